"""The paged 8-bit latent cache on a B200 against the float64 reference: append
with the rotation, gather, and attention (causal and windowed)."""
import numpy as np
import pytest

import cache_reference as ref
from dsa_test_util import dev, dev_bf16, host_bf16_as_f32, torch_mod

pytestmark = pytest.mark.gpu

DIMS = {512: 64, 64: 16}


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_prefill_dsa_b200 import build

    build.build()
    import sparse_attention_prefill_dsa_b200 as m

    m.library()
    return m


def bf16(x):
    """float values -> bf16 bits (nearest even) and their float64 values."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    bits = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return bits, (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Setup:
    """Random pool and batch. Rows of no sequence, and of pages of none, hold
    any bytes (NaN codes among them); unused page table entries are far out."""

    def __init__(self, lens, new, page=64, dc=512, heads=32, seed=0, pad=0, stride_pages=1,
                 spread=1.0, shared=False):
        rng = np.random.default_rng(seed)
        self.rng, self.dc, self.dr, self.page, self.heads = rng, dc, DIMS[dc], page, heads
        pages = [(n + page - 1) // page for n in lens]
        self.n_pages = sum(pages) + 2
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), max(max(pages), 1) + 1), 1 << 29, np.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        if shared:  # the first page of every sequence is one and the same
            self.table[:, 0] = self.table[0, 0]
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.lens = np.array(lens, np.int32)
        self.n_tok = int(self.cu[-1]) + pad
        w = dc + self.dr
        x = rng.standard_normal((self.n_pages, page, w)) * spread ** rng.integers(-2, 3, (self.n_pages, 1, 1))
        self.scale = np.array([ref.need_scale(np.abs(v).max()) for v in x], np.float32)
        codes = ref.encode(x / self.scale[:, None, None])
        junk = rng.integers(0, 256, codes.shape).astype(np.uint8)
        live = np.zeros((self.n_pages, page), bool)
        for b, n in enumerate(lens):
            pos = np.arange(n)
            live[self.table[b, pos // page], pos % page] = True
        codes = np.where(live[..., None], codes, junk)
        self.latent, self.rope = codes[..., :dc].copy(), codes[..., dc:].copy()
        t = torch_mod()
        self.stride_pages = stride_pages
        self.d_latent = t.zeros(self.n_pages, stride_pages, page, dc, dtype=t.uint8,
                                device="cuda")[:, stride_pages - 1]
        self.d_rope = t.zeros(self.n_pages, stride_pages, page, self.dr, dtype=t.uint8,
                              device="cuda")[:, stride_pages - 1]
        self.d_latent.copy_(dev(self.latent))
        self.d_rope.copy_(dev(self.rope))
        self.d_scale = dev(self.scale)
        self.d_table, self.d_cu, self.d_lens = dev(self.table), dev(self.cu), dev(self.lens)

    def structs(self, dsa):
        c = dsa.make_cache(self.d_latent, self.d_rope, self.d_scale)
        return c, dsa.make_batch(self.d_table, self.d_cu, self.d_lens, self.n_tok)

    def workspace(self, dsa, c, b):
        t = torch_mod()
        return t.full((dsa.dsa_cache_workspace_size(c, b, self.heads),), 0xA5, dtype=t.uint8,
                      device="cuda")

    def reference(self):
        return ref.Cache(self.latent, self.rope, self.scale, self.table, self.cu, self.lens)

    def inv_freq(self):
        i = np.arange(self.dr // 2)
        return (10000.0 ** (-2.0 * i / self.dr)).astype(np.float32)


# ---------------------------------------------------------------------- append

def run_append(dsa, s, style, heads=32, wide=False, with_q=True, spread=1.0):
    """One append through the library and the reference; compares everything."""
    t = torch_mod()
    rng = s.rng
    size = spread ** rng.integers(-3, 4, (s.n_tok, 1))
    lat_b, lat = bf16(rng.standard_normal((s.n_tok, s.dc)) * size)
    rope_b, rope = bf16(rng.standard_normal((s.n_tok, s.dr)) * 3 * size)
    qr_b, qr = bf16(rng.standard_normal((s.n_tok, heads, s.dr)))
    f = s.inv_freq()
    c, b = s.structs(dsa)
    ws = t.full((256,), 0xA5, dtype=t.uint8, device="cuda")
    d_lat, d_rope, d_qr = dev_bf16(lat_b), dev_bf16(rope_b), dev_bf16(qr_b)
    if wide:  # rows inside wider ones
        pad = lambda x, n: t.cat([x, t.full_like(x[..., :n], 7.0)], -1)[..., :x.shape[-1]]  # noqa: E731
        d_lat, d_rope, d_qr = pad(d_lat, 8), pad(d_rope, 16), pad(d_qr, 8)
    mark = -12.5
    q = t.full((s.n_tok, heads, s.dc + s.dr), mark, dtype=t.bfloat16, device="cuda")
    n_style = dsa.DSA_ROPE_HALVES if style else dsa.DSA_ROPE_INTERLEAVED
    r = s.reference()
    want_q = r.append(lat, rope, f, style, qr)
    for _ in range(2):  # a second call changes nothing
        dsa.check(dsa.dsa_cache_append(c, b, d_lat, d_rope, dev(f), n_style,
                                       d_qr if with_q else None, q if with_q else None, heads, ws))
        assert dsa.dsa_device_status(ws) == dsa.DSA_OK
        np.testing.assert_array_equal(s.d_scale.cpu().numpy(), r.scale.astype(np.float32))
        np.testing.assert_array_equal(s.d_latent.cpu().numpy(), r.latent)
        np.testing.assert_array_equal(s.d_rope.cpu().numpy(), r.rope)
        got = host_bf16_as_f32(q).astype(np.float64)
        assert (got[..., :s.dc] == mark).all()
        live = ~np.isnan(want_q) if with_q else np.zeros(want_q.shape, bool)
        got_r = got[..., s.dc:]
        assert (got_r[~live] == mark).all()
        # half a bf16 step of the value, and float32 cos, sin and two products
        # (each within 2^-24 of a term below |x| + |y| <= 2 max|q_rope|)
        tol = np.abs(want_q) * 2.0 ** -8 + 2 * np.abs(qr).max() * 4 * 2.0 ** -24
        assert (np.abs(got_r - want_q)[live] <= tol[live]).all()


@pytest.mark.parametrize("style", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dc", [512, 64])
def test_append_ragged(dsa, dc, page, style):
    s = Setup([1, 17, 64, 130, 300, 129, 5, 128], [1, 3, 64, 66, 1, 129, 0, 1], page=page, dc=dc, seed=page,
              pad=3)
    run_append(dsa, s, style, heads=3)


@pytest.mark.parametrize("heads", [1, 5, 32, 128])
def test_append_heads_and_strides(dsa, heads):
    s = Setup([40, 7], [9, 7], seed=heads, stride_pages=3)
    run_append(dsa, s, False, heads=heads, wide=True)


def test_append_without_queries(dsa):
    s = Setup([40, 700], [9, 650], page=32, seed=2)
    run_append(dsa, s, True, with_q=False)


def test_append_scales_that_grow_and_shrink(dsa):
    """Rows of very different size: some pages' earlier rows are re-expressed
    (some down to zero), others keep their scale."""
    s = Setup(list(range(20, 84)), [1 + i % 5 for i in range(64)], page=16, seed=3, spread=16.0)
    run_append(dsa, s, False, heads=2, spread=64.0)


def test_append_far_positions(dsa):
    """Angles of 10^5 radians: only the page of the new row has to exist."""
    n, page = 131071, 16
    s = Setup([n % page], [1], page=page, seed=4)
    j = n // page
    table = np.full((1, j + 1), -1, np.int32)
    table[0, j] = s.table[0, 0]
    s.table, s.lens = table, np.array([n], np.int32)
    s.d_table, s.d_lens = dev(s.table), dev(s.lens)
    run_append(dsa, s, True, heads=4)


def test_append_zero_rows_and_zero_values(dsa):
    s = Setup([64, 20], [64, 4], page=16, seed=5)
    t = torch_mod()
    c, b = s.structs(dsa)
    ws = t.empty(256, dtype=t.uint8, device="cuda")
    z = t.zeros(s.n_tok, s.dc, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_append(c, b, z, z[:, :64], dev(s.inv_freq()), 0, None, None, 1, ws))
    dsa.check(dsa.dsa_device_status(ws))
    r = s.reference()
    r.append(np.zeros((s.n_tok, s.dc)), np.zeros((s.n_tok, s.dr)), s.inv_freq(), False)
    np.testing.assert_array_equal(s.d_scale.cpu().numpy(), r.scale.astype(np.float32))
    np.testing.assert_array_equal(s.d_latent.cpu().numpy(), r.latent)


def test_append_reports_and_skips_what_is_wrong(dsa):
    s = Setup([70, 40, 33, 90], [5, 3, 4, 30], page=32, seed=6)
    s.lens[2] = 2           # fewer rows than new tokens
    s.table[0, 2] = -1      # the page of row 69 of sequence 0 (rows 65.. are new)
    s.table[3, 1] = s.n_pages  # outside the pool: rows 60..63 of sequence 3
    s.d_table, s.d_lens = dev(s.table), dev(s.lens)
    t = torch_mod()
    lat_b, lat = bf16(s.rng.standard_normal((s.n_tok, s.dc)))
    rope_b, rope = bf16(s.rng.standard_normal((s.n_tok, s.dr)))
    c, b = s.structs(dsa)
    ws = t.empty(256, dtype=t.uint8, device="cuda")
    dsa.check(dsa.dsa_cache_append(c, b, dev_bf16(lat_b), dev_bf16(rope_b), dev(s.inv_freq()), 0,
                                   None, None, 1, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_ERR_RANGE
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK  # reading it clears it
    r = s.reference()
    r.append(lat, rope, s.inv_freq(), False)
    np.testing.assert_array_equal(s.d_latent.cpu().numpy(), r.latent)
    np.testing.assert_array_equal(s.d_rope.cpu().numpy(), r.rope)
    # a sound call on the same workspace reports nothing
    s2 = Setup([70], [5], page=32, seed=7)
    c2, b2 = s2.structs(dsa)
    dsa.check(dsa.dsa_cache_append(c2, b2, dev_bf16(lat_b), dev_bf16(rope_b), dev(s.inv_freq()), 0,
                                   None, None, 1, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK


# ---------------------------------------------------------------------- gather

@pytest.mark.parametrize("page,dc,pos0,n", [(16, 512, 0, 1), (16, 64, 3, 200), (32, 512, 31, 2),
                                            (64, 512, 5, 330), (128, 512, 127, 208), (128, 64, 0, 335)])
def test_gather_is_exact(dsa, page, dc, pos0, n):
    t = torch_mod()
    s = Setup([20, 335], [1, 1], page=page, dc=dc, seed=page + n, stride_pages=2, spread=32.0)
    c, b = s.structs(dsa)
    ws = t.full((256,), 0xA5, dtype=t.uint8, device="cuda")
    lat = t.full((n + 1, dc), 3.0, dtype=t.bfloat16, device="cuda")
    rope = t.full((n + 1, s.dr), 3.0, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_gather(c, b, 1, pos0, n, lat, rope, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK
    want, _ = s.reference().rows(1, np.arange(pos0, pos0 + n))
    np.testing.assert_array_equal(host_bf16_as_f32(lat)[:n], want[:, :dc])
    np.testing.assert_array_equal(host_bf16_as_f32(rope)[:n], want[:, dc:])
    assert (host_bf16_as_f32(lat)[n] == 3.0).all() and (host_bf16_as_f32(rope)[n] == 3.0).all()


def test_gather_reports_rows_that_are_not_there(dsa):
    t = torch_mod()
    s = Setup([100], [1], page=32, seed=8)
    s.table[0, 1] = -7
    s.d_table = dev(s.table)
    c, b = s.structs(dsa)
    ws = t.empty(256, dtype=t.uint8, device="cuda")
    lat = t.full((110, s.dc), 3.0, dtype=t.bfloat16, device="cuda")
    rope = t.full((110, s.dr), 3.0, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_gather(c, b, 0, 0, 64, lat, rope, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_ERR_RANGE
    want, _ = s.reference().rows(0, np.arange(32))
    got = host_bf16_as_f32(lat)
    np.testing.assert_array_equal(got[:32], want[:, :512])
    assert (got[32:] == 3.0).all()
    dsa.check(dsa.dsa_cache_gather(c, b, 0, 96, 10, lat, rope, ws))  # six rows too many
    assert dsa.dsa_device_status(ws) == dsa.DSA_ERR_RANGE
    assert (host_bf16_as_f32(lat)[4:32] == want[4:, :512]).all()
    dsa.check(dsa.dsa_cache_gather(c, b, 0, 0, 0, lat, rope, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK


# ------------------------------------------------------------------- attention

MARK = -77.0


def queries(s, spread=1.0):
    """bf16 queries; with spread > 1 the rows are of different size."""
    size = spread ** s.rng.integers(-2, 3, (s.n_tok, s.heads, 1))
    return bf16(s.rng.standard_normal((s.n_tok, s.heads, s.dc + s.dr)) * size)


def check_attn(got_out, got_lse, want):
    """Tolerances, all derived: the output's own rounding (half a bf16 step of
    the value, 2^-8); the weights p carry at least 8 significant bits (2^-8 of
    sum p|v| / sum p), plus 2^-12 of it for float32 sums, exp2 and weights that
    are too small for that; the logits are sums of 576 products in float32:
    600 * 2^-24 of sum |q_c k_c|, which shifts lse by as much and p by that
    factor."""
    out, lse, mag, zabs = want
    live = ~np.isnan(lse)
    dz = 600 * 2.0 ** -24 * zabs
    np.testing.assert_array_equal(got_out[~live], MARK)
    tol = (np.abs(out) * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -12 + 2 * dz[..., None]))[live]
    bad = np.abs(got_out[live] - out[live]) > tol
    assert not bad.any(), (bad.sum(), np.abs(got_out[live] - out[live]).max())
    if got_lse is not None:
        np.testing.assert_array_equal(got_lse[~live], np.float32(MARK))
        g, w = got_lse[live], lse[live]
        np.testing.assert_array_equal(np.isinf(g), np.isinf(w))
        f = np.isfinite(w)
        err = np.abs(g[f] - w[f])
        assert (err <= dz[live][f] + 2.0 ** -20 + np.abs(w[f]) * 2.0 ** -22).all(), err.max()


def run_attn(dsa, s, window=0, n_sink=0, want_lse=True, spread=1.0, scale=None, want_status=None):
    t = torch_mod()
    q_b, q = queries(s, spread)
    c, b = s.structs(dsa)
    ws = s.workspace(dsa, c, b)
    scale = float(np.float32(scale or (s.dc + s.dr) ** -0.5))
    out = t.full((s.n_tok, s.heads, s.dc), MARK, dtype=t.bfloat16, device="cuda")
    lse = t.full((s.n_tok, s.heads), MARK, dtype=t.float32, device="cuda") if want_lse else None
    d_q = dev_bf16(q_b)
    dsa.check(dsa.dsa_cache_attn(c, b, d_q, s.heads, scale, window, n_sink, out, lse, ws))
    assert dsa.dsa_device_status(ws) == (dsa.DSA_OK if want_status is None else want_status)
    got, got_lse = host_bf16_as_f32(out), lse.cpu().numpy() if want_lse else None
    want = s.reference().attend(q, scale, window, n_sink)
    check_attn(got, got_lse, want)
    # the same call gives the same bits
    out2 = t.full_like(out, MARK)
    dsa.check(dsa.dsa_cache_attn(c, b, d_q, s.heads, scale, window, n_sink, out2, None, ws))
    assert t.equal(out.view(t.int16), out2.view(t.int16))
    return got, want


LENS = [1, 2, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("dc,heads", [(512, 32), (64, 4)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attn_decode(dsa, dc, heads, page):
    run_attn(dsa, Setup(LENS, [1] * len(LENS), page=page, dc=dc, heads=heads, seed=page, pad=2))


@pytest.mark.parametrize("heads", [1, 3, 8, 16, 31, 33, 64, 128])
def test_attn_heads(dsa, heads):
    run_attn(dsa, Setup([5, 260, 129], [1, 1, 2], heads=heads, seed=heads))


@pytest.mark.parametrize("dc,heads", [(512, 32), (512, 5), (64, 4)])
def test_attn_chunks(dsa, dc, heads):
    """Prefill chunks: from nothing, from inside a page, zero tokens, one token."""
    run_attn(dsa, Setup([40, 300, 9, 131, 65], [40, 70, 0, 3, 1], page=32, dc=dc, heads=heads, seed=heads,
                        pad=5))


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (5, 4), (64, 0), (128, 16), (129, 130),
                                           (200, 1), (5000, 3)])
@pytest.mark.parametrize("dc,heads", [(512, 32), (64, 4)])
def test_attn_window(dsa, dc, heads, window, n_sink):
    run_attn(dsa, Setup([1, 4, 130, 517, 640], [1, 1, 2, 1, 33], page=16, dc=dc, heads=heads,
                        seed=window), window, n_sink)


@pytest.mark.parametrize("heads", [4, 32])
def test_attn_pages_outside_the_window_are_not_read(dsa, heads):
    """Their page table entries are garbage, and rows of the window's pages
    that no token sees hold NaN codes."""
    s = Setup([700, 390], [1, 2], page=16, heads=heads, seed=11)
    window, n_sink = 100, 5
    for b, (n, m) in enumerate(zip(s.lens, np.diff(s.cu))):
        lo = n - m - window + 1
        for j in range(n_sink // 16 + 1, lo // 16):
            s.table[b, j] = -1 if j % 2 else 1 << 30
        for pos in list(range(n_sink, 16)) + list(range(lo // 16 * 16, lo)):
            p = s.table[b, pos // 16]
            s.latent[p, pos % 16], s.rope[p, pos % 16] = 0x7F, 0xFF
    s.d_latent.copy_(dev(s.latent))
    s.d_rope.copy_(dev(s.rope))
    s.d_table = dev(s.table)
    run_attn(dsa, s, window, n_sink)


@pytest.mark.parametrize("spread", [4.0, 64.0])
def test_attn_pages_and_queries_of_different_size(dsa, spread):
    """Scales that differ from page to page, rows of q that differ by far."""
    run_attn(dsa, Setup([900, 333], [1, 3], page=16, seed=12, spread=spread), scale=0.02)
    run_attn(dsa, Setup([900, 333], [1, 3], page=64, seed=13), spread=spread, scale=0.01)


def test_attn_sharp_logits_that_keep_growing(dsa):
    """A key's weight exceeds all earlier ones by far, again and again."""
    s = Setup([1500], [2], seed=14)
    grow = np.linspace(0.02, 4.0, 1500)
    x = s.rng.standard_normal((1500, s.dc + s.dr)) * grow[:, None]
    for j in range(0, 1500, 64):
        p = s.table[0, j // 64]
        v = x[j:j + 64]
        s.scale[p] = ref.need_scale(np.abs(v).max())
        codes = ref.encode(v / s.scale[p])
        s.latent[p, :len(v)], s.rope[p, :len(v)] = codes[:, :s.dc], codes[:, s.dc:]
    s.d_latent.copy_(dev(s.latent))
    s.d_rope.copy_(dev(s.rope))
    s.d_scale = dev(s.scale)
    run_attn(dsa, s, scale=0.3)


def test_attn_one_weight_far_above_the_rest(dsa):
    """One key holds almost all of one row's weight, and it comes first: later
    tiles add next to nothing."""
    s = Setup([2000], [1], seed=15)
    p = s.table[0, 0]
    s.latent[p, 3] = ref.encode(np.full(s.dc, 6.0) / s.scale[p])
    s.d_latent.copy_(dev(s.latent))
    t = torch_mod()
    q_b, q = bf16(np.full((1, s.heads, s.dc + s.dr), 0.5))
    c, b = s.structs(dsa)
    ws = s.workspace(dsa, c, b)
    out = t.full((1, s.heads, s.dc), MARK, dtype=t.bfloat16, device="cuda")
    lse = t.full((1, s.heads), MARK, dtype=t.float32, device="cuda")
    dsa.check(dsa.dsa_cache_attn(c, b, dev_bf16(q_b), s.heads, 0.04, 0, 0, out, lse, ws))
    dsa.check(dsa.dsa_device_status(ws))
    want = s.reference().attend(q, float(np.float32(0.04)), 0, 0)
    check_attn(host_bf16_as_f32(out), lse.cpu().numpy(), want)


def test_attn_long_context_over_many_sms(dsa):
    """20,000 rows for one token (split over SMs) beside sequences of one row."""
    run_attn(dsa, Setup([1, 20000, 1], [1, 1, 1], page=128, heads=32, seed=16))
    run_attn(dsa, Setup([9000], [3], page=64, heads=16, seed=17), window=6000, n_sink=300)


@pytest.mark.parametrize("window,n_sink", [(0, 0), (200, 4)])
@pytest.mark.parametrize("lens,new,heads", [([700, 1300], [300, 40], 32), ([520] * 90, [1] * 90, 32),
                                            ([900, 40, 1500], [128, 40, 3], 128)])
def test_attn_sms_that_take_several_sequences(dsa, lens, new, heads, window, n_sink):
    """More tiles than SMs: an SM goes through parts of several items, each of
    several tiles, with whole items between the parts that cross SMs."""
    run_attn(dsa, Setup(lens, new, heads=heads, page=32, seed=26), window, n_sink)


def test_attn_shared_prefix_page(dsa):
    run_attn(dsa, Setup([200, 90, 300], [2, 1, 1], seed=18, shared=True))


def test_attn_strided_pool_and_no_lse(dsa):
    run_attn(dsa, Setup([200, 90], [2, 1], seed=19, stride_pages=3), want_lse=False)


@pytest.mark.parametrize("dc,heads", [(512, 32), (64, 4)])
def test_attn_reports_and_skips_what_is_wrong(dsa, dc, heads):
    s = Setup([70, 40, 300, 5], [1, 1, 2, 1], page=32, dc=dc, heads=heads, seed=20)
    s.lens[1] = 0           # a token, and no row for it
    s.table[2, 3] = -1      # rows 96..127 of sequence 2 are not seen
    s.table[3, 0] = s.n_pages  # sequence 3 sees nothing: out = 0, lse = -inf
    s.d_table, s.d_lens = dev(s.table), dev(s.lens)
    got, want = run_attn(dsa, s, want_status=dsa.DSA_ERR_RANGE)
    assert (got[4] == 0).all() and np.isneginf(want[1][4]).all()


def test_attn_wrong_cu_seqlens_is_reported(dsa):
    t = torch_mod()
    s = Setup([70, 40], [1, 1], seed=21)
    c, b = s.structs(dsa)
    q_b, _ = queries(s)
    out = t.full((s.n_tok, s.heads, s.dc), MARK, dtype=t.bfloat16, device="cuda")
    for cu in ([0, -5, 2], [0, 7, 9], [3, 1, 2], [-1, 1 << 30, -(1 << 30)]):
        s.d_cu.copy_(dev(np.array(cu, np.int32)))
        ws = s.workspace(dsa, c, b)
        dsa.check(dsa.dsa_cache_attn(c, b, dev_bf16(q_b), s.heads, 0.04, 0, 0, out, None, ws))
        assert dsa.dsa_device_status(ws) == dsa.DSA_ERR_RANGE
        x = t.zeros(s.n_tok, 512, dtype=t.bfloat16, device="cuda")
        dsa.check(dsa.dsa_cache_append(c, b, x, x, dev(s.inv_freq()), 0, None, None, 1, ws))
        assert dsa.dsa_device_status(ws) == dsa.DSA_ERR_RANGE


def test_nothing_to_do(dsa):
    t = torch_mod()
    s = Setup([70, 40], [1, 1], seed=22)
    c, _ = s.structs(dsa)
    empty = dsa.make_batch(s.d_table, s.d_cu, s.d_lens, 0)
    ws = s.workspace(dsa, c, empty)
    x = t.zeros(16, 576, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_attn(c, empty, x, 32, 0.04, 0, 0, x, None, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK
    dsa.check(dsa.dsa_cache_append(c, empty, x, x, dev(s.inv_freq()), 0, None, None, 1, ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK
    assert float(x.abs().max()) == 0.0


def test_sequences_without_new_tokens_and_many_of_them(dsa):
    """Nothing but sequences without tokens; then 1,500 sequences, most of them
    so (more than a block has threads), in both calls."""
    s = Setup([70, 40], [0, 0], seed=27, pad=3)
    run_attn(dsa, s)
    run_append(dsa, s, False, heads=2, with_q=False)
    rng = np.random.default_rng(28)
    lens = rng.integers(1, 40, 1500).tolist()
    new = [int(rng.random() < 0.05) for _ in lens]
    s = Setup(lens, new, page=16, seed=28)
    run_attn(dsa, s)
    run_append(dsa, s, True, heads=3)


# --------------------------------------------------------------- used together

def test_append_then_attend_then_gather_into_the_sparse_layer(dsa):
    """Three steps of two sequences (a prefill chunk, then single tokens), and the
    gathered rows given to the sparse attention with every key selected: both
    attentions see the same values."""
    t = torch_mod()
    page, heads = 64, 32
    s = Setup([200, 75], [200, 75], page=page, heads=heads, seed=23)
    r = s.reference()
    f = s.inv_freq()
    scale = float(np.float32(576 ** -0.5))
    for new in ([190, 70], [1, 1], [1, 1]):
        s.lens = np.array([190, 70], np.int32) if new[0] > 1 else s.lens + 1
        s.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s.d_lens, s.d_cu = dev(s.lens), dev(s.cu)
        s.n_tok = int(s.cu[-1])
        r.lens, r.cu = s.lens, s.cu
        c, b = s.structs(dsa)
        ws = s.workspace(dsa, c, b)
        lat_b, lat = bf16(s.rng.standard_normal((s.n_tok, 512)))
        rope_b, rope = bf16(s.rng.standard_normal((s.n_tok, 64)))
        q_b, _ = bf16(s.rng.standard_normal((s.n_tok, heads, 576)))
        q = dev_bf16(q_b)
        q_rope = q[..., 512:].clone()
        dsa.check(dsa.dsa_cache_append(c, b, dev_bf16(lat_b), dev_bf16(rope_b), dev(f), 0, q_rope, q,
                                       heads, ws))
        out = t.empty(s.n_tok, heads, 512, dtype=t.bfloat16, device="cuda")
        lse = t.empty(s.n_tok, heads, dtype=t.float32, device="cuda")
        dsa.check(dsa.dsa_cache_attn(c, b, q, heads, scale, 0, 0, out, lse, ws))
        dsa.check(dsa.dsa_device_status(ws))
        r.append(lat, rope, f, False)
        np.testing.assert_array_equal(s.d_latent.cpu().numpy(), r.latent)
        want = r.attend(host_bf16_as_f32(q).astype(np.float64), scale, 0, 0)
        check_attn(host_bf16_as_f32(out), lse.cpu().numpy(), want)
    n = int(s.lens[0])
    g_lat = t.empty(n, 512, dtype=t.bfloat16, device="cuda")
    g_rope = t.empty(n, 64, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_gather(c, b, 0, 0, n, g_lat, g_rope, ws))
    import workloads

    d = workloads.make_dims(1, n - 1, n, heads, 512, 64, 32, 128, 256)
    idx = np.full((1, 256), -1, np.int32)
    idx[0, :n] = np.arange(n)
    out2 = t.empty(1, heads, 512, dtype=t.bfloat16, device="cuda")
    lse2 = t.empty(1, heads, dtype=t.float32, device="cuda")
    ws2 = t.empty(dsa.dsa_workspace_size(d, dsa.DSA_WS_ATTN), dtype=t.uint8, device="cuda")
    dsa.check(dsa.dsa_sparse_attn_prefill(d, q[:1], g_lat, g_rope, dev(idx), out2, lse2, ws2))
    dsa.check(dsa.dsa_device_status(ws2))
    # each is within its bound of the same exact value: the sum of the two
    # (bf16 weights and output of the sparse attention: 2^-8 of each)
    got = host_bf16_as_f32(out2).astype(np.float64)
    tol = 2 * (np.abs(want[0][:1]) * 2.0 ** -8 + want[2][:1] * (2.0 ** -8 + 2.0 ** -11))
    assert (np.abs(got - host_bf16_as_f32(out)[:1]) <= tol).all()
    assert np.abs(lse2.cpu().numpy() - lse.cpu().numpy()[:1]).max() < 2e-3


def test_captured_steps_replay_with_new_lengths(dsa):
    """Append and attention in one CUDA graph; the batch arrays change between
    replays, and a second graph with a workspace of its own runs beside it."""
    t = torch_mod()
    s = Setup([100, 300], [1, 1], seed=24)
    s.lens = np.array([50, 200], np.int32)
    r = s.reference()
    c, b = s.structs(dsa)
    f = dev(s.inv_freq())
    lat, rope = (t.zeros(2, n, dtype=t.bfloat16, device="cuda") for n in (512, 64))
    q = t.zeros(2, 32, 576, dtype=t.bfloat16, device="cuda")
    runs = []
    for k in range(2):
        ws = s.workspace(dsa, c, b)
        out = t.empty(2, 32, 512, dtype=t.bfloat16, device="cuda")
        lse = t.empty(2, 32, dtype=t.float32, device="cuda")
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            if k == 0:
                dsa.check(dsa.dsa_cache_append(c, b, lat, rope, f, 0, None, None, 1, ws))
            dsa.check(dsa.dsa_cache_attn(c, b, q, 32, 0.04, 150 * k, 4 * k, out, lse, ws))
        runs.append((g, ws, out, lse))
    for step in range(3):
        s.lens = s.lens + 1
        r.lens = s.lens
        s.d_lens.copy_(dev(s.lens))
        lat_b, lat_h = bf16(s.rng.standard_normal((2, 512)))
        rope_b, rope_h = bf16(s.rng.standard_normal((2, 64)))
        q_b, q_h = bf16(s.rng.standard_normal((2, 32, 576)))
        lat.copy_(dev_bf16(lat_b))
        rope.copy_(dev_bf16(rope_b))
        q.copy_(dev_bf16(q_b))
        r.append(lat_h, rope_h, s.inv_freq(), False)
        t.cuda.synchronize()
        runs[0][0].replay()
        t.cuda.synchronize()
        other = t.cuda.Stream()
        with t.cuda.stream(other):
            runs[1][0].replay()
        runs[0][0].replay()
        t.cuda.synchronize()
        for k, (_, ws, out, lse) in enumerate(runs):
            assert dsa.dsa_device_status(ws) == dsa.DSA_OK
            want = r.attend(q_h, float(np.float32(0.04)), 150 * k, 4 * k)
            check_attn(host_bf16_as_f32(out), lse.cpu().numpy(), want)


def test_two_streams_with_their_own_workspaces(dsa):
    t = torch_mod()
    s = Setup([3000, 50], [1, 2], seed=25)
    q_b, q = queries(s)
    c, b = s.structs(dsa)
    d_q = dev_bf16(q_b)
    got = []
    t.cuda.synchronize()
    for k in range(4):
        st = t.cuda.Stream()
        with t.cuda.stream(st):
            ws = s.workspace(dsa, c, b)
            out = t.full((s.n_tok, s.heads, s.dc), MARK, dtype=t.bfloat16, device="cuda")
            dsa.check(dsa.dsa_cache_attn(c, b, d_q, s.heads, 0.04, 0, 0, out, None, ws))
        got.append((st, ws, out))
    t.cuda.synchronize()
    want = s.reference().attend(q, float(np.float32(0.04)), 0, 0)
    for st, ws, out in got:
        assert dsa.dsa_device_status(ws, st) == dsa.DSA_OK
        check_attn(host_bf16_as_f32(out), None, want)
