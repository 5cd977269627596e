"""Attention over the paged 8-bit cache where the softmax weights of a row are far
apart: one key holds most of the weight (a first token, or one in the middle), and a
long flat tail of keys the rest; or one page has a far larger scale than the others.
The outputs have to be within check_attn's bound of the float64 reference.

That bound counts 2^-8 of every weight. The keys that share a tile of 128 with the
large one are held less exactly, to 2^-3 of themselves at worst: 127 roundings of
weights that differ (their logits' sd is 0.5) average to less than 1 % of those
keys' sum, of which the tail holds at least 16 times as much."""
import functools

import numpy as np
import pytest

import cache_reference as ref
from dsa_test_util import dev, dev_bf16, host_bf16_as_f32, torch_mod
from test_gpu_cache import MARK, Setup, bf16, check_attn, dsa, run_attn  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

DC, DR = 512, 64
SCALE = float(np.float32((DC + DR) ** -0.5))


@functools.lru_cache(maxsize=1)
def tail(n, page):
    """Codes and scales of n rows of similar size, their rotary part 0."""
    rng = np.random.default_rng(n)
    pages = (n + page - 1) // page
    some = rng.standard_normal((1024, DC)) + 0.5  # values that do not average out
    x = np.zeros((pages * page, DC + DR))
    x[:, :DC] = some[rng.integers(0, len(some), len(x))]
    x = x.reshape(pages, page, DC + DR)
    s = np.array([ref.need_scale(v) for v in np.abs(x).max((1, 2))])
    return ref.encode(x / s[:, None, None]), s


class Long:
    """One stored sequence of n rows with a large key at `at`, and n_seq batch
    entries that all refer to it, each with `new` tokens."""

    def __init__(self, n, at, weight, seen, n_seq, new, heads, seed, page=64):
        rng = np.random.default_rng(seed)
        self.n, self.at, self.heads, self.page = n, at, heads, page
        pages = (n + page - 1) // page
        self.n_pages = pages + 2
        codes, s = (x.copy() for x in tail(n, page))
        # The large key's logit comes from its rotary part, against queries whose
        # rotary part is 1. Its value is a tenth of the others' size.
        z = np.log(weight / (1 - weight)) + np.log(seen) + 0.125
        j = at // page
        x = ref.VALUES[codes[j]] * s[j]
        x[at % page, :DC] *= 0.1
        x[at % page, DC:] = z / (DR * SCALE)
        s[j] = ref.need_scale(np.abs(x).max())
        codes[j] = ref.encode(x / s[j])
        order = rng.permutation(self.n_pages)[:pages]
        self.codes = np.full((self.n_pages, page, DC + DR), 0x7F, np.uint8)  # NaN elsewhere
        self.codes[order] = codes
        self.codes[order[-1], (n - 1) % page + 1:] = 0x7F
        self.scale = np.ones(self.n_pages, np.float32)
        self.scale[order] = s
        self.table = np.repeat(order[None].astype(np.int32), n_seq, 0)
        self.new, self.n_tok = new, n_seq * new
        q = rng.standard_normal((self.n_tok, heads, DC + DR)) * 0.48
        q[..., DC:] = 1.0
        self.q_bits, self.q = bf16(q)

    def run(self, dsa, window, n_sink, sample, weight=None):
        t = torch_mod()
        d = (dev(self.codes[..., :DC].copy()), dev(self.codes[..., DC:].copy()), dev(self.scale))
        c = dsa.make_cache(*d)
        n_seq = len(self.table)
        cu = np.arange(n_seq + 1, dtype=np.int32) * self.new
        b = dsa.make_batch(dev(self.table), dev(cu), dev(np.full(n_seq, self.n, np.int32)), self.n_tok)
        ws = t.empty(dsa.dsa_cache_workspace_size(c, b, self.heads), dtype=t.uint8, device="cuda")
        out = t.full((self.n_tok, self.heads, DC), MARK, dtype=t.bfloat16, device="cuda")
        lse = t.full((self.n_tok, self.heads), MARK, dtype=t.float32, device="cuda")
        dsa.check(dsa.dsa_cache_attn(c, b, dev_bf16(self.q_bits), self.heads, SCALE, window, n_sink,
                                     out, lse, ws))
        dsa.check(dsa.dsa_device_status(ws))
        got, got_lse = host_bf16_as_f32(out), lse.cpu().numpy()
        assert np.isfinite(got).all() and np.isfinite(got_lse).all()
        # the sampled tokens as sequences of their own
        tok = np.unique(np.linspace(0, self.n_tok - 1, sample).astype(int))
        lens = self.n - self.new + tok % self.new + 1
        r = ref.Cache(self.codes[..., :DC], self.codes[..., DC:], self.scale,
                      np.repeat(self.table[:1], len(tok), 0), np.arange(len(tok) + 1), lens)
        want = r.attend(self.q[tok], SCALE, window, n_sink)
        if weight is not None:  # the case is what it is meant to be
            row, _ = r.rows(0, np.array([self.at]))
            w = np.exp(SCALE * (self.q[tok] @ row[0]) - want[1])
            assert abs(w.mean() - weight) < 0.12, w.mean()
        check_attn(got[tok], got_lse[tok], want)


@pytest.mark.parametrize("at", ["first", "middle"])
@pytest.mark.parametrize("weight", [0.5, 0.8, 0.95])
@pytest.mark.parametrize("n,n_seq,new,heads", [
    (17408, 148, 1, 32),   # 32 rows an item, a sequence's tiles in one or two SMs
    (17408, 1, 300, 32),   # 64 rows
    (131071, 1, 3, 32),    # 64 rows, a sequence over all SMs
    (131071, 40, 1, 32),   # 32 rows, four SMs a sequence
    (4100, 5, 120, 16)])   # 64 rows, several tokens an item
def test_a_large_weight_and_a_long_tail(dsa, n, n_seq, new, heads, weight, at):  # noqa: F811
    pos = 0 if at == "first" else n // 2 + 5
    s = Long(n, pos, weight, n, n_seq, new, heads, seed=n + int(100 * weight))
    s.run(dsa, 0, 0, 2 if n > 20000 else 4, weight)


@pytest.mark.parametrize("weight", [0.5, 0.8, 0.95])
@pytest.mark.parametrize("n_seq,new", [(90, 1), (1, 500)])
def test_a_first_token_beside_a_window(dsa, n_seq, new, weight):  # noqa: F811
    s = Long(17408, 0, weight, 2064, n_seq, new, 32, seed=int(100 * weight))
    s.run(dsa, 2048, 16, 6, weight)


@pytest.mark.parametrize("grow", [4, 14, 20])
@pytest.mark.parametrize("n_seq,new", [(148, 1), (1, 300)])
def test_a_page_with_a_far_larger_scale(dsa, n_seq, new, grow):  # noqa: F811
    """One outlier element 2^grow above the rest in a page near the beginning: its
    tile's weights and those of the others are 2^grow apart in the products."""
    n = 8192
    s = Long(n, 4000, 0.01, n, n_seq, new, 32, seed=grow)
    p = s.table[0, 3]
    x = ref.VALUES[s.codes[p]] * s.scale[p]
    x[7, 100] = 2.0 ** grow
    s.scale[p] = ref.need_scale(np.abs(x).max())
    s.codes[p] = ref.encode(x / s.scale[p])
    s.q_bits[..., 100] = 0  # (it is in no logit)
    s.q[..., 100] = 0.0
    s.run(dsa, 0, 0, 6)


@pytest.mark.parametrize("n_seq,new", [(148, 1), (1, 300)])
def test_weights_that_fall_and_rise_again(dsa, n_seq, new):  # noqa: F811
    """Logits that fall by 50 (in powers of two) from tile to tile and come back: a
    row's reference follows, and stops 2^40 below its highest."""
    n = 6000
    s = Long(n, 0, 0.01, n, n_seq, new, 32, seed=9)
    pos = np.arange(n)
    fall = -50 * np.log(2) * np.abs(np.interp(pos, [0, 2500, 3000, 5990, n], [0, 1, 1, 0, 0]))
    for j, p in enumerate(s.table[0]):
        z = fall[j * 64:(j + 1) * 64]
        x = ref.VALUES[s.codes[p]] * s.scale[p]
        x[:len(z), DC:] = z[:, None] / (DR * SCALE)
        s.scale[p] = ref.need_scale(np.nanmax(np.abs(x)))
        with np.errstate(invalid="ignore"):
            codes = ref.encode(np.nan_to_num(x) / s.scale[p])
        s.codes[p, :len(z)] = codes[:len(z)]
    s.run(dsa, 0, 0, 6)


@pytest.mark.parametrize("scale", [0.08, 0.13, 0.3])
@pytest.mark.parametrize("lens,new", [([2900, 700] * 8, [1, 1] * 8), ([2500, 900], [60, 70])])
def test_logits_of_every_spread(dsa, lens, new, scale):  # noqa: F811
    """Standard deviations of 2, 3 and 7: the references move up and down all the time."""
    run_attn(dsa, Setup(lens, new, page=32, seed=int(100 * scale)), scale=scale)
