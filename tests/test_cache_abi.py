"""The paged 8-bit latent cache on the CPU: struct layouts, workspace sizes and
the refusals that come before any device is touched; and pins of the float64
reference that the GPU tests compare with. No test here launches a kernel."""
import ctypes
import os
import re

import numpy as np
import pytest

import cache_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dsa.h")
FAKE = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_prefill_dsa_b200 import build

    build.build()
    import sparse_attention_prefill_dsa_b200 as m

    m.library()
    return m


def cache_of(dsa, **over):
    a = dict(latent=FAKE, rope=FAKE, scale=FAKE, latent_page_stride=64 * 512,
             rope_page_stride=64 * 64, n_pages=10, page_size=64, d_latent=512, d_rope=64)
    a.update(over)
    return dsa.dsa_cache(*[a[f] for f, _ in dsa.dsa_cache._fields_])


def batch_of(dsa, **over):
    a = dict(page_table=FAKE, cu_seqlens=FAKE, seq_lens=FAKE, n_seq=2, max_pages=4, n_tok=5,
             reserved=0)
    a.update(over)
    return dsa.dsa_batch(*[a[f] for f, _ in dsa.dsa_batch._fields_])


def append(dsa, c, b, **over):
    a = dict(latent=FAKE, rope=FAKE, inv_freq=FAKE, rope_style=0, q_rope=FAKE, q=FAKE, n_heads=32,
             workspace=FAKE, workspace_bytes=1 << 30, stream=0)
    a.update(over)
    return dsa.dsa_cache_append(c, b, **a)


def gather(dsa, c, b, **over):
    a = dict(seq=0, pos0=0, n_rows=1, latent=FAKE, rope=FAKE, workspace=FAKE,
             workspace_bytes=1 << 30, stream=0)
    a.update(over)
    return dsa.dsa_cache_gather(c, b, **a)


def attn(dsa, c, b, **over):
    a = dict(q=FAKE, n_heads=32, softmax_scale=0.04, window=0, n_sink=0, out=FAKE, lse=None,
             workspace=FAKE, workspace_bytes=1 << 30, stream=0)
    a.update(over)
    return dsa.dsa_cache_attn(c, b, **a)


@pytest.mark.parametrize("name", ["dsa_cache", "dsa_batch"])
def test_struct_layout_matches_header(dsa, name):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = text[text.index("typedef struct %s {" % name):text.index("} %s;" % name)]
    fields = re.findall(r"([a-z_0-9]+);", body)
    struct = getattr(dsa, name)
    assert fields == [f for f, _ in struct._fields_]
    assert ctypes.sizeof(struct) == (56 if name == "dsa_cache" else 40)


@pytest.mark.parametrize("call", [append, gather, attn])
def test_refusals_of_cache_and_batch(dsa, call):
    c, b = cache_of(dsa), batch_of(dsa)
    for over, want in (
            (dict(latent=None), dsa.DSA_ERR_NULL), (dict(rope=None), dsa.DSA_ERR_NULL),
            (dict(scale=None), dsa.DSA_ERR_NULL), (dict(latent=FAKE + 8), dsa.DSA_ERR_ALIGN),
            (dict(rope=FAKE + 4), dsa.DSA_ERR_ALIGN), (dict(scale=FAKE + 4), dsa.DSA_ERR_ALIGN),
            (dict(page_size=48), dsa.DSA_ERR_DIMS), (dict(page_size=256), dsa.DSA_ERR_DIMS),
            (dict(page_size=0), dsa.DSA_ERR_DIMS), (dict(d_latent=256), dsa.DSA_ERR_DIMS),
            (dict(d_rope=16), dsa.DSA_ERR_DIMS), (dict(n_pages=0), dsa.DSA_ERR_DIMS),
            (dict(latent_page_stride=64 * 512 - 16), dsa.DSA_ERR_DIMS),
            (dict(rope_page_stride=64 * 64 - 16), dsa.DSA_ERR_DIMS),
            (dict(latent_page_stride=64 * 512 + 8), dsa.DSA_ERR_ALIGN),
            (dict(latent_page_stride=(1 << 39) + 16), dsa.DSA_ERR_DIMS)):
        assert call(dsa, cache_of(dsa, **over), b) == want, over
    for over, want in (
            (dict(page_table=None), dsa.DSA_ERR_NULL), (dict(cu_seqlens=None), dsa.DSA_ERR_NULL),
            (dict(seq_lens=None), dsa.DSA_ERR_NULL), (dict(seq_lens=FAKE + 4), dsa.DSA_ERR_ALIGN),
            (dict(n_seq=-1), dsa.DSA_ERR_DIMS), (dict(max_pages=0), dsa.DSA_ERR_DIMS),
            (dict(max_pages=(1 << 24) + 1), dsa.DSA_ERR_DIMS), (dict(n_tok=-1), dsa.DSA_ERR_DIMS),
            (dict(n_tok=1 << 24), dsa.DSA_ERR_DIMS), (dict(reserved=1), dsa.DSA_ERR_DIMS)):
        assert call(dsa, c, batch_of(dsa, **over)) == want, over
    assert call(dsa, c, b, workspace=None) == dsa.DSA_ERR_WORKSPACE
    assert call(dsa, c, b, workspace=FAKE + 8) == dsa.DSA_ERR_ALIGN
    assert call(dsa, c, b, workspace_bytes=255) == dsa.DSA_ERR_WORKSPACE


def test_refusals_of_append(dsa):
    c, b = cache_of(dsa), batch_of(dsa)
    for over, want in (
            (dict(latent=None), dsa.DSA_ERR_NULL), (dict(rope=None), dsa.DSA_ERR_NULL),
            (dict(inv_freq=None), dsa.DSA_ERR_NULL), (dict(q=None), dsa.DSA_ERR_NULL),
            (dict(q_rope=None), dsa.DSA_ERR_NULL), (dict(rope_style=2), dsa.DSA_ERR_DIMS),
            (dict(n_heads=0), dsa.DSA_ERR_DIMS), (dict(n_heads=129), dsa.DSA_ERR_DIMS),
            (dict(latent=FAKE + 2), dsa.DSA_ERR_ALIGN), (dict(q=FAKE + 8), dsa.DSA_ERR_ALIGN),
            (dict(ld_latent=504), dsa.DSA_ERR_DIMS), (dict(ld_latent=516), dsa.DSA_ERR_ALIGN),
            (dict(ld_rope=56), dsa.DSA_ERR_DIMS), (dict(ld_rope=68), dsa.DSA_ERR_ALIGN),
            (dict(ld_q_tok=-8), dsa.DSA_ERR_DIMS), (dict(ld_q_head=68), dsa.DSA_ERR_ALIGN)):
        assert append(dsa, c, b, **over) == want, over


def test_refusals_of_gather(dsa):
    c, b = cache_of(dsa), batch_of(dsa)
    for over, want in (
            (dict(latent=None), dsa.DSA_ERR_NULL), (dict(rope=FAKE + 2), dsa.DSA_ERR_ALIGN),
            (dict(seq=-1), dsa.DSA_ERR_DIMS), (dict(seq=2), dsa.DSA_ERR_DIMS),
            (dict(pos0=-1), dsa.DSA_ERR_DIMS), (dict(n_rows=-1), dsa.DSA_ERR_DIMS),
            (dict(pos0=256, n_rows=1), dsa.DSA_ERR_DIMS)):
        assert gather(dsa, c, b, **over) == want, over


def test_refusals_of_attention(dsa):
    c, b = cache_of(dsa), batch_of(dsa)
    for over, want in (
            (dict(q=None), dsa.DSA_ERR_NULL), (dict(out=None), dsa.DSA_ERR_NULL),
            (dict(q=FAKE + 8), dsa.DSA_ERR_ALIGN), (dict(lse=FAKE + 4), dsa.DSA_ERR_ALIGN),
            (dict(n_heads=0), dsa.DSA_ERR_DIMS), (dict(n_heads=129), dsa.DSA_ERR_DIMS),
            (dict(window=-1), dsa.DSA_ERR_DIMS), (dict(n_sink=-1), dsa.DSA_ERR_DIMS),
            (dict(softmax_scale=0.0), dsa.DSA_ERR_DIMS),
            (dict(softmax_scale=float("nan")), dsa.DSA_ERR_DIMS)):
        assert attn(dsa, c, b, **over) == want, over
    need = dsa.dsa_cache_workspace_size(c, b, 32)
    assert attn(dsa, c, b, workspace_bytes=need - 1) == dsa.DSA_ERR_WORKSPACE


def test_workspace_size(dsa):
    c, b = cache_of(dsa), batch_of(dsa)
    assert dsa.dsa_cache_workspace_size(c, b, 32) >= 256
    assert dsa.dsa_cache_workspace_size(c, b, 0) == 0
    assert dsa.dsa_cache_workspace_size(cache_of(dsa, page_size=8), b, 32) == 0
    # sizes only: no pointer is looked at
    assert dsa.dsa_cache_workspace_size(cache_of(dsa, latent=None), batch_of(dsa, seq_lens=None),
                                        32) == dsa.dsa_cache_workspace_size(c, b, 32)


def test_valid_calls_without_gpu_report_a_device_error(dsa):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    c, b = cache_of(dsa), batch_of(dsa)
    for call in (append, gather, attn):
        assert call(dsa, c, b) in (dsa.DSA_ERR_CUDA, dsa.DSA_ERR_DEVICE)


def test_descriptor_helpers_check_their_tensors(dsa):
    import torch

    lat, rope = torch.zeros(3, 16, 512, dtype=torch.uint8), torch.zeros(3, 16, 64, dtype=torch.uint8)
    c = dsa.make_cache(lat, rope, torch.ones(3))
    assert (c.n_pages, c.page_size, c.d_latent, c.d_rope) == (3, 16, 512, 64)
    assert (c.latent_page_stride, c.rope_page_stride) == (16 * 512, 16 * 64)
    wide = torch.zeros(3, 2, 16, 512, dtype=torch.uint8)[:, 1]  # a pool of two layers
    assert dsa.make_cache(wide, rope, torch.ones(3)).latent_page_stride == 2 * 16 * 512
    for bad in ((lat.float(), rope, torch.ones(3)), (lat[:2], rope, torch.ones(3)),
                (lat, rope, torch.ones(2)), (lat, rope, torch.ones(3).double()),
                (lat[..., ::2], rope, torch.ones(3))):
        with pytest.raises(ValueError):
            dsa.make_cache(*bad)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    b = dsa.make_batch(i(2, 7), i(3), i(2), 9)
    assert (b.n_seq, b.max_pages, b.n_tok, b.reserved) == (2, 7, 9, 0)
    for bad in ((i(3, 7), i(3), i(2), 9), (i(2, 7), i(2), i(2), 9), (i(2, 7).long(), i(3), i(2), 9),
                (i(7, 2).t(), i(3), i(2), 9)):
        with pytest.raises(ValueError):
            dsa.make_batch(*bad)


def test_reference_codes_are_e4m3():
    import torch

    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.VALUES, want)
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * s
                        for s in (1e-3, 0.02, 1.0, 100.0)]).clip(-448, 448)
    mid = (ref.VALUES[:126] + ref.VALUES[1:127]) / 2  # ties
    x = np.concatenate([x, mid, -mid, [0.0, -0.0, 448.0, -448.0]])
    got = torch.from_numpy(x).float().double().numpy()
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.encode(got), want)


def test_reference_append_by_hand():
    """Two pages of two rows, d_rope = 2 at angle t * pi / 2: a quarter turn a token."""
    c = ref.Cache(np.zeros((3, 2, 2), np.uint8), np.zeros((3, 2, 2), np.uint8), np.ones(3),
                  np.array([[2, 0]]), np.array([0, 3]), np.array([3]))
    lat = np.array([[1.0, 2.0], [448.0, 0.0], [449.0, 0.5]])
    c.append(lat, np.array([[1.0, 0.0]] * 3), np.array([np.pi / 2]), False)
    assert c.scale[2] == 1.0 and c.scale[0] == 2.0 and c.scale[1] == 1.0
    val = ref.VALUES
    np.testing.assert_array_equal(val[c.latent[2]] * 1.0, lat[:2])
    np.testing.assert_array_equal(val[c.latent[0, 0]] * 2.0, [448.0, 0.5])
    np.testing.assert_array_equal(val[c.rope[2]], [[1.0, 0.0], [0.0, 1.0]])
    np.testing.assert_array_equal(val[c.rope[0, 0]] * 2.0, [-1.0, 0.0])
    # one more row that needs a larger scale: row 0 of its page is re-expressed
    c.cu, c.lens = np.array([0, 1]), np.array([4])
    c.append(np.array([[448.0 * 8, 0.0]]), np.array([[0.0, 0.0]]), np.array([np.pi / 2]), False)
    assert c.scale[0] == 8.0
    np.testing.assert_array_equal(val[c.latent[0, 0]] * 8.0, [448.0, 0.5])
