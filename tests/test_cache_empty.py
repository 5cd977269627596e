"""Batches and ranges with nothing in them, as torch's empty tensors (address 0) make
them: accepted by the three calls of the paged cache, with a cleared status."""
import pytest

FAKE = 1 << 20  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def dsa():
    from sparse_attention_prefill_dsa_b200 import build

    build.build()
    import sparse_attention_prefill_dsa_b200 as m

    m.library()
    return m


def calls(dsa, c, b, ws, x, none):
    """Each call with empty token tensors where `none` says so, else with x."""
    e = None if none else x
    yield dsa.dsa_cache_append(c, b, e, e, x, 0, e, e, 32, ws, 1 << 30, 0, ld_latent=512, ld_rope=64,
                               ld_q_tok=2048, ld_q_head=64)
    yield dsa.dsa_cache_append(c, b, e, e, x, 0, e, x, 32, ws, 1 << 30, 0, ld_latent=512, ld_rope=64,
                               ld_q_tok=2048, ld_q_head=64)
    yield dsa.dsa_cache_attn(c, b, e, 32, 0.04, 0, 0, e, None, ws, 1 << 30, 0)


def test_nothing_is_not_a_null_pointer(dsa):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    passed = (dsa.DSA_ERR_CUDA, dsa.DSA_ERR_DEVICE)  # every argument check
    c = dsa.dsa_cache(FAKE, FAKE, FAKE, 64 * 512, 64 * 64, 10, 64, 512, 64)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    empty = dsa.make_batch(i(0, 4), i(1), i(0), 0)
    empty.cu_seqlens = FAKE
    assert empty.page_table is None and empty.seq_lens is None  # (torch's address of nothing)
    idle = dsa.dsa_batch(FAKE, FAKE, FAKE, 2, 4, 0, 0)
    for b in (empty, idle):
        for none in (True, False):
            for status in calls(dsa, c, b, FAKE, FAKE, none):
                assert status in passed
    assert dsa.dsa_cache_gather(c, idle, 1, 3, 0, None, None, FAKE, 1 << 30, 0) in passed
    # something to do still needs its pointers
    b = dsa.dsa_batch(FAKE, FAKE, FAKE, 2, 4, 1, 0)
    assert all(s == dsa.DSA_ERR_NULL for s in calls(dsa, c, b, FAKE, FAKE, True))
    for table, lens in ((None, FAKE), (FAKE, None)):
        b = dsa.dsa_batch(table, FAKE, lens, 2, 4, 0, 0)
        assert all(s == dsa.DSA_ERR_NULL for s in calls(dsa, c, b, FAKE, FAKE, False))
    assert dsa.dsa_cache_gather(c, idle, 1, 3, 1, None, FAKE, FAKE, 1 << 30, 0) == dsa.DSA_ERR_NULL
    assert dsa.dsa_cache_gather(c, empty, 0, 0, 0, None, None, FAKE, 1 << 30, 0) == dsa.DSA_ERR_DIMS


@pytest.mark.gpu
def test_nothing_clears_the_status(dsa):
    import torch

    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    h = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    c = dsa.make_cache(torch.zeros(3, 64, 512, dtype=torch.uint8, device="cuda"),
                       torch.zeros(3, 64, 64, dtype=torch.uint8, device="cuda"),
                       torch.ones(3, device="cuda"))
    freq = torch.ones(32, device="cuda")
    for b in (dsa.make_batch(i(0, 4), i(1), i(0), 0), dsa.make_batch(i(2, 4), i(3), i(2), 0)):
        n = dsa.dsa_cache_workspace_size(c, b, 32)
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
        dsa.check(dsa.dsa_cache_append(c, b, h(0, 512), h(0, 64), freq, 0, h(0, 32, 64),
                                       h(0, 32, 576), 32, ws))
        assert dsa.dsa_device_status(ws) == dsa.DSA_OK
        ws.fill_(0xA5)
        dsa.check(dsa.dsa_cache_attn(c, b, h(0, 32, 576), 32, 0.04, 0, 0, h(0, 32, 512),
                                     torch.empty(0, 32, device="cuda"), ws))
        assert dsa.dsa_device_status(ws) == dsa.DSA_OK
    ws.fill_(0xA5)
    dsa.check(dsa.dsa_cache_gather(c, b, 1, 0, 0, h(0, 512), h(0, 64), ws))
    assert dsa.dsa_device_status(ws) == dsa.DSA_OK
