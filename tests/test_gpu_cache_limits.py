"""The paged cache at the ends of its ranges."""
import numpy as np
import pytest

from dsa_test_util import dev, dev_bf16, host_bf16_as_f32, torch_mod
from test_gpu_cache import MARK, Setup, bf16, check_attn, dsa, run_attn  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-1, 1 << 30, np.iinfo(np.int32).max, np.iinfo(np.int32).min])
@pytest.mark.parametrize("dc,heads", [(512, 32), (64, 4)])
def test_attn_reports_every_page_outside_the_pool(dsa, dc, heads, entry):  # noqa: F811
    s = Setup([70, 300], [1, 2], page=32, dc=dc, heads=heads, seed=3)
    s.table[1, 3] = entry  # rows 96..127
    s.d_table = dev(s.table)
    run_attn(dsa, s, want_status=dsa.DSA_ERR_RANGE)


@pytest.mark.parametrize("pinned", [False, True])
def test_a_workspace_in_host_memory_is_refused(dsa, pinned):  # noqa: F811
    t = torch_mod()
    s = Setup([70], [1], seed=4)
    c, b = s.structs(dsa)
    ws = t.zeros(dsa.dsa_cache_workspace_size(c, b, 32), dtype=t.uint8, pin_memory=pinned)
    x = t.zeros(1, 32, 576, dtype=t.bfloat16, device="cuda")
    freq = dev(s.inv_freq())
    assert dsa.dsa_cache_attn(c, b, x, 32, 0.04, 0, 0, x, None, ws) == dsa.DSA_ERR_DEVICE
    assert dsa.dsa_cache_append(c, b, x[:, 0], x[:, 0, :64], freq, 0, None, None, 1, ws,
                                ld_latent=512, ld_rope=64) == dsa.DSA_ERR_DEVICE
    assert dsa.dsa_cache_gather(c, b, 0, 0, 1, x, x, ws) == dsa.DSA_ERR_DEVICE


@pytest.mark.parametrize("page", [16, 64])
def test_a_page_that_fills_token_by_token(dsa, page):  # noqa: F811
    """Its scale is read, kept or raised, and written at every step."""
    t = torch_mod()
    s = Setup([page], [1], page=page, seed=page)
    r, f = s.reference(), s.inv_freq()
    c, _ = s.structs(dsa)
    ws = t.empty(256, dtype=t.uint8, device="cuda")
    for i in range(page):
        lat_b, lat = bf16(s.rng.standard_normal((1, 512)) * 2.0 ** ((i * 7) % 11 + i // 4))
        rope_b, rope = bf16(s.rng.standard_normal((1, 64)))
        r.lens = np.array([i + 1], np.int32)
        r.append(lat, rope, f, False)
        b = dsa.make_batch(s.d_table, s.d_cu, dev(r.lens), 1)
        dsa.check(dsa.dsa_cache_append(c, b, dev_bf16(lat_b), dev_bf16(rope_b), dev(f), 0, None, None,
                                       1, ws))
        dsa.check(dsa.dsa_device_status(ws))
        np.testing.assert_array_equal(s.d_scale.cpu().numpy(), r.scale.astype(np.float32))
        np.testing.assert_array_equal(s.d_latent.cpu().numpy(), r.latent)
        np.testing.assert_array_equal(s.d_rope.cpu().numpy(), r.rope)


def test_the_largest_values(dsa):  # noqa: F811
    """The largest bf16 below 2^127 and a rotary pair whose turn comes as near: finite
    through append, gather and attention. (Queries of 0: the logits are 0.)"""
    t = torch_mod()
    s = Setup([70], [70], page=64, seed=8)
    r, f = s.reference(), s.inv_freq()
    c, b = s.structs(dsa)
    ws = s.workspace(dsa, c, b)
    top = 2.0 ** 127 - 2.0 ** 119
    lat_b, lat = bf16(np.where(s.rng.random((70, 512)) < 0.1, top, s.rng.standard_normal((70, 512))))
    lat_b[:, ::7] ^= 0x8000
    lat[:, ::7] *= -1
    rope_b, rope = bf16(np.full((70, 64), top / 2))
    r.append(lat, rope, f, False)
    dsa.check(dsa.dsa_cache_append(c, b, dev_bf16(lat_b), dev_bf16(rope_b), dev(f), 0, None, None, 1,
                                   ws))
    dsa.check(dsa.dsa_device_status(ws))
    assert r.scale[s.table[0, 0]] == 2.0 ** 119
    np.testing.assert_array_equal(s.d_scale.cpu().numpy(), r.scale.astype(np.float32))
    np.testing.assert_array_equal(s.d_latent.cpu().numpy(), r.latent)
    np.testing.assert_array_equal(s.d_rope.cpu().numpy(), r.rope)
    g_lat = t.empty(70, 512, dtype=t.bfloat16, device="cuda")
    g_rope = t.empty(70, 64, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_gather(c, b, 0, 0, 70, g_lat, g_rope, ws))
    want, _ = r.rows(0, np.arange(70))
    assert np.isfinite(want).all() and np.abs(want).max() == 2.0 ** 127
    np.testing.assert_array_equal(host_bf16_as_f32(g_lat), want[:, :512])
    np.testing.assert_array_equal(host_bf16_as_f32(g_rope), want[:, 512:])
    q = t.zeros(70, 32, 576, dtype=t.bfloat16, device="cuda")
    out = t.full((70, 32, 512), MARK, dtype=t.bfloat16, device="cuda")
    lse = t.full((70, 32), MARK, dtype=t.float32, device="cuda")
    dsa.check(dsa.dsa_cache_attn(c, b, q, 32, 0.04, 0, 0, out, lse, ws))
    dsa.check(dsa.dsa_device_status(ws))
    check_attn(host_bf16_as_f32(out), lse.cpu().numpy(),
               r.attend(np.zeros((70, 32, 576)), float(np.float32(0.04)), 0, 0))


def test_statuses_of_calls_that_are_checked_together(dsa):  # noqa: F811
    """Each call has the workspace of its own that the README gives it: what append
    finds is there after the attention."""
    t = torch_mod()
    s = Setup([70, 40], [6, 1], page=32, seed=6)
    s.lens[1] = 0  # a token, and no row for it
    s.d_lens = dev(s.lens)
    c, b = s.structs(dsa)
    ws, ws2 = s.workspace(dsa, c, b), s.workspace(dsa, c, b)
    x = t.zeros(7, 32, 576, dtype=t.bfloat16, device="cuda")
    out = t.zeros(7, 32, 512, dtype=t.bfloat16, device="cuda")
    dsa.check(dsa.dsa_cache_append(c, b, out[:, 0], x[:, 0, 512:], dev(s.inv_freq()), 0, None, None, 1,
                                   ws))
    sound = Setup([70, 40], [6, 1], page=32, seed=6)
    c2, b2 = sound.structs(dsa)
    dsa.check(dsa.dsa_cache_attn(c2, b2, x, 32, 0.04, 0, 0, out, None, ws2))
    assert dsa.dsa_device_status(ws) == dsa.DSA_ERR_RANGE
    assert dsa.dsa_device_status(ws2) == dsa.DSA_OK
