"""The failure path of the paged cache's attention: waits with limits too short for
the kernel's own steps run out here and there, the blocks end, the status says so, and
the next call on the same workspace is right. (The order of the barriers on that path
is checked on the CPU, in test_cache_protocol.py.)"""
import numpy as np
import pytest

from dsa_test_util import dev_bf16, torch_mod
from test_gpu_cache import MARK, Setup, dsa, queries  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

LIMITS = [1 << 31, 100000, 30000, 10000, 5000, 2500, 1200, 600, 300, 0]


@pytest.mark.parametrize("window,n_sink", [(0, 0), (300, 20)])
@pytest.mark.parametrize("lens,new,heads", [
    ([700], [1], 32),                 # 32 rows, a tile an SM
    ([3000, 40, 900] * 24, [1] * 72, 32),  # 32 rows, several sequences an SM
    ([900, 2500], [130, 700], 32)])   # 64 rows, several items an SM
def test_waits_that_run_out_end_the_call(dsa, lens, new, heads, window, n_sink):  # noqa: F811
    t = torch_mod()
    s = Setup(lens, new, heads=heads, page=64, seed=len(lens))
    q_b, _ = queries(s)
    q = dev_bf16(q_b)
    c, b = s.structs(dsa)
    ws = s.workspace(dsa, c, b)

    def call(limit):
        out = t.full((s.n_tok, heads, s.dc), MARK, dtype=t.bfloat16, device="cuda")
        lse = t.full((s.n_tok, heads), MARK, dtype=t.float32, device="cuda")
        a = (c, b, q, heads, 0.04, window, n_sink, out, lse)
        dsa.check(dsa.dsa_cache_attn(*a, ws) if limit is None else
                  dsa.dsa_selftest_cache_wait(*a, limit, ws))
        return dsa.dsa_device_status(ws), out.view(t.int16), lse

    status, want, want_lse = call(None)
    assert status == dsa.DSA_OK
    seen = []
    for limit in LIMITS:
        for _ in range(3):
            status, got, lse = call(limit)
            seen.append(status)
            assert status in (dsa.DSA_OK, dsa.DSA_ERR_TIMEOUT)
            if status == dsa.DSA_OK:
                assert t.equal(got, want) and t.equal(lse, want_lse)
            status, got, lse = call(None)
            assert status == dsa.DSA_OK and t.equal(got, want) and t.equal(lse, want_lse)
    assert seen[:3] == [dsa.DSA_OK] * 3  # a limit of about a second
    assert seen[-3:] == [dsa.DSA_ERR_TIMEOUT] * 3
    assert np.isfinite(want_lse.cpu().numpy()).all()
