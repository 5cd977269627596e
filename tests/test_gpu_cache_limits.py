"""The paged cache at the ends of its ranges."""
import numpy as np
import pytest

from dsa_test_util import dev
from test_gpu_cache import Setup, dsa, run_attn  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-1, 1 << 30, np.iinfo(np.int32).max, np.iinfo(np.int32).min])
@pytest.mark.parametrize("dc,heads", [(512, 32), (64, 4)])
def test_attn_reports_every_page_outside_the_pool(dsa, dc, heads, entry):  # noqa: F811
    s = Setup([70, 300], [1, 2], page=32, dc=dc, heads=heads, seed=3)
    s.table[1, 3] = entry  # rows 96..127
    s.d_table = dev(s.table)
    run_attn(dsa, s, want_status=dsa.DSA_ERR_RANGE)
