"""The paged cache's kernels in the checking build (libdsa_check.so): the same tests,
whose calls have to leave a clean status, so that no index was found out of bounds."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

TESTS = os.path.dirname(os.path.abspath(__file__))


def test_checking_build_is_clean_on_the_paged_cache():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_prefill_dsa_b200 import build

    build.build(variant="check")
    code = ("import sys, pytest\nsys.path.insert(0, %r)\n"
            "import sparse_attention_prefill_dsa_b200 as dsa\n"
            "assert dsa.LIB_PATH.endswith('libdsa_check.so'), dsa.LIB_PATH\n"
            "sys.exit(pytest.main(['-x', '-q', '-p', 'no:cacheprovider', '-k', %r, %r]))" % (
                os.path.dirname(TESTS),
                "append or gather or attn_chunks or attn_window or sms or wrong or without or captured",
                os.path.join(TESTS, "test_gpu_cache.py")))
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, DSA_LIBRARY="check"),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
