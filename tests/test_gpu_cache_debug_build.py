"""The paged cache's suites again, on the build with device bounds checks (see
test_gpu_debug_build.py): page-table reads, rows written and read, workspace slots and
output rows are tested against their buffers, and no check may fail."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("suite,only", [("tests/test_gpu_cache.py", ""),
                                        ("tests/test_gpu_cache_numbers.py", "test_numbers or own_powers")])
def test_cache_suites_pass_on_debug_build_with_clean_bounds(suite, only):
    from attention_score_reduction_b200 import build
    lib = build.build(debug=True)
    env = dict(os.environ, KVZIP_LIBRARY=lib, KVZIP_EXPECT_DEBUG="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        *(["-k", only] if only else []), suite], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
