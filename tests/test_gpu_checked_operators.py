"""The suites of the 16-bit operators run again against the checked build
(libmilo_checked.so, see test_gpu_checked.py), in a child process whose library
the child confirms before it starts."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys, pytest
import int3_gemm_rank_b200 as m
m.lib()
assert m.LIB_PATH.endswith('libmilo_checked.so'), m.LIB_PATH
sys.exit(pytest.main(['tests/test_gpu_exchange.py', 'tests/test_gpu_dense.py', 'tests/test_gpu_operator_edges.py',
                      '-m', 'gpu', '-x', '-q', '-p', 'no:cacheprovider']))
"""


def test_operator_suites_pass_on_the_checked_build():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int3_gemm_rank_b200 import build
    build.build(checked=True)
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, env=dict(os.environ, MILO_LIBRARY="checked"),
                       capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
