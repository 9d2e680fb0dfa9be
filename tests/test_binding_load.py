"""Loading the Python binding of the small calls (host only)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("fault", [
    'sys.modules["invariant_verify_gb300._biv_torch"] = None',       # its import raises
    'torch.__version__ = "1.0.0"',                                   # it was built for another torch
])
def test_the_library_loads_without_the_binding(fault):
    """Every call has its way through ctypes: a binding that cannot be used costs time only."""
    from invariant_verify_gb300 import build
    build.build()
    r = subprocess.run([sys.executable, "-c", "import sys, torch\n" + fault + CALLS], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


CALLS = """
import warnings
from invariant_verify_gb300 import abi as B
with warnings.catch_warnings(record=True) as w:
    warnings.simplefilter("always")
    assert B.biv_status_string(2)
    assert len(w) == 1 and "_biv_torch" in str(w[0].message), w
z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)
for fn, args in ((B.biv_gemm_bias_act, (z(4, 64), z(64, 64), z(4, 64))),
                 (B.biv_softmax, (z(4, 8, t=torch.float32), z(4, 8, t=torch.float32), 1.0))):
    try:
        fn(*args)
    except B.BivError as e:
        assert e.status == 7, e                              # the tensors' place, found by abi.py's own checks
    else:
        raise AssertionError(fn)
"""
