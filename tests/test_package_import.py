"""What importing the package needs: the operators on torch tensors need torch and the compiled
module, everything else does not."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_star_import_needs_no_torch():
    r = python("import sys; sys.modules['torch'] = None\n"
               "from weight_only_bit_moe_amd import *\n"
               "print(moe_wna16_status_string is not None, forward is not None)")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["True", "True"]


def test_operators_are_listed_and_reached_by_name():
    import weight_only_bit_moe_amd as M
    names = ("add_rmsnorm", "route_topk", "gemm_w8a8", "gemm_w8a8_workspace_for", "swiglu_quant",
             "moe_wna16_add_rmsnorm", "moe_wna16_route_topk", "moe_wna16_gemm_w8a8",
             "moe_wna16_gemm_w8a8_workspace_size", "moe_wna16_swiglu_quant")
    assert set(names) <= set(dir(M)) and set(M.__all__) <= set(dir(M))
    assert all(callable(getattr(M, n)) for n in names)
    with pytest.raises(AttributeError):
        M.no_such_operator
