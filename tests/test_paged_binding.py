"""The compiled binding of the paged functions: when it is loaded, when it is
built again, and how it passes errors on."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytest.importorskip("depth_kv_attention_b200",
                    reason="libmoda.so not built (python depth_kv_attention_b200/csrc/build.py)")


def test_dense_functions_work_without_the_binding():
    """Without a loadable binding the package imports and its ctypes functions
    work; a paged function says what is missing."""
    code = """
import sys
sys.modules["depth_kv_attention_b200._moda_torch"] = None   # an import of it fails
import torch
import depth_kv_attention_b200 as moda
assert moda.moda_status_string(1)
assert moda.moda_pack_depth_bytes(1, 8, 2, 128, 4, torch.bfloat16) > 0
assert moda.moda_fwd_paged_workspace_bytes(4, 2, 2, 8, 2, 128, 5, 16, torch.bfloat16) > 0
z = torch.zeros(1)
for call in (lambda: moda.moda_paged_append(z, z, z, z, z, z, z, z), lambda: moda.moda_fwd_paged(z, z, z, z, z, z, 1)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e), e
    else:
        raise SystemExit("no ImportError")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr + r.stdout
