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


def build_module():
    spec = importlib.util.spec_from_file_location(
        "moda_build_under_test", os.path.join(ROOT, "depth_kv_attention_b200", "csrc", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_binding_is_built_again_when_torch_changes(tmp_path, monkeypatch):
    """The object depends on the installed torch and Python and on the compile
    command as much as on its source."""
    mod = build_module()
    monkeypatch.setattr(mod, "BIND", str(tmp_path / "_moda_torch.so"))
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "_build"))
    runs = []

    def compile_(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("object")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mod.subprocess, "run", compile_)
    mod.build_binding()
    mod.build_binding()
    assert len(runs) == 1
    with monkeypatch.context() as m:
        m.setattr("importlib.metadata.version", lambda name: "99.0")
        mod.build_binding()
        mod.build_binding()
    assert len(runs) == 2
    with monkeypatch.context() as m:
        m.setattr("sysconfig.get_config_var", lambda name: ".other-python.so")
        mod.build_binding()
    assert len(runs) == 3
    mod.build_binding(force=True)
    assert len(runs) == 4
    os.remove(mod.BIND)
    mod.build_binding()
    assert len(runs) == 5


def test_a_failed_compile_leaves_no_key(tmp_path, monkeypatch):
    mod = build_module()
    monkeypatch.setattr(mod, "BIND", str(tmp_path / "_moda_torch.so"))
    monkeypatch.setattr(mod, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(mod.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no header"))
    for _ in range(2):
        with pytest.raises(RuntimeError, match="no header"):
            mod.build_binding()


def test_binding_of_another_torch_is_refused(monkeypatch):
    import torch

    import depth_kv_attention_b200 as moda
    monkeypatch.setattr(moda, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    z = torch.zeros(1)
    with pytest.raises(ImportError, match="0.0.1"):
        moda.moda_fwd_paged(z, z, z, z, z, z, 1)


def test_a_binding_that_does_not_say_its_torch_is_refused(monkeypatch):
    import types

    import torch

    import depth_kv_attention_b200 as moda
    old = types.ModuleType("_moda_torch")
    monkeypatch.setattr(moda, "_bind", None)
    monkeypatch.setitem(sys.modules, "depth_kv_attention_b200._moda_torch", old)
    monkeypatch.setattr(moda, "_moda_torch", old, raising=False)
    z = torch.zeros(1)
    with pytest.raises(ImportError, match="build it again"):
        moda.moda_fwd_paged(z, z, z, z, z, z, 1)


def test_a_flag_without_a_truth_value_is_refused():
    """Before anything runs, and not as a result with an error pending."""
    import torch

    import depth_kv_attention_b200 as moda
    z = torch.zeros(1)
    with pytest.raises(ValueError, match="interleaved"):
        moda.moda_paged_append(z, z, z, z, z, z, z, z, interleaved=torch.zeros(2))


def out_of_memory():
    import torch

    import depth_kv_attention_b200 as moda

    def z(*s, t=torch.bfloat16):
        return torch.zeros(s, dtype=t, device="cuda")

    q, kp, table = z(4096, 32, 128), z(8, 4, 16, 128), z(1, 8, t=torch.int32)
    k = z(4096, 4, 128)
    cu, ctx = torch.tensor([0, 4096], dtype=torch.int32).cuda(), torch.tensor([128], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.0)  # the allocator takes nothing more from the driver
    with pytest.raises(torch.OutOfMemoryError):
        moda.moda_fwd_paged(q, kp, kp, table, cu, ctx, 4096)
    with pytest.raises(torch.OutOfMemoryError):
        moda.moda_paged_append(q, k, k, kp, kp, table, cu, ctx)


@pytest.mark.gpu
def test_out_of_memory_is_torchs():
    """An allocation that fails raises what torch's own functions raise. In a
    process of its own, whose allocator holds nothing that would serve it."""
    code = "import sys; sys.path[:0] = ['.', 'tests']; import test_paged_binding as t; t.out_of_memory()"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
