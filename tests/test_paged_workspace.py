"""The workspace that the paged attention asks for, and what it does with one."""
import pytest
import torch

import oracle
from paged_util import Paged, check_rows, make

moda = pytest.importorskip("depth_kv_attention_b200",
                           reason="libmoda.so not built (python depth_kv_attention_b200/csrc/build.py)")


def size(max_q=90, Hq=8, Hkv=2, d=128, pages=1000, page=16, dtype=torch.bfloat16, q8=True, **kw):
    return moda.moda_fwd_paged_workspace_bytes(99, 2, max_q, Hq, Hkv, d, pages, page, dtype, q8, **kw)


def test_none_where_the_scalar_path_runs():
    """8-bit rows that TMA cannot address (d % 16), fp32, odd pages."""
    assert size(d=72) == 0
    assert size(d=72, max_q=1) == 0
    assert size(d=72, q8=False) > 0
    assert size(dtype=torch.float32) == 0
    assert size(page=24) == 0


def run(x, c, **kw):
    return moda.moda_fwd_paged_q8(x["q"], x["k_pages"], x["v_pages"], x["k_scale"], x["v_scale"], x["table"], x["cu_q"],
                                  x["ctx"], x["max_q"], kd=x["kd"], vd=x["vd"], Ld=c.Ld, **kw)


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


def check(got, x, c, scale=None):
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    w = oracle.paged_forward(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], x["kd"], x["vd"], c.Ld,
                             scale or c.d ** -0.5, x["k_scale"], x["v_scale"])
    check_rows(*got, w, c.dtype, 800, c.d)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(impl="simt"), dict(scale=-0.1)], ids=["simt", "negative_scale"])
def test_no_more_than_the_kernel_that_runs_needs(kw):
    """Chunks over 8-bit pages that do not take the kernel with the bf16 copy run
    without room for one."""
    c = Paged("ws", ((300, 70), (90, 40)), Hq=8, Hkv=1, Ld=2, cap=2)
    x = make(c, q8=True)
    few = moda.moda_fwd_paged_workspace_bytes(c.N, 2, 4, 8, 1, c.d, x["k_pages"].shape[0], c.P, torch.bfloat16, True)
    ws = torch.empty(few, dtype=torch.uint8, device="cuda")
    check(run(cuda(x), c, workspace=ws, **kw), x, c, kw.get("scale"))
