"""The workspace that the paged attention asks for, and what it does with one."""
import os
import subprocess
import sys

import pytest
import torch

import oracle
from paged_util import Paged, check_rows, make

moda = pytest.importorskip("depth_kv_attention_b200",
                           reason="libmoda.so not built (python depth_kv_attention_b200/csrc/build.py)")


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


def check(got, x, c, scale=None, keys=302):
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    w = oracle.paged_forward(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], x["kd"], x["vd"], c.Ld,
                             scale or c.d ** -0.5, x["k_scale"], x["v_scale"])
    check_rows(*got, w, c.dtype, keys, c.d)


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


def test_goes_by_the_call_where_the_width_is_known():
    """Chunks over 8-bit pages: room for the table's entries, not for the pool."""
    parts = size(q8=False)
    page = 2 * 16 * 128 * 2                                   # bytes of a bf16 page of 2 heads
    for pages in (1000, 100000):
        n = size(pages=pages, max_blocks=6)
        assert parts + 2 * 12 * page <= n <= parts + 2 * 12 * page + 2048
        assert size(pages=pages) >= parts + 2 * pages * page
    assert size(pages=1000, max_blocks=900) == size(pages=1000)   # never more than for the pool
    assert size(max_blocks=6, q8=False) == parts
    assert size(max_blocks=6, max_q=1) == size(max_q=1)
    assert size(max_blocks=6, impl="simt") == 0
    assert size(max_blocks=0) == 0
    for pages in range(8, 40):
        for blocks in range(1, 25):
            n = size(pages=pages, max_blocks=blocks, Hkv=1)
            assert n <= size(pages=pages, Hkv=1)


# two sequences in a cache of many pages
LARGE = Paged("large", ((300, 70), (95, 40)), Hq=8, Hkv=2, Ld=2, cap=2)


def in_a_large_cache(c, pages):
    """The call's pages scattered over a pool of `pages`; scales elsewhere NaN."""
    x = make(c, q8=True)
    n = x["k_pages"].shape[0]
    at = torch.arange(n) * (pages // n) + 3
    g = cuda(x)
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        fill = float("nan") if name.endswith("scale") else 77
        pool = torch.full((pages, *x[name].shape[1:]), fill, dtype=x[name].dtype, device="cuda")
        pool[at] = g[name]
        g[name] = pool
    g["table"] = torch.where(x["table"] < 0, x["table"], at[x["table"].clamp(min=0)].to(torch.int32)).cuda()
    return x, g


@pytest.mark.gpu
def test_a_chunk_in_a_large_cache_takes_little():
    c = LARGE
    x, g = in_a_large_cache(c, 20000)
    pool = g["k_pages"].numel() * 2 * 2                      # bytes of both bf16 pools
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    got = run(g, c)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < pool / 4
    check(got, x, c)


@pytest.mark.gpu
@pytest.mark.parametrize("pages", [40, 20000], ids=["small_pool", "large_pool"])
@pytest.mark.parametrize("copy", [True, False], ids=["with_copy", "without_copy"])
@pytest.mark.parametrize("shift", [0, 16])
def test_exactly_the_bytes_asked_for(pages, copy, shift):
    """A workspace of the size asked for, or of the size for 16-bit pages: right
    rows, and nothing behind or before it is written."""
    c = LARGE
    x, g = in_a_large_cache(c, pages)
    n = moda.moda_fwd_paged_workspace_bytes(c.N, 2, x["max_q"], c.Hq, c.Hkv, c.d, pages, c.P, torch.bfloat16, copy,
                                            max_blocks=x["table"].shape[1])
    whole = torch.full((256 + n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    ws = whole[256 + shift:256 + shift + n]
    check(run(g, c, workspace=ws), x, c)
    assert torch.all(whole[:256 + shift] == 0xAB) and torch.all(whole[256 + shift + n:] == 0xAB)
    with pytest.raises(moda.ModaError):
        few = moda.moda_fwd_paged_workspace_bytes(c.N, 2, 8, c.Hq, c.Hkv, c.d, pages, c.P, torch.bfloat16, False)
        run(g, c, workspace=whole[:few - 256])


def copy_does_not_fit():
    c = Paged("full", ((9000, 70), (8700, 40)), Hq=8, Hkv=8, Ld=2, cap=2)
    x = make(c, q8=True)
    g = cuda(x)
    n = moda.moda_fwd_paged_workspace_bytes(c.N, 2, x["max_q"], c.Hq, c.Hkv, c.d, x["k_pages"].shape[0], c.P,
                                            torch.bfloat16, True, max_blocks=x["table"].shape[1])
    few = moda.moda_fwd_paged_workspace_bytes(c.N, 2, x["max_q"], c.Hq, c.Hkv, c.d, x["k_pages"].shape[0], c.P,
                                              torch.bfloat16, False)
    assert n > few + (60 << 20)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_allocated()
    limit = torch.cuda.memory_reserved() + few + (24 << 20)   # room for the parts, not for the copy
    torch.cuda.set_per_process_memory_fraction(limit / torch.cuda.get_device_properties(0).total_memory)
    got = run(g, c)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < few + (24 << 20)
    torch.cuda.set_per_process_memory_fraction(1.0)
    check(got, x, c, keys=9002)


@pytest.mark.gpu
def test_a_chunk_runs_where_the_copy_does_not_fit():
    """In a process of its own, whose allocator holds nothing that would serve it."""
    code = "import sys; sys.path[:0] = ['.', 'tests']; import test_paged_workspace as t; t.copy_does_not_fit()"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


@pytest.mark.parametrize("change,code", [
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(q=None), 1), (dict(max_q=0), 1), (dict(scale=float("nan")), 1),
    (dict(impl=3), 2), (dict(d=20), 2), (dict(kp=0x10008), 3), (dict(ws=0x10008), 3),
    (dict(ws=None), 4), (dict(nbytes=-1), 4), (dict(nbytes=0), 4),
])
def test_refusals_of_the_c_entry(change, code):
    """Decided before any CUDA call (fake addresses, never dereferenced).
    nbytes -1: one less than the kernel for few rows needs."""
    import ctypes
    A = 0x10000
    vp, i = ctypes.c_void_p, ctypes.c_int
    x = dict(q=A, kp=A, vp=A, ks=A, vs=A, max_q=90, d=128, scale=0.1, ws=A, nbytes=1 << 40, impl=0)
    x.update(change)
    if x["nbytes"] == -1:
        x["nbytes"] = moda.moda_fwd_paged_workspace_bytes(99, 2, 8, 8, 2, 128, 1000, 16, torch.bfloat16, False) - 1
    fn = moda.lib.moda_fwd_paged_q8_ex
    fn.restype = i
    fn.argtypes = [vp] * 10 + [i] * 12 + [ctypes.c_float, vp, vp, vp, ctypes.c_size_t, vp, i]
    assert fn(x["q"], x["kp"], x["vp"], x["ks"], x["vs"], None, None, A, A, A, 99, 2, x["max_q"], 8, 2, x["d"], 0, 0, 1000,
              16, 3, 0, x["scale"], A, A, x["ws"], x["nbytes"], None, x["impl"]) == code


def test_sizes_whose_indexes_would_pass_32_bits_take_another_kernel():
    """The last row tile's end, and the conversion's index over the table's
    entries behind the last one, have to fit 32 bits too."""
    def n(N, Hq=1, B=2, max_blocks=6, q8=False, max_q=90, d=8):
        return moda.moda_fwd_paged_workspace_bytes(N, B, max_q, Hq, 1, d, 1 << 30, 16, torch.bfloat16, q8,
                                                   max_blocks=max_blocks)
    assert n(0x7fffff00 - 1) > 0
    assert n(0x7fffff00) == 0 and n(0x7fffffff) == 0          # the scalar path, which needs none
    few = n(99, max_q=32, d=16)
    assert n(99, B=1, max_blocks=0x7fff0000, q8=True, d=16) > few   # the copy of the pages
    assert n(99, B=1, max_blocks=0x7fff0001, q8=True, d=16) == few  # the kernel for few rows
