"""Refusals of the paged cache's entry points, decided before any CUDA call
(fake 16-byte aligned addresses, never dereferenced), and those of the Python
binding on CPU tensors."""
import ctypes

import pytest
import torch

moda = pytest.importorskip("depth_kv_attention_b200",
                           reason="libmoda.so not built (python depth_kv_attention_b200/csrc/build.py)")

_vp, _i, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong


def entry(name, args):
    fn = getattr(moda.lib, name)
    fn.restype, fn.argtypes = _i, args
    return fn


_APPEND = [_vp] * 3 + [_ll] * 3 + [_vp, _i, _i, _i] + [_vp] * 3 + [_i] * 9
_FWD = [_vp] * 5 + [_i] * 12 + [ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp, _i]
c_append = entry("moda_paged_append", _APPEND + [_vp] * 5 + [_i, _i, _vp])
c_append_q8 = entry("moda_paged_append_q8", _APPEND + [_vp] * 7 + [_i, _i, _vp])
c_fwd_paged = entry("moda_fwd_paged", [_vp] * 3 + _FWD)
c_fwd_paged_q8 = entry("moda_fwd_paged_q8", [_vp] * 5 + _FWD)

P = 0x10000
DIMS = dict(N=4, B=2, Hq=8, Hkv=2, d=128, pages=5, page=16, blocks=3, dt=0)


def append(q=P, k=P, v=P, sq=1024, sk=256, sv=256, rope=P, rope_len=64, rot=128, cu=P, ctx=P, table=P, kp=P, vp=P,
           qo=P, kd=P, vd=P, Ld=4, slot=1, scales=None, **kw):
    x = dict(DIMS, **kw)
    dims = [x["N"], x["B"], x["Hq"], x["Hkv"], x["d"], x["pages"], x["page"], x["blocks"], x["dt"]]
    args = [q, k, v, sq, sk, sv, rope, rope_len, rot, 0, cu, ctx, table, *dims, kp, vp]
    if scales is None:
        return c_append(*args, qo, kd, vd, Ld, slot, None)
    return c_append_q8(*args, *scales, qo, kd, vd, Ld, slot, None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(cu=None), 1),
    (dict(ctx=None), 1), (dict(table=None), 1), (dict(q=None), 1), (dict(qo=None), 1), (dict(kd=None), 1),
    (dict(vd=None), 1), (dict(N=0), 1), (dict(B=0), 1), (dict(pages=0), 1), (dict(page=0), 1), (dict(blocks=0), 1),
    (dict(Hq=7), 1), (dict(dt=5), 1), (dict(slot=4), 1), (dict(slot=-1), 1), (dict(rot=0), 1), (dict(rot=130), 1),
    (dict(rot=63), 1), (dict(rope_len=0), 1), (dict(sq=1016), 1), (dict(sk=248), 1), (dict(sv=0), 1),
    (dict(scales=(None, P)), 1), (dict(scales=(P, None)), 1),
    (dict(d=136, sq=1088, sk=272, sv=272), 2), (dict(d=12, rot=8), 2), (dict(d=6, rot=2, dt=1), 2),
    (dict(page=1 << 28), 2),
    (dict(q=P + 8), 3), (dict(k=P + 2), 3), (dict(kp=P + 4), 3), (dict(qo=P + 2), 3), (dict(kd=P + 8), 3),
    (dict(rope=P + 2), 3), (dict(cu=P + 1), 3), (dict(table=P + 2), 3), (dict(sq=1028), 3), (dict(sk=260), 3),
    (dict(scales=(P + 2, P)), 3),
])
def test_append_refusals(kw, code):
    assert append(**kw) == code


def fwd(q=P, kp=P, vp=P, kd=P, vd=P, cu=P, ctx=P, table=P, max_q=2, Ld=2, cap=4, scale=0.1, out=P, lse=P, ws=P,
        nws=1 << 40, impl=0, scales=None, **kw):
    x = dict(DIMS, **kw)
    tail = [kd, vd, cu, ctx, table, x["N"], x["B"], max_q, x["Hq"], x["Hkv"], x["d"], Ld, cap, x["pages"], x["page"],
            x["blocks"], x["dt"], scale, out, lse, ws, nws, None, impl]
    if scales is None:
        return c_fwd_paged(q, kp, vp, *tail)
    return c_fwd_paged_q8(q, kp, vp, *scales, *tail)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(out=None), 1), (dict(kd=None), 1),
    (dict(vd=None), 1), (dict(cu=None), 1), (dict(ctx=None), 1), (dict(table=None), 1), (dict(max_q=0), 1),
    (dict(Ld=-1), 1), (dict(Ld=5), 1), (dict(N=0), 1), (dict(Hq=3), 1), (dict(dt=9), 1), (dict(impl=9), 1),
    (dict(scale=float("nan")), 1), (dict(scales=(None, P)), 1), (dict(scales=(P, None)), 1),
    (dict(d=256), 2), (dict(d=20), 2), (dict(impl=3), 2), (dict(impl=2, dt=1), 2),
    (dict(impl=2, page=24), 2),
    (dict(q=P + 2), 3), (dict(kp=P + 8), 3), (dict(lse=P + 2), 3), (dict(kd=P + 8), 3), (dict(ctx=P + 2), 3),
    (dict(scales=(P, P + 1)), 3),
])
def test_fwd_refusals(kw, code):
    assert fwd(**kw) == code


def test_workspace_refusals():
    n = moda._c_paged_ws(4, 2, 2, 8, 2, 128, 5, 16, 0, 0)
    assert n > 0
    assert fwd(ws=None) == 4
    assert fwd(nws=n - 1) == 4
    assert fwd(ws=P + 8) == 3
    # chunks over 8-bit pages: two bf16 pools beside the parts of cut units
    a, b = (moda._c_paged_ws(99, 2, 90, 8, 2, 128, 1000, 16, 0, q8) for q8 in (0, 1))
    assert b - a >= 2 * 1000 * 2 * 16 * 128 * 2
    assert fwd(max_q=90, N=99, pages=1000, nws=b - 1, scales=(P, P)) == 4
    for bad in ((0, 2, 2, 8, 2, 128, 5, 16, 0, 0), (4, 2, 2, 7, 2, 128, 5, 16, 0, 0), (4, 2, 2, 8, 2, 128, 0, 16, 0, 0)):
        assert moda._c_paged_ws(*bad) == 0
    assert moda._c_paged_ws(4, 2, 2, 8, 2, 128, 5, 16, 1, 0) == 0  # fp32 needs none


def cpu_call():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    return dict(q=z(3, 4, 64), k=z(3, 2, 64), v=z(3, 2, 64), kp=z(5, 2, 16, 64), vp=z(5, 2, 16, 64),
                table=z(2, 3, t=torch.int32), cu=z(3, t=torch.int32), ctx=z(2, t=torch.int32))


@pytest.mark.parametrize("change", [
    dict(kp=torch.zeros(5, 2, 16, 32, dtype=torch.bfloat16)), dict(vp=torch.zeros(5, 2, 8, 64, dtype=torch.bfloat16)),
    dict(cu=torch.zeros(2, dtype=torch.int32)), dict(ctx=torch.zeros(3, dtype=torch.int32)),
    dict(table=torch.zeros(2, 3, dtype=torch.int64)), dict(kp=torch.zeros(5, 2, 16, 64), vp=torch.zeros(5, 2, 16, 64)),
    dict(v=torch.zeros(3, 1, 64, dtype=torch.bfloat16)), dict(k=torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2)),
    dict(q=torch.zeros(3, 4, 64)), dict(kp=torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)),
    dict(),  # CPU tensors
])
def test_binding_refusals(change):
    x = dict(cpu_call(), **change)
    with pytest.raises((ValueError, RuntimeError)):
        moda.moda_paged_append(x["q"], x["k"], x["v"], x["kp"], x["vp"], x["table"], x["cu"], x["ctx"])
    if "v" in change or "k" in change:
        return
    with pytest.raises((ValueError, RuntimeError)):
        moda.moda_fwd_paged(x["q"], x["kp"], x["vp"], x["table"], x["cu"], x["ctx"], 1)


def test_binding_refuses_8bit_mistakes():
    x = cpu_call()
    s = torch.zeros(5, 2)
    with pytest.raises(ValueError):  # bf16 pages with scales
        moda.moda_fwd_paged_q8(x["q"], x["kp"], x["vp"], s, s, x["table"], x["cu"], x["ctx"], 1)
    k8 = torch.zeros(5, 2, 16, 64, dtype=torch.int8)
    with pytest.raises(ValueError):  # scales of another shape
        moda.moda_fwd_paged_q8(x["q"], k8, k8, s[:4], s, x["table"], x["cu"], x["ctx"], 1)
    with pytest.raises(ValueError):
        moda.moda_paged_append_q8(x["q"], x["k"], x["v"], k8, k8, s.half(), s, x["table"], x["cu"], x["ctx"])
    with pytest.raises(ValueError):  # int8 pages without scales
        moda.moda_fwd_paged(x["q"], k8, k8, x["table"], x["cu"], x["ctx"], 1)
