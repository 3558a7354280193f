"""Attention over 8-bit pages whose value scales lie far from one: the smallest
scale that the append writes (2^-126), large ones, and both in one sequence."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

moda = pytest.importorskip("depth_kv_attention_b200")

P, D, BLOCKS = 16, 128, 20


def call(exponents, G, Ld, seed=3):
    """One sequence of 20 pages. The first key of every page has a logit 7 above
    the others' and values of zero, so that what comes out is carried by keys of
    small weight (e^-7 of the largest) alone. exponents: of the pages' value scales."""
    g = torch.Generator("cpu")
    g.manual_seed(seed)
    kc = torch.zeros(BLOCKS, 1, P, D, dtype=torch.int8)
    kc[:, :, 0, 0] = 112                     # q . k = 1 * 112 / 16 = 7
    vc = torch.randint(112, 128, (BLOCKS, 1, P, D), generator=g).to(torch.int8)
    vc[:, :, 0] = 0
    order = torch.randperm(BLOCKS, generator=g)
    vs = torch.empty(BLOCKS, 1)
    e = torch.tensor([exponents[i % len(exponents)] for i in range(BLOCKS)])
    vs[order, 0] = torch.exp2(e.double()).float()
    q = torch.zeros(1, G, D, dtype=torch.bfloat16)
    q[..., 0] = 1
    low = 2.0 ** min(exponents)
    kd = torch.zeros(1, Ld, 1, D, dtype=torch.bfloat16) if Ld else None
    vd = ((112 + 15 * torch.rand(1, Ld, 1, D, generator=g)) * low).to(torch.bfloat16) if Ld else None
    return dict(q=q, kp=kc, vp=vc, ks=torch.full((BLOCKS, 1), 2.0 ** -4), vs=vs,
                table=order.to(torch.int32)[None].contiguous(), cu=torch.tensor([0, 1], dtype=torch.int32),
                ctx=torch.tensor([BLOCKS * P - 3], dtype=torch.int32), kd=kd, vd=vd)


@pytest.mark.parametrize("exponents", [(-126,), (-126, -120, -118), (-100,), (0,), (3, -4, 5), (110,)],
                         ids=lambda e: "_".join(map(str, e)))
@pytest.mark.parametrize("G,Ld,impl", [(1, 0, "auto"), (8, 0, "auto"), (8, 3, "auto"), (16, 0, "auto"), (32, 2, "auto"),
                                       (40, 0, "auto"), (8, 0, "simt")])
def test_value_scales(exponents, G, Ld, impl):
    x = call(exponents, G, Ld)
    g = {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}
    out, lse = moda.moda_fwd_paged_q8(g["q"], g["kp"], g["vp"], g["ks"], g["vs"], g["table"], g["cu"], g["ctx"], 1,
                                      kd=g["kd"], vd=g["vd"], Ld=Ld, scale=1.0, impl=impl)
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    w, wl, absv, _ = oracle.paged_forward(x["q"], x["kp"], x["vp"], x["table"], x["cu"], x["ctx"], x["kd"], x["vd"], Ld,
                                          1.0, x["ks"], x["vs"])
    assert np.all(np.abs(lse.cpu().numpy() - wl) <= 2.0 ** -18 * (1 + np.abs(wl)))
    # P in bf16 and the result in bf16: half a step each; the rest (exp2, fp32
    # sums of 320 keys) stays below 2^-14. Nothing here is below bf16's smallest
    # normal number, 2^-126 (the result is 112 * 15 / (e^7 + 18) 2^-126 = 1.5 of it at least).
    err = np.abs(out.double().cpu().numpy() - w)
    assert np.all(err <= (2.0 ** -8 + 2.0 ** -14) * absv + 2.0 ** -8 * np.abs(w)), (err / absv).max()
