"""Shared pieces of the paged-cache tests: random caches and error bounds."""
from dataclasses import dataclass

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@dataclass(frozen=True)
class Paged:
    """A paged call: per sequence (tokens with the new ones, new tokens)."""
    name: str
    seqs: tuple
    Hq: int = 8
    Hkv: int = 2
    d: int = 128
    P: int = 16
    Ld: int = 0
    cap: int = 0
    dtype: str = "bf16"
    rot: int = 0
    inter: bool = False
    spare_rows: int = 0   # packed rows behind the last sequence
    seed: int = 1

    @property
    def N(self):
        return sum(n for _, n in self.seqs) + self.spare_rows


def make(c: Paged, q8=False, dev="cpu"):
    """Tensors of a call. Rows of a page past its sequence's end, and pages of
    no sequence, hold NaN (codes: any) and scales of untouched pages NaN."""
    g = torch.Generator("cpu")
    g.manual_seed(c.seed)
    dt = DT[c.dtype]
    blocks = [max(0, -(-n // c.P)) for n, _ in c.seqs]
    pages = sum(blocks) + 2
    order = torch.randperm(pages, generator=g).tolist()
    width = max(1, max(blocks))
    table = torch.full((len(c.seqs), width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cu = [0]
    for _, n in c.seqs:
        cu.append(cu[-1] + n)
    N, shape = c.N, (pages, c.Hkv, c.P, c.d)

    def rnd(*s):
        return torch.randn(s, generator=g).to(dt)

    x = dict(table=table, cu_q=torch.tensor(cu, dtype=torch.int32),
             ctx=torch.tensor([n for n, _ in c.seqs], dtype=torch.int32),
             q=rnd(N, c.Hq, c.d), k=rnd(N, c.Hkv, c.d), v=rnd(N, c.Hkv, c.d), max_q=max(1, max(n for _, n in c.seqs)))
    held = torch.zeros(pages, c.P, dtype=torch.bool)
    for b, (n, _) in enumerate(c.seqs):
        for j in range(max(0, n)):
            held[int(table[b, j // c.P]), j % c.P] = True
    if q8:
        for n in ("k", "v"):
            x[n + "_pages"] = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
            s = 2.0 ** torch.randint(-8, -3, (pages, c.Hkv), generator=g).float()
            s[~held.any(1)] = float("nan")
            x[n + "_scale"] = s
    else:
        for n in ("k", "v"):
            p = rnd(*shape)
            p.masked_fill_(~held[:, None, :, None], float("nan"))
            x[n + "_pages"] = p
    cap = max(c.cap, c.Ld)
    x["kd"], x["vd"] = (rnd(N, cap, c.Hkv, c.d), rnd(N, cap, c.Hkv, c.d)) if cap else (None, None)
    if cap > c.Ld:  # slots a layer does not read yet
        x["kd"][:, c.Ld:] = float("nan")
        x["vd"][:, c.Ld:] = float("nan")
    x["rope"] = None
    if c.rot:
        far = max(n for n, _ in c.seqs)
        a = torch.arange(max(1, far), dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, c.rot, 2, dtype=torch.float64) / c.rot)
        x["rope"] = torch.cat([a.cos(), a.sin()], 1).float()
    if dev != "cpu":
        x = {n: t.to(dev) if torch.is_tensor(t) else t for n, t in x.items()}
    return x


def check_rows(got_out, got_lse, want, dtype, keys, d, what=""):
    """Element-wise against the float64 rows, by error bounds that follow from
    the arithmetic.

    Logits: fp32 accumulation of d exact products, one scaling: at most
    dz = (d + 4) 2^-24 zabs. lse: dz + 2^-19 (1 + |lse|) for exp2 / log2 and
    the fp32 sum. P: 2 dz + 2^-19 relative. out: that times sum P|v|, plus the
    sum's fp32 rounding (keys 2^-24), plus for bf16 half a step 2^-8 of each
    P and of the result (P is a bf16 matrix operand there)."""
    out, lse, absv, zabs = want
    rows = ~np.isnan(lse)
    got_out = got_out.detach().double().cpu().numpy()[rows]
    got_lse = got_lse.detach().double().cpu().numpy()[rows]
    out, lse, absv, zabs = out[rows], lse[rows], absv[rows], zabs[rows]
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), empty), what
    assert np.all(got_out[empty] == 0), what
    dz = (d + 4) * 2.0 ** -24 * zabs
    fin = ~empty
    err = np.abs(got_lse[fin] - lse[fin])
    assert np.all(err <= (dz[fin] + 2.0 ** -19 * (1 + np.abs(lse[fin])))), (what, "lse", err.max())
    rel = 2 * dz + 2.0 ** -19 + keys * 2.0 ** -24
    bound = rel[..., None] * absv
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * absv + 2.0 ** -8 * np.abs(out)
    else:
        bound = bound + 2.0 ** -24 * np.abs(out)
    err = np.abs(got_out - out)
    assert np.all(np.isfinite(got_out)), what
    worst = (err / np.maximum(bound, 1e-30)).max() if err.size else 0.0
    assert np.all(err <= bound + 1e-30), (what, "out", err.max(), worst)
    return worst
