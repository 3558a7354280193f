"""The serving operators of the MoDA library as cases to measure: the paged
sequence cache (append with the position rotation, 16/32-bit or 8-bit pages)
and the attention that reads it together with a token's depth keys.

``run`` computes a case in its plain form (elementary torch operations) or,
where ``own`` is true, through the library's entry points. ``exact`` restates
the definitions in float64, one sequence at a time.

Shared layout: B sequences with new tokens packed along one axis (``cu_q``
[B+1]); ``ctx`` [B] counts each sequence's tokens with the new ones, so new
token i of n sits at position ctx - n + i; ``table`` [B, blocks] gives the page
of every block of ``page`` positions; pages are [pages, Hkv, page, d].
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    base = dict(dtype="bf16", heads=32, kv_heads=4, dim=128, depth=0, slots=0, rot=0, inter=False)
    return [
        # one decode step of a batch: one token per sequence, every q and k
        # rotated, the pair also written to a slot of the token's depth rows
        dict(base, name="append_step", op="append", seqs=64, new=1, ctx=1000, spread=0.8, page=16, slots=28, rot=128),
        # two long prompts written at once
        dict(base, name="append_prompt", op="append", seqs=2, new=16384, ctx=16384, spread=0.0, page=64, slots=4,
             rot=128),
        # ragged chunks in fp32, a partial rotation of neighbouring pairs and
        # pages of 24 tokens
        dict(base, name="append_ragged_f32", op="append", dtype="f32", seqs=7, new=250, ctx=700, spread=0.9, page=24,
             heads=4, kv_heads=1, dim=64, slots=4, rot=32, inter=True),
        # a decode step into the 8-bit cache
        dict(base, name="append_q8_step", op="append_q8", seqs=64, new=1, ctx=100, spread=0.8, page=16, slots=28,
             rot=128),
        # chunks of prompts into the 8-bit cache, most start inside a page
        dict(base, name="append_q8_chunk", op="append_q8", seqs=8, new=2000, ctx=2500, spread=0.7, page=32, slots=4,
             rot=128),
        # the smallest call: a few short sequences, fp32, where latency counts
        dict(base, name="attend_tiny_f32", op="attend", dtype="f32", seqs=4, new=1, ctx=128, spread=0.5, page=16,
             heads=4, kv_heads=1, dim=64, depth=4, slots=4),
        # the usual decode step: many sequences of mixed lengths
        dict(base, name="attend_step", op="attend", seqs=64, new=1, ctx=8192, spread=0.75, page=16, depth=28,
             slots=28),
        # one user with a long context: few rows, one long axis
        dict(base, name="attend_step_64k", op="attend", seqs=1, new=1, ctx=65536, spread=0.0, page=64, depth=28,
             slots=28),
        # several drafted tokens checked at once, 32 heads on one kv-head, at
        # a layer whose buffer is not yet full
        dict(base, name="attend_draft_g32", op="attend", seqs=16, new=4, ctx=8192, spread=0.5, page=32, heads=32,
             kv_heads=1, depth=20, slots=28),
        # chunks of long prompts over what the cache holds already
        dict(base, name="attend_chunk", op="attend", seqs=3, new=1024, ctx=16384, spread=0.5, page=64, depth=16,
             slots=16),
        # the decode step and the chunk over the 8-bit cache
        dict(base, name="attend_q8_step", op="attend_q8", seqs=64, new=1, ctx=8192, spread=0.75, page=16, depth=28,
             slots=28),
        dict(base, name="attend_q8_chunk", op="attend_q8", seqs=2, new=1024, ctx=16384, spread=0.5, page=64, depth=16,
             slots=16),
    ]


def _span(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "attend", "attend", "attend_q8", "attend_q8"])
    f32 = op in ("append", "attend") and rng.random() < 0.2
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 7, 8, 16, 32])
    while kv * group > 64:
        group = rng.choice([1, 2, 4, 7, 8])
    dim = rng.choice([64, 72, 128]) if f32 else rng.choice([64, 96, 128, 128, 128])
    c = dict(op=op, dtype="f32" if f32 else "bf16", heads=kv * group, kv_heads=kv, dim=dim,
             page=rng.choice([16, 24, 64]) if f32 else rng.choice([16, 32, 48, 64, 128]),
             spread=round(rng.uniform(0.0, 0.9), 2), depth=0, slots=0, rot=0, inter=False)
    c["seqs"] = _span(rng, 1, 16 if f32 else 96)
    if op.startswith("append"):
        c["new"] = 1 if rng.random() < 0.5 else _span(rng, 2, 4000)
        c["ctx"] = c["new"] + _span(rng, 1, 1000)
        c["slots"] = rng.choice([0, 4, 12])
        c["rot"] = rng.choice([0, dim, dim, dim // 2])
        c["inter"] = rng.random() < 0.3
        most = {"append": 60e6, "append_q8": 12e6}[op]
        while c["seqs"] * c["ctx"] * (kv + (c["heads"] if c["new"] > 1 else 0)) * dim > most and c["ctx"] > 8:
            c["new"] = max(1, c["new"] // 2)
            c["ctx"] = max(c["new"], c["ctx"] // 2)
    else:
        c["new"] = rng.choice([1, 1, 1, _span(rng, 2, 8), _span(rng, 9, 1024)])
        c["ctx"] = max(c["new"], _span(rng, 1, 1500 if f32 else 65536))
        c["slots"] = rng.choice([0, 4, 16, 28, 33])
        c["depth"] = c["slots"] if rng.random() < 0.7 else rng.randint(0, c["slots"])
        if f32:
            c["new"] = min(c["new"], 16)
        while c["ctx"] > 64 and (work(c)["bytes"] > 6e8 or work(c)["flops"] > 2.5e11):
            c["ctx"] //= 2
            c["new"] = max(1, min(c["new"], c["ctx"]) * 3 // 4) if c["new"] > 8 else min(c["new"], c["ctx"])
    return c


def _lengths(case):
    """(ctx, new) of every sequence: the case's largest for the first, shorter
    ones after it; with three sequences or more the second has nothing new."""
    B, ctx, new = case["seqs"], [], []
    for b in range(B):
        part = 1.0 - case["spread"] * ((b * 29) % B) / B
        n = max(1, int(case["new"] * part))
        if B >= 3 and b == 1 and case["new"] > 1:
            n = 0
        ctx.append(max(n, 1, int(case["ctx"] * part)))
        new.append(n)
    return ctx, new


def work(case):
    ctx, new = _lengths(case)
    N, Hq, Hkv, d, L = sum(new), case["heads"], case["kv_heads"], case["dim"], case["depth"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("append"):
        q8 = case["op"] == "append_q8"
        read = N * (Hq + 2 * Hkv) * d * e + N * case["rot"] * 4
        write = N * Hq * d * e + N * 2 * Hkv * d * (1 if q8 else e) + (N * 2 * Hkv * d * e if case["slots"] else 0)
        return {"bytes": read + write, "flops": N * (Hq + Hkv) * case["rot"] * 3 + (N * 2 * Hkv * d * 2 if q8 else 0)}
    seen = [c if n else 0 for c, n in zip(ctx, new)]
    pairs = sum(n * c - n * (n - 1) // 2 for c, n in zip(ctx, new)) + N * L
    kv_bytes = sum(seen) * Hkv * d * 2 * (1 if case["op"] == "attend_q8" else e)
    return {"bytes": kv_bytes + 2 * N * Hq * d * e + N * Hq * 4 + N * L * Hkv * d * 2 * e, "flops": 4 * d * Hq * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(int(seed))
    dev, dt = "cuda", _DT[case["dtype"]]
    Hq, Hkv, d, P = case["heads"], case["kv_heads"], case["dim"], case["page"]
    ctx, new = _lengths(case)
    N, B = sum(new), len(ctx)
    blocks = [-(-c // P) for c in ctx]
    pages = sum(blocks) + 3  # three pages of the pool are nobody's
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max(blocks)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = dict(case=dict(case), table=table, cu_q=torch.tensor(cu, dtype=torch.int32, device=dev),
             ctx=torch.tensor(ctx, dtype=torch.int32, device=dev), max_q=max(new), scale=1.0 / math.sqrt(d))
    if case["op"].endswith("q8"):
        s["k_pages"] = (torch.randn((pages, Hkv, P, d), generator=g, device=dev) * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["v_pages"] = (torch.randn((pages, Hkv, P, d), generator=g, device=dev) * 32).round_().clamp_(-127, 127).to(torch.int8)
        for name in ("k_scale", "v_scale"):
            e = torch.randint(-6, -3, (pages, Hkv), generator=g, device=dev)
            s[name] = _power(e)
    else:
        s["k_pages"], s["v_pages"] = normal(pages, Hkv, P, d), normal(pages, Hkv, P, d)
    if case["slots"]:
        s["kd"], s["vd"] = normal(N, case["slots"], Hkv, d), normal(N, case["slots"], Hkv, d)
    else:
        s["kd"] = s["vd"] = None
    if case["op"].startswith("append"):
        # q, k and v as a model's one projection leaves them: columns of one matrix
        qkv = normal(N, (Hq + 2 * Hkv) * d)
        s["q"] = qkv[:, :Hq * d].view(N, Hq, d)
        s["k"] = qkv[:, Hq * d:(Hq + Hkv) * d].view(N, Hkv, d)
        s["v"] = qkv[:, (Hq + Hkv) * d:].view(N, Hkv, d)
        s["slot"] = case["slots"] // 2
        s["rope"] = None
        if case["rot"]:
            far = max(ctx)
            f = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
            a = torch.arange(far, device=dev, dtype=torch.float64)[:, None] * f
            s["rope"] = torch.cat([a.cos(), a.sin()], 1).float()
    else:
        # logits of a trained model spread wider than unit queries give
        s["q"] = (2 * torch.randn((N, Hq, d), generator=g, device=dev)).to(dt)
    return s


def _power(e):
    """2^e of whole e in [-126, 127], as fp32."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


# ------------------------------------------------------------ plain forms
def _positions(s):
    """Of every new token: its sequence, its position, its page and its row there."""
    P, i = s["case"]["page"], torch.arange(s["k"].shape[0], device=s["k"].device)
    cu, ctx = s["cu_q"].long(), s["ctx"].long()
    b = torch.searchsorted(cu[1:], i, right=True)
    pos = ctx[b] - cu[b + 1] + i
    return pos, s["table"].long()[b, pos // P], pos % P


def _rotate(x, rope, inter):
    if rope is None:
        return x
    h = rope.shape[-1] // 2
    c, n = rope[:, None, :h], rope[:, None, h:]
    y = x.clone()
    a, b = (x[..., 0:2 * h:2], x[..., 1:2 * h:2]) if inter else (x[..., :h], x[..., h:2 * h])
    u, w = a * c - b * n, b * c + a * n
    if inter:
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = u, w
    else:
        y[..., :h], y[..., h:2 * h] = u, w
    return y


def _append(s):
    pos, page, row = _positions(s)
    rope = None if s["rope"] is None else s["rope"][pos]
    q = _rotate(s["q"].float(), rope, s["case"]["inter"]).to(s["q"].dtype)
    k, v = _rotate(s["k"].float(), rope, s["case"]["inter"]), s["v"]
    if s["case"]["op"] == "append_q8":
        _into_q8(s["k_pages"], s["k_scale"], k, page, row)
        _into_q8(s["v_pages"], s["v_scale"], v.float(), page, row)
    else:
        s["k_pages"][page, :, row] = k.to(s["k_pages"].dtype)
        s["v_pages"][page, :, row] = v
    if s["kd"] is not None:
        s["kd"][:, s["slot"]] = k.to(s["kd"].dtype)
        s["vd"][:, s["slot"]] = v
    return q


def _into_q8(codes, scale, x, page, row):
    """Rows x [N, Hkv, d] into (page, row) of the 8-bit pages, in place."""
    top = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
    first = torch.full((codes.shape[0],), codes.shape[2], device=x.device, dtype=torch.int64)
    first = first.index_reduce_(0, page, row, "amin")[:, None]
    m, e = torch.frexp(top)
    e = (e - 7 + (m > 127 / 128).to(e.dtype)).clamp(-126, 120)
    fresh = torch.where(top > 0, _power(e), 0.0)
    touched = first < codes.shape[2]
    held = torch.where(touched & (first == 0), 0.0, scale)
    now = torch.where(touched, torch.maximum(held, fresh), scale)
    ratio = torch.where(now > 0, held / now, 0.0)
    before = torch.arange(codes.shape[2], device=x.device) < first
    moved = torch.round(codes.float() * ratio[:, :, None, None]).to(torch.int8)
    codes.copy_(torch.where((touched & before)[:, None, :, None], moved, codes))
    by = now[page][..., None]
    codes[page, :, row] = torch.where(by > 0, torch.round(x / by), 0.0).clamp(-127, 127).to(torch.int8)
    scale.copy_(now)


def _attend(s):
    case = s["case"]
    Hkv, d, P, L = case["kv_heads"], case["dim"], case["page"], case["depth"]
    q, table, cu, ctx = s["q"], s["table"].long(), s["cu_q"].long(), s["ctx"].long()
    N, Hq = q.shape[:2]
    B, n, G = table.shape[0], s["max_q"], Hq // Hkv
    dev = q.device

    def gathered(pages, scale):
        x = pages[table.clamp(min=0)].float()
        if scale is not None:
            x = x * scale[table.clamp(min=0)][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, d)  # [B, Hkv, keys, d]

    k, v = gathered(s["k_pages"], s.get("k_scale")), gathered(s["v_pages"], s.get("v_scale"))
    i = torch.arange(n, device=dev)
    there = i < (cu[1:] - cu[:-1])[:, None]                      # [B, n]
    tok = (cu[:-1, None] + i).clamp(max=N - 1)
    pos = (ctx - cu[1:] + cu[:-1])[:, None] + i
    x = q[tok].float().view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    j = torch.arange(k.shape[2], device=dev)
    seen = (j <= pos[..., None]) & (table >= 0).repeat_interleave(P, 1)[:, None]   # [B, n, keys]
    z = (x @ k.transpose(-1, -2)).view(B, Hkv, n, G, -1) * s["scale"]
    z = z.masked_fill(~seen[:, None, :, None], -math.inf)
    top = z.amax(-1)
    if L:
        kd, vd = s["kd"][tok, :L].float(), s["vd"][tok, :L].float()   # [B, n, L, Hkv, d]
        zd = torch.einsum("bhngd,bnlhd->bhngl", x.view(B, Hkv, n, G, d), kd) * s["scale"]
        top = torch.maximum(top, zd.amax(-1))
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(z - top[..., None])
    total = p.sum(-1)
    o = (p.view(B, Hkv, n * G, -1) @ v).view(B, Hkv, n, G, d)
    if L:
        pd = torch.exp(zd - top[..., None])
        total = total + pd.sum(-1)
        o = o + torch.einsum("bhngl,bnlhd->bhngd", pd, vd)
    o = o / torch.where(total > 0, total, 1.0)[..., None]
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    o = o.permute(0, 2, 1, 3, 4).reshape(B * n, Hq, d)
    lse = lse.permute(0, 2, 1, 3).reshape(B * n, Hq)
    at = torch.where(there, tok, N).view(-1)                      # rows that are not there go to a spare one
    out, low = torch.empty((N + 1, Hq, d), device=dev, dtype=q.dtype), torch.empty((N + 1, Hq), device=dev)
    out[at], low[at] = o.to(q.dtype), lse
    return out[:N], low[:N]


def _stands_for(codes, scale):
    """The values that 8-bit pages stand for: exact in bf16, as a scale is a power of two."""
    return codes.to(torch.bfloat16) * scale.to(torch.bfloat16)[:, :, None, None]


# --------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    if op.startswith("append"):
        if own:
            import depth_kv_attention_b200 as moda
            extra = dict(rope=s["rope"], interleaved=s["case"]["inter"], kd=s["kd"], vd=s["vd"], slot=s["slot"])
            if op == "append_q8":
                q = moda.moda_paged_append_q8(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scale"],
                                              s["v_scale"], s["table"], s["cu_q"], s["ctx"], **extra)
            else:
                q = moda.moda_paged_append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"],
                                           s["ctx"], **extra)
        else:
            q = _append(s)
        res = {"q": q}
        if op == "append_q8":
            res["k_pages"] = _stands_for(s["k_pages"], s["k_scale"])
            res["v_pages"] = _stands_for(s["v_pages"], s["v_scale"])
        else:
            res["k_pages"], res["v_pages"] = s["k_pages"], s["v_pages"]
        if s["kd"] is not None:
            res["kd"], res["vd"] = s["kd"], s["vd"]
        return res
    if own:
        import depth_kv_attention_b200 as moda
        if op == "attend_q8":
            out, lse = moda.moda_fwd_paged_q8(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                              s["table"], s["cu_q"], s["ctx"], s["max_q"], kd=s["kd"], vd=s["vd"],
                                              Ld=s["case"]["depth"], scale=s["scale"])
        else:
            out, lse = moda.moda_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cu_q"], s["ctx"],
                                           s["max_q"], kd=s["kd"], vd=s["vd"], Ld=s["case"]["depth"],
                                           scale=s["scale"])
    else:
        out, lse = _attend(s)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"].startswith("append") else _exact_attend(s)


def _exact_append(s):
    case, dev = s["case"], s["q"].device
    P, q8 = case["page"], case["op"] == "append_q8"
    cu, ctx, table = s["cu_q"].tolist(), s["ctx"].tolist(), s["table"].tolist()
    q, k, v = (s[n].double().clone() for n in ("q", "k", "v"))
    if case["rot"]:
        R = case["rot"]
        first = torch.arange(0, R, 2, device=dev) if case["inter"] else torch.arange(R // 2, device=dev)
        second = first + (1 if case["inter"] else R // 2)
        at = torch.cat([torch.arange(c - (cu[b + 1] - cu[b]), c, device=dev) for b, c in enumerate(ctx)])
        turn = torch.complex(s["rope"][at, :R // 2].double(), s["rope"][at, R // 2:].double())[:, None]
        for x in (q, k):
            w = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = w.real, w.imag
    pages = []
    for name, x in (("k", k), ("v", v)):
        held = s[name + "_pages"].double()
        if q8:
            held = held * s[name + "_scale"].double()[:, :, None, None]
            codes, scale = s[name + "_pages"].double(), s[name + "_scale"].double().clone()
        for b, c in enumerate(ctx):
            p, stop = c - (cu[b + 1] - cu[b]), c
            while p < stop:  # page by page
                last = min(stop, (p // P + 1) * P)
                page, r0 = table[b][p // P], p % P
                rows = x[cu[b + 1] - (stop - p):cu[b + 1] - (stop - last)].transpose(0, 1)   # [Hkv, rows, d]
                if q8:
                    top = rows.abs().amax((1, 2))
                    step = torch.exp2(torch.ceil(torch.log2(top / 127).clamp(min=-126)))
                    step = torch.where(top > 127 * step, 2 * step, torch.where(top <= 63.5 * step, step / 2, step))
                    step = torch.where(top > 0, step, 0.0)
                    if r0:
                        step = torch.maximum(step, scale[page])
                        codes[page, :, :r0] = torch.round(codes[page, :, :r0] * (scale[page] / step)[:, None, None])
                    codes[page, :, r0:r0 + last - p] = torch.round(rows / step[:, None, None]).clamp(-127, 127)
                    scale[page] = step
                    held[page] = codes[page] * step[:, None, None]
                else:
                    held[page, :, r0:r0 + last - p] = rows
                p = last
        pages.append(held)
    res = {"q": q, "k_pages": pages[0], "v_pages": pages[1]}
    if s["kd"] is not None:
        res["kd"], res["vd"] = s["kd"].double(), s["vd"].double()
        res["kd"][:, s["slot"]], res["vd"][:, s["slot"]] = k, v
    return res


def _exact_attend(s):
    case = s["case"]
    Hkv, d, P, L = case["kv_heads"], case["dim"], case["page"], case["depth"]
    N, Hq = s["q"].shape[:2]
    dev = s["q"].device
    out = torch.zeros((N, Hq, d), device=dev, dtype=torch.float64)
    lse = torch.zeros((N, Hq), device=dev, dtype=torch.float64)
    cu, ctx = s["cu_q"].tolist(), s["ctx"].tolist()
    for b, c in enumerate(ctx):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        ids = s["table"][b, :-(-c // P)].long()
        pos = torch.arange(c - (hi - lo), c, device=dev)
        hidden = torch.arange(c, device=dev) > pos[:, None]
        for h in range(Hkv):
            kk, vv = (s[n + "_pages"][ids, h].double() for n in ("k", "v"))
            if case["op"] == "attend_q8":
                kk, vv = kk * s["k_scale"][ids, h].double()[:, None, None], vv * s["v_scale"][ids, h].double()[:, None, None]
            kk, vv = kk.reshape(-1, d)[:c], vv.reshape(-1, d)[:c]
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["q"][lo:hi, hs].double() * s["scale"]                          # [n, G, d]
            z = (x @ kk.T).masked_fill_(hidden[:, None], -math.inf)              # [n, G, c]
            if L:
                z = torch.cat([z, x @ s["kd"][lo:hi, :L, h].double().transpose(1, 2)], -1)
            lse[lo:hi, hs] = torch.logsumexp(z, -1)
            w = z.sub_(lse[lo:hi, hs, None]).exp_()
            out[lo:hi, hs] = w[..., :c] @ vv
            if L:
                out[lo:hi, hs] += w[..., c:] @ s["vd"][lo:hi, :L, h].double()
    return {"out": out, "lse": lse}
