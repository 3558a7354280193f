"""GPU parity of appending to the paged cache (moda_paged_append,
moda_paged_append_q8) with the float64 oracle.

The definition fixes every operation in fp32, so the same steps in numpy
float32 give the same bits; against float64 the rotated values are off by at
most three fp32 roundings and one to the storage type."""
import numpy as np
import pytest
import torch

import oracle
from paged_util import DT, Paged, make

pytestmark = pytest.mark.gpu

moda = pytest.importorskip("depth_kv_attention_b200")

CASES = [
    Paged("one_token", ((1, 1),), rot=128, cap=3),
    Paged("steps", tuple((17 + 13 * b, 1) for b in range(37)), Hq=32, Hkv=4, rot=128, cap=5),
    Paged("chunks", ((100, 100), (77, 30), (40, 0), (16, 16), (33, 17), (1, 1)), Hq=7, Hkv=7, rot=64, P=16, cap=2,
          spare_rows=3),
    Paged("inter", ((50, 20), (31, 31)), rot=128, inter=True, P=8),
    Paged("inter_part", ((50, 20), (31, 31)), rot=48, inter=True, P=32, d=96, Hq=14, Hkv=2, cap=1),
    Paged("odd_half", ((50, 20), (31, 31)), rot=36, d=72, dtype="f32", P=5, Hq=3, Hkv=1, cap=2),
    Paged("odd_inter", ((50, 20), (31, 31)), rot=34, d=64, inter=True, P=7, Hq=4, Hkv=1),
    Paged("odd_half_bf16", ((50, 20), (31, 31)), rot=20, d=64, P=24, Hq=4, Hkv=2, cap=1),
    Paged("no_rot", ((300, 300), (5, 2)), d=8, P=64, Hq=5, Hkv=5, cap=2),
    Paged("f32", ((130, 129), (64, 1), (65, 2)), d=128, dtype="f32", rot=128, P=64, Hq=16, Hkv=2, cap=1),
    Paged("f32_small", ((9, 9), (12, 4)), d=4, dtype="f32", rot=4, P=1, Hq=2, Hkv=1),
    # enough bytes for the bulk-copy form: one and several parts per token,
    # fp32, no rotation, sequences without new tokens and rows of none
    Paged("bulk", ((400, 390), (77, 0), (300, 220), (5, 5)), Hq=32, Hkv=4, rot=128, cap=2, spare_rows=3),
    Paged("bulk_parts", ((350, 349), (64, 33)), Hq=64, Hkv=8, rot=64, P=24, inter=True),
    Paged("bulk_f32", ((500, 480), (300, 211)), Hq=16, Hkv=2, d=72, rot=40, inter=True, dtype="f32", P=48, cap=1),
    Paged("bulk_plain", ((700, 650),), Hq=24, Hkv=3, P=32),
    Paged("many", tuple((3 + b % 5, b % 3) for b in range(1500)), d=16, rot=16, P=16, Hq=1, Hkv=1),
]


def bits(t):
    """Exact comparison that takes equal NaN as equal."""
    return torch.nan_to_num(t.float(), nan=12345.0)


@pytest.mark.parametrize("c", CASES, ids=[c.name for c in CASES])
def test_append(c):
    x = make(c)
    g = {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}
    mark = torch.full_like(g["q"], 7.0)
    slot = max(c.cap - 1, 0)
    q = moda.moda_paged_append(g["q"], g["k"], g["v"], g["k_pages"], g["v_pages"], g["table"], g["cu_q"], g["ctx"],
                               rope=g["rope"], interleaved=c.inter, q_out=mark, kd=g["kd"], vd=g["vd"], slot=slot)
    torch.cuda.synchronize()
    assert q is mark
    args = (x["q"], x["k"], x["v"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], x["rope"], c.inter,
            x["kd"], x["vd"], slot, torch.full_like(x["q"], 7.0))
    same = oracle.paged_append(*args, dtype=np.float32)
    near = oracle.paged_append(*args)
    half = torch.finfo(DT[c.dtype]).eps / 2
    for what, got, s, w in zip(("q", "k", "v", "kd", "vd"), (q, g["k_pages"], g["v_pages"], g["kd"], g["vd"]), same,
                               near):
        if got is None:
            continue
        got = got.cpu()
        assert torch.equal(bits(got), bits(torch.from_numpy(s).to(DT[c.dtype]))), what
        ok = ~np.isnan(w)
        # |a c| + |b s| <= sqrt(2) * 6 for these normals; three fp32 roundings of it
        err = np.abs(got.double().numpy() - w)[ok]
        assert np.all(err <= half * np.abs(w[ok]) + 3 * 2.0 ** -24 * 9), what


@pytest.mark.parametrize("c", CASES, ids=[c.name for c in CASES])
def test_append_q8(c):
    x = make(c, q8=True)
    g = {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}
    slot = max(c.cap - 1, 0)
    q = moda.moda_paged_append_q8(g["q"], g["k"], g["v"], g["k_pages"], g["v_pages"], g["k_scale"], g["v_scale"],
                                  g["table"], g["cu_q"], g["ctx"], rope=g["rope"], interleaved=c.inter,
                                  q_out=torch.full_like(g["q"], 7.0), kd=g["kd"], vd=g["vd"], slot=slot)
    torch.cuda.synchronize()
    qo, _, _, kd, vd = oracle.paged_append(x["q"], x["k"], x["v"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"],
                                           x["ctx"], x["rope"], c.inter, x["kd"], x["vd"], slot,
                                           torch.full_like(x["q"], 7.0), dtype=np.float32)
    dt = DT[c.dtype]
    assert torch.equal(bits(q.cpu()), bits(torch.from_numpy(qo).to(dt)))
    if kd is not None:
        assert torch.equal(bits(g["kd"].cpu()), bits(torch.from_numpy(kd).to(dt)))
        assert torch.equal(bits(g["vd"].cpu()), bits(torch.from_numpy(vd).to(dt)))
    kc, vc, ks, vs = oracle.paged_append_q8(x["k"], x["v"], x["k_pages"], x["v_pages"], x["k_scale"], x["v_scale"],
                                            x["table"], x["cu_q"], x["ctx"], x["rope"], c.inter)
    for name, want in (("k_pages", kc), ("v_pages", vc), ("k_scale", ks), ("v_scale", vs)):
        np.testing.assert_array_equal(g[name].double().cpu().numpy(), want, err_msg=name)


@pytest.mark.parametrize("seqs", [((40, 9), (25, 25)), ((2500, 2400), (1500, 1000))], ids=["few", "bulk"])
def test_columns_of_one_projection(seqs):
    """q, k and v as column blocks of one matrix (a token stride, dense heads)."""
    c = Paged("cols", seqs, Hq=8, Hkv=2, d=64, rot=64)
    x = make(c, dev="cuda")
    whole = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)], 1)
    q, k, v = whole[:, :512].view(-1, 8, 64), whole[:, 512:640].view(-1, 2, 64), whole[:, 640:].view(-1, 2, 64)
    res = []
    for a, b, e in ((x["q"], x["k"], x["v"]), (q, k, v)):
        kp, vp = x["k_pages"].clone(), x["v_pages"].clone()
        qo = moda.moda_paged_append(a, b, e, kp, vp, x["table"], x["cu_q"], x["ctx"], rope=x["rope"])
        res.append([bits(t) for t in (qo, kp, vp)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_q8_token_by_token_grows_and_matches():
    """A cache filled token by token (values growing, so codes move at most
    steps) equals the oracle's after every call, and each value is within one
    step of what was appended."""
    c = Paged("grow", ((40, 40),), Hq=2, Hkv=2, d=16, P=16, dtype="f32")
    x = make(c, q8=True)
    grow = 1.25 ** torch.arange(40).view(40, 1, 1)
    k, v = x["k"] * grow, x["v"] / grow
    g = [x[n].cuda() for n in ("k_pages", "v_pages", "k_scale", "v_scale")]
    w = [x[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")]
    cu = torch.tensor([0, 1], dtype=torch.int32)
    for t in range(40):
        ctx = torch.tensor([t + 1], dtype=torch.int32)
        moda.moda_paged_append_q8(None, k[t:t + 1].cuda(), v[t:t + 1].cuda(), *g, x["table"].cuda(), cu.cuda(), ctx.cuda())
        w = list(oracle.paged_append_q8(k[t:t + 1], v[t:t + 1], *w, x["table"], cu, ctx))
    torch.cuda.synchronize()
    for got, want in zip(g, w):
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    for codes, scale, src in ((g[0], g[2], k), (g[1], g[3], v)):
        for t in range(40):
            p = int(x["table"][0, t // 16])
            got = codes[p, :, t % 16].double().cpu() * scale[p].double().cpu()[:, None]
            assert torch.all((got - src[t].double()).abs() <= scale[p].double().cpu()[:, None])


def test_q8_unusual_values():
    """Zero rows (scale 0), NaN (code 0), infinities (+-127), ties to even and
    values at the smallest scale."""
    d, P = 16, 16
    k = torch.zeros(4, 1, d)
    k[1, 0, :8] = torch.tensor([127.0, 2.5, 3.5, -2.5, -3.5, 0.5, 1.5, -127.0])
    k[2, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0])
    k[3, 0, :3] = torch.tensor([1e-45, -1e-40, 1e-38])
    kp = torch.full((4, 1, P, d), 5, dtype=torch.int8).cuda()
    vp, ks, vs = kp.clone(), torch.full((4, 1), float("nan")).cuda(), torch.full((4, 1), float("nan")).cuda()
    table = torch.arange(4, dtype=torch.int32).view(4, 1)
    args = (table, torch.arange(5, dtype=torch.int32), torch.ones(4, dtype=torch.int32))
    w = oracle.paged_append_q8(k, k, kp.cpu(), vp.cpu(), ks.cpu(), vs.cpu(), *args)
    moda.moda_paged_append_q8(None, k.cuda(), k.cuda(), kp, vp, ks, vs, *(t.cuda() for t in args))
    torch.cuda.synchronize()
    for got, want in zip((kp, vp, ks, vs), w):
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    assert ks.cpu().flatten()[:2].tolist() == [0.0, 1.0]
    assert kp[1, 0, 0, :8].cpu().tolist() == [127, 2, 4, -2, -4, 0, 2, -127]
    assert kp[2, 0, 0, :4].cpu().tolist() == [0, 127, -127, 64]


@pytest.mark.parametrize("q8", [False, True])
def test_bad_positions_and_pages_are_left_out(q8):
    """No page (-1 or past the pool), a table that ends too early, a negative
    position, a position past the rope table: nothing is written there."""
    c = Paged("bad", ((20, 20), (20, 4), (30, 3), (2, 5), (40, 2)), Hq=2, Hkv=1, d=16, rot=16, P=16, cap=1)
    x = make(c, q8=q8)
    x["table"][0, 1], x["table"][1, 1] = -1, 10 ** 6
    x["table"] = x["table"][:, :2].contiguous()   # sequence 4's last block is out of the table
    x["rope"] = x["rope"][:29].contiguous()       # position 29 of sequence 2 is not in the rope table
    g = {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}
    fill = torch.full_like(g["q"], 7.0)
    common = dict(rope=g["rope"], q_out=fill, kd=g["kd"], vd=g["vd"])
    if q8:
        moda.moda_paged_append_q8(g["q"], g["k"], g["v"], g["k_pages"], g["v_pages"], g["k_scale"], g["v_scale"],
                                  g["table"], g["cu_q"], g["ctx"], **common)
        want = oracle.paged_append_q8(x["k"], x["v"], x["k_pages"], x["v_pages"], x["k_scale"], x["v_scale"],
                                      x["table"], x["cu_q"], x["ctx"], x["rope"])
        torch.cuda.synchronize()
        for name, w in zip(("k_pages", "v_pages", "k_scale", "v_scale"), want):
            np.testing.assert_array_equal(g[name].double().cpu().numpy(), w)
    else:
        moda.moda_paged_append(g["q"], g["k"], g["v"], g["k_pages"], g["v_pages"], g["table"], g["cu_q"], g["ctx"],
                               **common)
        torch.cuda.synchronize()
    qo, kp, vp, kd, vd = oracle.paged_append(x["q"], x["k"], x["v"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"],
                                             x["ctx"], x["rope"], False, x["kd"], x["vd"], 0,
                                             torch.full_like(x["q"], 7.0), dtype=np.float32)
    pairs = [(fill, qo), (g["kd"], kd), (g["vd"], vd)] + ([] if q8 else [(g["k_pages"], kp), (g["v_pages"], vp)])
    for got, w in pairs:
        assert torch.equal(bits(got.cpu()), bits(torch.from_numpy(w).to(torch.bfloat16)))


def test_without_queries():
    """q left out: keys and values only, in both forms."""
    for seqs in (((40, 9),), ((2500, 2400), (1500, 1000))):
        c = Paged("kv", seqs, Hq=8, Hkv=8, d=128, rot=128)
        x = make(c, dev="cuda")
        res = []
        for q in (x["q"], None):
            kp, vp = x["k_pages"].clone(), x["v_pages"].clone()
            qo = moda.moda_paged_append(q, x["k"], x["v"], kp, vp, x["table"], x["cu_q"], x["ctx"], rope=x["rope"])
            assert (qo is None) == (q is None)
            res.append([bits(kp), bits(vp)])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*res))
        assert moda.moda_device_status() == 0


def test_expired_wait_is_reported():
    """The bulk form's waits are bounded: with a cap of one poll some expire,
    the call's kernels end and the status word says so."""
    c = Paged("bulk", ((3000, 2900),), Hq=32, Hkv=4, rot=128)
    x = make(c, dev="cuda")
    torch.cuda.synchronize()
    moda.moda_debug_set_wait_limit(1)
    try:
        moda.moda_paged_append(x["q"], x["k"], x["v"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"],
                               rope=x["rope"])
        assert moda.moda_device_status() == 6
    finally:
        moda.moda_debug_set_wait_limit(0)
    assert moda.moda_device_status() == 0


def test_other_stream_and_graph():
    """On a side stream, and captured once and replayed after the inputs, the
    lengths and the table changed in place."""
    c = Paged("graph", ((40, 9), (25, 25)), Hq=8, Hkv=2, d=64, rot=64, cap=1)
    x, y = make(c, dev="cuda"), make(Paged("graph", ((40, 9), (25, 25)), Hq=8, Hkv=2, d=64, rot=64, cap=1, seed=9), dev="cuda")
    y["ctx"] = torch.tensor([31, 40], dtype=torch.int32, device="cuda")
    y["rope"], y["k_pages"], y["v_pages"] = x["rope"], x["k_pages"], x["v_pages"]

    def call(t, pages, stream=None, q_out=None):
        return moda.moda_paged_append(t["q"], t["k"], t["v"], *pages, t["table"], t["cu_q"], t["ctx"], rope=t["rope"],
                                      kd=t["kd"], vd=t["vd"], q_out=q_out, stream=stream)
    want = []
    for t in (x, y):
        pages = [t["k_pages"].clone(), t["v_pages"].clone()]
        want.append([bits(call(t, pages))] + [bits(p) for p in pages])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pages = [x["k_pages"].clone(), x["v_pages"].clone()]
    side.wait_stream(torch.cuda.current_stream())
    q = call(x, pages, stream=side, q_out=torch.empty_like(x["q"]))
    side.synchronize()
    assert all(torch.equal(bits(a), b) for a, b in zip([q] + pages, want[0]))
    buf = {n: t.clone() if torch.is_tensor(t) else t for n, t in x.items()}
    pages = [x["k_pages"].clone(), x["v_pages"].clone()]
    out = torch.empty_like(x["q"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(buf, pages, q_out=out)
    for t, w in ((x, want[0]), (y, want[1])):
        for n in ("q", "k", "v", "table", "cu_q", "ctx", "kd", "vd"):
            buf[n].copy_(t[n])
        pages[0].copy_(t["k_pages"])
        pages[1].copy_(t["v_pages"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), b) for a, b in zip([out] + pages, w))


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_pages_past_32_bits(q8):
    """The same rows arrive in pages whose elements lie 2^31 from the pool's start."""
    c = Paged("far", ((300, 200), (77, 1)), Hq=8, Hkv=1, rot=64, P=64)
    x = make(c, dev="cuda")
    n = x["k_pages"].shape[0]
    first = 2 ** 31 // (c.Hkv * c.P * c.d) - 3
    dt = torch.int8 if q8 else torch.bfloat16
    pools = []
    for pages in (n, first + n):
        kv = [torch.empty((pages, c.Hkv, c.P, c.d), dtype=dt, device="cuda") for _ in range(2)]
        sc = [torch.empty((pages, c.Hkv), device="cuda") for _ in range(2)] if q8 else []
        for t in kv + sc:
            t[-n:] = 0
        table = torch.where(x["table"] < 0, x["table"], x["table"] + (pages - n))
        f = moda.moda_paged_append_q8 if q8 else moda.moda_paged_append
        f(x["q"], x["k"], x["v"], *kv, *sc, table, x["cu_q"], x["ctx"], rope=x["rope"])
        pools.append(kv + sc)
    torch.cuda.synchronize()
    for near, far in zip(*pools):
        assert near.any() and torch.equal(near, far[first:])


def test_what_follows_finds_8bit_append_done():
    """Many queries beside few keys: the kernel after the call, in a stream and
    in a replayed graph, reads finished queries, codes and scales."""
    c = Paged("after", ((4100, 4096),), Hq=64, Hkv=1, rot=128, P=64)
    x = make(c, q8=True, dev="cuda")
    pools = [x[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")]
    src = [x[n].clone() for n in ("q", "k", "v")]
    out = torch.empty_like(x["q"])

    def call():
        moda.moda_paged_append_q8(*src, *pools, x["table"], x["cu_q"], x["ctx"], rope=x["rope"], q_out=out)
        return [t.clone() for t in (out, *pools)]

    wanted = []
    for f in (1, -2):
        for n, t in zip(("q", "k", "v"), src):
            t.copy_(x[n] * f)
        call()
        torch.cuda.synchronize()
        wanted.append([t.clone() for t in (out, *pools)])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for rep in range(6):
        f = rep % 2
        for n, t in zip(("q", "k", "v"), src):
            t.copy_(x[n] * (1, -2)[f])
        out.zero_()
        if rep < 4:
            graph.replay()
            seen = [t.clone() for t in got]
        else:
            seen = call()
        torch.cuda.synchronize()
        # (the page that holds earlier tokens keeps the larger scale of the two calls)
        assert torch.equal(bits(seen[0]), bits(wanted[f][0]))
        last = x["table"][0].long()[1:]
        for a, b in zip(seen[1:], wanted[f][1:]):
            assert torch.equal(bits(a[last]), bits(b[last]))
