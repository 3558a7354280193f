"""GPU parity of the attention over the paged cache (moda_fwd_paged,
moda_fwd_paged_q8) with the float64 oracle, by bounds that follow from the
arithmetic (paged_util.check_rows). Everything a row must not see holds NaN."""
import pytest
import torch

import oracle
from paged_util import Paged, check_rows, make

pytestmark = pytest.mark.gpu

moda = pytest.importorskip("depth_kv_attention_b200")


def steps(*ctx):
    return tuple((c, 1) for c in ctx)


CASES = [
    Paged("one_key", steps(1)),
    Paged("one_key_depth", steps(1), Ld=3, cap=3),
    Paged("tails", steps(*range(1, 35)), Hq=4, Hkv=1, Ld=2, cap=5),
    Paged("mixed", steps(700, 3, 64, 65, 129, 1024, 333), Hq=32, Hkv=4, Ld=28, cap=28),
    Paged("long", steps(5000), Hq=8, Hkv=1, Ld=4, cap=4, P=64),
    Paged("g1", steps(100, 257), Hq=4, Hkv=4, Ld=5, cap=8),
    Paged("g7", steps(100, 257), Hq=14, Hkv=2, Ld=5, cap=5, P=48),
    Paged("g16", steps(90, 31), Hq=16, Hkv=1, P=32),
    Paged("g20", steps(90, 31), Hq=20, Hkv=1, P=32, Ld=17, cap=17),
    Paged("g32", steps(200, 77), Hq=32, Hkv=1, Ld=28, cap=33, P=32),
    Paged("g71", steps(100), Hq=71, Hkv=1, Ld=1, cap=1),
    Paged("d64", steps(130, 40), d=64, Ld=4, cap=4),
    Paged("d96", steps(130, 40), d=96, Ld=4, cap=4, P=128),
    Paged("d8", steps(130, 40), d=8, Hq=6, Hkv=2),
    Paged("d72", steps(130, 40), d=72, Hq=6, Hkv=2, Ld=9, cap=9),
    Paged("draft", ((300, 4), (65, 5), (20, 0), (130, 3)), Hq=8, Hkv=2, Ld=6, cap=6, spare_rows=2),
    Paged("draft_g32", ((300, 4), (64, 4)), Hq=32, Hkv=1, Ld=20, cap=28, P=32),
    Paged("chunk", ((200, 100), (130, 130), (64, 1)), Hq=8, Hkv=2, Ld=3, cap=3),
    Paged("chunk_g8", ((700, 300), (90, 33)), Hq=8, Hkv=1, Ld=16, cap=16, P=64),
    Paged("chunk_g1", ((300, 150),), Hq=2, Hkv=2, Ld=7, cap=7, d=128),
    Paged("chunk_g7", ((300, 90),), Hq=7, Hkv=1, Ld=2, cap=2, d=96),
    Paged("chunk_g5_d64", ((330, 70), (20, 20), (9, 0)), Hq=10, Hkv=2, Ld=5, cap=6, d=64, P=32),
    Paged("chunk_g3_d72", ((150, 150), (33, 32)), Hq=3, Hkv=1, Ld=17, cap=17, d=72, spare_rows=1),
    Paged("chunk_g71", ((60, 9), (130, 2)), Hq=71, Hkv=1, Ld=2, cap=2, P=128),
    Paged("chunk_g100_d8", ((40, 5),), Hq=100, Hkv=1, Ld=1, cap=1, d=8),
    Paged("chunk_g130", ((40, 3),), Hq=130, Hkv=1, d=64),
    Paged("chunk_many", tuple((20 + 7 * b, (5 * b) % 17) for b in range(40)), Hq=12, Hkv=2, Ld=3, cap=3),
    Paged("chunk_short_ctx", ((5, 70), (3, 40), (0, 30)), Hq=4, Hkv=1),
    Paged("chunk_short_depth", ((5, 70), (3, 40), (0, 30)), Hq=4, Hkv=1, Ld=4, cap=4),
    Paged("chunk_long_g33", ((2100, 11), (700, 3)), Hq=33, Hkv=1, Ld=20, cap=20, d=64, P=48),
    Paged("chunk_sees_nothing", ((0, 30), (5, 70), (300, 20)), Hq=4, Hkv=1, P=128),
    Paged("chunk_sees_nothing_g1", ((0, 50),), Hq=2, Hkv=2, P=64, d=64),
    Paged("rows33", ((900, 33), (1500, 9)), Hq=4, Hkv=4, Ld=4, cap=4, d=96),
    Paged("deep", steps(40), Hq=4, Hkv=1, Ld=130, cap=140),
    Paged("short_ctx", ((2, 5), (0, 1), (3, 3)), Hq=8, Hkv=2),
    Paged("short_ctx_depth", ((2, 5), (0, 1), (3, 3)), Hq=8, Hkv=2, Ld=3, cap=3),
    Paged("odd_page", steps(100, 33), P=24, Ld=2, cap=2),
    Paged("page1", steps(20, 7), P=1, d=16, Hq=2, Hkv=1),
    Paged("f32", ((128, 1), (70, 3), (300, 1)), Hq=4, Hkv=1, d=64, Ld=4, cap=4, dtype="f32"),
    Paged("f32_d72", ((50, 2), (9, 9)), Hq=6, Hkv=3, d=72, P=5, Ld=3, cap=4, dtype="f32"),
    Paged("f32_d128", steps(400, 1), Hq=8, Hkv=1, d=128, P=64, dtype="f32"),
    Paged("many", tuple((1 + b % 70, b % 3) for b in range(1100)), d=32, Hq=2, Hkv=1, Ld=1, cap=1),
]


def run(x, c, q8, impl="auto", **kw):
    if q8:
        return moda.moda_fwd_paged_q8(x["q"], x["k_pages"], x["v_pages"], x["k_scale"], x["v_scale"], x["table"],
                                      x["cu_q"], x["ctx"], x["max_q"], kd=x["kd"], vd=x["vd"], Ld=c.Ld, impl=impl, **kw)
    return moda.moda_fwd_paged(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], x["max_q"],
                               kd=x["kd"], vd=x["vd"], Ld=c.Ld, impl=impl, **kw)


def want(x, c):
    return oracle.paged_forward(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], x["kd"], x["vd"],
                                c.Ld, c.d ** -0.5, x.get("k_scale"), x.get("v_scale"))


def keys_of(c):
    return max(n for n, _ in c.seqs) + c.Ld


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


@pytest.mark.parametrize("impl", ["auto", "simt"])
@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
@pytest.mark.parametrize("c", CASES, ids=[c.name for c in CASES])
def test_parity(c, q8, impl):
    x = make(c, q8=q8)
    # rows behind the last sequence stay as they were
    out = torch.full((c.N, c.Hq, c.d), 9.0, dtype=x["q"].dtype, device="cuda")
    lse = torch.full((c.N, c.Hq), 9.0, device="cuda")
    got = run(cuda(x), c, q8, impl, out=out, lse=lse)
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    assert got[0] is out and got[1] is lse
    check_rows(out, lse, want(x, c), c.dtype, keys_of(c), c.d, c.name)
    n = c.N - c.spare_rows
    assert torch.all(out[n:] == 9) and torch.all(lse[n:] == 9)


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_long_chunks(q8):
    """Many key tiles per part; parts that end inside a unit and begin in the next."""
    c = Paged("chunk_long", ((3000, 300), (2500, 260)), Hq=16, Hkv=2, Ld=5, cap=5, P=64, d=96)
    x = make(c, q8=q8)
    got = run(cuda(x), c, q8)
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    check_rows(*got, want(x, c), c.dtype, keys_of(c), c.d)


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_peaked_logits(q8):
    """Queries of large norm: one key takes nearly all the weight, running
    maxima jump, and far keys underflow."""
    c = Paged("peak", ((600, 1), (200, 3)), Hq=16, Hkv=2, Ld=5, cap=5)
    x = make(c, q8=q8)
    x["q"] = x["q"] * 12
    got = run(cuda(x), c, q8)
    torch.cuda.synchronize()
    check_rows(*got, want(x, c), c.dtype, keys_of(c), c.d)


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_pages_that_are_not_there(q8):
    """Holes in the table (an id below 0 or past the pool, whole tiles of them
    too) and a table shorter than the context: those positions are not seen."""
    c = Paged("holes", ((400, 2), (300, 1), (500, 1)), Hq=8, Hkv=2, Ld=2, cap=2)
    x = make(c, q8=q8)
    x["table"][0, 3], x["table"][0, 24], x["table"][1, 0:16] = -1, 10 ** 6, -7
    x["table"][2, :] = -1
    x["table"] = x["table"][:, :28].contiguous()
    got = run(cuda(x), c, q8)
    torch.cuda.synchronize()
    check_rows(*got, want(x, c), c.dtype, keys_of(c), c.d)


def test_nan_where_a_row_does_not_look():
    """NaN and infinities in the values and keys of a later new token and in
    another token's depth rows reach only the rows that see them."""
    c = Paged("nan", ((70, 4),), Hq=8, Hkv=1, Ld=3, cap=3)
    x = make(c)
    clean = want(x, c)
    page, row = int(x["table"][0, 69 // 16]), 69 % 16   # the last token's key and value
    x["k_pages"][page, :, row], x["v_pages"][page, :, row] = float("nan"), float("inf")
    x["vd"][2, 1], x["kd"][2, 0] = float("nan"), float("inf")
    out, lse = run(cuda(x), c, False)
    torch.cuda.synchronize()
    ok = [0, 1]
    check_rows(out[ok], lse[ok], tuple(w[ok] for w in clean), c.dtype, keys_of(c), c.d)
    assert torch.isnan(out[2:]).all() and torch.isnan(lse[3]).all()


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
@pytest.mark.parametrize("G", [8, 7])
def test_nan_in_a_chunk(G, q8):
    """The same in a chunk of many rows, whose tiles of 128 keys are masked row
    by row: a non-finite value of a late token and of one token's depth rows
    reaches exactly the rows and features that see it."""
    c = Paged("nanchunk", ((300, 120), (90, 40)), Hq=G, Hkv=1, Ld=3, cap=3, d=96)
    x = make(c, q8=q8)
    clean = want(x, c)
    at = 250                                             # position of new token 70 of sequence 0
    if not q8:
        x["v_pages"][int(x["table"][0, at // 16]), :, at % 16, 5] = float("inf")
    x["vd"][33, 1, 0, 7] = float("nan")
    out, lse = run(cuda(x), c, q8)
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    hit = torch.zeros(c.N, G, c.d, dtype=torch.bool)
    if not q8:
        hit[70:120, :, 5] = True
        assert torch.isinf(out[70:120, :, 5]).all()
    hit[33, :, 7] = True
    assert torch.isnan(out[33, :, 7]).all()
    got = torch.where(hit.cuda(), torch.tensor(0.0, dtype=out.dtype, device="cuda"), out)
    o, l, a, z = clean
    o, a = o.copy(), a.copy()
    o[hit.numpy()], a[hit.numpy()] = 0.0, 1.0
    check_rows(got, lse, (o, l, a, z), c.dtype, keys_of(c), c.d)


@pytest.mark.parametrize("seqs", [((900, 1), (400, 1)), ((300, 90),)], ids=["steps", "chunk"])
def test_expired_waits_are_reported(seqs):
    """Every wait in the kernels is bounded: with a cap of one poll they give
    up, the call ends and the status word says so; the next call is sound."""
    c = Paged("limit", seqs, Hq=8, Hkv=1, Ld=2, cap=2)
    x = make(c)
    g = cuda(x)
    torch.cuda.synchronize()
    moda.moda_debug_set_wait_limit(1)
    try:
        run(g, c, False)
        assert moda.moda_device_status() == 6
    finally:
        moda.moda_debug_set_wait_limit(0)
    got = run(g, c, False)
    assert moda.moda_device_status() == 0
    check_rows(*got, want(x, c), c.dtype, keys_of(c), c.d)


@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scale_of_zero_and_below(scale):
    c = Paged("scale", ((60, 30), (33, 1)), Hq=8, Hkv=1, d=64)
    x = make(c)
    out, lse = moda.moda_fwd_paged(*(x[n].cuda() for n in ("q", "k_pages", "v_pages", "table", "cu_q", "ctx")), 30,
                                   scale=scale)
    torch.cuda.synchronize()
    w = oracle.paged_forward(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], None, None, 0, scale)
    check_rows(out, lse, w, c.dtype, keys_of(c), c.d)


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_twice_the_same_and_shared_workspace(q8):
    """The same call twice gives the same bits, also through a workspace that
    holds NaN; two captured graphs that share it replay one after the other."""
    c = Paged("again", ((3000, 1), (1500, 2), (10, 1)), Hq=32, Hkv=4, Ld=6, cap=6)
    x = cuda(make(c, q8=q8))
    n = moda.moda_fwd_paged_workspace_bytes(c.N, len(c.seqs), x["max_q"], c.Hq, c.Hkv, c.d,
                                            x["k_pages"].shape[0], c.P, torch.bfloat16, q8)
    ws = torch.full((max(n, 16) // 4,), float("nan"), device="cuda").view(torch.uint8)
    a = run(x, c, q8)
    b = run(x, c, q8, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    y = dict(x, q=x["q"] * 2)
    wanted = [a, run(y, c, q8)]
    graphs, outs = [], []
    for t in (x, y):
        outs.append([torch.empty_like(a[0]), torch.empty_like(a[1])])
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            run(t, c, q8, workspace=ws, out=outs[-1][0], lse=outs[-1][1])
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, wanted):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_graph_follows_the_lengths():
    """A captured decode step serves later steps: only device arrays change."""
    c = Paged("replay", ((200, 1), (90, 1)), Hq=8, Hkv=1, Ld=2, cap=2)
    x = make(c)
    x["k_pages"], x["v_pages"] = torch.nan_to_num(x["k_pages"], nan=0.5), torch.nan_to_num(x["v_pages"], nan=0.5)
    g = cuda(x)
    out, lse = torch.empty_like(g["q"]), torch.empty((c.N, c.Hq), device="cuda")
    run(g, c, False, out=out, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(g, c, False, out=out, lse=lse)
    for ctx in ((200, 90), (201, 1), (16, 96), (0, 33)):
        x["ctx"] = torch.tensor(ctx, dtype=torch.int32)
        g["ctx"].copy_(x["ctx"])
        graph.replay()
        torch.cuda.synchronize()
        check_rows(out, lse, want(x, c), c.dtype, keys_of(c), c.d, str(ctx))


def test_other_stream():
    c = Paged("stream", ((900, 1), (90, 1)), Hq=32, Hkv=4, Ld=2, cap=2)
    x = cuda(make(c))
    a = run(x, c, False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = run(x, c, False, stream=side, out=torch.empty_like(x["q"]))
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_max_q_is_a_hint():
    """Any max_q gives the oracle's rows (it only selects the kernel)."""
    c = Paged("hint", ((150, 40), (33, 1)), Hq=8, Hkv=1, Ld=2, cap=2)
    x = make(c)
    w = want(x, c)
    for m in (1, 3, 17, 1000):
        got = run(dict(cuda(x), max_q=m), c, False)
        torch.cuda.synchronize()
        check_rows(*got, w, c.dtype, keys_of(c), c.d, str(m))


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_layers_of_steps(q8):
    """As they are used together: per step and layer append (rotated, and into
    the layer's depth slot), then attend to the cache and the slots of the
    layers before; prompts first, then single tokens. Every attention call
    matches the oracle on the cache that the calls before it left."""
    Hq, Hkv, d, P, layers = 8, 2, 64, 16, 3
    g = torch.Generator("cpu")
    g.manual_seed(5)
    pages = 12
    table = torch.randperm(pages, generator=g)[:8].view(2, 4).to(torch.int32).cuda()
    f = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    a = torch.arange(64, dtype=torch.float64)[:, None] * f
    rope = torch.cat([a.cos(), a.sin()], 1).float().cuda()
    kv = torch.int8 if q8 else torch.bfloat16
    cache = [[torch.zeros(pages, Hkv, P, d, dtype=kv, device="cuda") for _ in range(2)] for _ in range(layers)]
    scale = [[torch.zeros(pages, Hkv, device="cuda") for _ in range(2)] for _ in range(layers)]
    ctx = [0, 0]
    for new in ((21, 14), (1, 1), (1, 1), (2, 0), (1, 3)):
        N = sum(new)
        ctx = [c + n for c, n in zip(ctx, new)]
        cu = torch.tensor([0, new[0], N], dtype=torch.int32).cuda()
        lens = torch.tensor(ctx, dtype=torch.int32).cuda()
        kd = torch.full((N, layers, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        vd = kd.clone()
        for layer in range(layers):
            q, k, v = (torch.randn(N, h, d, generator=g).to(torch.bfloat16).cuda() for h in (Hq, Hkv, Hkv))
            pg, sc = cache[layer], scale[layer]
            kw = dict(rope=rope, kd=kd, vd=vd, slot=layer)
            if q8:
                qr = moda.moda_paged_append_q8(q, k, v, *pg, *sc, table, cu, lens, **kw)
                out, lse = moda.moda_fwd_paged_q8(qr, *pg, *sc, table, cu, lens, max(new), kd=kd, vd=vd, Ld=layer)
            else:
                qr = moda.moda_paged_append(q, k, v, *pg, table, cu, lens, **kw)
                out, lse = moda.moda_fwd_paged(qr, *pg, table, cu, lens, max(new), kd=kd, vd=vd, Ld=layer)
            torch.cuda.synchronize()
            w = oracle.paged_forward(qr, *pg, table.cpu(), cu.cpu(), lens.cpu(), kd, vd, layer, d ** -0.5,
                                     *(sc if q8 else (None, None)))
            check_rows(out, lse, w, "bf16", max(ctx) + layer, d)
            turned = oracle.rotate(k[0].double().cpu().numpy(), rope[ctx[0] - new[0]].double().cpu().numpy(), False)
            assert abs(kd[0, layer].double().cpu().numpy() - turned).max() <= 2.0 ** -8 * abs(turned).max() + 1e-5


@pytest.mark.parametrize("new", [1, 40], ids=["step", "chunk"])
@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_sequences_with_a_common_beginning(q8, new):
    """Pages that stand in several tables, and twice in one."""
    c = Paged("prefix", ((200, new), (170, new), (96, new)), Hq=8, Hkv=2, Ld=2, cap=2, P=16)
    x = make(c, q8=q8)
    x["table"][1, :6] = x["table"][0, :6]
    x["table"][2, :3] = x["table"][0, 3:6]
    x["table"][2, 3:6] = x["table"][0, 3:6]
    got = run(cuda(x), c, q8)
    torch.cuda.synchronize()
    check_rows(*got, want(x, c), c.dtype, keys_of(c), c.d)


@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
def test_two_streams_at_once(q8):
    """Steps and chunks side by side on two streams, each with what it allocates."""
    calls = []
    for seqs in (((3000, 1), (1500, 2), (10, 1)), ((1200, 300), (90, 64))):
        c = Paged("side", seqs, Hq=32, Hkv=4, Ld=6, cap=6)
        calls.append((c, cuda(make(c, q8=q8))))
    alone = [run(x, c, q8) for c, x in calls]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(20):
        for i, (c, x) in enumerate(calls):
            got[i].append(run(x, c, q8, stream=side[i]))
    torch.cuda.synchronize()
    assert moda.moda_device_status() == 0
    for a, g in zip(alone, got):
        for o, l in g:
            assert torch.equal(o, a[0]) and torch.equal(l, a[1])


@pytest.mark.parametrize("impl", ["auto", "simt"])
@pytest.mark.parametrize("q8", [False, True], ids=["kv16", "kv8"])
@pytest.mark.parametrize("new", [1, 40], ids=["step", "chunk"])
def test_pages_past_32_bits(new, q8, impl):
    """Pages whose elements lie 2^31 and more from the pool's start."""
    c = Paged("far", ((300, new), (77, new)), Hq=8, Hkv=1, Ld=2, cap=2, P=64)
    x = make(c, q8=q8)
    n = x["k_pages"].shape[0]
    first = 2 ** 31 // (c.Hkv * c.P * c.d) - 3   # of n pages that lie across the mark
    far = cuda(x)
    for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
        if name in far:
            pool = torch.empty((first + n, *x[name].shape[1:]), dtype=x[name].dtype, device="cuda")
            pool[first:] = far[name]
            far[name] = pool
    far["table"] = torch.where(far["table"] < 0, far["table"], far["table"] + first)
    got = run(far, c, q8, impl)
    torch.cuda.synchronize()
    check_rows(*got, want(x, c), c.dtype, keys_of(c), c.d)
