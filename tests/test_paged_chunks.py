"""GPU tests of the paged attention's documented properties for chunks as well
as steps, on both page types: captured calls follow the device arrays, any
max_q gives the same rows, and a shared workspace carries nothing over."""
import pytest
import torch

import oracle
from paged_util import Paged, check_rows, make

pytestmark = pytest.mark.gpu

moda = pytest.importorskip("depth_kv_attention_b200")

KINDS = ["kv16", "kv8"]


def padded(c, q8, N, pages, width):
    """The tensors of `c` in buffers of given sizes: packed rows behind the last
    sequence, pages that no table names, table entries that name no page."""
    x = make(c, q8=q8)
    n, more = c.N, pages - x["k_pages"].shape[0]

    def grow(t, k, fill):
        return torch.cat([t, torch.full((k, *t.shape[1:]), fill, dtype=t.dtype)])

    for name in ("k_pages", "v_pages"):
        x[name] = grow(x[name], more, 99 if q8 else float("nan"))
    for name in ("k_scale", "v_scale") if q8 else ():
        x[name] = grow(x[name], more, float("nan"))
    for name in ("q", "kd", "vd"):
        x[name] = grow(x[name], N - n, 0.5)
    t = torch.full((x["table"].shape[0], width), -1, dtype=torch.int32)
    t[:, :x["table"].shape[1]] = x["table"]
    x["table"] = t
    return x


def run(x, Ld, q8, max_q, **kw):
    a = [x["q"], x["k_pages"], x["v_pages"]] + ([x["k_scale"], x["v_scale"]] if q8 else [])
    fn = moda.moda_fwd_paged_q8 if q8 else moda.moda_fwd_paged
    return fn(*a, x["table"], x["cu_q"], x["ctx"], max_q, kd=x["kd"], vd=x["vd"], Ld=Ld, **kw)


def check(got, x, Ld, q8, d, keys, what=""):
    w = oracle.paged_forward(x["q"], x["k_pages"], x["v_pages"], x["table"], x["cu_q"], x["ctx"], x["kd"], x["vd"], Ld,
                             d ** -0.5, x.get("k_scale"), x.get("v_scale"))
    check_rows(*got, w, "bf16", keys, d, what)


def cuda(x):
    return {n: t.cuda() if torch.is_tensor(t) else t for n, t in x.items()}


@pytest.mark.parametrize("q8", [False, True], ids=KINDS)
@pytest.mark.parametrize("pages,width", [(60, 30), (400, 30)], ids=["small_pool", "large_pool"])
@pytest.mark.parametrize("max_q", [1, 60], ids=["step", "chunk"])
def test_replay_follows_the_arrays(q8, pages, width, max_q):
    """One captured call serves batches of other lengths, tables, cache contents
    and numbers of new tokens, from a workspace of NaN each time."""
    G, Ld, d = 8, 3, 64
    batches = [((200, 60), (90, 20), (33, 1)), ((201, 1), (400, 40), (5, 5)), ((16, 16), (96, 0), (480, 64)),
               ((0, 7), (3, 40), (300, 33)), ((200, 60), (90, 20), (33, 1)), ((130, 1), (131, 1), (132, 1))]
    N = 90
    cases = [Paged(f"r{i}", b, Hq=2 * G, Hkv=2, d=d, Ld=Ld, cap=4, seed=i + 1) for i, b in enumerate(batches)]
    x = padded(cases[0], q8, N, pages, width)
    g = cuda(x)
    n = moda.moda_fwd_paged_workspace_bytes(N, 3, max_q, 2 * G, 2, d, pages, 16, torch.bfloat16, q8)
    ws = torch.empty(n // 4, device="cuda")
    out, lse = torch.empty_like(g["q"]), torch.empty((N, 2 * G), device="cuda")
    kw = dict(workspace=ws, out=out, lse=lse)
    run(g, Ld, q8, max_q, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(g, Ld, q8, max_q, **kw)
    for c in cases:
        x = padded(c, q8, N, pages, width)
        for name, t in x.items():
            if torch.is_tensor(t) and name not in ("k", "v"):
                g[name].copy_(t)
        ws.fill_(float("nan"))
        out.fill_(9.0)
        lse.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert moda.moda_device_status() == 0
        check((out, lse), x, Ld, q8, d, 500, c.name)
        assert torch.all(out[c.N:] == 9) and torch.all(lse[c.N:] == 9)


@pytest.mark.parametrize("q8", [False, True], ids=KINDS)
@pytest.mark.parametrize("seqs", [((150, 40), (33, 1)), ((700, 130), (90, 1), (257, 3), (20, 0))], ids=["two", "four"])
def test_any_max_q(q8, seqs):
    c = Paged("hint", seqs, Hq=16, Hkv=2, Ld=2, cap=2)
    x = make(c, q8=q8)
    g = cuda(x)
    for m in (1, 2, 3, 5, 17, 1000):
        got = run(g, 2, q8, m)
        torch.cuda.synchronize()
        assert moda.moda_device_status() == 0
        check(got, x, 2, q8, c.d, 800, str(m))


def test_a_shared_workspace_carries_nothing_over():
    """Chunks and steps over both page types, of other sizes and pools, through
    one workspace: each gives what it gives with its own."""
    calls = []
    for i, (q8, seqs, d) in enumerate([(True, ((300, 70), (90, 40)), 128), (False, ((500, 100),), 128),
                                       (True, ((700, 1), (90, 1)), 64), (True, ((260, 200), (40, 40), (33, 1)), 128)]):
        c = Paged(f"ws{i}", seqs, Hq=8, Hkv=1, d=d, Ld=2, cap=2, seed=i + 1)
        calls.append((c, q8, cuda(make(c, q8=q8))))
    need = max(moda.moda_fwd_paged_workspace_bytes(c.N, len(c.seqs), x["max_q"], 8, 1, c.d, x["k_pages"].shape[0], c.P,
                                                   torch.bfloat16, q8) for c, q8, x in calls)
    ws = torch.full((need // 4 + 4,), float("nan"), device="cuda")
    own = [run(x, 2, q8, x["max_q"]) for c, q8, x in calls]
    for i in (0, 1, 3, 2, 0, 3, 1, 0):
        c, q8, x = calls[i]
        out, lse = run(x, 2, q8, x["max_q"], workspace=ws)
        assert torch.equal(out, own[i][0]) and torch.equal(lse, own[i][1]), i
