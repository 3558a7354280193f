"""Float64 CPU oracle of the paged sequence cache (TEST INFRASTRUCTURE).

The same rules as ``moda_oracle``: imports nothing from the product, plain
loops over sequences, tokens and pages. B sequences' new tokens are rows
cu_q[b] .. cu_q[b+1]-1 of one packed axis; ctx_lens counts a sequence's tokens
with the new ones, so row i of sequence b sits at position
ctx_lens[b] - (cu_q[b+1] - i). Pages are [num_pages, Hkv, page_size, d].
"""
from __future__ import annotations

import numpy as np

from .moda_oracle import to_f64

__all__ = ["paged_positions", "rotate", "paged_append", "paged_append_q8", "paged_forward", "scale_for"]


def _ints(x):
    return [int(v) for v in (x.tolist() if hasattr(x, "tolist") else x)]


def _table(block_table):
    return [_ints(r) for r in block_table]


def paged_positions(cu_q, ctx_lens, N):
    """Per packed row: (sequence, position), or None for a row of no sequence."""
    cu, ctx = _ints(cu_q), _ints(ctx_lens)
    at = [None] * N
    for b in range(len(ctx)):
        for i in range(max(cu[b], 0), min(cu[b + 1], N)):
            at[i] = (b, ctx[b] - (cu[b + 1] - i))
    return at


def _page(table, b, pos, P, pages):
    blk = pos // P
    if pos < 0 or blk >= len(table[b]):
        return -1
    p = table[b][blk]
    return p if 0 <= p < pages else -1


def rotate(x, row, interleaved, dtype=np.float64):
    """x [H, d] rotated by one table row (cos | sin halves), each operation in ``dtype``."""
    x = np.array(x, dtype=dtype)
    if row is None:
        return x
    R = len(row)
    c, s = np.asarray(row[:R // 2], dtype=dtype), np.asarray(row[R // 2:], dtype=dtype)
    y = x.copy()
    for j in range(R // 2):
        f, g = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        y[:, f] = x[:, f] * c[j] - x[:, g] * s[j]
        y[:, g] = x[:, g] * c[j] + x[:, f] * s[j]
    return y


def _taken(at, rope):
    return at is not None and at[1] >= 0 and (rope is None or at[1] < len(rope))


def paged_append(q, k, v, k_pages, v_pages, block_table, cu_q, ctx_lens, rope=None, interleaved=False, kd=None,
                 vd=None, slot=0, q_out=None, dtype=np.float64):
    """The cache after the append: (q_out, k_pages, v_pages, kd, vd) as
    unrounded ``dtype`` arrays. ``q_out`` gives the rows no token writes."""
    q, k, v = (None if x is None else np.asarray(to_f64(x), dtype=dtype) for x in (q, k, v))
    kp, vp = np.array(to_f64(k_pages), dtype=dtype), np.array(to_f64(v_pages), dtype=dtype)
    kd, vd = (None if x is None else np.array(to_f64(x), dtype=dtype) for x in (kd, vd))
    qo = None if q is None else (np.array(to_f64(q_out), dtype=dtype) if q_out is not None else np.zeros_like(q))
    rp = None if rope is None else to_f64(rope)
    table, P = _table(block_table), kp.shape[2]
    for i, at in enumerate(paged_positions(cu_q, ctx_lens, k.shape[0])):
        if not _taken(at, rp):
            continue
        b, pos = at
        row = None if rp is None else rp[pos]
        ki = rotate(k[i], row, interleaved, dtype)
        if q is not None:
            qo[i] = rotate(q[i], row, interleaved, dtype)
        if kd is not None:
            kd[i, slot], vd[i, slot] = ki, v[i]
        page = _page(table, b, pos, P, kp.shape[0])
        if page >= 0:
            kp[page, :, pos % P], vp[page, :, pos % P] = ki, v[i]
    return qo, kp, vp, kd, vd


def scale_for(amax):
    """The smallest power of two 2^e, e >= -126, with amax <= 127 * 2^e (0 for 0)."""
    if not amax > 0:
        return 0.0
    e = -126
    while amax > 127 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def paged_append_q8(k, v, k_pages, v_pages, k_scale, v_scale, block_table, cu_q, ctx_lens, rope=None,
                    interleaved=False, dtype=np.float32):
    """(k_codes, v_codes, k_scale, v_scale) after the append. The rotation runs
    in ``dtype`` (the definition fixes fp32 there); the rest is exact."""
    out = []
    at = paged_positions(cu_q, ctx_lens, k.shape[0])
    rp = None if rope is None else to_f64(rope)
    table = _table(block_table)
    for x, codes, scale, turned in ((k, k_pages, k_scale, True), (v, v_pages, v_scale, False)):
        x, codes, scale = to_f64(x), np.array(to_f64(codes)), np.array(to_f64(scale))
        pages, Hkv, P, d = codes.shape
        runs = {}
        for i, a in enumerate(at):
            if not _taken(a, rp):
                continue
            page = _page(table, a[0], a[1], P, pages)
            if page >= 0:
                row = rp[a[1]] if turned and rp is not None else None
                runs.setdefault((a[0], a[1] // P, page), []).append(
                    (a[1] % P, rotate(x[i], row, interleaved, dtype).astype(np.float64)))
        for (_, _, page), rows in runs.items():
            first = min(r for r, _ in rows)
            for h in range(Hkv):
                vals = np.array([y[h] for _, y in rows])
                fin = np.where(np.isfinite(vals), np.abs(vals), 0.0)
                now = scale_for(fin.max())
                if first:
                    now = max(now, scale[page, h])
                    ratio = scale[page, h] / now if now > 0 else 0.0
                    codes[page, h, :first] = np.rint(codes[page, h, :first] * ratio)
                for r, y in rows:
                    with np.errstate(all="ignore"):
                        c = np.rint(y[h] / now) if now > 0 else np.zeros(d)
                    codes[page, h, r] = np.clip(np.where(np.isnan(c), 0.0, c), -127, 127)
                scale[page, h] = now
        out.append((codes, scale))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def paged_forward(q, k_pages, v_pages, block_table, cu_q, ctx_lens, kd, vd, Ld, scale, k_scale=None, v_scale=None):
    """(out [N,Hq,d], lse [N,Hq], absv, zabs): float64 results, NaN in rows of
    no sequence; absv = sum P |v| per output element and zabs = the largest
    scale * sum |q||k| of a row, the two sizes error bounds go by."""
    q, kp, vp = to_f64(q), to_f64(k_pages), to_f64(v_pages)
    if k_scale is not None:
        kp = kp * to_f64(k_scale)[:, :, None, None]
        vp = vp * to_f64(v_scale)[:, :, None, None]
    kd, vd = (None if Ld == 0 else to_f64(x) for x in (kd, vd))
    N, Hq, d = q.shape
    pages, Hkv, P, _ = kp.shape
    table = _table(block_table)
    out, absv = np.full((N, Hq, d), np.nan), np.full((N, Hq, d), np.nan)
    lse, zabs = np.full((N, Hq), np.nan), np.zeros((N, Hq))
    for i, at in enumerate(paged_positions(cu_q, ctx_lens, N)):
        if at is None:
            continue
        b, pos = at
        where = [(_page(table, b, j, P, pages), j % P) for j in range(pos + 1)]
        where = [w for w in where if w[0] >= 0]
        pg, rw = [w[0] for w in where], [w[1] for w in where]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            kk, vv = kp[pg, g, rw].reshape(-1, d), vp[pg, g, rw].reshape(-1, d)
            if Ld:
                kk, vv = np.concatenate([kk, kd[i, :Ld, g]]), np.concatenate([vv, vd[i, :Ld, g]])
            if not len(kk):
                out[i, h], absv[i, h], lse[i, h] = 0.0, 0.0, -np.inf
                continue
            z = kk @ q[i, h] * scale
            m = z.max()
            e = np.exp(z - m)
            p = e / e.sum()
            out[i, h], absv[i, h] = p @ vv, p @ np.abs(vv)
            lse[i, h] = m + np.log(e.sum())
            zabs[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, absv, zabs
