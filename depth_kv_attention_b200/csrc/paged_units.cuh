// Work units of the paged attention and their distribution over CTAs.
//
// A unit is (sequence, kv-head, tile of MR rows); a row is a (token, head of
// the group) pair of the sequence, flattened token-major, so every row of a
// tile reads the same K and V. A unit's keys come in stages: KEYS sequence keys
// each, then depth stages of DS slices of 16 slots of one token. All units'
// stages form one list (sequence-major, then kv-head, then tile) that the
// CTAs cut into equal parts, so a ragged batch loads every SM alike, whatever
// its lengths; a unit that is cut is joined from its parts afterwards. The
// lengths are known on the device only: every CTA scans them itself.
#pragma once

#include <cstdint>

#include "paged_common.cuh"

namespace moda {

// First element of part x of W equal parts of [0, total): floor(total x / W),
// in 32 bits where they hold it (a 64-bit division costs ten times as much).
__device__ __forceinline__ long long part_begin(long long total, int x, int W) {
    if (total < (1LL << 31)) {
        const uint32_t t = (uint32_t)total, q = t / (uint32_t)W, r = t - q * W;
        return (long long)q * x + r * (uint32_t)x / (uint32_t)W;  // r x < W^2
    }
    return total * x / W;
}

struct SeqInfo {
    int q0, n;  // packed rows q0 .. q0+n-1
    int pos0;   // position of the first
};

__device__ __forceinline__ SeqInfo seq_info(const PagedCache& c, int b) {
    SeqInfo s;
    const int lo = __ldg(c.cu_q + b), hi = __ldg(c.cu_q + b + 1);
    s.q0 = min(max(lo, 0), c.N);
    s.n = max(min(hi, c.N) - s.q0, 0);
    const long long pos = (long long)__ldg(c.ctx_lens + b) - ((long long)hi - s.q0);
    s.pos0 = (int)max(pos, -(1LL << 30));
    return s;
}

struct UnitShape {
    int r0, rows;      // rows of the sequence in this tile
    int tok0, ntok;    // tokens they belong to
    int nk;            // sequence keys the last token sees
    int st_seq, st;    // sequence stages, all stages (at least one)
};

// Tile rt of MR rows of a sequence with n tokens. DSL: 16-slot slices of one
// token's depth rows; DS: slices per depth stage; max_keys: what the block
// table can hold.
template <int MR, int KEYS>
__device__ __forceinline__ UnitShape unit_shape(const SeqInfo& s, int rt, int G, int DSL, int DS, long long max_keys) {
    UnitShape u;
    u.r0 = rt * MR;
    u.rows = min(MR, s.n * G - u.r0);
    u.tok0 = u.r0 / G;
    u.ntok = (u.r0 + u.rows - 1) / G - u.tok0 + 1;
    const long long last = (long long)s.pos0 + u.tok0 + u.ntok;  // position of the last token + 1
    u.nk = (int)max(0LL, min(last, max_keys));
    u.st_seq = (u.nk + KEYS - 1) / KEYS;
    u.st = max(u.st_seq + (u.ntok * DSL + DS - 1) / DS, 1);
    return u;
}

template <int MR, int KEYS>
__device__ __forceinline__ long long seq_stages(const SeqInfo& s, int G, int DSL, int DS, long long max_keys) {
    long long t = 0;
    const int tiles = (s.n * G + MR - 1) / MR;
    for (int rt = 0; rt < tiles; ++rt) t += unit_shape<MR, KEYS>(s, rt, G, DSL, DS, max_keys).st;
    return t;
}

}  // namespace moda
