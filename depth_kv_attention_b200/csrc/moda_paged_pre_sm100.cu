// Attention over the paged sequence cache for many query rows per sequence
// (chunks of prompts, wide drafts), on tcgen05. bf16 pages; 8-bit ones
// are turned into bf16 once, ahead of it (see the end of the file).
//
// What it computes: as moda_paged_dec_sm100.cu, one softmax over the sequence
// keys a new token sees and its own depth keys ("动态混合深度注意力机制MoDA技术解析",
// mhpn.cn, §1.2 formula, §2.2 online-softmax state and dual mask).
//
// How: the tile machinery of the dense forward (moda_fwd_sm100.cu): two
// 128-row query tiles of 2n = 2 * 128/G tokens and one kv-head, S and O in
// TMEM, softmax one thread per row, the two tiles' MMAs and softmaxes
// alternating; one MMA thread, one TMA warp, a five-slot ring of 128-key K and
// V tiles. What differs:
//  * A key tile is eight slices of 16 rows, each from its own page (TMA boxes;
//    page ids fetched 32 slices at a time, a batch ahead). Depth tiles are
//    eight slices of 16 slots of one token.
//  * The items of all units form one list that the CTAs (one per SM) cut into
//    equal parts (paged_units.cuh): chunks are ragged and a few units rarely
//    fill the GPU evenly. Roles run from piece to piece; a unit that is cut
//    leaves (m, l, O) in the workspace for the join.
//  * Value tiles in which some row is masked pass through two conditioning
//    warps, which clear their non-finite elements (a masked P is 0, and 0 * NaN
//    is not); rows that do see one get it added back when the piece ends.
//  * Code is kept small where a piece begins and ends: with short sequences the
//    roles of 12 warps together miss the instruction cache all the time, and
//    each piece of unrolled code cost more than it saved. For the same reason
//    nothing spills: shared memory leaves the L1 cache almost no room.
//
// What bounds it: the products, while a unit is long (1024 tokens over 16K,
// G = 8: 423 us, 65 % of the cuBLAS rate; a tile's softmax, 1 us an item, and
// its own products alternate, so the two tiles together fill about 70 %). A
// piece costs about 6 us besides: queries, first products, the last tile's
// values and the epilogue follow each other (216-token sequences: 184 us for 42
// us of products; one 2048-token prompt 98 for 21).
//  * Every mbarrier wait is bounded, as in the dense forward.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "depth_mask.cuh"
#include "fwd_softmax.cuh"
#include "paged_join.cuh"
#include "paged_ptx.cuh"
#include "paged_units.cuh"
#include "tmap_host.h"

namespace moda {
namespace {

constexpr int kD = 128;         // features of a tile; rows of fewer are padded with zeros by TMA
constexpr int kTileBytes = 128 * kD * 2;
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kRows = 256;      // rows of a unit: two tiles
constexpr int kItemKeys = 128;
constexpr int kSlices = 8;      // 16-row slices of an item
constexpr int kParts = 148;     // one CTA per SM
constexpr int kMeta = 8;        // items whose slice notes are kept (the rings hold fewer than 5)
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kPieces = 8;      // pieces described at a time
constexpr int kPieceUsers = 11; // warps that read a piece: softmax 8, MMA, conditioning 2
constexpr uint32_t kNoPollLimit = 0;

struct PreParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_kd, tm_vd;
    PagedCache c;
    const __nv_bfloat16* v_pages;  // values, read again only for rows that see
    const __nv_bfloat16* vd;       // a non-finite one
    __nv_bfloat16* out;
    float* lse;
    float* part_o;
    float* part_ml;
    int4* desc;
    int Hq, G, n, Ld, Ld_cap, DSL;  // a tile has n tokens, n * G of its 128 rows
    int lg_step;                    // 2n = 1 << lg_step <= 128, or -1
    int box_rows;  // rows of a page box: the largest power of two that divides the page size, at most 128
    float sl2;
    unsigned int* status;
    unsigned int wait_limit;
};

// Warpgroups 0, 1: softmax of tiles 0, 1. Warps 8, 9: producer, MMA; 10, 11
// condition. Registers at launch and after reallocation:
// 384 x 168 = 256 x 200 + 128 x 104. (With 216 and 72 the control warps spilled:
// 1024 tokens over 16K 473 us, with these 455.)
constexpr int kThreads = 384;
constexpr int kCondFirst = 10;
constexpr int kCond = 64;        // conditioning threads
constexpr int kSoftmaxRegs = 200;
constexpr int kControlRegs = 104;
constexpr int kStages = 5;

struct __align__(8) PreBars {
    uint64_t q_full[2], q_empty[2];
    uint64_t full[kStages], empty[kStages];
    uint64_t raw_full[kStages];      // a value tile that is to be conditioned has landed
    uint64_t s_full[2], p_full[2], o_final[2], o_empty[2];
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t drain;
    uint32_t holes[kMeta];           // per item: slices without a page
    int bad_piece[kMeta];            // last piece that met a non-finite value a row may see
    long long scan[16];
    long long total, hi;             // items in all, end of this CTA's part
    int W;                           // parts
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kCtl = 2048;
constexpr int kSmemBytes = (2 + kStages) * kTileBytes + kCtl + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

__device__ __forceinline__ void flag_timeout(PreParams const& p, PreBars* bars) {
    *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    atomicOr(p.status, 1u);
}

// A unit: tokens tok0 .. tok0 + ntok - 1 of a sequence (tile i: n of them). Its
// depth chunks (128 rows: eight slices) belong to one tile each, but for one
// that both may share. Where none is shared they come in turns, tile 0's, tile
// 1's, tile 0's .. : while one tile's softmax runs the other's next product can.
struct Unit {
    int tok0, ntok;
    int nk;                 // sequence keys its last token sees
    int n_seq, n_items;
    int nkv0, nkv1;         // sequence items tile 0 / 1 takes part in
    int pairs;              // leading pairs of depth items in turns
    int c0_end, c1_begin, chunks;  // chunks of tile 0: [0, c0_end), of tile 1: [c1_begin, chunks)
    // depth chunk of item n_seq + e, and back
    __device__ __forceinline__ int chunk(int e) const {
        return e < 2 * pairs ? (e & 1 ? c1_begin : 0) + (e >> 1) : e - pairs;
    }
    __device__ __forceinline__ int item_of(int c) const {
        if (pairs == 0) return n_seq + c;
        return n_seq + (c >= c1_begin ? 2 * (c - c1_begin) + 1 : c < pairs ? 2 * c : c + pairs);
    }
    __device__ __forceinline__ bool part(int i, int x) const {
        if (x < n_seq) return x < (i ? nkv1 : nkv0);
        const int c = chunk(x - n_seq);
        return i ? c >= c1_begin && c < chunks : c < c0_end;
    }
};

__device__ __forceinline__ int keys_seen(const SeqInfo& s, int tok, long long max_keys) {
    return (int)max(0LL, min((long long)s.pos0 + tok + 1, max_keys));
}

__device__ __forceinline__ Unit make_unit(const PreParams& p, const SeqInfo& s, int rt, long long max_keys) {
    Unit u;
    const int n = p.n;
    u.tok0 = rt * 2 * n;
    u.ntok = min(2 * n, s.n - u.tok0);
    const int nv0 = min(n, u.ntok), nv1 = u.ntok - nv0;
    u.nk = keys_seen(s, u.tok0 + u.ntok - 1, max_keys);
    u.n_seq = (u.nk + kItemKeys - 1) / kItemKeys;
    u.nkv0 = (keys_seen(s, u.tok0 + nv0 - 1, max_keys) + kItemKeys - 1) / kItemKeys;
    u.nkv1 = nv1 ? u.n_seq : 0;
    const int dep0 = nv0 * p.DSL, dep = u.ntok * p.DSL;  // slices
    const int chunks = u.chunks = (dep + kSlices - 1) / kSlices;
    u.c0_end = (dep0 + kSlices - 1) / kSlices;
    u.c1_begin = nv1 ? dep0 / kSlices : chunks;
    u.pairs = u.c0_end == u.c1_begin ? chunks - u.c1_begin : 0;  // (tile 1 never has more than tile 0)
    u.n_items = max(u.n_seq + chunks, 1);
    return u;
}

// Sum of floor((a i + b) / m) over i < n, by Euclid's algorithm on (a, m).
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
    long long t = 0;
    for (;;) {
        t += (n - 1) * n / 2 * (a / m) + n * (b / m);
        a %= m;
        b %= m;
        const long long y = a * n + b;
        if (y < m) return t;
        n = y / m;
        b = y % m;
        const long long x = m;
        m = a;
        a = x;
    }
}
// Items of the sequence's first `tiles` units. Unit rt sees
// min(pos0 + 2n (rt + 1), pos0 + n_tokens) keys; where no unit is clipped by
// position 0 or by the table, ceil(keys / 128) over the whole units is a sum of
// floors, so it needs no loop over them. With 2n a power of two that divides
// 128 the floors are those of t / m, m = 128 / 2n, over consecutive t.
__device__ __forceinline__ long long items_before(const PreParams& p, const SeqInfo& s, int tiles, long long max_keys) {
    const int step = 2 * p.n;
    const long long last = (long long)s.pos0 + s.n;
    if (s.pos0 < 0 || last > max_keys) {
        long long t = 0;
        for (int rt = 0; rt < tiles; ++rt) t += make_unit(p, s, rt, max_keys).n_items;
        return t;
    }
    const int whole = min(tiles, p.lg_step >= 0 ? s.n >> p.lg_step : s.n / step);
    long long t;
    if (p.lg_step >= 0) {
        const int lg_m = 7 - p.lg_step, m = 1 << lg_m;
        const int q = (int)(((long long)s.pos0 + step + kItemKeys - 1) >> p.lg_step);  // ceil(K / 128) = floor((q + rt) / m)
        auto f = [&](int x) {                                                          // sum of floor(t / m), t < x
            const long long k = x >> lg_m;
            return ((k * (k - 1) / 2) << lg_m) + k * (x & (m - 1));
        };
        t = f(q + whole) - f(q);
    } else {
        t = whole ? floor_sum(whole, kItemKeys, step, (long long)s.pos0 + step + kItemKeys - 1) : 0;
    }
    t += (long long)whole * ((step * p.DSL + kSlices - 1) / kSlices);
    if (tiles > whole) t += make_unit(p, s, whole, max_keys).n_items;
    return t;
}
__device__ __forceinline__ long long seq_items(const PreParams& p, const SeqInfo& s, long long max_keys) {
    return items_before(p, s, (s.n + 2 * p.n - 1) / (2 * p.n), max_keys);
}
__device__ __forceinline__ long long table_keys(const PagedCache& c) {
    return min((long long)c.max_blocks * c.page_size, 0x7fffff00LL);
}

// A piece of this CTA's part: items [first, end) of a unit. The producer, which
// is ahead of the others, walks from piece to piece and describes each in a
// ring of them; walking takes about as long as half an item.
struct Piece {
    int b, kvh, rt, first, end, left;  // left: items of the part from here on
    SeqInfo sq;
    Unit u;
    __device__ __forceinline__ void shape(const PreParams& p) {
        u = make_unit(p, sq, rt, table_keys(p.c));
        end = min(u.n_items, first + left);
    }
    __device__ __forceinline__ bool next(const PreParams& p) {  // false: the part is done
        left -= end - first;
        if (left <= 0) return false;
        first = 0;
        if (++rt * 2 * p.n >= sq.n) {
            rt = 0;
            if (++kvh == p.c.Hkv) {
                kvh = 0;
                do {
                    sq = seq_info(p.c, ++b);
                } while (sq.n == 0 && b + 1 < p.c.B);
            }
        }
        shape(p);
        return true;
    }
};

static_assert(sizeof(PreBars) + kPieces * sizeof(Piece) <= kCtl && sizeof(PreBars) % 8 == 0, "control block");

// softmax_item for an item of which the row sees columns [lo, hi) less those
// in `holes` (bit k: columns 16 k ..). In chunks of 32 columns, read twice, in
// rolled loops: items like this are a few per unit, and the unrolled code of
// 128 masked columns (26 KB of it) pushed everything else out of the
// instruction cache wherever units are short.
__device__ __forceinline__ void softmax_masked(uint32_t tS, uint32_t tO, int lo, int hi, uint32_t holes, float sl2, int it,
                                               float& m, float& l) {
    // (chunks no row of the warp sees are skipped: of a depth item the 32 / G
    // tokens of a warp see a part, of a diagonal one the first columns)
    auto load = [&](int c, float (&s)[32]) {
        const int a = min(max(lo - 32 * c, 0), 32), e = min(max(hi - 32 * c, 0), 32);  // columns [a, e) of the chunk
        uint32_t vis = (e >= 32 ? 0xffffffffu : (1u << e) - 1u) & ~(a >= 32 ? 0xffffffffu : (1u << a) - 1u);
        if ((holes >> (2 * c)) & 1) vis &= 0xffff0000u;
        if ((holes >> (2 * c + 1)) & 1) vis &= 0x0000ffffu;
        if (!__any_sync(0xffffffffu, vis != 0)) return false;
        uint32_t su[32];
        ptx::tmem_ld32(tS + c * 32, su);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = (vis >> k) & 1 ? __uint_as_float(su[k]) : -INFINITY;
        return true;
    };
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        float s[32];
        if (!load(c, s)) continue;
#pragma unroll
        for (int k = 0; k < 32; ++k) mx = fmaxf(mx, s[k]);
    }
    const float mxs = mx * sl2;
    if (__any_sync(0xffffffffu, mxs > m + kRescaleThreshold)) {
        const float mnew = fmaxf(m, mxs);
        const float corr = (mnew == -INFINITY) ? 1.f : ptx::ex2(m - mnew);
        if (it > 0) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                ptx::tmem_ld32(tO + c * 32, o);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                ptx::tmem_st32(tO + c * 32, o);
            }
        }
        l *= corr;
        m = mnew;
    }
    const float ref = (m == -INFINITY) ? 0.f : m;
    float acc = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        float s[32];
        uint32_t pk[16] = {};
        if (load(c, s)) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float p0 = ptx::ex2(fmaf(s[2 * k], sl2, -ref)), p1 = ptx::ex2(fmaf(s[2 * k + 1], sl2, -ref));
                acc += p0 + p1;
                pk[k] = ptx::pack_bf16x2(p0, p1);
            }
        }
        ptx::tmem_st16(tS + c * 16, pk);  // over columns whose S has been read
    }
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    l += acc;
}

// Sets the non-finite elements of a bf16 value tile to 0. Returns whether this
// thread met one in a row below `rows` (rows past it nobody sees). The usual
// tile has none: 0 * x summed over everything is NaN exactly when one is there.
__device__ __forceinline__ bool clear_nonfinite(uint8_t* slot, int ct, int rows, int halves) {
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
    __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 8
    for (int ch = ct; ch < halves * (kHalfBytes / 16); ch += kCond) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot + ch * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            __nv_bfloat162 x;
            memcpy(&x, &w[e], 4);
            acc[e] = __hfma2(x, zero, acc[e]);
        }
    }
    const __nv_bfloat162 sum = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
    const float2 f = __bfloat1622float2(sum);
    if (f.x == 0.f && f.y == 0.f) return false;
    bool met = false;
    for (int ch = ct; ch < halves * (kHalfBytes / 16); ch += kCond) {
        uint4* at = reinterpret_cast<uint4*>(slot + ch * 16);
        const uint4 v = *at;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        bool any = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if ((w[e] & 0x7f80u) == 0x7f80u) { w[e] &= 0xffff0000u; any = true; }
            if ((w[e] & 0x7f800000u) == 0x7f800000u) { w[e] &= 0x0000ffffu; any = true; }
        }
        if (any) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            met |= ((ch >> 3) & 127) < rows;
        }
    }
    return met;
}

// HALVES: 64-feature halves of a row in use.
template <int HALVES>
__global__ void __launch_bounds__(kThreads, 1) paged_pre_kernel(const __grid_constant__ PreParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sRing = smem + 2 * kTileBytes;
    PreBars* bars = reinterpret_cast<PreBars*>(sRing + kStages * kTileBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t wait_limit = p.wait_limit;
    volatile int* abort_flag = &bars->abort_flag;
    const PagedCache& c = p.c;
    const int cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bars->full[s], 1);
            ptx::mbar_init(&bars->empty[s], 1);
            ptx::mbar_init(&bars->raw_full[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars->q_full[i], 1);
            ptx::mbar_init(&bars->q_empty[i], 1);
            ptx::mbar_init(&bars->s_full[i], 1);
            ptx::mbar_init(&bars->p_full[i], 4);
            ptx::mbar_init(&bars->o_final[i], 1);
            ptx::mbar_init(&bars->o_empty[i], 4);
        }
        for (int i = 0; i < kPieces; ++i) {
            ptx::mbar_init(&bars->piece_full[i], 1);
            ptx::mbar_init(&bars->piece_empty[i], kPieceUsers);
        }
        ptx::mbar_init(&bars->drain, 1);
        for (int i = 0; i < kMeta; ++i) bars->bad_piece[i] = -1;
        bars->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        p.desc[cta] = make_int4(0, 0, 0, 0);
    }
    // ---- the list of items: each thread sums a run of sequences, then a scan
    Piece* pieces = reinterpret_cast<Piece*>(bars + 1);
    {
        const long long max_keys = table_keys(c);
        const int per = (c.B + kThreads - 1) / kThreads;
        const int b0 = min((int)threadIdx.x * per, c.B), b1 = min(b0 + per, c.B);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += seq_items(p, seq_info(c, b), max_keys);
        long long incl = mine * c.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) bars->scan[warp] = incl;
        if (warp == 0) {
            ptx::tmem_alloc(&bars->tmem_base, 512);
            ptx::tmem_relinquish();
        }
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        long long total = 0, pre = 0;
        for (int x = 0; x < kThreads / 32; ++x) {
            if (x < warp) pre += bars->scan[x];
            total += bars->scan[x];
        }
        incl += pre;
        const int W = (int)max(1LL, min((long long)kParts, total));
        if (cta >= W || total == 0) {
            if (warp == 0) ptx::tmem_dealloc(bars->tmem_base, 512);
            return;
        }
        const long long lo = part_begin(total, cta, W), hi = part_begin(total, cta + 1, W);
        long long at = incl - mine * c.Hkv;
        if (lo >= at && lo < incl) {  // one thread: the part begins in its run
            Piece w;
            for (w.b = b0; w.b < b1; ++w.b) {
                w.sq = seq_info(c, w.b);
                const long long k = seq_items(p, w.sq, max_keys);
                if (lo < at + k * c.Hkv) {
                    long long in = lo - at;
                    w.kvh = (int)(in / k);
                    in -= w.kvh * k;
                    int x = 0, y = (w.sq.n + 2 * p.n - 1) / (2 * p.n) - 1;  // last unit that starts at or before `in`
                    while (x < y) {
                        const int mid = (x + y + 1) / 2;
                        if (items_before(p, w.sq, mid, max_keys) <= in) x = mid; else y = mid - 1;
                    }
                    w.rt = x;
                    w.first = (int)(in - items_before(p, w.sq, x, max_keys));
                    break;
                }
                at += k * c.Hkv;
            }
            w.left = (int)(hi - lo);
            w.shape(p);
            pieces[0] = w;
            bars->total = total;
            bars->hi = hi;
            bars->W = W;
        }
        __syncthreads();
    }
    const uint32_t tmem = bars->tmem_base;
    const int n = p.n;
    // piece k's description, once it is there (nullptr: the wait ran out)
    auto take_piece = [&](int k) -> const Piece* {
        const bool got = ptx::mbar_wait(&bars->piece_full[k % kPieces], (k / kPieces) & 1, wait_limit, abort_flag);
        return got ? pieces + k % kPieces : nullptr;
    };

    if (warp >= 8) ptx::setmaxnreg_dec<kControlRegs>();
    if (warp == kProducerWarp) {
        // -------------------------------------------------------- TMA warp
        int st = 0;
        uint32_t ph = 1, used = 0, full_par = 0, raw_par = 0, last_raw = 0;  // per-stage bits for the drain
        int q_loads = 0;  // of tiles 0 and 1 in turn
        bool ok = true;
        int item = 0;  // items of the part so far
        if (lane == 0) {
            ptx::prefetch_tmap(&p.tm_q);
            ptx::prefetch_tmap(&p.tm_k);
            ptx::prefetch_tmap(&p.tm_v);
            if (p.Ld > 0) {
                ptx::prefetch_tmap(&p.tm_kd);
                ptx::prefetch_tmap(&p.tm_vd);
            }
        }
        for (int piece = 0; ok; ++piece) {
            const Piece* w = pieces + piece % kPieces;
            if (lane == 0) ptx::mbar_arrive(&bars->piece_full[piece % kPieces]);
            const int first = w->first, end = w->end, kvh = w->kvh, b = w->b;
            const int n_seq = w->u.n_seq, nk = w->u.nk, ntok = w->u.ntok;
            const int row0 = w->sq.q0 + w->u.tok0, pos_first = w->sq.pos0 + w->u.tok0;
            const int sl0 = first * kSlices;
            auto fetch = [&](int sl) {
                int pg = -1;
                if (sl < n_seq * kSlices && sl * 16 < nk) pg = page_of(c, b, sl * 16 / c.page_size);
                return pg;
            };
            int page = fetch(sl0 + lane), page_next = fetch(sl0 + 32 + lane);
            for (int x = first; x < end && ok; ++x, ++item) {
                const bool seq = x < n_seq;
                const int rel = x * kSlices - sl0;
                if (seq && rel && (rel & 31) == 0) {
                    page = page_next;
                    page_next = fetch(sl0 + rel + 32 + lane);
                }
                const uint32_t none =
                    __ballot_sync(0xffffffffu, __shfl_sync(0xffffffffu, page, (rel & 31) + (lane & 7)) < 0) & 0xffu;
                for (int kv = 0; kv < 2; ++kv) {
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bars->empty[st], ph, wait_limit, abort_flag))) {
                        if (lane == 0) flag_timeout(p, bars);
                        ok = false;
                        break;
                    }
                    uint8_t* dst = sRing + st * kTileBytes;
                    const bool raw = kv && (!seq || (x + 1) * kItemKeys - 1 > pos_first);
                    uint64_t* bar = raw ? &bars->raw_full[st] : &bars->full[st];
                    const uint32_t bit = 1u << st;
                    if (raw) raw_par ^= bit;
                    full_par ^= bit;
                    last_raw = raw ? last_raw | bit : last_raw & ~bit;
                    used |= bit;
                    if (kv == 0 && lane == 0) bars->holes[item % kMeta] = seq ? none : 0;
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, HALVES * kHalfBytes);
                    __syncwarp();
                    if (seq) {
                        // boxes of box_rows rows and half of the features
                        const int half = lane & 1, r0 = (lane >> 1) * p.box_rows;
                        const int pg = __shfl_sync(0xffffffffu, page, ((rel & 31) + (r0 >> 4)) & 31);
                        if (r0 < kItemKeys && half < HALVES)
                            // a page that is not there lies outside the map: zeros
                            ptx::tma_load_4d(dst + half * kHalfBytes + r0 * 128, kv ? &p.tm_v : &p.tm_k, bar, half * 64,
                                             pg < 0 ? 0 : (x * kItemKeys + r0) % c.page_size, kvh,
                                             pg < 0 ? c.num_pages : pg);
                    } else {
                        const int sl = lane & 7, half = (lane >> 3) & 1;
                        const int y = w->u.chunk(x - n_seq) * kSlices + sl;
                        const int tok = p.DSL ? y / p.DSL : 0, s16 = p.DSL ? y % p.DSL : 0;
                        if (lane < 16 && half < HALVES)
                            ptx::tma_load_4d(dst + half * kHalfBytes + sl * 2048, kv ? &p.tm_vd : &p.tm_kd, bar,
                                             half * 64, kvh, s16 * 16, p.DSL && tok < ntok ? row0 + tok : c.N);
                    }
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                    if (kv == 0 && x == first && ok) {
                        // this piece's queries, once the piece before has used its own
                        for (int i = 0; i < 2 && ok; ++i) {
                            if (piece > 0 &&
                                !__all_sync(0xffffffffu, ptx::mbar_wait(&bars->q_empty[i], (piece - 1) & 1, wait_limit, abort_flag))) {
                                if (lane == 0) flag_timeout(p, bars);
                                ok = false;
                                break;
                            }
                            if (lane == 0) ptx::mbar_arrive_expect_tx(&bars->q_full[i], HALVES * n * p.G * 128);
                            __syncwarp();
                            if (lane < HALVES)
                                ptx::tma_load_4d(sQ + i * kTileBytes + lane * kHalfBytes, &p.tm_q, &bars->q_full[i], lane * 64,
                                                 kvh * p.G, row0 + i * n, 0);
                            ++q_loads;
                        }
                    }
                    if (!ok) break;
                }
            }
            // describe the next piece
            if (!ok || w->left <= end - first) break;
            const int nx = (piece + 1) % kPieces;
            if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bars->piece_empty[nx], (((piece + 1) / kPieces) & 1) ^ 1, wait_limit,
                                                        abort_flag))) {
                if (lane == 0) flag_timeout(p, bars);
                break;
            }
            if (lane == 0) {
                Piece v = *w;
                v.next(p);
                pieces[nx] = v;
            }
            __syncwarp();
        }
        // every load this CTA issued lands before it exits
        for (int i = 0; i < 2; ++i)
            if (q_loads > i) ptx::mbar_wait(&bars->q_full[i], ((q_loads - 1 - i) / 2) & 1, kNoPollLimit, nullptr);
        for (int s = 0; s < kStages; ++s) {
            if (!((used >> s) & 1)) continue;
            if ((last_raw >> s) & 1) ptx::mbar_wait(&bars->raw_full[s], ((raw_par >> s) & 1) ^ 1, kNoPollLimit, nullptr);
            else ptx::mbar_wait(&bars->full[s], ((full_par >> s) & 1) ^ 1, kNoPollLimit, nullptr);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // -------------------------------------------------------- MMA warp
        // One lane issues. The loop over plain items is that lane's alone; at a
        // piece's ends, where instruction fetch is what costs, the whole warp
        // walks and one lane's predicate issues: the code is smaller so.
        const uint32_t lead = lane == 0;
        constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(128, kItemKeys, 0, 0);
        constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, HALVES * 64, 0, 1);
        const uint32_t sQa = ptx::smem_u32(sQ), sRa = ptx::smem_u32(sRing);
        const uint64_t q0 = ptx::umma_desc_sw128(sQa, 16, 1024);
        const uint64_t k0 = ptx::umma_desc_sw128(sRa, 16, 1024);
        const uint64_t v0 = ptx::umma_desc_sw128(sRa, kHalfBytes, 1024);
        constexpr uint64_t kSlotUnits = kTileBytes >> 4;
        auto wait_one = [&](uint64_t* bar, uint32_t parity) {
            const bool got = ptx::mbar_wait(bar, parity, wait_limit, abort_flag);
            if (got) ptx::tc_fence_after();
            else flag_timeout(p, bars);
            return got;
        };
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            const bool got = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, wait_limit, abort_flag));
            if (got) ptx::tc_fence_after();
            else if (lead) flag_timeout(p, bars);
            return got;
        };
        auto issue_s_one = [&](int i, int st) {
            const uint64_t kd_ = k0 + (uint64_t)st * kSlotUnits, qd_ = q0 + (uint64_t)i * kSlotUnits;
#pragma unroll
            for (int k = 0; k < 4 * HALVES; ++k) {
                const uint64_t off = (uint64_t)((k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2);
                ptx::mma_ss(tmem + i * 128, qd_ + off, kd_ + off, idesc_qk, k > 0);
            }
            ptx::mma_commit(&bars->s_full[i]);
        };
        auto issue_pv_one = [&](int i, uint64_t vd, bool add) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                ptx::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8, vd + (uint64_t)(k * 128), idesc_pv,
                            (add || k > 0) ? 1u : 0u);
        };
        uint32_t pp = 0;                 // p_full phases, a bit per tile
        int st = 0;
        uint32_t ph = 0;
        auto advance = [&]() {
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
        };
        bool ok = true;
        bool more = true;
        for (int piece = 0; more && ok; ++piece) {
            const Piece* w = take_piece(piece);
            if (!__all_sync(0xffffffffu, w != nullptr)) {
                if (lead) flag_timeout(p, bars);
                break;
            }
            const Unit u = w->u;
            const int first = w->first, end = w->end;
            more = w->left > end - first;
            __syncwarp();
            if (lead) ptx::mbar_arrive(&bars->piece_empty[piece % kPieces]);
            // the last item of each tile in the piece (first - 1: none)
            int last0 = end - 1, last1 = u.ntok > n ? end - 1 : first - 1;
            while (last0 >= first && !u.part(0, last0)) --last0;
            while (last1 >= first && !u.part(1, last1)) --last1;
            // Rolled, for the items at a piece's ends: unrolled, a batch of 216-token
            // sequences took 230 us instead of 204
            auto issue_tail = [&](int i, int x, int slot) {
                const uint64_t kd_ = k0 + (uint64_t)slot * kSlotUnits, qd_ = q0 + (uint64_t)i * kSlotUnits;
#pragma unroll 1
                for (int k = 0; k < 4 * HALVES; ++k) {
                    const uint64_t off = (uint64_t)((k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2);
                    ptx::mma_ss_lead(tmem + i * 128, qd_ + off, kd_ + off, idesc_qk, k > 0, lead);
                }
                ptx::mma_commit_lead(&bars->s_full[i], lead);
                // after its last product the tile's queries may go
                if (x == (i ? last1 : last0)) ptx::mma_commit_lead(&bars->q_empty[i], lead);
            };
            // o_final may run at most one piece ahead of either tile's warps,
            // also of a tile that takes no part in these pieces
            auto finish = [&](int i) {
                if (piece > 0 && !wait_all(&bars->o_empty[i], (piece - 1) & 1)) return false;
                ptx::mma_commit_lead(&bars->o_final[i], lead);
                return true;
            };
            auto who = [&](int x) { return (u.part(0, x) ? 1u : 0u) | (u.part(1, x) ? 2u : 0u); };
            uint32_t cur = who(first), started = 0;
            ok = wait_all(&bars->full[st], ph);
#pragma unroll 1
            for (int i = 0; i < 2 && ok; ++i) {
                ok = wait_all(&bars->q_full[i], piece & 1);
                if (!ok) break;
                if ((cur >> i) & 1) issue_tail(i, first, st);
                if ((i ? last1 : last0) < first) {
                    ptx::mma_commit_lead(&bars->q_empty[i], lead);
                    ok = finish(i);
                }
            }
            if (!ok) break;
            ptx::mma_commit_lead(&bars->empty[st], lead);
            advance();
            // Items that both tiles take part in, as in the next one, and that
            // are nobody's last: the loop that has to keep the tensor core fed
            const int plain = min(end - 2, min(u.nkv0, u.nkv1) - 2);
            int x = first;
            if (lead) {
                for (; x < plain; ++x) {
                    const int st_v = st;
                    if (!(ok = wait_one(&bars->full[st], ph))) break;
                    advance();
                    const uint64_t vd = v0 + (uint64_t)st_v * kSlotUnits;
#pragma unroll 1
                    for (int i = 0; i < 2 && ok; ++i) {
                        if (!(ok = wait_one(&bars->p_full[i], (pp >> i) & 1))) break;
                        issue_pv_one(i, vd, x > first);
                        if (i == 0 && !(ok = wait_one(&bars->full[st], ph))) break;
                        issue_s_one(i, st);
                    }
                    if (!ok) break;
                    ptx::mma_commit(&bars->empty[st_v]);
                    ptx::mma_commit(&bars->empty[st]);
                    advance();
                    pp ^= 3;
                    started = 3;
                }
            }
            __syncwarp();
            x = __shfl_sync(0xffffffffu, x, 0);
            st = __shfl_sync(0xffffffffu, st, 0);
            ph = __shfl_sync(0xffffffffu, ph, 0);
            pp = __shfl_sync(0xffffffffu, pp, 0);
            started = __shfl_sync(0xffffffffu, started, 0);
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            if (x > first) cur = 3;
            for (; x < end && ok; ++x) {
                const int st_v = st;
                ok = wait_all(&bars->full[st], ph);
                if (!ok) break;
                advance();
                const bool next = x + 1 < end;
                const uint64_t vd = v0 + (uint64_t)st_v * kSlotUnits;
                const uint32_t nxt = next ? who(x + 1) : 0u;
                bool k_ready = false;
                // round 0: a tile that sits this item out can go ahead with the
                // next; then tile 0's and tile 1's P V and next S
#pragma unroll 1
                for (int step = 0; step < 4 && ok; ++step) {
                    const int i = step & 1;
                    const bool in = (cur >> i) & 1;
                    if (step < 2 ? in : !in) continue;
                    if (in) {
                        // (P also says that this tile's warps have read the O of the
                        // piece before, which the piece's first P V overwrites)
                        if (!wait_all(&bars->p_full[i], (pp >> i) & 1)) {
                            ok = false;
                            break;
                        }
                        pp ^= 1u << i;
#pragma unroll 1
                        for (int k = 0; k < 8; ++k)
                            ptx::mma_ts_lead(tmem + 256 + i * 128, tmem + i * 128 + k * 8, vd + (uint64_t)(k * 128), idesc_pv,
                                        ((started >> i) & 1) | (k > 0 ? 1u : 0u), lead);
                        started |= 1u << i;
                        if (x == (i ? last1 : last0) && !finish(i)) {
                            ok = false;
                            break;
                        }
                    }
                    if ((nxt >> i) & 1) {
                        if (!k_ready && !wait_all(&bars->full[st], ph)) {
                            ok = false;
                            break;
                        }
                        k_ready = true;
                        issue_tail(i, x + 1, st);
                    }
                }
                if (!ok) break;
                ptx::mma_commit_lead(&bars->empty[st_v], lead);
                if (next) {
                    ptx::mma_commit_lead(&bars->empty[st], lead);
                    advance();
                }
                cur = nxt;
            }
        }
        ptx::mma_commit_lead(&bars->drain, lead);
        ptx::mbar_wait(&bars->drain, 0, kNoPollLimit, nullptr);
        __syncwarp();
    } else if (warp >= kCondFirst) {
        // ---------------------------------------------------- conditioning
        const int ct = threadIdx.x - kCondFirst * 32;
        int st = 0;
        uint32_t raw_par = 0;
        bool ok = true;
        bool more = true;
        for (int piece = 0; more && ok; ++piece) {
            const Piece* w = take_piece(piece);
            if (!ptx::bar_and(1, kCond, w != nullptr)) {
                if (ct == 0) flag_timeout(p, bars);
                break;
            }
            const int first = w->first, end = w->end, n_seq = w->u.n_seq, nk = w->u.nk;
            const int pos_first = w->sq.pos0 + w->u.tok0;
            more = w->left > end - first;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->piece_empty[piece % kPieces]);
            for (int x = first; x < end && ok; ++x) {
                const bool seq = x < n_seq;
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    uint8_t* slot = sRing + st * kTileBytes;
                    uint64_t* full = &bars->full[st];
                    if (kv && (!seq || (x + 1) * kItemKeys - 1 > pos_first)) {
                        const bool got = ptx::mbar_wait(&bars->raw_full[st], (raw_par >> st) & 1, wait_limit, abort_flag);
                        raw_par ^= 1u << st;
                        if (!ptx::bar_and(1, kCond, got)) {
                            if (ct == 0) flag_timeout(p, bars);
                            ok = false;
                            break;
                        }
                        const int rows = seq ? min(nk - x * kItemKeys, kItemKeys) : kItemKeys;
                        if (clear_nonfinite(slot, ct, rows, HALVES)) bars->bad_piece[piece % kMeta] = piece;
                        ptx::fence_proxy_async_smem();
                        ptx::bar_sync(1, kCond);
                        if (ct == 0) ptx::mbar_arrive(full);
                    }
                    if (++st == kStages) st = 0;
                }
            }
        }
    } else if (warp < 8) {
        // ---------------------------------------------- softmax warpgroups
        ptx::setmaxnreg_inc<kSoftmaxRegs>();
        const int i = warp / 4;
        const int r = (warp % 4) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t tS = tmem + lane_off + i * 128, tO = tmem + lane_off + 256 + i * 128;
        const bool used = r < n * p.G;        // (n G may be less than 128)
        const int tl = used ? i * n + r / p.G : 2 * n;  // token of the unit
        const int hh = r % p.G;
        bool ok = true;
        uint32_t sp = 0;                      // s_full phase
        int item = 0;
        bool more = true;
        for (int piece = 0; more && ok; ++piece) {
            const Piece* w = take_piece(piece);
            if (!__all_sync(0xffffffffu, w != nullptr)) {
                if (lane == 0) flag_timeout(p, bars);
                break;
            }
            const int first = w->first, end = w->end, n_seq = w->u.n_seq;
            more = w->left > end - first;
            const int pos = used ? w->sq.pos0 + w->u.tok0 + tl : -1;
            float m = -INFINITY, l = 0.f;
            int it = 0;
            const int nkv = i ? w->u.nkv1 : w->u.nkv0;
            for (int x = first; x < end; ++x, ++item) {
                if (x < n_seq ? x >= nkv : !w->u.part(i, x)) continue;
                const bool got = ptx::mbar_wait(&bars->s_full[i], sp, wait_limit, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    if (lane == 0) flag_timeout(p, bars);
                    ok = false;
                    break;
                }
                sp ^= 1;
                ptx::tc_fence_after();
                const bool seq = x < n_seq;
                const int kbase = x * kItemKeys;
                const uint32_t holes = bars->holes[item % kMeta];
                // the columns this row sees
                int lo = 0, hi = pos - kbase + 1;
                if (!seq) {
                    lo = (tl * p.DSL - w->u.chunk(x - n_seq) * kSlices) * 16;
                    hi = lo + p.Ld;
                }
                if (__all_sync(0xffffffffu, seq && hi >= 128) && !holes)
                    softmax_item(tS, tO, true, 0, 127, 0, 0, false, 0, p.sl2, it, m, l);  // nothing to mask
                else
                    softmax_masked(tS, tO, lo, hi, holes, p.sl2, it, m, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bars->p_full[i]);
                ++it;
            }
            if (!ok) break;
            const bool got = ptx::mbar_wait(&bars->o_final[i], piece & 1, wait_limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) flag_timeout(p, bars);
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const int kvh = w->kvh;
            const bool valid = tl < w->u.ntok;
            const bool whole = first == 0 && end == w->u.n_items;
            const int ps = 2 * cta + (first == 0 ? 1 : 0);
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            const long long row = (long long)(w->sq.q0 + w->u.tok0 + tl) * p.Hq + kvh * p.G + hh;
            const bool bad = *reinterpret_cast<volatile int*>(&bars->bad_piece[piece % kMeta]) == piece;
#pragma unroll 1
            for (int cc = 0; cc < 4 && cc * 32 < c.d; ++cc) {
                uint32_t o[32];
                if (it > 0) {
                    ptx::tmem_ld32(tO + cc * 32, o);
                    ptx::tmem_wait_ld();
                } else {  // no item of the piece was this tile's: O holds nothing
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                }
                if (bad && valid) {
                    // the non-finite values that were cleared, for the rows that see them
                    auto add = [&](const __nv_bfloat16* v) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (cc * 32 + e >= c.d) break;
                            const float f = __bfloat162float(v[cc * 32 + e]);
                            if (!(fabsf(f) <= 3.4e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
                        }
                    };
                    {
                        const int pf = w->sq.pos0 + w->u.tok0;  // tiles that end past it were cleared
                        const int x0 = max(first, max(0, pf + 1) / kItemKeys), x1 = min(end, n_seq);
                        for (int j = x0 * kItemKeys; j < min(x1 * kItemKeys, min(pos + 1, w->u.nk)); ++j) {
                            const int pg = page_of(c, w->b, j / c.page_size);
                            if (pg >= 0)
                                add(p.v_pages + (((long long)pg * c.Hkv + kvh) * c.page_size + j % c.page_size) * c.d);
                        }
                    }
                    for (int s = 0; s < p.Ld; ++s) {
                        const int xi = w->u.item_of((tl * p.DSL + s / 16) / kSlices);
                        if (xi >= first && xi < end)
                            add(p.vd + (((long long)(w->sq.q0 + w->u.tok0 + tl) * p.Ld_cap + s) * c.Hkv + kvh) * c.d);
                    }
                }
                if (!valid) continue;
                if (whole) {
                    uint32_t q[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        q[e] = ptx::pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row * c.d + cc * 32);
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (cc * 32 + 8 * v < c.d) dst[v] = make_uint4(q[4 * v], q[4 * v + 1], q[4 * v + 2], q[4 * v + 3]);
                } else {
                    float* dst = p.part_o + ((long long)ps * kRows + i * 128 + r) * kD + cc * 32;
#pragma unroll
                    for (int v = 0; v < 4; ++v) ptx::st_global_32b(dst + 8 * v, &o[8 * v]);
                }
            }
            if (valid) {
                if (!whole && first == 0 && threadIdx.x == 0) {
                    // parts of the unit, up to the one that holds its last item
                    const long long last = bars->hi - w->left + w->u.n_items;
                    const int c_last = (int)((last * bars->W + bars->total - 1) / bars->total) - 1;
                    p.desc[cta] = make_int4(w->sq.q0, kvh, w->rt, (c_last - cta + 1) | (w->u.ntok <= n ? w->u.ntok * p.G : 128 + (w->u.ntok - n) * p.G) << 16);
                }
                if (!whole)
                    *reinterpret_cast<float2*>(p.part_ml + ((long long)ps * kRows + i * 128 + r) * 2) = make_float2(m, l);
                else if (p.lse)
                    p.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
            }
            // O has been read
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(&bars->o_empty[i]);
                ptx::mbar_arrive(&bars->piece_empty[piece % kPieces]);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    // the join may be scheduled once every CTA is about here; earlier its
    // waiting blocks would take issue slots from this kernel
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int HALVES>
cudaError_t launch_halves(const PagedFwdArgs& a, char* ws, cudaStream_t s) {
    PreParams p;
    memset(static_cast<void*>(&p), 0, sizeof(p));
    const PagedCache& c = a.c;
    const cuuint64_t P = c.page_size, Hkv = c.Hkv;
    p.n = 128 / a.G;
    p.lg_step = -1;
    for (int lg = 1; lg <= 7; ++lg)
        if (2 * p.n == 1 << lg) p.lg_step = lg;
    const cuuint64_t d = c.d;
    {
        const cuuint64_t dims[4] = {d, (cuuint64_t)a.Hq, (cuuint64_t)c.N, 1};
        const cuuint64_t st[3] = {d * 2, (cuuint64_t)a.Hq * d * 2, (cuuint64_t)c.N * a.Hq * d * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)a.G, (cuuint32_t)p.n, 1};
        if (!make_tmap_bf16_4d(&p.tm_q, a.q, dims, st, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[4] = {d, P, Hkv, (cuuint64_t)c.num_pages};
        const cuuint64_t st[3] = {d * 2, P * d * 2, Hkv * P * d * 2};
        p.box_rows = std::min(c.page_size & -c.page_size, kItemKeys);
        const cuuint32_t box[4] = {64, (cuuint32_t)p.box_rows, 1, 1};
        if (!make_tmap_bf16_4d(&p.tm_k, a.k_pages, dims, st, box) || !make_tmap_bf16_4d(&p.tm_v, a.v_pages, dims, st, box))
            return cudaErrorInvalidValue;
    }
    {
        // Without depth rows a unit that sees no key still has one item, all of
        // it masked: boxes of the same size, anywhere in the pages.
        const bool any = a.Ld > 0;
        const cuuint64_t dims[4] = {d, Hkv, any ? (cuuint64_t)a.Ld : P, (cuuint64_t)(any ? c.N : c.num_pages)};
        const cuuint64_t st[3] = {any ? d * 2 : P * d * 2, any ? Hkv * d * 2 : d * 2,
                                  (cuuint64_t)(any ? a.Ld_cap : P) * Hkv * d * 2};
        const cuuint32_t box[4] = {64, 1, 16, 1};
        if (!make_tmap_bf16_4d(&p.tm_kd, any ? a.kd : a.k_pages, dims, st, box) ||
            !make_tmap_bf16_4d(&p.tm_vd, any ? a.vd : a.v_pages, dims, st, box))
            return cudaErrorInvalidValue;
    }
    p.c = c;
    p.v_pages = static_cast<const __nv_bfloat16*>(a.v_pages);
    p.vd = static_cast<const __nv_bfloat16*>(a.vd);
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.Hq = a.Hq; p.G = a.G; p.Ld = a.Ld; p.Ld_cap = a.Ld_cap; p.DSL = (a.Ld + 15) / 16;
    p.sl2 = a.scale * 1.4426950408889634f;
    p.status = a.status;
    p.wait_limit = a.wait_limit;
    p.desc = reinterpret_cast<int4*>(ws);
    // [desc | part_ml | part_o], part_o at a 32-byte boundary
    p.part_ml = reinterpret_cast<float*>(ws + kParts * sizeof(int4));
    p.part_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(p.part_ml + (size_t)2 * kParts * kRows * 2) + 31) & ~uintptr_t(31));
    static SmemLimit limit;
    const auto kern = paged_pre_kernel<HALVES>;
    cudaError_t err = limit.raise(reinterpret_cast<const void*>(kern), kSmemBytes);
    if (err != cudaSuccess) return err;
    kern<<<kParts, kThreads, kSmemBytes, s>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    JoinParams j{p.c, p.out, p.lse, p.part_o, p.part_ml, p.desc, p.Hq, p.G, p.n};
    return launch_paged_join<kRows, kD, kParts>(j, s);
}

cudaError_t launch(const PagedFwdArgs& a, char* ws, cudaStream_t s) {
    return a.c.d <= 64 ? launch_halves<1>(a, ws, s) : launch_halves<2>(a, ws, s);
}

// 8-bit pages to bf16 pages, for the pages this call
// reads: value = code * scale, exact, as the scale is a power of two. Every
// unit of a chunk would otherwise convert the same tiles again: in the kernel
// the conversion shared the SM with the softmax and took two and a half times
// the matrix products' time, here it is one pass over the cache (1 byte read,
// 2 written per element), and what it writes is still in L2 when it is read.
// One CTA per (block of the table, kv-head): 16 codes per thread and step.
// The copies have the pages' own numbers, or, with `table`, those of the block
// table's entries, which then names them for the attention.
__global__ void __launch_bounds__(256) paged_dequant_kernel(const PagedCache c, const int8_t* kc, const int8_t* vc,
                                                            const float* ks, const float* vs, __nv_bfloat16* ko,
                                                            __nv_bfloat16* vo, int32_t* table) {
    const int h = blockIdx.y;
    const int total = c.B * c.max_blocks;
    for (int x = blockIdx.x; x < total; x += gridDim.x) {
        const int b = x / c.max_blocks, blk = x % c.max_blocks;
        const SeqInfo s = seq_info(c, b);
        const long long keys = (long long)s.pos0 + s.n;  // seen by the last new token
        const bool seen = s.n != 0 && (long long)blk * c.page_size < keys;
        const int page = seen ? page_of(c, b, blk) : -1;
        if (table && h == 0 && threadIdx.x == 0) table[x] = page < 0 ? -1 : x;
        if (page < 0) continue;
        const long long row = (long long)page * c.Hkv + h, to_row = table ? (long long)x * c.Hkv + h : row;
        const float k1 = __ldg(ks + row), v1 = __ldg(vs + row);
        const long long at = row * c.page_size * c.d, to = to_row * c.page_size * c.d;
        const int n16 = (int)min((long long)c.page_size, keys - (long long)blk * c.page_size) * (c.d / 16);
        for (int e = threadIdx.x; e < n16; e += blockDim.x) {
            const uint4 a = *reinterpret_cast<const uint4*>(kc + at + e * 16), d = *reinterpret_cast<const uint4*>(vc + at + e * 16);
            auto put = [&](const uint4& w, float sc, __nv_bfloat16* dst) {
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                uint32_t o[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int i0 = (int)(u[q] << 24) >> 24, i1 = (int)(u[q] << 16) >> 24, i2 = (int)(u[q] << 8) >> 24, i3 = (int)u[q] >> 24;
                    o[2 * q] = ptx::pack_bf16x2(i0 * sc, i1 * sc);
                    o[2 * q + 1] = ptx::pack_bf16x2(i2 * sc, i3 * sc);
                }
                ptx::st_global_32b(dst, o);
            };
            put(a, k1, ko + to + e * 16);
            put(d, v1, vo + to + e * 16);
        }
    }
}

size_t join_bytes() {
    return kParts * sizeof(int4) + 2 * (size_t)kParts * kRows * (kD + 2) * sizeof(float) + 32;
}
size_t up(size_t n, size_t to) { return (n + to - 1) & ~(to - 1); }
// bytes of a pool of `pages` bf16 pages
size_t pool_bytes(const PagedCache& c, long long pages) {
    return up((size_t)pages * c.Hkv * c.page_size * c.d * 2, 256);
}
// The bf16 copy of 8-bit pages: with room for every page of the cache, by its
// number, or for the block table's entries, by theirs, with a table, where that
// halves it (a call on a few sequences of a large cache). The table is not free:
// 63 prompts of 216 tokens in a cache of 255 pages took 127 us by page and 131 by
// entry. max_blocks == 0: not known.
struct Copy {
    bool by_entry;
    size_t table, pool;  // bytes of the table and of each of K and V
};
Copy copy_of(const PagedCache& c) {
    const Copy by_page = {false, 0, pool_bytes(c, c.num_pages)};
    const long long entries = (long long)c.B * c.max_blocks;
    if (entries == 0 || 2 * entries > c.num_pages) return by_page;
    const Copy by_entry = {true, up((size_t)entries * sizeof(int32_t), 256), pool_bytes(c, entries)};
    return by_entry.table + 2 * by_entry.pool < 2 * by_page.pool ? by_entry : by_page;  // (never more than by page)
}

}  // namespace

bool paged_pre_supported(const PagedFwdArgs& a) {
    // (a scale <= 0 goes to the other kernels: the dense softmax step takes a
    // row's maximum before it scales)
    // (the copy's grid, and its index, which runs past the entries by up to a grid)
    if (a.k_scale && ((long long)a.c.B * a.c.max_blocks > 0x7fff0000LL || a.c.Hkv > 65535)) return false;
    return a.dtype == MODA_BF16 && a.c.d % 8 == 0 && a.G <= 128 && a.c.page_size % 16 == 0 && a.scale > 0.f &&
           (long long)a.c.N * a.Hq < 0x7fffff00LL;  // rows in 32 bits, the last tile's end among them
}

size_t paged_pre_workspace(const PagedCache& c, bool q8) {
    const size_t parts = up(join_bytes(), 256);
    if (!q8) return parts;
    const Copy copy = copy_of(c);
    return parts + copy.table + 2 * copy.pool + 32;
}

cudaError_t launch_paged_pre(const PagedFwdArgs& a, cudaStream_t s) {
    char* ws = static_cast<char*>(a.workspace);
    if (!a.k_scale) return launch(a, ws, s);
    // [parts | table | bf16 K pages | bf16 V pages], the pages at 32-byte boundaries
    const PagedCache& c = a.c;
    const Copy copy = copy_of(c);
    char* at = reinterpret_cast<char*>(up(reinterpret_cast<uintptr_t>(ws + up(join_bytes(), 256)), 32));
    int32_t* table = copy.by_entry ? reinterpret_cast<int32_t*>(at) : nullptr;
    at += copy.table;
    PagedFwdArgs f = a;
    f.k_pages = at;
    f.v_pages = at + copy.pool;
    f.k_scale = f.v_scale = nullptr;
    const long long blocks = (long long)c.B * c.max_blocks;
    if (copy.by_entry) {
        f.c.block_table = table;
        f.c.num_pages = (int)blocks;
    }
    paged_dequant_kernel<<<dim3((unsigned)std::min(blocks, 4096LL), c.Hkv), 256, 0, s>>>(
        c, static_cast<const int8_t*>(a.k_pages), static_cast<const int8_t*>(a.v_pages), a.k_scale, a.v_scale,
        reinterpret_cast<__nv_bfloat16*>(at), reinterpret_cast<__nv_bfloat16*>(at + copy.pool), table);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch(f, ws, s) : e;
}

}  // namespace moda
