// Attention over the paged sequence cache for many query rows per sequence
// (chunks of prompts, wide drafts): bf16 or 8-bit pages, d = 128, on tcgen05.
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
//  * Conditioning warps see the tiles that cannot go to the tensor core as
//    they came. 8-bit tiles become bf16 in place (a code times its page's
//    power-of-two scale, exact). Value tiles in which some row is masked are
//    cleared of non-finite elements (a masked P is 0, and 0 * NaN is not);
//    rows that do see one get it added back when the piece ends.
//  * Every mbarrier wait is bounded, as in the dense forward.
#include <cuda_bf16.h>

#include <cmath>
#include <cstring>

#include "depth_mask.cuh"
#include "fwd_softmax.cuh"
#include "paged_join.cuh"
#include "paged_units.cuh"
#include "sm100_ptx.cuh"
#include "tmap_host.h"

namespace moda {
namespace {

constexpr int kD = 128;
constexpr int kTileBytes = 128 * kD * 2;
constexpr int kHalfBytes = kTileBytes / 2;
constexpr int kStages = 5;
constexpr int kRows = 256;      // rows of a unit: two tiles
constexpr int kItemKeys = 128;
constexpr int kSlices = 8;      // 16-row slices of an item
constexpr int kParts = 148;     // one CTA per SM
constexpr int kMeta = 8;        // items whose slice notes are kept (the ring holds at most 3)
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr uint32_t kNoPollLimit = 0;

struct PreParams {
    CUtensorMap tm_q, tm_k, tm_v, tm_kd, tm_vd;
    PagedCache c;
    const float* k_scale;
    const float* v_scale;
    const __nv_bfloat16* v_pages;  // bf16 pages and depth values, read again only
    const __nv_bfloat16* vd;       // for rows that see a non-finite value
    __nv_bfloat16* out;
    float* lse;
    float* part_o;
    float* part_ml;
    int4* desc;
    int Hq, G, n, Ld, Ld_cap, DSL;
    float sl2;
    unsigned int* status;
    unsigned int wait_limit;
};

// Warpgroups 0, 1: softmax of tiles 0, 1. Warps 8, 9: producer, MMA. bf16:
// warps 10-11 condition (16-bit tiles rarely need it); 8-bit: a fourth
// warpgroup does, one key row per thread. Registers at launch and after
// reallocation: 384 x 168 = 256 x 216 + 128 x 72; 512 x 128 = 256 x 200 + 256 x 56.
template <bool Q8>
struct Roles {
    static constexpr int kThreads = Q8 ? 512 : 384;
    static constexpr int kCondFirst = Q8 ? 12 : 10;
    static constexpr int kCond = Q8 ? 128 : 64;  // conditioning threads
    static constexpr int kSoftmaxRegs = Q8 ? 200 : 216;
    static constexpr int kControlRegs = Q8 ? 56 : 72;
};

struct __align__(8) PreBars {
    uint64_t q_full, q_empty;
    uint64_t full[kStages], empty[kStages], raw_full[kStages];
    uint64_t s_full[2], p_full[2], o_final[2], o_empty[2];
    uint64_t drain;
    float scale[kStages][kSlices];   // 8-bit: scale of each slice of a tile
    uint32_t holes[kMeta];           // per item: slices without a page
    int bad_piece[kMeta];            // last piece that met a non-finite value a row may see
    long long scan[16];
    long long begin_in_seq;
    int begin_seq;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kSmemBytes = 2 * kTileBytes + kStages * kTileBytes + 1024 + 1024;
static_assert(sizeof(PreBars) <= 1024, "barrier block");
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

__device__ __forceinline__ void flag_timeout(PreParams const& p, PreBars* bars) {
    *reinterpret_cast<volatile int*>(&bars->abort_flag) = 1;
    atomicOr(p.status, 1u);
}

// A unit: tokens tok0 .. tok0 + ntok - 1 of a sequence (tile i: n of them).
struct Unit {
    int tok0, ntok;
    int nk;                 // sequence keys its last token sees
    int n_seq, n_items;
    int nkv0, nkv1;         // sequence items tile 0 / 1 takes part in
    int dhi0, dlo1, dhi1;   // depth items of tile 0: [n_seq, dhi0), of tile 1: [dlo1, dhi1)
    __device__ __forceinline__ bool part(int i, int x) const {
        return i ? x < nkv1 || (x >= dlo1 && x < dhi1) : x < nkv0 || (x >= n_seq && x < dhi0);
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
    u.dhi0 = u.n_seq + (dep0 + kSlices - 1) / kSlices;
    u.dlo1 = u.n_seq + dep0 / kSlices;
    u.dhi1 = nv1 ? u.n_seq + (dep + kSlices - 1) / kSlices : u.dlo1;
    u.n_items = max(u.n_seq + (dep + kSlices - 1) / kSlices, 1);
    return u;
}

__device__ __forceinline__ long long seq_items(const PreParams& p, const SeqInfo& s, long long max_keys) {
    long long t = 0;
    for (int rt = 0; rt * 2 * p.n < s.n; ++rt) t += make_unit(p, s, rt, max_keys).n_items;
    return t;
}

// The pieces of this CTA's part, walked alike by every role.
struct Walk {
    const PreParams& p;
    long long max_keys, left;
    int b, kvh, rt, first, piece;
    SeqInfo sq;
    Unit u;
    int end;
    __device__ __forceinline__ void shape() {
        u = make_unit(p, sq, rt, max_keys);
        end = (int)min((long long)u.n_items, first + left);
    }
    __device__ __forceinline__ bool next() {  // false: the part is done
        left -= end - first;
        if (left <= 0) return false;
        first = 0;
        ++piece;
        if (++rt * 2 * p.n >= sq.n) {
            rt = 0;
            if (++kvh == p.c.Hkv) {
                kvh = 0;
                do {
                    sq = seq_info(p.c, ++b);
                } while (sq.n == 0 && b + 1 < p.c.B);
            }
        }
        shape();
        return true;
    }
};

// Two codes in bytes 0 and 2 of w, times the power of two in both halves of
// sc2, as a bf16 pair (exact): (0x4300 | low 7 bits) is 128 + them,
// (0x4300 | sign bit) is 128 or 256.
__device__ __forceinline__ uint32_t scaled_codes(uint32_t w, __nv_bfloat162 sc2) {
    const uint32_t y = (w & 0x007f007fu) | 0x43004300u, base = (w & 0x00800080u) | 0x43004300u;
    __nv_bfloat162 a, b;
    memcpy(&a, &y, 4);
    memcpy(&b, &base, 4);
    const __nv_bfloat162 r = __hmul2(__hsub2(a, b), sc2);
    uint32_t o;
    memcpy(&o, &r, 4);
    return o;
}

// Row r of a tile of 128 x 128 codes (plain 128-byte lines in the slot's
// second half) to bf16 in the swizzled K-major layout of the whole slot. The
// thread reads its row before it writes, and only its own line lies where it
// writes features 64-127. Chunks are taken in an order that starts at the
// row's number, so that neighbouring rows hit different banks.
__device__ __forceinline__ void dequant_row(uint8_t* slot, int r, float scale) {
    uint4 in[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        in[j] = *reinterpret_cast<const uint4*>(slot + kHalfBytes + r * 128 + (((j + r) & 7) << 4));
    const __nv_bfloat162 sc2 = __float2bfloat162_rn(scale);
#pragma unroll
    for (int jj = 0; jj < 8; ++jj) {
        const int j = (jj + r) & 7;  // codes 16 j .. 16 j + 15
        const uint32_t w[4] = {in[jj].x, in[jj].y, in[jj].z, in[jj].w};
        uint32_t o[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t lo = scaled_codes(w[q], sc2), hi = scaled_codes(w[q] >> 8, sc2);  // (0, 2), (1, 3)
            o[2 * q] = __byte_perm(lo, hi, 0x5410);
            o[2 * q + 1] = __byte_perm(lo, hi, 0x7632);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int oc = 2 * j + v;  // output chunk of 8 features
            *reinterpret_cast<uint4*>(slot + (oc >> 3) * kHalfBytes + r * 128 + (((oc & 7) ^ (r & 7)) << 4)) =
                make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        }
    }
}

// Sets the non-finite elements of a bf16 value tile to 0. Returns whether this
// thread met one in a row below `rows` (rows past it nobody sees).
template <int THREADS>
__device__ __forceinline__ bool clear_nonfinite(uint8_t* slot, int ct, int rows) {
    bool met = false;
#pragma unroll 4
    for (int ch = ct; ch < kTileBytes / 16; ch += THREADS) {
        uint4* at = reinterpret_cast<uint4*>(slot + ch * 16);
        uint4 v = *at;
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

__device__ __forceinline__ void load_box(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2, int c3) {
    ptx::tma_load_4d(dst, m, bar, c0, c1, c2, c3);
}

template <bool Q8>
__global__ void __launch_bounds__(Roles<Q8>::kThreads, 1) paged_pre_kernel(const __grid_constant__ PreParams p) {
    using R = Roles<Q8>;
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

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        ptx::mbar_init(&bars->q_full, 1);
        ptx::mbar_init(&bars->q_empty, 1);
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&bars->full[s], 1);
            ptx::mbar_init(&bars->empty[s], 1);
            ptx::mbar_init(&bars->raw_full[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars->s_full[i], 1);
            ptx::mbar_init(&bars->p_full[i], 4);
            ptx::mbar_init(&bars->o_final[i], 1);
            ptx::mbar_init(&bars->o_empty[i], 4);
        }
        ptx::mbar_init(&bars->drain, 1);
        for (int i = 0; i < kMeta; ++i) bars->bad_piece[i] = -1;
        bars->abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        p.desc[cta] = make_int4(0, 0, 0, 0);
    }
    // ---- the list of items: each thread sums a run of sequences, then a scan
    Walk w{p};
    w.max_keys = min((long long)c.max_blocks * c.page_size, 0x7fffff00LL);
    {
        const int per = (c.B + R::kThreads - 1) / R::kThreads;
        const int b0 = min((int)threadIdx.x * per, c.B), b1 = min(b0 + per, c.B);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += seq_items(p, seq_info(c, b), w.max_keys);
        long long incl = mine * c.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) bars->scan[warp] = incl;
        __syncthreads();
        long long total = 0, pre = 0;
        for (int x = 0; x < R::kThreads / 32; ++x) {
            if (x < warp) pre += bars->scan[x];
            total += bars->scan[x];
        }
        incl += pre;
        const int W = (int)max(1LL, min((long long)kParts, total));
        if (cta >= W || total == 0) return;
        const long long lo = total * cta / W, hi = total * (cta + 1) / W;
        long long at = incl - mine * c.Hkv;
        if (lo >= at && lo < incl) {
            for (int b = b0; b < b1; ++b) {
                const long long k = seq_items(p, seq_info(c, b), w.max_keys) * c.Hkv;
                if (lo < at + k) {
                    bars->begin_seq = b;
                    bars->begin_in_seq = lo - at;
                    break;
                }
                at += k;
            }
        }
        if (warp == 0) {
            ptx::tmem_alloc(&bars->tmem_base, 512);
            ptx::tmem_relinquish();
        }
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        w.b = bars->begin_seq;
        w.sq = seq_info(c, w.b);
        long long in = bars->begin_in_seq;
        const long long k = max(seq_items(p, w.sq, w.max_keys), 1LL);
        w.kvh = (int)(in / k);
        in -= w.kvh * k;
        w.rt = 0;
        for (;; ++w.rt) {
            const int items = make_unit(p, w.sq, w.rt, w.max_keys).n_items;
            if (in < items) break;
            in -= items;
        }
        w.first = (int)in;
        w.left = hi - lo;
        w.piece = 0;
        w.shape();
        // the first part of a cut unit says where its parts are
        if (threadIdx.x == 0) {
            Walk v = w;
            long long at2 = lo;
            for (;;) {
                if (v.first == 0 && v.end < v.u.n_items) {
                    const long long last = at2 + v.u.n_items - 1;
                    const int c_last = (int)(((last + 1) * W + total - 1) / total) - 1;
                    p.desc[cta] = make_int4(v.b, v.kvh, v.rt, (c_last - cta + 1) | min(v.u.ntok * p.G, kRows) << 16);
                }
                at2 += v.end - v.first;
                if (!v.next()) break;
            }
        }
    }
    const uint32_t tmem = bars->tmem_base;
    const int n = p.n;

    if (warp >= 8) ptx::setmaxnreg_dec<R::kControlRegs>();
    if (warp == kProducerWarp) {
        // -------------------------------------------------------- TMA warp
        int st = 0;
        uint32_t ph = 1, used = 0, full_par = 0, raw_par = 0, last_raw = 0;  // per-stage bits for the drain
        uint32_t q_par = 0;
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
        for (bool more = true; more && ok; more = w.next()) {
            const Unit& u = w.u;
            const int sl0 = w.first * kSlices;
            auto fetch = [&](int sl) {
                int pg = -1;
                if (sl < u.n_seq * kSlices && sl * 16 < u.nk) pg = page_of(c, w.b, sl * 16 / c.page_size);
                return pg;
            };
            auto scales = [&](int pg, float& a, float& e) {
                a = e = 1.f;
                if (Q8 && pg >= 0) {
                    a = __ldg(p.k_scale + (long long)pg * c.Hkv + w.kvh);
                    e = __ldg(p.v_scale + (long long)pg * c.Hkv + w.kvh);
                }
            };
            int page = fetch(sl0 + lane), page_next = fetch(sl0 + 32 + lane);
            float ks, vs, ks_next = 1.f, vs_next = 1.f;
            scales(page, ks, vs);
            const int pos_first = w.sq.pos0 + u.tok0;
            for (int x = w.first; x < w.end && ok; ++x, ++item) {
                const bool seq = x < u.n_seq;
                const int rel = x * kSlices - sl0;
                if (seq && rel && (rel & 31) == 0) {
                    page = page_next;
                    ks = ks_next;
                    vs = vs_next;
                    page_next = fetch(sl0 + rel + 32 + lane);
                }
                if (seq && (rel & 31) == 16) scales(page_next, ks_next, vs_next);
                for (int kv = 0; kv < 2; ++kv) {
                    if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bars->empty[st], ph, wait_limit, abort_flag))) {
                        if (lane == 0) flag_timeout(p, bars);
                        ok = false;
                        break;
                    }
                    uint8_t* dst = sRing + st * kTileBytes;
                    const bool raw = seq ? (Q8 || (kv && (x + 1) * kItemKeys - 1 > pos_first)) : kv;
                    uint64_t* bar = raw ? &bars->raw_full[st] : &bars->full[st];
                    const uint32_t bit = 1u << st;
                    if (raw) raw_par ^= bit;
                    full_par ^= bit;
                    last_raw = raw ? last_raw | bit : last_raw & ~bit;
                    used |= bit;
                    if (seq) {
                        const int sl = lane & 7, half = (lane >> 3) & 1;
                        const int src = (rel & 31) + sl;
                        const int pg = __shfl_sync(0xffffffffu, page, src);
                        const float sc = __shfl_sync(0xffffffffu, kv ? vs : ks, src);
                        const uint32_t none = __ballot_sync(0xffffffffu, lane < 8 && pg < 0);
                        if (Q8 && lane < 8) bars->scale[st][sl] = pg < 0 ? 0.f : sc;
                        if (!kv && lane == 0) bars->holes[item % kMeta] = none;
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, Q8 ? kHalfBytes : kTileBytes);
                        __syncwarp();
                        const int row = pg < 0 ? 0 : (x * kSlices + sl) * 16 % c.page_size;
                        const int pgc = pg < 0 ? c.num_pages : pg;  // outside the map: zeros
                        if (Q8) {
                            if (lane < 8)
                                load_box(dst + kHalfBytes + sl * 2048, kv ? &p.tm_v : &p.tm_k, bar, 0, row, w.kvh, pgc);
                        } else if (lane < 16) {
                            load_box(dst + half * kHalfBytes + sl * 2048, kv ? &p.tm_v : &p.tm_k, bar, half * 64, row,
                                     w.kvh, pgc);
                        }
                    } else {
                        const int sl = lane & 7, half = (lane >> 3) & 1;
                        const int y = (x - u.n_seq) * kSlices + sl;
                        const int tok = p.DSL ? y / p.DSL : 0, s16 = p.DSL ? y % p.DSL : 0;
                        if (!kv && lane == 0) bars->holes[item % kMeta] = 0;
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive_expect_tx(bar, kTileBytes);
                        __syncwarp();
                        if (lane < 16)
                            load_box(dst + half * kHalfBytes + sl * 2048, kv ? &p.tm_vd : &p.tm_kd, bar, half * 64, w.kvh,
                                     s16 * 16, p.DSL && tok < u.ntok ? w.sq.q0 + u.tok0 + tok : c.N);
                    }
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                if (x == w.first && ok) {
                    // this piece's queries, once the piece before has used its own
                    if (w.piece > 0) {
                        if (!__all_sync(0xffffffffu, ptx::mbar_wait(&bars->q_empty, (w.piece - 1) & 1, wait_limit, abort_flag))) {
                            if (lane == 0) flag_timeout(p, bars);
                            ok = false;
                            break;
                        }
                    }
                    if (lane == 0) ptx::mbar_arrive_expect_tx(&bars->q_full, 2 * kTileBytes);
                    __syncwarp();
                    if (lane < 4)
                        load_box(sQ + (lane >> 1) * kTileBytes + (lane & 1) * kHalfBytes, &p.tm_q, &bars->q_full,
                                 (lane & 1) * 64, w.kvh * p.G, w.sq.q0 + u.tok0 + (lane >> 1) * n, 0);
                    q_par = w.piece + 1;  // query loads issued
                }
            }
        }
        // every load this CTA issued lands before it exits
        if (q_par) ptx::mbar_wait(&bars->q_full, (q_par - 1) & 1, kNoPollLimit, nullptr);
        for (int s = 0; s < kStages; ++s) {
            if (!((used >> s) & 1)) continue;
            if ((last_raw >> s) & 1) ptx::mbar_wait(&bars->raw_full[s], ((raw_par >> s) & 1) ^ 1, kNoPollLimit, nullptr);
            else ptx::mbar_wait(&bars->full[s], ((full_par >> s) & 1) ^ 1, kNoPollLimit, nullptr);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------ MMA thread
        if (lane == 0) {
            constexpr uint32_t idesc_qk = ptx::idesc_bf16_f32(128, kItemKeys, 0, 0);
            constexpr uint32_t idesc_pv = ptx::idesc_bf16_f32(128, kD, 0, 1);
            const uint32_t sQa = ptx::smem_u32(sQ), sRa = ptx::smem_u32(sRing);
            const uint64_t q0 = ptx::umma_desc_sw128(sQa, 16, 1024);
            const uint64_t k0 = ptx::umma_desc_sw128(sRa, 16, 1024);
            const uint64_t v0 = ptx::umma_desc_sw128(sRa, kHalfBytes, 1024);
            constexpr uint64_t kSlotUnits = kTileBytes >> 4;
            auto wait_all = [&](uint64_t* bar, uint32_t parity) {
                const bool got = ptx::mbar_wait(bar, parity, wait_limit, abort_flag);
                if (!got) flag_timeout(p, bars);
                else ptx::tc_fence_after();
                return got;
            };
            auto issue_s = [&](int i, int st) {
                const uint64_t kd_ = k0 + (uint64_t)st * kSlotUnits, qd_ = q0 + (uint64_t)i * kSlotUnits;
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const uint64_t off = (uint64_t)((k >> 2) * (kHalfBytes >> 4) + (k & 3) * 2);
                    ptx::mma_ss(tmem + i * 128, qd_ + off, kd_ + off, idesc_qk, k > 0);
                }
                ptx::mma_commit(&bars->s_full[i]);
            };
            uint32_t pp0 = 0, pp1 = 0;       // p_full phases
            int st = 0;
            uint32_t ph = 0;
            auto advance = [&]() {
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            };
            bool ok = true;
            for (bool more = true; more && ok; more = w.next()) {
                const Unit& u = w.u;
                ok = wait_all(&bars->q_full, w.piece & 1);
                if (!ok) break;
                ok = wait_all(&bars->full[st], ph);
                if (!ok) break;
                if (u.part(0, w.first)) issue_s(0, st);
                if (u.part(1, w.first)) issue_s(1, st);
                ptx::mma_commit(&bars->empty[st]);
                advance();
                int cnt0 = 0, cnt1 = 0;      // items of this piece each tile has taken part in
                for (int x = w.first; x < w.end && ok; ++x) {
                    const int st_v = st;
                    ok = wait_all(&bars->full[st], ph);
                    if (!ok) break;
                    advance();
                    const bool next = x + 1 < w.end;
                    const uint64_t vd = v0 + (uint64_t)st_v * kSlotUnits;
                    bool k_ready = false;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (!ok) break;
                        if (u.part(i, x)) {
                            const int cnt = i ? cnt1 : cnt0;
                            // (P also says that this tile's warps have read the O of the
                            // piece before, which the piece's first P V overwrites)
                            if (!wait_all(&bars->p_full[i], i ? pp1 : pp0)) {
                                ok = false;
                                break;
                            }
                            if (i) pp1 ^= 1; else pp0 ^= 1;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                ptx::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8, vd + (uint64_t)(k * 128), idesc_pv,
                                            (cnt > 0 || k > 0) ? 1u : 0u);
                            if (i) ++cnt1; else ++cnt0;
                        }
                        if (next && u.part(i, x + 1)) {
                            if (!k_ready) {
                                if (!wait_all(&bars->full[st], ph)) {
                                    ok = false;
                                    break;
                                }
                                k_ready = true;
                            }
                            issue_s(i, st);
                        }
                    }
                    if (!ok) break;
                    ptx::mma_commit(&bars->empty[st_v]);
                    if (next) {
                        ptx::mma_commit(&bars->empty[st]);
                        advance();
                    }
                }
                // o_final may run at most one piece ahead of either tile's warps,
                // also of a tile that takes no part in these pieces
                if (ok && w.piece > 0)
                    ok = wait_all(&bars->o_empty[0], (w.piece - 1) & 1) && wait_all(&bars->o_empty[1], (w.piece - 1) & 1);
                if (ok) {
                    ptx::mma_commit(&bars->q_empty);
                    ptx::mma_commit(&bars->o_final[0]);
                    ptx::mma_commit(&bars->o_final[1]);
                }
            }
            ptx::mma_commit(&bars->drain);
            ptx::mbar_wait(&bars->drain, 0, kNoPollLimit, nullptr);
        }
        __syncwarp();
    } else if (warp >= R::kCondFirst) {
        // ---------------------------------------------------- conditioning
        const int ct = threadIdx.x - R::kCondFirst * 32;
        int st = 0;
        uint32_t raw_par = 0;
        bool ok = true;
        for (bool more = true; more && ok; more = w.next()) {
            const Unit& u = w.u;
            const int pos_first = w.sq.pos0 + u.tok0;
            for (int x = w.first; x < w.end && ok; ++x)
                for (int kv = 0; kv < 2; ++kv) {
                    const bool seq = x < u.n_seq;
                    const bool raw = seq ? (Q8 || (kv && (x + 1) * kItemKeys - 1 > pos_first)) : kv;
                    const int s = st;
                    if (++st == kStages) st = 0;
                    if (!raw) continue;
                    const bool got = ptx::mbar_wait(&bars->raw_full[s], (raw_par >> s) & 1, wait_limit, abort_flag);
                    raw_par ^= 1u << s;
                    if (!ptx::bar_and(1, R::kCond, got)) {
                        if (ct == 0) flag_timeout(p, bars);
                        ok = false;
                        break;
                    }
                    uint8_t* slot = sRing + s * kTileBytes;
                    if (Q8 && seq) {
                        dequant_row(slot, ct, bars->scale[s][ct >> 4]);
                    } else {
                        const int rows = seq ? min(u.nk - x * kItemKeys, kItemKeys) : kItemKeys;
                        if (clear_nonfinite<R::kCond>(slot, ct, rows)) bars->bad_piece[w.piece % kMeta] = w.piece;
                    }
                    ptx::fence_proxy_async_smem();  // generic writes before the tensor core's reads
                    ptx::bar_sync(1, R::kCond);
                    if (ct == 0) ptx::mbar_arrive(&bars->full[s]);
                }
        }
    } else if (warp < 8) {
        // ---------------------------------------------- softmax warpgroups
        ptx::setmaxnreg_inc<R::kSoftmaxRegs>();
        const int i = warp / 4;
        const int r = (warp % 4) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t tS = tmem + lane_off + i * 128, tO = tmem + lane_off + 256 + i * 128;
        const int tl = i * n + r / p.G;       // token of the unit
        const int hh = r % p.G;
        bool ok = true;
        uint32_t sp = 0;                      // s_full phase
        int item = 0;
        for (bool more = true; more && ok; more = w.next()) {
            const Unit& u = w.u;
            const int pos = w.sq.pos0 + u.tok0 + tl;
            float m = -INFINITY, l = 0.f;
            int it = 0;
            for (int x = w.first; x < w.end; ++x, ++item) {
                if (!u.part(i, x)) continue;
                const bool got = ptx::mbar_wait(&bars->s_full[i], sp, wait_limit, abort_flag);
                if (!__all_sync(0xffffffffu, got)) {
                    if (lane == 0) flag_timeout(p, bars);
                    ok = false;
                    break;
                }
                sp ^= 1;
                ptx::tc_fence_after();
                const bool seq = x < u.n_seq;
                const int kbase = x * kItemKeys;
                const uint32_t holes = bars->holes[item % kMeta];
                softmax_columns(
                    tS, tO,
                    [&](float (&s)[128]) {
                        if (seq) {
                            if (kbase + 127 > pos) {
#pragma unroll
                                for (int k = 0; k < 128; ++k)
                                    if (kbase + k > pos) s[k] = -INFINITY;
                            }
                            if (holes) {
#pragma unroll
                                for (int k = 0; k < 128; ++k)
                                    if ((holes >> (k >> 4)) & 1) s[k] = -INFINITY;
                            }
                        } else {
                            uint32_t vis[4];
                            depth_col_mask((tl * p.DSL - (x - u.n_seq) * kSlices) * 16, p.Ld, false, 0ull, vis);
#pragma unroll
                            for (int k = 0; k < 128; ++k)
                                if (!((vis[k >> 5] >> (k & 31)) & 1u)) s[k] = -INFINITY;
                        }
                    },
                    p.sl2, it, m, l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&bars->p_full[i]);
                ++it;
            }
            if (!ok) break;
            const bool got = ptx::mbar_wait(&bars->o_final[i], w.piece & 1, wait_limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) flag_timeout(p, bars);
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            const bool valid = tl < u.ntok;
            const bool whole = w.first == 0 && w.end == u.n_items;
            const int ps = 2 * cta + (w.first == 0 ? 1 : 0);
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            const long long row = (long long)(w.sq.q0 + u.tok0 + tl) * p.Hq + w.kvh * p.G + hh;
            const bool bad = *reinterpret_cast<volatile int*>(&bars->bad_piece[w.piece % kMeta]) == w.piece;
#pragma unroll 1
            for (int cc = 0; cc < 4; ++cc) {
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
                            const float f = __bfloat162float(v[cc * 32 + e]);
                            if (!(fabsf(f) <= 3.4e38f)) o[e] = __float_as_uint(__uint_as_float(o[e]) + f);
                        }
                    };
                    if (!Q8) {
                        const int pf = w.sq.pos0 + u.tok0;  // tiles that end past it were cleared
                        const int x0 = max(w.first, max(0, pf + 1) / kItemKeys), x1 = min(w.end, u.n_seq);
                        for (int j = x0 * kItemKeys; j < min(x1 * kItemKeys, min(pos + 1, u.nk)); ++j) {
                            const int pg = page_of(c, w.b, j / c.page_size);
                            if (pg >= 0)
                                add(p.v_pages + (((long long)pg * c.Hkv + w.kvh) * c.page_size + j % c.page_size) * kD);
                        }
                    }
                    for (int s = 0; s < p.Ld; ++s) {
                        const int xi = u.n_seq + (tl * p.DSL + s / 16) / kSlices;
                        if (xi >= w.first && xi < w.end)
                            add(p.vd + (((long long)(w.sq.q0 + u.tok0 + tl) * p.Ld_cap + s) * c.Hkv + w.kvh) * kD);
                    }
                }
                if (!valid) continue;
                if (whole) {
                    uint32_t q[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        q[e] = ptx::pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row * kD + cc * 32);
#pragma unroll
                    for (int v = 0; v < 4; ++v) dst[v] = make_uint4(q[4 * v], q[4 * v + 1], q[4 * v + 2], q[4 * v + 3]);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(p.part_o + ((long long)ps * kRows + i * 128 + r) * kD + cc * 32);
#pragma unroll
                    for (int v = 0; v < 8; ++v) dst[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                }
            }
            if (valid) {
                if (!whole)
                    *reinterpret_cast<float2*>(p.part_ml + ((long long)ps * kRows + i * 128 + r) * 2) = make_float2(m, l);
                else if (p.lse)
                    p.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
            }
            // O has been read
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->o_empty[i]);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <bool Q8>
cudaError_t launch(const PagedFwdArgs& a, cudaStream_t s) {
    PreParams p;
    memset(static_cast<void*>(&p), 0, sizeof(p));
    const PagedCache& c = a.c;
    const cuuint64_t P = c.page_size, Hkv = c.Hkv, e = Q8 ? 1 : 2;
    p.n = 128 / a.G;
    {
        const cuuint64_t dims[4] = {kD, (cuuint64_t)a.Hq, (cuuint64_t)c.N, 1};
        const cuuint64_t st[3] = {kD * 2, (cuuint64_t)a.Hq * kD * 2, (cuuint64_t)c.N * a.Hq * kD * 2};
        const cuuint32_t box[4] = {64, (cuuint32_t)a.G, (cuuint32_t)p.n, 1};
        if (!make_tmap_bf16_4d(&p.tm_q, a.q, dims, st, box)) return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[4] = {kD, P, Hkv, (cuuint64_t)c.num_pages};
        const cuuint64_t st[3] = {kD * e, P * kD * e, Hkv * P * kD * e};
        const cuuint32_t box[4] = {Q8 ? 128u : 64u, 16, 1, 1};
        const bool ok = Q8 ? make_tmap_u8_4d(&p.tm_k, a.k_pages, dims, st, box) && make_tmap_u8_4d(&p.tm_v, a.v_pages, dims, st, box)
                           : make_tmap_bf16_4d(&p.tm_k, a.k_pages, dims, st, box) && make_tmap_bf16_4d(&p.tm_v, a.v_pages, dims, st, box);
        if (!ok) return cudaErrorInvalidValue;
    }
    if (a.Ld > 0) {
        const cuuint64_t dims[4] = {kD, Hkv, (cuuint64_t)a.Ld, (cuuint64_t)c.N};
        const cuuint64_t st[3] = {kD * 2, Hkv * kD * 2, (cuuint64_t)a.Ld_cap * Hkv * kD * 2};
        const cuuint32_t box[4] = {64, 1, 16, 1};
        if (!make_tmap_bf16_4d(&p.tm_kd, a.kd, dims, st, box) || !make_tmap_bf16_4d(&p.tm_vd, a.vd, dims, st, box))
            return cudaErrorInvalidValue;
    } else {
        p.tm_kd = p.tm_k;
        p.tm_vd = p.tm_v;
    }
    p.c = c;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.v_pages = Q8 ? nullptr : static_cast<const __nv_bfloat16*>(a.v_pages);
    p.vd = static_cast<const __nv_bfloat16*>(a.vd);
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.Hq = a.Hq; p.G = a.G; p.Ld = a.Ld; p.Ld_cap = a.Ld_cap; p.DSL = (a.Ld + 15) / 16;
    p.sl2 = a.scale * 1.4426950408889634f;
    p.status = a.status;
    p.wait_limit = a.wait_limit;
    char* ws = static_cast<char*>(a.workspace);
    p.desc = reinterpret_cast<int4*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + kParts * sizeof(int4));
    p.part_o = p.part_ml + (size_t)2 * kParts * kRows * 2;
    auto kern = paged_pre_kernel<Q8>;
    static SmemLimit limit;
    cudaError_t err = limit.raise(reinterpret_cast<const void*>(kern), kSmemBytes);
    if (err != cudaSuccess) return err;
    kern<<<kParts, Roles<Q8>::kThreads, kSmemBytes, s>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    JoinParams j{p.c, p.out, p.lse, p.part_o, p.part_ml, p.desc, p.Hq, p.G};
    return launch_paged_join<kRows, kD, kParts>(j, s);
}

}  // namespace

bool paged_pre_supported(const PagedFwdArgs& a) {
    // (a scale <= 0 goes to the other kernels: the dense softmax step takes a
    // row's maximum before it scales)
    return a.dtype == MODA_BF16 && a.c.d == kD && a.G <= 128 && 128 % a.G == 0 && a.c.page_size % 16 == 0 && a.scale > 0.f &&
           (long long)a.c.N * a.Hq < (1LL << 31);
}

size_t paged_pre_workspace() {
    return kParts * sizeof(int4) + 2 * (size_t)kParts * kRows * (kD + 2) * sizeof(float);
}

cudaError_t launch_paged_pre(const PagedFwdArgs& a, cudaStream_t s) {
    return a.k_scale ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace moda
