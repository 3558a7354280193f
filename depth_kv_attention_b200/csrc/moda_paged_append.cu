// Appending to the paged sequence cache: the new tokens' keys (rotated by
// their position), values and rotated queries, in one launch (8-bit pages with
// many queries: two, side by side).
//
// What it computes, per token at position p of its sequence and per head:
//   (x1, x2) -> (x1 cos - x2 sin, x2 cos + x1 sin)   over the rot/2 pairs
// with cos / sin read from the caller's table row p, each product and sum one
// IEEE fp32 operation, rounded once to the storage type. Keys and values go to
// row p % page_size of page block_table[b][p / page_size]; optionally also to
// the token's depth slot (the write step of "Mixture-of-Depths Attention",
// gist.science German summary §2, Write-Step), which saves the separate pass.
//
// 8-bit pages hold int8 codes and one power-of-two scale per (page, kv-head):
// the smallest 2^e with amax <= 127 * 2^e over the rows written, or the page's
// old scale if that is larger and the page holds earlier tokens. A power of
// two makes every step but the rounding to a code exact, in any precision, and
// lets a page grow: earlier codes move to a larger scale by an exact shift
// with one rounding, so that after any number of moves a code is within one
// step of its value (1/2 + 1/4 + ... steps). An arbitrary scale would lose
// half a step at each move.
//
// Memory-bound: every input and output byte moves once. One warp serves a
// token (or a share of its heads), a lane keeps the same pairs of every head,
// so cos and sin stay in registers across heads. Two forms, by size:
//  * few bytes: a warp per (token, share of heads) straight from global memory,
//    as many warps as there are shares;
//  * many: resident warps walk runs of tokens and bulk copies bring the next
//    token's rows into shared memory meanwhile, which keeps more bytes in
//    flight than registers can and looks up sequence and page once a run.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "paged_common.cuh"
#include "paged_ptx.cuh"
#include "smem_limit.h"

namespace moda {
namespace {

constexpr int kWarps = 4;

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Chunk {
    T x[VEC];
};

template <int VEC>
struct Turn {
    float c[VEC], s[VEC];
};

// cos / sin of pairs pair0 .. pair0 + N - 1 of a table row; N of them at once
// (rows and halves are aligned to min(16, 4 N) bytes where N > 1).
template <int N>
struct alignas(N >= 4 ? 16 : 4 * N) Row {
    float x[N >= 4 ? 4 : N];
};
template <int VEC, int N>
__device__ __forceinline__ void load_turn(Turn<VEC>& t, const float* row, int rot, int pair0) {
    constexpr int W = N >= 4 ? 4 : N;
#pragma unroll
    for (int e = 0; e < N; e += W) {
        const Row<N> c = *reinterpret_cast<const Row<N>*>(row + pair0 + e);
        const Row<N> s = *reinterpret_cast<const Row<N>*>(row + rot / 2 + pair0 + e);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            t.c[e + k] = c.x[k];
            t.s[e + k] = s.x[k];
        }
    }
}

__device__ __forceinline__ void turn_pair(float a, float b, float c, float s, float& u, float& w) {
    u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    w = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// A head row is cut into units: rotation units first, then plain chunks.
//   half split:  unit = chunk i and chunk i + rot/2           (2 VEC features)
//   interleaved: unit = one chunk of VEC features = VEC/2 pairs
//                (VEC = 1: the two features of one pair)
struct Units {
    int rot_units, plain_units, total;
    __host__ __device__ Units(int d, int rot, int interleaved, int vec) {
        const int span = interleaved ? (vec == 1 ? 2 : vec) : 2 * vec;
        rot_units = rot / span;
        plain_units = (d - rot) / vec;
        total = rot_units + plain_units;
    }
};

// Features [f0, f0 + VEC) and, for two-part units, [f1, f1 + VEC) of unit u.
template <int VEC, bool INTER>
struct Unit {
    int f0, f1;
    bool two, turned;
    Turn<VEC> t;
    // where the unit's features are,
    __device__ __forceinline__ void place(int u, const Units& n, int rot) {
        turned = u < n.rot_units;
        two = turned && (!INTER || VEC == 1);
        if (!turned) f0 = rot + (u - n.rot_units) * VEC;
        else f0 = u * (INTER && VEC == 1 ? 2 : VEC);
        f1 = INTER ? f0 + 1 : f0 + rot / 2;
    }
    // and its cos / sin too
    __device__ __forceinline__ void set(int u, const Units& n, int rot, const float* row) {
        place(u, n, rot);
        if (turned) {
            if (INTER) {
                load_turn<VEC, VEC == 1 ? 1 : VEC / 2>(t, row, rot, VEC == 1 ? u : u * VEC / 2);
            } else {
                load_turn<VEC, VEC>(t, row, rot, f0);
            }
        }
    }
    // The unit's features of one head row as they are stored,
    template <typename T>
    __device__ __forceinline__ void load(const T* row, Chunk<T, VEC>& ca, Chunk<T, VEC>& cb) const {
        ca = *reinterpret_cast<const Chunk<T, VEC>*>(row + f0);
        if (two) cb = *reinterpret_cast<const Chunk<T, VEC>*>(row + f1);
    }
    // and rotated, as fp32.
    template <typename T>
    __device__ __forceinline__ void turn(const Chunk<T, VEC>& ca, const Chunk<T, VEC>& cb, float (&a)[VEC],
                                         float (&b)[VEC]) const {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            a[e] = pg_to_f(ca.x[e]);
            b[e] = two ? pg_to_f(cb.x[e]) : 0.f;
        }
        if (!turned) return;
        if (INTER && VEC > 1) {
#pragma unroll
            for (int e = 0; e < VEC / 2; ++e) {
                const float x = a[2 * e], y = a[2 * e + 1];
                turn_pair(x, y, t.c[e], t.s[e], a[2 * e], a[2 * e + 1]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float x = a[e], y = b[e];
                turn_pair(x, y, t.c[e], t.s[e], a[e], b[e]);
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&a)[VEC], const float (&b)[VEC]) const {
        Chunk<T, VEC> ca, cb;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            ca.x[e] = pg_from_f<T>(a[e]);
            cb.x[e] = pg_from_f<T>(b[e]);
        }
        *reinterpret_cast<Chunk<T, VEC>*>(row + f0) = ca;
        if (two) *reinterpret_cast<Chunk<T, VEC>*>(row + f1) = cb;
    }
};

// Token i: its sequence, position and whether the call takes it at all.
struct Token {
    int b;
    long long pos;
    bool taken;
};
__device__ __forceinline__ Token find_token(const AppendArgs& a, int i) {
    Token t;
    t.b = seq_of_token(a.c, i);
    t.taken = t.b < a.c.B && i >= __ldg(a.c.cu_q + (t.b < a.c.B ? t.b : 0));
    t.pos = -1;
    if (t.taken) {
        t.pos = (long long)__ldg(a.c.ctx_lens + t.b) - ((long long)__ldg(a.c.cu_q + t.b + 1) - i);
        t.taken = t.pos >= 0 && (!a.rope || t.pos < a.rope_len);
    }
    return t;
}

// One warp: heads [h0, h1) of token i, in the order q heads, k heads, v heads,
// from rows at q, k, v (head h of q at q + h d) and the token's table row.
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void put_heads(const AppendArgs& a, int i, int page, int row, int h0, int h1, const T* q,
                                          const T* k, const T* v, const float* rope) {
    const PagedCache& c = a.c;
    const int lane = threadIdx.x % 32, P = c.page_size, d = c.d;
    const int rot = rope ? a.rot : 0;
    const Units n(d, rot, INTER, VEC);
    T* kp = static_cast<T*>(a.k_pages) + (((long long)page * c.Hkv) * P + row) * d;
    T* vp = static_cast<T*>(a.v_pages) + (((long long)page * c.Hkv) * P + row) * d;
    T* kdp = a.kd ? static_cast<T*>(a.kd) + ((long long)i * a.Ld + a.slot) * c.Hkv * d : nullptr;
    T* vdp = a.vd ? static_cast<T*>(a.vd) + ((long long)i * a.Ld + a.slot) * c.Hkv * d : nullptr;
    const bool paged = page >= 0 && !a.k_scale;
    const int nk = a.Hq + c.Hkv;
    // q and k heads
    {
        const int per = n.total < 32 ? 32 / n.total : 1;  // heads at a time
        const int hg = n.total < 32 ? lane / n.total : 0;
        for (int u = n.total < 32 ? lane % n.total : lane; u < n.total; u += 32) {
            if (hg >= per) break;
            Unit<VEC, INTER> un;
            un.set(u, n, rot, rope);
            const int end = h1 < nk ? h1 : nk;
            constexpr int kBatch = 4;  // heads in flight: all loads before the first store
            for (int h = h0 + hg; h < end; h += kBatch * per) {
                Chunk<T, VEC> ca[kBatch], cb[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int hj = h + j * per;
                    if (hj >= end) break;
                    un.load(hj < a.Hq ? q + (long long)hj * d : k + (long long)(hj - a.Hq) * d, ca[j], cb[j]);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int hj = h + j * per;
                    if (hj >= end) break;
                    float x[VEC], y[VEC];
                    un.turn(ca[j], cb[j], x, y);
                    if (hj < a.Hq) {
                        un.store(static_cast<T*>(a.q_out) + ((long long)i * a.Hq + hj) * d, x, y);
                    } else {
                        if (paged) un.store(kp + (long long)(hj - a.Hq) * P * d, x, y);
                        if (kdp) un.store(kdp + (long long)(hj - a.Hq) * d, x, y);
                    }
                }
            }
        }
    }
    // v heads: copied
    const int v0 = h0 > nk ? h0 : nk;
    if (h1 > v0) {
        const int chunks = d / VEC;
        for (int x = lane; x < (h1 - v0) * chunks; x += 32) {
            const int h = v0 - nk + x / chunks, f = x % chunks * VEC;
            const Chunk<T, VEC> ch = *reinterpret_cast<const Chunk<T, VEC>*>(v + (long long)h * d + f);
            if (paged) *reinterpret_cast<Chunk<T, VEC>*>(vp + (long long)h * P * d + f) = ch;
            if (vdp) *reinterpret_cast<Chunk<T, VEC>*>(vdp + (long long)h * d + f) = ch;
        }
    }
}

template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void token_heads(const AppendArgs& a, int i, int h0, int h1) {
    const Token t = find_token(a, i);
    if (!t.taken) return;
    put_heads<T, VEC, INTER>(a, i, page_of(a.c, t.b, t.pos / a.c.page_size), (int)(t.pos % a.c.page_size), h0, h1,
                             static_cast<const T*>(a.q) + i * a.sq, static_cast<const T*>(a.k) + i * a.sk,
                             static_cast<const T*>(a.v) + i * a.sv, a.rope ? a.rope + t.pos * a.rot : nullptr);
}

// Warp w of the launch serves share w % shares of the heads of token w / shares.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) paged_append_kernel(const AppendArgs a, int shares, int h_first, int h_all) {
    const long long w = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
    const int i = (int)(w / shares), part = (int)(w % shares);
    if (w / shares >= a.c.N) return;
    const int per = (h_all - h_first + shares - 1) / shares;
    const int h0 = h_first + part * per, h1 = min(h0 + per, h_all);
    if (h0 < h1) token_heads<T, VEC, INTER>(a, i, h0, h1);
}

// The form for many bytes. Every warp has two buffers, each for heads_per heads
// of one token and its table row, and walks a run of (token, part) items in
// order: part x = heads [h_first + x heads_per, ...). Bulk copies need 16-byte
// aligned rows, which the vector form has.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kWarps * 32) paged_append_bulk_kernel(const AppendArgs a, int parts, int heads_per,
                                                                        int h_first, int h_all) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ uint64_t bars[kWarps][2];
    const PagedCache& c = a.c;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, d = c.d;
    const int row_bytes = heads_per * d * (int)sizeof(T), rope_bytes = a.rope ? a.rot * 4 : 0;
    uint8_t* buf = smem + (size_t)warp * 2 * (row_bytes + rope_bytes);
    // the keys and values of 8-bit pages, which need nothing of this, may start
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lane == 0) {
        ptx::mbar_init(&bars[warp][0], 1);
        ptx::mbar_init(&bars[warp][1], 1);
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    __syncwarp();
    const long long items = (long long)c.N * parts, warps = (long long)gridDim.x * kWarps;
    const long long w = (long long)blockIdx.x * kWarps + warp;
    const long long lo = items * w / warps, hi = items * (w + 1) / warps;
    // the sequence and page of the last token looked at
    int b = -1, seq_lo = 0, seq_hi = 0, page = -1;
    long long pos0 = 0, blk = -1;
    struct Item {
        int i, h0, h1, page, row;  // h1 == h0: not taken
    };
    auto fetch = [&](long long x, int s) {  // item x into buffer s
        Item it;
        it.i = (int)(x / parts);
        it.h0 = h_first + (int)(x % parts) * heads_per;
        it.h1 = min(it.h0 + heads_per, h_all);
        if (b < 0 || it.i >= seq_hi || it.i < seq_lo) {
            b = seq_of_token(c, it.i);
            blk = -1;
            if (b < c.B) {
                seq_lo = __ldg(c.cu_q + b);
                seq_hi = __ldg(c.cu_q + b + 1);
                pos0 = (long long)__ldg(c.ctx_lens + b) - seq_hi;  // position = pos0 + row
            } else {
                seq_lo = it.i;  // behind the last sequence
                seq_hi = c.N;
            }
        }
        const long long pos = pos0 + it.i;
        if (b >= c.B || it.i < seq_lo || pos < 0 || (a.rope && pos >= a.rope_len)) {
            it.h1 = it.h0;
            return it;
        }
        const long long bk = pos / c.page_size;
        if (bk != blk) {
            blk = bk;
            page = page_of(c, b, bk);
        }
        it.page = page;
        it.row = (int)(pos - bk * c.page_size);
        if (lane == 0) {
            uint8_t* dst = buf + s * (row_bytes + rope_bytes);
            uint64_t* bar = &bars[warp][s];
            const int nk = a.Hq + c.Hkv;
            ptx::mbar_arrive_expect_tx(bar, (it.h1 - it.h0) * d * (int)sizeof(T) + rope_bytes);
            auto copy = [&](int from, int to, const void* base, long long stride, int first) {
                from = max(from, it.h0);
                to = min(to, it.h1);
                if (from < to)
                    ptx::bulk_load(dst + (size_t)(from - it.h0) * d * sizeof(T),
                                   static_cast<const T*>(base) + it.i * stride + (long long)(from - first) * d,
                                   (to - from) * d * (int)sizeof(T), bar);
            };
            copy(0, a.Hq, a.q, a.sq, 0);
            copy(a.Hq, nk, a.k, a.sk, a.Hq);
            copy(nk, nk + c.Hkv, a.v, a.sv, nk);
            if (rope_bytes) ptx::bulk_load(dst + row_bytes, a.rope + pos * a.rot, rope_bytes, bar);
        }
        return it;
    };
    uint32_t par = 0;  // bit s: phase of buffer s
    Item cur = {}, nxt = {};
    if (lo < hi) cur = fetch(lo, 0);
    for (long long x = lo; x < hi; ++x) {
        const int s = (int)(x - lo) & 1;
        if (x + 1 < hi) nxt = fetch(x + 1, s ^ 1);
        if (cur.h1 > cur.h0) {
            const bool got = ptx::mbar_wait(&bars[warp][s], (par >> s) & 1, a.wait_limit, nullptr);
            par ^= 1u << s;
            if (!__all_sync(0xffffffffu, got)) {
                if (lane == 0) atomicOr(a.status, 1u);
                // what is in flight lands before the warp ends
                ptx::mbar_wait(&bars[warp][s], ((par >> s) & 1) ^ 1, 0, nullptr);
                if (x + 1 < hi && nxt.h1 > nxt.h0) ptx::mbar_wait(&bars[warp][s ^ 1], (par >> (s ^ 1)) & 1, 0, nullptr);
                return;
            }
            const uint8_t* src = buf + s * (row_bytes + rope_bytes);
            const T* base = reinterpret_cast<const T*>(src) - (long long)cur.h0 * d;  // head h at base + h d
            put_heads<T, VEC, INTER>(a, cur.i, cur.page, cur.row, cur.h0, cur.h1, base, base + (long long)a.Hq * d,
                                     base + (long long)(a.Hq + c.Hkv) * d,
                                     rope_bytes ? reinterpret_cast<const float*>(src + row_bytes) : nullptr);
        }
        __syncwarp();  // the buffer has been read before its next copy
        cur = nxt;
    }
}

// ------------------------------------------------------------- 8-bit pages
// Scale of values up to amax (finite, >= 0): the smallest 2^e, e >= -126, with
// amax <= 127 * 2^e; 0 for amax = 0. amax = m * 2^E with 1 <= m < 2:
// e = E - 6 when m <= 127/64, else E - 5.
__device__ __forceinline__ float scale_for(float amax) {
    if (!(amax > 0.f)) return 0.f;
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127 - 6 + ((u & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    e = max(e, -126);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y <= 3.402823466e38f ? y : 0.f;
}
// rhe(x / scale) clamped to +-127, as 1/scale is a power of two (0 for NaN).
__device__ __forceinline__ int code_of(float x, float inv) {
    const float y = __fmul_rn(x, inv);
    return y == y ? (int)fminf(fmaxf(rintf(y), -127.f), 127.f) : 0;
}

// The codes of VEC values. Without non-finite ones among them (`odd`) no code
// is out of range, and adding 1.5 * 2^23 rounds x / scale to a whole number,
// half to even, in the sum's low byte: x * inv is exact, so the fused add rounds
// once.
template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* dst, const float (&x)[VEC], float inv, bool odd) {
    if (odd || VEC < 4) {
        Chunk<int8_t, VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.x[e] = (int8_t)code_of(x[e], inv);
        *reinterpret_cast<Chunk<int8_t, VEC>*>(dst) = o;
        return;
    }
    uint32_t w[VEC >= 4 ? VEC / 4 : 1];
#pragma unroll
    for (int e = 0; e + 3 < VEC; e += 4) {
        uint32_t b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(__fmaf_rn(x[e + k], inv, 12582912.f));
        w[e / 4] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    if (VEC == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[VEC / 8]);
    else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

// One CTA: the rows of one page that start at token i (the first token of its
// sequence or of a page), for one kv-head: the first half of its threads the
// keys (kv = 0), the second the values. Two passes, the largest value and the
// codes; the second finds the rows in L1. The loops stay rolled, and the passes
// share one body: a run is a few rounds, and unrolled the code took longer to
// fetch than to run.
constexpr int kRunThreads = 128;  // of each half

template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void page_run(const AppendArgs& a, int i, const Token& t, int g, float* red) {
    const PagedCache& c = a.c;
    const int P = c.page_size, d = c.d, kv = threadIdx.x / kRunThreads, tid = threadIdx.x % kRunThreads;
    const int page = page_of(c, t.b, t.pos / P);
    const int r0 = (int)(t.pos % P);
    float* scales = (kv ? a.v_scale : a.k_scale) + (long long)max(page, 0) * c.Hkv + g;
    const float old = r0 && page >= 0 ? *scales : 0.f;
    long long rows = min((long long)__ldg(c.cu_q + t.b + 1), (long long)c.N) - i;
    if (rows > P - r0) rows = P - r0;
    if (a.rope && rows > a.rope_len - t.pos) rows = a.rope_len - t.pos;
    const int rot = (kv == 0 && a.rope) ? a.rot : 0;
    Units n(d, rot, INTER, VEC);
    // rows without a rotation: two chunks a unit as well, where they are even
    const bool pairs = rot == 0 && d % (2 * VEC) == 0;
    if (pairs) n.total = d / (2 * VEC);
    const T* src = kv ? static_cast<const T*>(a.v) + (long long)g * d : static_cast<const T*>(a.k) + (long long)g * d;
    const long long ss = kv ? a.sv : a.sk;
    T* dep = static_cast<T*>(kv ? a.vd : a.kd);
    const int total = (int)rows * n.total;
    int8_t* codes = static_cast<int8_t*>(kv ? a.v_pages : a.k_pages) + ((long long)max(page, 0) * c.Hkv + g) * P * d;
    float amax = 0.f, none = 0.f;  // none: 0 * every value, NaN when one is not finite
    float now = old, inv = 0.f;
    bool odd = false;
    // pass 0: the largest value; 1: the largest finite one, where some are not; 2: the codes
#pragma unroll 1
    for (int pass = 0; pass < 3; pass += pass || odd ? 1 : 2) {
        if (pass == 2) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (tid % 32 == 0) red[threadIdx.x / 32] = amax;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kRunThreads / 32; ++w) amax = fmaxf(amax, red[kv * (kRunThreads / 32) + w]);
            now = fmaxf(old, scale_for(amax));
            inv = now > 0.f ? 1.f / now : 0.f;  // exact: a power of two
            if (r0 && old != now) {
                const float ratio = __fmul_rn(old, inv);
#pragma unroll 1
                for (int x = tid; x < r0 * (d / VEC); x += kRunThreads) {
                    Chunk<int8_t, VEC>* at = reinterpret_cast<Chunk<int8_t, VEC>*>(codes + (long long)x * VEC);
                    Chunk<int8_t, VEC> ch = *at;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ch.x[e] = (int8_t)code_of((float)ch.x[e], ratio);
                    *at = ch;
                }
            }
        }
#pragma unroll 1
        for (int x = tid; x < total; x += kRunThreads) {
            const int r = x / n.total, u = x - r * n.total;
            Unit<VEC, INTER> un;
            un.set(u, n, rot, rot ? a.rope + (t.pos + r) * a.rot : nullptr);
            if (pairs) {
                un.f0 = u * VEC;
                un.f1 = un.f0 + d / 2;
                un.two = true;
            }
            Chunk<T, VEC> ca, cb;
            un.load(src + (i + r) * ss, ca, cb);
            float p[VEC], q[VEC];  // (q is 0 where a unit has one part)
            un.turn(ca, cb, p, q);
            if (pass == 0) {
                if (dep) un.store(dep + (((long long)(i + r) * a.Ld + a.slot) * c.Hkv + g) * d, p, q);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    amax = fmaxf(amax, fmaxf(fabsf(p[e]), fabsf(q[e])));
                    none = fmaf(p[e], 0.f, fmaf(q[e], 0.f, none));
                }
            } else if (pass == 1) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fmaxf(finite_abs(p[e]), finite_abs(q[e])));
            } else {
                int8_t* dst = codes + (long long)(r0 + r) * d;
                store_codes<VEC>(dst + un.f0, p, inv, odd);
                if (un.two) store_codes<VEC>(dst + un.f1, q, inv, odd);
            }
        }
        if (pass == 0) {
            if (page < 0) return;  // uniform over the CTA
            odd = __syncthreads_or(!(none == 0.f));
            if (odd) amax = 0.f;
        }
    }
    __syncthreads();  // everyone has read the old scale and `red`
    if (tid == 0) *scales = now;
}

// Blocks [0, q_blocks): q heads of the tokens, one warp per share. The rest:
// block x serves the page runs that start in tokens [chunk*x', chunk*(x'+1))
// for one kv-head. Without Q (no queries, or the bulk form takes them) the code
// for them is not there. Three CTAs per SM even at the price of some spills in
// the queries' part: with one, a decode step of 64 tokens ran in two waves (10.0
// us, with three 5.8). 8 chunks, 9975 tokens, into pages of 32 rows, 4 kv-heads:
// 23 us, and 33 us for the queries (163 MB: 4.9 TB/s).
template <typename T, int VEC, bool INTER, bool Q>
__global__ void __launch_bounds__(2 * kRunThreads, 3)
paged_append_q8_kernel(const AppendArgs a, int shares, int q_blocks, int chunk) {
    if (Q && (int)blockIdx.x < q_blocks) {
        const long long w = (long long)blockIdx.x * (2 * kRunThreads / 32) + threadIdx.x / 32;
        if (w / shares >= a.c.N) return;
        const int per = (a.Hq + shares - 1) / shares, h0 = (int)(w % shares) * per;
        if (h0 < a.Hq) token_heads<T, VEC, INTER>(a, (int)(w / shares), h0, min(h0 + per, a.Hq));
        return;
    }
    __shared__ float red[2 * kRunThreads / 32];
    const int x = blockIdx.x - q_blocks, g = x % a.c.Hkv;
    const long long i0 = (long long)(x / a.c.Hkv) * chunk;
    // lane e looks at token i0 + e. A run starts where the sequence's new
    // tokens start (counting from the first one with a position) and at each
    // page's first row.
    const PagedCache& c = a.c;
    const int lane = threadIdx.x % 32;
    Token t;
    t.b = seq_of_token(c, (int)i0);
    t.taken = false;
    t.pos = -1;
    const int i = (int)i0 + lane;
    bool head = false;
    if (lane < chunk && i0 + lane < c.N) {
        while (t.b < c.B && __ldg(c.cu_q + t.b + 1) <= i) ++t.b;
        if (t.b < c.B) {
            const int lo = __ldg(c.cu_q + t.b);
            t.pos = (long long)__ldg(c.ctx_lens + t.b) - ((long long)__ldg(c.cu_q + t.b + 1) - i);
            t.taken = i >= lo && t.pos >= 0 && (!a.rope || t.pos < a.rope_len);
            head = t.taken && (t.pos % c.page_size == 0 || i == lo || i == 0);
        }
    }
    for (uint32_t heads = __ballot_sync(0xffffffffu, head); heads; heads &= heads - 1) {
        const int e = __ffs(heads) - 1;
        Token run;
        run.b = __shfl_sync(0xffffffffu, t.b, e);
        run.pos = __shfl_sync(0xffffffffu, t.pos, e);
        run.taken = true;
        page_run<T, VEC, INTER>(a, (int)i0 + e, run, g, red);
    }
    // Beside the bulk form's queries (see launch): what comes next in the stream
    // has to find those done too, so one block outlasts them.
    if (!Q && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// From this many bytes of q, k and v the bulk form is the faster one. Measured
// (bf16, 32 + 2 * 4 heads of 128, rotated, one slot written; direct / bulk):
// 128 tokens 4.0 / 5.7 us, 256 tokens (2.6 MB) 6.4 / 5.9, 1024 tokens 11.1 /
// 6.7, 32768 tokens 213 / 144 us (80 % of the copy bandwidth).
constexpr long long kBulkBytes = 5LL << 19;
constexpr int kBulkBuffer = 10 * 1024;  // two of them a warp, four warps a CTA, two CTAs per SM

// heads [h_first, h_all) of every token
template <typename T, int VEC, bool INTER>
cudaError_t launch_bulk(const AppendArgs& a, int h_first, int h_all, cudaStream_t s) {
    const PagedCache& c = a.c;
    const int heads = h_all - h_first, head_bytes = c.d * (int)sizeof(T);
    const int most = kBulkBuffer / head_bytes > 0 ? kBulkBuffer / head_bytes : 1;
    const int parts = (heads + most - 1) / most, per = (heads + parts - 1) / parts;
    const int bytes = kWarps * 2 * (per * head_bytes + (a.rope ? a.rot * 4 : 0));
    auto kern = paged_append_bulk_kernel<T, VEC, INTER>;
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void*>(kern), kWarps * 2 * (kBulkBuffer + 512));
    if (e != cudaSuccess) return e;
    kern<<<2 * 148, kWarps * 32, bytes, s>>>(a, parts, per, h_first, h_all);
    return cudaGetLastError();
}

template <typename T, int VEC, bool INTER>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    const PagedCache& c = a.c;
    const int rot = a.rope ? a.rot : 0;
    const Units n(c.d, rot, INTER, VEC);
    const int per_pass = n.total < 32 ? 32 / n.total : 1;  // heads a warp serves at a time
    const bool q8 = a.k_scale != nullptr;
    const int h_first = a.q ? 0 : a.Hq, h_all = q8 ? a.Hq : a.Hq + 2 * c.Hkv;
    const int heads = h_all - h_first;  // of the token warps (8-bit pages: q only)
    const bool bulk = VEC > 1 && (long long)c.N * heads * c.d * (long long)sizeof(T) >= kBulkBytes;
    if constexpr (VEC > 1) {
        if (bulk) {
            const cudaError_t e = launch_bulk<T, VEC, INTER>(a, h_first, h_all, s);
            if (e != cudaSuccess || !q8) return e;
        }
    }
    // few tokens: split a token's heads until about 16 warps per SM are busy
    int shares = 1;
    while (shares * 2 * per_pass <= heads && (long long)c.N * shares < 148 * 16) shares *= 2;
    const long long blocks = ((long long)c.N * shares + kWarps - 1) / kWarps;
    if (!q8) {
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        paged_append_kernel<T, VEC, INTER><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a, shares, h_first, h_all);
    } else {
        // tokens whose page runs a CTA serves: one while the CTAs fit the GPU
        // about at once (every CTA looks up its tokens first), a page at most
        const long long waves = (long long)c.N * c.Hkv / (148 * 4);
        const int chunk = (int)std::max(1LL, std::min<long long>(waves, std::min(c.page_size, 32)));
        const long long q_blocks = a.q && !bulk ? ((long long)c.N * shares + 7) / 8 : 0;
        const long long all = q_blocks + ((long long)c.N + chunk - 1) / chunk * c.Hkv;
        if (all > 0x7fffffffLL) return cudaErrorInvalidValue;
        if (q_blocks) {
            paged_append_q8_kernel<T, VEC, INTER, true><<<(unsigned)all, 2 * kRunThreads, 0, s>>>(a, shares, (int)q_blocks, chunk);
        } else {
            // beside the queries' kernel, where that went ahead (8 chunks, 9975 tokens: 56 us
            // one after the other, 51 side by side; one of 4096 37 and 30)
            cudaLaunchConfig_t cfg;
            std::memset(&cfg, 0, sizeof(cfg));
            cfg.gridDim = dim3((unsigned)all);
            cfg.blockDim = dim3(2 * kRunThreads);
            cfg.stream = s;
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            at[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = at;
            cfg.numAttrs = bulk ? 1 : 0;
            return cudaLaunchKernelEx(&cfg, paged_append_q8_kernel<T, VEC, INTER, false>, a, shares, 0, chunk);
        }
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const AppendArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int rot = a.rope ? a.rot : 0;
    // vectors of 16 bytes need whole ones in each rotated part and an aligned table
    const bool vec = (a.interleaved ? rot : rot / 2) % V == 0 && (reinterpret_cast<uintptr_t>(a.rope) & 15u) == 0;
    if (a.interleaved) return vec ? launch<T, V, true>(a, s) : launch<T, 1, true>(a, s);
    return vec ? launch<T, V, false>(a, s) : launch<T, 1, false>(a, s);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t s) {
    return a.dtype == MODA_F32 ? pick<float>(a, s) : pick<__nv_bfloat16>(a, s);
}

}  // namespace moda
