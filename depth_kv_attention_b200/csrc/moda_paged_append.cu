// Appending to the paged sequence cache: the new tokens' keys (rotated by
// their position), values and rotated queries, in one launch.
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
// token (or a share of its heads when there are few tokens), a lane keeps the
// same pairs of every head, so cos and sin stay in registers across heads.
#include <cuda_bf16.h>

#include "paged_common.cuh"

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

// cos / sin of the VEC pairs of unit u (identity when there is no rotation).
template <int VEC>
__device__ __forceinline__ void load_turn(Turn<VEC>& t, const float* row, int rot, int pair0, int n) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        t.c[e] = e < n ? __ldg(row + pair0 + e) : 1.f;
        t.s[e] = e < n ? __ldg(row + rot / 2 + pair0 + e) : 0.f;
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
    __device__ __forceinline__ void set(int u, const Units& n, int rot, const float* row) {
        turned = u < n.rot_units;
        if (turned) {
            if (INTER) {
                f0 = u * (VEC == 1 ? 2 : VEC);
                f1 = f0 + 1;
                two = VEC == 1;
                load_turn<VEC>(t, row, rot, VEC == 1 ? u : u * VEC / 2, VEC == 1 ? 1 : VEC / 2);
            } else {
                f0 = u * VEC;
                f1 = f0 + rot / 2;
                two = true;
                load_turn<VEC>(t, row, rot, f0, VEC);
            }
        } else {
            f0 = rot + (u - n.rot_units) * VEC;
            f1 = 0;
            two = false;
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

// One warp: heads [h0, h1) of token i, in the order q heads, k heads, v heads.
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void token_heads(const AppendArgs& a, int i, int h0, int h1) {
    const Token t = find_token(a, i);
    if (!t.taken) return;
    const PagedCache& c = a.c;
    const int lane = threadIdx.x % 32, P = c.page_size, d = c.d;
    const int page = page_of(c, t.b, t.pos / P);
    const int row = (int)(t.pos % P);
    const float* rope = a.rope ? a.rope + t.pos * a.rot : nullptr;
    const Units n(d, a.rope ? a.rot : 0, INTER, VEC), nv(d, 0, INTER, VEC);
    const int rot = a.rope ? a.rot : 0;
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
                    un.load(hj < a.Hq ? static_cast<const T*>(a.q) + i * a.sq + (long long)hj * d
                                      : static_cast<const T*>(a.k) + i * a.sk + (long long)(hj - a.Hq) * d,
                            ca[j], cb[j]);
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
            const Chunk<T, VEC> ch =
                *reinterpret_cast<const Chunk<T, VEC>*>(static_cast<const T*>(a.v) + i * a.sv + (long long)h * d + f);
            if (paged) *reinterpret_cast<Chunk<T, VEC>*>(vp + (long long)h * P * d + f) = ch;
            if (vdp) *reinterpret_cast<Chunk<T, VEC>*>(vdp + (long long)h * d + f) = ch;
        }
    }
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

template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* dst, const float (&x)[VEC], float inv) {
    Chunk<int8_t, VEC> o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o.x[e] = (int8_t)code_of(x[e], inv);
    *reinterpret_cast<Chunk<int8_t, VEC>*>(dst) = o;
}

// One CTA: the rows of one page that start at token i (the first token of its
// sequence or of a page), for one kv-head, keys (kv = 0) or values.
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void page_run(const AppendArgs& a, int i, const Token& t, int g, int kv, float* red) {
    const PagedCache& c = a.c;
    const int P = c.page_size, d = c.d, tid = threadIdx.x;
    const int page = page_of(c, t.b, t.pos / P);
    const int r0 = (int)(t.pos % P);
    long long rows = min((long long)__ldg(c.cu_q + t.b + 1), (long long)c.N) - i;
    if (rows > P - r0) rows = P - r0;
    if (a.rope && rows > a.rope_len - t.pos) rows = a.rope_len - t.pos;
    const int rot = (kv == 0 && a.rope) ? a.rot : 0;
    const Units n(d, rot, INTER, VEC);
    const T* src = kv ? static_cast<const T*>(a.v) + (long long)g * d : static_cast<const T*>(a.k) + (long long)g * d;
    const long long ss = kv ? a.sv : a.sk;
    T* dep = static_cast<T*>(kv ? a.vd : a.kd);
    const int total = (int)rows * n.total;
    float amax = 0.f;
    for (int x = tid; x < total; x += kWarps * 32) {
        const int r = x / n.total, u = x % n.total;
        Unit<VEC, INTER> un;
        un.set(u, n, rot, rot ? a.rope + (t.pos + r) * a.rot : nullptr);
        Chunk<T, VEC> cp, cq;
        un.load(src + (i + r) * ss, cp, cq);
        float p[VEC], q[VEC];
        un.turn(cp, cq, p, q);
        if (dep) un.store(dep + (((long long)(i + r) * a.Ld + a.slot) * c.Hkv + g) * d, p, q);
#pragma unroll
        for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, finite_abs(p[e]));
        if (un.two)
#pragma unroll
            for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, finite_abs(q[e]));
    }
    if (page < 0) return;  // uniform over the CTA
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float* scales = (kv ? a.v_scale : a.k_scale) + (long long)page * c.Hkv + g;
    const float old = r0 ? *scales : 0.f;
    if (tid % 32 == 0) red[tid / 32] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) amax = fmaxf(amax, red[w]);
    const float now = fmaxf(old, scale_for(amax));
    const float inv = now > 0.f ? 1.f / now : 0.f;  // exact: a power of two
    int8_t* codes = static_cast<int8_t*>(kv ? a.v_pages : a.k_pages) + ((long long)page * c.Hkv + g) * P * d;
    if (r0 && old != now) {
        const float ratio = __fmul_rn(old, inv);
        for (int x = tid; x < r0 * (d / VEC); x += kWarps * 32) {
            Chunk<int8_t, VEC>* at = reinterpret_cast<Chunk<int8_t, VEC>*>(codes + (long long)x * VEC);
            Chunk<int8_t, VEC> ch = *at;
#pragma unroll
            for (int e = 0; e < VEC; ++e) ch.x[e] = (int8_t)code_of((float)ch.x[e], ratio);
            *at = ch;
        }
    }
    for (int x = tid; x < total; x += kWarps * 32) {
        const int r = x / n.total, u = x % n.total;
        Unit<VEC, INTER> un;
        un.set(u, n, rot, rot ? a.rope + (t.pos + r) * a.rot : nullptr);
        Chunk<T, VEC> cp, cq;
        un.load(src + (i + r) * ss, cp, cq);
        float p[VEC], q[VEC];
        un.turn(cp, cq, p, q);
        int8_t* dst = codes + (long long)(r0 + r) * d;
        store_codes<VEC>(dst + un.f0, p, inv);
        if (un.two) store_codes<VEC>(dst + un.f1, q, inv);
    }
    __syncthreads();  // everyone has read the old scale and `red`
    if (tid == 0) *scales = now;
}

// Blocks [0, q_blocks): q heads of the tokens, one warp per share. The rest:
// block x serves the page runs that start in tokens [chunk*x', chunk*(x'+1))
// for one (kv-head, keys or values).
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kWarps * 32)
paged_append_q8_kernel(const AppendArgs a, int shares, int q_blocks, int chunk) {
    if ((int)blockIdx.x < q_blocks) {
        const long long w = (long long)blockIdx.x * kWarps + threadIdx.x / 32;
        if (w / shares >= a.c.N) return;
        const int per = (a.Hq + shares - 1) / shares, h0 = (int)(w % shares) * per;
        if (h0 < a.Hq) token_heads<T, VEC, INTER>(a, (int)(w / shares), h0, min(h0 + per, a.Hq));
        return;
    }
    __shared__ float red[kWarps];
    const int jobs = 2 * a.c.Hkv, x = blockIdx.x - q_blocks;
    const int job = x % jobs;
    const long long i0 = (long long)(x / jobs) * chunk;
    for (int e = 0; e < chunk && i0 + e < a.c.N; ++e) {
        const int i = (int)i0 + e;
        const Token t = find_token(a, i);
        // a run starts where the sequence's new tokens start (counting from
        // the first one with a position) and at each page's first row
        const bool head = t.taken && (t.pos % a.c.page_size == 0 || i == __ldg(a.c.cu_q + t.b) || i == 0);
        if (head) page_run<T, VEC, INTER>(a, i, t, job >> 1, job & 1, red);
    }
}

template <typename T, int VEC, bool INTER>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    const PagedCache& c = a.c;
    const int rot = a.rope ? a.rot : 0;
    const Units n(c.d, rot, INTER, VEC);
    const int per_pass = n.total < 32 ? 32 / n.total : 1;  // heads a warp serves at a time
    const bool q8 = a.k_scale != nullptr;
    const int h_first = a.q ? 0 : a.Hq;
    const int heads = q8 ? (a.q ? a.Hq : 0) : a.Hq + 2 * c.Hkv - h_first;
    // few tokens: split a token's heads until about 16 warps per SM are busy
    int shares = 1;
    while (shares * 2 * per_pass <= heads && (long long)c.N * shares < 148 * 16) shares *= 2;
    const long long blocks = ((long long)c.N * shares + kWarps - 1) / kWarps;
    if (!q8) {
        if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
        paged_append_kernel<T, VEC, INTER><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a, shares, h_first, a.Hq + 2 * c.Hkv);
    } else {
        const int chunk = c.N <= 2048 ? 1 : min(c.page_size, 32);
        const long long q_blocks = a.q ? blocks : 0;
        const long long all = q_blocks + ((long long)c.N + chunk - 1) / chunk * 2 * c.Hkv;
        if (all > 0x7fffffffLL) return cudaErrorInvalidValue;
        paged_append_q8_kernel<T, VEC, INTER><<<(unsigned)all, kWarps * 32, 0, s>>>(a, shares, (int)q_blocks, chunk);
    }
    return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const AppendArgs& a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int rot = a.rope ? a.rot : 0;
    if (a.interleaved) return rot % V ? launch<T, 1, true>(a, s) : launch<T, V, true>(a, s);
    return (rot / 2) % V ? launch<T, 1, false>(a, s) : launch<T, V, false>(a, s);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t s) {
    return a.dtype == MODA_F32 ? pick<float>(a, s) : pick<__nv_bfloat16>(a, s);
}

}  // namespace moda
