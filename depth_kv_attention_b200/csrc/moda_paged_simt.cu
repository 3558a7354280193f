// Scalar (SIMT, fp32 FMA) attention over the paged sequence cache: the path
// for fp32 and for the shapes the tensor-core kernels do not take (pages that
// are no multiple of 16 rows, 8-bit pages with d no multiple of 16).
//
// One softmax over the token's visible sequence keys and its own depth keys
// ("动态混合深度注意力机制MoDA技术解析", mhpn.cn, §1.2 formula; §2.2 online softmax
// state and the dual mask). One CTA per (token, query head); eight lanes share
// a key (four consecutive features of every 32 each), each lane group has two
// keys in flight and its own running (m, l, o), so a warp works on eight keys
// at once. Small calls are a chain of loads (four short sequences, one token each: 6 us);
// larger ones are bound by instructions, about 50 per key and lane. The states are
// joined by shuffles within a warp and through shared memory across warps.
// Only visible keys are touched, so nothing masked can reach a sum.
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "paged_common.cuh"

namespace moda {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDMax = 128;
constexpr int kMaxWarps = 16;
constexpr int kKeys = 2;  // keys a lane group has in flight

template <typename T>
struct alignas(sizeof(T) * 4) Four {
    T x[4];
};

// Features 32c + 4l .. +3 of a row, c < F / 4 (zero past d; d % 4 == 0).
template <int F, typename T>
__device__ __forceinline__ void load_row(const T* row, int d, int l, T (&x)[F]) {
#pragma unroll
    for (int c = 0; c < F / 4; ++c) {
        const int f = 32 * c + 4 * l;
        Four<T> v{};
        if (f < d) v = *reinterpret_cast<const Four<T>*>(row + f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * c + e] = v.x[e];
    }
}

// F features a lane: 8 for d <= 64, else 16.
template <int F>
struct State {
    float m, l, o[F];
    // Keys with logits s (log2 domain) and values v times sv; a logit of -inf
    // adds nothing (its values are zeros then).
    template <typename KV>
    __device__ __forceinline__ void add(const float (&s)[kKeys], const KV (&v)[kKeys][F], const float (&sv)[kKeys]) {
        float mn = m;
#pragma unroll
        for (int u = 0; u < kKeys; ++u) mn = fmaxf(mn, s[u]);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float corr = exp2f(m - ref);
        l *= corr;
#pragma unroll
        for (int e = 0; e < F; ++e) o[e] *= corr;
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const float p = exp2f(s[u] - ref), pv = p * sv[u];
            l += p;
#pragma unroll
            for (int e = 0; e < F; ++e) o[e] = fmaf(pv, pg_to_f(v[u][e]), o[e]);
        }
        m = mn;
    }
    __device__ __forceinline__ void join_lanes(int mask) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, mask), l2 = __shfl_xor_sync(0xffffffffu, l, mask);
        const float mn = fmaxf(m, m2);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float c1 = exp2f(m - ref), c2 = exp2f(m2 - ref);
        l = l * c1 + l2 * c2;
#pragma unroll
        for (int e = 0; e < F; ++e) o[e] = o[e] * c1 + __shfl_xor_sync(0xffffffffu, o[e], mask) * c2;
        m = mn;
    }
};

template <typename T, typename KV, int F>
__global__ void __launch_bounds__(kMaxWarps * 32) paged_fwd_simt_kernel(const PagedFwdArgs a) {
    __shared__ float sm[kMaxWarps], sl[kMaxWarps], so[kMaxWarps][kDMax];
    const PagedCache& c = a.c;
    const int i = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, g = h / a.G, d = c.d, P = c.page_size;
    const int b = seq_of_token(c, i);
    if (b >= c.B || i < __ldg(c.cu_q + b)) return;  // a row of no sequence stays as it was
    const long long pos = (long long)__ldg(c.ctx_lens + b) - ((long long)__ldg(c.cu_q + b + 1) - i);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const int grp = warp * 4 + lane / 8, groups = warps * 4, l8 = lane % 8;
    T q[F];
    load_row(static_cast<const T*>(a.q) + ((long long)i * a.Hq + h) * d, d, l8, q);
    const float sl2 = a.scale * kLog2e;
    State<F> st;
    st.m = -INFINITY;
    st.l = 0.f;
#pragma unroll
    for (int e = 0; e < F; ++e) st.o[e] = 0.f;
    // One step: keys `on` says, their rows at k + at[u] and v + at[u].
    auto step = [&](const auto* k, const auto* v, const long long (&at)[kKeys], const bool (&on)[kKeys],
                    const float (&ks)[kKeys], const float (&vs)[kKeys]) {
        using KT = std::remove_cv_t<std::remove_pointer_t<decltype(k)>>;
        KT kx[kKeys][F] = {}, vx[kKeys][F] = {};
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
            if (on[u]) load_row(k + at[u], d, l8, kx[u]);
#pragma unroll
        for (int u = 0; u < kKeys; ++u)
            if (on[u]) load_row(v + at[u], d, l8, vx[u]);
        float s[kKeys];
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < F; ++e) s[u] = fmaf(pg_to_f(q[e]), pg_to_f(kx[u][e]), s[u]);
        }
        // the eight lanes of a key take part together (their loop bounds are equal)
        const unsigned lanes = 0xffu << (lane & 24);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int u = 0; u < kKeys; ++u) s[u] += __shfl_xor_sync(lanes, s[u], o);
#pragma unroll
        for (int u = 0; u < kKeys; ++u) s[u] = on[u] ? s[u] * ks[u] : -INFINITY;
        st.add(s, vx, vs);
    };
    long long at[kKeys];
    bool on[kKeys];
    float ks[kKeys], vs[kKeys];
    // positions are below 2^31, steps of kKeys * groups <= 128 keep j below 2^32
    const unsigned nk = (unsigned)max(0LL, min(pos + 1, (long long)c.max_blocks * P));
    for (unsigned j = grp; j < nk; j += kKeys * groups) {
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            const unsigned ju = j + u * groups, blk = ju / (unsigned)P;
            const int page = ju < nk ? page_of(c, b, blk) : -1;
            const long long hrow = (long long)max(page, 0) * c.Hkv + g;
            on[u] = page >= 0;
            at[u] = (hrow * P + (ju - blk * P)) * d;
            ks[u] = sl2;
            vs[u] = 1.f;
            if (a.k_scale && on[u]) {
                ks[u] *= __ldg(a.k_scale + hrow);
                vs[u] = __ldg(a.v_scale + hrow);
            }
        }
        step(static_cast<const KV*>(a.k_pages), static_cast<const KV*>(a.v_pages), at, on, ks, vs);
    }
    for (int x = grp; x < a.Ld; x += kKeys * groups) {
#pragma unroll
        for (int u = 0; u < kKeys; ++u) {
            on[u] = x + u * groups < a.Ld;
            at[u] = (((long long)i * a.Ld_cap + x + u * groups) * c.Hkv + g) * d;
            ks[u] = sl2;
            vs[u] = 1.f;
        }
        step(static_cast<const T*>(a.kd), static_cast<const T*>(a.vd), at, on, ks, vs);
    }
    __syncwarp();
    st.join_lanes(8);
    st.join_lanes(16);
    if (lane < 8) {
#pragma unroll
        for (int e = 0; e < F; ++e) so[warp][32 * (e / 4) + 4 * l8 + e % 4] = st.o[e];
        if (lane == 0) {
            sm[warp] = st.m;
            sl[warp] = st.l;
        }
    }
    __syncthreads();
    float m = -INFINITY, l = 0.f;
    for (int w = 0; w < warps; ++w) m = fmaxf(m, sm[w]);
    const float ref = m == -INFINITY ? 0.f : m;
    for (int w = 0; w < warps; ++w) l += sl[w] * exp2f(sm[w] - ref);
    // an empty row (nothing visible): zeros and lse = -inf
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int f = threadIdx.x; f < d; f += blockDim.x) {
        float o = 0.f;
        for (int w = 0; w < warps; ++w) o += so[w][f] * exp2f(sm[w] - ref);
        static_cast<T*>(a.out)[((long long)i * a.Hq + h) * d + f] = pg_from_f<T>(o * inv);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[(long long)i * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename T, typename KV>
void launch(const PagedFwdArgs& a, unsigned grid, unsigned th, cudaStream_t s) {
    if (a.c.d <= 64) paged_fwd_simt_kernel<T, KV, 8><<<grid, th, 0, s>>>(a);
    else paged_fwd_simt_kernel<T, KV, 16><<<grid, th, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_paged_fwd_simt(const PagedFwdArgs& a, cudaStream_t s) {
    const PagedCache& c = a.c;
    const long long grid = (long long)c.N * a.Hq;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    // a warp takes eight keys at a time: up to four rounds before more warps
    // help, and no more of them than keep the SMs busy: rows beside each other
    // hide each other's joins (160 tokens of 8 heads over 1018 keys: 104 us with
    // 16 warps a row, 84 with two)
    const long long keys = (long long)c.max_blocks * c.page_size;
    int warps = 2;
    while (warps < kMaxWarps && keys > (long long)warps * 32 && grid * warps < 148 * 16) warps *= 2;
    const unsigned th = warps * 32;
    if (a.dtype == MODA_F32) {
        if (a.k_scale) launch<float, int8_t>(a, (unsigned)grid, th, s);
        else launch<float, float>(a, (unsigned)grid, th, s);
    } else {
        if (a.k_scale) launch<__nv_bfloat16, int8_t>(a, (unsigned)grid, th, s);
        else launch<__nv_bfloat16, __nv_bfloat16>(a, (unsigned)grid, th, s);
    }
    return cudaGetLastError();
}

}  // namespace moda
