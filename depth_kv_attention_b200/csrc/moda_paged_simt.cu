// Scalar (SIMT, fp32 FMA) attention over the paged sequence cache: the path
// for fp32 and for the shapes the tensor-core kernels do not take (pages that
// are no multiple of 16 rows, d no multiple of 8).
//
// One softmax over the token's visible sequence keys and its own depth keys
// ("动态混合深度注意力机制MoDA技术解析", mhpn.cn, §1.2 formula; §2.2 online softmax
// state and the dual mask). One CTA per (token, query head); eight lanes share
// a key (four consecutive features of every 32 each), so a warp works on four
// keys at once, each lane group with its own running (m, l, o). The states are
// joined by shuffles within a warp and through shared memory across warps.
// Only visible keys are touched, so nothing masked can reach a sum.
#include <cuda_bf16.h>

#include <cmath>

#include "paged_common.cuh"

namespace moda {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDMax = 128;
constexpr int kMaxWarps = 16;

template <typename T>
struct alignas(sizeof(T) * 4) Four {
    T x[4];
};

// Features 32c + 4l .. +3 of a row, c = 0..3 (zero past d; d % 4 == 0).
template <typename T>
__device__ __forceinline__ void load16(const T* row, int d, int l, float (&x)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int f = 32 * c + 4 * l;
        Four<T> v;
        if (f < d) v = *reinterpret_cast<const Four<T>*>(row + f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * c + e] = f < d ? pg_to_f(v.x[e]) : 0.f;
    }
}

struct State {
    float m, l, o[16];
    // One key with logit s (log2 domain) and values v.
    __device__ __forceinline__ void add(float s, const float (&v)[16]) {
        const float mn = fmaxf(m, s);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float corr = exp2f(m - ref), p = exp2f(s - ref);
        l = l * corr + p;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = fmaf(o[e], corr, p * v[e]);
        m = mn;
    }
    __device__ __forceinline__ void join_lanes(int mask) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, mask), l2 = __shfl_xor_sync(0xffffffffu, l, mask);
        const float mn = fmaxf(m, m2);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float c1 = exp2f(m - ref), c2 = exp2f(m2 - ref);
        l = l * c1 + l2 * c2;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = o[e] * c1 + __shfl_xor_sync(0xffffffffu, o[e], mask) * c2;
        m = mn;
    }
};

template <typename T, typename KV>
__global__ void __launch_bounds__(kMaxWarps * 32) paged_fwd_simt_kernel(const PagedFwdArgs a) {
    __shared__ float sm[kMaxWarps], sl[kMaxWarps], so[kMaxWarps][kDMax];
    const PagedCache& c = a.c;
    const int i = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, g = h / a.G, d = c.d, P = c.page_size;
    const int b = seq_of_token(c, i);
    if (b >= c.B || i < __ldg(c.cu_q + b)) return;  // a row of no sequence stays as it was
    const long long pos = (long long)__ldg(c.ctx_lens + b) - ((long long)__ldg(c.cu_q + b + 1) - i);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
    const int grp = warp * 4 + lane / 8, groups = warps * 4, l8 = lane % 8;
    float q[16];
    load16(static_cast<const T*>(a.q) + ((long long)i * a.Hq + h) * d, d, l8, q);
    const float sl2 = a.scale * kLog2e;
    State st;
    st.m = -INFINITY;
    st.l = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) st.o[e] = 0.f;
    auto dot = [&](const float (&k)[16]) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s = fmaf(q[e], k[e], s);
        // the eight lanes of a key take part together (their loop bounds are equal)
        const unsigned lanes = 0xffu << (lane & 24);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(lanes, s, o);
        return s * sl2;
    };
    const long long nk = min(pos + 1, (long long)c.max_blocks * P);
    for (long long j = grp; j < nk; j += groups) {
        const int page = page_of(c, b, j / P);
        if (page < 0) continue;
        const long long hrow = (long long)page * c.Hkv + g, at = (hrow * P + j % P) * d;
        float k[16], v[16];
        load16(static_cast<const KV*>(a.k_pages) + at, d, l8, k);
        load16(static_cast<const KV*>(a.v_pages) + at, d, l8, v);
        float s = dot(k);
        if (a.k_scale) {
            s *= __ldg(a.k_scale + hrow);
            const float sv = __ldg(a.v_scale + hrow);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= sv;
        }
        st.add(s, v);
    }
    for (int x = grp; x < a.Ld; x += groups) {
        const long long at = (((long long)i * a.Ld_cap + x) * c.Hkv + g) * d;
        float k[16], v[16];
        load16(static_cast<const T*>(a.kd) + at, d, l8, k);
        load16(static_cast<const T*>(a.vd) + at, d, l8, v);
        st.add(dot(k), v);
    }
    __syncwarp();
    st.join_lanes(8);
    st.join_lanes(16);
    if (lane < 8) {
#pragma unroll
        for (int e = 0; e < 16; ++e) so[warp][32 * (e / 4) + 4 * l8 + e % 4] = st.o[e];
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

}  // namespace

cudaError_t launch_paged_fwd_simt(const PagedFwdArgs& a, cudaStream_t s) {
    const PagedCache& c = a.c;
    const long long grid = (long long)c.N * a.Hq;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    // a warp takes four keys at a time: about eight rounds before more warps help
    const long long keys = (long long)c.max_blocks * c.page_size;
    int warps = 2;
    while (warps < kMaxWarps && keys > (long long)warps * 32) warps *= 2;
    const unsigned th = warps * 32;
    if (a.dtype == MODA_F32) {
        if (a.k_scale) paged_fwd_simt_kernel<float, int8_t><<<(unsigned)grid, th, 0, s>>>(a);
        else paged_fwd_simt_kernel<float, float><<<(unsigned)grid, th, 0, s>>>(a);
    } else {
        if (a.k_scale) paged_fwd_simt_kernel<__nv_bfloat16, int8_t><<<(unsigned)grid, th, 0, s>>>(a);
        else paged_fwd_simt_kernel<__nv_bfloat16, __nv_bfloat16><<<(unsigned)grid, th, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace moda
