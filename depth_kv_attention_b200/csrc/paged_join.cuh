// Joining the parts of work units that the paged attention kernels cut (see
// paged_units.cuh).
#pragma once

#include <cmath>
#include <cstring>

#include "paged_units.cuh"
#include "sm100_ptx.cuh"
#include "smem_limit.h"

namespace moda {

struct JoinParams {
    PagedCache c;
    __nv_bfloat16* out;
    float* lse;
    const float* part_o;   // [2W][MR][D]: CTA x's first part in 2x, its last (the start of a unit) in 2x + 1
    const float* part_ml;  // [2W][MR][2]
    const int4* desc;      // [W]: {sequence, kv-head, tile, parts | rows << 16}, 0: no unit is cut there
    int Hq, G;
};

// Joins the parts of cut units, always in their order. Every block lists the
// cut units (CTA x of the attention wrote the first part of desc[x]'s) and
// takes its share of the passes over them: a pass is eight rows with a warp
// each, or, with many parts, one row whose parts eight warps share.
constexpr int kJoinWarps = 8;
constexpr int kShareParts = 8;  // more parts than this: eight warps a row

__device__ __forceinline__ int join_passes(const int4& ds) {
    const int parts = ds.w & 0xffff, rows = ds.w >> 16;
    return parts == 0 ? 0 : parts > kShareParts ? rows : (rows + kJoinWarps - 1) / kJoinWarps;
}

template <int MR, int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const JoinParams p) {
    constexpr int E = D / 32;
    __shared__ int sums[kJoinWarps + 1], ends[W];
    __shared__ float sml[kJoinWarps][2], so[kJoinWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // running sum of passes over the CTAs: warp w scans kPer of them
    constexpr int kPer = (W + kJoinWarps - 1) / kJoinWarps;
    static_assert(kPer <= 64, "two loads a lane");
    const int at0 = warp * kPer + lane, at1 = at0 + 32;
    const bool in0 = lane < kPer && at0 < W, in1 = lane + 32 < kPer && at1 < W;
    const int n0 = in0 ? join_passes(p.desc[at0]) : 0, n1 = in1 ? join_passes(p.desc[at1]) : 0;
    int i0 = n0, i1 = n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v0 = __shfl_up_sync(0xffffffffu, i0, o), v1 = __shfl_up_sync(0xffffffffu, i1, o);
        if (lane >= o) {
            i0 += v0;
            i1 += v1;
        }
    }
    i1 += __shfl_sync(0xffffffffu, i0, 31);
    if (lane == 31) sums[warp] = i1;
    __syncthreads();
    int pre = 0;
    for (int w = 0; w < warp; ++w) pre += sums[w];
    if (in0) ends[at0] = pre + i0;
    if (in1) ends[at1] = pre + i1;
    __syncthreads();
    const int all = ends[W - 1];
    for (int item = blockIdx.x; item < all; item += gridDim.x) {
        int lo = 0, hi = W - 1;  // first CTA whose running sum passes the item
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (ends[mid] <= item) lo = mid + 1; else hi = mid;
        }
        const int x = lo;
        const int4 ds = p.desc[x];
        const int parts = ds.w & 0xffff, rows = ds.w >> 16;
        const int pass = item - (x ? ends[x - 1] : 0);
        const bool shared = parts > kShareParts;
        const int r = shared ? pass : pass * kJoinWarps + warp;
        const int row = ds.z * MR + r;
        auto slot = [&](int i) { return (long long)(i == 0 ? 2 * x + 1 : 2 * (x + i)) * MR + r; };
        float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        if (r < rows) {
            for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[slot(i) * 2]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll 8
            for (int i = shared ? warp : 0; i < parts; i += shared ? kJoinWarps : 1) {
                const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(i) * 2);
                const float w = ptx::ex2(ml.x - ref);
                const float* po = p.part_o + slot(i) * D + lane * E;
                l += ml.y * w;
                if (E == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(po);
                    acc[0] += v.x * w; acc[1] += v.y * w; acc[E - 2] += v.z * w; acc[E - 1] += v.w * w;
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(po);
                    acc[0] += v.x * w; acc[1] += v.y * w;
                }
            }
        }
        if (shared) {  // the eight warps' sums, in their order
#pragma unroll
            for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
            if (lane == 0) sml[warp][1] = l;
            __syncthreads();
            l = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.f;
            if (warp == 0)
                for (int w = 0; w < kJoinWarps; ++w) {
                    l += sml[w][1];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += so[w][lane * E + e];
                }
            __syncthreads();
        }
        if (r < rows && (!shared || warp == 0)) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const SeqInfo sq = seq_info(p.c, ds.x);
            const long long orow = (long long)(sq.q0 + row / p.G) * p.Hq + ds.y * p.G + row % p.G;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                if (lane * E + e < p.c.d)
                    *reinterpret_cast<uint32_t*>(p.out + orow * p.c.d + lane * E + e) =
                        ptx::pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
            if (lane == 0 && p.lse) p.lse[orow] = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
        }
    }
}

template <int MR, int D, int W>
cudaError_t launch_paged_join(const JoinParams& p, cudaStream_t s) {
    // launched while the attention drains; waits for its end on the device
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(2 * 148);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<MR, D, W>, p);
}

}  // namespace moda
