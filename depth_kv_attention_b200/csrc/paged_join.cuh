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
    const int4* desc;      // [W]: {first row of the sequence, kv-head, tile, parts | rows << 16}, 0: no unit is cut there
    int Hq, G;
    int n;  // tokens of a 128-row tile (rows past n G unused), or 0: rows are (token, head) without gaps
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

// Parts a warp loads at a time, and blocks per SM. A pass is a chain of loads
// (about 1.5 us), so what counts is how many are under way: two parts are the
// rule where units are large and cut once, and batches of four leave room for
// four blocks (148 units of 256 rows: 28 us with two blocks and batches of
// eight). Decode units may have hundreds of parts.
template <int MR>
struct JoinCfg {
    static constexpr int kBatch = MR == 256 ? 4 : 8, kBlocks = MR == 256 ? 4 : 2;
};

template <int MR, int D, int W>
__global__ void __launch_bounds__(kJoinWarps * 32, JoinCfg<MR>::kBlocks) paged_join_kernel(const JoinParams p) {
    constexpr int E = D / 32, kBatch = JoinCfg<MR>::kBatch;
    __shared__ int sums[kJoinWarps], ends[W];
    __shared__ int4 descs[W];
    __shared__ float sml[kJoinWarps][2], so[kJoinWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // running sum of passes over the CTAs: warp w scans kPer of them
    constexpr int kPer = (W + kJoinWarps - 1) / kJoinWarps;
    static_assert(kPer <= 64, "two loads a lane");
    const int at0 = warp * kPer + lane, at1 = at0 + 32;
    const bool in0 = lane < kPer && at0 < W, in1 = lane + 32 < kPer && at1 < W;
    int n0 = 0, n1 = 0;
    if (in0) n0 = join_passes(descs[at0] = p.desc[at0]);
    if (in1) n1 = join_passes(descs[at1] = p.desc[at1]);
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
        int x = 0;  // first CTA whose running sum passes the item
#pragma unroll
        for (int w = 0; w < W; w += 32)
            x += __popc(__ballot_sync(0xffffffffu, w + lane < W && ends[min(w + lane, W - 1)] <= item));
        const int4 ds = descs[x];
        const int parts = ds.w & 0xffff, rows = ds.w >> 16;
        const int pass = item - (x ? ends[x - 1] : 0);
        const bool shared = parts > kShareParts;
        const int r = shared ? pass : pass * kJoinWarps + warp;
        // row r of the tile: token and head
        const int rr = p.n ? r & 127 : ds.z * MR + r;
        const int tok = p.n ? (2 * ds.z + (r >> 7)) * p.n + rr / p.G : rr / p.G;
        const bool there = r < rows && (!p.n || rr < p.n * p.G);
        auto slot = [&](int i) { return (long long)(i == 0 ? 2 * x + 1 : 2 * (x + i)) * MR + r; };
        float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        if (there) {
            // all loads of a batch in flight together
            const int step = shared ? kJoinWarps : 1;
            for (int i0 = shared ? warp : 0; i0 < parts; i0 += kBatch * step) {
                float2 ml[kBatch];
                float v[kBatch][E];
                float mn = m;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * step;
                    ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[k][e] = 0.f;
                    if (i < parts) {
                        ml[k] = *reinterpret_cast<const float2*>(p.part_ml + slot(i) * 2);
                        const float* po = p.part_o + slot(i) * D + lane * E;
                        if (E == 4) {
                            const float4 f = *reinterpret_cast<const float4*>(po);
                            v[k][0] = f.x; v[k][1] = f.y; v[k][E - 2] = f.z; v[k][E - 1] = f.w;
                        } else {
                            const float2 f = *reinterpret_cast<const float2*>(po);
                            v[k][0] = f.x; v[k][1] = f.y;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ml[k].x);
                const float ref = mn == -INFINITY ? 0.f : mn, corr = ptx::ex2(m - ref);
                l *= corr;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] *= corr;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const float w = ptx::ex2(ml[k].x - ref);
                    l += ml[k].y * w;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += v[k][e] * w;
                }
                m = mn;
            }
        }
        if (shared) {  // the eight warps' sums, in their order
#pragma unroll
            for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
            if (lane == 0) {
                sml[warp][0] = m;
                sml[warp][1] = l;
            }
            __syncthreads();
            if (warp == 0) {
                m = -INFINITY;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sml[w][0]);
                const float ref = m == -INFINITY ? 0.f : m;
                l = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) {
                    const float c = ptx::ex2(sml[w][0] - ref);
                    l += sml[w][1] * c;
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] += so[w][lane * E + e] * c;
                }
            }
            __syncthreads();
        }
        if (there && (!shared || warp == 0)) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long orow = (long long)(ds.x + tok) * p.Hq + ds.y * p.G + rr % p.G;
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
    cfg.gridDim = dim3(JoinCfg<MR>::kBlocks * 148);
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
