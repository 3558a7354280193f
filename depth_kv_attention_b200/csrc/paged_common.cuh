// Where a token of the packed axis lives in the paged cache, shared by the
// append and the attention kernels.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "moda_paged.h"

namespace moda {

__device__ __forceinline__ float pg_to_f(float x) { return x; }
__device__ __forceinline__ float pg_to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float pg_to_f(int8_t x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T pg_from_f(float x);
template <>
__device__ __forceinline__ float pg_from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 pg_from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Number of sequences whose tokens all lie before token i, i.e. the sequence
// of token i when cu_q is non-decreasing; B when no sequence holds it. Called
// by whole warps; the count of a ballot costs one load per 32 sequences, all
// in flight together, against a chain of log2(B) dependent loads.
__device__ __forceinline__ int seq_of_token(const PagedCache& c, int i) {
    const int lane = threadIdx.x % 32;
    int b = 0;
    if (c.B <= 1024) {
        for (int s = 0; s < c.B; s += 32) {
            const bool before = s + lane < c.B && __ldg(c.cu_q + s + lane + 1) <= i;
            b += __popc(__ballot_sync(0xffffffffu, before));
        }
    } else {
        int lo = 0, hi = c.B;  // first sequence whose end lies behind i
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (__ldg(c.cu_q + mid + 1) <= i) lo = mid + 1; else hi = mid;
        }
        b = lo;
    }
    return b;
}

// Page of block `blk` of sequence b, or -1 when the table does not reach that
// far or holds no page of the pool there.
__device__ __forceinline__ int page_of(const PagedCache& c, int b, long long blk) {
    if (blk < 0 || blk >= c.max_blocks) return -1;
    const int p = __ldg(c.block_table + (long long)b * c.max_blocks + blk);
    return p >= 0 && p < c.num_pages ? p : -1;
}

}  // namespace moda
