// Instructions that only the paged-cache kernels use.
#pragma once

#include <cstdint>

#include "sm100_ptx.cuh"

namespace moda {
namespace ptx {

// Untiled bulk copy into this CTA's shared memory: both addresses 16-byte
// aligned, a multiple of 16 bytes; completion counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// One 32-byte store (a whole sector); the address is 32-byte aligned.
__device__ __forceinline__ void st_global_32b(void* dst, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

}  // namespace ptx
}  // namespace moda
