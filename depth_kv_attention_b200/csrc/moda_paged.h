// Internal declarations of the paged sequence cache (append and attention).
// Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/moda.h"

namespace moda {

// The cache as both operators see it. B sequences; sequence b's new tokens are
// rows cu_q[b] .. cu_q[b+1]-1 of the packed token axis [0, N) and ctx_lens[b]
// counts its tokens with the new ones, so token i sits at position
// ctx_lens[b] - (cu_q[b+1] - i).
struct PagedCache {
    const int32_t* cu_q;         // [B+1]
    const int32_t* ctx_lens;     // [B]
    const int32_t* block_table;  // [B, max_blocks]
    int N, B, Hkv, d;
    int num_pages, page_size, max_blocks;
};

struct AppendArgs {
    PagedCache c;
    const void* q;  // [N, Hq, d], token stride sq; may be null with q_out null
    const void* k;  // [N, Hkv, d], token stride sk
    const void* v;
    long long sq, sk, sv;
    const float* rope;  // [rope_len, rot] cos | sin halves, or null
    int rope_len, rot, interleaved;
    int Hq;
    moda_dtype dtype;
    void* q_out;    // [N, Hq, d] or null
    void* k_pages;  // [num_pages, Hkv, page_size, d]: input dtype, or int8 codes
    void* v_pages;
    float* k_scale;  // 8-bit pages: [num_pages, Hkv], else null
    float* v_scale;
    void* kd;  // [N, Ld, Hkv, d] or null
    void* vd;
    int Ld, slot;
    unsigned int* status;     // device status word
    unsigned int wait_limit;  // bounded-wait polls (0 = default)
};

struct PagedFwdArgs {
    PagedCache c;
    const void* q;  // [N, Hq, d]
    const void* k_pages;
    const void* v_pages;
    const float* k_scale;  // 8-bit pages: [num_pages, Hkv], else null
    const float* v_scale;
    const void* kd;  // [N, Ld_cap, Hkv, d], slots 0 .. Ld-1 are attended to
    const void* vd;
    int Hq, G, Ld, Ld_cap, max_q;
    float scale;
    moda_dtype dtype;
    void* out;   // [N, Hq, d]
    float* lse;  // [N, Hq] or null
    void* workspace;
    unsigned int* status;
    unsigned int wait_limit;
};

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t s);
// Tensor-core attention for few rows per sequence (moda_paged_dec_sm100.cu).
bool paged_dec_supported(const PagedFwdArgs& a);
size_t paged_dec_workspace(int max_q, int G, int d);
cudaError_t launch_paged_dec(const PagedFwdArgs& a, cudaStream_t s);
// tcgen05 attention for many rows per sequence (moda_paged_pre_sm100.cu).
bool paged_pre_supported(const PagedFwdArgs& a);
size_t paged_pre_workspace(const PagedCache& c, bool q8);  // c.max_blocks may be 0: not known
cudaError_t launch_paged_pre(const PagedFwdArgs& a, cudaStream_t s);
// Rows per sequence and kv-head from which it is the one that runs. 48
// sequences of 3000 tokens, 4 kv-heads of 128, in us, this kernel / the other:
// 32 rows 87 / 81 (8-bit pages 162 / 96), 40 rows 87 / 140 (164 / 169), 64 rows
// 90 / 144 (165 / 172), 128 rows 95 / 264 (171 / 323); G = 1 and 8 alike.
constexpr int kPagedPreRows = 33;
// Every shape (moda_paged_simt.cu).
cudaError_t launch_paged_fwd_simt(const PagedFwdArgs& a, cudaStream_t s);

}  // namespace moda
