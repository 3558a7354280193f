// Attention over the paged sequence cache for few query rows per sequence
// (decode, drafted tokens, ragged mixes): bf16 or 8-bit pages, d <= 128.
//
// What it computes: one softmax over the sequence keys a new token sees and
// its own depth keys ("动态混合深度注意力机制MoDA技术解析", mhpn.cn, §1.2 formula,
// §2.2 online-softmax state and dual mask), all heads of a GQA group together.
//
// What bounds it: a token's G rows share every key, so a step reads K and V
// once and does 4 G d operations per key and head: memory-bound up to about
// G * tokens = 64. (From 33 rows on the tcgen05 kernel is the faster one, so
// this one has tiles of up to 32.) The design keeps loads in flight and everything else out of
// the way:
//  * The stages of all units (paged_units.cuh) are cut into equal parts, two or
//    three CTAs per SM; cut units leave (m, l, O) in the workspace and a small
//    second kernel joins them in a fixed order.
//  * One producer warp fills a ring of K and V slots (64 or 128 keys) by TMA, one box of
//    16 rows per page slice, so any page size that is a multiple of 16 works;
//    page ids and scales are fetched 32 slices at a time, one batch ahead.
//  * The products are mma.sync m16n8k16 with the KEYS as the 16 rows (S^T = K Q^T,
//    O^T = V^T P^T): query rows then come in eights, which is what a decode step
//    has (G heads of a token), where a tcgen05 tile would be 128 rows high. Four
//    consumer warps, each with its own keys of a stage and its own softmax state,
//    joined at the unit's end; with 32 rows two of them take 16 rows each of the
//    same keys. Up to 8 rows three CTAs fit an SM, else two. For d > 64 that
//    takes some spills: 92 and 180 bytes of stores a thread with 16 and 32 rows,
//    over 8-bit pages 84, 308 and 308 with 8, 16 and 32. P^T is
//    what the second product wants as its B operand, once its 8 x 8 blocks are
//    transposed between lanes (movmatrix).
//  * 8-bit pages: a lane reads whole 16-byte pieces of a row and turns codes
//    into bf16 exactly, two at a time with two instructions (codes_to_bf16). The
//    order in which a lane holds features is free in a product's contracted
//    index (queries are laid out alike) and only permutes the output rows.
//    A key's scale multiplies its logit, a value's scale its codes or its P
//    (code_factor, p_factor): all exact, as scales are powers of two.
//  * Rounding: logits, P, l, O in fp32; P is rounded to bf16 as the operand of
//    P V (l sums the unrounded P).
//  * A value that a row must not see may be anything: a masked P is exactly 0,
//    but 0 * NaN is not. Stages in which some row is masked look for
//    non-finite values, add those to the rows that do see them on the CUDA
//    cores and clear them before the product.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "paged_join.cuh"
#include "paged_units.cuh"
#include "sm100_ptx.cuh"
#include "tmap_host.h"

namespace moda {
namespace {

constexpr int kSliceRows = 16;
constexpr float kLazy = 8.f;                    // log2 units before a running max moves

struct DecParams {
    CUtensorMap tm_k, tm_v, tm_kd, tm_vd;
    PagedCache c;
    const __nv_bfloat16* q;
    const float* k_scale;
    const float* v_scale;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;   // [2W][MR][D]
    float* part_ml;  // [2W][MR][2]
    int4* desc;      // [W]: as in JoinParams
    int Hq, G, Ld, DSL, W;
    int split;       // units may be cut (else each stays with one CTA)
    float sl2;
    unsigned int* status;
    unsigned int wait_limit;
};

constexpr int kSeqs = 64;    // sequences whose lengths are kept in shared memory
constexpr int kCtl = 2048;   // barriers and those

// NH: 64-feature halves of a row; NR: 8-row tiles of a warp; WR: warps along the
// query rows, the others split the keys.
template <bool Q8, int NH, int NR, int WR>
struct Cfg {
    static constexpr int D = 64 * NH;
    static constexpr int kWarps = 4;                         // consumers
    static constexpr int kPerSM = NR == 1 ? 3 : 2;           // CTAs
    static constexpr int kParts = kPerSM * 148;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int MR = 8 * NR * WR;
    static constexpr int WK = kWarps / WR;                   // warps that share a stage's keys
    static constexpr int SL = WR == 2 || Q8 ? 2 : 1;  // slices of a stage per warp
    static constexpr int SPS = SL * WK;                      // slices of a stage
    static constexpr int KEYS = 16 * SPS;
    static constexpr int kSeqSlice = Q8 ? 2048 : 2048 * NH;  // bytes of 16 keys
    static constexpr int kDepSlice = 2048 * NH;
    static constexpr int kSlot = SPS * kSeqSlice;
    static constexpr int DS = kSlot / kDepSlice;             // depth slices per stage
    static constexpr int NS = kSlot == 8192 ? 8 : kSlot == 16384 ? (kPerSM == 3 ? 4 : 5) : 3;  // ring slots
    static constexpr int kMergeBufs = WK / 2 * WR;
    static constexpr int kMergeFloats = 8 * NR * D;
    static constexpr int kSmem = 1024 + NS * kSlot + kMergeBufs * kMergeFloats * 4 + kCtl;
};

struct __align__(8) DecBars {
    uint64_t full[8], empty[8];
    float scale[8][8];   // per slot and slice. Keys: scale (1 for bf16), -1: no page; values: factor of P
    uint32_t code_mul[8][8];  // 8-bit values: factor of the codes
    float ml[4][16][2];
    long long scan[9];
    long long begin_in_seq;
    int begin_seq;
    int abort_flag;
    SeqInfo seqs[kSeqs];
};
static_assert(sizeof(DecBars) <= kCtl, "barrier block");

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 0x00800080 in a register that the compiler does not see through: with two
// constants (w ^ m) & c would be two instructions.
__device__ __forceinline__ uint32_t magic_reg() {
    uint32_t r;
    asm volatile("mov.u32 %0, 0x00800080;" : "=r"(r));
    return r;
}
// Two int8 codes c, in bytes 0 and 2 of w, as a bf16 pair c / kCodeUnit (exact):
// the bits 0 .. 255 are the bf16 numbers u 2^-133 (subnormal below 128, one
// binade above), so u = c + 128 needs one fused multiply-add by 2^127.
constexpr float kCodeUnit = 64.f;
constexpr uint32_t kCodeMul = 0x7f007f00u, kCodeOff = 0xc000c000u;  // 2^127, -2
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t w, uint32_t magic, uint32_t mul = kCodeMul, uint32_t off = kCodeOff) {
    uint32_t u, o;
    asm("lop3.b32 %0, %1, %2, 0x00ff00ff, 0x28;" : "=r"(u) : "r"(w), "r"(magic));  // (w ^ magic) & m
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o) : "r"(u), "r"(mul), "r"(off));
    return o;
}
// A page's value scale s, 0 or a power of two, as a factor of its codes and one
// of P, of which one is 1. A scale below one goes to the codes, with the
// fused multiply-add that converts them anyway (by 2^127 s and -2 s): c s / 64 is
// exact in bf16 for every s >= 2^-126. As a factor of P it would leave P few bits,
// or none, where s is small: P s is rounded to bf16, whose step is 2^-133 there.
// A scale of one and more goes to P. The producer splits the scale (64 sequences
// up to 8K: 73.0 us, 74.3 with the split in the consumers, 72.3 with all of it on P).
__device__ __forceinline__ uint32_t code_factor(float s) {  // 2^127 min(s, 1) as a bf16 pair
    const uint32_t e = __bfloat16_as_ushort(__float2bfloat16_rn(s > 0.f ? fminf(s, 1.f) : 1.f));
    return (e + (127u << 7)) * 0x10001u;
}
__device__ __forceinline__ float p_factor(float s) { return s > 0.f ? fmaxf(s, 1.f) : 0.f; }

// Byte address of feature f of row r of a bf16 slice (64-feature halves of 16
// rows, 128-byte swizzle).
__device__ __forceinline__ uint32_t bf16_at(uint32_t slice, int r, int f) {
    return slice + (f >> 6) * 2048 + r * 128 + ((((f >> 3) & 7) ^ (r & 7)) << 4) + (f & 7) * 2;
}

// S^T += K Q^T of one 16-key slice: keys g, g + 8 of a lane's fragment, query
// rows 2t, 2t + 1 of each 8-row tile.
template <int NH, int NR>
__device__ __forceinline__ void qk_bf16(uint32_t slice, const uint32_t (&qf)[NR][NH * 4][2], float (&s)[NR][4], int lane) {
    const int r = lane & 15, hi = lane >> 4;
#pragma unroll
    for (int k = 0; k < NH * 4; ++k) {
        uint32_t a[4];
        ldsm4(bf16_at(slice, r, 16 * k + 8 * hi), a);
#pragma unroll
        for (int x = 0; x < NR; ++x) mma_bf16(s[x], a[0], a[1], a[2], a[3], qf[x][k][0], qf[x][k][1]);
    }
}
// O^T += V^T P^T: output tile m = features 16 m + g, + 8.
template <int NH, int NR>
__device__ __forceinline__ void pv_bf16(uint32_t slice, const uint32_t (&pf)[NR][2], float (&o)[NR][NH * 4][4], int lane) {
    const int r = (lane & 7) + ((lane >> 4) << 3), hi = (lane >> 3) & 1;
#pragma unroll
    for (int m = 0; m < NH * 4; ++m) {
        uint32_t a[4];
        ldsm4t(bf16_at(slice, r, 16 * m + 8 * hi), a);
#pragma unroll
        for (int x = 0; x < NR; ++x) mma_bf16(o[x][m], a[0], a[1], a[2], a[3], pf[x][0], pf[x][1]);
    }
}

// 8-bit kernels hold features permuted: lane t of a quad owns features
// t * D/4 .. of a key; k-step s takes its features 4s, 4s+2 and 4s+1, 4s+3.
// Output tile m, row g / g + 8 = feature g * D/8 + 2m / + 1.
template <int NH, int NR>
__device__ __forceinline__ void qk_q8(uint32_t slice, const uint32_t (&qf)[NR][NH * 4][2], float (&s)[NR][4], int lane,
                                      uint32_t magic) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < NH; ++c) {  // 16 codes = 4 k-steps
        const uint32_t at = slice + g * 128 + (((t * NH + c) ^ g) << 4);
        const uint4 w0 = lds128(at), w1 = lds128(at + 1024);  // keys g, g + 8
        const uint32_t a[4] = {w0.x, w0.y, w0.z, w0.w}, b[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = codes_to_bf16(a[e], magic), a1 = codes_to_bf16(b[e], magic);
            const uint32_t a2 = codes_to_bf16(a[e] >> 8, magic), a3 = codes_to_bf16(b[e] >> 8, magic);
#pragma unroll
            for (int x = 0; x < NR; ++x) mma_bf16(s[x], a0, a1, a2, a3, qf[x][4 * c + e][0], qf[x][4 * c + e][1]);
        }
    }
}
template <int NH, int NR>
__device__ __forceinline__ void pv_q8(uint32_t slice, const uint32_t (&pf)[NR][2], float (&o)[NR][NH * 4][4], int lane,
                                      uint32_t magic, uint32_t mul) {
    const uint32_t off = mul + (kCodeOff - kCodeMul);  // -2 s beside 2^127 s
    const int g = lane >> 2, t = lane & 3;
    uint32_t w[4][NH * 2];  // 8 NH codes of keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int r = 2 * t + (x & 1) + 8 * (x >> 1);
        if (NH == 2) {
            const uint4 v = lds128(slice + r * 128 + ((g ^ (r & 7)) << 4));
            w[x][0] = v.x; w[x][1] = v.y; w[x][NH * 2 - 2] = v.z; w[x][NH * 2 - 1] = v.w;
        } else {
            const uint2 v = lds64(slice + r * 128 + (((g >> 1) ^ (r & 7)) << 4) + (g & 1) * 8);
            w[x][0] = v.x; w[x][1] = v.y;
        }
    }
#pragma unroll
    for (int m = 0; m < NH * 4; ++m) {
        const int q = m >> 1;
        const uint32_t s0 = (m & 1) ? 0x6622u : 0x4400u, s1 = (m & 1) ? 0x7733u : 0x5511u;  // codes 2m, 2m + 1 of two keys
        const uint32_t a0 = codes_to_bf16(__byte_perm(w[0][q], w[1][q], s0), magic, mul, off);
        const uint32_t a1 = codes_to_bf16(__byte_perm(w[0][q], w[1][q], s1), magic, mul, off);
        const uint32_t a2 = codes_to_bf16(__byte_perm(w[2][q], w[3][q], s0), magic, mul, off);
        const uint32_t a3 = codes_to_bf16(__byte_perm(w[2][q], w[3][q], s1), magic, mul, off);
#pragma unroll
        for (int x = 0; x < NR; ++x) mma_bf16(o[x][m], a0, a1, a2, a3, pf[x][0], pf[x][1]);
    }
}
// bf16 depth slices in the same permuted order.
template <int NH, int NR>
__device__ __forceinline__ void qk_bf16_perm(uint32_t slice, const uint32_t (&qf)[NR][NH * 4][2], float (&s)[NR][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < NH * 2; ++c) {  // 8 features = 2 k-steps
        const uint4 w0 = lds128(bf16_at(slice, g, t * 16 * NH + 8 * c)), w1 = lds128(bf16_at(slice, g + 8, t * 16 * NH + 8 * c));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t l0 = e ? w0.z : w0.x, h0 = e ? w0.w : w0.y, l1 = e ? w1.z : w1.x, h1 = e ? w1.w : w1.y;
            const uint32_t a0 = __byte_perm(l0, h0, 0x5410), a2 = __byte_perm(l0, h0, 0x7632);
            const uint32_t a1 = __byte_perm(l1, h1, 0x5410), a3 = __byte_perm(l1, h1, 0x7632);
#pragma unroll
            for (int x = 0; x < NR; ++x) mma_bf16(s[x], a0, a1, a2, a3, qf[x][2 * c + e][0], qf[x][2 * c + e][1]);
        }
    }
}
template <int NH, int NR>
__device__ __forceinline__ void pv_bf16_perm(uint32_t slice, const uint32_t (&pf)[NR][2], float (&o)[NR][NH * 4][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int c = 0; c < NH; ++c) {  // 8 of the lane's 8 NH features
        uint32_t w[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint4 v = lds128(bf16_at(slice, 2 * t + (x & 1) + 8 * (x >> 1), g * 8 * NH + 8 * c));
            w[x][0] = v.x; w[x][1] = v.y; w[x][2] = v.z; w[x][3] = v.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5410), a1 = __byte_perm(w[0][e], w[1][e], 0x7632);
            const uint32_t a2 = __byte_perm(w[2][e], w[3][e], 0x5410), a3 = __byte_perm(w[2][e], w[3][e], 0x7632);
#pragma unroll
            for (int x = 0; x < NR; ++x) mma_bf16(o[x][4 * c + e], a0, a1, a2, a3, pf[x][0], pf[x][1]);
        }
    }
}

// Feature of row g (hi = 0) or g + 8 (hi = 1) of output tile m.
template <bool Q8, int NH>
__device__ __forceinline__ int out_col(int m, int hi, int g) {
    return Q8 ? g * (8 * NH) + 2 * m + hi : 16 * m + g + 8 * hi;
}

// Keys of a bf16 slice with a non-finite value, as a 16-bit mask.
template <int NH>
__device__ __forceinline__ uint32_t nonfinite_keys(uint32_t slice, int lane) {
    bool bad = false;
    const int r = lane >> 1;
#pragma unroll
    for (int x = 0; x < NH * 4; ++x) {
        const uint4 v = lds128(slice + (x >> 2) * 2048 + r * 128 + (((lane & 1) * 4 + (x & 3)) << 4));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bad |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
    }
    const uint32_t b = __ballot_sync(0xffffffffu, bad);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) m |= ((b >> (2 * k)) & 3u) ? 1u << k : 0u;
    return m;
}

// Adds P V of the keys in `bad` to the rows whose P is not 0.
template <bool Q8, int NH, int NR>
__device__ __forceinline__ void add_nonfinite(uint32_t slice, uint32_t bad, const float (&p)[NR][4], float (&o)[NR][NH * 4][4],
                                              int lane) {
    const int g = lane >> 2, t = lane & 3;
    for (; bad; bad &= bad - 1) {
        const int k = __ffs(bad) - 1, src = (k & 7) * 4 + t;
        float pr[NR][2];
        bool any = false;
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                pr[x][e] = __shfl_sync(0xffffffffu, (k & 8) ? p[x][2 + e] : p[x][e], src);
                any |= pr[x][e] != 0.f;
            }
        if (!__any_sync(0xffffffffu, any)) continue;  // what an unused row of a page held
#pragma unroll
        for (int m = 0; m < NH * 4; ++m)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                uint16_t raw;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(raw) : "r"(bf16_at(slice, k, out_col<Q8, NH>(m, hi, g))) : "memory");
                const float v = __uint_as_float((uint32_t)raw << 16);
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (pr[x][e] != 0.f) o[x][m][2 * hi + e] += pr[x][e] * v;
            }
    }
}
template <int NH>
__device__ __forceinline__ void clear_keys(uint32_t slice, uint32_t bad, int lane) {
    for (; bad; bad &= bad - 1) {
        const int k = __ffs(bad) - 1;
        if (lane < NH * 8)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(slice + (lane >> 3) * 2048 + k * 128 + (lane & 7) * 16), "r"(0) : "memory");
    }
}

// Box of 16 rows x 64 bf16 (or 128 codes) to a shared memory address: as
// ptx::tma_load_4d, whose generic pointer took registers here (28 bytes more of spills).
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, uint64_t* bar, int x, int row, int h, int page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(ptx::smem_u32(bar)), "r"(x), "r"(row), "r"(h), "r"(page)
        : "memory");
}

template <bool Q8, int NH, int NR, int WR>
__global__ void __launch_bounds__(Cfg<Q8, NH, NR, WR>::kThreads, Cfg<Q8, NH, NR, WR>::kPerSM) paged_dec_kernel(const __grid_constant__ DecParams p) {
    using C = Cfg<Q8, NH, NR, WR>;
    constexpr int kThreads = C::kThreads;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t ring = (ptx::smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (ring - ptx::smem_u32(smem_raw));
    float* merge = reinterpret_cast<float*>(base + C::NS * C::kSlot);
    DecBars* bars = reinterpret_cast<DecBars*>(base + C::NS * C::kSlot + C::kMergeBufs * C::kMergeFloats * 4);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const PagedCache& c = p.c;
    const long long max_keys = min((long long)c.max_blocks * c.page_size, 0x7fffff00LL);
    const int cta = blockIdx.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NS; ++s) {
            ptx::mbar_init(&bars->full[s], 1);
            ptx::mbar_init(&bars->empty[s], C::kWarps);
        }
        bars->abort_flag = 0;
        ptx::prefetch_tmap(&p.tm_k);
        ptx::prefetch_tmap(&p.tm_v);
        if (p.Ld > 0) {
            ptx::prefetch_tmap(&p.tm_kd);
            ptx::prefetch_tmap(&p.tm_vd);
        }
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
        p.desc[cta] = make_int4(0, 0, 0, 0);
    }
    // ---- the list of stages, and where this CTA's part of it begins
    auto seq_at = [&](int b) { return b < kSeqs ? bars->seqs[b] : seq_info(c, b); };
    long long total, lo, hi, in_seq, seq_n;  // all stages; the part; its start and the stages per kv-head in its sequence
    int b, W;
    SeqInfo sq;
    auto cut_list = [&]() {  // false: no part for this CTA
        W = (int)max(1LL, min((long long)p.W, total));
        if (cta >= W || total == 0) return false;
        lo = part_begin(total, cta, W);
        hi = part_begin(total, cta + 1, W);
        return true;
    };
    if (c.B <= 32) {
        // a sequence per lane, every warp for itself: one round of loads and no
        // exchange through shared memory
        SeqInfo mine = {0, 0, 0};
        if (lane < c.B) mine = seq_info(c, lane);
        const long long n = lane < c.B ? seq_stages<C::MR, C::KEYS>(mine, p.G, p.DSL, C::DS, max_keys) : 0;
        if (warp == 0 && lane < c.B) bars->seqs[lane] = mine;
        long long incl = n * c.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        total = __shfl_sync(0xffffffffu, incl, 31);
        if (!cut_list()) return;
        b = __ffs(__ballot_sync(0xffffffffu, lo < incl)) - 1;
        in_seq = lo - __shfl_sync(0xffffffffu, incl - n * c.Hkv, b);
        seq_n = __shfl_sync(0xffffffffu, n, b);
        sq.q0 = __shfl_sync(0xffffffffu, mine.q0, b);
        sq.n = __shfl_sync(0xffffffffu, mine.n, b);
        sq.pos0 = __shfl_sync(0xffffffffu, mine.pos0, b);
        __syncthreads();
    } else {
        // each thread sums a run of sequences, then a scan over the threads
        const int per = (c.B + kThreads - 1) / kThreads;
        const int b0 = min((int)threadIdx.x * per, c.B), b1 = min(b0 + per, c.B);
        long long mine = 0;
        for (int x = b0; x < b1; ++x) {
            const SeqInfo s = seq_info(c, x);
            if (x < kSeqs) bars->seqs[x] = s;
            mine += seq_stages<C::MR, C::KEYS>(s, p.G, p.DSL, C::DS, max_keys);
        }
        long long incl = mine * c.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) bars->scan[warp] = incl;
        __syncthreads();
        total = 0;
        long long pre = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) pre += bars->scan[w];
            total += bars->scan[w];
        }
        incl += pre;
        if (!cut_list()) return;
        long long at = incl - mine * c.Hkv;
        if (lo >= at && lo < incl) {  // one thread: the part begins in its run
            for (int x = b0; x < b1; ++x) {
                const long long n = seq_stages<C::MR, C::KEYS>(seq_at(x), p.G, p.DSL, C::DS, max_keys) * c.Hkv;
                if (lo < at + n) {
                    bars->begin_seq = x;
                    bars->begin_in_seq = lo - at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        b = bars->begin_seq;
        in_seq = bars->begin_in_seq;
        sq = seq_at(b);
        seq_n = seq_stages<C::MR, C::KEYS>(sq, p.G, p.DSL, C::DS, max_keys);
    }
    volatile int* abort_flag = &bars->abort_flag;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(p.status, 1u);
    };

    // ---- the units of this part, walked alike by every warp
    int kvh, rt = 0, first;     // first: first stage of the current unit's piece
    long long left = hi - lo;   // stages still to do
    if (in_seq < (1LL << 31) && seq_n < (1LL << 31)) kvh = (int)((uint32_t)in_seq / (uint32_t)seq_n);
    else kvh = (int)(in_seq / seq_n);
    for (long long in = in_seq - kvh * seq_n;; ++rt) {
        const int st = unit_shape<C::MR, C::KEYS>(sq, rt, p.G, p.DSL, C::DS, max_keys).st;
        if (in < st) {
            first = (int)in;
            break;
        }
        in -= st;
    }
    auto next_unit = [&]() {
        first = 0;
        if (++rt * C::MR < sq.n * p.G) return;
        rt = 0;
        if (++kvh < c.Hkv) return;
        kvh = 0;
        do {
            sq = seq_at(++b);
        } while (sq.n == 0 && b + 1 < c.B);  // `left` > 0: a later sequence has stages
    };

    if (!p.split && first > 0) {  // the unit belongs to the CTA it starts in
        left -= unit_shape<C::MR, C::KEYS>(sq, rt, p.G, p.DSL, C::DS, max_keys).st - first;
        if (left > 0) next_unit();
    }

    if (warp == C::kWarps) {
        int slot = 0, ph = 1, issued = 0;
        bool ok = true;
        while (left > 0) {
            const UnitShape u = unit_shape<C::MR, C::KEYS>(sq, rt, p.G, p.DSL, C::DS, max_keys);
            const int end = p.split ? (int)min((long long)u.st, first + left) : u.st;
            // page slices [SPS first, ...) of the unit, 32 at a time: lane l
            // holds slice 32 batch + l of the piece; the next batch's page ids
            // are in flight while this one's boxes are issued
            const int sl0 = first * C::SPS, sl_all = u.st_seq * C::SPS;
            auto fetch = [&](int sl) {  // page of slice sl, num_pages: none
                const int key = sl * kSliceRows;
                int pg = -1;
                if (sl < sl_all && key < u.nk) pg = page_of(c, b, key / c.page_size);
                return pg;
            };
            int page = fetch(sl0 + lane), page_next = fetch(sl0 + 32 + lane);
            float ks = 1.f, vs = 1.f, ks_next = 1.f, vs_next = 1.f;
            auto scales = [&](int pg, float& a, float& e) {
                a = pg < 0 ? -1.f : 1.f;
                e = 1.f;
                if (Q8 && pg >= 0) {
                    a = __ldg(p.k_scale + (long long)pg * c.Hkv + kvh);
                    e = __ldg(p.v_scale + (long long)pg * c.Hkv + kvh);
                }
            };
            scales(page, ks, vs);
            for (int st = first; st < end; ++st) {
                const bool seq = st < u.st_seq;
                const int rel = st * C::SPS - sl0;
                if (seq && rel && (rel & 31) == 0) {
                    page = page_next;
                    ks = ks_next;
                    vs = vs_next;
                    page_next = fetch(sl0 + rel + 32 + lane);
                }
                if (seq && (rel & 31) == 16) scales(page_next, ks_next, vs_next);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (ok && !__all_sync(0xffffffffu, ptx::mbar_wait(&bars->empty[slot], ph, p.wait_limit, abort_flag))) {
                        if (lane == 0) fail();
                        ok = false;
                    }
                    if (ok) {
                        uint64_t* bar = &bars->full[slot];
                        const uint32_t dst = ring + slot * C::kSlot;
                        if (seq) {
                            const int per_slice = Q8 ? 1 : NH;
                            const int sl = lane / per_slice, half = lane % per_slice;
                            const int src = (rel & 31) + (sl & (C::SPS - 1));
                            const int pg = __shfl_sync(0xffffffffu, page, src);
                            const float sc = __shfl_sync(0xffffffffu, kv ? vs : ks, src);
                            if (lane < C::SPS * per_slice && half == 0) {
                                bars->scale[slot][sl] = Q8 && kv ? p_factor(sc) : sc;
                                if (Q8 && kv) bars->code_mul[slot][sl] = code_factor(sc);
                            }
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, C::kSlot);
                            __syncwarp();
                            if (lane < C::SPS * per_slice) {
                                const int key = (st * C::SPS + sl) * kSliceRows;
                                // a page that is not there lies outside the map: zeros
                                load_box(dst + sl * C::kSeqSlice + half * 2048, kv ? &p.tm_v : &p.tm_k, bar, half * 64,
                                         pg < 0 ? 0 : key % c.page_size, kvh, pg < 0 ? c.num_pages : pg);
                            }
                        } else {
                            const int sl = lane / NH, half = lane % NH;
                            const int x = (st - u.st_seq) * C::DS + sl;
                            if (lane == 0) ptx::mbar_arrive_expect_tx(bar, C::kSlot);
                            __syncwarp();
                            if (lane < C::DS * NH) {
                                const int tok = p.DSL ? x / p.DSL : 0, sl16 = p.DSL ? x % p.DSL : 0;
                                const bool in = tok < u.ntok && p.DSL;
                                load_box(dst + sl * C::kDepSlice + half * 2048, kv ? &p.tm_vd : &p.tm_kd, bar, half * 64, kvh,
                                         sl16 * kSliceRows, in ? sq.q0 + u.tok0 + tok : c.N);
                            }
                        }
                        ++issued;
                    }
                    if (++slot == C::NS) {
                        slot = 0;
                        ph ^= 1;
                    }
                }
            }
            left -= end - first;
            if (left > 0) next_unit();
        }
        // every copy this CTA issued lands before it exits
        for (int s = issued > C::NS ? issued - C::NS : 0; s < issued; ++s)
            ptx::mbar_wait(&bars->full[s % C::NS], (s / C::NS) & 1, 0, nullptr);
        return;
    }

    // ------------------------------------------------------ consumer warps
    const int wr = warp / C::WK, wk = warp % C::WK;  // rows 8 NR wr .., keys of slices wk, wk + WK, ..
    const int g = lane >> 2, t = lane & 3;
    const uint32_t magic = magic_reg();
    int slot = 0, ph = 0;
    bool ok = true;
    while (left > 0) {
        const UnitShape u = unit_shape<C::MR, C::KEYS>(sq, rt, p.G, p.DSL, C::DS, max_keys);
        const int end = p.split ? (int)min((long long)u.st, first + left) : u.st;
        const int row0 = u.r0 + 8 * NR * wr, rows = u.rows - 8 * NR * wr;  // this warp's rows (rows may be <= 0)
        auto out_row = [&](int r) {  // packed row and head of row r of the sequence
            return (long long)(sq.q0 + r / p.G) * p.Hq + kvh * p.G + r % p.G;
        };
        // queries of row g of each tile, and token and position of rows 2t, 2t + 1
        uint32_t qf[NR][NH * 4][2];
        int tok[NR][2], pos[NR][2];
#pragma unroll
        for (int x = 0; x < NR; ++x) {
            const bool in = 8 * x + g < rows;
            const __nv_bfloat16* row = p.q + (in ? out_row(row0 + 8 * x + g) : 0) * c.d;
#pragma unroll
            for (int k = 0; k < NH * 4; ++k) {
                if (Q8) {
                    const int f = t * 16 * NH + 4 * k;  // features f .. f+3
                    uint2 w = make_uint2(0, 0);
                    if (in && f < c.d) w = *reinterpret_cast<const uint2*>(row + f);
                    qf[x][k][0] = __byte_perm(w.x, w.y, 0x5410);
                    qf[x][k][1] = __byte_perm(w.x, w.y, 0x7632);
                } else {
                    const int f = 16 * k + 2 * t;
                    qf[x][k][0] = in && f < c.d ? *reinterpret_cast<const uint32_t*>(row + f) : 0u;
                    qf[x][k][1] = in && f + 8 < c.d ? *reinterpret_cast<const uint32_t*>(row + f + 8) : 0u;
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * x + 2 * t + e;
                tok[x][e] = r < rows ? (row0 + r) / p.G : -1;
                pos[x][e] = r < rows ? sq.pos0 + tok[x][e] : -1;
            }
        }
        float o[NR][NH * 4][4];
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int x = 0; x < NR; ++x) {
#pragma unroll
            for (int n = 0; n < NH * 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][n][e] = 0.f;
            m[x][0] = m[x][1] = -INFINITY;
            l[x][0] = l[x][1] = 0.f;
        }

        const int pos_first = sq.pos0 + u.tok0;  // keys up to here are seen by every row of the tile
        for (int st = first; st < end; ++st) {
            const bool seq = st < u.st_seq;
            const int kslot = slot, kph = ph;
            if (++slot == C::NS) { slot = 0; ph ^= 1; }
            const int vslot = slot, vph = ph;
            if (++slot == C::NS) { slot = 0; ph ^= 1; }
            if (ok && !__all_sync(0xffffffffu, ptx::mbar_wait(&bars->full[kslot], kph, p.wait_limit, abort_flag))) {
                if (lane == 0) fail();
                ok = false;
            }
            const uint32_t ka = ring + kslot * C::kSlot, va = ring + vslot * C::kSlot;
            const uint32_t bytes = seq ? C::kSeqSlice : C::kDepSlice;
            float s[C::SL][NR][4];
            const bool some = !seq || st * C::KEYS + C::KEYS - 1 > pos_first;  // some row is masked somewhere in the stage
            bool part[C::SL];                                                // this warp's slice i takes part
#pragma unroll
            for (int i = 0; i < C::SL; ++i) {
                const int sl = wk + i * C::WK;
                part[i] = seq || sl < C::DS;
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][x][e] = 0.f;
                float ksc = 1.f;
                if (ok && part[i]) {
                    if (seq) {
                        ksc = bars->scale[kslot][sl];
                        if (Q8) qk_q8<NH, NR>(ka + sl * bytes, qf, s[i], lane, magic);
                        else qk_bf16<NH, NR>(ka + sl * bytes, qf, s[i], lane);
                    } else {
                        if (Q8) qk_bf16_perm<NH, NR>(ka + sl * bytes, qf, s[i], lane);
                        else qk_bf16<NH, NR>(ka + sl * bytes, qf, s[i], lane);
                    }
                }
                const float mul = p.sl2 * (Q8 && seq ? kCodeUnit : 1.f);
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[i][x][e] *= mul;
                        if (Q8) s[i][x][e] *= ksc;
                    }
                if (!part[i]) {
#pragma unroll
                    for (int x = 0; x < NR; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[i][x][e] = -INFINITY;
                } else if (some || ksc < 0.f) {
                    const int key0 = (st * C::SPS + sl) * kSliceRows;
                    const int dx = (st - u.st_seq) * C::DS + sl;
                    const int dtok = seq || !p.DSL ? 0 : u.tok0 + dx / p.DSL, dsl = seq || !p.DSL ? 0 : dx % p.DSL * kSliceRows;
#pragma unroll
                    for (int x = 0; x < NR; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = g + 8 * (e >> 1), r = e & 1;
                            const bool see = seq ? key0 + k <= pos[x][r] && key0 + k < u.nk && ksc >= 0.f
                                                 : tok[x][r] == dtok && dsl + k < p.Ld;
                            if (!see) s[i][x][e] = -INFINITY;
                        }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->empty[kslot]);
            // ---- online softmax over this warp's keys of the stage
            float mx[NR][2];
            bool moves = false;
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(s[0][x][e], s[0][x][2 + e]);
#pragma unroll
                    for (int i = 1; i < C::SL; ++i) v = fmaxf(v, fmaxf(s[i][x][e], s[i][x][2 + e]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mx[x][e] = v;
                    moves |= v > m[x][e] + kLazy;
                }
            if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mn = fmaxf(m[x][e], mx[x][e]);
                        const float corr = mn == -INFINITY ? 1.f : ptx::ex2(m[x][e] - mn);
                        l[x][e] *= corr;
                        m[x][e] = mn;
#pragma unroll
                        for (int n = 0; n < NH * 4; ++n) {
                            o[x][n][e] *= corr;
                            o[x][n][2 + e] *= corr;
                        }
                    }
            }
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const float ref[2] = {m[x][0] == -INFINITY ? 0.f : m[x][0], m[x][1] == -INFINITY ? 0.f : m[x][1]};
#pragma unroll
                for (int i = 0; i < C::SL; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[i][x][e] = ptx::ex2(s[i][x][e] - ref[e & 1]);
                        l[x][e & 1] += s[i][x][e];
                    }
            }
            if (ok && !__all_sync(0xffffffffu, ptx::mbar_wait(&bars->full[vslot], vph, p.wait_limit, abort_flag))) {
                if (lane == 0) fail();
                ok = false;
            }
            // ---- values a row must not see may be non-finite (codes are not)
            if (some && (!Q8 || !seq)) {
                uint32_t bad[C::SL];
#pragma unroll
                for (int i = 0; i < C::SL; ++i) {
                    bad[i] = 0;
                    if (ok && part[i]) {
                        bad[i] = nonfinite_keys<NH>(va + (wk + i * C::WK) * bytes, lane);
                        if (bad[i]) add_nonfinite<Q8, NH, NR>(va + (wk + i * C::WK) * bytes, bad[i], s[i], o, lane);
                    }
                }
                // warps that share the keys have all read them before they are cleared
                if (WR > 1) ptx::bar_sync(2, C::kWarps * 32); else __syncwarp();
#pragma unroll
                for (int i = 0; i < C::SL; ++i)
                    if (bad[i]) clear_keys<NH>(va + (wk + i * C::WK) * bytes, bad[i], lane);
                ptx::fence_proxy_async_smem();  // before the slot's next copy
                if (WR > 1) ptx::bar_sync(2, C::kWarps * 32); else __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < C::SL; ++i) {
                const int sl = wk + i * C::WK;
                if (!ok || !part[i]) continue;
                // (an 8-bit kernel's O is in units of kCodeUnit)
                float vsc = 1.f / kCodeUnit;
                if (Q8 && seq) vsc = bars->scale[vslot][sl];
                uint32_t pf[NR][2];
#pragma unroll
                for (int x = 0; x < NR; ++x)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pf[x][h] = transpose8x8(Q8 ? ptx::pack_bf16x2(s[i][x][2 * h] * vsc, s[i][x][2 * h + 1] * vsc)
                                                   : ptx::pack_bf16x2(s[i][x][2 * h], s[i][x][2 * h + 1]));
                if (seq) {
                    if (Q8) pv_q8<NH, NR>(va + sl * bytes, pf, o, lane, magic, bars->code_mul[vslot][sl]);
                    else pv_bf16<NH, NR>(va + sl * bytes, pf, o, lane);
                } else {
                    if (Q8) pv_bf16_perm<NH, NR>(va + sl * bytes, pf, o, lane);
                    else pv_bf16<NH, NR>(va + sl * bytes, pf, o, lane);
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars->empty[vslot]);
        }
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int sh = 4; sh < 32; sh *= 2) l[x][e] += __shfl_xor_sync(0xffffffffu, l[x][e], sh);
        // ---- join the warps that shared the rows: upper half into lower half
        if (C::WK > 1) {
#pragma unroll
            for (int half = C::WK / 2; half >= 1; half /= 2) {
                ptx::bar_sync(1, C::kWarps * 32);  // the buffers are free
                const int buf = wr * (C::WK / 2) + wk % half;
                float* mo = merge + buf * C::kMergeFloats;
                if (wk >= half && wk < 2 * half) {
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
#pragma unroll
                        for (int n = 0; n < NH * 4; ++n)
                            *reinterpret_cast<float4*>(mo + ((x * NH * 4 + n) * 32 + lane) * 4) =
                                make_float4(o[x][n][0], o[x][n][1], o[x][n][2], o[x][n][3]);
                        if (g == 0) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                bars->ml[buf][8 * x + 2 * t + e][0] = m[x][e];
                                bars->ml[buf][8 * x + 2 * t + e][1] = l[x][e];
                            }
                        }
                    }
                }
                ptx::bar_sync(1, C::kWarps * 32);
                if (wk < half) {
#pragma unroll
                    for (int x = 0; x < NR; ++x) {
                        float c1[2], c2[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float m2 = bars->ml[buf][8 * x + 2 * t + e][0], l2 = bars->ml[buf][8 * x + 2 * t + e][1];
                            const float mn = fmaxf(m[x][e], m2), rf = mn == -INFINITY ? 0.f : mn;
                            c1[e] = ptx::ex2(m[x][e] - rf);
                            c2[e] = ptx::ex2(m2 - rf);
                            l[x][e] = l[x][e] * c1[e] + l2 * c2[e];
                            m[x][e] = mn;
                        }
#pragma unroll
                        for (int n = 0; n < NH * 4; ++n) {
                            const float4 v = *reinterpret_cast<const float4*>(mo + ((x * NH * 4 + n) * 32 + lane) * 4);
                            o[x][n][0] = o[x][n][0] * c1[0] + v.x * c2[0];
                            o[x][n][1] = o[x][n][1] * c1[1] + v.y * c2[1];
                            o[x][n][2] = o[x][n][2] * c1[0] + v.z * c2[0];
                            o[x][n][3] = o[x][n][3] * c1[1] + v.w * c2[1];
                        }
                    }
                }
            }
        }
        const bool whole = first == 0 && end == u.st;
        if (wk == 0 && whole) {
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                float inv[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) inv[e] = l[x][e] == 0.f ? 0.f : (Q8 ? kCodeUnit : 1.f) / l[x][e];
                if (Q8) {  // 8 NH consecutive features of rows 2t, 2t + 1
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * x + 2 * t + e, f0 = g * 8 * NH;
                        if (r >= rows) continue;
                        __nv_bfloat16* dst = p.out + out_row(row0 + r) * c.d + f0;
#pragma unroll
                        for (int n = 0; n < NH * 4; n += 4)
                            if (f0 + 2 * n < c.d)
                                *reinterpret_cast<uint4*>(dst + 2 * n) =
                                    make_uint4(ptx::pack_bf16x2(o[x][n][e] * inv[e], o[x][n][2 + e] * inv[e]),
                                               ptx::pack_bf16x2(o[x][n + 1][e] * inv[e], o[x][n + 1][2 + e] * inv[e]),
                                               ptx::pack_bf16x2(o[x][n + 2][e] * inv[e], o[x][n + 2][2 + e] * inv[e]),
                                               ptx::pack_bf16x2(o[x][n + 3][e] * inv[e], o[x][n + 3][2 + e] * inv[e]));
                    }
                } else {  // 8 x 8 blocks (feature, row) transposed: features 2t, 2t + 1 of row g
                    const bool in = 8 * x + g < rows;
                    __nv_bfloat16* dst = p.out + (in ? out_row(row0 + 8 * x + g) : 0) * c.d;
#pragma unroll
                    for (int n = 0; n < NH * 4; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t w = transpose8x8(ptx::pack_bf16x2(o[x][n][2 * h] * inv[0], o[x][n][2 * h + 1] * inv[1]));
                            const int f = 16 * n + 8 * h + 2 * t;
                            if (in && f < c.d) *reinterpret_cast<uint32_t*>(dst + f) = w;
                        }
                }
                if (g == 0 && p.lse)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (8 * x + 2 * t + e < rows)
                            p.lse[out_row(row0 + 8 * x + 2 * t + e)] =
                                l[x][e] == 0.f ? -INFINITY : (m[x][e] + __log2f(l[x][e])) * 0.6931471805599453f;
            }
        } else if (wk == 0) {
            // a part: the one that starts the unit goes to slot 2 cta + 1
            const int ps = 2 * cta + (first == 0 ? 1 : 0);
            const long long pr = (long long)ps * C::MR + 8 * NR * wr;
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * x + 2 * t + e;
                    if (r >= rows) continue;
                    float* po = p.part_o + (pr + r) * C::D;
#pragma unroll
                    for (int n = 0; n < NH * 4; ++n) {
                        if (Q8) {
                            *reinterpret_cast<float2*>(po + out_col<true, NH>(n, 0, g)) =
                                make_float2(o[x][n][e] * kCodeUnit, o[x][n][2 + e] * kCodeUnit);
                        } else {
                            po[out_col<false, NH>(n, 0, g)] = o[x][n][e];
                            po[out_col<false, NH>(n, 1, g)] = o[x][n][2 + e];
                        }
                    }
                    if (g == 0) *reinterpret_cast<float2*>(p.part_ml + (pr + r) * 2) = make_float2(m[x][e], l[x][e]);
                }
            if (first == 0 && warp == 0 && lane == 0) {
                // parts up to the one that holds the unit's last stage
                const long long last = hi - left + u.st - 1;  // its index in the list (this piece starts at hi - left)
                const int c_last = (int)(((last + 1) * W + total - 1) / total) - 1;
                p.desc[cta] = make_int4(sq.q0, kvh, rt, (c_last - cta + 1) | u.rows << 16);
            }
        }
        left -= end - first;
        if (left > 0) next_unit();
    }
    // the join may be scheduled once every CTA is about here; earlier its
    // waiting blocks would take issue slots from this kernel
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Query rows of a unit by the rows a sequence has: 8, 16 or 32.
int rows_of(int max_q, int G) {
    const long long r = (long long)max_q * G;
    return r <= 8 ? 8 : r <= 16 ? 16 : 32;
}

// Map of 8-bit pages with the swizzle of the bf16 ones.
bool make_tmap_codes(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[4], const cuuint64_t (&strides)[3],
                     const cuuint32_t (&box)[4]) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool Q8, int NH, int NR, int WR>
cudaError_t launch(const PagedFwdArgs& a, cudaStream_t s) {
    using C = Cfg<Q8, NH, NR, WR>;
    DecParams p;
    memset(&p, 0, sizeof(p));
    const PagedCache& c = a.c;
    const cuuint64_t d = c.d, P = c.page_size, e = Q8 ? 1 : 2;
    {
        const cuuint64_t dims[4] = {d, P, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
        const cuuint64_t st[3] = {d * e, P * d * e, c.Hkv * P * d * e};
        const cuuint32_t box[4] = {Q8 ? 128u : 64u, (cuuint32_t)kSliceRows, 1, 1};
        auto make = [&](CUtensorMap* m, const void* pages) {
            return Q8 ? make_tmap_codes(m, pages, dims, st, box) : make_tmap_bf16_4d(m, pages, dims, st, box);
        };
        if (!make(&p.tm_k, a.k_pages) || !make(&p.tm_v, a.v_pages)) return cudaErrorInvalidValue;
    }
    if (a.Ld > 0) {
        // dimensions: feature, kv-head, slot (those in use), token
        const cuuint64_t dims[4] = {d, (cuuint64_t)c.Hkv, (cuuint64_t)a.Ld, (cuuint64_t)c.N};
        const cuuint64_t st[3] = {d * 2, c.Hkv * d * 2, (cuuint64_t)a.Ld_cap * c.Hkv * d * 2};
        const cuuint32_t box[4] = {64, 1, (cuuint32_t)kSliceRows, 1};
        if (!make_tmap_bf16_4d(&p.tm_kd, a.kd, dims, st, box) || !make_tmap_bf16_4d(&p.tm_vd, a.vd, dims, st, box))
            return cudaErrorInvalidValue;
    } else {
        p.tm_kd = p.tm_k;
        p.tm_vd = p.tm_v;
    }
    p.c = c;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.Hq = a.Hq; p.G = a.G; p.Ld = a.Ld; p.DSL = (a.Ld + kSliceRows - 1) / kSliceRows;
    p.W = C::kParts;
    // The longest unit that the block table allows, in stages. Up to two stay
    // whole and save the join (one sequence of 16 tokens, G = 4: 8.6 us against
    // 9.4). Longer ones are cut to use the idle CTAs (one of 256 tokens: 9.8
    // against 12.0), but for those of up to six stages when there are units for
    // a share of the CTAs anyway (64 sequences of 128 tokens, four of them new,
    // G = 4: 33.1 cut, 23.8 whole).
    const long long keys = (long long)c.max_blocks * c.page_size;
    const long long toks = std::min((C::MR + a.G - 2) / a.G + 1, a.max_q);
    const long long stages = (keys + C::KEYS - 1) / C::KEYS + (toks * p.DSL + C::DS - 1) / C::DS;
    const long long units = (long long)c.B * c.Hkv * (((long long)a.max_q * a.G + C::MR - 1) / C::MR);
    p.split = stages > 6 || (stages > 2 && stages * C::kParts > 10 * units);
    p.sl2 = a.scale * 1.4426950408889634f;
    p.status = a.status;
    p.wait_limit = a.wait_limit;
    char* ws = static_cast<char*>(a.workspace);
    p.desc = reinterpret_cast<int4*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + C::kParts * sizeof(int4));
    p.part_o = p.part_ml + (size_t)2 * C::kParts * C::MR * 2;
    auto kern = paged_dec_kernel<Q8, NH, NR, WR>;
    static SmemLimit limit;
    cudaError_t err = limit.raise(reinterpret_cast<const void*>(kern), C::kSmem);
    if (err != cudaSuccess) return err;
    kern<<<C::kParts, C::kThreads, C::kSmem, s>>>(p);
    err = cudaGetLastError();
    if (err != cudaSuccess || !p.split) return err;
    JoinParams j{p.c, p.out, p.lse, p.part_o, p.part_ml, p.desc, p.Hq, p.G, 0};
    return launch_paged_join<C::MR, C::D, C::kParts>(j, s);
}

template <bool Q8, int NH>
cudaError_t by_rows(const PagedFwdArgs& a, cudaStream_t s) {
    switch (rows_of(a.max_q, a.G)) {
        case 8: return launch<Q8, NH, 1, 1>(a, s);
        case 16: return launch<Q8, NH, 2, 1>(a, s);
        default: return launch<Q8, NH, 2, 2>(a, s);
    }
}

}  // namespace

bool paged_dec_supported(const PagedFwdArgs& a) {
    const PagedCache& c = a.c;
    if (a.dtype != MODA_BF16 || c.d % 8 || c.page_size % kSliceRows) return false;
    if (a.k_scale && c.d % 16) return false;  // TMA strides are multiples of 16 bytes
    return (long long)c.N * a.Hq < 0x7fffff00LL;  // rows in 32 bits, the last tile's end among them
}

size_t paged_dec_workspace(int max_q, int G, int d) {
    const size_t mr = rows_of(max_q, G), D = d <= 64 ? 64 : 128;
    const size_t parts = (mr == 8 ? 3 : 2) * 148;
    return parts * sizeof(int4) + 2 * parts * mr * (D + 2) * sizeof(float);
}

cudaError_t launch_paged_dec(const PagedFwdArgs& a, cudaStream_t s) {
    if (a.k_scale) return a.c.d <= 64 ? by_rows<true, 1>(a, s) : by_rows<true, 2>(a, s);
    return a.c.d <= 64 ? by_rows<false, 1>(a, s) : by_rows<false, 2>(a, s);
}

}  // namespace moda
