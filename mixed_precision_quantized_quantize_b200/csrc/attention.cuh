// attention.cuh -- what the attention kernels share: their parameters, what a
// sequence holds, which new tokens a row sees, the conversion of codes and a
// few one-instruction wrappers.  Included once by each kernel file.
#pragma once

#include "quik_internal.h"
#include "sm100.cuh"

#include <cuda_fp16.h>

namespace quik {

struct AttnParams {
    int tokens, sequences, q_heads, heads, group, max_tokens, max_pages, mask_words;
    int pages, page_shift, splits, row_blocks;
    float scale_log2;
    const uint16_t *q;
    int64_t q_stride;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *page_table, *context, *cu;
    const uint32_t *mask;
    uint16_t *out;
    int64_t out_stride;
    float *lse;
    float *part_o;   // [splits][tokens * q_heads][D]
    float2 *part_ml; // [splits][tokens * q_heads]
    // up to 8 rows: pieces (workers + items of them), each 8 rows as the warps hold them
    int workers;
    int mode;          // who takes an item
    float4 *piece_o;   // [pieces][D / 16][32]
    float2 *piece_ml;  // [pieces][8]
    int *item_span;    // [items][2]: the workers that hold an item's first and last tile
};

// The tcgen05 form (tree_attention_wide.cu): `blocks` (1 or 2) blocks of 128
// rows a CTA, p.row_blocks of those and p.splits set by the caller.
quik_status launch_attention_wide(const AttnParams &p, int kv_type, int head_dim, int blocks,
                                  cudaStream_t stream);

// Indices out of range met by the kernels of this file (page numbers, lengths,
// offsets): only ever grows; quik_sync_check reports the increase.
static __device__ unsigned int g_attn_bad_index;

namespace {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 (or 4) bytes global -> shared, zeros where !ok (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void group_sync(int id, int threads) {
    if (threads == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pick(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void load_matrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void load_matrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t (&w)[BYTES / 4], uint32_t addr) {
    if constexpr (BYTES == 16)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr)
                     : "memory");
    else if constexpr (BYTES == 8)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
}

// Codes to fp16, exactly: a code's bits, its sign bit flipped (that adds 128 or
// 8), are put into the mantissa of 2^10 (or, four bits up, of 2^6), and that
// base plus the offset is subtracted.  (Without the subtraction, the codes as
// fp16 subnormals and the offset taken off the sums, a product lost up to ten
// bits: the tensor cores align subnormals by their nominal exponent.)
// bytes 0, 1 (hi: 2, 3) of x, already ^ 0x80808080, as a pair
__device__ __forceinline__ uint32_t pair8(uint32_t x, bool hi) {
    return half2_sub(pick(x, 0x64006400u, hi ? 0x5352u : 0x5150u), 0x64806480u);  // 1024 + 128
}
// the nibbles at bits 0 and 16 (up: 4 and 20) of x as a pair
__device__ __forceinline__ uint32_t pair4(uint32_t x, bool up) {
    const uint32_t c = up ? 0x54805480u : 0x64086408u;  // 64 + 8, 1024 + 8
    uint32_t r;  // (x & mask) ^ c
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(x), "r"(up ? 0x00f000f0u : 0x000f000fu), "r"(c));
    return half2_sub(r, c);
}

// What a sequence holds; n == 0: nothing to do.
struct Seq {
    int first, n, ctx, total;
};
__device__ __forceinline__ Seq sequence(const AttnParams &p, int b, bool report) {
    Seq s;
    s.first = p.cu[b];
    const int end = p.cu[b + 1];
    s.ctx = p.context[b];
    const int64_t cap = min(static_cast<int64_t>(p.max_pages) << p.page_shift,
                            static_cast<int64_t>(0x7fffff00));
    int64_t total = static_cast<int64_t>(s.ctx) + (static_cast<int64_t>(end) - s.first);
    bool bad = s.first < 0 || end < s.first || end > p.tokens || s.ctx < 0;
    if (!bad) bad = end - s.first > p.max_tokens;
    s.n = bad ? 0 : end - s.first;
    if (!bad && total > cap) {
        total = cap;
        if (report) atomicAdd(&g_attn_bad_index, 1u);
    }
    if (bad && report) atomicAdd(&g_attn_bad_index, 1u);
    s.total = bad ? 0 : static_cast<int>(total);
    return s;
}

// Which of the 32 tokens from new token j0 on (negative: context) new token
// `tok` sees; tok < 0 (no such row): all of them.
__device__ __forceinline__ unsigned seen(const AttnParams &p, int first, int tok, int j0) {
    if (tok < 0 || j0 + 32 <= 0) return 0xffffffffu;
    if (p.mask == nullptr) {
        const int top = tok - j0;  // last visible position of the tile
        return top < 0 ? 0u : top >= 31 ? 0xffffffffu : (2u << top) - 1u;
    }
    const uint32_t *row = p.mask + static_cast<int64_t>(first + tok) * p.mask_words;
    if (j0 < 0) return (row[0] << -j0) | ((1u << -j0) - 1u);
    const int w = j0 / 32;
    const uint32_t lo = w < p.mask_words ? row[w] : 0u;
    const uint32_t hi = w + 1 < p.mask_words ? row[w + 1] : 0u;
    return __funnelshift_r(lo, hi, j0 % 32);
}

// The unit of the values' scales: the exponent above the largest finite one
// (given by its bits).
__device__ __forceinline__ int top_exponent(unsigned top) {
    return min(max(static_cast<int>(top >> 23) - 126, -100), 126);
}
// 2^-R, for R from -126 to 126.
__device__ __forceinline__ float unit_of(int R) { return __uint_as_float(static_cast<unsigned>(127 - R) << 23); }
// 1 / u of such a power of two.
__device__ __forceinline__ float inverse_unit(float u) { return __uint_as_float((254u << 23) - __float_as_uint(u)); }
__device__ __forceinline__ unsigned finite_bits(float x) {
    const unsigned u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

}  // namespace
}  // namespace quik
