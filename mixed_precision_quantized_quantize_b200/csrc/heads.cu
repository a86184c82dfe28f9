// heads.cu -- the row kernels between the QKV projection and the attention:
// the per-head RMS norm with the rotation (qk_norm_rope), the append of K and
// V rows to the paged cache (kv_append) and the read-back (kv_gather).
//
// A row is one head of one token, D = 64 or 128 channels.  In the first two
// D / 16 lanes hold a row, sixteen channels each, so a warp holds 8 or 4 rows
// and all reductions over a row are shuffles inside that lane group.  A lane's
// channels are two runs of eight (16-byte loads), placed so that both channels
// of every rotated pair are in the same lane: with pairs (i, i + rotary_dim / 2)
// a run and the one rotary_dim / 2 further on, otherwise two adjacent runs.  The
// rotation then needs no exchange between lanes.  The table entries of a token
// are loaded once and serve all the rows that a warp takes of it.
//
// Every channel is read once and written once, but at these sizes the kernels
// are bound by instructions as much as by memory, so the arithmetic is paired
// (two fp32 an instruction).  Norm and rotation of 2048 x 64 heads of 128: 18.6 us
// with eight channels a lane and the partner's shuffled in, 15.3 with two runs of
// four, 14.6 with two runs of eight and four CTAs an SM (10.4 by the bytes).
// Appends of 2048 x 32 heads of 128 in fp16 take 14.4 us (10.4 by the bytes) and
// read back 12.9 (10.2), of 4093 x 8 in INT8 8.4 and read back 6.1 (6.7 for both),
// of 4096 x 32 in INT4 27.7 and read back 17.5 (23.5 for both).
#include "quik_internal.h"
#include "sm100.cuh"

#include <cuda_fp16.h>

namespace quik {

// Rows whose position or slot was outside its range: only ever grows;
// quik_sync_check reports the increase.
__device__ unsigned int g_kv_bad_index;

namespace {

using ptx::f2;
using ptx::f2_add;
using ptx::f2_fma;
using ptx::f2_mul;
using ptx::f2_split;
using ptx::f2_sub;

__device__ __forceinline__ uint4 load16(const void *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void store16(void *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }

// Eight fp16 channels as four fp32 pairs, and back (rounded to nearest).
__device__ __forceinline__ void unpack8(uint4 v, uint64_t *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[i] = f2(f.x, f.y);
    }
}
__device__ __forceinline__ uint4 pack8(const uint64_t *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_split(x[i], a, b);
        const __half2 h = __floats2half2_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's channels: runs of eight at a and b.
struct Runs {
    int a, b;
};
template <bool INTER>
__device__ __forceinline__ Runs runs_of(int rotary, int i) {
    const int half = rotary / 2;
    Runs r;
    if (!INTER && 8 * i < half) {
        r.a = 8 * i;
        r.b = half + 8 * i;
    } else {
        r.a = 16 * i;  // (half-split: lanes half / 8 on go on at rotary_dim)
        r.b = r.a + 8;
    }
    return r;
}

// The rotation of one token, as this lane needs it.  Half-split: cosines and
// sines of its eight pairs, two a word.  Adjacent pairs: one angle a word, twice,
// the sine with the sign of its channel.
template <bool INTER>
struct Turn {
    uint64_t c[INTER ? 8 : 4], s[INTER ? 8 : 4];
    uint64_t zero;  // -0, -0, not known to the compiler
    bool on;        // this lane's channels are rotated
};

template <bool INTER>
__device__ __forceinline__ Turn<INTER> load_turn(const RotaryArgs &r, int token, int i) {
    Turn<INTER> t;
    const int half = r.rotary / 2;
    t.on = 8 * i < half;
    t.zero = f2(r.minus_zero, r.minus_zero);
    if (r.rotary == 0) return t;
    int pos = r.positions[token];
    if (pos < 0 || pos >= r.rows) {
        if (threadIdx.x % 32 == 0) atomicAdd(&g_kv_bad_index, 1u);
        pos = 0;
    }
    if (t.on) {
        // pairs 8 i .. 8 i + 7 in both forms
        const int64_t at = static_cast<int64_t>(pos) * half + 8 * i;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 c = *reinterpret_cast<const float4 *>(r.cos + at + 4 * h);
            const float4 s = *reinterpret_cast<const float4 *>(r.sin + at + 4 * h);
            if constexpr (INTER) {
                t.c[4 * h] = f2(c.x, c.x), t.c[4 * h + 1] = f2(c.y, c.y);
                t.c[4 * h + 2] = f2(c.z, c.z), t.c[4 * h + 3] = f2(c.w, c.w);
                t.s[4 * h] = f2(-s.x, s.x), t.s[4 * h + 1] = f2(-s.y, s.y);
                t.s[4 * h + 2] = f2(-s.z, s.z), t.s[4 * h + 3] = f2(-s.w, s.w);
            } else {
                t.c[2 * h] = f2(c.x, c.y), t.c[2 * h + 1] = f2(c.z, c.w);
                t.s[2 * h] = f2(s.x, s.y), t.s[2 * h + 1] = f2(s.z, s.w);
            }
        }
    }
    return t;
}

// x c + y s (MINUS: x c - y s).  EXACT: in IEEE steps, each product and the sum rounded: the
// values, and so the codes made of them, are then the same wherever they are
// computed.  (A paired product followed by a paired sum came out with one
// rounding instead of two; as a sum with a -0 that the compiler does not know
// the product is rounded by itself.)
template <bool EXACT, bool MINUS>
__device__ __forceinline__ uint64_t turned(uint64_t x, uint64_t c, uint64_t y, uint64_t s, uint64_t zero) {
    const uint64_t a = EXACT ? f2_fma(x, c, zero) : f2_mul(x, c), b = EXACT ? f2_fma(y, s, zero) : f2_mul(y, s);
    return MINUS ? f2_sub(a, b) : f2_add(a, b);
}

// Rotate a lane's channels x (words 0-3: the run at a; 4-7: the run at b).
template <bool INTER, bool EXACT>
__device__ __forceinline__ void rotate(const Turn<INTER> &t, uint64_t (&x)[8]) {
    if (!t.on) return;
    if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, b;
            f2_split(x[i], a, b);
            x[i] = turned<EXACT, false>(x[i], t.c[i], f2(b, a), t.s[i], t.zero);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t a = x[i], b = x[i + 4];
            x[i] = turned<EXACT, true>(a, t.c[i], b, t.s[i], t.zero);
            x[i + 4] = turned<EXACT, false>(b, t.c[i], a, t.s[i], t.zero);
        }
    }
}

// Which token and which rows of it a warp takes: a CTA holds `wt` warps of
// each of its `tpc` tokens.
struct Place {
    int token, row0;
    bool ok;
};
template <int ROWS>
__device__ __forceinline__ Place place(int tokens, int wt, int tpc, int rows) {
    const int w = threadIdx.x / 32;
    Place p;
    p.token = static_cast<int>(blockIdx.x * static_cast<unsigned>(tpc)) + w / wt;
    p.row0 = (blockIdx.y * wt + w % wt) * ROWS;
    p.ok = p.token < tokens && p.token >= 0 && p.row0 < rows;
    return p;
}

// ------------------------------------------------------------------ norm + rotation
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(256, INTER ? 3 : 4) qk_norm_rope_kernel(const QkArgs a, int wt, int tpc) {
    constexpr int LPR = D / 16, RPW = 32 / LPR;
    const int rows = a.q_heads + a.kv_heads;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR;
    const Runs e = runs_of<INTER>(a.rot.rotary, lane % LPR);
    // (row r of k is k[(r - q_heads) D], so its base is moved back by the q heads)
    const uint16_t *q = a.q + p.token * a.q_stride;
    const uint16_t *k = a.k + p.token * a.k_stride - static_cast<int64_t>(a.q_heads) * D;
    uint4 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            const uint16_t *src = (r < a.q_heads ? q : k) + r * D;
            raw[u][0] = load16(src + e.a);
            raw[u][1] = load16(src + e.b);
        }
    }
    const Turn<INTER> t = load_turn<INTER>(a.rot, p.token, lane % LPR);
    uint16_t *qo = a.q_out + p.token * a.q_out_stride;
    uint16_t *ko = a.k_out + p.token * a.k_out_stride - static_cast<int64_t>(a.q_heads) * D;
    const uint16_t *held = nullptr;  // the weight that g holds
    uint4 g[2] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        const bool is_q = r < a.q_heads;
        uint64_t x[8];
        unpack8(raw[u][0], x);
        unpack8(raw[u][1], x + 4);
        const uint16_t *gamma = is_q ? a.q_gamma : a.k_gamma;
        if (gamma != held) {
            held = gamma;
            if (gamma != nullptr) g[0] = load16(gamma + e.a), g[1] = load16(gamma + e.b);
        }
        // the sum of squares in fp32: 64 or 128 terms, at most 2^39
        uint64_t s2 = f2_mul(x[0], x[0]), s3 = f2_mul(x[4], x[4]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = f2_fma(x[i], x[i], s2), s3 = f2_fma(x[4 + i], x[4 + i], s3);
        float ss, s1;
        f2_split(f2_add(s2, s3), ss, s1);
        ss += s1;
#pragma unroll
        for (int m = 1; m < LPR; m *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (gamma != nullptr) {
            const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
            const uint64_t r2 = f2(rs, rs);
            uint64_t w[8];
            unpack8(g[0], w);
            unpack8(g[1], w + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = f2_mul(f2_mul(x[i], r2), w[i]);
        }
        if (a.rot.rotary != 0) rotate<INTER, false>(t, x);
        if (r < rows) {
            uint16_t *dst = (is_q ? qo : ko) + r * D;
            store16(dst + e.a, pack8(x));
            store16(dst + e.b, pack8(x + 4));
        }
    }
}

// ------------------------------------------------------------------ append
// The codes of sixteen channels, each in the low bits of its word (INT4: code + 8,
// which four of add up to a word of nibbles).  The product t with the
// reciprocal is within 127 * 2^-23 = 1.6e-5 of the quotient and the rounded
// quotient within 0.8e-5 of it, so unless t lies within 4e-5 of a half-integer
// both round alike; t is rounded (half to even) by adding 1.5 * 2^23, whose low
// mantissa bits then are the code.  One channel in 12500 divides.
template <int BITS>
__device__ __forceinline__ void codes_of(const uint64_t (&x)[8], float s, float inv, uint32_t (&c)[16]) {
    constexpr int top = BITS == 4 ? 7 : 127, bias = BITS == 4 ? 8 : 0;
    const float kRound = 12582912.0f + bias;
    const uint64_t i2 = f2(inv, inv), k2 = f2(kRound, kRound);
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint64_t t = f2_mul(x[i], i2), m = f2_add(t, k2), d = f2_sub(t, f2_sub(m, k2));
        float a, b;
        f2_split(m, a, b);
        c[2 * i] = __float_as_uint(a);
        c[2 * i + 1] = __float_as_uint(b);
        f2_split(d, a, b);
        far = fmaxf(fmaxf(far, fabsf(a)), fabsf(b));
    }
    // outside this range the reciprocal or the products may leave fp32's
    if (!(far <= 0.49996f && s >= 1e-30f && s <= 1e30f)) {
        // the IEEE quotient; 0 / 0 and what an infinite or NaN scale gives
        // convert to zero
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a, b;
            f2_split(x[i], a, b);
            c[2 * i] = bias + max(-top, min(top, __float2int_rn(__fdiv_rn(a, s))));
            c[2 * i + 1] = bias + max(-top, min(top, __float2int_rn(__fdiv_rn(b, s))));
        }
    }
}

// The largest magnitude of sixteen channels, as bits (non-negative values order
// alike): NaN > infinity > finite, so a row that holds one keeps it in its
// scale.  The maximum itself ignores NaN; the sum of products with zero is NaN
// where a channel is not finite, and the bits are compared then.
__device__ __forceinline__ uint32_t largest(const uint64_t (&x)[8]) {
    float m = 0.0f;
    uint64_t z = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float a, b;
        f2_split(x[i], a, b);
        m = fmaxf(fmaxf(m, fabsf(a)), fabsf(b));
        z = f2_fma(x[i], 0ull, z);
    }
    uint32_t u = __float_as_uint(m);
    float z0, z1;
    f2_split(z, z0, z1);
    if (z0 + z1 != 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u = max(u, max(static_cast<uint32_t>(x[i]) & 0x7fffffffu,
                           static_cast<uint32_t>(x[i] >> 32) & 0x7fffffffu));
    }
    return u;
}

template <int D, bool INTER, int BITS, int U>
__global__ void __launch_bounds__(256, INTER ? 3 : 4) kv_append_kernel(const AppendArgs a, int wt, int tpc) {
    constexpr int LPR = D / 16, RPW = 32 / LPR, RB = D * BITS / 8;
    const int H = a.cache.heads, rows = 2 * H;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR;
    const int64_t slot = a.slots[p.token];
    const Runs e = runs_of<INTER>(a.rot.rotary, lane % LPR);
    // (row r of v is v[(r - H) D], so its base is moved back by the k heads)
    const uint16_t *ks = a.k + p.token * a.k_stride;
    const uint16_t *vs = a.v + p.token * a.v_stride - static_cast<int64_t>(H) * D;
    uint4 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            const uint16_t *src = (r < H ? ks : vs) + r * D;
            raw[u][0] = load16(src + e.a);
            raw[u][1] = load16(src + e.b);
        }
    }
    // (the slot is looked at only now: the rows are on their way meanwhile)
    const int64_t limit = static_cast<int64_t>(a.cache.pages) * a.cache.page_size;
    if (slot < 0 || slot >= limit) {  // a padded token, or a slot outside the cache: nothing is written
        if (slot >= limit && lane == 0) atomicAdd(&g_kv_bad_index, 1u);
        return;
    }
    const int shift = __ffs(a.cache.page_size) - 1;  // a power of two
    const int64_t page = slot >> shift, off = slot & (a.cache.page_size - 1);
    const int64_t row0 = ((page * H) << shift) + off;  // the token's row of head 0
    uint8_t *kd = static_cast<uint8_t *>(a.cache.k) + row0 * RB, *vd = static_cast<uint8_t *>(a.cache.v) + row0 * RB;
    Turn<INTER> t;
    t.on = false;
    if (a.rot.rotary != 0 && p.row0 < H) t = load_turn<INTER>(a.rot, p.token, lane % LPR);
    uint64_t x[U][8];
    float mine = 0.0f;  // of row u where lane % U == u: its largest magnitude
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        unpack8(raw[u][0], x[u]);
        unpack8(raw[u][1], x[u] + 4);
        if (r < H) rotate<INTER, true>(t, x[u]);
        if (BITS == 16) continue;
        uint32_t m = largest(x[u]);
#pragma unroll
        for (int s = 1; s < LPR; s *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
        if (lane % U == u) mine = __uint_as_float(m);
    }
    // the two divisions of a row are made by one lane in U
    constexpr int top = BITS == 4 ? 7 : 127;
    float scale_u = 0.0f, inv_u = 0.0f;
    if (BITS != 16) {
        scale_u = __fdiv_rn(mine, static_cast<float>(top));
        inv_u = __frcp_rn(scale_u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        const bool is_k = r < H;
        const int at_head = (is_k ? r : r - H) << shift;  // rows from the token's first head
        uint8_t *dst = (is_k ? kd : vd) + at_head * RB;
        if (BITS == 16) {
            if (r < rows) {
                store16(dst + 2 * e.a, pack8(x[u]));
                store16(dst + 2 * e.b, pack8(x[u] + 4));
            }
            continue;
        }
        const int src = (lane & ~(LPR - 1)) | u;
        const float scale = __shfl_sync(0xffffffffu, scale_u, src);
        const float inv = __shfl_sync(0xffffffffu, inv_u, src);
        if (r >= rows) continue;
        uint32_t c[16];
        codes_of<BITS>(x[u], scale, inv, c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // the run at a, the run at b
            const uint32_t *q = c + 8 * i;
            const int at = i ? e.b : e.a;
            if (BITS == 8) {
                uint32_t w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    w[j] = __byte_perm(__byte_perm(q[4 * j], q[4 * j + 1], 0x0040),
                                       __byte_perm(q[4 * j + 2], q[4 * j + 3], 0x0040), 0x5410);
                *reinterpret_cast<uint2 *>(dst + at) = make_uint2(w[0], w[1]);
            } else {  // 8 more in every nibble is its top bit flipped
                *reinterpret_cast<uint32_t *>(dst + at / 2) =
                    __byte_perm(q[0] + q[1] * 16 + q[2] * 256 + q[3] * 4096,
                                q[4] + q[5] * 16 + q[6] * 256 + q[7] * 4096, 0x5410) ^
                    0x88888888u;
            }
        }
        if (lane % LPR == 0) (is_k ? a.cache.k_scale : a.cache.v_scale)[row0 + at_head] = scale;
    }
}

// ------------------------------------------------------------------ read back
template <int D, int BITS, int U>
__global__ void __launch_bounds__(256) kv_gather_kernel(const GatherArgs a, int wt, int tpc) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, RB = D * BITS / 8;
    const int H = a.cache.heads, rows = 2 * H;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR, e0 = lane % LPR * 8;
    const int64_t slot = a.slots[p.token];
    const int64_t limit = static_cast<int64_t>(a.cache.pages) * a.cache.page_size;
    const bool live = slot >= 0 && slot < limit;
    if (slot >= limit && lane == 0) atomicAdd(&g_kv_bad_index, 1u);
    const int shift = __ffs(a.cache.page_size) - 1;  // a power of two
    const int64_t page = live ? slot >> shift : 0, off = live ? slot & (a.cache.page_size - 1) : 0;
    const int64_t row0 = ((page * H) << shift) + off;  // the token's row of head 0
    const uint8_t *kd = static_cast<const uint8_t *>(a.cache.k) + row0 * RB;
    const uint8_t *vd = static_cast<const uint8_t *>(a.cache.v) + row0 * RB;
    uint4 raw[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u] = make_uint4(0, 0, 0, 0);
        scale[u] = 0.0f;
        if (r < rows && live) {
            const bool is_k = r < H;
            const int at_head = (is_k ? r : r - H) << shift;
            const uint8_t *src = (is_k ? kd : vd) + at_head * RB;
            if (BITS == 16) raw[u] = *reinterpret_cast<const uint4 *>(src + 2 * e0);
            if (BITS == 8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src + e0);
                raw[u].x = w.x;
                raw[u].y = w.y;
            }
            if (BITS == 4) raw[u].x = *reinterpret_cast<const uint32_t *>(src + e0 / 2);
            if (BITS != 16) scale[u] = (is_k ? a.cache.k_scale : a.cache.v_scale)[row0 + at_head];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        if (r >= rows) continue;
        uint4 out = raw[u];
        if (BITS != 16) {
            // a code's bits (offset to be non-negative) under the exponent of
            // 2^10, or four bits up of 2^6, of an fp16: that plus the code
            uint32_t h[4];
            if (BITS == 8) {
                const uint32_t w0 = raw[u].x ^ 0x80808080u, w1 = raw[u].y ^ 0x80808080u;
                h[0] = __byte_perm(w0, 0x64006400u, 0x5150), h[1] = __byte_perm(w0, 0x64006400u, 0x5352);
                h[2] = __byte_perm(w1, 0x64006400u, 0x5150), h[3] = __byte_perm(w1, 0x64006400u, 0x5352);
            } else {  // pairs (0, 4), (1, 5), (2, 6), (3, 7)
                const uint32_t w = raw[u].x, y = w >> 8;
                h[0] = ((w ^ 0x88888888u) & 0x000f000fu) | 0x64006400u;
                h[1] = ((w ^ 0x88888888u) & 0x00f000f0u) | 0x54005400u;
                h[2] = ((y ^ 0x88888888u) & 0x000f000fu) | 0x64006400u;
                h[3] = ((y ^ 0x88888888u) & 0x00f000f0u) | 0x54005400u;
            }
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float base = BITS == 8 ? 1152.0f : i % 2 ? 72.0f : 1032.0f;
                const float2 v = __half22float2(__hsub2(*reinterpret_cast<const __half2 *>(&h[i]),
                                                        __float2half2_rn(base)));
                f[BITS == 8 ? 2 * i : i] = v.x;
                f[BITS == 8 ? 2 * i + 1 : i + 4] = v.y;
            }
            uint64_t x[4];
            const uint64_t s2 = f2(scale[u], scale[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2(f[2 * i], f[2 * i + 1]), s2);
            out = live ? pack8(x) : make_uint4(0, 0, 0, 0);
        }
        uint16_t *o = r < H ? a.k_out + p.token * a.k_stride + r * D
                            : a.v_out + p.token * a.v_stride + (r - H) * D;
        *reinterpret_cast<uint4 *>(o + e0) = out;
    }
}

// Warps of a token, tokens of a CTA and the grid, when a warp takes `per` rows.
struct Launch {
    dim3 grid;
    int threads, wt, tpc;
};
Launch plan(int tokens, int rows, int per) {
    const int chunks = (rows + per - 1) / per;
    Launch l;
    l.wt = chunks < 8 ? chunks : 8;
    l.tpc = 8 / l.wt;
    l.threads = 32 * l.wt * l.tpc;
    l.grid = dim3((tokens + static_cast<unsigned>(l.tpc) - 1) / l.tpc, (chunks + l.wt - 1) / l.wt);
    return l;
}

// Rows in flight per lane group: several hide the memory latency of a long call
// (a warp then has 2 to 4 KB of loads outstanding); a call with too few rows to
// fill the SMs that way takes one row a lane group, for more warps.
bool deep(int tokens, int rows, int per) {
    return static_cast<int64_t>(tokens) * rows >= static_cast<int64_t>(sm_count()) * 16 * per;
}

template <int D, bool INTER>
cudaError_t run_qk(const QkArgs &a, cudaStream_t stream) {
    constexpr int RPW = 512 / D, U = 2;
    const int rows = a.q_heads + a.kv_heads;
    if (deep(a.tokens, rows, U * RPW)) {
        const Launch l = plan(a.tokens, rows, U * RPW);
        qk_norm_rope_kernel<D, INTER, U><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    } else {
        const Launch l = plan(a.tokens, rows, RPW);
        qk_norm_rope_kernel<D, INTER, 1><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    }
    return cudaGetLastError();
}

template <int D, bool INTER, int BITS>
cudaError_t run_append(const AppendArgs &a, cudaStream_t stream) {
    constexpr int RPW = 512 / D, U = 2;
    const int rows = 2 * a.cache.heads;
    if (deep(a.tokens, rows, U * RPW)) {
        const Launch l = plan(a.tokens, rows, U * RPW);
        kv_append_kernel<D, INTER, BITS, U><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    } else {
        const Launch l = plan(a.tokens, rows, RPW);
        kv_append_kernel<D, INTER, BITS, 1><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    }
    return cudaGetLastError();
}

template <int D, int BITS>
cudaError_t run_gather(const GatherArgs &a, cudaStream_t stream) {
    constexpr int RPW = 256 / D;
    const int rows = 2 * a.cache.heads;
    if (deep(a.tokens, rows, 4 * RPW)) {
        const Launch l = plan(a.tokens, rows, 4 * RPW);
        kv_gather_kernel<D, BITS, 4><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    } else {
        const Launch l = plan(a.tokens, rows, RPW);
        kv_gather_kernel<D, BITS, 1><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    }
    return cudaGetLastError();
}

template <int D, bool INTER>
cudaError_t append_bits(const AppendArgs &a, cudaStream_t stream) {
    if (a.cache.kv_type == QUIK_KV_INT4) return run_append<D, INTER, 4>(a, stream);
    if (a.cache.kv_type == QUIK_KV_INT8) return run_append<D, INTER, 8>(a, stream);
    return run_append<D, INTER, 16>(a, stream);
}

template <int D>
cudaError_t gather_bits(const GatherArgs &a, cudaStream_t stream) {
    if (a.cache.kv_type == QUIK_KV_INT4) return run_gather<D, 4>(a, stream);
    if (a.cache.kv_type == QUIK_KV_INT8) return run_gather<D, 8>(a, stream);
    return run_gather<D, 16>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t stream) {
    if (a.head_dim == 64)
        return a.rot.interleaved ? run_qk<64, true>(a, stream) : run_qk<64, false>(a, stream);
    return a.rot.interleaved ? run_qk<128, true>(a, stream) : run_qk<128, false>(a, stream);
}

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t stream) {
    if (a.cache.head_dim == 64)
        return a.rot.interleaved ? append_bits<64, true>(a, stream) : append_bits<64, false>(a, stream);
    return a.rot.interleaved ? append_bits<128, true>(a, stream) : append_bits<128, false>(a, stream);
}

cudaError_t launch_kv_gather(const GatherArgs &a, cudaStream_t stream) {
    return a.cache.head_dim == 64 ? gather_bits<64>(a, stream) : gather_bits<128>(a, stream);
}

unsigned int take_row_errors() {
    unsigned int word = 0;
    if (cudaMemcpyFromSymbol(&word, g_kv_bad_index, sizeof(word)) != cudaSuccess) return 0;
    return counter_increase(kCounterBadRow, word);
}

}  // namespace quik
