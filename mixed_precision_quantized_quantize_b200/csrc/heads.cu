// heads.cu -- the row kernels between the QKV projection and the attention:
// the per-head RMS norm with the rotation (qk_norm_rope), the append of K and
// V rows to the paged cache (kv_append) and the read-back (kv_gather).
//
// A row is one head of one token, D = 64 or 128 channels.  D / 8 lanes hold a
// row, eight channels each, so a warp holds 4 or 2 rows and all reductions over
// a row are shuffles inside that lane group.  A lane's eight channels are two
// runs of four, placed so that both channels of every rotated pair are in the
// same lane: with pairs (i, i + rotary_dim / 2) a run and the one rotary_dim / 2
// further on, otherwise two adjacent runs.  The rotation then needs no exchange
// between lanes.  (With 16-byte loads and the partner's channels shuffled in,
// norm and rotation of 2048 x 64 heads took 18.6 us.)  The table entries of a
// token are loaded once and serve all the rows that a warp takes of it.
//
// All three kernels are bound by memory: every channel is read once and
// written once.
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

__device__ __forceinline__ uint2 load8(const void *p) { return *reinterpret_cast<const uint2 *>(p); }
__device__ __forceinline__ void store8(void *p, uint2 v) { *reinterpret_cast<uint2 *>(p) = v; }

// Four fp16 channels as two fp32 pairs, and back (rounded to nearest).
__device__ __forceinline__ void unpack4(uint2 v, uint64_t *x) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
    x[0] = f2(a.x, a.y);
    x[1] = f2(b.x, b.y);
}
__device__ __forceinline__ uint2 pack4(const uint64_t *x) {
    float a, b;
    uint2 v;
    f2_split(x[0], a, b);
    __half2 h = __floats2half2_rn(a, b);
    v.x = *reinterpret_cast<const uint32_t *>(&h);
    f2_split(x[1], a, b);
    h = __floats2half2_rn(a, b);
    v.y = *reinterpret_cast<const uint32_t *>(&h);
    return v;
}

// A lane's channels: runs of four at a and b.
struct Runs {
    int a, b;
};
template <bool INTER>
__device__ __forceinline__ Runs runs_of(int rotary, int i) {
    const int half = rotary / 2;
    Runs r;
    if (!INTER && 4 * i < half) {
        r.a = 4 * i;
        r.b = half + 4 * i;
    } else {
        r.a = 8 * i;  // (half-split: the i-th run pair from rotary_dim on is at 2 * 4 i, too)
        r.b = r.a + 4;
    }
    return r;
}

// The rotation of one token, as this lane needs it: cosines and sines of its
// four pairs.
struct Turn {
    float c[4], s[4];
    bool on;  // this lane's channels are rotated
};

template <bool INTER>
__device__ __forceinline__ Turn load_turn(const RotaryArgs &r, int token, int i) {
    Turn t;
    const int half = r.rotary / 2;
    t.on = 4 * i < half;
    if (r.rotary == 0) return t;
    int pos = r.positions[token];
    if (pos < 0 || pos >= r.rows) {
        if (threadIdx.x % 32 == 0) atomicAdd(&g_kv_bad_index, 1u);
        pos = 0;
    }
    if (t.on) {
        // pairs 4 i .. 4 i + 3 in both forms
        const int64_t at = static_cast<int64_t>(pos) * half + 4 * i;
        const float4 c = *reinterpret_cast<const float4 *>(r.cos + at);
        const float4 s = *reinterpret_cast<const float4 *>(r.sin + at);
        t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
        t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
    }
    return t;
}

// Rotate a lane's channels x (pairs 0, 1: the run at a; 2, 3: the run at b) in
// IEEE steps, each product and each sum rounded: the values, and so the codes
// made of them, are then the same wherever they are computed.  (Paired
// products followed by a paired sum came out with one rounding instead of two.)
template <bool INTER>
__device__ __forceinline__ void rotate(const Turn &t, uint64_t (&x)[4]) {
    if (!t.on) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(x[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : i + 4;
        const float a = v[ia], b = v[ib];
        v[ia] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
        v[ib] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f2(v[2 * i], v[2 * i + 1]);
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
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkArgs a, int wt, int tpc) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int rows = a.q_heads + a.kv_heads;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR;
    const Runs e = runs_of<INTER>(a.rot.rotary, lane % LPR);
    const uint16_t *q = a.q + p.token * a.q_stride, *k = a.k + p.token * a.k_stride;
    uint2 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u][0] = raw[u][1] = make_uint2(0, 0);
        if (r < rows) {
            const uint16_t *src = r < a.q_heads ? q + r * D : k + (r - a.q_heads) * D;
            raw[u][0] = load8(src + e.a);
            raw[u][1] = load8(src + e.b);
        }
    }
    const Turn t = load_turn<INTER>(a.rot, p.token, lane % LPR);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        const bool is_q = r < a.q_heads;
        uint64_t x[4];
        unpack4(raw[u][0], x);
        unpack4(raw[u][1], x + 2);
        const uint16_t *gamma = is_q ? a.q_gamma : a.k_gamma;
        // the sum of squares in fp32: 64 or 128 terms, at most 2^39
        uint64_t s2 = f2_mul(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) s2 = f2_fma(x[i], x[i], s2);
        float ss, s1;
        f2_split(s2, ss, s1);
        ss += s1;
#pragma unroll
        for (int m = 1; m < LPR; m *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (gamma != nullptr) {
            const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
            const uint64_t r2 = f2(rs, rs);
            uint64_t g[4];
            unpack4(load8(gamma + e.a), g);
            unpack4(load8(gamma + e.b), g + 2);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = f2_mul(f2_mul(x[i], r2), g[i]);
        }
        if (a.rot.rotary != 0) rotate<INTER>(t, x);
        if (r < rows) {
            uint16_t *dst = is_q ? a.q_out + p.token * a.q_out_stride + r * D
                                 : a.k_out + p.token * a.k_out_stride + (r - a.q_heads) * D;
            store8(dst + e.a, pack4(x));
            store8(dst + e.b, pack4(x + 2));
        }
    }
}

// ------------------------------------------------------------------ append
// The codes of eight channels, each in the low bits of its word (INT4: code + 8,
// which four of add up to a word of nibbles).  The product t with the
// reciprocal is within 127 * 2^-23 = 1.6e-5 of the quotient and the rounded
// quotient within 0.8e-5 of it, so unless t lies within 4e-5 of a half-integer
// both round alike; t is rounded (half to even) by adding 1.5 * 2^23, whose low
// mantissa bits then are the code.  One channel in 12500 divides.
template <int BITS>
__device__ __forceinline__ void codes_of(const uint64_t (&x)[4], float s, float inv, uint32_t (&c)[8]) {
    constexpr int top = BITS == 4 ? 7 : 127, bias = BITS == 4 ? 8 : 0;
    const float kRound = 12582912.0f + bias;
    const uint64_t i2 = f2(inv, inv), k2 = f2(kRound, kRound);
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_split(x[i], a, b);
            c[2 * i] = bias + max(-top, min(top, __float2int_rn(__fdiv_rn(a, s))));
            c[2 * i + 1] = bias + max(-top, min(top, __float2int_rn(__fdiv_rn(b, s))));
        }
    }
}

// The largest magnitude of eight channels, as bits (non-negative values order
// alike): NaN > infinity > finite, so a row that holds one keeps it in its
// scale.  The maximum itself ignores NaN; the sum of products with zero is NaN
// where a channel is not finite, and the bits are compared then.
__device__ __forceinline__ uint32_t largest(const uint64_t (&x)[4]) {
    float m = 0.0f;
    uint64_t z = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
        for (int i = 0; i < 4; ++i)
            u = max(u, max(static_cast<uint32_t>(x[i]) & 0x7fffffffu,
                           static_cast<uint32_t>(x[i] >> 32) & 0x7fffffffu));
    }
    return u;
}

template <int D, bool INTER, int BITS, int U>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(const AppendArgs a, int wt, int tpc) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, RB = D * BITS / 8;
    const int H = a.cache.heads, rows = 2 * H;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR;
    const int64_t slot = a.slots[p.token];
    const int64_t limit = static_cast<int64_t>(a.cache.pages) * a.cache.page_size;
    if (slot < 0 || slot >= limit) {  // a padded token, or a slot outside the cache: nothing is written
        if (slot >= limit && lane == 0) atomicAdd(&g_kv_bad_index, 1u);
        return;
    }
    const Runs e = runs_of<INTER>(a.rot.rotary, lane % LPR);
    const uint16_t *ks = a.k + p.token * a.k_stride, *vs = a.v + p.token * a.v_stride;
    uint2 raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u][0] = raw[u][1] = make_uint2(0, 0);
        if (r < rows) {
            const uint16_t *src = r < H ? ks + r * D : vs + (r - H) * D;
            raw[u][0] = load8(src + e.a);
            raw[u][1] = load8(src + e.b);
        }
    }
    const int shift = __ffs(a.cache.page_size) - 1;  // a power of two
    const int64_t page = slot >> shift, off = slot & (a.cache.page_size - 1);
    const int64_t row0 = ((page * H) << shift) + off;  // the token's row of head 0
    uint8_t *kd = static_cast<uint8_t *>(a.cache.k) + row0 * RB, *vd = static_cast<uint8_t *>(a.cache.v) + row0 * RB;
    Turn t;
    t.on = false;
    if (a.rot.rotary != 0 && p.row0 < H) t = load_turn<INTER>(a.rot, p.token, lane % LPR);
    uint64_t x[U][4];
    float mine = 0.0f;  // of row u where lane % U == u: its largest magnitude
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        unpack4(raw[u][0], x[u]);
        unpack4(raw[u][1], x[u] + 2);
        if (r < H) rotate<INTER>(t, x[u]);
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
                store8(dst + 2 * e.a, pack4(x[u]));
                store8(dst + 2 * e.b, pack4(x[u] + 2));
            }
            continue;
        }
        const int src = (lane & ~(LPR - 1)) | u;
        const float scale = __shfl_sync(0xffffffffu, scale_u, src);
        const float inv = __shfl_sync(0xffffffffu, inv_u, src);
        if (r >= rows) continue;
        uint32_t c[8];
        codes_of<BITS>(x[u], scale, inv, c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // the run at a, the run at b
            const uint32_t *q = c + 4 * i;
            const int at = i ? e.b : e.a;
            if (BITS == 8)
                *reinterpret_cast<uint32_t *>(dst + at) =
                    __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
            else  // 8 more in every nibble is its top bit flipped
                *reinterpret_cast<uint16_t *>(dst + at / 2) =
                    static_cast<uint16_t>((q[0] + q[1] * 16 + q[2] * 256 + q[3] * 4096) ^ 0x8888u);
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
                const uint2 w = load8(src + e0);
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
            const uint2 lo = pack4(x), hi = pack4(x + 2);
            out = live ? make_uint4(lo.x, lo.y, hi.x, hi.y) : make_uint4(0, 0, 0, 0);
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

// Rows in flight per lane group: four hide the memory latency of a long call
// (each warp then has 2 KB of loads outstanding); a call with too few rows to
// fill the SMs that way takes one row a lane group, for more warps.
bool deep(int tokens, int rows, int rpw) {
    return static_cast<int64_t>(tokens) * rows >= static_cast<int64_t>(sm_count()) * 16 * 4 * rpw;
}

template <int D, bool INTER>
cudaError_t run_qk(const QkArgs &a, cudaStream_t stream) {
    constexpr int RPW = 256 / D;
    const int rows = a.q_heads + a.kv_heads;
    if (deep(a.tokens, rows, RPW)) {
        const Launch l = plan(a.tokens, rows, 4 * RPW);
        qk_norm_rope_kernel<D, INTER, 4><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    } else {
        const Launch l = plan(a.tokens, rows, RPW);
        qk_norm_rope_kernel<D, INTER, 1><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
    }
    return cudaGetLastError();
}

template <int D, bool INTER, int BITS>
cudaError_t run_append(const AppendArgs &a, cudaStream_t stream) {
    constexpr int RPW = 256 / D;
    const int rows = 2 * a.cache.heads;
    if (deep(a.tokens, rows, RPW)) {
        const Launch l = plan(a.tokens, rows, 4 * RPW);
        kv_append_kernel<D, INTER, BITS, 4><<<l.grid, l.threads, 0, stream>>>(a, l.wt, l.tpc);
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
    if (deep(a.tokens, rows, RPW)) {
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
