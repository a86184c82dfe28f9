// heads.cu -- the row kernels between the QKV projection and the attention:
// the per-head RMS norm with the rotation (qk_norm_rope), the append of K and
// V rows to the paged cache (kv_append) and the read-back (kv_gather).
//
// A row is one head of one token, D = 64 or 128 channels.  D / 8 lanes hold a
// row, eight channels (one 16-byte load) each, so a warp holds 4 or 2 rows,
// and all reductions over a row are shuffles inside that lane group.  The
// rotation's partner of a channel lies in the same lane (adjacent pairs) or
// rotary_dim / 2 channels away, a whole number of lanes (rotary_dim % 16 ==
// 0): one shuffle.  The table entries of a token are loaded once and serve
// all the rows that a warp takes of that token.
//
// All three kernels are bound by memory: every channel is read once and
// written once, in 16-byte units.
#include "quik_internal.h"

#include <cuda_fp16.h>

namespace quik {

// Rows whose position or slot was outside its range: only ever grows;
// quik_sync_check reports the increase.
__device__ unsigned int g_kv_bad_index;

namespace {

__device__ __forceinline__ uint4 load16(const void *p) {
    return *reinterpret_cast<const uint4 *>(p);
}

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The rotation of one token, as this lane needs it: cosines and sines of its
// channels (adjacent pairs: the first four entries).  In the half-split form
// the sine carries the sign, so that both halves are own * c + partner * s.
struct Turn {
    float c[8], s[8];
    int lanes;  // distance to the partner's lane (half-split)
    bool on;    // this lane's channels are rotated
};

template <bool INTER>
__device__ __forceinline__ Turn load_turn(const RotaryArgs &r, int token, int e0) {
    Turn t;
    t.on = e0 < r.rotary;
    t.lanes = 0;
    if (r.rotary == 0) return t;
    int pos = r.positions[token];
    if (pos < 0 || pos >= r.rows) {
        if (threadIdx.x % 32 == 0) atomicAdd(&g_kv_bad_index, 1u);
        pos = 0;
    }
    const int half = r.rotary / 2;
    const int64_t at = static_cast<int64_t>(pos) * half;
    if (INTER) {
        if (t.on) {
            const float4 c = *reinterpret_cast<const float4 *>(r.cos + at + e0 / 2);
            const float4 s = *reinterpret_cast<const float4 *>(r.sin + at + e0 / 2);
            t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
            t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
        }
    } else {
        const bool low = e0 < half;
        t.lanes = t.on ? (low ? half / 8 : -(half / 8)) : 0;
        if (t.on) {
            const int64_t i = at + (low ? e0 : e0 - half);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 c = *reinterpret_cast<const float4 *>(r.cos + i + 4 * h);
                const float4 s = *reinterpret_cast<const float4 *>(r.sin + i + 4 * h);
                t.c[4 * h] = c.x, t.c[4 * h + 1] = c.y, t.c[4 * h + 2] = c.z, t.c[4 * h + 3] = c.w;
                t.s[4 * h] = low ? -s.x : s.x, t.s[4 * h + 1] = low ? -s.y : s.y;
                t.s[4 * h + 2] = low ? -s.z : s.z, t.s[4 * h + 3] = low ? -s.w : s.w;
            }
        }
    }
    return t;
}

// Rotate x (eight channels of a row) in IEEE steps, each product and each sum
// rounded: the values (and so the codes made of them) are then the same
// whatever the compiler would contract.  Every lane of the warp calls it.
template <bool INTER>
__device__ __forceinline__ void rotate(const Turn &t, float (&x)[8]) {
    if (INTER) {
        if (t.on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
                x[2 * i + 1] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
            }
        }
    } else {
        const int src = (threadIdx.x + t.lanes) & 31;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, x[i], src);
            if (t.on) x[i] = __fadd_rn(__fmul_rn(x[i], t.c[i]), __fmul_rn(o, t.s[i]));
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
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkArgs a, int wt, int tpc) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int rows = a.q_heads + a.kv_heads;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR, e0 = lane % LPR * 8;
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (r < a.q_heads)
            raw[u] = load16(a.q + p.token * a.q_stride + r * D + e0);
        else if (r < rows)
            raw[u] = load16(a.k + p.token * a.k_stride + (r - a.q_heads) * D + e0);
    }
    const Turn t = load_turn<INTER>(a.rot, p.token, e0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        const bool is_q = r < a.q_heads;
        float x[8];
        unpack8(raw[u], x);
        const uint16_t *gamma = is_q ? a.q_gamma : a.k_gamma;
        // the sum of squares in fp32: 64 or 128 terms, at most 2^39
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = 1; m < LPR; m *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        if (gamma != nullptr) {
            const float rs = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            float g[8];
            unpack8(load16(gamma + e0), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * g[i];
        }
        if (a.rot.rotary != 0) rotate<INTER>(t, x);
        if (r < rows) {
            uint16_t *o = is_q ? a.q_out + p.token * a.q_out_stride + r * D
                               : a.k_out + p.token * a.k_out_stride + (r - a.q_heads) * D;
            *reinterpret_cast<uint4 *>(o + e0) = pack8(x);
        }
    }
}

// ------------------------------------------------------------------ append
// rint(v / s) with the IEEE quotient, for |v / s| <= 127 (+ rounding).  The
// product with the reciprocal is within 127 * 2^-23 of the quotient, so
// wherever it is further than 1e-4 from a half-integer both round alike; the
// rest (and every non-finite case, where the comparison fails) divides.
__device__ __forceinline__ int code_of(float v, float s, float inv, int top) {
    const float t = v * inv;
    float q = rintf(t);
    if (!(fabsf(t - q) <= 0.4999f)) q = rintf(__fdiv_rn(v, s));
    const int c = __float2int_rn(q);  // NaN gives 0
    return max(-top, min(top, c));
}

template <int D, bool INTER, int BITS, int U>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a, int wt, int tpc) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, RB = D * BITS / 8;
    const int H = a.cache.heads, rows = 2 * H;
    const Place p = place<U * RPW>(a.tokens, wt, tpc, rows);
    if (!p.ok) return;
    const int lane = threadIdx.x % 32, sub = lane / LPR, e0 = lane % LPR * 8;
    const int64_t slot = a.slots[p.token];
    const int64_t limit = static_cast<int64_t>(a.cache.pages) * a.cache.page_size;
    if (slot < 0 || slot >= limit) {  // a padded token, or a slot outside the cache: nothing is written
        if (slot >= limit && lane == 0) atomicAdd(&g_kv_bad_index, 1u);
        return;
    }
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (r < H)
            raw[u] = load16(a.k + p.token * a.k_stride + r * D + e0);
        else if (r < rows)
            raw[u] = load16(a.v + p.token * a.v_stride + (r - H) * D + e0);
    }
    const int64_t page = slot / a.cache.page_size, off = slot % a.cache.page_size;
    Turn t;
    const bool any_k = a.rot.rotary != 0 && p.row0 < H;
    if (any_k) t = load_turn<INTER>(a.rot, p.token, e0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        const bool is_k = r < H;
        const int h = is_k ? r : r - H;
        float x[8];
        unpack8(raw[u], x);
        if (any_k) {
            // a warp may hold rows of both: the shuffles are for all, the result for K
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i];
            rotate<INTER>(t, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = is_k ? y[i] : x[i];
        }
        const int64_t row = (page * H + h) * a.cache.page_size + off;
        uint8_t *dst = static_cast<uint8_t *>(is_k ? a.cache.k : a.cache.v) + row * RB;
        if (BITS == 16) {
            if (r < rows) *reinterpret_cast<uint4 *>(dst + 2 * e0) = pack8(x);
            continue;
        }
        // the row's largest magnitude, on the bits: NaN > infinity > finite, so
        // a row that holds one keeps it in its scale
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
        for (int s = 1; s < LPR; s *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, s));
        constexpr int top = BITS == 4 ? 7 : 127;
        const float scale = __fdiv_rn(__uint_as_float(m), static_cast<float>(top));
        int c[8] = {};
        if (scale != 0.0f) {
            const float inv = __frcp_rn(scale);
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = code_of(x[i], scale, inv, top);
        }
        if (r >= rows) continue;
        if (BITS == 8) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = (c[4 * i] & 255) | (c[4 * i + 1] & 255) << 8 | (c[4 * i + 2] & 255) << 16 |
                       static_cast<uint32_t>(c[4 * i + 3]) << 24;
            *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(w[0], w[1]);
        } else {
            uint32_t w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= static_cast<uint32_t>(c[i] & 15) << (4 * i);
            *reinterpret_cast<uint32_t *>(dst + e0 / 2) = w;
        }
        if (e0 == 0) (is_k ? a.cache.k_scale : a.cache.v_scale)[row] = scale;
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
    const int64_t page = live ? slot / a.cache.page_size : 0, off = live ? slot % a.cache.page_size : 0;
    uint4 raw[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        raw[u] = make_uint4(0, 0, 0, 0);
        scale[u] = 0.0f;
        if (r < rows && live) {
            const bool is_k = r < H;
            const int64_t row = (page * H + (is_k ? r : r - H)) * a.cache.page_size + off;
            const uint8_t *src = static_cast<const uint8_t *>(is_k ? a.cache.k : a.cache.v) + row * RB;
            if (BITS == 16) raw[u] = load16(src + 2 * e0);
            if (BITS == 8) {
                const uint2 w = *reinterpret_cast<const uint2 *>(src + e0);
                raw[u].x = w.x;
                raw[u].y = w.y;
            }
            if (BITS == 4) raw[u].x = *reinterpret_cast<const uint32_t *>(src + e0 / 2);
            if (BITS != 16) scale[u] = (is_k ? a.cache.k_scale : a.cache.v_scale)[row];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int r = p.row0 + u * RPW + sub;
        if (r >= rows) continue;
        uint4 out = raw[u];
        if (BITS != 16) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int c;
                if (BITS == 8)
                    c = static_cast<int8_t>((i < 4 ? raw[u].x : raw[u].y) >> (8 * (i % 4)));
                else
                    c = static_cast<int>(raw[u].x << (28 - 4 * i)) >> 28;
                x[i] = __fmul_rn(static_cast<float>(c), scale[u]);
            }
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
