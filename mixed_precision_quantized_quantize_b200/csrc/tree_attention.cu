// tree_attention.cu -- attention of drafted tokens over the paged KV cache
// (fp16, INT8 or packed INT4 rows).
//
// Per sequence and key head, the G = q_heads / heads query heads of the new
// tokens are the rows of one small matrix (row r: new token r / G, head r % G),
// so that a cached row is read once for all of them.  For tiles of 32 cached
// tokens:
//     S = Q K^T             m16n8k16 products, fp32 sums
//     t = scale * log2(e) * k_scale * S
//     m' = max(m, max t), p = 2^(t - m' + 14), l += p, O = O 2^(m - m') + p V
// The running maximum and sum are fp32.  p is rounded to fp16 for its product
// with V; the factor 2^14 (it cancels in O / l) keeps p's far below the maximum
// out of fp16's subnormal range, and p <= 2^14 stays below its largest value.
// Quantised values enter the product as their integer codes, exact in fp16;
// their scale multiplies p in fp32 before that rounding, relative to a row's running
// power of two 2^R above every scale that the row has seen so far (its O then is
// in units of 2^R), so p stays within fp16 whatever the scales are, and a token
// that the row does not see has no part in it.
#include "attention.cuh"

namespace quik {

namespace {

using Params = AttnParams;
constexpr int kTile = 32;          // cached tokens per tile
constexpr float kShift = 14.0f;    // p carries 2^14
constexpr int kMaxSplits = 64;
constexpr float kFirstUnit = 0x1p100f;  // 2^-R, no scale seen yet
// WR warps share a tile, 16 rows each; NW / WR such groups take tiles in turn.
template <int BITS_, int D_, int WR_, int NW_>
struct Cfg {
    static constexpr int BITS = BITS_, D = D_, WR = WR_, NW = NW_;
    static constexpr int TG = NW / WR;
    static constexpr int RB = D * BITS / 8;  // bytes of a cached row
    static constexpr int CPR = RB / 16;
    // row pitches in shared memory: with 16 bytes of padding the 8 rows that a
    // fragment load touches fall into different banks; rows of 32 or 64 bytes
    // of K are read whole, in order, and need none
    static constexpr int KS = RB >= 128 ? RB + 16 : RB;
    static constexpr int VS = RB + 16;
    static constexpr int SCALES = BITS == 16 ? 0 : 2 * kTile * 4;
    static constexpr int STAGE = kTile * (KS + VS) + SCALES + 16;
    static constexpr int STAGES = 3;
    static constexpr int RING = TG * STAGES * STAGE;
    static constexpr int OP = D + 4;  // pitch of an output row at the merge (floats)
    static constexpr int MERGE = NW * 16 * OP * 4 + NW * 16 * 8;
    static constexpr int SMEM = RING > MERGE ? RING : MERGE;
    static constexpr int ROWS = 16 * WR;
    static constexpr int STEPS = D / 16;  // products along a head
    static constexpr int NT = D / 8;      // output column tiles
};

// The cached rows of one sequence and key head, tile by tile, into a ring of
// stages in shared memory.  TH threads (a warp, or the WR warps that share a
// tile) copy together.  Pages hold 16 tokens or more, so each half of a tile is
// contiguous in memory: two row offsets, one page number each, place it all.
template <class C>
struct Tiles {
    static constexpr int TH = 32 * C::WR;
    const uint8_t *k, *v;   // this thread's place in the head's rows of page 0
    const float *ks, *vs;   // this lane's scale there
    const int32_t *table;
    uint8_t *ring;
    unsigned page_rows;     // rows of a page, all heads
    int page_shift, pages, end, total;
    int gt;                 // thread among the TH
    bool report;

    // Page of the half of the tile that this lane stands for (lanes 0-15, 16-31); -1: none.
    __device__ __forceinline__ int page_of(int tile) const {
        const int pos = tile * kTile + (threadIdx.x & 16);
        if (tile >= end || pos >= total) return -1;
        const int id = table[pos >> page_shift];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(pages)) return id;
        if (report && (threadIdx.x & 15) == 0) atomicAdd(&g_attn_bad_index, 1u);
        return -1;
    }
    // Start the copies of a tile (id: page_of of it).
    __device__ __forceinline__ void issue(int tile, int stage, int id) const {
        uint8_t *st = ring + stage * C::STAGE;
        const int t = gt / C::CPR, c = gt % C::CPR;
        const uint32_t ka = smem_addr(st) + t * C::KS + c * 16;
        const uint32_t va = smem_addr(st) + kTile * C::KS + t * C::VS + c * 16;
        const int left = total - tile * kTile;  // tokens from the tile's first one on
        const int p0 = __shfl_sync(0xffffffffu, id, 0), p1 = __shfl_sync(0xffffffffu, id, 16);
        const int in_page = tile * kTile & ((1 << page_shift) - 1);
        const int in_page1 = (tile * kTile + 16) & ((1 << page_shift) - 1);
        // the row of the tile's first token; of its 16th from there, less 16: both
        // halves then go by the token's number in the tile
        const int64_t r0 = static_cast<int64_t>(static_cast<uint64_t>(static_cast<unsigned>(p0)) * page_rows) + in_page;
        const int64_t r1 =
            static_cast<int64_t>(static_cast<uint64_t>(static_cast<unsigned>(p1)) * page_rows) + (in_page1 - 16);
        constexpr int N = kTile * C::CPR, HALF = N / 2, STEP = TH / C::CPR;  // STEP tokens a round
        uint8_t *tail = st + kTile * (C::KS + C::VS);
        if (left >= kTile && (p0 | p1) >= 0) {
            const uint8_t *k0 = k + r0 * C::RB, *k1 = k + r1 * C::RB, *v0 = v + r0 * C::RB, *v1 = v + r1 * C::RB;
#pragma unroll
            for (int i = 0; i < (N + TH - 1) / TH; ++i) {
                if (N % TH != 0 && gt >= N) break;
                const bool second = HALF % TH == 0 ? i * TH >= HALF : gt >= HALF;
                copy16(ka + i * STEP * C::KS, (second ? k1 : k0) + i * TH * 16, true);
                copy16(va + i * STEP * C::VS, (second ? v1 : v0) + i * TH * 16, true);
            }
            if (gt < 32) {
                if constexpr (C::BITS != 16) {
                    const int64_t r = gt >= 16 ? r1 : r0;
                    copy4(smem_addr(tail) + 4 * gt, ks + r, true);
                    copy4(smem_addr(tail) + 4 * (kTile + gt), vs + r, true);
                }
                if (gt == 0) *reinterpret_cast<unsigned *>(tail + C::SCALES) = 0xffffffffu;
            }
        } else {  // the last tile, or one with a bad page: zeros where there is nothing
#pragma unroll
            for (int i = 0; i < (N + TH - 1) / TH; ++i) {
                if (N % TH != 0 && gt >= N) break;
                const bool second = HALF % TH == 0 ? i * TH >= HALF : gt >= HALF;
                const bool ok = (second ? p1 : p0) >= 0 && t + i * STEP < left;
                const int64_t off = ok ? (second ? r1 : r0) * C::RB + i * TH * 16 : 0;
                copy16(ka + i * STEP * C::KS, k + off, ok);
                copy16(va + i * STEP * C::VS, v + off, ok);
            }
            if (gt < 32) {
                const bool ok = (gt >= 16 ? p1 : p0) >= 0 && gt < left;
                if constexpr (C::BITS != 16) {
                    const int64_t r = ok ? (gt >= 16 ? r1 : r0) : 0;
                    copy4(smem_addr(tail) + 4 * gt, ks + r, ok);
                    copy4(smem_addr(tail) + 4 * (kTile + gt), vs + r, ok);
                }
                const unsigned live = __ballot_sync(0xffffffffu, ok);
                if (gt == 0) *reinterpret_cast<unsigned *>(tail + C::SCALES) = live;
            }
        }
    }
};

template <class C>
__device__ __forceinline__ Tiles<C> tiles_of(const Params &p, const Seq &sq, int b, int h, int end, uint8_t *ring,
                                             int gt, bool report) {
    Tiles<C> t;
    const int64_t head = static_cast<int64_t>(h) << p.page_shift;
    t.k = p.k + head * C::RB + gt * 16, t.v = p.v + head * C::RB + gt * 16;
    t.ks = p.ks + head + gt % 32, t.vs = p.vs + head + gt % 32;
    t.table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
    t.ring = ring;
    t.page_rows = static_cast<unsigned>(p.heads) << p.page_shift;
    t.page_shift = p.page_shift, t.pages = p.pages;
    t.end = end, t.total = sq.total, t.gt = gt, t.report = report;
    return t;
}

// Four channels from d on of row r of a block (row g of its sequence): the
// warp groups' results, `step` rows apart in shared memory, joined and written.
template <class C>
__device__ __forceinline__ void finish_row(const Params &p, const Seq &sq, const uint8_t *smem, int split, int h,
                                           int g, int r, int step, int groups, int d) {
    const float *mo = reinterpret_cast<const float *>(smem);
    const float2 *ml = reinterpret_cast<const float2 *>(smem + groups * step * C::OP * 4);
    float M = -INFINITY;
    for (int k = 0; k < groups; ++k) M = fmaxf(M, ml[k * step + r].x);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = 0; k < groups; ++k) {
        const float2 a = ml[k * step + r];
        const float f = exp2_fast(a.x - base);
        const float4 v = *reinterpret_cast<const float4 *>(mo + (k * step + r) * C::OP + d);
        L = fmaf(f, a.y, L);
        acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
    }
    const int head = h * p.group + g % p.group, token = sq.first + g / p.group;
    const int64_t row = static_cast<int64_t>(token) * p.q_heads + head;
    if (p.splits == 1) {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        *reinterpret_cast<uint2 *>(p.out + static_cast<int64_t>(token) * p.out_stride + head * C::D + d) =
            make_uint2(half2_of(acc.x * inv, acc.y * inv), half2_of(acc.z * inv, acc.w * inv));
        if (d == 0 && p.lse != nullptr)
            p.lse[row] = L == 0.0f ? -INFINITY : (M - kShift + log2f(L)) * 0.693147180559945f;
    } else {
        const int64_t at = static_cast<int64_t>(split) * p.tokens * p.q_heads + row;
        *reinterpret_cast<float4 *>(p.part_o + at * C::D + d) = acc;
        if (d == 0) p.part_ml[at] = make_float2(M, L);
    }
}

template <class C>
__global__ void __launch_bounds__(C::NW * 32) tree_attention_kernel(const Params p) {
    constexpr int BITS = C::BITS, D = C::D, WR = C::WR, TG = C::TG;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int tg = warp / WR, wr = warp % WR;
    const int split = blockIdx.x % p.splits, rb = blockIdx.x / p.splits;
    const int h = blockIdx.y, b = blockIdx.z;
    const Seq sq = sequence(p, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
    const int rows = sq.n * p.group;
    if (rb * C::ROWS >= rows) return;

    // this split's tiles
    const int tiles = (sq.total + kTile - 1) / kTile;
    const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / p.splits);
    const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / p.splits);

    // ---- the query rows of this lane, as the products' first operand
    const int q4 = lane & 3, q8 = lane >> 2;
    int tok[2];  // new token of rows q8 and q8 + 8 of this warp, -1: no such row
    uint32_t qf[C::STEPS][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = rb * C::ROWS + wr * 16 + q8 + 8 * e;
        tok[e] = r < rows ? r / p.group : -1;
        const uint16_t *src = p.q;
        if (tok[e] >= 0)
            src += static_cast<int64_t>(sq.first + tok[e]) * p.q_stride +
                   static_cast<int64_t>(h * p.group + r % p.group) * D;
        if constexpr (BITS == 16) {
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    qf[s][e + 2 * x] =
                        tok[e] >= 0 ? *reinterpret_cast<const uint32_t *>(src + 16 * s + 8 * x + 2 * q4) : 0u;
        } else {
            // a lane's K operand is D / 4 consecutive channels; the order in
            // which its words give them up is the order of q here
            uint32_t w[D / 8];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (tok[e] >= 0) u = *reinterpret_cast<const uint4 *>(src + q4 * (D / 4) + 8 * i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) {
                if constexpr (BITS == 8) {
                    qf[s][e] = w[2 * s], qf[s][e + 2] = w[2 * s + 1];
                } else {
                    // eight codes of a word: pairs (0, 4), (1, 5), then (2, 6), (3, 7)
                    const uint32_t lo = w[4 * (s / 2) + s % 2], hi = w[4 * (s / 2) + 2 + s % 2];
                    qf[s][e] = pick(lo, hi, 0x5410u), qf[s][e + 2] = pick(lo, hi, 0x7632u);
                }
            }
        }
    }

    const Tiles<C> src = tiles_of<C>(p, sq, b, h, t1, smem + tg * C::STAGES * C::STAGE, wr * 32 + lane,
                                     wr == 0 && rb == 0);
    uint8_t *ring = src.ring;
    float o[C::NT][4];
#pragma unroll
    for (int i = 0; i < C::NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float unit[2] = {kFirstUnit, kFirstUnit};  // of o's rows, 2^-R (quantised values)

    int next = t0 + tg;  // tile to be issued next, and its pages
    int id = src.page_of(next);
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
        if (next < t1) src.issue(next, s, id);
        copy_commit();
        next += TG;
        id = src.page_of(next);
    }

    int stage = 0;
    for (int t = t0 + tg; t < t1; t += TG) {
        copy_wait<C::STAGES - 2>();
        group_sync(1 + tg, 32 * WR);
        {
            int free_stage = stage + C::STAGES - 1;
            if (free_stage >= C::STAGES) free_stage -= C::STAGES;
            if (next < t1) src.issue(next, free_stage, id);
            copy_commit();
            next += TG;
            id = src.page_of(next);
        }
        const uint8_t *st = ring + stage * C::STAGE;
        const uint32_t ka = smem_addr(st), va = ka + kTile * C::KS;
        const uint8_t *tail = st + kTile * (C::KS + C::VS);
        if (++stage == C::STAGES) stage = 0;

        // ---- S = Q K^T: column 8 n + 2 q4 + e is token 8 n + 2 q4 + e of the tile
        float s[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n][j] = 0.0f;
            if constexpr (BITS == 16) {
#pragma unroll
                for (int k = 0; k < C::STEPS / 2; ++k) {
                    uint32_t f[4];
                    load_matrix4(f, ka + (8 * n + (lane & 7)) * C::KS + (4 * k + (lane >> 3)) * 16);
                    mma(s[n], qf[2 * k], f[0], f[1]);
                    mma(s[n], qf[2 * k + 1], f[2], f[3]);
                }
            } else {
                constexpr int LB = C::RB / 4, UB = LB < 16 ? LB : 16;
                const uint32_t at = ka + (8 * n + q8) * C::KS + q4 * LB;
#pragma unroll
                for (int u = 0; u < LB / UB; ++u) {
                    uint32_t w[UB / 4];
                    load_words<UB>(w, at + u * UB);
#pragma unroll
                    for (int i = 0; i < UB / 4; ++i) {
                        if constexpr (BITS == 8) {
                            const uint32_t x = w[i] ^ 0x80808080u;
                            mma(s[n], qf[u * (UB / 4) + i], pair8(x, false), pair8(x, true));
                        } else {
                            const uint32_t x = w[i], y = x >> 8;
                            const int k = 2 * (u * (UB / 4) + i);
                            mma(s[n], qf[k], pair4(x, false), pair4(x, true));
                            mma(s[n], qf[k + 1], pair4(y, false), pair4(y, true));
                        }
                    }
                }
            }
        }
        // ---- scores in log2 units, unseen ones -infinity
        float vsc[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float2 ksc = make_float2(1.0f, 1.0f);
            if constexpr (BITS != 16) {
                ksc = *reinterpret_cast<const float2 *>(tail + 4 * (8 * n + 2 * q4));
                const float2 v2 = *reinterpret_cast<const float2 *>(tail + 4 * (kTile + 8 * n + 2 * q4));
                vsc[n][0] = v2.x, vsc[n][1] = v2.y;
            }
            const float a = ksc.x * p.scale_log2, c = ksc.y * p.scale_log2;
            s[n][0] *= a, s[n][1] *= c, s[n][2] *= a, s[n][3] *= c;
        }
        const unsigned live = *reinterpret_cast<const unsigned *>(tail + C::SCALES);
        const int j0 = t * kTile - sq.ctx;  // new token at the tile's first position
        unsigned see[2] = {live, live};
        const bool masked = live != 0xffffffffu || j0 + kTile > 0;
        if (masked) {
            see[0] &= seen(p, sq.first, tok[0], j0);
            see[1] &= seen(p, sq.first, tok[1], j0);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!((see[j >> 1] >> (8 * n + 2 * q4 + (j & 1))) & 1u)) s[n][j] = -INFINITY;
        }
        // ---- running maximum
        float alpha[2], base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = m[e];
#pragma unroll
            for (int n = 0; n < 4; ++n) x = fmaxf(x, fmaxf(s[n][2 * e], s[n][2 * e + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            base[e] = x == -INFINITY ? 0.0f : x;
            alpha[e] = exp2_fast(m[e] - base[e]);
            m[e] = x;
            l[e] *= alpha[e];
            base[e] -= kShift;
        }
        // ---- the rows' units of the values' scales
        if constexpr (BITS != 16) {
            // only a scale above a unit (or one that is not finite) has a closer look
            float big = 0.0f;
#pragma unroll
            for (int n = 0; n < 4; ++n) big = fmaxf(fmaxf(big, fabsf(vsc[n][0])), fabsf(vsc[n][1]));
            if (__any_sync(0xffffffffu, big * fmaxf(unit[0], unit[1]) > 1.0f)) {
                unsigned top[2] = {0, 0};  // largest finite magnitudes that the rows see, by their bits
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const unsigned u = finite_bits(vsc[n][j]), bit = 8 * n + 2 * q4 + j;
                        top[0] = max(top[0], (see[0] >> bit) & 1u ? u : 0u);
                        if (masked) top[1] = max(top[1], (see[1] >> bit) & 1u ? u : 0u);
                    }
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[e] = max(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                        top[e] = max(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                    }
                } else {  // (all rows see all of it)
                    top[0] = top[1] = __reduce_max_sync(0xffffffffu, top[0]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float u = unit_of(top_exponent(top[e]));
                    if (u < unit[e]) {
                        alpha[e] *= u * inverse_unit(unit[e]);
                        unit[e] = u;
                    }
                }
            }
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
            for (int i = 0; i < C::NT; ++i) {
                o[i][0] *= alpha[0], o[i][1] *= alpha[0];
                o[i][2] *= alpha[1], o[i][3] *= alpha[1];
            }
        }
        // ---- p
        uint32_t pf[2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = exp2_fast(s[n][j] - base[j >> 1]);
                l[j >> 1] += x[j];
            }
            if constexpr (BITS != 16) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    ptx::f2_split(ptx::f2_mul(ptx::f2(x[2 * e], x[2 * e + 1]),
                                              ptx::f2_mul(ptx::f2(vsc[n][0], vsc[n][1]), ptx::f2(unit[e], unit[e]))),
                                  x[2 * e], x[2 * e + 1]);
                if (masked) {  // an unseen token's scale may be anything
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (!((see[j >> 1] >> (8 * n + 2 * q4 + (j & 1))) & 1u)) x[j] = 0.0f;
                }
            }
            pf[n / 2][2 * (n % 2)] = half2_of(x[0], x[1]);
            pf[n / 2][2 * (n % 2) + 1] = half2_of(x[2], x[3]);
        }
        // ---- O += P V
        if constexpr (BITS == 16) {
            // stored infinities and NaN in a tile that some row does not see
            // whole: 0 * infinity would reach that row through the product
            unsigned odd = 0;
            if (masked) {
                bool any = false;
#pragma unroll
                for (int c = 0; c < C::CPR; ++c) {
                    uint32_t w[4];
                    load_words<16>(w, va + lane * C::VS + 16 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        any |= (w[i] & 0x7c00u) == 0x7c00u || (w[i] & 0x7c000000u) == 0x7c000000u;
                }
                odd = __ballot_sync(0xffffffffu, any);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const unsigned o2 = odd >> (16 * k + 2 * q4);
                const uint32_t keep0 = ~((o2 & 1u ? 0xffffu : 0u) | (o2 & 2u ? 0xffff0000u : 0u));
                const uint32_t keep1 = ~((o2 & 256u ? 0xffffu : 0u) | (o2 & 512u ? 0xffff0000u : 0u));
#pragma unroll
                for (int i = 0; i < C::NT; i += 2) {
                    uint32_t f[4];
                    load_matrix4_t(f, va + (16 * k + (lane & 15)) * C::VS + (i + (lane >> 4)) * 16);
                    if (odd != 0) f[0] &= keep0, f[1] &= keep1, f[2] &= keep0, f[3] &= keep1;
                    mma(o[i], pf[k], f[0], f[1]);
                    mma(o[i + 1], pf[k], f[2], f[3]);
                }
            }
            // the tokens left out above, one by one, for the rows that see them
            while (odd != 0) {
                const int x = __ffs(odd) - 1;
                odd &= odd - 1;
                float pr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mine = 0.0f;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (8 * n + 2 * q4 + j == x) {
                                const uint32_t w = pf[n / 2][2 * (n % 2) + e];
                                const __half2 h2 = *reinterpret_cast<const __half2 *>(&w);
                                mine = j ? __high2float(h2) : __low2float(h2);
                            }
                    pr[e] = __shfl_sync(0xffffffffu, mine, (lane & ~3) | ((x % 8) / 2));
                }
#pragma unroll
                for (int i = 0; i < C::NT; ++i) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(
                        st + kTile * C::KS + x * C::VS + (8 * i + 2 * q4) * 2);
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                    if ((see[0] >> x) & 1u) o[i][0] = fmaf(pr[0], v.x, o[i][0]), o[i][1] = fmaf(pr[0], v.y, o[i][1]);
                    if ((see[1] >> x) & 1u) o[i][2] = fmaf(pr[1], v.x, o[i][2]), o[i][3] = fmaf(pr[1], v.y, o[i][3]);
                }
            }
        } else {
            // a lane's V operand is D / 8 consecutive channels of four tokens
            // (column i of output tile c is channel c D / 8 + i)
            constexpr int LB = C::RB / 8;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t w[4][LB / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    load_words<LB>(w[x], va + (16 * k + 2 * q4 + (x & 1) + 8 * (x >> 1)) * C::VS + q8 * LB);
#pragma unroll
                for (int i = 0; i < LB / 4; ++i) {
                    if constexpr (BITS == 8) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t sel = y ? 0x7362u : 0x5140u;
                            const uint32_t a = pick(w[0][i], w[1][i], sel) ^ 0x80808080u;
                            const uint32_t c = pick(w[2][i], w[3][i], sel) ^ 0x80808080u;
                            mma(o[4 * i + 2 * y], pf[k], pair8(a, false), pair8(c, false));
                            mma(o[4 * i + 2 * y + 1], pf[k], pair8(a, true), pair8(c, true));
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t sel = y ? 0x7632u : 0x5410u;
                            const uint32_t a = pick(w[0][i], w[1][i], sel), a2 = a >> 8;
                            const uint32_t c = pick(w[2][i], w[3][i], sel), c2 = c >> 8;
                            mma(o[8 * i + 4 * y], pf[k], pair4(a, false), pair4(c, false));
                            mma(o[8 * i + 4 * y + 1], pf[k], pair4(a, true), pair4(c, true));
                            mma(o[8 * i + 4 * y + 2], pf[k], pair4(a2, false), pair4(c2, false));
                            mma(o[8 * i + 4 * y + 3], pf[k], pair4(a2, true), pair4(c2, true));
                        }
                    }
                }
            }
        }
    }

    // ---- join the warp groups' results in shared memory (the ring is done with)
    copy_wait<0>();
    __syncthreads();
    float *mo = reinterpret_cast<float *>(smem) + warp * 16 * C::OP;
    float2 *ml = reinterpret_cast<float2 *>(smem + C::NW * 16 * C::OP * 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float up = BITS == 16 ? 1.0f : inverse_unit(unit[e]);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        if (q4 == 0) ml[warp * 16 + q8 + 8 * e] = make_float2(m[e], l[e]);
#pragma unroll
        for (int i = 0; i < C::NT; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int d = BITS == 16 ? 8 * i + 2 * q4 + j : (2 * q4 + j) * (D / 8) + i;
                mo[(q8 + 8 * e) * C::OP + d] = o[i][2 * e + j] * up;
            }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < C::ROWS * (D / 4); x += C::NW * 32) {
        const int r = x / (D / 4), d = x % (D / 4) * 4;
        const int g = rb * C::ROWS + r;
        if (g >= rows) break;
        finish_row<C>(p, sq, smem, split, h, g, r, C::ROWS, TG, d);
    }
}

// ------------------------------------------------------------------ up to 8 rows
// The transposed products, S^T = K Q^T and O^T = V^T P^T: with the cached
// tokens (then the channels) as the 16 rows of an m16n8k16 product and the
// query rows as its 8 columns, a decoding step's few rows cost half the
// products, accumulators and exponentials.  P^T turns from the accumulators'
// layout into the second product's operand by movmatrix.
//
// A token over 200 of INT8, 32 heads: 6.4 to 6.6 us; one of 16 sequences over up to 2048
// of INT4, 32 heads: 37 us with the join (16.9 by the bytes; the conversion of codes
// keeps the ALU half busy at 16 warps an SM); one over 65536, 64 / 8 heads: fp16 54 us
// (40.9 by the bytes), INT8 39 (21.1), INT4 32 (10.9).
//
// Short contexts: see FewMode.  Otherwise the work, tiles of all sequences, key heads
// and blocks of 8 rows one after the other, is cut into equal runs, one a warp, whatever the sequences'
// lengths: no warp waits for another, and all end together.  A run crosses
// from one item (sequence, key head, row block) to the next without emptying
// its ring.  What a warp finds for an item is a piece; a second kernel joins an
// item's pieces.  Piece number = worker + item: along the runs one or the other
// goes up at every step, so no two pieces share a number.  (CTAs of four warps
// on 1 / 2 of an item each, joined in shared memory: 44.5 us for 16 sequences
// over INT4, of which 28 us remained without any arithmetic.)
template <int BITS_, int D_>
struct FewCfg {
    static constexpr int BITS = BITS_, D = D_, WR = 1;
    static constexpr int RB = D * BITS / 8, CPR = RB / 16;
    static constexpr int KS = RB >= 128 ? RB + 16 : RB, VS = RB + 16;
    static constexpr int SCALES = BITS == 16 ? 0 : 2 * kTile * 4;
    static constexpr int STAGE = kTile * (KS + VS) + SCALES + 32;
    // warps of a CTA and stages of each: what fills an SM's shared memory with
    // warps (one warp takes microseconds for a tile: their number counts)
    static constexpr int NW = STAGE > 6000 ? 6 : 4;
    static constexpr int STAGES = STAGE > 4000 ? 2 : 3;
    static constexpr int SMEM = NW * STAGES * STAGE;
    static constexpr int STEPS = D / 16, MT = D / 16;
    // resident CTAs of an SM: by 228 KB of shared memory and 65536 registers
    static constexpr int BY_SMEM = 233472 / (SMEM + 1024);
    static constexpr int CTAS = BY_SMEM < 4 ? BY_SMEM : 4;
    static constexpr int WORKERS = CTAS * NW;  // of an SM
};

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// Tiles of an item of sequence b, and its items.
struct Load {
    int tiles, items;
};
__device__ __forceinline__ Load load_of(const Params &p, const Seq &s) {
    Load l;
    l.tiles = (s.total + kTile - 1) / kTile;
    l.items = s.n == 0 ? 0 : p.heads * ((s.n * p.group + 7) / 8);
    return l;
}

// A place in the work: an item of sequence b and a tile of it.
struct Cursor {
    int b, item, tile, tiles, items;
    Seq sq;
};
// The next sequence that has any work, from b on.
__device__ __forceinline__ void enter(const Params &p, Cursor &c, int b) {
    for (; b < p.sequences; ++b) {
        c.sq = sequence(p, b, false);
        const Load l = load_of(p, c.sq);
        c.b = b, c.tiles = l.tiles, c.items = l.items;
        if (l.tiles > 0 && l.items > 0) return;
    }
}

// Who takes an item.  Short contexts are not streamed: a second kernel would take
// as long as the first.  Then a warp has an item to itself, or the CTA's warps
// share one and join what they found in shared memory; both write its rows.
enum FewMode { kStream, kWarp, kGroup };

template <class C, int MODE>
__global__ void __launch_bounds__(C::NW * 32, C::CTAS) tree_attention_few_kernel(const Params p) {
    constexpr int BITS = C::BITS, D = C::D;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int worker = blockIdx.x * C::NW + warp;

    int left;  // tiles still to be issued
    Cursor at;
    at.item = 0, at.tile = 0;
    if constexpr (MODE != kStream) {
        const int per = p.heads * p.row_blocks, index = MODE == kWarp ? worker : blockIdx.x;
        at.b = index / per;
        if (at.b >= p.sequences) return;
        at.item = index % per;
        at.sq = sequence(p, at.b, at.item == 0 && lane == 0 && (MODE == kWarp || warp == 0));
        const Load l = load_of(p, at.sq);
        if (at.item >= l.items) return;
        at.tiles = l.tiles, at.items = l.items;
        left = l.tiles;
        if constexpr (MODE == kGroup) {
            at.tile = static_cast<int>(static_cast<int64_t>(l.tiles) * warp / C::NW);
            left = static_cast<int>(static_cast<int64_t>(l.tiles) * (warp + 1) / C::NW) - at.tile;
        }
    } else {
        // ---- this worker's run: the tiles of all sequences, 32 sequences at a time
        // (the first 32 are looked at once: the usual number, and this is latency)
        const bool report = blockIdx.x == 0 && warp == 0;
        Seq mine{};
        if (lane < p.sequences) mine = sequence(p, lane, report);
        const Load mine_load = load_of(p, mine);
        const int64_t mine_tiles = static_cast<int64_t>(mine_load.tiles) * mine_load.items;
        int64_t all = mine_tiles;
        for (int b = 32 + lane; b < p.sequences; b += 32) {
            const Load l = load_of(p, sequence(p, b, report));
            all += static_cast<int64_t>(l.tiles) * l.items;
        }
#pragma unroll
        for (int x = 1; x < 32; x *= 2) all += __shfl_xor_sync(0xffffffffu, all, x);
        // no more workers than tiles: every worker between an item's first and last has a piece of it
        const int64_t workers = all < p.workers ? all : p.workers;
        if (worker >= workers) return;
        const int64_t from = all * worker / workers;
        left = static_cast<int>(all * (worker + 1) / workers - from);
        {
            int64_t before = 0;
            for (int b0 = 0; b0 < p.sequences; b0 += 32) {
                int64_t own = mine_tiles;
                if (b0 > 0) {
                    const Load l = load_of(p, b0 + lane < p.sequences ? sequence(p, b0 + lane, false) : Seq{});
                    own = static_cast<int64_t>(l.tiles) * l.items;
                }
                int64_t to = own;  // tiles up to and with this lane's sequence
#pragma unroll
                for (int x = 1; x < 32; x *= 2) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, to, x);
                    if (lane >= x) to += y;
                }
                to += before;
                const unsigned past = __ballot_sync(0xffffffffu, to > from);
                if (past != 0) {
                    const int src = __ffs(past) - 1;
                    const int64_t ahead = from - __shfl_sync(0xffffffffu, to - own, src);
                    if (b0 == 0) {
                        at.b = src;
                        at.sq.first = __shfl_sync(0xffffffffu, mine.first, src);
                        at.sq.n = __shfl_sync(0xffffffffu, mine.n, src);
                        at.sq.ctx = __shfl_sync(0xffffffffu, mine.ctx, src);
                        at.sq.total = __shfl_sync(0xffffffffu, mine.total, src);
                        const Load l = load_of(p, at.sq);
                        at.tiles = l.tiles, at.items = l.items;
                    } else {
                        enter(p, at, b0 + src);
                    }
                    at.item = static_cast<int>(ahead / at.tiles);
                    at.tile = static_cast<int>(ahead % at.tiles);
                    break;
                }
                before = __shfl_sync(0xffffffffu, to, 31);
            }
        }
    }
    int todo = left;
    const int first_b = at.b, first_item = at.item;

    uint8_t *ring = smem + warp * C::STAGES * C::STAGE;
    // of the place to be issued next: its rows, its page number
    Tiles<C> src;
    int id;
    auto locate = [&]() {
        const int blocks = at.items / p.heads;
        src = tiles_of<C>(p, at.sq, at.b, at.item / blocks, at.tiles, ring, lane, at.item % blocks == 0);
    };
    locate();
    id = src.page_of(at.tile);
    const int first_items = at.items, first_n = at.sq.n;
    // copies of the next tile, what the products need to know of it, and one step on
    bool start = true;
    auto issue = [&](int stage) {
        if (left == 0) return;
        src.issue(at.tile, stage, id);
        const bool last = left == 1 || at.tile + 1 == at.tiles;
        if (lane == 0) {
            // beside `live`: first new token of the tile, item, sequence, and whether
            // the tile is the first or last of a piece, the first or last of its item
            uint8_t *tail = ring + stage * C::STAGE + kTile * (C::KS + C::VS) + C::SCALES;
            *reinterpret_cast<int4 *>(tail + 16) =
                make_int4(at.tile * kTile - at.sq.ctx, at.item, at.b,
                          (start ? 1 : 0) | (last ? 2 : 0) | (at.tile == 0 ? 4 : 0) |
                              (at.tile + 1 == at.tiles ? 8 : 0));
        }
        start = last;
        if (--left == 0) return;
        if (++at.tile == at.tiles) {
            at.tile = 0;
            if (++at.item == at.items) {
                at.item = 0;
                enter(p, at, at.b + 1);
            }
            locate();
        }
        id = src.page_of(at.tile);
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
        issue(s);
        copy_commit();
    }

    const int q4 = lane & 3, q8 = lane >> 2;
    uint32_t qf[C::STEPS][2];  // the query rows as the products' second operand
    int tok[2], first = 0;     // new token of rows 2 q4, 2 q4 + 1; the sequence's first row
    float o[C::MT][4], m[2], l[2];
    // Of p as it enters the product (with the values' scale): what its rounding added,
    // and its sum before that, one half a row.  Kept for short contexts, where a row
    // may see a token or two (20 of a tile's 750 instructions).
    constexpr bool MEND = MODE != kStream;
    uint64_t added = 0, exact = 0;
    float unit[2];  // of O's rows, 2^-R (quantised values)

    // A new item: this lane's query row is q8, and of it the channels that the
    // lanes' K words give up together.
    auto open = [&](int b, int item) {
        first = p.cu[b];
        const int rows = (p.cu[b + 1] - first) * p.group, blocks = (rows + 7) / 8;
        const int h = item / blocks, r0 = item % blocks * 8;
        const int r = r0 + q8;
        const bool ok = r < rows;
        const uint16_t *row = p.q;
        if (ok)
            row += static_cast<int64_t>(first + r / p.group) * p.q_stride +
                   static_cast<int64_t>(h * p.group + r % p.group) * D;
        if constexpr (BITS == 16) {
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    qf[s][x] = ok ? *reinterpret_cast<const uint32_t *>(row + 16 * s + 8 * x + 2 * q4) : 0u;
        } else {
            uint32_t w[D / 8];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (ok) u = *reinterpret_cast<const uint4 *>(row + q4 * (D / 4) + 8 * i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
#pragma unroll
            for (int s = 0; s < C::STEPS; ++s) {
                if constexpr (BITS == 8) {
                    qf[s][0] = w[2 * s], qf[s][1] = w[2 * s + 1];
                } else {
                    // words of eight channels: step 2 i even nibbles (0, 4), (2, 6), step 2 i + 1
                    // odd ones (1, 5), (3, 7)
                    const int i = 4 * (s / 2);
                    const uint32_t sel = s % 2 ? 0x7632u : 0x5410u;
                    qf[s][0] = pick(w[i], w[i + 2], sel), qf[s][1] = pick(w[i + 1], w[i + 3], sel);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int x = r0 + 2 * q4 + e;
            tok[e] = x < rows ? x / p.group : -1;
            m[e] = -INFINITY, l[e] = 0.0f;
        }
        added = exact = 0;
        unit[0] = unit[1] = kFirstUnit;
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    };
    // The factor that takes the roundings' common part out of row e's O: a token that
    // has most of the weight would else give its own rounding to the whole row (three
    // tokens: 1.6 times the error of the output's rounding alone).  Weights of one
    // sign have theirs within 2^-11; anything else is left as it is.
    auto mend = [&](int e, float sum) {
        float d, w, other;
        if (e == 0)
            ptx::f2_split(added, d, other), ptx::f2_split(exact, w, other);
        else
            ptx::f2_split(added, other, d), ptx::f2_split(exact, other, w);
#pragma unroll
        for (int y = 4; y < 32; y *= 2) {
            d += __shfl_xor_sync(0xffffffffu, d, y);
            if constexpr (BITS != 16) w += __shfl_xor_sync(0xffffffffu, w, y);
        }
        if constexpr (BITS == 16) w = sum;
        return w > 0.0f && fabsf(d) <= w * 0x1p-10f ? w / (w + d) : 1.0f;
    };
    // (of the first item while its first tile is on the way)
    open(first_b, first_item);
    bool opened = true;

    int stage = 0;
    for (; todo > 0; --todo) {
        copy_wait<C::STAGES - 2>();
        __syncwarp();
        issue(stage + C::STAGES - 1 >= C::STAGES ? stage - 1 : stage + C::STAGES - 1);
        copy_commit();
        const uint8_t *st = ring + stage * C::STAGE;
        const uint32_t ka = smem_addr(st), va = ka + kTile * C::KS;
        const uint8_t *tail = st + kTile * (C::KS + C::VS);
        if (++stage == C::STAGES) stage = 0;
        const unsigned live = *reinterpret_cast<const unsigned *>(tail + C::SCALES);
        const int4 place = *reinterpret_cast<const int4 *>(tail + C::SCALES + 16);
        const int j0 = place.x;
        if ((place.w & 1) && !opened) open(place.z, place.y);
        opened = false;

        // ---- S^T: s[i][2 f + e] is token 16 i + 8 f + q8, row 2 q4 + e
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
            if constexpr (BITS == 16) {
#pragma unroll
                for (int k = 0; k < C::STEPS; ++k) {
                    uint32_t f[4];
                    load_matrix4(f, ka + (16 * i + (lane & 15)) * C::KS + (2 * k + (lane >> 4)) * 16);
                    mma(s[i], f, qf[k][0], qf[k][1]);
                }
            } else {
                constexpr int LB = C::RB / 4, UB = LB < 16 ? LB : 16;
                const uint32_t at = ka + (16 * i + q8) * C::KS + q4 * LB;
#pragma unroll
                for (int u = 0; u < LB / UB; ++u) {
                    uint32_t w[2][UB / 4];
                    load_words<UB>(w[0], at + u * UB);
                    load_words<UB>(w[1], at + 8 * C::KS + u * UB);
#pragma unroll
                    for (int k = 0; k < UB / 4; ++k) {
                        if constexpr (BITS == 8) {
                            const uint32_t x = w[0][k] ^ 0x80808080u, y = w[1][k] ^ 0x80808080u;
                            const uint32_t f[4] = {pair8(x, false), pair8(y, false), pair8(x, true),
                                                   pair8(y, true)};
                            const int step = u * (UB / 4) + k;
                            mma(s[i], f, qf[step][0], qf[step][1]);
                        } else {
                            const uint32_t x = w[0][k], y = w[1][k], x2 = x >> 8, y2 = y >> 8;
                            const uint32_t f[4] = {pair4(x, false), pair4(y, false), pair4(x2, false),
                                                   pair4(y2, false)};
                            const uint32_t g[4] = {pair4(x, true), pair4(y, true), pair4(x2, true),
                                                   pair4(y2, true)};
                            const int step = 2 * (u * (UB / 4) + k);
                            mma(s[i], f, qf[step][0], qf[step][1]);
                            mma(s[i], g, qf[step + 1][0], qf[step + 1][1]);
                        }
                    }
                }
            }
        }
        // ---- scores in log2 units, unseen ones -infinity
        float vsc[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                float ksc = p.scale_log2;
                if constexpr (BITS != 16) {
                    ksc *= *reinterpret_cast<const float *>(tail + 4 * (16 * i + 8 * f + q8));
                    vsc[i][f] = *reinterpret_cast<const float *>(tail + 4 * (kTile + 16 * i + 8 * f + q8));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) s[i][2 * f + e] *= ksc;
            }
        unsigned see[2] = {live, live};
        const bool masked = live != 0xffffffffu || j0 + kTile > 0;
        if (masked) {
            see[0] &= seen(p, first, tok[0], j0);
            see[1] &= seen(p, first, tok[1], j0);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!((see[j & 1] >> (16 * i + 8 * (j >> 1) + q8)) & 1u)) s[i][j] = -INFINITY;
        }
        // ---- running maximum
        float alpha[2], base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = fmaxf(fmaxf(s[0][e], s[0][2 + e]), fmaxf(s[1][e], s[1][2 + e]));
#pragma unroll
            for (int y = 4; y < 32; y *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, y));
            x = fmaxf(x, m[e]);
            base[e] = x == -INFINITY ? 0.0f : x;
            alpha[e] = exp2_fast(m[e] - base[e]);
            m[e] = x;
            l[e] *= alpha[e];
            base[e] -= kShift;
        }
        // ---- the rows' units of the values' scales
        if constexpr (BITS != 16) {
            // only a scale above a unit (or one that is not finite) has a closer look
            const float big = fmaxf(fmaxf(fabsf(vsc[0][0]), fabsf(vsc[0][1])),
                                    fmaxf(fabsf(vsc[1][0]), fabsf(vsc[1][1])));
            if (__any_sync(0xffffffffu, big * fmaxf(unit[0], unit[1]) > 1.0f)) {
                unsigned top[2] = {0, 0};  // largest finite magnitudes that the rows see, by their bits
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const unsigned u = finite_bits(vsc[i][f]), bit = 16 * i + 8 * f + q8;
                        top[0] = max(top[0], (see[0] >> bit) & 1u ? u : 0u);
                        if (masked) top[1] = max(top[1], (see[1] >> bit) & 1u ? u : 0u);
                    }
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int y = 4; y < 32; y *= 2) top[e] = max(top[e], __shfl_xor_sync(0xffffffffu, top[e], y));
                } else {  // (all rows see all of it)
                    top[0] = top[1] = __reduce_max_sync(0xffffffffu, top[0]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float u = unit_of(top_exponent(top[e]));
                    if (u < unit[e]) {
                        alpha[e] *= u * inverse_unit(unit[e]);
                        unit[e] = u;
                    }
                }
            }
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
            for (int i = 0; i < C::MT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= alpha[j & 1];
        }
        if constexpr (MEND) added = ptx::f2_mul(added, ptx::f2(alpha[0], alpha[1]));
        if constexpr (MEND && BITS != 16) exact = ptx::f2_mul(exact, ptx::f2(alpha[0], alpha[1]));
        // ---- p, transposed into the second operand
        uint32_t pf[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                float x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = exp2_fast(s[i][2 * f + e] - base[e]);
                    l[e] += x[e];
                }
                if constexpr (BITS != 16) {
                    ptx::f2_split(ptx::f2_mul(ptx::f2(x[0], x[1]), ptx::f2_mul(ptx::f2(vsc[i][f], vsc[i][f]),
                                                                               ptx::f2(unit[0], unit[1]))),
                                  x[0], x[1]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)  // an unseen token's scale may be anything
                        if (masked && !((see[e] >> (16 * i + 8 * f + q8)) & 1u)) x[e] = 0.0f;
                }
                const __half2 h2 = __floats2half2_rn(x[0], x[1]);
                if constexpr (MEND) {
                    const float2 r = __half22float2(h2);
                    const uint64_t x2 = ptx::f2(x[0], x[1]);
                    added = ptx::f2_add(added, ptx::f2_sub(ptx::f2(r.x, r.y), x2));
                    if constexpr (BITS != 16) exact = ptx::f2_add(exact, x2);
                }
                pf[i][f] = transpose8(*reinterpret_cast<const uint32_t *>(&h2));
            }
        // ---- O^T += V^T P^T
        if constexpr (BITS == 16) {
            // stored infinities and NaN in a tile that some row does not see
            // whole: 0 * infinity would reach that row through the product
            unsigned odd = 0;
            if (masked) {
                bool any = false;
#pragma unroll
                for (int c = 0; c < C::CPR; ++c) {
                    uint32_t w[4];
                    load_words<16>(w, va + lane * C::VS + 16 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        any |= (w[i] & 0x7c00u) == 0x7c00u || (w[i] & 0x7c000000u) == 0x7c000000u;
                }
                odd = __ballot_sync(0xffffffffu, any);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned o2 = odd >> (16 * i + 2 * q4);
                const uint32_t keep0 = ~((o2 & 1u ? 0xffffu : 0u) | (o2 & 2u ? 0xffff0000u : 0u));
                const uint32_t keep1 = ~((o2 & 256u ? 0xffffu : 0u) | (o2 & 512u ? 0xffff0000u : 0u));
#pragma unroll
                for (int c = 0; c < C::MT; ++c) {
                    uint32_t f[4];
                    load_matrix4_t(f, va + (16 * i + (lane & 7) + ((lane >> 4) & 1) * 8) * C::VS +
                                          (2 * c + ((lane >> 3) & 1)) * 16);
                    if (odd != 0) f[0] &= keep0, f[1] &= keep0, f[2] &= keep1, f[3] &= keep1;
                    mma(o[c], f, pf[i][0], pf[i][1]);
                }
            }
            // the tokens left out above, one by one, for the rows that see them
            while (odd != 0) {
                const int x = __ffs(odd) - 1;
                odd &= odd - 1;
                // lane 4 r + (x % 8) / 2 holds row r's p of this token
                float pr[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const uint32_t y = __shfl_sync(0xffffffffu, pf[i][f], 4 * (2 * q4 + e) + (x % 8) / 2);
                            if (x / 8 == 2 * i + f) w = y;
                        }
                    const __half2 h2 = *reinterpret_cast<const __half2 *>(&w);
                    pr[e] = x % 2 ? __high2float(h2) : __low2float(h2);
                }
#pragma unroll
                for (int c = 0; c < C::MT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float v = __half2float(*reinterpret_cast<const __half *>(
                            st + kTile * C::KS + x * C::VS + (16 * c + 8 * (j >> 1) + q8) * 2));
                        if ((see[j & 1] >> x) & 1u) o[c][j] = fmaf(pr[j & 1], v, o[c][j]);
                    }
            }
        } else {
            // a lane's V operand is D / 8 consecutive channels of four tokens:
            // rows q8 and q8 + 8 of tile c are channels 2 c and 2 c + 1 of them
            constexpr int LB = C::RB / 8;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t w[4][LB / 4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    load_words<LB>(w[x], va + (16 * i + 2 * q4 + (x & 1) + 8 * (x >> 1)) * C::VS + q8 * LB);
#pragma unroll
                for (int k = 0; k < LB / 4; ++k) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        if constexpr (BITS == 8) {
                            const uint32_t sel = y ? 0x7362u : 0x5140u;
                            const uint32_t a = pick(w[0][k], w[1][k], sel) ^ 0x80808080u;
                            const uint32_t c = pick(w[2][k], w[3][k], sel) ^ 0x80808080u;
                            const uint32_t f[4] = {pair8(a, false), pair8(a, true), pair8(c, false),
                                                   pair8(c, true)};
                            mma(o[2 * k + y], f, pf[i][0], pf[i][1]);
                        } else {
                            const uint32_t sel = y ? 0x7632u : 0x5410u;
                            const uint32_t a = pick(w[0][k], w[1][k], sel), a2 = a >> 8;
                            const uint32_t c = pick(w[2][k], w[3][k], sel), c2 = c >> 8;
                            const uint32_t f[4] = {pair4(a, false), pair4(a, true), pair4(c, false),
                                                   pair4(c, true)};
                            const uint32_t g[4] = {pair4(a2, false), pair4(a2, true), pair4(c2, false),
                                                   pair4(c2, true)};
                            mma(o[4 * k + 2 * y], f, pf[i][0], pf[i][1]);
                            mma(o[4 * k + 2 * y + 1], g, pf[i][0], pf[i][1]);
                        }
                    }
                }
            }
        }
        if constexpr (MODE != kStream) continue;
        const int64_t item = place.z * (static_cast<int64_t>(p.heads) * p.row_blocks) + place.y;
        if (lane == 0 && (place.w & 4)) p.item_span[2 * item] = worker;
        if (lane == 0 && (place.w & 8)) p.item_span[2 * item + 1] = worker;
        if (place.w & 2) {
            // ---- the piece, as the lanes hold it; rows that do not exist are left out
            const int64_t piece = worker + item;
            const float up0 = BITS == 16 ? 1.0f : inverse_unit(unit[0]);
            const float up1 = BITS == 16 ? 1.0f : inverse_unit(unit[1]);
            float4 *dst = p.piece_o + piece * (C::MT * 32) + lane;
            if (tok[0] >= 0) {
#pragma unroll
                for (int c = 0; c < C::MT; ++c)
                    dst[c * 32] = make_float4(o[c][0] * up0, o[c][1] * up1, o[c][2] * up0, o[c][3] * up1);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[e];
#pragma unroll
                for (int y = 4; y < 32; y *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, y);
                if (q8 == 0) p.piece_ml[piece * 8 + 2 * q4 + e] = make_float2(m[e], sum);
            }
        }
    }
    if constexpr (MODE == kWarp) {
        // ---- the rows, through shared memory into their order (the ring is done with)
        copy_wait<0>();
        __syncwarp();
        static_assert(8 * (D + 4) * 4 + 32 <= C::STAGES * C::STAGE, "the rows fit the warp's ring");
        float *rows = reinterpret_cast<float *>(ring), *lse = rows + 8 * (D + 4);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float up = BITS == 16 ? 1.0f : inverse_unit(unit[e]);
            float sum = l[e];
#pragma unroll
            for (int y = 4; y < 32; y *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, y);
            const float f = (sum == 0.0f ? 0.0f : up / sum) * mend(e, sum);
            if (q8 == 0)
                lse[2 * q4 + e] = sum == 0.0f ? -INFINITY : (m[e] - kShift + log2f(sum)) * 0.693147180559945f;
#pragma unroll
            for (int c = 0; c < C::MT; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    rows[(2 * q4 + e) * (D + 4) + (BITS == 16 ? 16 * c + 8 * x + q8 : q8 * (D / 8) + 2 * c + x)] =
                        o[c][2 * x + e] * f;
        }
        __syncwarp();
        const int blocks = first_items / p.heads, h = first_item / blocks, r0 = first_item % blocks * 8;
        constexpr int PER = 8, LANES = D / PER;  // 16 bytes a lane
#pragma unroll
        for (int x = lane / LANES; x < 8; x += 32 / LANES) {
            const int g = r0 + x;
            if (g >= first_n * p.group) break;
            const int64_t token = first + g / p.group, head = h * p.group + g % p.group;
            const float *src8 = rows + x * (D + 4) + lane % LANES * PER;
            const float4 a = *reinterpret_cast<const float4 *>(src8), c = *reinterpret_cast<const float4 *>(src8 + 4);
            *reinterpret_cast<uint4 *>(p.out + token * p.out_stride + head * D + lane % LANES * PER) =
                make_uint4(half2_of(a.x, a.y), half2_of(a.z, a.w), half2_of(c.x, c.y), half2_of(c.z, c.w));
            if (lane % LANES == 0 && p.lse != nullptr) p.lse[token * p.q_heads + head] = lse[x];
        }
    }
    if constexpr (MODE == kGroup) {
        // ---- every warp's rows, maxima and sums in its ring (which is done with); then
        // a thread joins eight channels of a row
        constexpr int PITCH = D + 4;
        copy_wait<0>();
        __syncwarp();
        float *rows = reinterpret_cast<float *>(ring), *ml = rows + 8 * PITCH;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float up = BITS == 16 ? 1.0f : inverse_unit(unit[e]);
            float sum = l[e];
#pragma unroll
            for (int y = 4; y < 32; y *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, y);
            const float f = up * mend(e, sum);
            if (q8 == 0) ml[2 * (2 * q4 + e)] = m[e], ml[2 * (2 * q4 + e) + 1] = sum;
#pragma unroll
            for (int c = 0; c < C::MT; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    rows[(2 * q4 + e) * PITCH + (BITS == 16 ? 16 * c + 8 * x + q8 : q8 * (D / 8) + 2 * c + x)] =
                        o[c][2 * x + e] * f;
        }
        __syncthreads();
        const int blocks = first_items / p.heads, h = first_item / blocks, r0 = first_item % blocks * 8;
        constexpr int PER = 8, LANES = D / PER;
        static_assert(8 * LANES <= C::NW * 32, "a thread each");
        static_assert(8 * PITCH * 4 + 64 <= C::STAGES * C::STAGE, "they fit the ring");
        const int x = threadIdx.x / LANES, d = threadIdx.x % LANES * PER, g = r0 + x;
        if (x >= 8 || g >= first_n * p.group) return;
        const float *all = reinterpret_cast<const float *>(smem);
        constexpr int STEP = C::STAGES * C::STAGE / 4;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::NW; ++w) M = fmaxf(M, all[w * STEP + 8 * PITCH + 2 * x]);
        const float base = M == -INFINITY ? 0.0f : M;
        float L = 0.0f, acc[PER] = {};
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
            const float *mine = all + w * STEP;
            const float f = exp2_fast(mine[8 * PITCH + 2 * x] - base);
            L = fmaf(f, mine[8 * PITCH + 2 * x + 1], L);
            const float4 a = *reinterpret_cast<const float4 *>(mine + x * PITCH + d);
            const float4 c = *reinterpret_cast<const float4 *>(mine + x * PITCH + d + 4);
            acc[0] = fmaf(f, a.x, acc[0]), acc[1] = fmaf(f, a.y, acc[1]);
            acc[2] = fmaf(f, a.z, acc[2]), acc[3] = fmaf(f, a.w, acc[3]);
            acc[4] = fmaf(f, c.x, acc[4]), acc[5] = fmaf(f, c.y, acc[5]);
            acc[6] = fmaf(f, c.z, acc[6]), acc[7] = fmaf(f, c.w, acc[7]);
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const int64_t token = first + g / p.group, head = h * p.group + g % p.group;
        *reinterpret_cast<uint4 *>(p.out + token * p.out_stride + head * D + d) =
            make_uint4(half2_of(acc[0] * inv, acc[1] * inv), half2_of(acc[2] * inv, acc[3] * inv),
                       half2_of(acc[4] * inv, acc[5] * inv), half2_of(acc[6] * inv, acc[7] * inv));
        if (d == 0 && p.lse != nullptr)
            p.lse[token * p.q_heads + head] = L == 0.0f ? -INFINITY : (M - kShift + log2f(L)) * 0.693147180559945f;
    }
}

// Join an item's pieces: a block of W warps a row, each warp every W-th piece.
// A lane's 16 bytes of a piece hold two channels of this row (and of the row
// beside it); up to 4 W pieces are loaded at once, before their maximum is
// known.
template <class C, int W>
__global__ void __launch_bounds__(32 * W) tree_attention_few_join_kernel(const Params p) {
    constexpr int D = C::D, V = D / 64, AHEAD = 4;
    __shared__ float acc_s[W][D], sum_s[W], max_s[W];
    const int h = blockIdx.y, b = blockIdx.z, g = blockIdx.x;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const Seq sq = sequence(p, b, false);  // (not written by the kernel that is waited for)
    ptx::grid_dependency_wait();
    if (g >= sq.n * p.group) return;
    const Load ld = load_of(p, sq);
    const int r = g % 8, item = h * (ld.items / p.heads) + g / 8;
    const int64_t index = b * (static_cast<int64_t>(p.heads) * p.row_blocks) + item;
    int w0 = 0, count = 0;
    if (ld.tiles > 0) {
        const int2 span = *reinterpret_cast<const int2 *>(p.item_span + 2 * index);
        w0 = span.x;
        count = span.y - span.x + 1;
    }
    const int64_t piece0 = index + w0;
    const float2 *ml = p.piece_ml + piece0 * 8 + r;
    // tile c of the products, channel q8: lanes (c, q8), 4 tiles a load
    const int q8 = lane % 8, c0 = lane / 8;
    const float4 *src = p.piece_o + (piece0 * C::MT + c0) * 32 + q8 * 4 + r / 2;
    float2 a[AHEAD];
    float4 v[AHEAD][V];
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        const int s = warp + W * i;
        const bool ok = s < count;
        a[i] = ok ? ml[s * 8] : make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j)
            v[i][j] = ok ? src[static_cast<int64_t>(s) * (C::MT * 32) + j * 128] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        M = fmaxf(M, a[i].x);
    }
    for (int s = W * AHEAD + threadIdx.x; s < count; s += 32 * W) M = fmaxf(M, ml[s * 8].x);
#pragma unroll
    for (int y = 1; y < 32; y *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, y));
    if (lane == 0) max_s[warp] = M;
    __syncthreads();
#pragma unroll
    for (int y = 0; y < W; ++y) M = fmaxf(M, max_s[y]);
    const float base = M == -INFINITY ? 0.0f : M;
    float acc[V][2] = {}, L = 0.0f;
    auto add = [&](const float2 &m, const float4 (&x)[V]) {
        const float f = exp2_fast(m.x - base);
        L = fmaf(f, m.y, L);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            acc[j][0] = fmaf(f, r % 2 ? x[j].y : x[j].x, acc[j][0]);
            acc[j][1] = fmaf(f, r % 2 ? x[j].w : x[j].z, acc[j][1]);
        }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) add(a[i], v[i]);
#pragma unroll 4
    for (int s = W * AHEAD + warp; s < count; s += W) {
        float4 x[V];
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = src[static_cast<int64_t>(s) * (C::MT * 32) + j * 128];
        add(ml[s * 8], x);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int c = c0 + 4 * j;
            acc_s[warp][C::BITS == 16 ? 16 * c + 8 * x + q8 : q8 * (D / 8) + 2 * c + x] = acc[j][x];
        }
    if (lane == 0) sum_s[warp] = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int y = 0; y < W; ++y) L += sum_s[y];
    const int head = h * p.group + g % p.group, token = sq.first + g / p.group;
    if (threadIdx.x < D / 2) {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        const int e = 2 * threadIdx.x;
        float y0 = 0.0f, y1 = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) y0 += acc_s[i][e], y1 += acc_s[i][e + 1];
        *reinterpret_cast<uint32_t *>(p.out + static_cast<int64_t>(token) * p.out_stride + head * D + e) =
            half2_of(y0 * inv, y1 * inv);
    }
    if (threadIdx.x == 0 && p.lse != nullptr)
        p.lse[static_cast<int64_t>(token) * p.q_heads + head] =
            L == 0.0f ? -INFINITY : (M - kShift + log2f(L)) * 0.693147180559945f;
}

// Join the splits' results: a block of four warps a row, each warp every fourth
// split, eight loads in flight.  (One warp a row, one split after the other:
// 24 us for 64 splits.)
template <int D>
__global__ void __launch_bounds__(128) tree_attention_join_kernel(const Params p) {
    __shared__ float acc_s[4][D];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int h = blockIdx.y, b = blockIdx.z;
    const Seq sq = sequence(p, b, false);  // (not written by the kernel that is waited for)
    ptx::grid_dependency_wait();
    const int g = blockIdx.x;
    if (g >= sq.n * p.group) return;
    const int head = h * p.group + g % p.group, token = sq.first + g / p.group;
    const int64_t row = static_cast<int64_t>(token) * p.q_heads + head;
    const int64_t step = static_cast<int64_t>(p.tokens) * p.q_heads;
    // lanes hold the maxima and sums of up to 64 splits
    const float2 none = make_float2(-INFINITY, 0.0f);
    const float2 a0 = lane < p.splits ? p.part_ml[lane * step + row] : none;
    const float2 a1 = lane + 32 < p.splits ? p.part_ml[(lane + 32) * step + row] : none;
    float M = fmaxf(a0.x, a1.x);
#pragma unroll
    for (int x = 1; x < 32; x *= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    const float base = M == -INFINITY ? 0.0f : M;
    const float f0 = exp2_fast(a0.x - base), f1 = exp2_fast(a1.x - base);
    float L = fmaf(f0, a0.y, f1 * a1.y);
#pragma unroll
    for (int x = 1; x < 32; x *= 2) L += __shfl_xor_sync(0xffffffffu, L, x);
    constexpr int V = D / 32;
    float acc[V] = {};
#pragma unroll 8
    for (int s = warp; s < p.splits; s += 4) {
        const float f = __shfl_sync(0xffffffffu, s < 32 ? f0 : f1, s % 32);
        const float *src = p.part_o + (s * step + row) * D + lane * V;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(f, src[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc_s[warp][lane * V + i] = acc[i];
    __syncthreads();
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    if (threadIdx.x < D / 2) {
        const int d = 2 * threadIdx.x;
        float x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[i] = ((acc_s[0][d + i] + acc_s[1][d + i]) + (acc_s[2][d + i] + acc_s[3][d + i])) * inv;
        *reinterpret_cast<uint32_t *>(p.out + static_cast<int64_t>(token) * p.out_stride + head * D + d) =
            half2_of(x[0], x[1]);
    }
    if (threadIdx.x == 0 && p.lse != nullptr)
        p.lse[row] = L == 0.0f ? -INFINITY : (M - kShift + log2f(L)) * 0.693147180559945f;
}

// The same for up to four splits: a warp a row, every split's load in flight.
template <int D>
__global__ void __launch_bounds__(256) tree_attention_join4_kernel(const Params p) {
    const int lane = threadIdx.x % 32;
    const int h = blockIdx.y, b = blockIdx.z;
    const Seq sq = sequence(p, b, false);  // (not written by the kernel that is waited for)
    const int g = blockIdx.x * 8 + threadIdx.x / 32;
    ptx::grid_dependency_wait();
    if (g >= sq.n * p.group) return;
    const int head = h * p.group + g % p.group, token = sq.first + g / p.group;
    const int64_t row = static_cast<int64_t>(token) * p.q_heads + head;
    const int64_t step = static_cast<int64_t>(p.tokens) * p.q_heads;
    constexpr int V = D / 32;
    float2 a[4];
    float x[4][V];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s >= p.splits) break;
        a[s] = p.part_ml[s * step + row];
        const float *src = p.part_o + (s * step + row) * D + lane * V;
        if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src);
            x[s][0] = v.x, x[s][1] = v.y, x[s][2] = v.z, x[s][3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(src);
            x[s][0] = v.x, x[s][1] = v.y;
        }
    }
    float M = -INFINITY;
#pragma unroll
    for (int s = 0; s < 4; ++s)
        if (s < p.splits) M = fmaxf(M, a[s].x);
    const float base = M == -INFINITY ? 0.0f : M;
    float L = 0.0f, acc[V] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s >= p.splits) break;
        const float f = exp2_fast(a[s].x - base);
        L = fmaf(f, a[s].y, L);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(f, x[s][i], acc[i]);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint16_t *dst = p.out + static_cast<int64_t>(token) * p.out_stride + head * D + lane * V;
    if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(dst) =
            make_uint2(half2_of(acc[0] * inv, acc[1] * inv), half2_of(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t *>(dst) = half2_of(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[row] = L == 0.0f ? -INFINITY : (M - kShift + log2f(L)) * 0.693147180559945f;
}

// ------------------------------------------------------------------ host side
struct Plan {
    int wide;         // > 0: the tcgen05 form, with so many blocks of 128 rows a CTA
    int wr, row_blocks, splits;
    int workers;      // up to 8 rows: warps that share the tiles
    FewMode mode;     // ... and who takes an item
    int64_t pieces;
};

// Warps of a CTA, and of an SM.
struct FewWarps {
    int cta, sm;
};
template <int BITS>
FewWarps few_warps(int head_dim) {
    return head_dim == 64 ? FewWarps{FewCfg<BITS, 64>::NW, FewCfg<BITS, 64>::WORKERS}
                          : FewWarps{FewCfg<BITS, 128>::NW, FewCfg<BITS, 128>::WORKERS};
}

// Up to eight rows: who takes an item of at most `tiles` tiles.  Times are counted
// in tiles of 128 channels, about 0.8 us for a warp.  Measured, us, one token of
// each sequence over (a warp an item / a CTA an item / the stream and its join):
//     1 sequence, 32 heads of 128, INT8:     100 tokens 10.3 / 5.1 / 7.8
//         250 tokens 16.8 / 6.4 / 8.0, 600 tokens 33.7 / 9.6 / 8.8
//     16 sequences, 32 heads of 128, fp16:   60 tokens 8.1 / 16.2 / 10.5
//         150 tokens 13.9 / 21.1 / 14.7
//     128 sequences, 32 / 8 heads of 64, INT4: 60 tokens 6.3 / 9.2 / 15.7
//         250 tokens 12.6 / 14.1 / 21.2, 900 tokens 35.1 / 31.9 / 36.6
FewMode few_mode(const AttentionArgs &a, int64_t items, int64_t tiles, const FewWarps &w) {
    const int64_t resident = static_cast<int64_t>(sm_count()) * w.sm / w.cta, waves = (items + resident - 1) / resident;
    if (tiles <= 4) return waves == 1 ? kGroup : kWarp;
    if (tiles > 8 * w.cta) return kStream;  // (lengths then differ by more than the join takes)
    const double group = static_cast<double>(waves * ((tiles + w.cta - 1) / w.cta)) +
                         2.0 * static_cast<double>(waves - 1) * w.cta / w.sm;  // a CTA's start, unless others run
    const double stream = static_cast<double>(items * tiles) / static_cast<double>(resident * w.cta);
    const double rows = static_cast<double>(a.sequences) * a.q_heads * a.max_tokens;
    const double join = (2.5 + rows / 1024.0) * (128.0 / a.cache.head_dim);
    return group - (stream < 1.0 ? 1.0 : stream) <= join ? kGroup : kStream;
}

// The most rows of a key head that the warps' products take; more go to the
// tcgen05 form, whose tiles take as long for one row as for 128 and whose CTAs
// start slowly, but which reads and converts a tile once for all of them.  Both
// measured, 8 sequences of 4096 tokens, 8 key heads of 128, us (warps / tcgen05):
//     16 rows   INT4 28.3 / 41.9   INT8 33.9 / 39.3   fp16 44.2 / 35.2
//     32 rows   INT4 44.3 / 42.2   INT8 48.6 / 39.3   fp16 50.6 / 35.5
//     64 rows   INT4 66.8 / 42.6   INT8 71.5 / 39.8   fp16 74.4 / 36.0
// 32 sequences of 300 tokens, 32 rows: INT8 16.9 / 23.4.  Heads of 64, 64 rows:
// 2 sequences of 300 tokens INT8 9.4 / 10.2, 8 of 4096 tokens 50.0 / 37.2.
int narrow_rows(const AttentionArgs &a) {
    const bool long_context = a.max_context >= 2048;
    if (a.cache.head_dim == 64) return long_context ? 32 : 64;
    if (!long_context) return 32;
    return a.cache.kv_type == QUIK_KV_FP16 ? 8 : 16;
}

// Up to eight rows: the transposed form (wr 0); streamed, with as many workers as
// are resident at once, or one for each tile.
// More (narrow_rows): one or two row warps (a warp's products have 16), and splits of the
// cached tokens, enough CTAs for about two a resident slot, while each warp
// group keeps at least four tiles.
Plan plan_of(const AttentionArgs &a) {
    Plan r{};
    const int64_t rows = static_cast<int64_t>(a.max_tokens) * (a.q_heads / a.cache.heads);
    r.wr = rows <= 8 ? 0 : rows <= 16 ? 1 : 2;
    const int block = r.wr == 0 ? 8 : 16 * r.wr;
    r.row_blocks = static_cast<int>((rows + block - 1) / block);
    const int64_t items = static_cast<int64_t>(a.sequences) * a.cache.heads * r.row_blocks;
    const int64_t tiles = (static_cast<int64_t>(a.max_context) + a.max_tokens + kTile - 1) / kTile;
    if (rows > narrow_rows(a)) {
        r.wide = rows <= 128 ? 1 : 2;
        r.row_blocks = static_cast<int>((rows + 128 * r.wide - 1) / (128 * r.wide));
        const int64_t ctas = static_cast<int64_t>(a.sequences) * a.cache.heads * r.row_blocks;
        // one CTA an SM: the number of splits with the least time, counted in tiles
        // of 64 tokens (start and end of a CTA about four, joining about six)
        const int64_t sms = sm_count(), long_tiles = (tiles + 1) / 2;
        int64_t best = INT64_MAX;
        for (int s = 1; s <= kMaxSplits && (s == 1 || long_tiles >= 4 * s); ++s) {
            const int64_t cost = (ctas * s + sms - 1) / sms * ((long_tiles + s - 1) / s + 4) + (s > 1 ? 6 : 0);
            if (cost < best) best = cost, r.splits = s;
        }
        return r;
    }
    if (r.wr == 0) {
        const FewWarps w = a.cache.kv_type == QUIK_KV_INT4   ? few_warps<4>(a.cache.head_dim)
                           : a.cache.kv_type == QUIK_KV_INT8 ? few_warps<8>(a.cache.head_dim)
                                                             : few_warps<16>(a.cache.head_dim);
        r.mode = few_mode(a, items, tiles, w);
        const int64_t all = r.mode == kWarp ? items : r.mode == kGroup ? items * w.cta : items * tiles;
        const int64_t most = static_cast<int64_t>(sm_count()) * w.sm;
        const int64_t ctas = ((all < most || r.mode != kStream ? all : most) + w.cta - 1) / w.cta;
        r.workers = w.cta * static_cast<int>(ctas < 1 ? 1 : ctas);
        r.pieces = items + r.workers;
        return r;
    }
    const int64_t slots = static_cast<int64_t>(sm_count()) * 2;
    int64_t s = (2 * slots + items - 1) / items;
    const int64_t most = tiles / (4 * (4 / r.wr));
    s = s < most ? s : most;
    s = s < kMaxSplits ? s : kMaxSplits;
    r.splits = s < 1 ? 1 : static_cast<int>(s);
    return r;
}

size_t partial_bytes(const AttentionArgs &a, const Plan &r) {
    if (r.mode != kStream) return 0;
    if (r.wide == 0 && r.wr == 0)
        return static_cast<size_t>(r.pieces) * 8 * (a.cache.head_dim * 4 + 8) +
               static_cast<size_t>(r.pieces - r.workers) * 8;
    if (r.splits == 1) return 0;
    return static_cast<size_t>(r.splits) * a.tokens * a.q_heads * (a.cache.head_dim * 4 + 8);
}

// The join of a call's partial results, launched while the first kernel runs;
// it waits for that kernel's results.
quik_status launch_join(const Params &p, void (*kernel)(Params), int threads, cudaStream_t stream,
                        unsigned rows_a_block = 1) {
    cudaLaunchConfig_t cfg{};
    const unsigned rows = static_cast<unsigned>(p.max_tokens) * p.group;
    cfg.gridDim = dim3((rows + rows_a_block - 1) / rows_a_block, p.heads, p.sequences);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? QUIK_OK : QUIK_ERR_CUDA;
}

template <int D>
quik_status join_splits(const Params &p, cudaStream_t stream) {
    if (p.splits <= 4) return launch_join(p, &tree_attention_join4_kernel<D>, 256, stream, 8);
    return launch_join(p, &tree_attention_join_kernel<D>, 128, stream);
}

template <class C>
quik_status run_few(const Params &p, cudaStream_t stream) {
    void (*kernel)(Params) = p.mode == kStream ? &tree_attention_few_kernel<C, kStream>
                             : p.mode == kWarp ? &tree_attention_few_kernel<C, kWarp>
                                               : &tree_attention_few_kernel<C, kGroup>;
    if (!attribute_set_once(reinterpret_cast<const void *>(kernel), C::SMEM)) return QUIK_ERR_CUDA;
    kernel<<<p.workers / C::NW, C::NW * 32, C::SMEM, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return QUIK_ERR_CUDA;
    if (p.mode != kStream) return QUIK_OK;
    // many pieces an item: more warps, so that a few rounds of loads see them all
    const int64_t items = static_cast<int64_t>(p.sequences) * p.heads * p.row_blocks;
    if (p.workers >= 48 * items) return launch_join(p, &tree_attention_few_join_kernel<C, 16>, 512, stream);
    return launch_join(p, &tree_attention_few_join_kernel<C, 4>, 128, stream);
}

template <class C>
quik_status run(const Params &p, void (*kernel)(Params), cudaStream_t stream) {
    if (!attribute_set_once(reinterpret_cast<const void *>(kernel), C::SMEM)) return QUIK_ERR_CUDA;
    const dim3 grid(p.splits * p.row_blocks, p.heads, p.sequences);
    kernel<<<grid, C::NW * 32, C::SMEM, stream>>>(p);
    if (p.splits > 1) {
        const quik_status st = join_splits<C::D>(p, stream);
        if (st != QUIK_OK) return st;
    }
    return cudaGetLastError() == cudaSuccess ? QUIK_OK : QUIK_ERR_CUDA;
}

template <int BITS, int D>
quik_status run_rows(const Params &p, int wr, cudaStream_t stream) {
    if (wr == 0) return run_few<FewCfg<BITS, D>>(p, stream);
    if (wr == 1) return run<Cfg<BITS, D, 1, 4>>(p, &tree_attention_kernel<Cfg<BITS, D, 1, 4>>, stream);
    return run<Cfg<BITS, D, 2, 4>>(p, &tree_attention_kernel<Cfg<BITS, D, 2, 4>>, stream);
}

template <int BITS>
quik_status run_dim(const Params &p, int head_dim, int wr, cudaStream_t stream) {
    return head_dim == 64 ? run_rows<BITS, 64>(p, wr, stream) : run_rows<BITS, 128>(p, wr, stream);
}

}  // namespace

size_t attention_workspace(const AttentionArgs &a) { return partial_bytes(a, plan_of(a)); }

quik_status launch_tree_attention(const AttentionArgs &a, cudaStream_t stream) {
    const Plan plan = plan_of(a);
    Params p;
    p.tokens = a.tokens;
    p.sequences = a.sequences;
    p.q_heads = a.q_heads;
    p.heads = a.cache.heads;
    p.group = a.q_heads / a.cache.heads;
    p.max_tokens = a.max_tokens;
    p.max_pages = a.max_pages;
    p.mask_words = a.mask_words;
    p.pages = a.cache.pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.cache.page_size) ++p.page_shift;
    p.splits = plan.splits;
    p.row_blocks = plan.row_blocks;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.k = static_cast<const uint8_t *>(a.cache.k);
    p.v = static_cast<const uint8_t *>(a.cache.v);
    p.ks = a.cache.k_scale;
    p.vs = a.cache.v_scale;
    p.page_table = a.page_table;
    p.context = a.context;
    p.cu = a.cu_tokens;
    p.mask = a.mask;
    p.out = a.out;
    p.out_stride = a.out_stride;
    p.lse = a.lse;
    p.part_o = a.partial;
    p.part_ml = reinterpret_cast<float2 *>(
        a.partial + static_cast<size_t>(plan.splits) * a.tokens * a.q_heads * a.cache.head_dim);
    p.workers = plan.workers;
    p.mode = plan.mode;
    p.piece_o = reinterpret_cast<float4 *>(a.partial);
    p.piece_ml = reinterpret_cast<float2 *>(a.partial + static_cast<size_t>(plan.pieces) * 8 * a.cache.head_dim);
    p.item_span = reinterpret_cast<int *>(p.piece_ml + plan.pieces * 8);
    if (plan.wide > 0) {
        const quik_status st = launch_attention_wide(p, a.cache.kv_type, a.cache.head_dim, plan.wide, stream);
        if (st != QUIK_OK || p.splits == 1) return st;
        return a.cache.head_dim == 64 ? join_splits<64>(p, stream) : join_splits<128>(p, stream);
    }
    if (a.cache.kv_type == QUIK_KV_INT4) return run_dim<4>(p, a.cache.head_dim, plan.wr, stream);
    if (a.cache.kv_type == QUIK_KV_INT8) return run_dim<8>(p, a.cache.head_dim, plan.wr, stream);
    return run_dim<16>(p, a.cache.head_dim, plan.wr, stream);
}

unsigned int take_attention_errors() {
    unsigned int word = 0;
    if (cudaMemcpyFromSymbol(&word, g_attn_bad_index, sizeof(word)) != cudaSuccess) return 0;
    return counter_increase(kCounterBadPage, word);
}

}  // namespace quik
