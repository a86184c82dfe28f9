// tree_attention_wide.cu -- attention of many rows (trees of drafted tokens,
// chunks of a prompt) over the paged KV cache on the tcgen05 tensor cores.
//
// A CTA takes up to two blocks of 128 query rows of one sequence and key head
// and a run of its cached tokens, 64 at a time:
//     S = Q K^T    tcgen05 kind::f16, 128 x 64, both operands in shared memory
//     p            four warps a row block, a thread a row, as in tree_attention.cu
//     O += P V     P in tensor memory (over the S it came from), V in shared memory
// Six loader warps bring the cached rows in by cp.async; quantised rows land in a
// raw ring and are converted to fp16 (exact: they are integer codes) into the
// products' operand tiles, once for both row blocks.  A warp of its own brings
// the scales and works out their unit (by one of the loaders it made that one the
// slowest: 64 rows of 4096 INT8 tokens 45.1 -> 41.4 us without).  K and V tiles
// have one image, [64 tokens][64 channels] blocks in the 128-byte swizzle: K is
// read along its rows (K-major), V across them (MN-major, the transpose bit of
// B).  S is double-buffered, so the products of tile t + 1 run under the softmax
// of tile t, and the two row blocks' softmaxes under each other's products.
//
// The running maximum is only moved when a row's scores exceed it by 5 in log2
// (p carries 2^10 here, so p <= 2^15 < 65504): rescaling O is a trip through
// tensor memory, and after the first tiles it hardly ever happens.
//
// 256 rows x 64 tokens take 2300 to 2400 cycles, in which the softmax warps, two
// beside each other on a quarter of the SM, are never idle: 200 for the wait, 550
// to 900 to the maximum, 1400 for the exponentials (1024 of them the rate of the
// special-function units for both), 100 for P.  The products take 900 and the
// conversion 1800, beside them.  Around the tiles a CTA takes 6000 cycles to its
// first S and 5000 for its results.  64 drafted tokens over 8 x 4096 of INT8,
// 32 / 8 heads of 128: 55 to 56 us with the join, 17.4 by the products' rate.  A chunk
// of 2048 tokens of a prompt, the same heads: fp16 91 us, INT8 76, INT4 78 (21.3 by the
// products' rate; quantised rows skip the masks on tiles that all rows see whole).
// Tried and slower:
// two threads a row (more warps, the same time: 60.5 us), one row block by two
// groups that take tiles in turn (64 rows fp16 55.0 against 38.0 us), pieces by
// each sequence's own length (60.7 against 58.3 us: finding the place costs more).
#include <type_traits>

#include "attention.cuh"

namespace quik {

// Waits of this file's kernel that ran out: only ever grows.
static __device__ unsigned int g_wide_waits;

namespace {

constexpr int kPitch = 36;          // floats of a row in the write-out's shared memory (32 of them)
constexpr int kTok = 64;            // cached tokens per tile
constexpr float kLazy = 5.0f;        // how far scores may pass the running maximum (log2)
constexpr float kWideShift = 10.0f;  // p carries 2^10
constexpr float kJoinShift = 14.0f;  // what the join takes p to carry
constexpr int kLoaders = 192;        // threads; and a warp for the scales
constexpr int kOwnUnit = 512;        // marks a tile whose scales' unit goes by the row (added to -100 .. 126)

template <int BITS_, int D_, int QT_>
struct WideCfg {
    static constexpr int BITS = BITS_, D = D_, QT = QT_;
    static constexpr int RB = D * BITS / 8, CPR = RB / 16;
    static constexpr int THREADS = QT * 128 + kLoaders + 64;
    static constexpr int Q_BYTES = QT * 128 * D * 2;
    static constexpr int HALF = kTok * D * 2;  // a K or V tile
    static constexpr int STAGES = BITS == 16 ? 4 : 3;
    static constexpr int RAW = BITS == 16 ? 0 : 2 * kTok * RB + 2 * kTok * 4;
    static constexpr int RAWS = BITS == 16 ? 0 : BITS == 8 ? 3 : 4;
    static constexpr int META = 2 * kTok * 4 + 16 + kLoaders / 32 * 8;  // K scales, V scales, int4, an int2 a loader warp
    static constexpr int OUT_BYTES = QT * 128 * kPitch * 4;  // the write-out's, in Q's place
    static constexpr int OFF_KV = Q_BYTES > OUT_BYTES ? Q_BYTES : OUT_BYTES;
    static constexpr int OFF_RAW = OFF_KV + STAGES * 2 * HALF;
    static constexpr int OFF_META = OFF_RAW + RAWS * RAW;
    static constexpr int OFF_BAR = OFF_META + STAGES * META;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;  // + alignment of the base to 1024
    static constexpr int COLS = QT * (2 * kTok + D);   // tensor-memory columns
    static constexpr int ALLOC = COLS <= 256 ? 256 : 512;
    static constexpr int STEPS = D / 16;
};

struct WideBars {
    uint64_t kv_full[4], kv_empty[4], s_full[2][2], p_full[2][2], pv_done[2], q_full, drain;
    uint32_t tmem;
    int abort;
};

// Wait for a phase, for at most kWaitLimitNs and not once another role has given
// up.  Every lane of a warp waits for itself; a warp goes by all_of its answers.
__device__ __forceinline__ bool wide_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
#pragma unroll 1
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (ptx::global_timer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicAdd(&g_wide_waits, 1u);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool all_of(bool ok) { return __all_sync(0xffffffffu, ok); }

// D[tmem] += A[tmem] * B[smem desc], fp16 kind, A in tensor memory (lane = row,
// two fp16 a column, K in column order).
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc)
        : "memory");
}
// MN-major operand in the 128-byte swizzle: blocks of 64 elements x 8 k-rows of
// 128 bytes; 8-row groups 1024 bytes apart (stride), 64-element blocks HALF / 2
// (leading).
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t block_bytes) {
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(block_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The exponent of the unit when a scale's is e: with some room, so that it moves less often.
__device__ __forceinline__ int raised(int R, int e) { return e > R ? min(e + 1, 126) : R; }

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

// 16-byte chunk c (8 channels) of row r of an operand of `rows` rows.
__device__ __forceinline__ uint32_t swizzled(int r, int c, int rows) {
    return (c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// Whether any of eight fp16 values is an infinity or NaN.
__device__ __forceinline__ bool not_finite(uint4 w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) any |= (u[i] & 0x7c00u) == 0x7c00u || (u[i] & 0x7c000000u) == 0x7c000000u;
    return any;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) tree_attention_wide_kernel(const AttnParams p) {
    constexpr int BITS = C::BITS, D = C::D, QT = C::QT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
    WideBars *bars = reinterpret_cast<WideBars *>(smem + C::OFF_BAR);
    // (values broadcast from lane 0 are the same in the whole warp for the compiler
    // too: the products' descriptors and loop then live in uniform registers)
    const int lane = threadIdx.x % 32, warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
    const int split = blockIdx.x % p.splits;
    const int rb = p.row_blocks - 1 - blockIdx.x / p.splits;  // (a key head's blocks that see most start first)
    const int h = blockIdx.y, b = blockIdx.z;
    Seq sq = sequence(p, b, blockIdx.x == 0 && h == 0 && threadIdx.x == 0);
    const int rows = sq.n * p.group, row0 = rb * QT * 128;
    if (row0 >= rows) return;
    // without a mask, what is past the block's last token is seen by none of its rows
    if (p.mask == nullptr)
        sq.total = static_cast<int>(min(static_cast<int64_t>(sq.total),
                                        static_cast<int64_t>(sq.ctx) + (row0 + QT * 128 - 1) / p.group + 1));
    const int tiles = (sq.total + kTok - 1) / kTok;
    const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * split / p.splits);
    const int n = __shfl_sync(
        0xffffffffu, static_cast<int>(static_cast<int64_t>(tiles) * (split + 1) / p.splits) - t0, 0);

    constexpr int MMA_WARP = QT * 4 + kLoaders / 32 + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            ptx::mbar_init(&bars->kv_full[i], BITS == 16 ? kLoaders : kLoaders + 32);
            ptx::mbar_init(&bars->kv_empty[i], 1);
        }
        for (int g = 0; g < QT; ++g) {
            for (int i = 0; i < 2; ++i) {
                ptx::mbar_init(&bars->s_full[g][i], 1);
                ptx::mbar_init(&bars->p_full[g][i], 128);
            }
            ptx::mbar_init(&bars->pv_done[g], 1);
        }
        ptx::mbar_init(&bars->q_full, QT * 128);
        ptx::mbar_init(&bars->drain, 1);
        bars->abort = 0;
        ptx::fence_barrier_init();
    }
    if (warp == MMA_WARP) ptx::tmem_alloc(&bars->tmem, C::ALLOC);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);
    volatile int *abort = &bars->abort;
    const auto s_col = [&](int g, int buf) { return tmem + (g * 2 + buf) * kTok; };
    const auto o_col = [&](int g) { return tmem + QT * 2 * kTok + g * D; };

    // 8 warps of 184 registers a thread and 8 of 72 are the 16 of 128 that start.
    // All four warps of a warpgroup have to meet the same instruction, and the last
    // one's belong to two roles: so it comes before the roles part.
    if constexpr (QT == 2) {
        if (warp < QT * 4)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    }
    if (warp < QT * 4) {
        // ================================================ softmax: a thread a row
        const int g = warp / 4;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4) * 32 << 16;
        const int row = row0 + g * 128 + warp % 4 * 32 + lane;
        const int tok = row < rows ? row / p.group : -1;
        const int head = h * p.group + row - row / p.group * p.group;  // (of a row that is there)
        float m = -INFINITY, l = 0.0f;
        int R = -100;
        {
            // this warp's rows of Q (zeros past the last), a row's chunks by lanes beside
            // each other; where a row starts comes from its own lane
            constexpr int CH = D / 8;
            const int64_t start =
                tok < 0 ? -1 : static_cast<int64_t>(sq.first + tok) * p.q_stride + static_cast<int64_t>(head) * D;
            const uint32_t dst = ptx::smem_u32(smem) + g * (128 * D * 2);
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int r = i * (32 / CH) + lane / CH, c = lane % CH;
                const int64_t from = __shfl_sync(0xffffffffu, start, r);
                copy16(dst + swizzled(warp % 4 * 32 + r, c, 128), from < 0 ? p.q : p.q + from + 8 * c, from >= 0);
            }
            copy_commit();
            uint32_t z[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) ptx::tmem_st_32x32b_x32(o_col(g) + lanes + 32 * c, z);
            copy_wait<0>();
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&bars->q_full);
        }
        bool alive = true;
        for (int t = 0; t < n; ++t) {
            const int stage = t % C::STAGES, buf = t & 1;
            const uint8_t *meta = smem + C::OFF_META + stage * C::META;
            // (the tile's scales and masks come from the loaders, S from the products)
            // Both are done as a rule: asked for together, the answers' latencies overlap.
            const bool kv = ptx::mbar_try_wait(&bars->kv_full[stage], (t / C::STAGES) & 1);
            const bool sc = ptx::mbar_try_wait(&bars->s_full[g][buf], (t >> 1) & 1);
            alive = all_of((kv || wide_wait(&bars->kv_full[stage], (t / C::STAGES) & 1, abort)) &&
                           (sc || wide_wait(&bars->s_full[g][buf], (t >> 1) & 1, abort)));
            if (!alive) break;
            ptx::tc_fence_after();
            uint32_t s[64];
            float4 ks[BITS == 16 ? 1 : 16];
            {
                uint32_t lo[32], hi[32];
                ptx::tmem_ld_32x32b_x32(s_col(g, buf) + lanes, lo);
                ptx::tmem_ld_32x32b_x32(s_col(g, buf) + lanes + 32, hi);
                if constexpr (BITS != 16) {  // the keys' scales come meanwhile
#pragma unroll
                    for (int i = 0; i < 16; ++i) ks[i] = *reinterpret_cast<const float4 *>(meta + 16 * i);
                }
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) s[i] = lo[i], s[32 + i] = hi[i];
            }
            const int4 info = *reinterpret_cast<const int4 *>(meta + 2 * kTok * 4);
            const int j0 = info.z;
            // ---- scores in log2 units
            const uint64_t sc2 = ptx::f2(p.scale_log2, p.scale_log2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                uint64_t k0 = sc2, k1 = sc2;
                if constexpr (BITS != 16) {
                    k0 = ptx::f2(ks[i].x, ks[i].y), k1 = ptx::f2(ks[i].z, ks[i].w);
                }
                float x, y;
                ptx::f2_split(ptx::f2_mul(ptx::f2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), k0), x, y);
                s[4 * i] = __float_as_uint(x), s[4 * i + 1] = __float_as_uint(y);
                ptx::f2_split(ptx::f2_mul(ptx::f2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), k1), x,
                              y);
                s[4 * i + 2] = __float_as_uint(x), s[4 * i + 3] = __float_as_uint(y);
            }
            unsigned see[2] = {static_cast<unsigned>(info.x), static_cast<unsigned>(info.y)};
            const bool own = BITS != 16 && info.w > 126;  // (rows see the tile each in their way)
            const bool masked = (see[0] & see[1]) != 0xffffffffu || (BITS == 16 ? j0 + kTok > 0 : own);
            if (masked) {
                see[0] &= seen(p, sq.first, tok, j0);
                see[1] &= seen(p, sq.first, tok, j0 + 32);
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (!((see[i / 32] >> (i % 32)) & 1u)) s[i] = 0xff800000u;
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // (four short chains, not one)
#pragma unroll
            for (int i = 0; i < 64; i += 2)
                tops[i / 2 % 4] = fmaxf(fmaxf(tops[i / 2 % 4], __uint_as_float(s[i])), __uint_as_float(s[i + 1]));
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            // ---- move the maximum and the unit of the values' scales only where they must
            const bool move = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
            int unit = R;
            if constexpr (BITS != 16) {
                if (!own) {
                    unit = info.w;
                } else if (info.w - kOwnUnit > R) {
                    // a scale above this row's unit, which the row may not see
                    unsigned most = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float4 v4 = *reinterpret_cast<const float4 *>(meta + kTok * 4 + 16 * i);
                        const float v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if ((see[i / 8] >> (4 * i % 32 + j)) & 1u) most = max(most, finite_bits(v[j]));
                    }
                    unit = raised(R, top_exponent(most));
                }
            }
            if (__any_sync(0xffffffffu, move || unit != R)) {
                const float to = move ? top : m;
                float alpha = move ? (m == -INFINITY ? 0.0f : exp2_fast(m - to)) : 1.0f;
                l *= alpha;
                m = to;
                if (unit != R) alpha *= exp2_fast(static_cast<float>(R - unit));
                R = unit;
                if (t > 0) {  // (O is zero before the first tile)
                    alive = all_of(wide_wait(&bars->pv_done[g], (t - 1) & 1, abort));
                    if (!alive) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        ptx::tmem_ld_32x32b_x16(o_col(g) + lanes + 16 * c, o);
                        ptx::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        ptx::tmem_st_32x32b_x16(o_col(g) + lanes + 16 * c, o);
                    }
                }
            }
            // ---- p
            const float base = (m == -INFINITY ? 0.0f : m) - kWideShift;
            const uint64_t b2 = ptx::f2(base, base);
            // what the scales as they stand in shared memory still lack
            const float rest = own ? unit_of(R) : 1.0f;
            const uint64_t rest2 = ptx::f2(rest, rest);
            uint64_t sum = 0;
            uint32_t pk[32];
            auto weights = [&](auto some) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float x[4];
                    ptx::f2_split(ptx::f2_sub(ptx::f2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), b2), x[0],
                                  x[1]);
                    ptx::f2_split(ptx::f2_sub(ptx::f2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), b2),
                                  x[2], x[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = exp2_fast(x[j]);
                    sum = ptx::f2_add(sum, ptx::f2_add(ptx::f2(x[0], x[1]), ptx::f2(x[2], x[3])));
                    if constexpr (BITS != 16) {
                        const float4 v4 = *reinterpret_cast<const float4 *>(meta + kTok * 4 + 16 * i);
                        uint64_t v0 = ptx::f2(v4.x, v4.y), v1 = ptx::f2(v4.z, v4.w);
                        if constexpr (decltype(some)::value) v0 = ptx::f2_mul(v0, rest2), v1 = ptx::f2_mul(v1, rest2);
                        ptx::f2_split(ptx::f2_mul(ptx::f2(x[0], x[1]), v0), x[0], x[1]);
                        ptx::f2_split(ptx::f2_mul(ptx::f2(x[2], x[3]), v1), x[2], x[3]);
                        if constexpr (decltype(some)::value) {  // an unseen token's scale may be anything
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (!((see[i / 8] >> (4 * i % 32 + j)) & 1u)) x[j] = 0.0f;
                        }
                    }
                    pk[2 * i] = half2_of(x[0], x[1]);
                    pk[2 * i + 1] = half2_of(x[2], x[3]);
                }
            };
            if (BITS != 16 && masked)
                weights(std::true_type{});
            else
                weights(std::false_type{});
            float a, c;
            ptx::f2_split(sum, a, c);
            l += a + c;
            if constexpr (BITS == 16) {
                // values that are not finite, in a tile that some row does not see whole:
                // the eight channels around them are zeros in shared memory, and the
                // rows that see the token add them here
                const uint4 w0 = *reinterpret_cast<const uint4 *>(meta + 2 * kTok * 4 + 16);
                const uint4 w1 = *reinterpret_cast<const uint4 *>(meta + 2 * kTok * 4 + 32);
                const uint4 w2 = *reinterpret_cast<const uint4 *>(meta + 2 * kTok * 4 + 48);
                const unsigned odds[2] = {w0.x | w0.z | w1.x | w1.z | w2.x | w2.z, w0.y | w0.w | w1.y | w1.w | w2.y | w2.w};
                if ((odds[0] | odds[1]) != 0) {
                    if (t > 0) {
                        alive = all_of(wide_wait(&bars->pv_done[g], (t - 1) & 1, abort));
                        if (!alive) break;
                        ptx::tc_fence_after();
                    }
                    ptx::tmem_st_wait();
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll 1
                        for (unsigned odd = odds[half]; odd != 0; odd &= odd - 1) {
                            const int x = __ffs(odd) - 1, pos = (t0 + t) * kTok + 32 * half + x;
                            const bool on = (see[half] >> x) & 1u;
                            uint32_t w = 0;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i == x / 2) w = pk[16 * half + i];
                            const __half2 h2 = *reinterpret_cast<const __half2 *>(&w);
                            const float pr = x % 2 ? __high2float(h2) : __low2float(h2);
                            const int id = p.page_table[static_cast<int64_t>(b) * p.max_pages + (pos >> p.page_shift)];
                            const int64_t vr = ((static_cast<int64_t>(id) * p.heads + h) << p.page_shift) +
                                               (pos & ((1 << p.page_shift) - 1));
                            const uint4 *v = reinterpret_cast<const uint4 *>(p.v + vr * C::RB);
#pragma unroll 1
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                ptx::tmem_ld_32x32b_x16(o_col(g) + lanes + 16 * q, o);
                                ptx::tmem_ld_wait();
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const uint4 v8 = v[2 * q + y];
                                    const uint32_t u[4] = {v8.x, v8.y, v8.z, v8.w};
                                    if (on && not_finite(v8)) {
#pragma unroll
                                        for (int i = 0; i < 4; ++i) {
                                            const float2 f2v = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
                                            uint32_t &a0 = o[8 * y + 2 * i], &a1 = o[8 * y + 2 * i + 1];
                                            a0 = __float_as_uint(fmaf(pr, f2v.x, __uint_as_float(a0)));
                                            a1 = __float_as_uint(fmaf(pr, f2v.y, __uint_as_float(a1)));
                                        }
                                    }
                                }
                                ptx::tmem_st_32x32b_x16(o_col(g) + lanes + 16 * q, o);
                                ptx::tmem_st_wait();
                            }
                        }
                }
            }
            // The last wait below is for the last product.  By its parity it would pass
            // while the product before that one is still under way: so that one is
            // waited for here, where the last cannot have started.
            if (t > 0 && t == n - 1) {
                alive = all_of(wide_wait(&bars->pv_done[g], (t - 1) & 1, abort));
                if (!alive) break;
            }
            ptx::tmem_st_32x32b_x32(s_col(g, buf) + lanes, pk);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bars->p_full[g][buf]);
        }
        if (alive && n > 0) alive = all_of(wide_wait(&bars->pv_done[g], (n - 1) & 1, abort));
        if (alive) {
            // ---- results, 32 channels at a time through shared memory (Q's place:
            // every product that reads it is done) into whole lines
            ptx::tmem_st_wait();
            ptx::tc_fence_after();
            float *buf = reinterpret_cast<float *>(smem) + warp * 32 * kPitch;
            const float up = BITS == 16 ? 1.0f : unit_of(-R);
            const float f = p.splits > 1 ? up : l == 0.0f ? 0.0f : up / l;
            const int64_t at = tok < 0 ? -1 : static_cast<int64_t>(sq.first + tok) * p.q_heads + head;
            const int64_t out_at =
                tok < 0 ? -1 : (sq.first + tok) * p.out_stride + static_cast<int64_t>(head) * D;
            if (tok >= 0) {
                if (p.splits > 1)
                    p.part_ml[static_cast<int64_t>(split) * p.tokens * p.q_heads + at] =
                        make_float2(m + (kJoinShift - kWideShift), l);
                else if (p.lse != nullptr)
                    p.lse[at] = l == 0.0f ? -INFINITY : (m - kWideShift + log2f(l)) * 0.693147180559945f;
            }
            float *const part_o = p.part_o + static_cast<int64_t>(split) * p.tokens * p.q_heads * D;
            if (n == 0 && tok >= 0) {
                // no tiles: zeros, and not through Q's place, which is still being filled
                float4 *po = reinterpret_cast<float4 *>(part_o + at * D);
                uint4 *qo = reinterpret_cast<uint4 *>(p.out + out_at);
#pragma unroll 1
                for (int i = 0; i < D / 4; ++i) {
                    if (p.splits > 1)
                        po[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    else if (i < D / 8)
                        qo[i] = make_uint4(0, 0, 0, 0);
                }
            }
            // where this lane writes: eight rows of partial results, or four of the output
            float *part[8];
            uint16_t *out[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t y = __shfl_sync(0xffffffffu, at, i * 4 + lane / 8);
                part[i] = y < 0 || n == 0 || p.splits == 1 ? nullptr : part_o + y * D + lane % 8 * 4;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t y = __shfl_sync(0xffffffffu, out_at, i * 8 + lane / 4);
                out[i] = y < 0 || n == 0 ? nullptr : p.out + y + lane % 4 * 8;
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                if (n == 0) break;
                uint32_t o[32];
                ptx::tmem_ld_32x32b_x32(o_col(g) + lanes + 32 * c, o);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(buf + lane * kPitch + 4 * i) =
                        make_float4(__uint_as_float(o[4 * i]) * f, __uint_as_float(o[4 * i + 1]) * f,
                                    __uint_as_float(o[4 * i + 2]) * f, __uint_as_float(o[4 * i + 3]) * f);
                __syncwarp();
                if (p.splits > 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (part[i] != nullptr)
                            *reinterpret_cast<float4 *>(part[i] + 32 * c) =
                                *reinterpret_cast<const float4 *>(buf + (i * 4 + lane / 8) * kPitch + lane % 8 * 4);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (out[i] == nullptr) continue;
                        const float *r = buf + (i * 8 + lane / 4) * kPitch + lane % 4 * 8;
                        const float4 x = *reinterpret_cast<const float4 *>(r);
                        const float4 y = *reinterpret_cast<const float4 *>(r + 4);
                        *reinterpret_cast<uint4 *>(out[i] + 32 * c) =
                            make_uint4(half2_of(x.x, x.y), half2_of(x.z, x.w), half2_of(y.x, y.y), half2_of(y.z, y.w));
                    }
                }
                __syncwarp();
            }
        }
    } else if (warp < MMA_WARP) {
        // ================================================ loaders
        const int lt = threadIdx.x - QT * 128;
        // a thread's chunks of K (and V): the same place in rows TSTEP apart
        constexpr int CHUNKS = kTok * C::CPR, PER = (CHUNKS + kLoaders - 1) / kLoaders;
        constexpr int TSTEP = kLoaders / C::CPR;
        static_assert(kLoaders % C::CPR == 0, "a thread keeps its place in the rows");
        const int tok0 = lt / C::CPR, ch = lt % C::CPR;
        const int32_t *table = p.page_table + static_cast<int64_t>(b) * p.max_pages;
        const int64_t head = static_cast<int64_t>(h) << p.page_shift;
        const unsigned page_rows = static_cast<unsigned>(p.heads) << p.page_shift;
        const int page_mask = (1 << p.page_shift) - 1;
        // Page numbers of a tile's four groups of 16 tokens, as the table has them (kNone:
        // no such tokens).  They are looked at (checked) a tile later, when the loads
        // are long done: looked at at once they cost every tile a memory latency.
        constexpr int kNone = INT32_MIN;
        // (reported by the last block, the one that comes to all of the sequence's tokens
        // without a mask too)
        const bool report = lt == 0 && row0 + QT * 128 >= rows;
        auto pages = [&](int t, int (&raw)[4]) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int pos = (t0 + t) * kTok + 16 * f;
                raw[f] = t < n && pos < sq.total ? table[pos >> p.page_shift] : kNone;
            }
        };
        auto checked = [&](const int (&raw)[4], int (&id)[4]) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                id[f] = static_cast<unsigned>(raw[f]) < static_cast<unsigned>(p.pages) ? raw[f] : -1;
                if (id[f] < 0 && raw[f] != kNone && report) atomicAdd(&g_attn_bad_index, 1u);
            }
        };
        auto id_of = [](const int (&id)[4], int f) { return f & 2 ? (f & 1 ? id[3] : id[2]) : (f & 1 ? id[1] : id[0]); };
        auto row_of = [&](int id, int t, int token) {
            return static_cast<int64_t>(static_cast<uint64_t>(static_cast<unsigned>(id)) * page_rows) + head +
                   (((t0 + t) * kTok + token) & page_mask);
        };
        auto live_of = [&](const int (&id)[4], int t, int half) {
            const int left = sq.total - (t0 + t) * kTok - 32 * half;
            const unsigned in = left >= 32 ? 0xffffffffu : left <= 0 ? 0u : (1u << left) - 1u;
            return in & ((id[2 * half] >= 0 ? 0xffffu : 0u) | (id[2 * half + 1] >= 0 ? 0xffff0000u : 0u));
        };
        // copies of a tile's rows, to where dst_of(token, 0 or 1 for V) says
        auto copies = [&](int t, const int (&id)[4], auto dst_of) {
            const bool whole = (t0 + t + 1) * kTok <= sq.total && (id[0] | id[1] | id[2] | id[3]) >= 0;
            if (whole && p.page_shift >= 6) {
                // in one page, and there: one offset places it all
                const int64_t off = row_of(id[0], t, 0) * C::RB + lt * 16;
                const uint8_t *k = p.k + off, *v = p.v + off;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (CHUNKS % kLoaders != 0 && lt + j * kLoaders >= CHUNKS) break;
                    copy16(dst_of(tok0 + j * TSTEP, 0), k + j * kLoaders * 16, true);
                    copy16(dst_of(tok0 + j * TSTEP, 1), v + j * kLoaders * 16, true);
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int token = tok0 + j * TSTEP;
                if (CHUNKS % kLoaders != 0 && lt + j * kLoaders >= CHUNKS) break;
                const int pid = id_of(id, token / 16);
                const bool ok = pid >= 0 && (t0 + t) * kTok + token < sq.total;
                const int64_t off = ok ? row_of(pid, t, token) * C::RB + ch * 16 : 0;
                copy16(dst_of(token, 0), p.k + off, ok);
                copy16(dst_of(token, 1), p.v + off, ok);
            }
        };
        int raw_id[4], id[4];
        pages(0, raw_id);
        if (lt >= kLoaders && BITS == 16) {
            // (no scales)
        } else if constexpr (BITS == 16) {
            // straight into the operand tiles, two tiles ahead of the one handed over
            constexpr int AHEAD = 2;
            unsigned live[AHEAD][2];  // of tiles t - AHEAD .. t - 1
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) live[i][0] = live[i][1] = 0;
            for (int t = 0; t < n + AHEAD; ++t) {
                // tile t - AHEAD is handed over before tile t's stage is waited for, which
                // comes free behind products with earlier tiles
                if (t >= AHEAD) {
                    copy_wait<AHEAD - 1>();
                    const int d = t - AHEAD;
                    const int stage = d % C::STAGES, j0 = (t0 + d) * kTok - sq.ctx;
                    uint8_t *meta = smem + C::OFF_META + stage * C::META + 2 * kTok * 4;
                    if (lt == 0)
                        *reinterpret_cast<int4 *>(meta) =
                            make_int4(static_cast<int>(live[0][0]), static_cast<int>(live[0][1]), j0, 0);
                    unsigned odd[2] = {0u, 0u};
                    if (j0 + kTok > 0) {
                        // new tokens, which some rows see and others not: an infinity or NaN
                        // in their values must not meet a p of zero in the product
                        uint8_t *v = smem + C::OFF_KV + stage * 2 * C::HALF + C::HALF;
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const int token = tok0 + j * TSTEP;
                            if (CHUNKS % kLoaders != 0 && lt + j * kLoaders >= CHUNKS) break;
                            uint4 *at = reinterpret_cast<uint4 *>(v + swizzled(token, ch, kTok));
                            if (not_finite(*at)) {
                                *at = make_uint4(0, 0, 0, 0);
                                odd[token / 32] |= 1u << (token % 32);
                            }
                        }
                    }
                    odd[0] = __reduce_or_sync(0xffffffffu, odd[0]);
                    odd[1] = __reduce_or_sync(0xffffffffu, odd[1]);
                    if (lane == 0)  // each loader warp has a word pair of its own
                        *reinterpret_cast<uint2 *>(meta + 16 + 8 * (lt / 32)) = make_uint2(odd[0], odd[1]);
                    ptx::fence_proxy_async_smem();
                    ptx::mbar_arrive(&bars->kv_full[stage]);
                }
#pragma unroll
                for (int i = 0; i < AHEAD - 1; ++i) live[i][0] = live[i + 1][0], live[i][1] = live[i + 1][1];
                if (t < n) {
                    const int stage = t % C::STAGES;
                    if (t >= C::STAGES &&
                        !all_of(wide_wait(&bars->kv_empty[stage], (t / C::STAGES - 1) & 1, abort)))
                        break;
                    const uint32_t at = ptx::smem_u32(smem) + C::OFF_KV + stage * 2 * C::HALF;
                    checked(raw_id, id);
                    pages(t + 1, raw_id);
                    copies(t, id, [&](int token, int v) { return at + v * C::HALF + swizzled(token, ch, kTok); });
                    live[AHEAD - 1][0] = live_of(id, t, 0), live[AHEAD - 1][1] = live_of(id, t, 1);
                }
                copy_commit();
            }
        } else {
            // a ring of tiles as they come: RAWS - 1 on their way
            uint8_t *raws = smem + C::OFF_RAW;
            // Eight lanes write eight 16-byte chunks at a time, the lanes of the second
            // half of a row's chunks (the second 64 channels, at the same place in their
            // own block) in the other order: no two then meet in a bank.
            const int turn = D == 128 ? ch / (C::CPR / 2) : 0;
            const bool scales = lt >= kLoaders;
            // The unit of the values' scales, 2^R above every one so far, of the tiles
            // that all rows see alike: the context, and without a mask what lies before
            // the block's first token.  Nothing of this kind comes after a tile of the
            // other kind, where a row's unit is its own, over the tokens that it sees (a
            // scale of another token would take the bits of its weights).
            int R = -100;
            const int alike = p.mask == nullptr ? row0 / p.group + 1 : 0;  // new tokens that all rows see
            auto issue = [&](int t) {
                checked(raw_id, id);
                pages(t + 1, raw_id);
                if (t < n) {
                    const uint32_t at = ptx::smem_u32(raws + t % C::RAWS * C::RAW);
                    if (!scales) {
                        copies(t, id, [&](int token, int v) { return at + (v * kTok + token) * C::RB + ch * 16; });
                    } else {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int token = lane + 32 * half, pid = id_of(id, token / 16);
                            const bool ok = pid >= 0 && (t0 + t) * kTok + token < sq.total;
                            const int64_t r = ok ? row_of(pid, t, token) : 0;
                            copy4(at + 2 * kTok * C::RB + 4 * token, p.ks + r, ok);
                            copy4(at + 2 * kTok * C::RB + 4 * (kTok + token), p.vs + r, ok);
                        }
                    }
                }
                copy_commit();
            };
            unsigned live[4][2];  // of the tiles in the raw ring
#pragma unroll
            for (int i = 0; i < 4; ++i) live[i][0] = live[i][1] = 0;
#pragma unroll
            for (int t = 0; t < C::RAWS - 1; ++t) {
                issue(t);
                live[t][0] = live_of(id, t, 0), live[t][1] = live_of(id, t, 1);
            }
            for (int t = 0; t < n; ++t) {
                copy_wait<C::RAWS - 2>();
                const int stage = t % C::STAGES;
                if (t >= C::STAGES && !all_of(wide_wait(&bars->kv_empty[stage], (t / C::STAGES - 1) & 1, abort))) break;
                const uint8_t *raw = raws + t % C::RAWS * C::RAW;
                uint8_t *kv = smem + C::OFF_KV + stage * 2 * C::HALF;
                if (scales) {
                    const float *sc = reinterpret_cast<const float *>(raw + 2 * kTok * C::RB);
                    float *ks = reinterpret_cast<float *>(smem + C::OFF_META + stage * C::META), *vs = ks + kTok;
                    const float v0 = sc[kTok + lane], v1 = sc[kTok + 32 + lane];
                    const int e = top_exponent(__reduce_max_sync(0xffffffffu, max(finite_bits(v0), finite_bits(v1))));
                    const int j0 = (t0 + t) * kTok - sq.ctx;
                    const bool own = j0 + kTok > alike;
                    if (!own) R = raised(R, e);
                    const float unit = own ? 1.0f : unit_of(R);
                    ks[lane] = sc[lane] * p.scale_log2, ks[32 + lane] = sc[32 + lane] * p.scale_log2;
                    vs[lane] = v0 * unit, vs[32 + lane] = v1 * unit;
                    if (lane == 0)
                        *reinterpret_cast<int4 *>(ks + 2 * kTok) =
                            make_int4(static_cast<int>(live[0][0]), static_cast<int>(live[0][1]), j0,
                                      own ? kOwnUnit + e : R);
                    ptx::mbar_arrive(&bars->kv_full[stage]);
                    issue(t + C::RAWS - 1);
                    live[C::RAWS - 1][0] = live_of(id, t + C::RAWS - 1, 0);
                    live[C::RAWS - 1][1] = live_of(id, t + C::RAWS - 1, 1);
#pragma unroll
                    for (int i = 0; i < C::RAWS - 1; ++i) live[i][0] = live[i + 1][0], live[i][1] = live[i + 1][1];
                    continue;
                }
                // this thread's own chunks, from codes to fp16: K's, then V's (loads first,
                // which the compiler cannot move over the stores)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    uint4 w4[PER];
#pragma unroll
                    for (int j = 0; j < PER; ++j)
                        if (CHUNKS % kLoaders == 0 || lt + j * kLoaders < CHUNKS)
                            w4[j] = *reinterpret_cast<const uint4 *>(raw + v * kTok * C::RB + (lt + j * kLoaders) * 16);
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        if (CHUNKS % kLoaders != 0 && lt + j * kLoaders >= CHUNKS) break;
                        const int token = tok0 + j * TSTEP;
                        const uint32_t w[4] = {w4[j].x, w4[j].y, w4[j].z, w4[j].w};
                        uint8_t *dst = kv + v * C::HALF;
                        if constexpr (BITS == 8) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t a = (turn ? w[2 - 2 * i] : w[2 * i]) ^ 0x80808080u;
                                const uint32_t c = (turn ? w[3 - 2 * i] : w[2 * i + 1]) ^ 0x80808080u;
                                *reinterpret_cast<uint4 *>(dst + swizzled(token, 2 * ch + (i ^ turn), kTok)) =
                                    make_uint4(pair8(a, false), pair8(a, true), pair8(c, false), pair8(c, true));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                // pairs (0, 4), (1, 5), (2, 6), (3, 7) into channel order
                                const uint32_t x = turn ? w[i ^ 2] : w[i], y = x >> 8;
                                const uint32_t a = pair4(x, false), c = pair4(x, true), d = pair4(y, false),
                                               f = pair4(y, true);
                                *reinterpret_cast<uint4 *>(dst + swizzled(token, 4 * ch + (i ^ (2 * turn)), kTok)) =
                                    make_uint4(pick(a, c, 0x5410u), pick(d, f, 0x5410u), pick(a, c, 0x7632u),
                                               pick(d, f, 0x7632u));
                            }
                        }
                    }
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(&bars->kv_full[stage]);
                // the raw slot of the tile before this one is free: refill it
                issue(t + C::RAWS - 1);
            }
        }
        copy_wait<0>();
    } else {
        // ================================================ products
        // (descriptors are sums of a base and constants: in the low word, whose
        // address field does not overflow below 256 KB)
        const uint32_t base = ptx::smem_u32(smem);
        constexpr uint32_t id_s = ptx::idesc_f16_f32(128, kTok), id_o = ptx::idesc_f16_f32(128, D) | (1u << 16);
        const uint64_t dq = ptx::sw128_kmajor_desc(base), dk = ptx::sw128_kmajor_desc(base + C::OFF_KV);
        const uint64_t dv = mn_desc(base + C::OFF_KV + C::HALF, kTok * 128);
        const bool leader = elect_one();
        auto pv = [&](int t) {  // O += P V of tile t, both row blocks
            const int stage = t % C::STAGES, buf = t & 1;
            const uint64_t v = dv + static_cast<uint32_t>(stage * (2 * C::HALF / 16));
#pragma unroll
            for (int g = 0; g < QT; ++g) {
                if (!all_of(wide_wait(&bars->p_full[g][buf], (t >> 1) & 1, abort))) return false;
                ptx::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        mma_f16_ts(o_col(g), s_col(g, buf) + 8 * k, v + k * (2048 / 16), id_o);
                    ptx::mma_commit(&bars->pv_done[g]);
                    if (g == QT - 1) ptx::mma_commit(&bars->kv_empty[stage]);
                }
            }
            return true;
        };
        bool alive = n == 0 || all_of(wide_wait(&bars->q_full, 0, abort));
        for (int t = 0; t < n && alive; ++t) {
            const int stage = t % C::STAGES, buf = t & 1;
            alive = all_of(wide_wait(&bars->kv_full[stage], (t / C::STAGES) & 1, abort));
            if (!alive) break;
            ptx::tc_fence_after();
            if (leader) {
                const uint64_t k = dk + static_cast<uint32_t>(stage * (2 * C::HALF / 16));
#pragma unroll
                for (int g = 0; g < QT; ++g) {
#pragma unroll
                    for (int i = 0; i < C::STEPS; ++i)
                        ptx::mma_f16(s_col(g, buf), dq + (g * (128 * D * 2) + i / 4 * 16384 + i % 4 * 32) / 16,
                                     k + (i / 4 * (kTok * 128) + i % 4 * 32) / 16, id_s, i > 0);
                    ptx::mma_commit(&bars->s_full[g][buf]);
                }
            }
            if (t > 0) alive = pv(t - 1);
            if (!alive) break;
        }
        if (alive && n > 0) pv(n - 1);
        // whatever was issued has to end before its memory is given back
        if (leader) ptx::mma_commit(&bars->drain);
        __syncwarp();
        int none = 0;
        wide_wait(&bars->drain, 0, &none);
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, C::ALLOC);
    }
}

template <class C>
quik_status run(const AttnParams &p, cudaStream_t stream) {
    void (*kernel)(AttnParams) = &tree_attention_wide_kernel<C>;
    if (!attribute_set_once(reinterpret_cast<const void *>(kernel), C::SMEM)) return QUIK_ERR_CUDA;
    kernel<<<dim3(p.splits * p.row_blocks, p.heads, p.sequences), C::THREADS, C::SMEM, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? QUIK_OK : QUIK_ERR_CUDA;
}

template <int BITS>
quik_status run_bits(const AttnParams &p, int head_dim, int blocks, cudaStream_t stream) {
    if (head_dim == 64)
        return blocks == 1 ? run<WideCfg<BITS, 64, 1>>(p, stream) : run<WideCfg<BITS, 64, 2>>(p, stream);
    return blocks == 1 ? run<WideCfg<BITS, 128, 1>>(p, stream) : run<WideCfg<BITS, 128, 2>>(p, stream);
}

}  // namespace

quik_status launch_attention_wide(const AttnParams &p, int kv_type, int head_dim, int blocks,
                                  cudaStream_t stream) {
    if (kv_type == QUIK_KV_INT4) return run_bits<4>(p, head_dim, blocks, stream);
    if (kv_type == QUIK_KV_INT8) return run_bits<8>(p, head_dim, blocks, stream);
    return run_bits<16>(p, head_dim, blocks, stream);
}

unsigned int take_wide_errors(unsigned int *waits) {
    unsigned int word = 0, w = 0;
    if (cudaMemcpyFromSymbol(&word, g_attn_bad_index, sizeof(word)) != cudaSuccess) return 0;
    if (cudaMemcpyFromSymbol(&w, g_wide_waits, sizeof(w)) != cudaSuccess) return 0;
    *waits = counter_increase(kCounterWideWaits, w);
    return counter_increase(kCounterWidePage, word);
}

}  // namespace quik
