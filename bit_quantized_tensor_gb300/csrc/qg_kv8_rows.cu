// Attention over the paged 8-bit cache (kv8_common.cuh): many query rows a sequence, on tcgen05.
//
// The mathematics is that of the kernel for few rows: codes as exact fp16 operands, a page's
// scales outside the products, weights 2^(x + log2 sv - M + 9) in fp16.  With
//   t_j = raw_j c_b + l_b,   c_b = factor sk_b,  l_b = log2 sv_b      (b: j's 16 tokens)
// a weight is one fused multiply-add and one 2^x, like a softmax without scales.
//
// A CTA takes 256 rows (two tiles of 128: the heads that share a key head, times tokens) of a
// sequence and key head, against its tokens 128 at a time:
//   warps 0-3   softmax of tile 0, thread = row (its lane of tensor memory)
//   warps 4-7   softmax of tile 1
//   warps 8-11  codes of K and V to fp16 in shared memory
//   warp 12     MMA issuer, owner of the tensor memory
// S (128 x 128 fp32) of either tile lies in tensor memory, its weights (fp16) over its first half,
// from where they are the A operand of the product with V; O (128 x D fp32) beside it.  One
// tile's products run while the other's weights are made.  Both K and V lie in shared memory as
// tokens by 64 values (128-byte swizzle), which is K's K-major and V's MN-major form, so they are
// converted alike.  A row's sums are rescaled, in tensor memory, only when its maximum grows by 2^6.
//
// Measured: 623 us, 980 TFLOP/s for 4 prompts of 1392 to 2048 tokens, 32 heads of 128 values on 8 key
// heads, over 3058 to 8192 tokens, half the rate of the tensor cores.  What a step takes, about 4000
// cycles, is the chain scores -> weights -> product of a tile: 2000 for the weights, 560 for each product
// and 100 to 200 for each of the barriers between them.  So a softmax thread keeps half of its 128 scores
// between the maximum and the weights and has the next ones on their way while it works.  Scores of 64
// tokens at a time, made while the last 64 are weighed, leave no softmax waiting but take 718 us: a
// product with 64 columns keeps the tensor cores as long as one with 128.  The 13 warps hold a thread to 128
// registers, of which it spills 52 to 92 bytes; two threads a row, with an equal share each, spill more.
#include <cuda.h>

#include "kv8_attn.cuh"
#include "norm_common.cuh"
#include "qg_gemm_host.h"
#include "tc_issue.cuh"

namespace qg {

constexpr int kRowsSoftmaxWarps = 8, kRowsCodeWarps = 4, kRowsMmaWarp = 12;
constexpr int kRowsThreads = 32 * (kRowsMmaWarp + 1);
constexpr int kRowsTile = 128;   // rows of a tile, tokens of a step
constexpr int kSiteRowsK = 421, kSiteRowsV = 422, kSiteRowsS = 423, kSiteRowsP = 424, kSiteRowsPv = 425,
              kSiteRowsFree = 426, kSiteRowsQ = 427, kSiteRowsDrain = 428, kSiteRowsRaw = 429;

template <int D>
struct RowsCfg {
    static constexpr int BLOCKS = D / 64;                  // 128-byte columns of a tile
    static constexpr int TILE_BYTES = 128 * 2 * D;         // 128 rows of fp16
    static constexpr int STAGES = 2;                       // of K and of V
    static constexpr int RING = 2 * TILE_BYTES;            // after the two tiles of Q
    static constexpr int RAW = RING + 2 * STAGES * TILE_BYTES;
    static constexpr int RAW_SLOTS = 2, RAW_BYTES = 32 * D;   // a warp's 32 tokens of K or V on their way
    static constexpr int BARS = RAW + kRowsCodeWarps * RAW_SLOTS * RAW_BYTES;
    // at least half an SM's, so that no two CTAs meet on one (each takes all tensor memory)
    static constexpr int SMEM = BARS + 512 + 1024 > 117760 ? BARS + 512 + 1024 : 117760;
    static constexpr uint32_t O_COL = 256;                 // S of tile t at 128 t, O at 256 + D t
    static constexpr uint32_t IDESC_S = make_idesc(0, 0, 128, 128);
    static constexpr uint32_t IDESC_O = make_idesc(0, 0, 128, D) | (1u << 16);  // B is MN-major
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(2 * SMEM > 233472, "one CTA an SM");
};

// A from tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t idesc, uint32_t accumulate,
                                       uint32_t elected) {
    asm volatile(
        "{\n.reg .pred p, q;\n.reg .b64 db;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
        "mov.b64 db, {%2, %6};\n"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}" ::"r"(d),
        "r"(a), "r"(blo), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kTileHi)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Units of a sequence: key heads times pairs of row tiles, of which those of the last rows see
// most.  How many take at least `steps` steps of 128 tokens:
template <bool SOME>  // only those of sequences that come here
__device__ __forceinline__ int64_t rows_units(const AttnParams& p, int b, int steps) {
    const Kv8Seq s = kv8_seq(p.bt, p.c, b);
    const int64_t rows = static_cast<int64_t>(s.n) * p.group, pairs = (rows + 2 * kRowsTile - 1) / (2 * kRowsTile);
    if (SOME && rows < p.from) return 0;
    int64_t from = 0;  // first pair of tiles
    if (steps > 0) {
        const int64_t tokens = static_cast<int64_t>(steps - 1) * kRowsTile;  // to see more than these
        if (s.len <= tokens) return 0;
        if (p.causal) {
            const int64_t row = (tokens - s.first) * p.group;  // the first row that does
            if (row >= rows) return 0;
            from = row > 0 ? row / (2 * kRowsTile) : 0;
        }
    }
    return p.c.heads * (pairs - from);
}
__device__ __forceinline__ int64_t rows_sum(int64_t v, int64_t* mem) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();  // `mem` may still be read
    if ((threadIdx.x & 31) == 0) mem[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kRowsThreads / 32; ++w) v += mem[w];
    return v;
}
// The u-th longest unit: its sequence, which of those of its length, and its steps; b = B
// without one.  Long units first leaves the SMs done together: 4 prompts of 1392 to 2048 tokens
// over 3058 to 8192 take 251 steps where their own order took 285 (245: all alike).
struct RowsPlace {
    int b, steps;
    int64_t at;
};
template <bool SOME>
__device__ __forceinline__ RowsPlace rows_find(const AttnParams& p, int64_t u, int64_t* mem) {
    auto at_least = [&](int steps) {
        int64_t mine = 0;
        for (int b = threadIdx.x; b < p.bt.B; b += kRowsThreads) mine += rows_units<SOME>(p, b, steps);
        return rows_sum(mine, mem);
    };
    if (at_least(0) <= u) return {p.bt.B, 0, 0};
    // the most steps that more than u units take at least
    int lo = 0, hi = static_cast<int>(((static_cast<int64_t>(p.c.table_cols) << p.c.page_log2) + kRowsTile - 1) / kRowsTile) + 1;
    int64_t longer = 0;  // units of more steps than `lo`
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        const int64_t n = at_least(mid);
        if (n > u) {
            lo = mid;
        } else {
            hi = mid;
            longer = n;
        }
    }
    const Kv8Place at = kv8_find<kRowsThreads>(p.bt.B, u - longer, 0, mem, [&](int b) {
        return rows_units<SOME>(p, b, lo) - rows_units<SOME>(p, b, lo + 1);
    });
    return {at.b, lo, at.at};
}

// The forms of the kernel: of all sequences, of those of p.from rows and more, and of these with a unit's
// steps shared out to p.splits CTAs.  (What the second asks ahead of its loop costs the first 4% by
// the registers it leaves: 573 us of 4 prompts of 2048 tokens became 596.)
// With fewer units than SMs the last form's CTAs leave fp32 sums that a second kernel joins: which rows
// a unit has, left for it, and a CTA's sums, 256 rows of O, M and the denominator.
enum RowsForm { kWhole, kSome, kSplit };
struct alignas(16) RowsUnit {
    int64_t row0;                 // the sequence's first row of Q
    int head, first, rows, cut;   // rows: 0 without a unit
    int blind;                    // the sequence's first so many rows see no token
};
constexpr int kRowsParts = 304;   // CTAs that may have sums to join
constexpr int kRowsSplits = 32;   // of a unit
template <int D>
__device__ __forceinline__ float* rows_part(const AttnParams& p, int64_t cta) {
    return reinterpret_cast<float*>(reinterpret_cast<RowsUnit*>(p.part) + kRowsParts) + cta * (2 * kRowsTile) * (D + 4);
}

template <class T, int D, int FORM>
__global__ void __launch_bounds__(kRowsThreads, 1) k_kv8_attention_rows(const AttnParams p) {
    using Cfg = RowsCfg<D>;
    constexpr int TILE = kRowsTile;
    constexpr bool SPLIT = FORM == kSplit;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    __shared__ int64_t mem[kRowsThreads / 32 + 2];
    // a step's 8 blocks' sk and log2 sv, and the next step's, for each softmax warp
    __shared__ float2 scales[kRowsSoftmaxWarps][2][8];
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + Cfg::BARS);
    const uint32_t bar0 = smem_u32(bars), smem0 = smem_u32(smem);
    auto k_full = [&](int s) { return bar0 + 8u * s; };
    auto k_free = [&](int s) { return bar0 + 16u + 8u * s; };
    auto v_full = [&](int s) { return bar0 + 32u + 8u * s; };
    auto v_free = [&](int s) { return bar0 + 48u + 8u * s; };
    auto s_full = [&](int t) { return bar0 + 64u + 8u * t; };   // scores of tile t
    auto p_full = [&](int t) { return bar0 + 80u + 8u * t; };   // its weights
    auto pv_done = [&](int t) { return bar0 + 96u + 8u * t; };  // its product with V
    const uint32_t q_full = bar0 + 112u, drain = bar0 + 120u;
    uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + 16);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full(i), kRowsCodeWarps);
            mbar_init(k_free(i), 1);
            mbar_init(v_full(i), kRowsCodeWarps);
            mbar_init(v_free(i), 1);
            mbar_init(s_full(i), 1);
            mbar_init(p_full(i), 4);
            mbar_init(pv_done(i), 1);
        }
        mbar_init(q_full, kRowsSoftmaxWarps);
        mbar_init(drain, 1);
        for (int i = 0; i < kRowsCodeWarps * Cfg::RAW_SLOTS; ++i) mbar_init(bar0 + 144u + 8u * i, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait_prior_grid();
    fence_proxy_async_global();  // the cache may have been written just before, with ordinary stores
    const int unit_no = SPLIT ? blockIdx.x / p.splits : blockIdx.x, split = SPLIT ? blockIdx.x - unit_no * p.splits : 0;
    const RowsPlace at = rows_find<FORM != kWhole>(p, unit_no, mem);
    if (at.b >= p.bt.B) {  // more CTAs than units; no tensor memory is held yet
        if (SPLIT && split == 0 && threadIdx.x == 0) reinterpret_cast<RowsUnit*>(p.part)[unit_no].rows = 0;
        return;
    }
    if (warp == kRowsMmaWarp) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before the tensor memory is held: the next kernel may take its own and then wait for this one
    pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);

    // the unit: among its sequence's of this length, which are consecutive pairs of tiles
    const Kv8Seq seq = kv8_seq(p.bt, p.c, at.b);
    const int heads = p.c.heads, all_rows = seq.n * p.group;
    const int head = static_cast<int>(at.at % heads);
    const int pairs = (all_rows + 2 * TILE - 1) / (2 * TILE);
    const int longer = static_cast<int>(rows_units<false>(p, at.b, at.steps + 1) / heads);
    const int row0 = (pairs - 1 - longer - static_cast<int>(at.at / heads)) * 2 * TILE;
    auto seen_by = [&](int row) {
        const int64_t n = p.causal ? seq.first + row / p.group + 1 : seq.len;
        return row >= all_rows || n < 0 ? 0 : n < seq.len ? static_cast<int>(n) : seq.len;
    };
    // steps of 128 tokens that either tile sees
    int steps[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = row0 + t * TILE, last = min(all_rows, first + TILE) - 1;
        steps[t] = first < all_rows ? (seen_by(last) + TILE - 1) / TILE : 0;
    }
    // this CTA's share of them, `base` the first
    int most = max(steps[0], steps[1]), base = 0;
    if constexpr (SPLIT) {
        base = static_cast<int>(static_cast<int64_t>(most) * split / p.splits);
        most = static_cast<int>(static_cast<int64_t>(most) * (split + 1) / p.splits) - base;
#pragma unroll
        for (int t = 0; t < 2; ++t) steps[t] = max(0, min(steps[t] - base, most));
        if (split == 0 && threadIdx.x == 0) {
            const int64_t ahead = p.causal && seq.first < 0 ? -seq.first * p.group : 0;
            const int blind = seq.len == 0 || ahead > all_rows ? all_rows : static_cast<int>(ahead);
            reinterpret_cast<RowsUnit*>(p.part)[unit_no] = {seq.row0, head, row0, all_rows, seq.cut, blind};
        }
    }
    const int page_log2 = p.c.page_log2;
    const int tokens = max(seen_by(min(all_rows, row0 + TILE) - 1), seen_by(min(all_rows, row0 + 2 * TILE) - 1));
    // page * heads + head of a 16-token block, -1 without a page or behind what is seen
    auto unit_of = [&](int block) {
        if (16 * block >= tokens) return -1;
        const int page = kv8_page(p.c, at.b, (16 * block) >> page_log2);
        return page < 0 ? -1 : page * heads + head;
    };
    const float nan = __uint_as_float(0x7fc00000u);

    if (warp < kRowsSoftmaxWarps) {
        // ------------------------------------------------ queries, softmax, result of a row
        const int t = warp >> 2, r = (warp & 3) * 32 + lane, row = row0 + t * TILE + r;
        const uint32_t quad = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_at = quad + 128u * t, o_at = quad + Cfg::O_COL + D * t;
        float factor = 0.f;
        {
            const bool in = row < all_rows;
            const T* q = static_cast<const T*>(p.Q) + (seq.row0 + row / p.group) * p.ldq +
                         (head * p.group + row % p.group) * D;
            uint32_t bits = 0;
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
                float f[8];
                load_some<T, 8>(q + 8 * i, in ? 8 : 0, p.q_align == 16, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) bits = max(bits, abs_bits(f[k]));
            }
            const RowPower power = row_power(bits);
            // the factor of a score is not negative: the scale's sign goes into the queries
            const float up = p.scale_log2 < 0.f ? -power.up : power.up;
            factor = power.down * fabsf(p.scale_log2);
            uint8_t* const to = smem + t * Cfg::TILE_BYTES + r * 128;
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
                float f[8];
                load_some<T, 8>(q + 8 * i, in ? 8 : 0, p.q_align == 16, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] *= up;
                *reinterpret_cast<uint4*>(to + (i >> 3) * 16384 + (((i & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack2<__half>(f[0], f[1]), pack2<__half>(f[2], f[3]), pack2<__half>(f[4], f[5]),
                               pack2<__half>(f[6], f[7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        // a row that is not there sees what the last one does, for its warp to take the short way
        const int sees = seen_by(min(row, all_rows - 1)) - base * TILE, mine = steps[t];
        // scales of a step's 8 blocks, one a lane: the page three steps ahead, its scales two, what
        // they come to one, so that no load is waited for
        auto page_of = [&](int step) {
            const int block = 8 * (base + step) + lane, col = (16 * block) >> page_log2;
            return lane < 8 && step < mine && 16 * block < tokens && col < p.c.table_cols
                       ? p.c.table[static_cast<int64_t>(at.b) * p.c.table_cols + col]
                       : -1;
        };
        auto scales_of = [&](int page) {
            const int unit = page * heads + head;
            return page >= 0 && page < p.c.pages ? make_float2(p.c.ks[unit], p.c.vs[unit]) : make_float2(nan, nan);
        };
        auto keep = [&](int step, float2 v) {
            if (lane < 8) scales[warp][step & 1][lane] = make_float2(v.x, page_log2_of(v.y));
            __syncwarp();
        };
        keep(0, scales_of(page_of(0)));
        float2 raw = scales_of(page_of(1));
        int page = page_of(2);
        float M = neg_inf(), den = 0.f;
        bool ok = true;
        for (int step = 0; step < mine; ++step) {
            keep(step + 1, raw);
            raw = scales_of(page);
            page = page_of(step + 3);
            const float2* const sc = scales[warp][step & 1];
            const int left = sees - step * TILE;  // of the step's tokens
            const bool whole = __all_sync(0xffffffffu, left >= TILE);
            if (!__all_sync(0xffffffffu, bounded_wait(s_full(t), step & 1, abort_flag, p.ctl, kSiteRowsS))) {
                ok = false;
                break;
            }
            tc_fence_after();
            // scores 32 at a time; the last two quarters first, and again for their weights
            uint32_t xa[32], xb[32];
            float top = neg_inf(), least = -neg_inf();  // the greatest of the step, the least of its blocks' greatest
            auto maximum = [&](auto all, const uint32_t(&v)[32], int ch) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int b = 2 * ch + h, o = 16 * h;
                    const float2 sl = sc[b];
                    const float c = factor * sl.x;
                    if constexpr (decltype(all)::value) {
                        float m[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            m[i] = max3(__uint_as_float(v[o + 3 * i]), __uint_as_float(v[o + 3 * i + 1]),
                                        __uint_as_float(v[o + 3 * i + 2]));
                        const float m4 = max3(__uint_as_float(v[o + 12]), __uint_as_float(v[o + 13]),
                                              __uint_as_float(v[o + 14]));
                        m[0] = max3(m[0], m[1], __uint_as_float(v[o + 15]));
                        m[2] = max3(m[2], m[3], m4);
                        const float t = fmaf(fmaxf(m[0], m[2]), c, sl.y);
                        top = fmaxf(top, t);
                        least = fminf(least, t);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (16 * b + i < left) top = fmaxf(top, fmaf(__uint_as_float(v[o + i]), c, sl.y));
                    }
                }
            };
            // no use of a load's registers moves ahead of its wait
            auto landed = [&](uint32_t(&v)[32]) {
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(v[i]));
            };
            auto maxima = [&](auto all) {
                tmem_ld_32x32b_x32(s_at + 64, xa);
                tmem_ld_32x32b_x32(s_at + 96, xb);
                landed(xa);
                landed(xb);
                maximum(all, xa, 2);
                tmem_ld_32x32b_x32(s_at, xa);
                maximum(all, xb, 3);
                tmem_ld_32x32b_x32(s_at + 32, xb);
                landed(xa);
                landed(xb);
                maximum(all, xa, 0);
                maximum(all, xb, 1);
            };
            if (whole)
                maxima(std::true_type{});
            else
                maxima(std::false_type{});
            // O is at rest: this step's scores were issued behind the last step's product with V
            if (__any_sync(0xffffffffu, top > M + kLazy)) {
                const float m = fmaxf(M, top);
                const float half = M == neg_inf() ? 0.f : exp2_fast(0.5f * (M - m)), f = half * half;
                M = m;
                den = den * half * half;
                if (step) {
#pragma unroll 1
                    for (int d = 0; d < D; d += 16) {
                        uint32_t y[16];
                        tmem_ld_32x32b_x16(o_at + d, y);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                        tmem_st_x16(o_at + d, y);
                    }
                }
            }
            const float base = weight_base(M);
            auto weights = [&](auto all, const uint32_t(&x)[32], int ch) {
                uint32_t w[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int b = 2 * ch + h;
                    const float2 sl = sc[b];
                    const float c = factor * sl.x, l = sl.y - base, isv = exp2_fast(kDenPower - sl.y);
                    const uint64_t cc = two(c, c), ll = two(l, l);
                    uint64_t sum = two(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int k = 16 * h + 2 * i;
                        float2 e = both(fma_two(two(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), cc, ll));
                        if constexpr (!decltype(all)::value) {
                            if (32 * ch + k >= left) e.x = neg_inf();
                            if (32 * ch + k + 1 >= left) e.y = neg_inf();
                        }
                        e.x = exp2_fast(e.x);
                        e.y = exp2_fast(e.y);
                        sum = add_two(sum, two(e.x, e.y));
                        w[8 * h + i] = pack2<__half>(e.x, e.y);
                    }
                    const float2 s2 = both(sum);
                    const float s = s2.x + s2.y;
                    if constexpr (decltype(all)::value) {
                        den = fmaf(s, isv, den);
                    } else {
                        // not the low ones, nor 0 times a NaN of tokens not seen
                        const bool low = s < kLowWeight;
                        if (!low) den = fmaf(s, isv, den);
                        if (__any_sync(0xffffffffu, low && 16 * b < left)) {
                            float d = 0.f;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (16 * b + i < left) d += exp2_fast(fmaf(__uint_as_float(x[16 * h + i]), c, kDenPower - base));
                            if (low) den += d;
                        }
                    }
                }
                tmem_st_x16(s_at + 16 * ch, w);  // over scores that have been read
            };
            auto all_weights = [&](auto all) {
                weights(all, xa, 0);
                tmem_ld_32x32b_x32(s_at + 64, xa);
                weights(all, xb, 1);
                landed(xa);
                tmem_ld_32x32b_x32(s_at + 96, xb);
                weights(all, xa, 2);
                landed(xb);
                weights(all, xb, 3);
            };
            if (whole && !__any_sync(0xffffffffu, least < base - 99.f))
                all_weights(std::true_type{});
            else
                all_weights(std::false_type{});
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(t));
        }
        if (ok && mine)
            ok = __all_sync(0xffffffffu, bounded_wait(pv_done(t), (mine - 1) & 1, abort_flag, p.ctl, kSiteRowsPv));
        tc_fence_after();
        if (ok) {
            float* const sums = SPLIT ? rows_part<D>(p, blockIdx.x) + (t * TILE + r) * (D + 4) : nullptr;
            T* out = static_cast<T*>(p.O) + (seq.row0 + row / p.group) * p.ldo + (head * p.group + row % p.group) * D;
            const bool sectors = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
            const float scale = kDenUnit / den;
            // a row that sees nothing is 0; without a sum, its scores are all -inf and their softmax 0 / 0
            const float none = seq.cut || sees > 0 ? nan : 0.f;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                uint32_t y[16];
                float f[16];
                if (mine) {
                    tmem_ld_32x32b_x16(o_at + d, y);
                    tmem_wait_ld();
                }
                if constexpr (SPLIT) {
                    if (row < all_rows) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *reinterpret_cast<uint4*>(sums + d + i) =
                                mine ? make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]) : make_uint4(0, 0, 0, 0);
                        if (d == 0) *reinterpret_cast<float2*>(sums + D) = make_float2(M, den);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        f[i] = seq.cut || den == 0.f ? none : __uint_as_float(y[i]) * scale;
                    if (row < all_rows) {
                        if (sectors)
                            store_sectors<T>(out + d, f);
                        else
                            store_some<T, 16>(out + d, 16, false, f);
                    }
                }
            }
        }
        tc_fence_before();
    } else if (warp < kRowsMmaWarp) {
        // ------------------------------------------------ codes to fp16
        // A warp takes 32 of a step's 128 tokens, of K and then of V.  Their bytes, 16 tokens in one
        // piece, come by bulk copies a step ahead into a ring of the warp's own; a pass ends in a
        // proxy fence, so it has to be a long one (16 tokens a pass: 1450 cycles each).
        constexpr int CH = D / 16, PASS = 32 / CH, N = 32 / PASS;  // 16-byte pieces of a token; tokens a pass; passes
        constexpr int SLOTS = Cfg::RAW_SLOTS;
        const uint32_t elected = elect_lane();
        const int chunk = lane % CH, tok0 = lane / CH, w = warp - kRowsSoftmaxWarps;
        const uint8_t* const raw = smem + Cfg::RAW + w * SLOTS * Cfg::RAW_BYTES;
        const uint32_t raw_u32 = smem_u32(raw);
        auto raw_full = [&](int slot) { return bar0 + 144u + 8u * (w * SLOTS + slot); };
        // page * heads + head of the warp's two blocks of 16 steps, one a lane
        auto fetch = [&](int step) {
            step += lane >> 1;
            return step < most ? unit_of(8 * (base + step) + 2 * w + (lane & 1)) : -1;
        };
        int now = fetch(0), next = fetch(16);
        // K (slot 0) or V (slot 1) of a step; only blocks that hold tokens
        auto copy = [&](int step, int units, int slot) {
            if (step >= most) return;
            const int u0 = __shfl_sync(0xffffffffu, units, 2 * (step & 15));
            const int u1 = __shfl_sync(0xffffffffu, units, 2 * (step & 15) + 1);
            const uint32_t bytes = (u0 >= 0 ? Cfg::RAW_BYTES / 2 : 0) + (u1 >= 0 ? Cfg::RAW_BYTES / 2 : 0);
            if (elected) {
                const int8_t* codes = slot ? p.c.vq : p.c.kq;
                const int token = (base + step) * TILE + 32 * w, mask = (1 << page_log2) - 1;
                mbar_arrive_expect_tx(raw_full(slot), bytes);
                const uint32_t to = raw_u32 + slot * Cfg::RAW_BYTES;
                if (u0 >= 0)
                    bulk_copy_g2s(to, codes + ((static_cast<int64_t>(u0) << page_log2) + (token & mask)) * D,
                                  Cfg::RAW_BYTES / 2, raw_full(slot));
                if (u1 >= 0)
                    bulk_copy_g2s(to + Cfg::RAW_BYTES / 2,
                                  codes + ((static_cast<int64_t>(u1) << page_log2) + ((token + 16) & mask)) * D,
                                  Cfg::RAW_BYTES / 2, raw_full(slot));
            }
            __syncwarp();
        };
        auto convert = [&](int step, int slot, int ahead) {
            const int s = step & 1;
            const bool in0 = __shfl_sync(0xffffffffu, now, 2 * (step & 15)) >= 0;
            const bool in1 = __shfl_sync(0xffffffffu, now, 2 * (step & 15) + 1) >= 0;
            if (!__all_sync(0xffffffffu, bounded_wait(raw_full(slot), step & 1, abort_flag, p.ctl, kSiteRowsRaw)))
                return false;
            uint4 from[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                from[j] = *reinterpret_cast<const uint4*>(raw + slot * Cfg::RAW_BYTES + (tok0 + j * PASS) * D + 16 * chunk);
                if (!(j < N / 2 ? in0 : in1)) from[j] = make_uint4(0, 0, 0, 0);  // zeros where there is no token
            }
            __syncwarp();  // all have read the slot
            copy(step + 1, ahead, slot);
            if (!__all_sync(0xffffffffu, bounded_wait(slot ? v_free(s) : k_free(s), ((step >> 1) & 1) ^ 1, abort_flag, p.ctl,
                                                      kSiteRowsFree)))
                return false;
            uint8_t* const to = smem + Cfg::RING + (2 * slot + s) * Cfg::TILE_BYTES + (chunk >> 2) * 16384 + w * 4096;
            const int odd = (chunk >> 2) & 1;  // the second columns' lanes store their halves in turn, not to meet in a bank
            const int c0 = 2 * (chunk & 3);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int tok = tok0 + j * PASS;
                uint32_t h[8];
                s8_to_f16(from[j].x, h[0], h[1]);
                s8_to_f16(from[j].y, h[2], h[3]);
                s8_to_f16(from[j].z, h[4], h[5]);
                s8_to_f16(from[j].w, h[6], h[7]);
                const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), b = make_uint4(h[4], h[5], h[6], h[7]);
                uint8_t* const at_row = to + tok * 128;
                *reinterpret_cast<uint4*>(at_row + (((c0 + odd) ^ (tok & 7)) << 4)) = odd ? b : a;
                *reinterpret_cast<uint4*>(at_row + (((c0 + 1 - odd) ^ (tok & 7)) << 4)) = odd ? a : b;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (elected) mbar_arrive(slot ? v_full(s) : k_full(s));
            return true;
        };
        copy(0, now, 0);
        copy(0, now, 1);
        bool ok = true;
        for (int step = 0; ok && step < most; ++step) {
            const int ahead = (step & 15) == 15 ? next : now;  // units of step + 1
            ok = convert(step, 0, ahead) && convert(step, 1, ahead);
            if ((step & 15) == 15) {
                now = next;
                next = fetch(step + 17);
            }
        }
        if (!ok && elected) {
            // copies may still be in flight: give them a fixed time to land
            const uint64_t start = global_timer_ns();
            while (global_timer_ns() - start < 1000000) {
            }
        }
    } else {
        // ------------------------------------------------ MMA issuer
        const uint32_t elected = elect_lane();
        auto wait = [&](uint32_t bar, uint32_t parity, int site) {
            return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag, p.ctl, site));
        };
        auto commit = [&](uint32_t bar) {
            if (elected) tc_commit(bar);
            __syncwarp();
        };
        // scores of tile t of a step: S = Q K^T
        auto scores = [&](int t, int step) {
            // descriptors as sums of 32-bit words: anything else is done in vector registers and moved
            const uint32_t q = tile_lo(smem0, 16) + t * (Cfg::TILE_BYTES / 16);
            const uint32_t k = tile_lo(smem0 + Cfg::RING, 16) + (step & 1) * (Cfg::TILE_BYTES / 16);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint32_t at_k = (i >> 2) * 1024u + (i & 3) * 2u;
                mma_ss(tmem + 128u * t, q + at_k, k + at_k, Cfg::IDESC_S, i > 0, elected);
            }
            commit(s_full(t));
        };
        auto values = [&](int t, int step) {
            const uint32_t v = tile_lo(smem0 + Cfg::RING + 2 * Cfg::TILE_BYTES, 16384) + (step & 1) * (Cfg::TILE_BYTES / 16);
#pragma unroll
            for (int i = 0; i < TILE / 16; ++i)
                mma_ts(tmem + Cfg::O_COL + D * t, tmem + 128u * t + 8u * i, v + 128u * i, Cfg::IDESC_O,
                       step > 0 || i > 0, elected);
            commit(pv_done(t));
        };
        bool ok = most == 0 || (wait(q_full, 0, kSiteRowsQ) && wait(k_full(0), 0, kSiteRowsK));
        if (ok && most) {
            tc_fence_after();
            if (steps[0]) scores(0, 0);
            if (steps[1]) scores(1, 0);
            commit(k_free(0));
        }
        for (int step = 0; ok && step < most; ++step) {
            const int s = step & 1;
            const uint32_t parity = (step >> 1) & 1;
            if (!(ok = wait(v_full(s), parity, kSiteRowsV))) break;
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (ok && step < steps[t]) {
                    if (!(ok = wait(p_full(t), step & 1, kSiteRowsP))) break;
                    tc_fence_after();
                    values(t, step);
                    if (t == 1 || step >= steps[1]) commit(v_free(s));
                }
                if (ok && step + 1 < steps[t]) {
                    if (!k_ready) ok = wait(k_full((step + 1) & 1), ((step + 1) >> 1) & 1, kSiteRowsK);
                    k_ready = true;
                    // the scores go where the weights lie that the product just issued reads
                    if (!ok || !(ok = wait(pv_done(t), step & 1, kSiteRowsPv))) break;
                    tc_fence_after();
                    scores(t, step + 1);
                    if (t == 1 || step + 1 >= steps[1]) commit(k_free((step + 1) & 1));
                }
            }
        }
        commit(drain);  // every MMA issued has completed before anything is released
        bounded_wait(drain, 0, nullptr, p.ctl, kSiteRowsDrain);
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kRowsMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// A warp a row, four rows a warp: the sums of the unit's CTAs, in their order.
constexpr int kRowsJoinThreads = 256, kRowsJoinRows = 4 * kRowsJoinThreads / 32;
template <class T, int D>
__global__ void __launch_bounds__(kRowsJoinThreads) k_kv8_attention_rows_join(const AttnParams p) {
    constexpr int E = D / 32;  // values a lane
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const RowsUnit u = reinterpret_cast<const RowsUnit*>(p.part)[blockIdx.x];
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < 4; ++i) {
        const int r = blockIdx.y * kRowsJoinRows + 4 * (threadIdx.x >> 5) + i, row = u.first + r;
        if (u.rows == 0 || row >= u.rows) return;
        const float* const sums = rows_part<D>(p, static_cast<int64_t>(blockIdx.x) * p.splits) + r * (D + 4);
        constexpr int64_t NEXT = 2 * kRowsTile * (D + 4);
        float2 top = make_float2(neg_inf(), 0.f);
        if (lane < p.splits) top = *reinterpret_cast<const float2*>(sums + lane * NEXT + D);
        float m = top.x;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float half = top.x == neg_inf() ? 0.f : exp2_fast(0.5f * (top.x - m)), weight = half * half;
        const float den = warp_sum(top.y * half * half);
        float o[E];
#pragma unroll
        for (int k = 0; k < E; ++k) o[k] = 0.f;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            alignas(16) float v[E];
            if constexpr (E == 4)
                *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(sums + s * NEXT + E * lane);
            else
                *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(sums + s * NEXT + E * lane);
            const float w = __shfl_sync(0xffffffffu, weight, s);
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = fmaf(v[k], w, o[k]);
        }
        const float scale = kDenUnit / den, none = u.cut || row >= u.blind ? __uint_as_float(0x7fc00000u) : 0.f;
        T* out = static_cast<T*>(p.O) + (u.row0 + row / p.group) * p.ldo + (u.head * p.group + row % p.group) * D + E * lane;
#pragma unroll
        for (int k = 0; k < E; ++k) out[k] = from_f32<T>(u.cut || den == 0.f ? none : o[k] * scale);
    }
}

size_t attention_rows_workspace(int64_t D) {
    return kRowsParts * (sizeof(RowsUnit) + sizeof(float) * 2 * kRowsTile * static_cast<size_t>(D + 4));
}

static int64_t table_steps(const AttnParams& p) {
    return ((static_cast<int64_t>(p.c.table_cols) << p.c.page_log2) + kRowsTile - 1) / kRowsTile;
}

// How many rows a sequence has to have for the kernel above; 1: all sequences go to it, INT32_MAX:
// none.  64 rows a sequence take it 97 us (8 sequences of 8192 tokens, 8 heads of 128 values) where
// the kernel for few rows takes 106, 32 rows 97 and 68.  With fewer units, whose CTAs' sums have to be
// joined, twice as many: 64 rows of one sequence of 32768 take it 98 and the other 64, 128 rows 101
// and 99, 256 rows 114 and 175.
// A batch may hold prompts next to single tokens, which the host cannot see.  On average few rows a
// sequence: both kernels run once what is over one token a sequence makes four units (512 tokens
// next to 63 single ones over 8192 tokens: 492 us by the kernel for few rows alone, 284 by both; 5 us
// more for a batch of equals).  On average many: all but one sequence may be single tokens, each of
// which then keeps a CTA a key head busy for all of its steps.  Both run where that could be 16384 steps
// (108 on each SM, 220 us).  Of 64 sequences of 8 key heads over 8192 tokens 1024 tokens next to 63 single
// ones take 282 us and 414 by this kernel alone, 4096 596 and 678, but 16 tokens of each sequence 333 and
// 308.  4096 tokens next to 15 single ones could be 7680 steps and take 520 us by both, 493 by this
// kernel; with 65536 tokens for each of the 15, 540 and 943.
int attention_rows_from(const AttnParams& p) {
    if (p.c.D == 256) return INT32_MAX;
    const int64_t rows = static_cast<int64_t>(p.bt.rows) * p.group, B = p.bt.B;
    const int from = B * p.c.heads < 64 ? 128 : 64;
    if (rows >= B * from) return (B - 1) * p.c.heads * table_steps(p) < 16384 ? 1 : from;
    return B > 1 && (p.bt.rows - B) * p.group >= 8 * kRowsTile ? from : INT32_MAX;
}

template <class T, int D>
static int launch_rows(AttnParams p, int dev, cudaStream_t s) {
    // units at most, and about as many as there are
    const int64_t rows = static_cast<int64_t>(p.bt.rows) * p.group, holds = p.from > 1 ? rows / p.from : p.bt.rows;
    const int64_t seqs = p.bt.B < holds ? p.bt.B : holds;
    const int64_t units = ((rows - seqs) / (2 * kRowsTile) + seqs) * p.c.heads;
    if (units > INT32_MAX) return QG_ERR_INVALID_ARG;
    const int64_t alike = (rows + seqs * 2 * kRowsTile - 1) / (seqs * 2 * kRowsTile) * seqs * p.c.heads;
    // CTAs for a unit: as many as there are SMs for, each with 4 steps at least of the longest.  A lone
    // sequence's 128 rows over 32768 tokens of 8 heads: 440 us by 8 CTAs, 101 by 152.
    const int64_t steps = table_steps(p);
    int64_t splits = num_sms(dev) / alike;
    splits = splits > kRowsParts / units ? kRowsParts / units : splits;
    splits = splits > kRowsSplits ? kRowsSplits : splits;
    splits = splits > steps / 4 ? steps / 4 : splits;
    p.splits = splits < 1 ? 1 : static_cast<int>(splits);
    struct Whole;
    struct Some;
    struct Split;
    const dim3 grid(static_cast<unsigned>(units * p.splits));
    auto launch = [&](auto kernel, int raised) {
        return raised ? raised : launch_serialized(kernel, grid, kRowsThreads, RowsCfg<D>::SMEM, 1, s, p);
    };
    if (p.splits == 1 && p.from == 1)
        return launch(k_kv8_attention_rows<T, D, kWhole>, raise_smem<Whole>(k_kv8_attention_rows<T, D, kWhole>));
    if (p.splits == 1)
        return launch(k_kv8_attention_rows<T, D, kSome>, raise_smem<Some>(k_kv8_attention_rows<T, D, kSome>));
    const int rc = launch(k_kv8_attention_rows<T, D, kSplit>, raise_smem<Split>(k_kv8_attention_rows<T, D, kSplit>));
    if (rc) return rc;
    return launch_serialized(k_kv8_attention_rows_join<T, D>,
                             dim3(static_cast<unsigned>(units), 2 * kRowsTile / kRowsJoinRows), kRowsJoinThreads, 0, 1, s,
                             p);
}

int attention_rows(int dtype, const AttnParams& p, int dev, cudaStream_t s) {
    if (dtype == QG_F16) return p.c.D == 64 ? launch_rows<__half, 64>(p, dev, s) : launch_rows<__half, 128>(p, dev, s);
    return p.c.D == 64 ? launch_rows<__nv_bfloat16, 64>(p, dev, s) : launch_rows<__nv_bfloat16, 128>(p, dev, s);
}

#define QG_ROWS_FORM_BUDGET(T, NAME, D, FORM, FORM_NAME)                                                 \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention_rows<" NAME "," #D "," FORM_NAME ">",                         \
                           (reinterpret_cast<const void*>(k_kv8_attention_rows<T, D, FORM>)),            \
                           kRowsThreads, RowsCfg<D>::SMEM, 512, 1, 1)
#define QG_ROWS_BUDGET(T, NAME, D)                                                                       \
    QG_ROWS_FORM_BUDGET(T, NAME, D, kWhole, "whole");                                                    \
    QG_ROWS_FORM_BUDGET(T, NAME, D, kSome, "some");                                                      \
    QG_ROWS_FORM_BUDGET(T, NAME, D, kSplit, "split");                                                    \
    QG_BLOCK_KERNEL_BUDGET("k_kv8_attention_rows_join<" NAME "," #D ">",                                 \
                           (reinterpret_cast<const void*>(k_kv8_attention_rows_join<T, D>)),             \
                           kRowsJoinThreads, 0, 0, 1, 1)
QG_ROWS_BUDGET(__half, "f16", 64);
QG_ROWS_BUDGET(__half, "f16", 128);
QG_ROWS_BUDGET(__nv_bfloat16, "bf16", 64);
QG_ROWS_BUDGET(__nv_bfloat16, "bf16", 128);

}  // namespace qg
