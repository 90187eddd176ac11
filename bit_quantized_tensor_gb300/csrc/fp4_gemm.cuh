// Product of two microscaled 4-bit operands on the block-scaled tensor cores:
//   Y[m][n] = alpha * sum_k (a[m][k] sa[m][k / B]) (b[n][k] sb[n][k / B]) + bias[n]
// with a, b e2m1 codes and sa, sb block scales (fp4_common.cuh), alpha the
// product of the tensor scales (fp4_alpha).  tcgen05.mma multiplies the codes, applies both
// block scales and accumulates in fp32 in tensor memory; each K step of 64
// needs the scales of its rows in tensor memory too, which tcgen05.cp brings
// there from shared memory in the layout that the packed scales already have.
#pragma once
#include <type_traits>

#include "fp4_common.cuh"
#include "qg_gemm_host.h"
#include "qg_ptx.cuh"

namespace qg {

// ------------------------------------------------ block-scaled instructions

// Instruction descriptor: B scale id (bits 4-5), e2m1 for A (7-9) and B
// (10-12), N / 8 (17-22), scale type (23: 0 = e4m3, 1 = e8m0), M / 16 (24-28),
// A scale id (29-30).  The id picks the first scale byte of a 32-bit column:
// a K step of 64 uses four (blocks of 16) or two (blocks of 32) of them.
template <int FMT>
__host__ __device__ constexpr uint32_t fp4_idesc(uint32_t m, uint32_t n, uint32_t scale_id) {
    return (scale_id << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) |
           ((FMT == kMx ? 1u : 0u) << 23) | ((m >> 4) << 24) | (scale_id << 29);
}

// The asynchronous instructions below are issued by whole warps with one
// elected lane's predicate, and never inside a branch on the lane: in
// convergent code the descriptors and addresses stay in uniform registers.
// Issued from inside `if (lane == 0)` every operand is moved there one by one,
// which was measured at 200 cycles an MMA and 52 a scale copy, whatever their
// size; like this an MMA of 256 x 256 x 64 takes its 128 cycles and the copies
// disappear behind it (12 copies and 4 MMAs: 534 cycles).
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}

// Shared-memory descriptors, of which only the low word (start address >> 4)
// differs: built as a 32-bit sum, since a 64-bit one costs dependent uniform
// instructions in front of every issue.  kRowsHi: rows of 128 bytes, 128-byte
// swizzle, 1024 bytes between groups of 8 rows; kScalesHi: a scale tile, 32 rows
// of 16 bytes, no swizzle, 128 bytes between groups of 8 rows; version 1.
constexpr uint32_t kRowsHi = (1024u >> 4) | (1u << 14) | (2u << 29), kScalesHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t rows_lo(uint32_t smem_addr) { return ((smem_addr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t scales_lo(uint32_t smem_addr) { return (smem_addr & 0x3FFFFu) >> 4; }

#define QG_FP4_MMA(GROUP, KIND)                                                                              \
    asm volatile("{\n.reg .pred p, q;\n.reg .b64 da, db;\nsetp.ne.b32 p, %6, 0;\nsetp.ne.b32 q, %7, 0;\n"   \
                 "mov.b64 da, {%1, %8};\nmov.b64 db, {%2, %8};\n"                                            \
                 "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %3, [%4], [%5], p;\n}" ::"r"( \
                     d_tmem),                                                                                \
                 "r"(alo), "r"(blo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(elected), "r"(kRowsHi) \
                 : "memory")

// PAIR: M = 256 across the two CTAs of a cluster, issued by the leader.
template <int FMT, bool PAIR>
__device__ __forceinline__ void fp4_mma(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate, uint32_t elected) {
    if constexpr (FMT == kNv && !PAIR)
        QG_FP4_MMA("1", "mxf4nvf4.block_scale.block16");
    else if constexpr (FMT == kNv)
        QG_FP4_MMA("2", "mxf4nvf4.block_scale.block16");
    else if constexpr (!PAIR)
        QG_FP4_MMA("1", "mxf4.block_scale.block32");
    else
        QG_FP4_MMA("2", "mxf4.block_scale.block32");
}

// One 512-byte scale tile from shared memory into four columns of tensor
// memory, repeated in each quarter of the lanes (PAIR: in both CTAs, each from
// its own shared memory).
#define QG_FP4_COPY(GROUP)                                                                                 \
    asm volatile("{\n.reg .pred q;\n.reg .b64 d;\nsetp.ne.b32 q, %2, 0;\nmov.b64 d, {%1, %3};\n"           \
                 "@q tcgen05.cp.cta_group::" GROUP ".32x128b.warpx4 [%0], d;\n}" ::"r"(tmem),               \
                 "r"(lo), "r"(elected), "r"(kScalesHi)                                                     \
                 : "memory")
template <bool PAIR>
__device__ __forceinline__ void fp4_copy_scales(uint32_t tmem, uint32_t lo, uint32_t elected) {
    if constexpr (PAIR)
        QG_FP4_COPY("2");
    else
        QG_FP4_COPY("1");
}

// tma_load_2d and tma_load_2d_pair of an elected lane.
__device__ __forceinline__ void fp4_load(uint32_t dst, const void* tmap, int32_t c0, int32_t c1, uint32_t bar,
                                         uint32_t elected) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %5, 0;\n"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(bar), "r"(elected)
        : "memory");
}
__device__ __forceinline__ void fp4_load_pair(uint32_t dst, const void* tmap, int32_t c0, int32_t c1,
                                              uint32_t cluster_bar, uint32_t elected) {
    asm volatile(
        "{\n.reg .pred q;\nsetp.ne.b32 q, %5, 0;\n"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];\n}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(cluster_bar), "r"(elected)
        : "memory");
}

// ------------------------------------------------ one CTA per tile
//
// The weights' rows are the 128 rows of the MMA and the tokens its NT columns,
// so that few tokens waste few columns and the weights, which are what a small
// batch has to read, move in whole 16 KB boxes.  Tiles of fewer than 128 tokens
// hold all tokens (M <= NT): scales start at a multiple of four columns of
// tensor memory, so a tile cannot begin inside 128 scale rows.  A cluster of S CTAs splits K:
// each CTA sends its fp32 sums of a column to the CTA that owns the column,
// which adds them up in rank order.
//   warp 4  TMA producer      warp 5  MMA issuer, owner of the tensor memory
//   warps 0-3  epilogue (their lane quarter of the accumulator); with QUANT
//              they first quantize the tokens' values of the CTA's K range into
//              the ring themselves, which spares a small batch a kernel
// With few tokens nothing but latency counts: the ring takes less than half an
// SM's shared memory, so that a call's CTAs can set up and fetch their weights
// while those of the call before it finish.  16 tokens of 4096 f16 values by
// 4096 rows of mx weights: 6.0 us a call in a chain, quantization included (9.0 MB,
// mostly weights that the L2 holds: 1.5 TB/s); 777 x 1001 x 2304: 10 us.
constexpr int kFp4Threads = 192;
constexpr int kFp4Bk = 256;  // K of a stage: one 128-byte swizzled row of codes

template <int FMT_, int NT_>
struct Fp4Cfg {
    static constexpr int FMT = FMT_, NT = NT_;
    static constexpr int ATOMS = FMT == kNv ? 4 : 2;            // scale tiles along K in a stage
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = NT * 128;
    static constexpr int S_BYTES = ATOMS * 512;                 // scales of 128 rows
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2 * S_BYTES;
    static constexpr int W_BYTES = A_BYTES + S_BYTES;           // of a stage, the weights' part
    static constexpr int STAGES = 4;
    static constexpr int BARRIER_BYTES = 256;
    static constexpr int JOIN_BYTES = NT * 128 * 4;             // sums from the cluster (S > 1)
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + BARRIER_BYTES + 1024;
    static constexpr int SMEM_JOIN_BYTES = SMEM_BYTES + JOIN_BYTES;
    static constexpr int SFA_COL = NT;                          // D at column 0
    static constexpr int SFB_COL = NT + 4 * ATOMS;
    static constexpr int COLS_USED = NT + 8 * ATOMS;
    static constexpr int TMEM_COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : 256;
    static_assert(NT % 16 == 0 && NT <= 128, "MMA columns");
    static_assert(COLS_USED <= TMEM_COLS, "tensor memory");
    static_assert(SMEM_JOIN_BYTES <= 232448, "shared memory");
    static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms of 1 KB");
};

struct Fp4Params {
    int M, N, K;         // tokens, weight rows, reduction
    int log_splits;      // 2^log_splits CTAs of a cluster share K (single CTAs)
    const float *ts_a, *ts_b;  // tensor scales of the tokens and the weights, or null
    const void* bias;    // N values of the output type, or null
    void* Y;
    int64_t ldy;
    int dtype;           // of Y and bias
    bool weights_ready;  // the weights were complete before the kernel ahead on the stream started
    const void* X;       // QUANT: the tokens' values
    int64_t ldx;
    bool x_aligned;
    Ctl ctl;
};

constexpr int kSiteFp4Empty = 301;
constexpr int kSiteFp4Full = 302;
constexpr int kSiteFp4Acc = 303;
constexpr int kSiteFp4Quant = 304;
constexpr int kSiteFp4Join = 305;

// The sums are multiplied by `first`, which is 1 where the product of the tensor
// scales is a normal fp32 number (alpha, `second`).  Where it is not, the result may
// still be one: a product below the normal range takes the larger scale first, one
// above it the smaller.
struct Fp4Alpha {
    float first, second;
};
__device__ __forceinline__ Fp4Alpha fp4_alpha(const Fp4Params& p) {
    const float a = p.ts_a ? *p.ts_a : 1.f, b = p.ts_b ? *p.ts_b : 1.f, ab = a * b;
    if (ab >= 0x1p-126f && ab <= 0x1.fffffep+127f) return {1.f, ab};
    return ab < 1.f ? Fp4Alpha{fmaxf(a, b), fminf(a, b)} : Fp4Alpha{fminf(a, b), fmaxf(a, b)};
}
// The first of the two, for sums that go on to fmaf(sum, second, bias): behind a branch,
// since 16 multiplications by 1 a step cost 0.15 us in 10 and 1.2 in 84.
template <int N>
__device__ __forceinline__ void fp4_first(float (&f)[N], const Fp4Alpha& alpha) {
    if (alpha.first != 1.f) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] *= alpha.first;
    }
}

__device__ __forceinline__ float typed_at(const void* v, int dtype, int64_t i) {
    if (dtype == QG_F16) return __half2float(static_cast<const __half*>(v)[i]);
    if (dtype == QG_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(v)[i]);
    return static_cast<const float*>(v)[i];
}
__device__ __forceinline__ void typed_store(void* v, int dtype, int64_t i, float x) {
    if (dtype == QG_F16)
        static_cast<__half*>(v)[i] = __float2half_rn(x);
    else if (dtype == QG_BF16)
        static_cast<__nv_bfloat16*>(v)[i] = __float2bfloat16_rn(x);
    else
        static_cast<float*>(v)[i] = x;
}

// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Waits, bounded, until `bar` has completed phase `parity`, whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, const Ctl& ctl,
                                          int site) {
    return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag, ctl, site));
}

// QUANT: the type of the tokens' values, or void with packed tokens.
template <class Cfg, class QUANT>
__global__ void __launch_bounds__(kFp4Threads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                    const Fp4Params p) {
    constexpr int NT = Cfg::NT, STAGES = Cfg::STAGES, FMT = Cfg::FMT;
    constexpr bool Q = !std::is_void<QUANT>::value;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    // per stage: weights' codes | tokens' codes | weights' scales | tokens' scales
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * Cfg::STAGE_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t acc_bar = bar0 + 8u * (2 * STAGES);
    const uint32_t join_bar = acc_bar + 8u;  // the cluster's sums of this CTA's columns have arrived
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    float* const join = reinterpret_cast<float*>(smem + STAGES * Cfg::STAGE_BYTES + Cfg::BARRIER_BYTES);
    const uint32_t ring0 = smem_u32(smem);
    auto a_smem = [&](int s) { return ring0 + static_cast<uint32_t>(s) * Cfg::STAGE_BYTES; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a cluster takes a tile; clusters along x take the rows of weights, of which there may
    // be more tiles than a grid's y or z counts
    const int splits = 1 << p.log_splits, split = static_cast<int>(blockIdx.x) & (splits - 1);
    const int n0 = static_cast<int>(blockIdx.x >> p.log_splits) * 128;
    const int m0 = static_cast<int>(blockIdx.y) * NT;
    const int num_kb = (p.K + kFp4Bk - 1) / kFp4Bk;
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * split / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (split + 1) / splits);
    const int cols = min(NT, p.M - m0);  // tokens of this tile
    const int per = (cols + splits - 1) / splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), Q ? 1 + 4 : 1);  // the producer, and the quantizing warps
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(acc_bar, 1);
        mbar_init(join_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        // column c belongs to CTA c / per, which gets its sums from every CTA
        if (splits > 1) mbar_arrive_expect_tx(join_bar, splits * max(0, min(cols - split * per, per)) * 512);
    }
    if (threadIdx.x == 128) {
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmSW);
        if constexpr (!Q) {
            tma_prefetch_desc(&tmX);
            tma_prefetch_desc(&tmSX);
        }
    }
    if (warp == 5) tmem_alloc(smem_u32(tmem_holder), Cfg::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (splits > 1) cluster_arrive();  // this CTA runs: its shared memory may be written (awaited below)
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);  // known to be uniform

    bool ok = true;
    // The bounded waits below start only when the previous kernel is done (they
    // must not count its time); the producer alone may run ahead of that.
    if (warp != 4) pdl_wait_prior_grid();
    if (warp == 4) {
        const uint32_t elected = elect_lane();
        const int tiles_k = static_cast<int>(fp4_col_tiles(FMT, p.K));
        auto arm = [&](int s) {
            if (elected) mbar_arrive_expect_tx(full_bar(s), Q ? Cfg::W_BYTES : Cfg::STAGE_BYTES);
            __syncwarp();
        };
        auto load_w = [&](int kb, int s) {
            fp4_load(a_smem(s), &tmW, kb * (kFp4Bk / 2), n0, full_bar(s), elected);
            fp4_load(a_smem(s) + Cfg::A_BYTES + Cfg::B_BYTES, &tmSW, 0, (n0 >> 7) * tiles_k + kb * Cfg::ATOMS,
                     full_bar(s), elected);
        };
        auto load_x = [&](int kb, int s) {
            if constexpr (!Q) {
                fp4_load(a_smem(s) + Cfg::A_BYTES, &tmX, kb * (kFp4Bk / 2), m0, full_bar(s), elected);
                fp4_load(a_smem(s) + Cfg::A_BYTES + Cfg::B_BYTES + Cfg::S_BYTES, &tmSX, 0,
                         (m0 >> 7) * tiles_k + kb * Cfg::ATOMS, full_bar(s), elected);
            }
        };
        // Weights that were complete before the previous kernel began may
        // be fetched while that kernel (which makes the tokens' codes) runs.
        const int ahead = min(kb1 - kb0, STAGES);
        if (!p.weights_ready) {
            pdl_wait_prior_grid();
            fence_proxy_async_global();
        }
        for (int i = 0; i < ahead; ++i) {
            arm(i);
            load_w(kb0 + i, i);
        }
        if (p.weights_ready) {
            pdl_wait_prior_grid();
            fence_proxy_async_global();
        }
        for (int i = 0; i < ahead; ++i) load_x(kb0 + i, i);
        Ring<STAGES> ps;
        for (int i = 0; i < ahead; ++i) ps.next();
        for (int kb = kb0 + ahead; kb < kb1; ++kb) {
            if (!warp_wait(empty_bar(ps.slot()), ps.parity() ^ 1u, abort_flag, p.ctl, kSiteFp4Empty)) break;
            arm(ps.slot());
            load_w(kb, ps.slot());
            load_x(kb, ps.slot());
            ps.next();
        }
    } else if (warp == 5) {
        const uint32_t elected = elect_lane();
        Ring<STAGES> ps;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(full_bar(ps.slot()), ps.parity(), abort_flag, p.ctl, kSiteFp4Full)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int steps = min(4, (p.K - kb * kFp4Bk + 63) / 64);  // none behind K: its scales may be stale
            const uint32_t at = a_smem(ps.slot());
            const uint32_t a = rows_lo(at), b = a + Cfg::A_BYTES / 16;
            const uint32_t sa = scales_lo(at) + (Cfg::A_BYTES + Cfg::B_BYTES) / 16, sb = sa + Cfg::S_BYTES / 16;
            const int atoms = FMT == kNv ? steps : (steps + 1) / 2;
#pragma unroll
            for (int j = 0; j < Cfg::ATOMS; ++j) {
                if (j >= atoms) break;
                fp4_copy_scales<false>(tmem + Cfg::SFA_COL + 4 * j, sa + 32 * j, elected);
                fp4_copy_scales<false>(tmem + Cfg::SFB_COL + 4 * j, sb + 32 * j, elected);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= steps) break;
                const uint32_t col = FMT == kNv ? 4u * j : 4u * (j >> 1);
                const uint32_t id = FMT == kNv ? 0u : 2u * (j & 1);
                fp4_mma<FMT, false>(tmem, a + 2u * j, b + 2u * j,
                                    fp4_idesc<FMT>(128, NT, id), tmem + Cfg::SFA_COL + col,
                                    tmem + Cfg::SFB_COL + col, (kb > kb0 || j > 0) ? 1u : 0u, elected);
            }
            if (elected) tc_commit(empty_bar(ps.slot()));
            __syncwarp();
            ps.next();
        }
        if (elected) tc_commit(acc_bar);
        __syncwarp();
    } else if constexpr (Q) {
        // the tokens' codes and scales of the CTA's K range, block by block, in
        // the places where TMA would put them: 128-byte rows, 16-byte pieces
        // exchanged by the row's low three bits; scales as in memory
        constexpr int B = fp4_block(FMT), BLOCKS = kFp4Bk / B;
        const TensorScale ts = tensor_scale(FMT == kNv ? p.ts_a : nullptr);
        Ring<STAGES> ps;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(empty_bar(ps.slot()), ps.parity() ^ 1u, abort_flag, p.ctl, kSiteFp4Quant)) break;
            uint8_t* const codes_at = smem + ps.slot() * Cfg::STAGE_BYTES + Cfg::A_BYTES;
            uint8_t* const scales_at = codes_at + Cfg::B_BYTES + Cfg::S_BYTES;
            for (int i = threadIdx.x; i < cols * BLOCKS; i += 128) {
                const int m = i / BLOCKS, blk = i % BLOCKS;
                const int k = kb * kFp4Bk + blk * B;
                float x[B];
                uint32_t codes[B / 8];
                load_some<QUANT, B>(static_cast<const QUANT*>(p.X) + (m0 + m) * p.ldx + k, min(p.K - k, B), p.x_aligned, x);
                const uint32_t byte = quantize_block<FMT>(x, ts, codes);
                uint8_t* const row = codes_at + m * 128;
                if constexpr (B == 16)
                    *reinterpret_cast<uint2*>(row + (((blk >> 1) ^ (m & 7)) << 4) + 8 * (blk & 1)) =
                        make_uint2(codes[0], codes[1]);
                else
                    *reinterpret_cast<uint4*>(row + ((blk ^ (m & 7)) << 4)) =
                        make_uint4(codes[0], codes[1], codes[2], codes[3]);
                scales_at[(blk >> 2) * 512 + (m & 31) * 16 + (m >> 5) * 4 + (blk & 3)] = static_cast<uint8_t>(byte);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full_bar(ps.slot()));
            ps.next();
        }
    }
    // Everyone waits for the accumulator: warps 0-3 read it, the others must
    // not leave (or let the ring be reused) before the MMAs and copies end.
    if (warp == 4) pdl_wait_prior_grid();
    const Fp4Alpha alpha = fp4_alpha(p);
    if (!bounded_wait(acc_bar, 0u, nullptr, p.ctl, kSiteFp4Acc)) ok = false;
    if (warp == 4 && lane == 0 && *abort_flag) {
        // copies may still be in flight: give them a fixed time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {
        }
    }
    tc_fence_after();
    pdl_launch_dependents();
    const bool good = __syncthreads_and(ok && !*abort_flag);
    const bool empty = kb1 == kb0;
    const int n = n0 + warp * 32 + lane;
    const float bias = warp < 4 && p.bias && n < p.N ? typed_at(p.bias, p.dtype, n) : 0.f;
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    if (splits == 1) {
        if (warp < 4 && good) {
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_wait_ld();
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = empty ? 0.f : __uint_as_float(r[i]);
                fp4_first(f, alpha);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n < p.N && c + i < cols)
                        typed_store(p.Y, p.dtype, (m0 + c + i) * p.ldy + n, fmaf(f[i], alpha.second, bias));
            }
        }
        tc_fence_before();
        __syncthreads();
    } else {
        // fp32 sums, column by column, over the idle ring; then each owner's
        // columns in one copy to join[rank][column][row] there
        float* const sums = reinterpret_cast<float*>(smem);
        if (warp < 4) {
#pragma unroll 1
            for (int c = 0; c < cols; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < cols) sums[(c + i) * 128 + warp * 32 + lane] = __uint_as_float(r[i]);
            }
            fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncthreads();
        cluster_wait();  // every CTA of the cluster runs and has armed its barrier
        if (threadIdx.x < splits) {
            const int owner = threadIdx.x, mine = min(cols - owner * per, per);
            if (mine > 0)
                bulk_copy_s2s_cluster(mapa_shared(smem_u32(join) + 512u * (split * per), owner),
                                      smem_u32(sums) + 512u * (owner * per), 512u * mine, mapa_shared(join_bar, owner));
        }
        __syncwarp();
        const int c1 = min(cols, (split + 1) * per);
        if (warp < 4 && split * per < cols) {
            const bool joined = warp_wait(join_bar, 0u, nullptr, p.ctl, kSiteFp4Join);
            if (good && joined && n < p.N)
                for (int c = split * per; c < c1; ++c) {
                    float acc[1] = {0.f};
                    for (int s = 0; s < splits; ++s) acc[0] += join[(s * per + c - split * per) * 128 + threadIdx.x];
                    fp4_first(acc, alpha);
                    typed_store(p.Y, p.dtype, (m0 + c) * p.ldy + n, fmaf(acc[0], alpha.second, bias));
                }
        }
        cluster_sync();  // nobody leaves while its sums may still be on their way
    }
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

}  // namespace qg
