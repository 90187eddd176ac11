// Product of two microscaled 4-bit operands on the block-scaled tensor cores:
//   Y[m][n] = alpha * sum_k (a[m][k] sa[m][k / B]) (b[n][k] sb[n][k / B]) + bias[n]
// with a, b e2m1 codes and sa, sb block scales (fp4_common.cuh), alpha the
// product of the tensor scales.  tcgen05.mma multiplies the codes, applies both
// block scales and accumulates in fp32 in tensor memory; each K step of 64
// needs the scales of its rows in tensor memory too, which tcgen05.cp brings
// there from shared memory in the layout that the packed scales already have.
#pragma once
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

template <int FMT>
__device__ __forceinline__ void fp4_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (FMT == kNv)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %6, 0;\n"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
                d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}

// One 512-byte scale tile from shared memory into four columns of tensor
// memory, repeated in each quarter of the lanes.
__device__ __forceinline__ void fp4_copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

// Shared-memory descriptor of a scale tile: 32 rows of 16 bytes, no swizzle,
// 128 bytes between groups of 8 rows, descriptor version 1.
__device__ __forceinline__ uint64_t fp4_scale_desc(uint32_t smem_addr) {
    return static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128u >> 4) << 32) |
           (static_cast<uint64_t>(1u) << 46);
}

// ------------------------------------------------ one CTA per tile
//
// The weights' rows are the 128 rows of the MMA and the tokens its NT columns,
// so that few tokens waste few columns and the weights, which are what a small
// batch has to read, move in whole 16 KB boxes.  A cluster of S CTAs splits K
// and joins the fp32 sums through distributed shared memory, in rank order.
//   warp 4  TMA producer      warp 5  MMA issuer, owner of the tensor memory
//   warps 0-3  epilogue (their lane quarter of the accumulator)
constexpr int kFp4Threads = 192;
constexpr int kFp4Bk = 256;  // K of a stage: one 128-byte swizzled row of codes

template <int FMT_, int NT_>
struct Fp4Cfg {
    static constexpr int FMT = FMT_, NT = NT_;
    static constexpr int ATOMS = FMT == kNv ? 4 : 2;            // scale tiles along K in a stage
    static constexpr int A_BYTES = 128 * 128;
    static constexpr int B_BYTES = NT * 128;
    static constexpr int S_BYTES = ATOMS * 512;                 // scales of 128 rows
    static constexpr int B_ALLOC = B_BYTES < 1024 ? 1024 : B_BYTES;  // swizzle atoms of 1 KB
    static constexpr int STAGE_BYTES = A_BYTES + B_ALLOC + 2 * S_BYTES;
    static constexpr int TX_BYTES = A_BYTES + B_BYTES + 2 * S_BYTES;
    static constexpr int STAGES = NT >= 128 ? 5 : 8;
    static constexpr int BARRIER_BYTES = 256;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + BARRIER_BYTES + 1024;
    static constexpr int SFA_COL = NT;                          // D at column 0
    static constexpr int SFB_COL = NT + 4 * ATOMS;
    static constexpr int COLS_USED = NT + 8 * ATOMS;
    static constexpr int TMEM_COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : 256;
    static_assert(NT % 16 == 0 && NT <= 128, "MMA columns");
    static_assert(COLS_USED <= TMEM_COLS, "tensor memory");
    static_assert(SMEM_BYTES <= 232448, "shared memory");
    static_assert(128 * NT * 4 <= STAGES * STAGE_BYTES, "the joined sums reuse the ring");
};

struct Fp4Params {
    int M, N, K;         // tokens, weight rows, reduction
    const float *ts_a, *ts_b;  // tensor scales of the tokens and the weights, or null
    const void* bias;    // N values of the output type, or null
    void* Y;
    int64_t ldy;
    int dtype;           // of Y and bias
    bool weights_ready;  // the weights were complete before the kernel ahead on the stream started
    Ctl ctl;
};

constexpr int kSiteFp4Empty = 301;
constexpr int kSiteFp4Full = 302;
constexpr int kSiteFp4Acc = 303;
constexpr int kSiteFp4DrainTma = 304;
constexpr int kSiteFp4DrainMma = 305;

__device__ __forceinline__ float fp4_alpha(const Fp4Params& p) {
    return (p.ts_a ? *p.ts_a : 1.f) * (p.ts_b ? *p.ts_b : 1.f);
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

template <class Cfg>
__global__ void __launch_bounds__(kFp4Threads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                    const Fp4Params p) {
    constexpr int NT = Cfg::NT, STAGES = Cfg::STAGES, FMT = Cfg::FMT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    // per stage: weights' codes | tokens' codes | weights' scales | tokens' scales
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * Cfg::STAGE_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t acc_bar = bar0 + 8u * (2 * STAGES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    auto a_smem = [&](int s) { return smem_u32(smem + s * Cfg::STAGE_BYTES); };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int splits = static_cast<int>(gridDim.x), split = static_cast<int>(blockIdx.x);  // the cluster
    const int n0 = static_cast<int>(blockIdx.y) * 128;
    const int m0 = static_cast<int>(blockIdx.z) * NT;
    const int num_kb = (p.K + kFp4Bk - 1) / kFp4Bk;
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * split / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (split + 1) / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(acc_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmSW);
        tma_prefetch_desc(&tmSX);
    }
    if (warp == 5) tmem_alloc(smem_u32(tmem_holder), Cfg::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    // The bounded waits below start only when the previous kernel is done (they
    // must not count its time); the producer alone may run ahead of that.
    if (warp != 4) pdl_wait_prior_grid();
    bool ok = true;
    if (warp == 4) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_normal();
            auto load_w = [&](int kb, int s) {
                tma_load_2d(a_smem(s), &tmW, kb * (kFp4Bk / 2), n0, full_bar(s), keep);
                tma_load_2d(a_smem(s) + Cfg::A_BYTES + Cfg::B_ALLOC, &tmSW, 0,
                            static_cast<int>(blockIdx.y * fp4_col_tiles(FMT, p.K)) + kb * Cfg::ATOMS, full_bar(s),
                            keep);
            };
            auto load_x = [&](int kb, int s) {
                tma_load_2d(a_smem(s) + Cfg::A_BYTES, &tmX, kb * (kFp4Bk / 2), m0, full_bar(s), keep);
                tma_load_2d(a_smem(s) + Cfg::A_BYTES + Cfg::B_ALLOC + Cfg::S_BYTES, &tmSX, 0,
                            static_cast<int>((m0 >> 7) * fp4_col_tiles(FMT, p.K)) + kb * Cfg::ATOMS, full_bar(s),
                            keep);
            };
            // Weights that were complete before the previous kernel began may
            // be fetched while that kernel (which makes the tokens' codes) runs.
            const int ahead = min(kb1 - kb0, STAGES);
            if (!p.weights_ready) pdl_wait_prior_grid();
            for (int i = 0; i < ahead; ++i) {
                mbar_arrive_expect_tx(full_bar(i), Cfg::TX_BYTES);
                load_w(kb0 + i, i);
            }
            if (p.weights_ready) pdl_wait_prior_grid();
            for (int i = 0; i < ahead; ++i) load_x(kb0 + i, i);
            Ring<STAGES> ps;
            for (int i = 0; i < ahead; ++i) ps.next();
            for (int kb = kb0 + ahead; kb < kb1; ++kb) {
                if (!bounded_wait(empty_bar(ps.slot()), ps.parity() ^ 1u, abort_flag, p.ctl, kSiteFp4Empty)) break;
                mbar_arrive_expect_tx(full_bar(ps.slot()), Cfg::TX_BYTES);
                load_w(kb, ps.slot());
                load_x(kb, ps.slot());
                ps.next();
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        if (lane == 0) {
            Ring<STAGES> ps;
            const uint32_t sfb_shift = static_cast<uint32_t>((m0 & 127) >> 5);  // tile inside its 128 scale rows
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!bounded_wait(full_bar(ps.slot()), ps.parity(), abort_flag, p.ctl, kSiteFp4Full)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int steps = min(4, (p.K - kb * kFp4Bk + 63) / 64);  // none behind K: its scales may be stale
                const uint32_t a = a_smem(ps.slot()), b = a + Cfg::A_BYTES;
                const uint32_t sa = b + Cfg::B_ALLOC, sb = sa + Cfg::S_BYTES;
                const int atoms = FMT == kNv ? steps : (steps + 1) / 2;
                for (int j = 0; j < atoms; ++j) {
                    fp4_copy_scales(tmem + Cfg::SFA_COL + 4 * j, fp4_scale_desc(sa + 512 * j));
                    fp4_copy_scales(tmem + Cfg::SFB_COL + 4 * j, fp4_scale_desc(sb + 512 * j));
                }
                for (int j = 0; j < steps; ++j) {
                    const uint32_t col = FMT == kNv ? 4u * j : 4u * (j >> 1);
                    const uint32_t id = FMT == kNv ? 0u : 2u * (j & 1);
                    fp4_mma<FMT>(tmem, smem_desc_sw128(a + 32u * j), smem_desc_sw128(b + 32u * j),
                                 fp4_idesc<FMT>(128, NT, id), tmem + Cfg::SFA_COL + col,
                                 tmem + Cfg::SFB_COL + col + sfb_shift, (kb > kb0 || j > 0) ? 1u : 0u);
                }
                tc_commit(empty_bar(ps.slot()));
                ps.next();
            }
            tc_commit(acc_bar);
        }
        __syncwarp();
    }
    if (warp == 4) pdl_wait_prior_grid();
    // Everyone waits for the accumulator: warps 0-3 read it, the others must
    // not leave (or let the ring be reused) before the MMAs and copies end.
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
    const float alpha = fp4_alpha(p);
    const bool empty = kb1 == kb0;

    if (splits == 1) {
        if (warp < 4 && good) {
            const int n = n0 + warp * 32 + lane;
            const float bias = p.bias && n < p.N ? typed_at(p.bias, p.dtype, n) : 0.f;
            const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int m = m0 + c + i;
                    const float acc = empty ? 0.f : __uint_as_float(r[i]);
                    if (n < p.N && m < p.M)
                        typed_store(p.Y, p.dtype, m * p.ldy + n, fmaf(acc, alpha, bias));
                }
            }
        }
        tc_fence_before();
        __syncthreads();
    } else {
        // fp32 sums to shared memory (the ring is idle), column by column
        float* red = reinterpret_cast<float*>(smem);
        if (warp < 4) {
            const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(taddr + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) red[(c + i) * 128 + warp * 32 + lane] = __uint_as_float(r[i]);
            }
        }
        tc_fence_before();
        __syncthreads();
        cluster_sync();
        const int per = (NT + splits - 1) / splits;
        const int c1 = min(NT, (split + 1) * per);
        const uint32_t red0 = smem_u32(red);
        if (warp < 4) {
            const int n = n0 + threadIdx.x;
            const float bias = p.bias && n < p.N ? typed_at(p.bias, p.dtype, n) : 0.f;
            for (int c = split * per; c < c1; ++c) {
                if (m0 + c >= p.M) break;
                float acc = 0.f;
                for (int s = 0; s < splits; ++s) {
                    float v;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(v)
                                 : "r"(mapa_shared(red0 + 4u * (c * 128 + threadIdx.x), s)));
                    acc += v;
                }
                if (good && n < p.N) typed_store(p.Y, p.dtype, (m0 + c) * p.ldy + n, fmaf(acc, alpha, bias));
            }
        }
        cluster_sync();  // nobody leaves while its sums may still be read
    }
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

}  // namespace qg
