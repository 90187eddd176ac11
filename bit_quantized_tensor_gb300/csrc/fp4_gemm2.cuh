// The same product on CTA pairs, for problems with many tokens: 256 x 256
// tiles, persistent.  Two CTAs of a cluster share a tile; CTA r holds 128 rows
// of the tokens and 128 rows of the weights, and the leader's cta_group::2 MMA
// reads both halves, so each SM loads half as many weights per product as with
// a tile of its own.  Each CTA also holds the scales of its own 128 token rows
// and of all 256 weight rows, since its half of the accumulator needs them all.
//
// Tensor memory (512 columns) cannot hold two 256-column accumulators and the
// scales.  The two accumulators therefore overlap by 48 columns:
//   [0, 256) accumulator 0, [208, 464) accumulator 1, [464, 512) scales.
// The epilogue drains the shared columns of a tile first and then lets the
// MMAs of the next tile go, which write the other accumulator.  That costs the
// tensor cores the time to drain 48 columns a tile instead of 256.
//
// Bound by the issuing warp: 4096 x 8192 x 8192 takes 86 us (6.4 PFLOP/s) with
// blocks of 16 and 77 us (7.2) with blocks of 32, whose scales are half as many
// copies.  With descriptors as 64-bit sums it took 95 us (84 without its epilogue,
// 76 without its loads, 62 with the MMAs alone); a stage unrolled around those 91.
// A first look at the next block's barrier while one is issued costs 5 us.  A warp
// of its own for the scale copies, with two sets of scales in tensor memory, took
// a quantizing call from 120 to 143 us, copies between the MMAs of a block to 154.
#pragma once
#include "fp4_gemm.cuh"
#include "tc_gemm.cuh"

namespace qg {

template <int FMT_>
struct Fp4PairCfg {
    static constexpr int FMT = FMT_;
    static constexpr int ATOMS = FMT == kNv ? 4 : 2;
    static constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128;
    static constexpr int S_BYTES = ATOMS * 512;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 3 * S_BYTES;
    static constexpr int BARRIER_BYTES = 256;
    static constexpr int EPI_WARPS = 8;
    static constexpr int OUT_BYTES = EPI_WARPS * 2048;  // 32 rows x 16 columns a warp, see fp4_store_rows
    static constexpr int STAGES = (232448 - BARRIER_BYTES - OUT_BYTES - 1024) / STAGE_BYTES;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + BARRIER_BYTES + OUT_BYTES + 1024;
    static constexpr int ACC_STEP = 208;              // first column of accumulator 1
    static constexpr int SHARED_COLS = 256 - ACC_STEP;
    static constexpr int SFA_COL = ACC_STEP + 256, SFB_COL = SFA_COL + 4 * ATOMS;
    static constexpr int THREADS = 32 * (2 + EPI_WARPS);
    static_assert(SFB_COL + 8 * ATOMS <= 512, "tensor memory");
    static_assert(STAGES >= 4 && SMEM_BYTES <= 232448 && 2 * SMEM_BYTES > 233472, "shared memory, one CTA per SM");
    static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms of 1 KB");
};

constexpr int kSiteFp4PairEmpty = 311;
constexpr int kSiteFp4PairAcc = 312;
constexpr int kSiteFp4PairFull = 313;
constexpr int kSiteFp4PairEpi = 314;
constexpr int kSiteFp4PairDrainTma = 315;
constexpr int kSiteFp4PairDrainMma = 316;

// 32 rows x 16 columns of a warp (lane = row) to Y where rows are not 32-byte
// aligned or end inside the 16 columns: turned in shared memory, so that
// neighbouring lanes store neighbouring words of a row.  One value a lane and
// store instead (32 rows an instruction) took 36 us for 777 x 1001 x 2304.
// `buf`: 512 words of the warp; 16-byte pieces are exchanged by the row, which
// keeps both directions free of bank conflicts.
template <class T>
__device__ __forceinline__ void fp4_store_rows(uint8_t* buf, const float (&f)[16], T* Y, int64_t ldy, int row0, int M,
                                               int col, int N) {
    constexpr int RB = 16 * static_cast<int>(sizeof(T)), PIECES = RB / 16;
    const int lane = threadIdx.x & 31;
    auto turn = [](int r) { return PIECES == 4 ? (r >> 1) & 3 : (r >> 2) & 1; };
    float g[16 / PIECES];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
#pragma unroll
        for (int j = 0; j < 16 / PIECES; ++j) g[j] = f[q * (16 / PIECES) + j];
        store_vec<T, 16 / PIECES>(reinterpret_cast<T*>(buf + lane * RB + ((q ^ turn(lane)) << 4)), g);
    }
    __syncwarp();
    constexpr int WORDS = RB / 4, PER = 4 / static_cast<int>(sizeof(T));  // words a row, values a word
    const int w = lane % WORDS, c = col + w * PER;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        const int r = i * (32 / WORDS) + lane / WORDS;
        const uint32_t v = *reinterpret_cast<const uint32_t*>(buf + r * RB + (((w >> 2) ^ turn(r)) << 4) + (w & 3) * 4);
        if (row0 + r >= M || c >= N) continue;
        T* dst = Y + (row0 + r) * ldy + c;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<uint32_t*>(dst) = v;
        } else if (c + 1 < N && (reinterpret_cast<uintptr_t>(dst) & 3) == 0) {
            *reinterpret_cast<uint32_t*>(dst) = v;
        } else {
            reinterpret_cast<uint16_t*>(dst)[0] = static_cast<uint16_t>(v);
            if (c + 1 < N) reinterpret_cast<uint16_t*>(dst)[1] = static_cast<uint16_t>(v >> 16);
        }
    }
    __syncwarp();
}

template <class Cfg>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg::THREADS, 1)
    fp4_gemm2_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmSX, const __grid_constant__ CUtensorMap tmSW,
                     const Fp4Params p) {
    constexpr int STAGES = Cfg::STAGES, FMT = Cfg::FMT, ATOMS = Cfg::ATOMS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    // per stage: token codes | weight codes | token scales | weight scales (two blocks of 128 rows)
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * Cfg::STAGE_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    const uint32_t next_bar = bar0 + 8u * (2 * STAGES + 2);  // leader: the next tile's MMAs may start
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 3);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 4);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    uint8_t* const out_smem = smem + STAGES * Cfg::STAGE_BYTES + Cfg::BARRIER_BYTES;
    const uint32_t ring0 = smem_u32(smem);
    auto stage_smem = [&](int s) { return ring0 + static_cast<uint32_t>(s) * Cfg::STAGE_BYTES; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(accf_bar(0), 1);
        mbar_init(accf_bar(1), 1);
        mbar_init(next_bar, 2 * Cfg::EPI_WARPS);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmSX);
        tma_prefetch_desc(&tmSW);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);  // known to be uniform
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int num_m = (p.M + 255) / 256, num_n = (p.N + 255) / 256;
    const int ntiles = num_m * num_n;
    const int num_kb = (p.K + kFp4Bk - 1) / kFp4Bk;
    const int col_tiles = static_cast<int>(fp4_col_tiles(FMT, p.K));

    if (warp == 0) {
        // ------------------------------------------------ TMA producer (both CTAs)
        fence_proxy_async_global();
        const uint32_t elected = elect_lane();
        Ring<STAGES> ps;
        uint32_t armed = 0, armed_phase = 0;
        bool ok = true;
        for (int t = pair; ok && t < ntiles; t += npairs) {
            int mb, nb;
            tile_coords(t, num_m, num_n, mb, nb, kGroupMPairs);
            const int arow = mb * 256 + static_cast<int>(rank) * 128;
            const int brow = nb * 256 + static_cast<int>(rank) * 128;
            for (int kb = 0; kb < num_kb; ++kb) {
                if (!__all_sync(0xffffffffu, bounded_wait(empty_bar(ps.slot()), ps.parity() ^ 1u, abort_flag, p.ctl,
                                                          kSiteFp4PairEmpty))) {
                    ok = false;
                    break;
                }
                const uint32_t full = mapa_shared(full_bar(ps.slot()), 0);
                if (leader) {
                    if (elected) mbar_arrive_expect_tx(full_bar(ps.slot()), 2 * Cfg::STAGE_BYTES);
                    __syncwarp();
                    armed |= 1u << ps.slot();
                    armed_phase = (armed_phase & ~(1u << ps.slot())) | (ps.parity() << ps.slot());
                }
                const uint32_t a = stage_smem(ps.slot()), b = a + Cfg::A_BYTES;
                const uint32_t sa = b + Cfg::B_BYTES, sb = sa + Cfg::S_BYTES;
                fp4_load_pair(a, &tmX, kb * (kFp4Bk / 2), arow, full, elected);
                fp4_load_pair(b, &tmW, kb * (kFp4Bk / 2), brow, full, elected);
                // rows of scale tiles past the operand read as 0
                fp4_load_pair(sa, &tmSX, 0, (arow >> 7) * col_tiles + kb * ATOMS, full, elected);
                fp4_load_pair(sb, &tmSW, 0, (nb * 2) * col_tiles + kb * ATOMS, full, elected);
                fp4_load_pair(sb + Cfg::S_BYTES, &tmSW, 0, (nb * 2 + 1) * col_tiles + kb * ATOMS, full, elected);
                ps.next();
            }
        }
        if (!ok) {
            if (leader) {
                for (int s = 0; s < STAGES; ++s)
                    if (armed & (1u << s))
                        bounded_wait(full_bar(s), (armed_phase >> s) & 1u, nullptr, p.ctl, kSiteFp4PairDrainTma);
            } else {
                // the leader's barrier cannot be polled from here: a fixed time to land
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 1000000) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            // ------------------------------------------------ MMA issuer (leader)
            const uint32_t elected = elect_lane();
            Ring<STAGES> ps;
            const int last_steps = (p.K - (num_kb - 1) * kFp4Bk + 63) / 64;  // of 64, in a row's last block
            int n = 0;  // tiles begun
            bool ok = true;
            for (int t = pair; ok && t < ntiles; t += npairs, ++n) {
                // tile n - 1 has handed over the shared columns, and with it all of tile n - 2
                if (n > 0 && !__all_sync(0xffffffffu, bounded_wait(next_bar, (n - 1) & 1u, abort_flag, p.ctl,
                                                                   kSiteFp4PairAcc)))
                    break;
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>((n & 1) * Cfg::ACC_STEP);
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!__all_sync(0xffffffffu, bounded_wait(full_bar(ps.slot()), ps.parity(), abort_flag, p.ctl,
                                                              kSiteFp4PairFull))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = stage_smem(ps.slot());
                    const uint32_t a = rows_lo(at), b = a + Cfg::A_BYTES / 16;
                    const uint32_t sa = scales_lo(at) + (Cfg::A_BYTES + Cfg::B_BYTES) / 16, sb = sa + Cfg::S_BYTES / 16;
                    auto scales = [&](int j) {
                        fp4_copy_scales<true>(tmem + Cfg::SFA_COL + 4 * j, sa + 32 * j, elected);
                        fp4_copy_scales<true>(tmem + Cfg::SFB_COL + 8 * j, sb + 32 * j, elected);
                        fp4_copy_scales<true>(tmem + Cfg::SFB_COL + 8 * j + 4, sb + Cfg::S_BYTES / 16 + 32 * j, elected);
                    };
                    auto mma = [&](int j) {
                        const uint32_t atom = FMT == kNv ? j : j >> 1;
                        const uint32_t id = FMT == kNv ? 0u : 2u * (j & 1);
                        fp4_mma<FMT, true>(d, a + 2u * j, b + 2u * j, fp4_idesc<FMT>(256, 256, id),
                                           tmem + Cfg::SFA_COL + 4 * atom, tmem + Cfg::SFB_COL + 8 * atom,
                                           (kb > 0 || j > 0) ? 1u : 0u, elected);
                    };
                    if (kb + 1 < num_kb || last_steps == 4) {
#pragma unroll
                        for (int j = 0; j < ATOMS; ++j) scales(j);
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma(j);
                    } else {  // nothing behind K: its scales may be stale
#pragma unroll
                        for (int j = 0; j < ATOMS; ++j)
                            if (j * (4 / ATOMS) < last_steps) scales(j);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < last_steps) mma(j);
                    }
                    if (elected) tc_commit_pair(empty_bar(ps.slot()), 0x3);
                    __syncwarp();
                    ps.next();
                }
                if (!ok) break;
                if (elected) tc_commit_pair(accf_bar(n & 1), 0x3);
                __syncwarp();
            }
            if (elected) tc_commit_pair(drain_bar, 0x1);
            __syncwarp();
            bounded_wait(drain_bar, 0u, nullptr, p.ctl, kSiteFp4PairDrainMma);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- epilogue (both CTAs)
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const Fp4Alpha alpha = fp4_alpha(p);
        const uint32_t next = mapa_shared(next_bar, 0);
        uint8_t* const buf = out_smem + (warp - 2) * 2048;
        const bool sectors = (reinterpret_cast<uintptr_t>(p.Y) & 31) == 0 &&
                             (p.ldy * (p.dtype == QG_F32 ? 4 : 2)) % 32 == 0;
        // 16 columns of the warp's rows, in the type of Y
        auto put = [&](auto* Y, const uint32_t(&r)[16], int row0, int col) {
            using T = typename std::remove_pointer<decltype(Y)>::type;
            const T* bias = static_cast<const T*>(p.bias);
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(r[j]);
            fp4_first(f, alpha);
            if (!bias) {
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] *= alpha.second;
            } else if (col + 16 <= p.N) {
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = fmaf(f[j], alpha.second, to_f32<T>(bias[col + j]));
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    f[j] = fmaf(f[j], alpha.second, to_f32<T>(bias[min(col + j, p.N - 1)]));
            }
            if (sectors && col + 16 <= p.N) {
                if (row0 + lane < p.M) store_sectors(Y + (row0 + lane) * p.ldy + col, f);
            } else {
                fp4_store_rows(buf, f, Y, p.ldy, row0, p.M, col, p.N);
            }
        };
        int n = 0;
        for (int t = pair; t < ntiles; t += npairs, ++n) {
            int mb, nb;
            tile_coords(t, num_m, num_n, mb, nb, kGroupMPairs);
            const int row0 = mb * 256 + static_cast<int>(rank) * 128 + quad * 32;
            const bool got = bounded_wait(accf_bar(n & 1), (n >> 1) & 1u, abort_flag, p.ctl, kSiteFp4PairEpi);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16) +
                                   static_cast<uint32_t>((n & 1) * Cfg::ACC_STEP);
            // Accumulator 0 shares its last 48 columns and accumulator 1 its first 48
            // with the other one.  A warp's arrival says that it has read those of its
            // half (whether they are shared or not) and all of the tile before.
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(next);
            };
            auto put_any = [&](const uint32_t(&r)[16], int c) {
                const int col = nb * 256 + c;
                if (row0 >= p.M || col >= p.N) return;
                if (p.dtype == QG_F16)
                    put(static_cast<__half*>(p.Y), r, row0, col);
                else if (p.dtype == QG_BF16)
                    put(static_cast<__nv_bfloat16*>(p.Y), r, row0, col);
                else
                    put(static_cast<float*>(p.Y), r, row0, col);
            };
            // 16 columns a step, half 1 from the top down, so that the shared ones are
            // the first of the half that has them: all of those are read before any is
            // stored, since the next tile's MMAs wait for them
            auto col_of = [&](int i) { return half ? 240 - 16 * i : 16 * i; };
            uint32_t r[Cfg::SHARED_COLS / 16][16];
#pragma unroll
            for (int i = 0; i < Cfg::SHARED_COLS / 16; ++i) tmem_ld_32x32b_x16(taddr + col_of(i), r[i]);
            tmem_wait_ld();
            release();
#pragma unroll
            for (int i = 0; i < Cfg::SHARED_COLS / 16; ++i) put_any(r[i], col_of(i));
#pragma unroll 1
            for (int i = Cfg::SHARED_COLS / 16; i < 8; ++i) {
                tmem_ld_32x32b_x16(taddr + col_of(i), r[0]);
                tmem_wait_ld();
                put_any(r[0], col_of(i));
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while its partner may still use it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace qg
