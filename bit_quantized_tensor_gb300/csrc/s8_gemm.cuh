// Product of 8-bit operands for up to some hundred tokens: the weights' codes stay 8 bits wide
// up to the SM and become fp16 in shared memory.
//
// The 128 rows of the MMA are weight rows and its NT columns tokens.  A cluster of S CTAs splits
// K.  Per stage of 128 values of K
//   warp 16     TMA producer: 128 x 128 codes, NT x 128 fp16 codes of the tokens
//   warps 0-15  two groups, a group every second stage: codes to fp16 in the MMA's layout (a pass is
//               bound by its latency, fence and barrier included, so two are under way)
//   warp 17     MMA issuer, owner of the tensor memory
// (Stages of 64 values, with boxes of 64-byte rows, took 1300 cycles each where the MMA takes 256.)
// Every 1024 values of K have an accumulator of their own, whose fp32 sums are whole numbers of
// at most 2^24; they are added up as 32-bit integers, over the accumulators and over the cluster
// (each CTA sends a token's sums to the CTA that owns the token).  Lanes are weight rows in the
// epilogue, so a warp stores 32 neighbouring outputs of a token whatever N is.
#pragma once
#include "fp4_gemm.cuh"
#include "s8_common.cuh"
#include "tc_issue.cuh"

namespace qg {

constexpr int kS8CodeWarps = 16, kS8Groups = 2, kS8GroupWarps = kS8CodeWarps / kS8Groups;
constexpr int kS8Threads = 32 * (kS8CodeWarps + 2);
constexpr int kS8Bk = 128;              // K of a stage: 128 bytes of codes, two 128-byte columns of fp16
constexpr int kS8Exact = 1024 / kS8Bk;  // stages of an accumulator

template <int NT_>
struct S8Cfg {
    static constexpr int NT = NT_;
    static constexpr int RAW_BYTES = 128 * kS8Bk;              // weights' codes of a stage
    static constexpr int X_BYTES = NT * kS8Bk * 2;
    static constexpr int STAGES = NT == 128 ? 3 : 4;
    static constexpr int W_BYTES = 128 * kS8Bk * 2, SLOTS = NT == 128 ? 2 : 3;  // fp16 weights
    static_assert(SLOTS < STAGES, "a slot's last use is told by its stage's barrier");
    static constexpr int W_AT = STAGES * (RAW_BYTES + X_BYTES);
    static constexpr int BARS_AT = W_AT + SLOTS * W_BYTES;
    static constexpr int SUM_BYTES = NT * 128 * 4;             // after the loop: sums to send, then sums received
    static constexpr int SMEM = BARS_AT + 256 + 1024;
    static constexpr int ACCS = 512 / NT;                      // accumulators that fit
    static constexpr uint32_t IDESC = make_idesc(0, 0, 128, NT);
    static_assert(NT % 32 == 0 && NT <= 128, "MMA columns; lanes and columns of the epilogue's warps");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(2 * SMEM > 233472, "one CTA an SM keeps all tensor memory free");
    static_assert(2 * SUM_BYTES <= BARS_AT, "the sums lie over the rings");
};

struct S8Params {
    int M, N, K;
    int log_splits;
    const float *sa, *sb;
    const void* bias;
    void* Y;
    int64_t ldy;
    int dtype;
    Ctl ctl;
};

constexpr int kSiteS8Empty = 321, kSiteS8Full = 322, kSiteS8Ready = 323, kSiteS8Free = 324, kSiteS8Acc = 325,
              kSiteS8Join = 326, kSiteS8Raw = 327;

// Barrier of the cluster without memory ordering: the copies carry their own completion.
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

template <class Cfg>
__global__ void __launch_bounds__(kS8Threads, 1)
    s8_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const S8Params p) {
    constexpr int NT = Cfg::NT, STAGES = Cfg::STAGES, SLOTS = Cfg::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                     ~static_cast<uintptr_t>(1023));
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + Cfg::BARS_AT);
    const uint32_t bar0 = smem_u32(bars), smem0 = smem_u32(smem);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };               // codes and tokens of a stage landed
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };    // ... and are done with
    auto ready_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };  // fp16 weights of a stage
    const uint32_t acc_bar = bar0 + 8u * (2 * STAGES + SLOTS), join_bar = acc_bar + 8u;
    uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + SLOTS + 2);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    // a stage's codes, then all stages' tokens (swizzle atoms of 1 KB)
    auto raw_at = [&](int s) { return s * Cfg::RAW_BYTES; };
    auto x_at = [&](int s) { return STAGES * Cfg::RAW_BYTES + s * Cfg::X_BYTES; };

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int splits = 1 << p.log_splits, split = static_cast<int>(blockIdx.x) & (splits - 1);
    const int n0 = static_cast<int>(blockIdx.x >> p.log_splits) * 128, m0 = static_cast<int>(blockIdx.y) * NT;
    const int num_kb = (p.K + kS8Bk - 1) / kS8Bk;
    const int kb0 = static_cast<int>(static_cast<int64_t>(num_kb) * split / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(num_kb) * (split + 1) / splits), count = kb1 - kb0;
    const int cols = min(NT, p.M - m0), per = (cols + splits - 1) / splits;  // tokens here; of a CTA of the cluster

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < SLOTS; ++b) mbar_init(ready_bar(b), kS8GroupWarps);
        mbar_init(acc_bar, 1);
        mbar_init(join_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (splits > 1) mbar_arrive_expect_tx(join_bar, splits * max(0, min(cols - split * per, per)) * 512);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    pdl_wait_prior_grid();
    if (warp == kS8CodeWarps + 1) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before the tensor memory is held: the next kernel may take its own and then wait for this one
    pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);

    bool ok = true;
    if (warp == kS8CodeWarps) {
        // ------------------------------------------------ TMA producer
        const uint32_t elected = elect_lane();
        fence_proxy_async_global();
        Ring<STAGES> ps;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(empty_bar(ps.slot()), ps.parity() ^ 1u, abort_flag, p.ctl, kSiteS8Empty)) break;
            if (elected) mbar_arrive_expect_tx(full_bar(ps.slot()), Cfg::RAW_BYTES + Cfg::X_BYTES);
            __syncwarp();
            fp4_load(smem0 + raw_at(ps.slot()), &tmW, kb * kS8Bk, n0, full_bar(ps.slot()), elected);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                fp4_load(smem0 + x_at(ps.slot()) + h * (Cfg::X_BYTES / 2), &tmX, kb * kS8Bk + 64 * h, m0,
                         full_bar(ps.slot()), elected);
            ps.next();
        }
    } else if (warp == kS8CodeWarps + 1) {
        // ------------------------------------------------ MMA issuer
        const uint32_t elected = elect_lane();
        Ring<STAGES> ps;
        Ring<SLOTS> bs;
        for (int i = 0; i < count; ++i) {
            if (!warp_wait(full_bar(ps.slot()), ps.parity(), abort_flag, p.ctl, kSiteS8Full) ||
                !warp_wait(ready_bar(bs.slot()), bs.parity(), abort_flag, p.ctl, kSiteS8Ready)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // descriptors as sums of 32-bit words: anything else is done in vector registers and moved
            const uint32_t w = tile_lo(smem0 + Cfg::W_AT, 16) + bs.slot() * (Cfg::W_BYTES / 16);
            const uint32_t x = tile_lo(smem0 + x_at(0), 16) + ps.slot() * (Cfg::X_BYTES / 16);
            const uint32_t d = tmem + static_cast<uint32_t>(i / kS8Exact * NT);
#pragma unroll
            for (int k = 0; k < kS8Bk / 16; ++k)
                mma_ss(d, w + (k >> 2) * (Cfg::W_BYTES / 32) + 2u * (k & 3), x + (k >> 2) * (Cfg::X_BYTES / 32) + 2u * (k & 3),
                       Cfg::IDESC, i % kS8Exact > 0 || k > 0, elected);
            if (elected) tc_commit(empty_bar(ps.slot()));  // the stage, and the slot of its weights
            __syncwarp();
            ps.next();
            bs.next();
        }
        if (elected) tc_commit(acc_bar);
        __syncwarp();
    } else {
        // ------------------------------------------------ codes to fp16
        const int group = warp / kS8GroupWarps, t = threadIdx.x & (32 * kS8GroupWarps - 1);
        // 16-byte pieces of a row's 128 codes, rows 32 apart; the lanes of the second column of fp16
        // store their halves in turn, not to meet in a bank
        const int chunk = t & 7, row = t >> 3, odd = chunk >> 2, c0 = 2 * (chunk & 3);
        for (int i = group; i < count; i += kS8Groups) {
            const int s = i % STAGES, b = i % SLOTS;
            if (!warp_wait(full_bar(s), (i / STAGES) & 1, abort_flag, p.ctl, kSiteS8Raw)) break;
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = *reinterpret_cast<const uint4*>(smem + raw_at(s) + (row + 32 * j) * kS8Bk + 16 * chunk);
            // the MMA is done with the slot's last stage; that stage's barrier cannot be a round further,
            // since it would take this stage's MMA to get there
            if (i >= SLOTS && !warp_wait(empty_bar((i - SLOTS) % STAGES), ((i - SLOTS) / STAGES) & 1, abort_flag, p.ctl,
                                         kSiteS8Free))
                break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = row + 32 * j;
                uint32_t h[8];
                s8_to_f16(w[j].x, h[0], h[1]);
                s8_to_f16(w[j].y, h[2], h[3]);
                s8_to_f16(w[j].z, h[4], h[5]);
                s8_to_f16(w[j].w, h[6], h[7]);
                const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                uint8_t* const at = smem + Cfg::W_AT + b * Cfg::W_BYTES + odd * (Cfg::W_BYTES / 2) + r * 128;
                *reinterpret_cast<uint4*>(at + (((c0 + odd) ^ (r & 7)) << 4)) = odd ? hi : lo;
                *reinterpret_cast<uint4*>(at + (((c0 + 1 - odd) ^ (r & 7)) << 4)) = odd ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready_bar(b));
        }
    }
    if (!bounded_wait(acc_bar, 0u, nullptr, p.ctl, kSiteS8Acc)) ok = false;
    if (warp == kS8CodeWarps && lane == 0 && *abort_flag) {
        // copies may still be in flight: give them a fixed time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {
        }
    }
    tc_fence_after();
    const bool good = __syncthreads_and(ok && !*abort_flag);

    // warp w: lanes' quarter w % 4, columns from 32 (w / 4) on, where there are as many
    const int quad = warp & 3, n = n0 + quad * 32 + lane, accs = (count + kS8Exact - 1) / kS8Exact;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    auto sums_of = [&](int c, int (&v)[16]) {  // 16 columns from c on
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0;
        for (int a = 0; a < accs; ++a) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(taddr + a * NT + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += __float2int_rn(__uint_as_float(r[i]));
        }
    };
    const bool mine = warp < kS8CodeWarps;
    const float sb = mine && n < p.N ? p.sb[n] : 0.f, bias = mine && p.bias && n < p.N ? typed_at(p.bias, p.dtype, n) : 0.f;
    // 16 tokens' results of a lane's row; the scales are read ahead of the stores
    auto store = [&](int c, int c1, const int (&v)[16]) {
        float f[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = c + i < c1 ? p.sa[m0 + c + i] : 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = s8_scaled(v[i], f[i], sb, bias);
        if (n >= p.N) return;
        auto all = [&](auto* y) {
            using Y = std::remove_pointer_t<decltype(y)>;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < c1) y[(m0 + c + i) * p.ldy + n] = from_f32<Y>(f[i]);
        };
        if (p.dtype == QG_F16)
            all(static_cast<__half*>(p.Y));
        else if (p.dtype == QG_BF16)
            all(static_cast<__nv_bfloat16*>(p.Y));
        else
            all(static_cast<float*>(p.Y));
    };
    if (splits == 1) {
        if (mine && good) {
            for (int c = 16 * (warp >> 2); c < cols; c += 64) {
                int v[16];
                sums_of(c, v);
                store(c, cols, v);
            }
        }
        tc_fence_before();
        __syncthreads();
    } else {
        int* const sums = reinterpret_cast<int*>(smem);
        const int* const join = reinterpret_cast<const int*>(smem + Cfg::SUM_BYTES);
        if (mine) {
            for (int c = 16 * (warp >> 2); c < cols; c += 64) {
                int v[16];
                sums_of(c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (c + i < cols) sums[(c + i) * 128 + quad * 32 + lane] = v[i];
            }
            fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncthreads();
        cluster_meet();  // every CTA of the cluster is past its loop: its rings may be written
        if (threadIdx.x < splits) {
            const int owner = threadIdx.x, count_of = min(cols - owner * per, per);
            if (count_of > 0)
                bulk_copy_s2s_cluster(mapa_shared(smem0 + Cfg::SUM_BYTES + 512u * (split * per), owner),
                                      smem0 + 512u * (owner * per), 512u * count_of, mapa_shared(join_bar, owner));
        }
        __syncwarp();
        const int c1 = min(cols, (split + 1) * per);
        if (mine && split * per < cols) {
            const bool joined = warp_wait(join_bar, 0u, nullptr, p.ctl, kSiteS8Join);
            if (good && joined)
                for (int c = split * per + 16 * (warp >> 2); c < c1; c += 64) {
                    int v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0;
                    for (int s = 0; s < splits; ++s) {
                        const int* from = join + (s * per + c - split * per) * 128 + quad * 32 + lane;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < c1) v[i] += from[i * 128];
                    }
                    store(c, c1, v);
                }
        }
        cluster_meet();  // nobody leaves while its sums may still be on their way
    }
    if (warp == kS8CodeWarps + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace qg
