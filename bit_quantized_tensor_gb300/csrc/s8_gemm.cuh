// Product of 8-bit operands for up to some hundred tokens: the weights' codes stay 8 bits wide
// up to the SM and become fp16 in shared memory.
//
// The 128 rows of the MMA are weight rows and its NT columns tokens.  A cluster of S CTAs splits
// K.  Per stage of 64 values of K
//   warp 16     TMA producer: 128 x 64 codes, NT x 64 fp16 codes of the tokens
//   warps 0-15  four groups, a group every fourth stage: codes to fp16 in the MMA's layout (a pass
//               is bound by its latency, fence and barrier included, so four are under way)
//   warp 17     MMA issuer, owner of the tensor memory
// Every 1024 values of K have an accumulator of their own, whose fp32 sums are whole numbers of
// at most 2^24; they are added up as 32-bit integers, over the accumulators and over the cluster
// (each CTA sends a token's sums to the CTA that owns the token).  Lanes are weight rows in the
// epilogue, so a warp stores 32 neighbouring outputs of a token whatever N is.
#pragma once
#include "fp4_gemm.cuh"
#include "s8_common.cuh"
#include "tc_issue.cuh"

namespace qg {

constexpr int kS8CodeWarps = 16, kS8Groups = 4, kS8GroupWarps = kS8CodeWarps / kS8Groups;
constexpr int kS8Threads = 32 * (kS8CodeWarps + 2);
constexpr int kS8Bk = 64;             // K of a stage: 128 bytes of fp16
constexpr int kS8Exact = 1024 / kS8Bk;  // stages of an accumulator

template <int NT_>
struct S8Cfg {
    static constexpr int NT = NT_;
    static constexpr int RAW_BYTES = 128 * kS8Bk;              // weights' codes of a stage
    static constexpr int X_BYTES = NT * kS8Bk * 2;
    static constexpr int STAGES = 4;
    static constexpr int W_BYTES = 128 * kS8Bk * 2, SLOTS = kS8Groups;  // fp16 weights
    static constexpr int W_AT = STAGES * (RAW_BYTES + X_BYTES);
    static constexpr int JOIN_AT = W_AT + SLOTS * W_BYTES;     // sums from the cluster
    static constexpr int JOIN_BYTES = NT * 128 * 4;
    static constexpr int BARS_AT = JOIN_AT + JOIN_BYTES;
    static constexpr int SMEM = BARS_AT + 256 + 1024;
    static constexpr int ACCS = 512 / NT;                      // accumulators that fit
    static constexpr uint32_t IDESC = make_idesc(0, 0, 128, NT);
    static_assert(NT % 32 == 0 && NT <= 128, "MMA columns; lanes and columns of the epilogue's warps");
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(2 * SMEM > 233472, "one CTA an SM keeps all tensor memory free");
    static_assert(NT * 128 * 4 <= W_AT, "the sums to send lie over the ring");
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
    auto free_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + SLOTS + b); };
    const uint32_t acc_bar = bar0 + 8u * (2 * STAGES + 2 * SLOTS), join_bar = acc_bar + 8u;
    uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 2 * SLOTS + 2);
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
        for (int b = 0; b < SLOTS; ++b) {
            mbar_init(ready_bar(b), kS8GroupWarps);
            mbar_init(free_bar(b), 1);
        }
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
    if (splits > 1) cluster_arrive();  // this CTA runs: its shared memory may be written (awaited below)
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
            fp4_load(smem0 + x_at(ps.slot()), &tmX, kb * kS8Bk, m0, full_bar(ps.slot()), elected);
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
            const uint32_t w = smem0 + Cfg::W_AT + bs.slot() * Cfg::W_BYTES, x = smem0 + x_at(ps.slot());
            const uint32_t d = tmem + static_cast<uint32_t>(i / kS8Exact * NT);
#pragma unroll
            for (int k = 0; k < kS8Bk / 16; ++k)
                mma_ss(d, tile_lo(w + 32u * k, 16), tile_lo(x + 32u * k, 16), Cfg::IDESC, i % kS8Exact > 0 || k > 0,
                       elected);
            if (elected) {
                tc_commit(empty_bar(ps.slot()));
                tc_commit(free_bar(bs.slot()));
            }
            __syncwarp();
            ps.next();
            bs.next();
        }
        if (elected) tc_commit(acc_bar);
        __syncwarp();
    } else {
        // ------------------------------------------------ codes to fp16
        const int group = warp / kS8GroupWarps, t = threadIdx.x & (32 * kS8GroupWarps - 1);
        const int chunk = t & 3, row = t >> 2;  // 16-byte pieces of a row's 64 codes; rows 32 apart
        for (int i = group; i < count; i += kS8Groups) {
            const int s = i % STAGES, b = i % SLOTS;
            if (!warp_wait(full_bar(s), (i / STAGES) & 1, abort_flag, p.ctl, kSiteS8Raw)) break;
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = *reinterpret_cast<const uint4*>(smem + raw_at(s) + (row + 32 * j) * kS8Bk + 16 * chunk);
            if (!warp_wait(free_bar(b), ((i / SLOTS) & 1) ^ 1u, abort_flag, p.ctl, kSiteS8Free)) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = row + 32 * j;
                uint32_t h[8];
                s8_to_f16(w[j].x, h[0], h[1]);
                s8_to_f16(w[j].y, h[2], h[3]);
                s8_to_f16(w[j].z, h[4], h[5]);
                s8_to_f16(w[j].w, h[6], h[7]);
                uint8_t* const at = smem + Cfg::W_AT + b * Cfg::W_BYTES + r * 128;
                *reinterpret_cast<uint4*>(at + (((2 * chunk) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(at + (((2 * chunk + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
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
    if (splits == 1) {
        if (mine && good) {
            for (int c = 16 * (warp >> 2); c < cols; c += 64) {
                int v[16];
                sums_of(c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (n < p.N && c + i < cols)
                        typed_store(p.Y, p.dtype, (m0 + c + i) * p.ldy + n,
                                    fmaf(static_cast<float>(v[i]) * p.sa[m0 + c + i], sb, bias));
            }
        }
        tc_fence_before();
        __syncthreads();
    } else {
        int* const sums = reinterpret_cast<int*>(smem);
        const int* const join = reinterpret_cast<const int*>(smem + Cfg::JOIN_AT);
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
        cluster_wait();  // every CTA of the cluster runs and has armed its barrier
        if (threadIdx.x < splits) {
            const int owner = threadIdx.x, count_of = min(cols - owner * per, per);
            if (count_of > 0)
                bulk_copy_s2s_cluster(mapa_shared(smem0 + Cfg::JOIN_AT + 512u * (split * per), owner),
                                      smem0 + 512u * (owner * per), 512u * count_of, mapa_shared(join_bar, owner));
        }
        __syncwarp();
        const int c1 = min(cols, (split + 1) * per);
        if (mine && split * per < cols) {
            const bool joined = warp_wait(join_bar, 0u, nullptr, p.ctl, kSiteS8Join);
            if (good && joined && n < p.N)
                for (int c = split * per + (warp >> 2); c < c1; c += 4) {
                    int v = 0;
                    for (int s = 0; s < splits; ++s) v += join[(s * per + c - split * per) * 128 + quad * 32 + lane];
                    typed_store(p.Y, p.dtype, (m0 + c) * p.ldy + n,
                                fmaf(static_cast<float>(v) * p.sa[m0 + c], sb, bias));
                }
        }
        cluster_sync();  // nobody leaves while its sums may still be on their way
    }
    if (warp == kS8CodeWarps + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace qg
