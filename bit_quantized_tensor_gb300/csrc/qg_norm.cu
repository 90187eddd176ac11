// Layer norm forward, to values or straight to microscaled 4-bit codes:
//   mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),
//   y = (x - mean) rstd gamma + beta
// Statistics are fp32.  Bound by memory: x is read and y (or its codes)
// written once; a row lives in the registers of its threads in between.
#include "norm_common.cuh"

namespace qg {

// Eight consecutive normalised values of a row per lane to codes: the lanes of
// a block find its maximum with shuffles, each lane stores its word of codes,
// and the first lane of every four blocks their scale word.  All lanes of the
// warp take part; positions behind D hold 0.  factors: fill_factors' table, or none
// (a division a block, where rows are too few to pay for the table).
template <int FMT>
__device__ __forceinline__ void quantize_lane8(const float (&y)[8], int64_t k, int64_t D, int64_t row,
                                               const TensorScale& ts, const float* factors, uint8_t* Xq,
                                               uint8_t* Xs) {
    constexpr int LANES = fp4_block(FMT) / 8;
    uint32_t m = absmax_bits<8>(y);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s = factors ? block_scale<FMT>(m, ts, factors) : block_scale<FMT>(m, ts);
    const int64_t ld = fp4_codes_ld(D), tiles = fp4_col_tiles(FMT, D);
    if (k < 2 * ld) *reinterpret_cast<uint32_t*>(Xq + row * ld + k / 2) = scaled_codes8(y, s.r);
    const int blk = (threadIdx.x & 31) / LANES;
    uint32_t word = s.byte << (8 * (blk & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, LANES);
    word |= __shfl_xor_sync(0xffffffffu, word, 2 * LANES);
    if ((threadIdx.x & (4 * LANES - 1)) == 0 && k / fp4_block(FMT) < 4 * tiles)
        *reinterpret_cast<uint32_t*>(Xs + fp4_scale_offset(row, k / fp4_block(FMT), tiles)) = word;
}

constexpr int kToValues = -1;  // FMT of the forward that writes y

struct NormParams {
    int64_t M, D;
    const void* X;
    int64_t ldx;
    RowBounds xb;
    const void *gamma, *beta;
    bool w_f32, x_vec, w_vec, y_vec;
    float eps;
    void* Y;        // FMT < 0
    int64_t ldy;
    uint8_t *Xq, *Xs;  // FMT >= 0
    const float* ts;
    float *mean, *rstd;
};

// Zeroes the scale words behind the last row, up to the whole tile of 128 rows:
// word i of a tile belongs to row i / 4 + 32 (i % 4).  (Row by row, with a division
// a word, a single row of 4096 waited 3 us for its one CTA to get through them.)
template <int FMT>
__device__ __forceinline__ void zero_scale_rows(int64_t M, int64_t D, uint8_t* Xs) {
    const int used = static_cast<int>(M & 127);  // rows of the last tile
    if (used == 0) return;
    const int64_t tiles = fp4_col_tiles(FMT, D);
    uint32_t* const last = reinterpret_cast<uint32_t*>(Xs + (M >> 7) * tiles * 512);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < tiles * 128;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int word = static_cast<int>(i & 127);
        if ((word >> 2) + ((word & 3) << 5) >= used) last[i] = 0;
    }
}

// TPR threads hold a row, VPT times 8 values each; VEC: 8 consecutive values a
// step (16-byte accesses where alignment allows), else one value a step,
// neighbours in neighbouring threads, for rows whose stride breaks alignment.
template <class T, int TPR, int VPT, int FMT, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) k_layer_norm(const NormParams p) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR;
    constexpr int E = 8 * VPT;
    static_assert(FMT < 0 || VEC, "codes are formed from consecutive values");
    __shared__ float red[2][32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / TPR) + threadIdx.x / TPR;
    const int t = threadIdx.x % TPR;
    if (row >= p.M) {  // whole warps: TPR >= 32
        if constexpr (FMT >= 0) zero_scale_rows<FMT>(p.M, p.D, p.Xs);
        return;
    }
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    const int D = static_cast<int>(p.D);
    float v[E];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            const int k = (i * TPR + t) * 8;
            float u[8];
            load_some<T, 8>(x + k, D - k, p.x_vec, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * i + j] = u[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = (8 * i + j) * TPR + t;
                v[8 * i + j] = k < D ? to_f32<T>(x[k]) : 0.f;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sum += v[e];
    // gamma and beta of 8 columns: on their way with the row where a thread has no
    // more (a few rows are all latency), else when they are used
    auto weights = [&](int i, float(&g)[8], float(&b)[8]) {
        if constexpr (VEC) {
            const int k = (i * TPR + t) * 8;
            weights8<T>(p.gamma, p.w_f32, p.w_vec, k, D - k, 1.f, g);
            weights8<T>(p.beta, p.w_f32, p.w_vec, k, D - k, 0.f, b);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = (8 * i + j) * TPR + t;
                g[j] = k < D && p.gamma ? weight_at<T>(p.gamma, p.w_f32, k) : 1.f;
                b[j] = k < D && p.beta ? weight_at<T>(p.beta, p.w_f32, k) : 0.f;
            }
        }
    };
    float g[8], b[8];
    if constexpr (VPT == 1) weights(0, g, b);
    if constexpr (FMT >= 0) zero_scale_rows<FMT>(p.M, p.D, p.Xs);
    const float mean = __fdiv_rn(row_sum<TPR>(sum, red[0]), static_cast<float>(D));
    auto index = [&](int e) { return VEC ? ((e >> 3) * TPR + t) * 8 + (e & 7) : e * TPR + t; };
    float var = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float c = v[e] - mean;
        if (index(e) < D) var = fmaf(c, c, var);
    }
    var = __fdiv_rn(row_sum<TPR>(var, red[1]), static_cast<float>(D));
    const float rstd = __frcp_rn(__fsqrt_rn(var + p.eps));
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    const TensorScale ts = tensor_scale(FMT == kNv ? p.ts : nullptr);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            const int k = (i * TPR + t) * 8;
            if (i > 0 && (i * TPR + (t & ~31)) * 8 >= (D + 127) / 128 * 128) continue;  // the warp is past the row
            float y[8];
            if constexpr (VPT > 1) weights(i, g, b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = k + j < D ? fmaf((v[8 * i + j] - mean) * rstd, g[j], b[j]) : 0.f;
            if constexpr (FMT >= 0)
                quantize_lane8<FMT>(y, k, p.D, row, ts, nullptr, p.Xq, p.Xs);
            else if (k < D)
                store_some<T, 8>(static_cast<T*>(p.Y) + row * p.ldy + k, D - k, p.y_vec, y);
        } else {
            if constexpr (VPT > 1) weights(i, g, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = (8 * i + j) * TPR + t;
                if (k < D)
                    static_cast<T*>(p.Y)[row * p.ldy + k] = from_f32<T>(fmaf((v[8 * i + j] - mean) * rstd, g[j], b[j]));
            }
        }
    }
}

__host__ __device__ constexpr int norm_threads(int tpr) { return tpr == 32 ? 256 : tpr; }
__host__ __device__ constexpr int norm_min_ctas(int tpr) { return tpr == 32 ? 2 : 512 / tpr; }

// A thread holds 8 consecutive columns a step, and gamma and beta of its
// columns stay in registers from row to row.  EDGES: rows may start or end
// inside a 16-byte piece; then all rows of a group start at the same place in
// one (the launch sees to it) and the columns are cut from there, in aligned
// pieces.  Codes cannot follow that (a code word takes eight columns from a
// multiple of eight on), so FMT >= 0 with EDGES reads the ring value by value.
//
// What bounds it besides memory is the number of instructions a value: at 32
// (scalar arithmetic, weights and guards for every row) 8192 x 8192 bf16 took
// 77 us, at 26 67 us; with pairs, 32 columns a thread and held weights it takes
// 47 us (5.7 TB/s, 86 % of a plain copy's rate).
template <class T, int TPR, int FMT, bool EDGES>
__global__ void __launch_bounds__(norm_threads(TPR), norm_min_ctas(TPR))
    k_layer_norm_rows(const NormParams p, int slots, const Ctl ctl) {
    constexpr int GROUPS = norm_threads(TPR) / TPR;
    constexpr int VPT = 4;
    constexpr bool PIECES = FMT < 0 || !EDGES;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ __align__(8) uint64_t bars[GROUPS][kRingMax];
    __shared__ float red[2][32];
    __shared__ int abort_flag;
    __shared__ float factors[FMT == kNv ? 128 : 1];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int D = static_cast<int>(p.D);
    RowRing ring;
    ring.bar0 = smem_u32(&bars[group][0]);
    ring.row_bytes = p.D * static_cast<int64_t>(sizeof(T));
    ring.slot_bytes = static_cast<int>(row_slot_bytes(ring.row_bytes));
    ring.slots = ring_smem + static_cast<int64_t>(group) * slots * ring.slot_bytes;
    if (t == 0) {
        for (int s = 0; s < slots; ++s) mbar_init(ring.bar0 + 8 * s, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    pdl_wait_prior_grid();
    fence_proxy_async_global();
    pdl_launch_dependents();
    if constexpr (FMT >= 0) zero_scale_rows<FMT>(p.M, p.D, p.Xs);
    const T* X = static_cast<const T*>(p.X);
    const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * GROUPS + group;
    for (int s = 0; s < slots; ++s)
        if (row + s * step < p.M) row_fetch<TPR, EDGES>(ring, s, X + (row + s * step) * p.ldx, row + s * step, p.xb);
    const TensorScale ts = tensor_scale(FMT == kNv ? p.ts : nullptr);
    if constexpr (FMT == kNv) fill_factors(factors, ts.ts);
    __syncthreads();
    const float inv_d = __frcp_rn(static_cast<float>(D));
    // values before column 0 in a row's first piece
    const int lead = FMT < 0 && EDGES
                         ? static_cast<int>((reinterpret_cast<uintptr_t>(X + row * p.ldx) & 15) / sizeof(T))
                         : 0;
    auto first = [&](int i) { return (i * TPR + t) * 8 - lead; };  // column of step i
    // what the row leaves of its first piece and of its last
    const int last_piece = (D - 1 + lead) / 8, last_step = last_piece / TPR;
    const PieceMask<T> head = piece_mask<T>(t == 0 ? -lead : 0, D < 8 ? 8 : D);
    const PieceMask<T> tail = piece_mask<T>(t == last_piece % TPR ? last_piece * 8 - lead : 0,
                                            t == last_piece % TPR ? D : 8);
    uint64_t hg[4 * VPT], hb[4 * VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        uint64_t g[4], b[4];
        weight_piece<T>(p.gamma, p.w_f32, p.w_vec, first(i), D, 1.f, g);
        weight_piece<T>(p.beta, p.w_f32, p.w_vec, first(i), D, 0.f, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            hg[4 * i + j] = g[j];
            hb[4 * i + j] = b[j];
        }
    }

    int s = 0;
    uint32_t phase = 0;
    for (; row < p.M; row += step) {
        // a wait that runs out is recorded, ends the fetching, and lets the
        // remaining rows through with whatever their slots hold
        bounded_wait(ring.bar0 + 8 * s, phase, &abort_flag, ctl, kSiteNormRow);
        const T* x = row_in_slot<T>(ring, s, X + row * p.ldx);
        uint64_t v[4 * VPT];
        uint64_t sum2 = 0;  // (0, 0)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = first(i);
            uint64_t u[4] = {0, 0, 0, 0};
            if (k < D) {
                if constexpr (PIECES) {
                    if constexpr (EDGES || FMT >= 0)
                        load_piece<T>(x + k, u, head, i == 0, tail, i == last_step);
                    else
                        load_pairs<T>(x + k, u);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        u[j] = two(k + 2 * j < D ? to_f32<T>(x[k + 2 * j]) : 0.f,
                                   k + 2 * j + 1 < D ? to_f32<T>(x[k + 2 * j + 1]) : 0.f);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[4 * i + j] = u[j];
                sum2 = add_two(sum2, u[j]);
            }
        }
        const float2 sum = both(sum2);
        const float mean = row_sum<TPR>(sum.x + sum.y, red[0]) * inv_d;
        // all threads have read the slot
        if constexpr (TPR == 32) __syncwarp();
        if (row + slots * step < p.M && !*static_cast<volatile int*>(&abort_flag))
            row_fetch<TPR, EDGES>(ring, s, X + (row + slots * step) * p.ldx, row + slots * step, p.xb);
        if (++s == slots) {
            s = 0;
            phase ^= 1u;
        }
        const uint64_t minus = two(-mean, -mean);
        uint64_t var2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            uint64_t c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = add_two(v[4 * i + j], minus);
            if (piece_cut(first(i), D)) cut_piece(c, first(i), D);  // nothing outside the row counts
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                var2 = fma_two(c[j], c[j], var2);
                v[4 * i + j] = c[j];
            }
        }
        const float2 var = both(var2);
        const float rstd = __frcp_rn(__fsqrt_rn(row_sum<TPR>(var.x + var.y, red[1]) * inv_d + p.eps));
        if (t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        uint64_t r2 = two(rstd, rstd);
        if constexpr (FMT >= 0) {
            // codes are 0 behind the row: x - mean, gamma and beta are 0 there, but 1 / std may be NaN
            // or infinite; then it is the row's own values that become NaN (tested once a row:
            // a cut of every piece costs 2 us in 39 at 8192 x 4096)
            if (!(rstd < INFINITY)) {
                r2 = two(1.f, 1.f);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    uint64_t c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[j] = two(NAN, NAN);
                    cut_piece(c, first(i), D);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[4 * i + j] = c[j];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = first(i);
            if (FMT < 0 && k >= D) continue;
            if (FMT >= 0 && i > 0 && (i * TPR + (t & ~31)) * 8 >= (D + 127) / 128 * 128) continue;  // the whole warp
            uint64_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fma_two(mul_two(v[4 * i + j], r2), hg[4 * i + j], hb[4 * i + j]);
            if constexpr (FMT >= 0) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 h = both(y[j]);
                    f[2 * j] = h.x;
                    f[2 * j + 1] = h.y;
                }
                quantize_lane8<FMT>(f, k, p.D, row, ts, factors, p.Xq, p.Xs);
            } else {
                store_piece<T>(static_cast<T*>(p.Y) + row * p.ldy, k, D, !EDGES || p.y_vec, y);
            }
        }
    }
    if (abort_flag) {  // copies may still be in flight: give them a fixed time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {
        }
    }
}

// Rows longer than the registers of a CTA hold: three passes over the row,
// the second and third from L2.
template <class T, int FMT>
__global__ void __launch_bounds__(kLongThreads) k_layer_norm_long(const NormParams p) {
    __shared__ float red[2][32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    if constexpr (FMT >= 0) zero_scale_rows<FMT>(p.M, p.D, p.Xs);
    const int64_t row = blockIdx.x, D = p.D;
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    float sum = 0.f;
    for (int64_t k = threadIdx.x * 8; k < D; k += kLongThreads * 8) {
        float u[8];
        load_some<T, 8>(x + k, static_cast<int>(min(D - k, int64_t(8))), p.x_vec, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += u[j];
    }
    const float mean = __fdiv_rn(row_sum<kLongThreads>(sum, red[0]), static_cast<float>(D));
    float var = 0.f;
    for (int64_t k = threadIdx.x * 8; k < D; k += kLongThreads * 8) {
        float u[8];
        load_some<T, 8>(x + k, static_cast<int>(min(D - k, int64_t(8))), p.x_vec, u);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < D) var = fmaf(u[j] - mean, u[j] - mean, var);
    }
    var = __fdiv_rn(row_sum<kLongThreads>(var, red[1]), static_cast<float>(D));
    const float rstd = __frcp_rn(__fsqrt_rn(var + p.eps));
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    const TensorScale ts = tensor_scale(FMT == kNv ? p.ts : nullptr);
    for (int64_t k0 = 0; k0 < D; k0 += kLongThreads * 8) {  // whole warps, for the shuffles
        const int64_t k = k0 + threadIdx.x * 8;
        const int n = static_cast<int>(max(int64_t(0), min(D - k, int64_t(8))));
        float u[8], g[8], b[8], y[8];
        load_some<T, 8>(x + k, n, p.x_vec, u);
        weights8<T>(p.gamma, p.w_f32, p.w_vec, k, n, 1.f, g);
        weights8<T>(p.beta, p.w_f32, p.w_vec, k, n, 0.f, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = j < n ? fmaf((u[j] - mean) * rstd, g[j], b[j]) : 0.f;
        if constexpr (FMT >= 0)
            quantize_lane8<FMT>(y, k, D, row, ts, nullptr, p.Xq, p.Xs);
        else if (n > 0)
            store_some<T, 8>(static_cast<T*>(p.Y) + row * p.ldy + k, n, p.y_vec, y);
    }
}

// ------------------------------------------------------- host side

constexpr int64_t kMaxHeldFwd = 1024 * 32;   // longest row that k_layer_norm holds
constexpr int64_t kMaxRingFwd = 512 * 32 - 8;  // longest row that k_layer_norm_rows holds, at any place in a piece

template <class T, int TPR, int VPT, int FMT, bool VEC>
static int launch_norm(const NormParams& p, cudaStream_t s) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR;
    constexpr int ROWS = THREADS / TPR;
    return launch_serialized(k_layer_norm<T, TPR, VPT, FMT, VEC>,
                             dim3(static_cast<unsigned>((p.M + ROWS - 1) / ROWS)), THREADS, 0, 1, s, p);
}

// Slots of a ring, 2 at least: the edges of a row show one synchronization
// after their copy.
static int norm_slots(int64_t slot_bytes, int tpr) {
    return ring_slots(slot_bytes, norm_threads(tpr) / tpr * norm_min_ctas(tpr), 2);
}

// Largest dynamic shared memory of an instance (rows of 32 columns a thread).
static int ring_bytes(int tpr, size_t elem) {
    const int64_t slot = row_slot_bytes(static_cast<int64_t>(tpr) * 32 * static_cast<int64_t>(elem));
    return static_cast<int>(slot * norm_slots(slot, tpr) * (norm_threads(tpr) / tpr));
}

template <class T, int TPR, int FMT, bool EDGES>
static int launch_norm_rows(const NormParams& p, int64_t same, int dev, cudaStream_t s) {
    constexpr int THREADS = norm_threads(TPR), GROUPS = THREADS / TPR, CTAS = norm_min_ctas(TPR);
    const Ctl ctl = host_ctl(dev);
    if (!ctl.status) return QG_ERR_CUDA;
    const int64_t slot = row_slot_bytes(p.D * static_cast<int64_t>(sizeof(T)));
    const int slots = norm_slots(slot, TPR);
    const int64_t smem = slot * slots * GROUPS;
    auto* f = k_layer_norm_rows<T, TPR, FMT, EDGES>;
    struct Flags {};
    const int rc = raise_smem<Flags>(f);
    if (rc) return rc;
    const int64_t ctas = norm_ctas(p.M, GROUPS, int64_t(CTAS) * num_sms(dev), same);
    return launch_serialized(f, dim3(static_cast<unsigned>(ctas)), THREADS, static_cast<size_t>(smem), 1, s, p, slots,
                             ctl);
}

// Threads a row: as few as hold it in 32 columns each.  Measured against the next
// count, 2^26 bf16 values, us: rows of 1024 47 (146 with 128 threads), 4096 46 (79 with
// 256), 8192 46 (83 with 512).
template <class T, int FMT, bool EDGES>
static int norm_rows_by_size(const NormParams& p, int64_t same, int dev, cudaStream_t s) {
    const int64_t D = p.D + (EDGES ? 8 : 0);  // its place in the first piece
    if (D <= 1024) return launch_norm_rows<T, 32, FMT, EDGES>(p, same, dev, s);
    if (D <= 4096) return launch_norm_rows<T, 128, FMT, EDGES>(p, same, dev, s);
    if (D <= 8192) return launch_norm_rows<T, 256, FMT, EDGES>(p, same, dev, s);
    return launch_norm_rows<T, 512, FMT, EDGES>(p, same, dev, s);
}

// With more rows than SMs the ring, as few threads a row as hold it; with fewer, one step
// of 8 values a thread, since then the row's own latency is all there is.  Measured
// (bf16, us in a graph, ring / one CTA a row): 152 x 4096 3.7 / 2.6, 304 x 4096 3.8 / 4.5,
// 1216 x 4096 5.9 / 15.7, 304 x 8192 4.3 / 4.8.  Rows of up to 2048 would gain from the
// latter to about 1200 rows (304 x 2048 3.8 / 2.3, 1216 x 2048 5.4 / 4.4).
template <class T, int FMT, bool VEC>
static int norm_by_size(const NormParams& p, int dev, cudaStream_t s) {
    // codes are written up to whole scale words, so a row ends at a multiple of 128 there
    const int64_t D = FMT < 0 ? p.D : (p.D + 127) / 128 * 128;
    if (p.M <= num_sms(dev)) {
        if (D <= 2048) return launch_norm<T, 256, 1, FMT, VEC>(p, s);
        if (D <= 8192) return launch_norm<T, 1024, 1, FMT, VEC>(p, s);
    } else if (D <= kMaxRingFwd) {
        const int64_t same = same_place_rows(p.ldx, sizeof(T));
        const bool edges = !p.x_vec || (FMT < 0 ? p.D % 8 : p.D * static_cast<int64_t>(sizeof(T)) % 16) != 0;
        // y is stored in pieces where its rows start at the same places as those of x
        NormParams q = p;
        q.y_vec = FMT >= 0 || (reinterpret_cast<uintptr_t>(p.X) % 16 == reinterpret_cast<uintptr_t>(p.Y) % 16 &&
                               (static_cast<size_t>(p.ldx) * sizeof(T)) % 16 == (static_cast<size_t>(p.ldy) * sizeof(T)) % 16);
        if (!edges && q.y_vec) return norm_rows_by_size<T, FMT, false>(q, 1, dev, s);
        return norm_rows_by_size<T, FMT, true>(q, FMT < 0 ? same : 1, dev, s);
    }
    if (D <= kMaxHeldFwd) return launch_norm<T, 1024, 4, FMT, VEC>(p, s);
    return launch_serialized(k_layer_norm_long<T, FMT>, dim3(static_cast<unsigned>(p.M)), kLongThreads, 0, 1, s, p);
}

template <class T>
static int norm_forward(int fmt, const NormParams& p, int dev, cudaStream_t s) {
    if (fmt == kNv) return norm_by_size<T, kNv, true>(p, dev, s);
    if (fmt == kMx) return norm_by_size<T, kMx, true>(p, dev, s);
    if (p.x_vec && p.y_vec) return norm_by_size<T, kToValues, true>(p, dev, s);
    return norm_by_size<T, kToValues, false>(p, dev, s);
}

int check_rows(int dtype, int64_t M, int64_t D, const void* X, int64_t ldx) {
    if (M && !X) return QG_ERR_INVALID_ARG;
    if (M > 1 && ldx < D) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype)) return QG_ERR_MISALIGNED;
    return QG_OK;
}

int check_weight(const void* w, int dtype) {
    return reinterpret_cast<uintptr_t>(w) % dtype_bytes(dtype) ? QG_ERR_MISALIGNED : QG_OK;
}

int check_f32(const float* v) { return check_weight(v, QG_F32); }

int check_norm(int dtype, int wdtype, int64_t M, int64_t D, float eps) {
    if (!dtype_ok(dtype) || (wdtype != dtype && wdtype != QG_F32)) return QG_ERR_UNSUPPORTED;
    if (M < 0 || D < 1 || M > INT32_MAX || D > INT32_MAX) return QG_ERR_INVALID_ARG;
    if (!(eps >= 0.f)) return QG_ERR_INVALID_ARG;
    return QG_OK;
}

static int norm_call(int fmt, int dtype, int64_t M, int64_t D, const void* X, int64_t ldx, const void* gamma,
                     const void* beta, int wdtype, float eps, void* Y, int64_t ldy, const float* ts, uint8_t* Xq,
                     uint8_t* Xs, float* mean, float* rstd, void* stream) {
    int rc = check_norm(dtype, wdtype, M, D, eps);
    if (!rc) rc = check_rows(dtype, M, D, X, ldx);
    if (!rc) rc = check_weight(gamma, wdtype);
    if (!rc) rc = check_weight(beta, wdtype);
    if (!rc) rc = check_f32(mean);
    if (!rc) rc = check_f32(rstd);
    if (rc) return rc;
    if (M == 0) return QG_OK;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    NormParams p = {};
    p.M = M; p.D = D; p.X = X; p.ldx = ldx; p.gamma = gamma; p.beta = beta; p.eps = eps;
    const int64_t elem = static_cast<int64_t>(dtype_bytes(dtype));
    p.xb = row_bounds(X, M, ldx * elem, D * elem);
    p.w_f32 = wdtype == QG_F32;
    p.x_vec = vec_ok(X, ldx, dtype_bytes(dtype), M);
    p.w_vec = aligned16(gamma) && aligned16(beta);
    p.y_vec = vec_ok(Y, ldy, dtype_bytes(dtype), M);
    p.Y = Y; p.ldy = ldy; p.Xq = Xq; p.Xs = Xs; p.ts = ts; p.mean = mean; p.rstd = rstd;
    return by_dtype(dtype, [&](auto t) {
        return norm_forward<decltype(t)>(fmt, p, dev, static_cast<cudaStream_t>(stream));
    });
}

#define QG_NORM_FWD(T, NAME, TPR, VPT, FMT, FNAME, VEC)                                                \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm<" NAME "," #TPR "," #VPT "," FNAME "," #VEC ">",              \
                           (reinterpret_cast<const void*>(k_layer_norm<T, TPR, VPT, FMT, VEC>)),       \
                           TPR < 128 ? 128 : TPR, 0, 0, 1, 1)
#define QG_NORM_FWD_SIZES(T, NAME, FMT, FNAME, VEC)       \
    QG_NORM_FWD(T, NAME, 256, 1, FMT, FNAME, VEC);        \
    QG_NORM_FWD(T, NAME, 1024, 1, FMT, FNAME, VEC);       \
    QG_NORM_FWD(T, NAME, 1024, 4, FMT, FNAME, VEC)
// shared memory of a full ring: the longest row the instance takes
#define QG_NORM_ROWS(T, NAME, TPR, FMT, FNAME, EDGES)                                                  \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_rows<" NAME "," #TPR "," FNAME "," #EDGES ">",                \
                           (reinterpret_cast<const void*>(k_layer_norm_rows<T, TPR, FMT, EDGES>)),     \
                           norm_threads(TPR), ring_bytes(TPR, sizeof(T)), 0, 1, norm_min_ctas(TPR))
#define QG_NORM_ROWS_SIZES(T, NAME, FMT, FNAME, EDGES) \
    QG_NORM_ROWS(T, NAME, 32, FMT, FNAME, EDGES);      \
    QG_NORM_ROWS(T, NAME, 128, FMT, FNAME, EDGES);     \
    QG_NORM_ROWS(T, NAME, 256, FMT, FNAME, EDGES);     \
    QG_NORM_ROWS(T, NAME, 512, FMT, FNAME, EDGES)
#define QG_NORM_LONG(T, NAME)                                                                              \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_long<" NAME ">", (reinterpret_cast<const void*>(k_layer_norm_long<T, kToValues>)), \
                           kLongThreads, 0, 0, 1, 1);                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_long<" NAME ",nv>", (reinterpret_cast<const void*>(k_layer_norm_long<T, kNv>)), \
                           kLongThreads, 0, 0, 1, 1);                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_long<" NAME ",mx>", (reinterpret_cast<const void*>(k_layer_norm_long<T, kMx>)), \
                           kLongThreads, 0, 0, 1, 1)
#define QG_NORM_BUDGETS(T, NAME)                              \
    QG_NORM_FWD_SIZES(T, NAME, kToValues, "y", true);         \
    QG_NORM_FWD_SIZES(T, NAME, kToValues, "y", false);        \
    QG_NORM_FWD_SIZES(T, NAME, kNv, "nv", true);              \
    QG_NORM_FWD_SIZES(T, NAME, kMx, "mx", true);              \
    QG_NORM_ROWS_SIZES(T, NAME, kToValues, "y", false);       \
    QG_NORM_ROWS_SIZES(T, NAME, kToValues, "y", true);        \
    QG_NORM_ROWS_SIZES(T, NAME, kNv, "nv", false);            \
    QG_NORM_ROWS_SIZES(T, NAME, kNv, "nv", true);             \
    QG_NORM_ROWS_SIZES(T, NAME, kMx, "mx", false);            \
    QG_NORM_ROWS_SIZES(T, NAME, kMx, "mx", true);             \
    QG_NORM_LONG(T, NAME)
QG_NORM_BUDGETS(__half, "f16");
QG_NORM_BUDGETS(__nv_bfloat16, "bf16");
QG_NORM_BUDGETS(float, "f32");

}  // namespace qg

using namespace qg;

extern "C" {

int layer_norm(int dtype, int64_t M, int64_t D, const void* X, int64_t ldx, const void* gamma, const void* beta,
               int wdtype, float eps, void* Y, int64_t ldy, float* mean, float* rstd, void* stream) {
    const NvtxRange nvtx_range("layer_norm");
    if (M > 0 && (!Y || (M > 1 && ldy < D))) return QG_ERR_INVALID_ARG;
    if (dtype_ok(dtype) && reinterpret_cast<uintptr_t>(Y) % dtype_bytes(dtype)) return QG_ERR_MISALIGNED;
    return norm_call(kToValues, dtype, M, D, X, ldx, gamma, beta, wdtype, eps, Y, ldy, nullptr, nullptr, nullptr,
                     mean, rstd, stream);
}

int layer_norm_fp4(int fmt, int dtype, int64_t M, int64_t D, const void* X, int64_t ldx, const void* gamma,
                   const void* beta, int wdtype, float eps, const float* tscale, uint8_t* Xq, uint8_t* Xs,
                   float* mean, float* rstd, void* stream) {
    const NvtxRange nvtx_range("layer_norm_fp4");
    if (!fmt_ok(fmt) || (tscale && fmt == kMx)) return QG_ERR_UNSUPPORTED;
    if (M > 0 && (!Xq || !Xs)) return QG_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Xs) || reinterpret_cast<uintptr_t>(tscale) % 4) return QG_ERR_MISALIGNED;
    return norm_call(fmt, dtype, M, D, X, ldx, gamma, beta, wdtype, eps, nullptr, 0, tscale, Xq, Xs, mean, rstd,
                     stream);
}

}  // extern "C"
