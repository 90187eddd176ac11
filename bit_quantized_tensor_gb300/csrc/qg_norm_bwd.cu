// Layer norm backward, and sums of partial rows.
//   xh = (x - mean) rstd,  d = dy gamma
//   dx = rstd (d - sum(d) / D - xh sum(d xh) / D)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
// Sums are fp32.  Bound by memory: x and dy are read and dx written once.
#include <algorithm>

#include "norm_common.cuh"

namespace qg {

// ------------------------------------------------------- sums of partials
//
// out[j] = sum over i of partial[i][j], in a fixed order: SLICES slices of the
// parts in parallel, each thread with up to eight loads in flight, then the
// slices pairwise.  Few columns leave latency alone to count, and take 32 slices
// (152 x 1030: 5.8 us; 7.6 with 8, whose threads wait for three rounds of loads);
// with more than an SM has CTAs for, the instructions of a slice's end count, and
// 8 slices do (152 x 16384, 10 MB: 6.6 us from launch to end, 9.8 with 32).
constexpr int kSumCols = 32;

template <int SLICES>
__global__ void __launch_bounds__(kSumCols* SLICES)
    k_sum_partials(const float* partial, int64_t parts, int64_t n, float* __restrict__ out0,
                   int64_t n0, float* __restrict__ out1) {
    __shared__ float acc[SLICES][kSumCols + 1];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int c = threadIdx.x % kSumCols, s = threadIdx.x / kSumCols;
    const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kSumCols, step = SLICES * n;
    const float* q = partial + s * n + col0 + c;
    int left = col0 + c < n ? (static_cast<int>(parts) - s + SLICES - 1) / SLICES : 0;  // rows of this slice
    float a = 0.f;
    for (; left > 0; left -= 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u, q += step) v[u] = u < left ? *q : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) a += v[u];
    }
    acc[s][c] = a;
    __syncthreads();
    // the slices of a column in neighbouring lanes
    constexpr int PER_WARP = 32 / SLICES;
    const int lane = threadIdx.x % 32, k = threadIdx.x / 32 * PER_WARP + lane / SLICES;
    a = acc[lane % SLICES][k];
#pragma unroll
    for (int o = SLICES / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (lane % SLICES == 0 && col0 + k < n) (col0 + k < n0 ? out0[col0 + k] : out1[col0 + k - n0]) = a;
}

static int sum_partials2(const float* partial, int64_t parts, int64_t n, float* out0, int64_t n0, float* out1,
                         cudaStream_t s) {
    if (n == 0) return QG_OK;
    const int64_t ctas = (n + kSumCols - 1) / kSumCols;
    const dim3 grid(static_cast<unsigned>(ctas));
    if (ctas <= num_sms(current_device()))
        return launch_serialized(k_sum_partials<32>, grid, kSumCols * 32, 0, 1, s, partial, parts, n, out0, n0, out1);
    return launch_serialized(k_sum_partials<8>, grid, kSumCols * 8, 0, 1, s, partial, parts, n, out0, n0, out1);
}

int sum_partials_run(const float* partial, int64_t parts, int64_t n, float* out, cudaStream_t s) {
    return sum_partials2(partial, parts, n, out, n, out, s);
}

// ------------------------------------------------------- backward
//
// A CTA of 512 threads walks over rows, TPR threads a row, each group with a
// ring of (x, dy) row pairs in shared memory (norm_common.cuh).  A thread
// meets the same columns in every row and keeps gamma and their sums for
// dgamma and dbeta in registers, which leaves an SM only 16 warps.  So that the
// exchange of a row's two sums between its warps does not show, it is split:
// the warps leave their part of row i + 1, arrive at a barrier, finish dx of
// row i from the ring, and only then wait.  At the end each CTA adds up its
// groups, in order, and leaves one row of partial sums.  8192 x 8192 bf16: 76 us with
// the sums of the partial rows (5.3 TB/s), bound by the latency of a row's
// arithmetic with four warps a scheduler; both of a row's sums exchanged at once
// with its neighbour's, two rows a barrier, read the ring more often (113 us).
// Rows that start inside a piece cost masks on top: from L2, sums included,
// 16411 x 515 f16 24 us, 16411 x 512 14 us.
constexpr int kBwdThreads = 512;
__host__ __device__ constexpr int bwd_sums(int tpr, int vpt) { return 8 * vpt * (tpr + 4); }  // places of a group's sums
constexpr int kSiteNormSums = 402;

// Sums of two values over a warp with one value's shuffles: the halves of the
// warp take one each.  Lanes 0-15 end with the sum of a, the others with that of b.
template <int LANES>
__device__ __forceinline__ float half_sums(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_sums_by_half(float a, float b) {
    const bool low = (threadIdx.x & 16) == 0;
    const float other = __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
    return half_sums<16>((low ? a : b) + other);
}
// The halves' sums to every lane: (a, b).
__device__ __forceinline__ float2 from_halves(float v) {
    const float other = __shfl_xor_sync(0xffffffffu, v, 16);
    return (threadIdx.x & 16) == 0 ? make_float2(v, other) : make_float2(other, v);
}

struct NormBwdParams {
    int64_t M, D;
    const void *dY, *X;
    int64_t lddy, ldx;
    RowBounds dyb, xb;
    const void* gamma;
    bool w_f32, x_vec, dy_vec, w_vec, dx_vec;
    const float *mean, *rstd;
    void* dX;
    int64_t lddx;
    float* partial;  // [gridDim.x][2][D]
};


// VEC: all rows of a group, of x, dy and dx alike, start at the same place
// inside a 16-byte piece, and come in aligned pieces of 8 columns from there
// (EDGES; else at its start and whole).  Without VEC (rows of different places)
// the columns of a step are neighbours in neighbouring threads, and gamma waits
// in shared memory behind the ring.
template <class T, int TPR, int VPT, bool VEC, bool EDGES>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_layer_norm_backward(const NormBwdParams p, int slots, const Ctl ctl) {
    constexpr int GROUPS = kBwdThreads / TPR, WARPS = TPR / 32;
    constexpr int E = 8 * VPT;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ __align__(8) uint64_t bars[GROUPS][kRingMax];
    __shared__ __align__(8) uint64_t sum_bars[GROUPS];
    __shared__ float red[2][GROUPS][2][16];  // a row's sums, per warp: d, d xh
    __shared__ int abort_flag;
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR, lane = threadIdx.x & 31;
    const int D = static_cast<int>(p.D);
    RowRing ring;
    ring.bar0 = smem_u32(&bars[group][0]);
    ring.row_bytes = p.D * static_cast<int64_t>(sizeof(T));
    ring.slot_bytes = static_cast<int>(2 * row_slot_bytes(ring.row_bytes));
    ring.slots = ring_smem + static_cast<int64_t>(group) * slots * ring.slot_bytes;
    const uint32_t sum_bar = smem_u32(&sum_bars[group]);
    if (t == 0) {
        for (int s = 0; s < slots; ++s) mbar_init(ring.bar0 + 8 * s, 1);
        mbar_init(sum_bar, WARPS);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    pdl_wait_prior_grid();
    fence_proxy_async_global();
    pdl_launch_dependents();
    const T* X = static_cast<const T*>(p.X);
    const T* dY = static_cast<const T*>(p.dY);
    const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * GROUPS + group;
    // whole rows of whole pieces leave nothing to copy by hand; xb's ends are dyb's too
    auto at_end = [&](int64_t r) { return (!VEC || EDGES) && p.xb.at_end(r); };
    for (int s = 0; s < slots; ++s) {
        const int64_t r = row + s * step;
        if (r < p.M) row_fetch2<TPR>(ring, s, X + r * p.ldx, dY + r * p.lddy, at_end(r), p.xb, p.dyb);
    }
    float* const sg = reinterpret_cast<float*>(ring_smem + static_cast<int64_t>(GROUPS) * slots * ring.slot_bytes);
    if constexpr (!VEC) stage_weights<T>(sg, p.gamma, p.w_f32, D, 1.f);
    __syncthreads();
    const float inv_d = __frcp_rn(static_cast<float>(D));
    // values before column 0 in a row's first piece
    const int lead =
        VEC && EDGES ? static_cast<int>((reinterpret_cast<uintptr_t>(X + row * p.ldx) & 15) / sizeof(T)) : 0;
    uint64_t dg[E / 2], db[E / 2], hg[VEC ? E / 2 : 1];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dg[e] = db[e] = 0;

    // column of value j of step i, and whether the thread has none left
    auto column = [&](int i, int j) { return VEC ? (i * TPR + t) * 8 - lead + j : (8 * i + j) * TPR + t; };
    auto step_done = [&](int i) { return VEC ? column(i, 0) >= D : 8 * i * TPR >= D; };
    // what the row leaves of its first piece and of its last
    const int last_piece = (D - 1 + lead) / 8, last_step = last_piece / TPR;
    const PieceMask<T> head = piece_mask<T>(t == 0 ? -lead : 0, D < 8 ? 8 : D);
    const PieceMask<T> tail = piece_mask<T>(t == last_piece % TPR ? last_piece * 8 - lead : 0,
                                            t == last_piece % TPR ? D : 8);
    auto values = [&](const T* x, int i, uint64_t(&v)[4]) {
        if constexpr (VEC && EDGES) {
            load_piece<T>(x + column(i, 0), v, head, i == 0, tail, i == last_step);
        } else if constexpr (VEC) {
            load_pairs<T>(x + column(i, 0), v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = column(i, 2 * j), l = column(i, 2 * j + 1);
                v[j] = two(k < D ? to_f32<T>(x[k]) : 0.f, l < D ? to_f32<T>(x[l]) : 0.f);
            }
        }
    };
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            uint64_t g[4];
            weight_piece<T>(p.gamma, p.w_f32, p.w_vec, column(i, 0), D, 1.f, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) hg[4 * i + j] = g[j];
        }
    }
    auto gammas = [&](int i, uint64_t(&g)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (VEC) {
                g[j] = hg[4 * i + j];
            } else {
                const int k = column(i, 2 * j), l = column(i, 2 * j + 1);
                g[j] = two(k < D ? sg[k] : 0.f, l < D ? sg[l] : 0.f);
            }
        }
    };
    // where a row lies in its slot: x, and dy half a slot on
    const bool moves = VEC ? false : true;  // its place in a piece changes from row to row
    auto place = [&](const T* base, int64_t ld, int64_t r) {
        return static_cast<int>(moves ? reinterpret_cast<uintptr_t>(base + r * ld) & 15 : lead * sizeof(T));
    };

    // part 1 of row r in slot s: dgamma, dbeta and the warp's part of the row's sums,
    // by halves of the warp (outside the row dy is 0, and with it every term);
    // the sums are those of d and d xh: of the size of the gradient, however large or
    // small the row is (d (x - mean) and rstd^2 may not be fp32 numbers)
    auto part1 = [&](int64_t r, int s, uint32_t phase, float mean, float rstd) {
        // a wait that runs out is recorded, ends the fetching, and lets the
        // remaining rows through with whatever their slots hold
        bounded_wait(ring.bar0 + 8 * s, phase, &abort_flag, ctl, kSiteNormRow);
        const uint8_t* slot = ring.slots + static_cast<int64_t>(s) * ring.slot_bytes;
        const T* x = reinterpret_cast<const T*>(slot + place(X, p.ldx, r));
        const T* dy = reinterpret_cast<const T*>(slot + ring.slot_bytes / 2 + place(dY, p.lddy, r));
        const uint64_t minus = two(-mean, -mean), r2 = two(rstd, rstd);
        uint64_t a1 = 0, a2 = 0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (step_done(i)) continue;
            uint64_t u[4], y[4], g[4];
            values(x, i, u);
            values(dy, i, y);
            gammas(i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint64_t xh = mul_two(add_two(u[j], minus), r2), d = mul_two(y[j], g[j]);
                dg[4 * i + j] = fma_two(y[j], xh, dg[4 * i + j]);
                db[4 * i + j] = add_two(db[4 * i + j], y[j]);
                a1 = add_two(a1, d);
                a2 = fma_two(d, xh, a2);
            }
        }
        const float2 f1 = both(a1), f2 = both(a2);
        return warp_sums_by_half(f1.x + f1.y, f2.x + f2.y);
    };
    // part 2: dx = (d - sum(d) / D - (x - mean) (sum(d xh) / D rstd)) rstd
    auto part2 = [&](int64_t r, int s, float mean, float rstd, float2 sum) {
        const uint8_t* slot = ring.slots + static_cast<int64_t>(s) * ring.slot_bytes;
        const T* x = reinterpret_cast<const T*>(slot + place(X, p.ldx, r));
        const T* dy = reinterpret_cast<const T*>(slot + ring.slot_bytes / 2 + place(dY, p.lddy, r));
        const float k0 = -(sum.x * inv_d), k1 = -(sum.y * inv_d) * rstd;
        const uint64_t b0 = two(k0, k0), b1 = two(k1, k1), r2 = two(rstd, rstd), minus = two(-mean, -mean);
        T* o = static_cast<T*>(p.dX) + r * p.lddx;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (step_done(i)) continue;
            uint64_t u[4], y[4], g[4];
            values(x, i, u);
            values(dy, i, y);
            gammas(i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = mul_two(fma_two(add_two(u[j], minus), b1, fma_two(y[j], g[j], b0)), r2);
            if constexpr (VEC && EDGES) {
                store_piece<T>(o, column(i, 0), D, true, y);
            } else if constexpr (VEC) {
                store_pairs<T>(o + column(i, 0), y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = both(y[j / 2]);
                    if (column(i, j) < D) o[column(i, j)] = from_f32<T>(j & 1 ? f.y : f.x);
                }
            }
        }
    };

    int s = 0, n = 0;  // slot and number of the row that part 1 takes next
    uint32_t phase = 0;
    float mean = 0.f, rstd = 0.f, mean1 = 0.f, rstd1 = 0.f;
    float2 sum = make_float2(0.f, 0.f);
    if (row < p.M) {
        mean1 = p.mean[row];
        rstd1 = p.rstd[row];
    }
    // in each round: part 1 of row `row`, part 2 of the row before it
    int s_before = 0;
    for (; row < p.M + step; row += step, ++n) {
        const bool here = row < p.M, next = row + step < p.M;
        float v = 0.f, mean2 = 0.f, rstd2 = 0.f;
        if (next) {
            mean2 = p.mean[row + step];
            rstd2 = p.rstd[row + step];
        }
        if (here) {
            v = part1(row, s, phase, mean1, rstd1);
            if constexpr (TPR > 32) {
                if ((lane & 15) == 0) red[n & 1][group][lane >> 4][t >> 5] = v;
                __syncwarp();
                if (lane == 0) mbar_arrive(sum_bar);
            }
        }
        if (n > 0) part2(row - step, s_before, mean, rstd, sum);
        if (here) {
            if constexpr (TPR > 32) {
                bounded_wait(sum_bar, n & 1, &abort_flag, ctl, kSiteNormSums);
                v = (lane & 15) < WARPS ? red[n & 1][group][lane >> 4][lane & 15] : 0.f;
                v = half_sums<WARPS>(v);
                v = __shfl_sync(0xffffffffu, v, lane & 16);
            } else {
                __syncwarp();
            }
            sum = from_halves(v);
        }
        // every warp has arrived for this row, so it is done with part 2 of the one two
        // rows back: that slot takes the row `slots - 2` ahead of this one
        const int64_t ahead = row + (slots - 2) * step;
        if (n > 1 && ahead < p.M && !*static_cast<volatile int*>(&abort_flag)) {
            const int free_slot = s >= 2 ? s - 2 : s + slots - 2;
            row_fetch2<TPR>(ring, free_slot, X + ahead * p.ldx, dY + ahead * p.lddy, at_end(ahead), p.xb, p.dyb);
        }
        if (n > 1 && ahead < p.M && at_end(ahead)) {  // what threads copied of the last rows
            if constexpr (TPR > 32)
                asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
            else
                __syncwarp();
        }
        mean = mean1;
        rstd = rstd1;
        mean1 = mean2;
        rstd1 = rstd2;
        s_before = s;
        if (++s == slots) {
            s = 0;
            phase ^= 1u;
        }
    }
    __syncthreads();
    if (abort_flag) {  // copies may still be in flight: give them a fixed time to land
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000) {
        }
    }
    // every group's sums over the idle ring, then one row of partials.  Value e of
    // thread t lies at e (TPR + 4) + t, where neighbouring threads write and
    // neighbouring columns are read without meeting in a bank (column by column,
    // eight lanes met in one, and the end of a CTA took 2 to 3 us)
    float* sums = reinterpret_cast<float*>(ring_smem);  // [GROUPS][2][SUMS]
    constexpr int SUMS = bwd_sums(TPR, VPT);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float2 fg = both(dg[e / 2]), fb = both(db[e / 2]);
        sums[2 * group * SUMS + e * (TPR + 4) + t] = e & 1 ? fg.y : fg.x;
        sums[(2 * group + 1) * SUMS + e * (TPR + 4) + t] = e & 1 ? fb.y : fb.x;
    }
    __syncthreads();
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
    const T* const first_row = X + static_cast<int64_t>(blockIdx.x) * GROUPS * p.ldx;
    for (int k = threadIdx.x; k < D; k += kBwdThreads) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            // the thread and value that held column k in this group
            int e = k / TPR, u = k % TPR;
            if constexpr (VEC) {
                const int l = k + (EDGES ? static_cast<int>((reinterpret_cast<uintptr_t>(first_row + g * p.ldx) & 15) / sizeof(T)) : 0);
                u = l / 8 % TPR;
                e = l / 8 / TPR * 8 + l % 8;
            }
            a += sums[2 * g * SUMS + e * (TPR + 4) + u];
            b += sums[(2 * g + 1) * SUMS + e * (TPR + 4) + u];
        }
        out[k] = a;
        out[p.D + k] = b;
    }
}

// Rows longer than 8192: dx in one kernel (two passes over the row, the second
// from L2), the sums over the rows in another (one thread a column, a slice of
// the rows a CTA).
template <class T>
__global__ void __launch_bounds__(kLongThreads) k_layer_norm_backward_long(const NormBwdParams p) {
    __shared__ float red[2][32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x, D = p.D;
    const T* x = static_cast<const T*>(p.X) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dY) + row * p.lddy;
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t k = threadIdx.x * 8; k < D; k += kLongThreads * 8) {
        const int n = static_cast<int>(min(D - k, int64_t(8)));
        float u[8], v[8], g[8];
        load_some<T, 8>(x + k, n, p.x_vec, u);
        load_some<T, 8>(dy + k, n, p.dy_vec, v);
        weights8<T>(p.gamma, p.w_f32, p.w_vec, k, n, 1.f, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = v[j] * g[j];  // 0 behind the row
            s1 += d;
            s2 = fmaf(d, (u[j] - mean) * rstd, s2);
        }
    }
    s1 = row_sum<kLongThreads>(s1, red[0]) / static_cast<float>(D);
    s2 = row_sum<kLongThreads>(s2, red[1]) / static_cast<float>(D);
    for (int64_t k = threadIdx.x * 8; k < D; k += kLongThreads * 8) {
        const int n = static_cast<int>(min(D - k, int64_t(8)));
        float u[8], v[8], g[8], y[8];
        load_some<T, 8>(x + k, n, p.x_vec, u);
        load_some<T, 8>(dy + k, n, p.dy_vec, v);
        weights8<T>(p.gamma, p.w_f32, p.w_vec, k, n, 1.f, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = rstd * (v[j] * g[j] - s1 - (u[j] - mean) * rstd * s2);
        store_some<T, 8>(static_cast<T*>(p.dX) + row * p.lddx + k, n, p.dx_vec, y);
    }
}

constexpr int kColThreads = 256;

template <class T>
__global__ void __launch_bounds__(kColThreads) k_layer_norm_columns(const NormBwdParams p, int64_t rows_per_cta) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int64_t k = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
    if (k >= p.D) return;
    const int64_t r0 = blockIdx.y * rows_per_cta, r1 = min(p.M, r0 + rows_per_cta);
    float dg = 0.f, db = 0.f;
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        const float y = to_f32<T>(static_cast<const T*>(p.dY)[r * p.lddy + k]);
        const float x = to_f32<T>(static_cast<const T*>(p.X)[r * p.ldx + k]);
        dg = fmaf(y, (x - p.mean[r]) * p.rstd[r], dg);
        db += y;
    }
    p.partial[blockIdx.y * 2 * p.D + k] = dg;
    p.partial[(blockIdx.y * 2 + 1) * p.D + k] = db;
}

// ------------------------------------------------------- host side

constexpr int64_t kMaxHeldBwd = 8192;  // longest row that k_layer_norm_backward takes

// Rows of partial sums, at most: one a CTA of k_layer_norm_backward, of which a GB300's
// 152 SMs take one each, or of k_layer_norm_columns, of which eight an SM share 33
// blocks of columns and more.
static int max_partials(int64_t D) { return D <= kMaxHeldBwd ? 160 : 40; }

// Dynamic shared memory of a launch: the rings, or the sums that follow them.
static int64_t bwd_smem(int tpr, int vpt, int64_t D, size_t elem, bool vec, int* slots) {
    const int groups = kBwdThreads / tpr;
    const int64_t slot = 2 * row_slot_bytes(D * static_cast<int64_t>(elem));
    *slots = ring_slots(slot, groups, 3, 200 * 1024);  // two rows are in use at a time
    const int64_t ring = slot * *slots * groups + (vec ? 0 : (D + 7) / 8 * 32);
    const int64_t sums = int64_t(groups) * 2 * bwd_sums(tpr, vpt) * 4;
    return ring > sums ? ring : sums;
}

template <class T, int TPR, int VPT, bool VEC, bool EDGES>
static int launch_norm_bwd(const NormBwdParams& p, int64_t same, int dev, int64_t* parts, cudaStream_t s) {
    constexpr int GROUPS = kBwdThreads / TPR;
    const Ctl ctl = host_ctl(dev);
    if (!ctl.status) return QG_ERR_CUDA;
    const int most = std::min(num_sms(dev), max_partials(p.D));
    const int64_t ctas = norm_ctas(p.M, GROUPS, most, same);
    *parts = ctas;
    int slots = 0;
    const int64_t smem = bwd_smem(TPR, VPT, p.D, sizeof(T), VEC, &slots);
    auto* f = k_layer_norm_backward<T, TPR, VPT, VEC, EDGES>;
    struct Flags {};
    const int rc = raise_smem<Flags>(f);
    if (rc) return rc;
    return launch_serialized(f, dim3(static_cast<unsigned>(ctas)), kBwdThreads, static_cast<size_t>(smem), 1, s, p,
                             slots, ctl);
}

// Threads a row: a warp while its lanes can hold the row's sums (up to 24
// columns each; fp32 rows 16, for their slots), above that as few as hold them
// in 16 columns each.  Measured against the next count, 2^26 bf16 values, us: rows of
// 512 69 (194 with 128 threads), 768 66 (132), 2048 78 (122 with 256), 4096 83 (111).
template <class T, bool VEC, bool EDGES>
static int norm_bwd_by_size(const NormBwdParams& p, int64_t same, int dev, int64_t* parts, cudaStream_t s) {
    const int64_t D = p.D + (VEC && EDGES ? 8 : 0);  // its place in the first piece
    if (D <= 256) return launch_norm_bwd<T, 32, 1, VEC, EDGES>(p, same, dev, parts, s);
    if (D <= 512) return launch_norm_bwd<T, 32, 2, VEC, EDGES>(p, same, dev, parts, s);
    if constexpr (VEC && sizeof(T) == 2)
        if (D <= 768) return launch_norm_bwd<T, 32, 3, VEC, EDGES>(p, same, dev, parts, s);
    if (D <= 1024) return launch_norm_bwd<T, 128, 1, VEC, EDGES>(p, same, dev, parts, s);
    if (D <= 2048) return launch_norm_bwd<T, 128, 2, VEC, EDGES>(p, same, dev, parts, s);
    if (D <= 4096) return launch_norm_bwd<T, 256, 2, VEC, EDGES>(p, same, dev, parts, s);
    return launch_norm_bwd<T, 512, 2, VEC, EDGES>(p, same, dev, parts, s);
}

template <class T>
static int norm_backward(const NormBwdParams& p, float* dgamma, float* dbeta, int dev, cudaStream_t s) {
    int64_t parts = 0;
    int rc = QG_OK;
    if (p.M > 0) {
        if (p.D <= kMaxHeldBwd) {
            // do rows of x, dy and dx start at the same places?
            const uintptr_t x = reinterpret_cast<uintptr_t>(p.X) % 16;
            const size_t lx = static_cast<size_t>(p.ldx) * sizeof(T) % 16;
            const bool alike = reinterpret_cast<uintptr_t>(p.dY) % 16 == x && reinterpret_cast<uintptr_t>(p.dX) % 16 == x &&
                               (p.M == 1 || (static_cast<size_t>(p.lddy) * sizeof(T) % 16 == lx &&
                                             static_cast<size_t>(p.lddx) * sizeof(T) % 16 == lx));
            const bool edges = lx || x || p.D % 8;
            if (alike && !edges)
                rc = norm_bwd_by_size<T, true, false>(p, 1, dev, &parts, s);
            else if (alike && p.D + 8 <= kMaxHeldBwd)
                rc = norm_bwd_by_size<T, true, true>(p, same_place_rows(p.ldx, sizeof(T)), dev, &parts, s);
            else
                rc = norm_bwd_by_size<T, false, false>(p, 1, dev, &parts, s);
        } else {
            rc = launch_serialized(k_layer_norm_backward_long<T>, dim3(static_cast<unsigned>(p.M)), kLongThreads, 0,
                                   1, s, p);
            if (rc) return rc;
            const int64_t cols = (p.D + kColThreads - 1) / kColThreads;
            int64_t want = 8 * num_sms(dev) / cols + 1;  // about 8 CTAs an SM
            if (want > max_partials(p.D)) want = max_partials(p.D);
            const int64_t per = (p.M + want - 1) / want;
            parts = (p.M + per - 1) / per;
            rc = launch_serialized(k_layer_norm_columns<T>,
                                   dim3(static_cast<unsigned>(cols), static_cast<unsigned>(parts)), kColThreads, 0, 1,
                                   s, p, per);
        }
    }
    if (rc) return rc;
    return sum_partials2(p.partial, parts, 2 * p.D, dgamma, p.D, dbeta, s);
}

size_t norm_backward_workspace(int64_t D) {
    return static_cast<size_t>(max_partials(D)) * 2 * static_cast<size_t>(D) * sizeof(float);
}

static int bwd_smem_most(int tpr, int vpt, size_t elem, bool vec) {
    int slots = 0;
    return static_cast<int>(bwd_smem(tpr, vpt, int64_t(tpr) * vpt * 8, elem, vec, &slots));
}

#define QG_NORM_BWD(T, NAME, TPR, VPT, VEC, EDGES)                                                     \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_backward<" NAME "," #TPR "," #VPT "," #VEC "," #EDGES ">",    \
                           (reinterpret_cast<const void*>(k_layer_norm_backward<T, TPR, VPT, VEC, EDGES>)), \
                           kBwdThreads, bwd_smem_most(TPR, VPT, sizeof(T), VEC), 0, 1, 1)
#define QG_NORM_BWD_SIZES(T, NAME, VEC, EDGES)                                                         \
    QG_NORM_BWD(T, NAME, 32, 1, VEC, EDGES); QG_NORM_BWD(T, NAME, 32, 2, VEC, EDGES);                  \
    QG_NORM_BWD(T, NAME, 128, 1, VEC, EDGES); QG_NORM_BWD(T, NAME, 128, 2, VEC, EDGES);                \
    QG_NORM_BWD(T, NAME, 256, 2, VEC, EDGES); QG_NORM_BWD(T, NAME, 512, 2, VEC, EDGES)
#define QG_NORM_BWD_BUDGETS(T, NAME)                                                                       \
    QG_NORM_BWD_SIZES(T, NAME, true, false);                                                               \
    QG_NORM_BWD_SIZES(T, NAME, true, true);                                                                \
    QG_NORM_BWD_SIZES(T, NAME, false, false);                                                              \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_backward_long<" NAME ">",                                         \
                           reinterpret_cast<const void*>(k_layer_norm_backward_long<T>), kLongThreads, 0, 0, 1, 1); \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_columns<" NAME ">",                                               \
                           reinterpret_cast<const void*>(k_layer_norm_columns<T>), kColThreads, 0, 0, 1, 4)
QG_NORM_BWD_BUDGETS(__half, "f16");
QG_NORM_BWD_BUDGETS(__nv_bfloat16, "bf16");
QG_NORM_BWD_BUDGETS(float, "f32");
QG_NORM_BWD(__half, "f16", 32, 3, true, false);
QG_NORM_BWD(__half, "f16", 32, 3, true, true);
QG_NORM_BWD(__nv_bfloat16, "bf16", 32, 3, true, false);
QG_NORM_BWD(__nv_bfloat16, "bf16", 32, 3, true, true);
QG_BLOCK_KERNEL_BUDGET("k_sum_partials<32>", reinterpret_cast<const void*>(k_sum_partials<32>), kSumCols * 32, 0, 0,
                       1, 1);
QG_BLOCK_KERNEL_BUDGET("k_sum_partials<8>", reinterpret_cast<const void*>(k_sum_partials<8>), kSumCols * 8, 0, 0, 1, 4);

}  // namespace qg

using namespace qg;

extern "C" {

int layer_norm_backward(int dtype, int64_t M, int64_t D, const void* dY, int64_t lddy, const void* X, int64_t ldx,
                        const void* gamma, int wdtype, const float* mean, const float* rstd, void* dX, int64_t lddx,
                        float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("layer_norm_backward");
    int rc = check_norm(dtype, wdtype, M, D, 0.f);
    if (!rc) rc = check_rows(dtype, M, D, X, ldx);
    if (!rc) rc = check_rows(dtype, M, D, dY, lddy);
    if (!rc) rc = check_rows(dtype, M, D, dX, lddx);
    if (!rc) rc = check_weight(gamma, wdtype);
    for (const float* v : {mean, rstd, static_cast<const float*>(dgamma), static_cast<const float*>(dbeta)})
        if (!rc) rc = check_f32(v);
    if (rc) return rc;
    if (!dgamma || !dbeta || (M > 0 && (!mean || !rstd))) return QG_ERR_INVALID_ARG;
    if (!ws || ws_bytes < norm_backward_workspace(D)) return QG_ERR_WORKSPACE;
    if (!aligned16(ws)) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    NormBwdParams p = {};
    p.M = M; p.D = D; p.dY = dY; p.X = X; p.lddy = lddy; p.ldx = ldx; p.gamma = gamma;
    const int64_t elem = static_cast<int64_t>(dtype_bytes(dtype));
    p.xb = row_bounds(X, M, ldx * elem, D * elem);
    p.dyb = row_bounds(dY, M, lddy * elem, D * elem);
    p.xb.near = std::max(p.xb.near, p.dyb.near);
    p.xb.far = M - p.xb.near;
    p.w_f32 = wdtype == QG_F32;
    p.x_vec = vec_ok(X, ldx, dtype_bytes(dtype), M);
    p.dy_vec = vec_ok(dY, lddy, dtype_bytes(dtype), M);
    p.dx_vec = vec_ok(dX, lddx, dtype_bytes(dtype), M);
    p.w_vec = aligned16(gamma);
    p.mean = mean; p.rstd = rstd; p.dX = dX; p.lddx = lddx;
    p.partial = static_cast<float*>(ws);
    return by_dtype(dtype, [&](auto t) {
        return norm_backward<decltype(t)>(p, dgamma, dbeta, dev, static_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
