// Layer norm backward, and sums of partial rows.
//   xh = (x - mean) rstd,  d = dy gamma
//   dx = rstd (d - sum(d) / D - xh sum(d xh) / D)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
// Sums are fp32.  Bound by memory: x and dy are read and dx written once.
#include "norm_common.cuh"

namespace qg {

// ------------------------------------------------------- sums of partials
//
// out[j] = sum over i of partial[i][j], in a fixed order: 8 slices of the
// parts in parallel, then the slices in order.
constexpr int kSumCols = 32, kSumSlices = 8;

__global__ void __launch_bounds__(kSumCols* kSumSlices)
    k_sum_partials(const float* __restrict__ partial, int64_t parts, int64_t n, float* __restrict__ out0,
                   int64_t n0, float* __restrict__ out1) {
    __shared__ float acc[kSumSlices][kSumCols];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int c = threadIdx.x % kSumCols, s = threadIdx.x / kSumCols;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kSumCols + c;
    float a = 0.f;
    if (j < n) {
#pragma unroll 4
        for (int64_t i = s; i < parts; i += kSumSlices) a += partial[i * n + j];
    }
    acc[s][c] = a;
    __syncthreads();
    if (s == 0 && j < n) {
#pragma unroll
        for (int i = 1; i < kSumSlices; ++i) a += acc[i][c];
        (j < n0 ? out0[j] : out1[j - n0]) = a;
    }
}

static int sum_partials2(const float* partial, int64_t parts, int64_t n, float* out0, int64_t n0, float* out1,
                         cudaStream_t s) {
    if (n == 0) return QG_OK;
    return launch_serialized(k_sum_partials, dim3(static_cast<unsigned>((n + kSumCols - 1) / kSumCols)),
                             kSumCols * kSumSlices, 0, 1, s, partial, parts, n, out0, n0, out1);
}

int sum_partials_run(const float* partial, int64_t parts, int64_t n, float* out, cudaStream_t s) {
    return sum_partials2(partial, parts, n, out, n, out, s);
}

// ------------------------------------------------------- backward
//
// A CTA of 512 threads walks over rows, TPR threads a row, each group with a
// ring of (x, dy) row pairs in shared memory (norm_common.cuh).  A thread
// meets the same columns in every row and keeps their sums for gamma and beta
// in registers; x and dy are read from the ring twice, for the row's two sums
// and for dx, rather than held in between.  A slot is refilled one row late,
// behind the next row's only barrier.  At the end the groups add up in shared
// memory, in order, and each CTA leaves one row of partial sums.
constexpr int kBwdThreads = 512;

struct NormBwdParams {
    int64_t M, D;
    const void *dY, *X;
    int64_t lddy, ldx;
    const void* gamma;
    bool w_f32, x_vec, dy_vec, w_vec, dx_vec;
    const float *mean, *rstd;
    void* dX;
    int64_t lddx;
    float* partial;  // [gridDim.x][2][D]
};


template <class T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(kBwdThreads, 1)
    k_layer_norm_backward(const NormBwdParams p, int slots, const Ctl ctl) {
    constexpr int GROUPS = kBwdThreads / TPR;
    constexpr int E = 8 * VPT;
    constexpr int COLS = TPR * E;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ __align__(8) uint64_t bars[GROUPS][kRingMax];
    __shared__ float2 red[2][kBwdThreads / 32];
    __shared__ int abort_flag;
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int D = static_cast<int>(p.D);
    RowRing ring;
    ring.bar0 = smem_u32(&bars[group][0]);
    ring.row_bytes = p.D * static_cast<int64_t>(sizeof(T));
    ring.slot_bytes = static_cast<int>(2 * row_slot_bytes(ring.row_bytes));
    ring.slots = ring_smem + static_cast<int64_t>(group) * slots * ring.slot_bytes;
    if (t == 0) {
        for (int s = 0; s < slots; ++s) mbar_init(ring.bar0 + 8 * s, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    __syncthreads();
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const T* X = static_cast<const T*>(p.X);
    const T* dY = static_cast<const T*>(p.dY);
    const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * GROUPS + group;
    for (int s = 0; s < slots; ++s) {
        const int64_t r = row + s * step;
        if (r < p.M) row_fetch2<TPR>(ring, s, X + r * p.ldx, dY + r * p.lddy);
    }
    // without VEC gamma waits in shared memory as fp32, behind the ring
    float* const sg = reinterpret_cast<float*>(ring_smem + static_cast<int64_t>(GROUPS) * slots * ring.slot_bytes);
    if constexpr (!VEC) stage_weights<T>(sg, p.gamma, p.w_f32, D, 1.f);
    __syncthreads();
    const float inv_d = __frcp_rn(static_cast<float>(D));
    uint64_t dg[E / 2], db[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) dg[e] = db[e] = 0;

    // column of value j of step i, and whether no lane of the warp has one left
    auto column = [&](int i, int j) { return VEC ? (i * TPR + t) * 8 + j : (8 * i + j) * TPR + t; };
    auto step_done = [&](int i) { return VEC ? (i * TPR + t) * 8 >= D : 8 * i * TPR >= D; };
    auto values = [&](const T* x, int i, uint64_t(&v)[4]) {
        if constexpr (VEC) {
            load_pairs<T>(x + column(i, 0), v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = column(i, 2 * j), l = column(i, 2 * j + 1);
                v[j] = two(k < D ? to_f32<T>(x[k]) : 0.f, l < D ? to_f32<T>(x[l]) : 0.f);
            }
        }
    };
    auto gammas = [&](int i, uint64_t(&g)[4]) {
        if constexpr (VEC) {
            weight_pairs<T>(p.gamma, p.w_f32, column(i, 0), 1.f, g);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = column(i, 2 * j), l = column(i, 2 * j + 1);
                g[j] = two(k < D ? sg[k] : 0.f, l < D ? sg[l] : 0.f);
            }
        }
    };

    float mean = 0.f, rstd = 0.f;
    if (row < p.M) {
        mean = p.mean[row];
        rstd = p.rstd[row];
    }
    int s = 0, before = slots - 1;
    uint32_t phase = 0;
    int flip = 0;
    bool first = true;
    for (; row < p.M; row += step, flip ^= 1) {
        float mean_next = 0.f, rstd_next = 0.f;
        if (row + step < p.M) {
            mean_next = p.mean[row + step];
            rstd_next = p.rstd[row + step];
        }
        // a wait that runs out is recorded, ends the fetching, and lets the
        // remaining rows through with whatever their slots hold
        bounded_wait(ring.bar0 + 8 * s, phase, &abort_flag, ctl, kSiteNormRow);
        const T* x = row_in_slot<T>(ring, s, X + row * p.ldx);
        const T* dy = reinterpret_cast<const T*>(reinterpret_cast<const uint8_t*>(
                          row_in_slot<T>(ring, s, dY + row * p.lddy)) + ring.slot_bytes / 2);
        // with c = x - mean: dgamma += (dy rstd) c, and the row's sums of d and of d c
        // (behind the row dy is 0, and with it every term)
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
                const uint64_t c = add_two(u[j], minus), d = mul_two(y[j], g[j]);
                dg[4 * i + j] = fma_two(mul_two(y[j], r2), c, dg[4 * i + j]);
                db[4 * i + j] = add_two(db[4 * i + j], y[j]);
                a1 = add_two(a1, d);
                a2 = fma_two(d, c, a2);
            }
        }
        float s1 = warp_sum(both(a1).x + both(a1).y);
        float s2 = warp_sum(both(a2).x + both(a2).y);
        if constexpr (TPR > 32) {
            float2* r = red[flip] + group * (TPR / 32);
            if ((threadIdx.x & 31) == 0) r[t >> 5] = make_float2(s1, s2);
            // the TPR threads of this row only
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
            const float2 w = (threadIdx.x & 31) < TPR / 32 ? r[threadIdx.x & 31] : make_float2(0.f, 0.f);
            s1 = warp_sum(w.x);
            s2 = warp_sum(w.y);
        } else {
            __syncwarp();
        }
        // everyone is done with the row before: its slot takes the row `slots - 1` ahead of this one
        const int64_t ahead = row + (slots - 1) * step;
        if (!first && ahead < p.M && !*static_cast<volatile int*>(&abort_flag))
            row_fetch2<TPR>(ring, before, X + ahead * p.ldx, dY + ahead * p.lddy);
        first = false;
        // dx = d rstd - (sum(d) / D) rstd - c (sum(d c) / D) rstd^3
        const float k0 = -(s1 * inv_d) * rstd, k1 = -((s2 * rstd) * inv_d) * rstd * rstd;
        const uint64_t b0 = two(k0, k0), b1 = two(k1, k1);
        T* o = static_cast<T*>(p.dX) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (step_done(i)) continue;
            uint64_t u[4], y[4], g[4];
            values(x, i, u);
            values(dy, i, y);
            gammas(i, g);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = fma_two(add_two(u[j], minus), b1, fma_two(mul_two(y[j], g[j]), r2, b0));
            if constexpr (VEC) {
                store_pairs<T>(o + column(i, 0), y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = both(y[j / 2]);
                    if (column(i, j) < D) o[column(i, j)] = from_f32<T>(j & 1 ? f.y : f.x);
                }
            }
        }
        mean = mean_next;
        rstd = rstd_next;
        before = s;
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
    // the groups' sums, in order, over the idle ring; then one row of partials
    float* sums = reinterpret_cast<float*>(ring_smem);
    for (int g = 0; g < GROUPS; ++g) {
        if (group == g) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float* a = sums + column(e / 8, e % 8);
                const float2 fg = both(dg[e / 2]), fb = both(db[e / 2]);
                const float vg = e & 1 ? fg.y : fg.x, vb = e & 1 ? fb.y : fb.x;
                a[0] = g ? a[0] + vg : vg;
                a[COLS] = g ? a[COLS] + vb : vb;
            }
        }
        __syncthreads();
    }
    float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
    for (int k = threadIdx.x; k < D; k += kBwdThreads) {
        out[k] = sums[k];
        out[p.D + k] = sums[COLS + k];
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
constexpr int kMaxPartials = 512;      // rows of partial sums, at most

// Dynamic shared memory of a launch: the rings, or the sums that follow them.
static int64_t bwd_smem(int tpr, int vpt, int64_t D, size_t elem, bool vec, int* slots) {
    const int groups = kBwdThreads / tpr;
    const int64_t slot = 2 * row_slot_bytes(D * static_cast<int64_t>(elem));
    // 3: the edges of a row are visible one barrier after their copy, which itself is one row late
    *slots = ring_slots(slot, groups, 3);
    const int64_t ring = slot * *slots * groups + (vec ? 0 : (D + 7) / 8 * 32), sums = int64_t(2) * tpr * vpt * 8 * 4;
    return ring > sums ? ring : sums;
}

template <class T, int TPR, int VPT, bool VEC>
static int launch_norm_bwd(const NormBwdParams& p, int dev, int64_t* parts, cudaStream_t s) {
    constexpr int GROUPS = kBwdThreads / TPR;
    const Ctl ctl = host_ctl(dev);
    if (!ctl.status) return QG_ERR_CUDA;
    int64_t ctas = (p.M + GROUPS - 1) / GROUPS;
    if (ctas > num_sms(dev)) ctas = num_sms(dev);
    if (ctas > kMaxPartials) ctas = kMaxPartials;
    *parts = ctas;
    int slots = 0;
    const int64_t smem = bwd_smem(TPR, VPT, p.D, sizeof(T), VEC, &slots);
    auto* f = k_layer_norm_backward<T, TPR, VPT, VEC>;
    if (smem > 44 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return map_cuda(e);
    }
    return launch_serialized(f, dim3(static_cast<unsigned>(ctas)), kBwdThreads, static_cast<size_t>(smem), 1, s, p,
                             slots, ctl);
}

// Threads a row: as few as hold the row's sums (16 or 32 columns a thread), so
// that an SM has several rows in different phases; limited by three slots of
// (x, dy) a group in shared memory, which halves the columns for fp32.
template <class T, bool VEC>
static int norm_bwd_by_size(const NormBwdParams& p, int dev, int64_t* parts, cudaStream_t s) {
    constexpr bool WIDE = sizeof(T) == 4;
    if (p.D <= 256) return launch_norm_bwd<T, 32, 1, VEC>(p, dev, parts, s);
    if (p.D <= 512) return launch_norm_bwd<T, 32, 2, VEC>(p, dev, parts, s);
    if constexpr (!WIDE)
        if (p.D <= 1024) return launch_norm_bwd<T, 32, 4, VEC>(p, dev, parts, s);
    if (p.D <= 2048) return launch_norm_bwd<T, 128, 2, VEC>(p, dev, parts, s);
    if (p.D <= 4096) return launch_norm_bwd<T, 256, 2, VEC>(p, dev, parts, s);
    if constexpr (WIDE)
        return launch_norm_bwd<T, 512, 2, VEC>(p, dev, parts, s);
    else
        return launch_norm_bwd<T, 256, 4, VEC>(p, dev, parts, s);
}

template <class T>
static int norm_backward(const NormBwdParams& p, float* dgamma, float* dbeta, int dev, cudaStream_t s) {
    int64_t parts = 0;
    int rc = QG_OK;
    if (p.M > 0) {
        if (p.D <= kMaxHeldBwd) {
            rc = p.x_vec && p.dy_vec && p.dx_vec && p.w_vec && p.D % 8 == 0
                     ? norm_bwd_by_size<T, true>(p, dev, &parts, s)
                     : norm_bwd_by_size<T, false>(p, dev, &parts, s);
        } else {
            rc = launch_serialized(k_layer_norm_backward_long<T>, dim3(static_cast<unsigned>(p.M)), kLongThreads, 0,
                                   1, s, p);
            if (rc) return rc;
            const int64_t cols = (p.D + kColThreads - 1) / kColThreads;
            int64_t want = 8 * num_sms(dev) / cols + 1;  // about 8 CTAs an SM
            if (want > kMaxPartials) want = kMaxPartials;
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
    return static_cast<size_t>(kMaxPartials) * 2 * static_cast<size_t>(D) * sizeof(float);
}

static int bwd_smem_most(int tpr, int vpt, size_t elem, bool vec) {
    int slots = 0;
    return static_cast<int>(bwd_smem(tpr, vpt, int64_t(tpr) * vpt * 8, elem, vec, &slots));
}

#define QG_NORM_BWD(T, NAME, TPR, VPT, VEC)                                                            \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_backward<" NAME "," #TPR "," #VPT "," #VEC ">",               \
                           (reinterpret_cast<const void*>(k_layer_norm_backward<T, TPR, VPT, VEC>)),   \
                           kBwdThreads, bwd_smem_most(TPR, VPT, sizeof(T), VEC), 0, 1, 1)
#define QG_NORM_BWD_SIZES(T, NAME, VEC)                                                                \
    QG_NORM_BWD(T, NAME, 32, 1, VEC); QG_NORM_BWD(T, NAME, 32, 2, VEC);                                \
    QG_NORM_BWD(T, NAME, 128, 2, VEC); QG_NORM_BWD(T, NAME, 256, 2, VEC)
#define QG_NORM_BWD_16(T, NAME, VEC) QG_NORM_BWD(T, NAME, 32, 4, VEC); QG_NORM_BWD(T, NAME, 256, 4, VEC)
#define QG_NORM_BWD_BUDGETS(T, NAME)                                                                       \
    QG_NORM_BWD_SIZES(T, NAME, true);                                                                      \
    QG_NORM_BWD_SIZES(T, NAME, false);                                                                     \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_backward_long<" NAME ">",                                         \
                           reinterpret_cast<const void*>(k_layer_norm_backward_long<T>), kLongThreads, 0, 0, 1, 1); \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_columns<" NAME ">",                                               \
                           reinterpret_cast<const void*>(k_layer_norm_columns<T>), kColThreads, 0, 0, 1, 4)
QG_NORM_BWD_BUDGETS(__half, "f16");
QG_NORM_BWD_BUDGETS(__nv_bfloat16, "bf16");
QG_NORM_BWD_BUDGETS(float, "f32");
QG_NORM_BWD_16(__half, "f16", true);
QG_NORM_BWD_16(__half, "f16", false);
QG_NORM_BWD_16(__nv_bfloat16, "bf16", true);
QG_NORM_BWD_16(__nv_bfloat16, "bf16", false);
QG_NORM_BWD(float, "f32", 512, 2, true);
QG_NORM_BWD(float, "f32", 512, 2, false);
QG_BLOCK_KERNEL_BUDGET("k_sum_partials", reinterpret_cast<const void*>(k_sum_partials), kSumCols* kSumSlices, 0, 0,
                       1, 4);

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
    if (rc) return rc;
    if (!dgamma || !dbeta || (M > 0 && (!mean || !rstd))) return QG_ERR_INVALID_ARG;
    if (!ws || ws_bytes < norm_backward_workspace(D)) return QG_ERR_WORKSPACE;
    if (!aligned16(ws)) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    NormBwdParams p = {};
    p.M = M; p.D = D; p.dY = dY; p.X = X; p.lddy = lddy; p.ldx = ldx; p.gamma = gamma;
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
