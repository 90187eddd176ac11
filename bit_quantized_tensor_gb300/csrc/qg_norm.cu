// Layer norm: forward (to values, or straight to microscaled 4-bit codes) and
// backward with the sums over the rows for gamma and beta.
//
//   mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),
//   xh = (x - mean) rstd,  y = xh gamma + beta
//   d = dy gamma,  dx = rstd (d - sum(d) / D - xh sum(d xh) / D)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// All statistics and sums are fp32.  Everything here is bound by memory: the
// forward reads x and writes y once, the backward reads x and dy and writes dx
// once.  A row lives in the registers of its threads between the passes.
#include "fp4_common.cuh"
#include "qg_ptx.cuh"

namespace qg {

// A value of gamma or beta: fp32, or the type T of the rows.
template <class T>
__device__ __forceinline__ float weight_at(const void* w, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(w)[i] : to_f32<T>(static_cast<const T*>(w)[i]);
}

// 8 values from index i on, i a multiple of 8 and w 16-byte aligned when `vec`.
template <class T>
__device__ __forceinline__ void weights8(const void* w, bool f32, bool vec, int64_t i, int n, float none,
                                         float (&g)[8]) {
    if (!w) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = none;
    } else if (f32) {
        load_some<float, 8>(static_cast<const float*>(w) + i, n, vec, g);
    } else {
        load_some<T, 8>(static_cast<const T*>(w) + i, n, vec, g);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the TPR threads of a row (the whole CTA where TPR > 32), the same
// value in all of them.  `red` holds one value a warp; two calls in a row use
// two of them, so one barrier a call is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = warp_sum((threadIdx.x & 31) < TPR / 32 ? red[threadIdx.x & 31] : 0.f);
    }
    return v;
}

// Eight consecutive normalised values of a row per lane to codes: the lanes of
// a block find its maximum with shuffles, each lane stores its word of codes,
// and the first lane of every four blocks their scale word.  All lanes of the
// warp take part; positions behind D hold 0.
template <int FMT>
__device__ __forceinline__ void quantize_lane8(const float (&y)[8], int64_t k, int64_t D, int64_t row, float ts,
                                               float six_ts, uint8_t* Xq, uint8_t* Xs) {
    constexpr int LANES = fp4_block(FMT) / 8;
    uint32_t m = absmax_bits<8>(y);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s = block_scale<FMT>(m, ts, six_ts);
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fmul_rn(y[j], s.r);
    const int64_t ld = fp4_codes_ld(D), tiles = fp4_col_tiles(FMT, D);
    if (k < 2 * ld) *reinterpret_cast<uint32_t*>(Xq + row * ld + k / 2) = e2m1x8(q);
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
    const void *gamma, *beta;
    bool w_f32, x_vec, w_vec, y_vec;
    float eps;
    void* Y;        // FMT < 0
    int64_t ldy;
    uint8_t *Xq, *Xs;  // FMT >= 0
    const float* ts;
    float *mean, *rstd;
};

// Rows whose scale words behind the last row are zeroed (up to whole tiles).
template <int FMT>
__device__ __forceinline__ void zero_scale_rows(int64_t M, int64_t D, uint8_t* Xs) {
    const int64_t tiles = fp4_col_tiles(FMT, D), pad = (M + 127) / 128 * 128 - M;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < pad * tiles;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        *reinterpret_cast<uint32_t*>(Xs + fp4_scale_offset(M + i / tiles, 4 * (i % tiles), tiles)) = 0;
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
    if constexpr (FMT >= 0) zero_scale_rows<FMT>(p.M, p.D, p.Xs);
    if (row >= p.M) return;  // whole warps: TPR >= 32
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
    const float ts = FMT == kNv && p.ts ? *p.ts : 1.f;
    const float six_ts = __fmul_rn(6.f, ts);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            const int k = (i * TPR + t) * 8;
            if (i > 0 && (i * TPR + (t & ~31)) * 8 >= (D + 127) / 128 * 128) continue;  // the warp is past the row
            float g[8], b[8], y[8];
            weights8<T>(p.gamma, p.w_f32, p.w_vec, k, D - k, 1.f, g);
            weights8<T>(p.beta, p.w_f32, p.w_vec, k, D - k, 0.f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                y[j] = k + j < D ? fmaf((v[8 * i + j] - mean) * rstd, g[j], b[j]) : 0.f;
            if constexpr (FMT >= 0)
                quantize_lane8<FMT>(y, k, p.D, row, ts, six_ts, p.Xq, p.Xs);
            else if (k < D)
                store_some<T, 8>(static_cast<T*>(p.Y) + row * p.ldy + k, D - k, p.y_vec, y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = (8 * i + j) * TPR + t;
                if (k >= D) continue;
                const float g = p.gamma ? weight_at<T>(p.gamma, p.w_f32, k) : 1.f;
                const float b = p.beta ? weight_at<T>(p.beta, p.w_f32, k) : 0.f;
                static_cast<T*>(p.Y)[row * p.ldy + k] = from_f32<T>(fmaf((v[8 * i + j] - mean) * rstd, g, b));
            }
        }
    }
}

// Rows longer than the registers of a CTA hold: three passes over the row,
// the second and third from L2.
constexpr int kLongThreads = 1024;

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
    const float ts = FMT == kNv && p.ts ? *p.ts : 1.f;
    const float six_ts = __fmul_rn(6.f, ts);
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
            quantize_lane8<FMT>(y, k, D, row, ts, six_ts, p.Xq, p.Xs);
        else if (n > 0)
            store_some<T, 8>(static_cast<T*>(p.Y) + row * p.ldy + k, n, p.y_vec, y);
    }
}

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
// A CTA of 512 threads walks over rows, TPR threads a row, and keeps the sums
// for gamma and beta of its rows in registers: each thread meets the same
// 8 VPT columns in every row.  The next row's x and dy are loaded before the
// current row's two sums are formed, so the loads stay in flight across the
// row's barrier.  At the end the CTA's groups add up in shared memory, in
// order, and each CTA leaves one row of partial sums.
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

// 8 values as they are in memory (packed for 16-bit types).
template <class T>
struct Raw8 {
    uint4 w[sizeof(T) == 4 ? 2 : 1];
};
template <class T>
__device__ __forceinline__ Raw8<T> raw_zero() {
    Raw8<T> r;
    r.w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(T) == 4) r.w[1] = r.w[0];
    return r;
}
template <class T>
__device__ __forceinline__ void raw_values(const Raw8<T>& r, float (&x)[8]) {
    load_vec<T, 8>(reinterpret_cast<const T*>(r.w), x);
}

template <class T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(kBwdThreads, 1) k_layer_norm_backward(const NormBwdParams p) {
    constexpr int GROUPS = kBwdThreads / TPR;
    constexpr int E = 8 * VPT;
    constexpr int COLS = TPR * E;
    extern __shared__ float sums[];  // 2 x COLS
    __shared__ float2 red[2][kBwdThreads / 32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int D = static_cast<int>(p.D);
    const float inv_d = __frcp_rn(static_cast<float>(D));
    const int64_t step = static_cast<int64_t>(gridDim.x) * GROUPS;
    float dg[E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) dg[e] = db[e] = 0.f;

    auto load = [&](const void* base, int64_t ld, bool vec, int64_t row, Raw8<T>(&r)[VPT]) {
        const T* x = static_cast<const T*>(base) + row * ld;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            r[i] = raw_zero<T>();
            if (row >= p.M) continue;
            T* e = reinterpret_cast<T*>(r[i].w);
            if constexpr (VEC) {
                const int k = (i * TPR + t) * 8;
                if (vec && k + 8 <= D) {
                    r[i].w[0] = reinterpret_cast<const uint4*>(x + k)[0];
                    if constexpr (sizeof(T) == 4) r[i].w[1] = reinterpret_cast<const uint4*>(x + k)[1];
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (k + j < D) e[j] = x[k + j];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = (8 * i + j) * TPR + t;
                    if (k < D) e[j] = x[k];
                }
            }
        }
    };
    auto index = [&](int e) { return VEC ? ((e >> 3) * TPR + t) * 8 + (e & 7) : e * TPR + t; };

    int64_t row = static_cast<int64_t>(blockIdx.x) * GROUPS + group;
    Raw8<T> rx[VPT], ry[VPT];
    float mean = 0.f, rstd = 0.f;
    load(p.X, p.ldx, p.x_vec, row, rx);
    load(p.dY, p.lddy, p.dy_vec, row, ry);
    if (row < p.M) {
        mean = p.mean[row];
        rstd = p.rstd[row];
    }
    int flip = 0;
    for (; row < p.M; row += step, flip ^= 1) {
        float xh[E], d[E];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float x[8], y[8], g[8];
            raw_values<T>(rx[i], x);
            raw_values<T>(ry[i], y);
            if constexpr (VEC) {
                const int k = (i * TPR + t) * 8;
                weights8<T>(p.gamma, p.w_f32, p.w_vec, k, D - k, 1.f, g);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = (8 * i + j) * TPR + t;
                    g[j] = k < D && p.gamma ? weight_at<T>(p.gamma, p.w_f32, k) : 1.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = 8 * i + j;
                xh[e] = index(e) < D ? (x[j] - mean) * rstd : 0.f;
                dg[e] = fmaf(y[j], xh[e], dg[e]);
                db[e] += y[j];
                d[e] = y[j] * g[j];
                s1 += d[e];
                s2 = fmaf(d[e], xh[e], s2);
            }
        }
        const float scale = rstd;
        load(p.X, p.ldx, p.x_vec, row + step, rx);
        load(p.dY, p.lddy, p.dy_vec, row + step, ry);
        if (row + step < p.M) {
            mean = p.mean[row + step];
            rstd = p.rstd[row + step];
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if constexpr (TPR > 32) {
            float2* r = red[flip] + group * (TPR / 32);
            if ((threadIdx.x & 31) == 0) r[t >> 5] = make_float2(s1, s2);
            // the TPR threads of this row only
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(TPR) : "memory");
            const float2 u = (threadIdx.x & 31) < TPR / 32 ? r[threadIdx.x & 31] : make_float2(0.f, 0.f);
            s1 = warp_sum(u.x);
            s2 = warp_sum(u.y);
        }
        s1 *= inv_d;
        s2 *= inv_d;
        T* o = static_cast<T*>(p.dX) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = 8 * i + j;
                y[j] = scale * (d[e] - s1 - xh[e] * s2);
            }
            if constexpr (VEC) {
                const int k = (i * TPR + t) * 8;
                if (k < D) store_some<T, 8>(o + k, D - k, p.dx_vec, y);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = (8 * i + j) * TPR + t;
                    if (k < D) o[k] = from_f32<T>(y[j]);
                }
            }
        }
    }
    // the groups' sums, in order, then one row of partials
    for (int g = 0; g < GROUPS; ++g) {
        if (group == g) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float* a = sums + index(e);
                a[0] = g ? a[0] + dg[e] : dg[e];
                a[COLS] = g ? a[COLS] + db[e] : db[e];
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

constexpr int64_t kMaxHeldFwd = 1024 * 32;   // longest row that k_layer_norm holds
constexpr int64_t kMaxHeldBwd = 512 * 16;    // longest row that k_layer_norm_backward holds
constexpr int kMaxPartials = 512;            // rows of partial sums, at most

static bool vec_ok(const void* p, int64_t ld, size_t elem, int64_t rows) {
    return aligned16(p) && (rows <= 1 || (static_cast<size_t>(ld) * elem) % 16 == 0);
}

template <class T, int TPR, int VPT, int FMT, bool VEC>
static int launch_norm(const NormParams& p, cudaStream_t s) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR;
    constexpr int ROWS = THREADS / TPR;
    return launch_serialized(k_layer_norm<T, TPR, VPT, FMT, VEC>,
                             dim3(static_cast<unsigned>((p.M + ROWS - 1) / ROWS)), THREADS, 0, 1, s, p);
}

// Threads a row: with enough rows to fill the SMs, as few as hold the row in 32
// registers each (many rows in flight, few barriers); with fewer rows than SMs,
// one step of 8 values a thread, since then the row's own latency is all there is.
template <class T, int FMT, bool VEC>
static int norm_by_size(const NormParams& p, int dev, cudaStream_t s) {
    // codes are written up to whole scale words, so a row ends at a multiple of 128 there
    const int64_t D = FMT < 0 ? p.D : (p.D + 127) / 128 * 128;
    if (p.M <= num_sms(dev)) {
        if (D <= 2048) return launch_norm<T, 256, 1, FMT, VEC>(p, s);
        if (D <= 8192) return launch_norm<T, 1024, 1, FMT, VEC>(p, s);
    }
    if (D <= 1024) return launch_norm<T, 32, 4, FMT, VEC>(p, s);
    if (D <= 4096) return launch_norm<T, 128, 4, FMT, VEC>(p, s);
    if (D <= 8192) return launch_norm<T, 256, 4, FMT, VEC>(p, s);
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

template <class T, int TPR, int VPT, bool VEC>
static int launch_norm_bwd(const NormBwdParams& p, int64_t ctas, cudaStream_t s) {
    constexpr int SMEM = 2 * TPR * VPT * 8 * 4;
    auto* f = k_layer_norm_backward<T, TPR, VPT, VEC>;
    if constexpr (SMEM > 48 * 1024 - 512) {
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return map_cuda(e);
    }
    return launch_serialized(f, dim3(static_cast<unsigned>(ctas)), kBwdThreads, SMEM, 1, s, p);
}

template <class T, bool VEC>
static int norm_bwd_by_size(const NormBwdParams& p, int dev, int64_t* parts, cudaStream_t s) {
    const int64_t D = p.D;
    const int groups = D <= 512 ? 16 : D <= 2048 ? 4 : 1;
    int64_t ctas = (p.M + groups - 1) / groups;
    if (ctas > num_sms(dev)) ctas = num_sms(dev);
    if (ctas > kMaxPartials) ctas = kMaxPartials;
    *parts = ctas;
    if (D <= 256) return launch_norm_bwd<T, 32, 1, VEC>(p, ctas, s);
    if (D <= 512) return launch_norm_bwd<T, 32, 2, VEC>(p, ctas, s);
    if (D <= 1024) return launch_norm_bwd<T, 128, 1, VEC>(p, ctas, s);
    if (D <= 2048) return launch_norm_bwd<T, 128, 2, VEC>(p, ctas, s);
    if (D <= 4096) return launch_norm_bwd<T, 512, 1, VEC>(p, ctas, s);
    return launch_norm_bwd<T, 512, 2, VEC>(p, ctas, s);
}

template <class T>
static int norm_backward(const NormBwdParams& p, float* dgamma, float* dbeta, int dev, cudaStream_t s) {
    int64_t parts = 0;
    int rc = QG_OK;
    if (p.M > 0) {
        if (p.D <= kMaxHeldBwd) {
            rc = p.x_vec && p.dy_vec && p.dx_vec ? norm_bwd_by_size<T, true>(p, dev, &parts, s)
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

static int check_rows(int dtype, int64_t M, int64_t D, const void* X, int64_t ldx) {
    if (M && !X) return QG_ERR_INVALID_ARG;
    if (M > 1 && ldx < D) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype)) return QG_ERR_MISALIGNED;
    return QG_OK;
}

static int check_weight(const void* w, int dtype) {
    return reinterpret_cast<uintptr_t>(w) % dtype_bytes(dtype) ? QG_ERR_MISALIGNED : QG_OK;
}

static int check_norm(int dtype, int wdtype, int64_t M, int64_t D, float eps) {
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
    if (rc) return rc;
    if (M == 0) return QG_OK;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    NormParams p = {};
    p.M = M; p.D = D; p.X = X; p.ldx = ldx; p.gamma = gamma; p.beta = beta; p.eps = eps;
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
    QG_NORM_FWD(T, NAME, 32, 4, FMT, FNAME, VEC);         \
    QG_NORM_FWD(T, NAME, 128, 4, FMT, FNAME, VEC);        \
    QG_NORM_FWD(T, NAME, 256, 4, FMT, FNAME, VEC);        \
    QG_NORM_FWD(T, NAME, 1024, 4, FMT, FNAME, VEC)
#define QG_NORM_BWD(T, NAME, TPR, VPT, VEC)                                                            \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_backward<" NAME "," #TPR "," #VPT "," #VEC ">",               \
                           (reinterpret_cast<const void*>(k_layer_norm_backward<T, TPR, VPT, VEC>)),   \
                           kBwdThreads, 2 * TPR * VPT * 8 * 4, 0, 1, 1)
#define QG_NORM_BWD_SIZES(T, NAME, VEC)                                                                \
    QG_NORM_BWD(T, NAME, 32, 1, VEC); QG_NORM_BWD(T, NAME, 32, 2, VEC);                                \
    QG_NORM_BWD(T, NAME, 128, 1, VEC); QG_NORM_BWD(T, NAME, 128, 2, VEC);                              \
    QG_NORM_BWD(T, NAME, 512, 1, VEC); QG_NORM_BWD(T, NAME, 512, 2, VEC)
#define QG_NORM_LONG(T, NAME)                                                                              \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_long<" NAME ">", (reinterpret_cast<const void*>(k_layer_norm_long<T, kToValues>)), \
                           kLongThreads, 0, 0, 1, 1);                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_long<" NAME ",nv>", (reinterpret_cast<const void*>(k_layer_norm_long<T, kNv>)), \
                           kLongThreads, 0, 0, 1, 1);                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_long<" NAME ",mx>", (reinterpret_cast<const void*>(k_layer_norm_long<T, kMx>)), \
                           kLongThreads, 0, 0, 1, 1);                                                      \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_backward_long<" NAME ">",                                         \
                           reinterpret_cast<const void*>(k_layer_norm_backward_long<T>), kLongThreads, 0, 0, 1, 1); \
    QG_BLOCK_KERNEL_BUDGET("k_layer_norm_columns<" NAME ">",                                               \
                           reinterpret_cast<const void*>(k_layer_norm_columns<T>), kColThreads, 0, 0, 1, 4)
#define QG_NORM_BUDGETS(T, NAME)                              \
    QG_NORM_FWD_SIZES(T, NAME, kToValues, "y", true);         \
    QG_NORM_FWD_SIZES(T, NAME, kToValues, "y", false);        \
    QG_NORM_FWD_SIZES(T, NAME, kNv, "nv", true);              \
    QG_NORM_FWD_SIZES(T, NAME, kMx, "mx", true);              \
    QG_NORM_BWD_SIZES(T, NAME, true);                         \
    QG_NORM_BWD_SIZES(T, NAME, false);                        \
    QG_NORM_LONG(T, NAME)
QG_NORM_BUDGETS(__half, "f16");
QG_NORM_BUDGETS(__nv_bfloat16, "bf16");
QG_NORM_BUDGETS(float, "f32");
QG_BLOCK_KERNEL_BUDGET("k_sum_partials", reinterpret_cast<const void*>(k_sum_partials), kSumCols* kSumSlices, 0, 0,
                       1, 4);

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
