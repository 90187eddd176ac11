// Products of 8-bit integers with a scale for each token and output channel:
//   Y[m][n] = sa[m] sb[n] sum_k qa[m][k] qb[n][k] + bias[n]
// and the quantizer that makes such operands (s8_common.cuh).  The integer sums
// are exact (K < 131072) and rounded once to fp32.
#include <cuda.h>
#include <cuda_fp16.h>

#include "qg_gemm_host.h"
#include "s8_common.cuh"
#include "s8_gemm.cuh"

namespace qg {

// ------------------------------------------------------------ quantizer

// One row a group of TPR threads, CHUNKS pieces of 8 values a thread in registers; LONG: any
// length, read twice.  OUT: int8_t (packed operand) or __half (the codes as fp16 numbers, the
// tensor cores' operand).  Bound by the bytes it reads and writes, so few threads hold a row, as it
// lies in memory, and many rows are under way.  Measured: 4096 x 8192 bf16 15.0 us, 6.7 TB/s; 777 x
// 2304 f16 2.5 us; rows read twice 4.3 TB/s of what they have to move.
template <class OUT>
__device__ __forceinline__ void store_codes(OUT* dst, const float (&x)[8], float r) {
    if constexpr (sizeof(OUT) == 1) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(s8_pack(x, r), s8_pack(x + 4, r));
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = s8_number(x[i], r);
        store_vec<OUT, 8>(dst, f);
    }
}

template <class T, class OUT, int TPR, int CHUNKS>  // CHUNKS 0: LONG
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    k_s8_quantize(int M, int K, const void* X, int64_t ldx, bool aligned, OUT* Q, int ldq, float* S) {
    constexpr int GROUPS = TPR < 128 ? 128 / TPR : 1;
    constexpr bool LONG = CHUNKS == 0;
    constexpr int C = LONG ? 1 : CHUNKS;
    __shared__ uint32_t red[32];
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    const int t = threadIdx.x % TPR;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * GROUPS + threadIdx.x / TPR;
    if (TPR <= 32 && row >= M) return;  // whole groups; wider groups have a row each
    const T* x = static_cast<const T*>(X) + row * ldx;
    OUT* q = Q + row * ldq;
    uint32_t amax = 0;
    S8Piece<T> v[C];
    if constexpr (LONG) {
        for (int k = 8 * t; k < K; k += 8 * TPR) {
            v[0].load(x + k, K - k, aligned);
            amax = v[0].largest(amax);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = 8 * (t + c * TPR);
            v[c].load(x + k, K - k, aligned);  // zeros behind K
        }
#pragma unroll
        for (int c = 0; c < C; ++c) amax = v[c].largest(amax);
    }
    amax = warp_max_u32(S8Piece<T>::bits(amax));
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
        __syncthreads();
        amax = warp_max_u32((threadIdx.x & 31) < TPR / 32 ? red[threadIdx.x & 31] : 0u);
    }
    const float s = s8_scale(amax, kRowScaleFloor), r = s8_inverse(s);
    if (t == 0) S[row] = s;
    float f[8];
    if constexpr (LONG) {
        for (int k = 8 * t; k < ldq; k += 8 * TPR) {
            v[0].load(x + k, K - k, aligned);
            v[0].values(f);
            store_codes(q + k, f, r);
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = 8 * (t + c * TPR);
            if (k >= ldq) break;
            v[c].values(f);
            store_codes(q + k, f, r);
        }
    }
}

template <class T, class OUT>
static int launch_quantize(int64_t M, int64_t K, const void* X, int64_t ldx, OUT* Q, float* S, cudaStream_t s) {
    const bool aligned = aligned16(X) && (M == 1 || ldx * sizeof(T) % 16 == 0);
    const int m = static_cast<int>(M), k = static_cast<int>(K), ldq = static_cast<int>(s8_codes_ld(K));
    const unsigned rows = static_cast<unsigned>(M);
    auto launch = [&](auto kernel, unsigned grid, int threads) {
        return launch_serialized(kernel, dim3(grid), threads, 0, 1, s, m, k, X, ldx, aligned, Q, ldq, S);
    };
    if (ldq <= 32 * 8 * 4) return launch(k_s8_quantize<T, OUT, 32, 4>, (rows + 3) / 4, 128);
    if (ldq <= 128 * 8 * 4) return launch(k_s8_quantize<T, OUT, 128, 4>, rows, 128);
    if (ldq <= 128 * 8 * 8) return launch(k_s8_quantize<T, OUT, 128, 8>, rows, 128);
    if (ldq <= 512 * 8 * 4) return launch(k_s8_quantize<T, OUT, 512, 4>, rows, 512);
    return launch(k_s8_quantize<T, OUT, 512, 0>, rows, 512);
}

// ------------------------------------------------------------ few tokens

// Up to 8 tokens: the weights' rows are the rows of the MMA and the tokens its
// columns.  A CTA takes 16 weight rows, its 16 warps every 16th block of 64 values
// along K; a thread's bytes of a row (16 at a time) are the values of four MMA steps,
// since a sum does not depend on the order of k.  Sums of a few blocks are exact in
// fp32; they are added up in 32-bit integers, over the warps as well.  A lone token
// is quantized by every CTA for itself into shared memory (QUANT), which costs less
// than a kernel ahead of this one; more come as codes, straight into registers (2 tokens
// inside 6.5 us, with that kernel 6.3).
//
// Measured, linear of 4096 x 4096 in a chain of calls: 1 token 5.6 us (3.0 TB/s of weights),
// 4 and 8 with the quantizer's kernel 6.4 and 6.7, by the next kernel 9.8; 16 tokens by
// that 9.9; 8192 x 8192 17.0 us for 1 token (3.9 TB/s), 8 tokens 20.3.
// Latency: a CTA's weights are one or two rounds of loads, which go out when the kernel ahead has ended;
// until then lines are only brought to the L2.  With the weights cold 7.1 and 19.2 us for 1 token.
constexpr int kGemvWarps = 16, kGemvThreads = 32 * kGemvWarps;
constexpr int kGemvBatch = 4;            // blocks of 64 values in flight a thread
constexpr int kGemvTokens = 8;
constexpr size_t kGemvSmem = 100 * 1024;  // two CTAs an SM

__host__ __device__ inline int64_t gemv_token_bytes(int64_t K) { return (K + 63) / 64 * 64 + 16; }
// Is a lone token quantized inside the product's kernel?  Its codes have to fit the shared memory.
static bool gemv_quantizes(int64_t M, int64_t K) {
    return M == 1 && static_cast<size_t>(gemv_token_bytes(K)) <= kGemvSmem;
}

struct GemvParams {
    int M, N, K, ldq;
    const void* X;        // QUANT: values, else int8 codes (rows of ldq)
    int64_t ldx;
    bool x_aligned;
    const float* sa;      // scales of given codes
    const int8_t* W;
    const float* sb;
    const void* bias;
    void* Y;
    int64_t ldy;
};

// The first n bytes of 16, the others 0.
__device__ __forceinline__ uint4 first_bytes(uint4 w, int n) {
    auto keep = [&](uint32_t v, int at) {
        const int have = n - at;
        return have >= 4 ? v : have <= 0 ? 0u : v & ((1u << (8 * have)) - 1u);
    };
    return make_uint4(keep(w.x, 0), keep(w.y, 4), keep(w.z, 8), keep(w.w, 12));
}

template <class T, bool QUANT>
__global__ void __launch_bounds__(kGemvThreads, 2) k_s8_gemv(const GemvParams p) {
    extern __shared__ __align__(16) uint8_t codes[];
    __shared__ uint32_t red_max[kGemvWarps];
    __shared__ float token_scale[kGemvTokens];
    __shared__ int sums[kGemvWarps][4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * 16;
    const int blocks = (p.ldq + 63) / 64;
    const bool has0 = n0 + g < p.N, has1 = n0 + g + 8 < p.N;
    const int8_t* const w0 = p.W + static_cast<int64_t>(n0 + g) * p.ldq + 16 * t;
    const int8_t* const w1 = w0 + 8 * static_cast<int64_t>(p.ldq);

    // The weights may still be written by the kernel ahead, so they are read after the
    // wait; a prefetch only moves lines to the L2, where that kernel's stores go too.
    for (int b = warp; b < blocks; b += kGemvWarps) {
        const int k = 64 * b + 16 * t;
        if (k < p.ldq) {
            if (has0) asm volatile("prefetch.global.L2 [%0];" ::"l"(w0 + 64 * b));
            if (has1) asm volatile("prefetch.global.L2 [%0];" ::"l"(w1 + 64 * b));
        }
    }
    pdl_wait_prior_grid();
    pdl_launch_dependents();

    uint4 a[kGemvBatch][2], xc[QUANT ? 1 : kGemvBatch];
    auto load = [&](int b0) {
#pragma unroll
        for (int j = 0; j < kGemvBatch; ++j) {
            const int b = b0 + j * kGemvWarps, k = 64 * b + 16 * t;
            const bool in = b < blocks && k < p.ldq;
            a[j][0] = a[j][1] = make_uint4(0, 0, 0, 0);
            if (in && has0) a[j][0] = *reinterpret_cast<const uint4*>(w0 + 64 * static_cast<int64_t>(b));
            if (in && has1) a[j][1] = *reinterpret_cast<const uint4*>(w1 + 64 * static_cast<int64_t>(b));
            if constexpr (!QUANT) {
                xc[j] = make_uint4(0, 0, 0, 0);
                if (in && g < p.M) {
                    xc[j] = *reinterpret_cast<const uint4*>(static_cast<const int8_t*>(p.X) +
                                                            static_cast<int64_t>(g) * p.ldq + k);
                    if (k + 16 > p.K) xc[j] = first_bytes(xc[j], p.K - k);  // what lies behind K does not count
                }
            }
        }
    };
    load(warp);

    if constexpr (QUANT) {
        const T* x = static_cast<const T*>(p.X);
        auto at = [&](int i) { return 8 * (static_cast<int>(threadIdx.x) + i * kGemvThreads); };
        const int pieces = (64 * blocks + 8 * kGemvThreads - 1) / (8 * kGemvThreads);
        constexpr int HELD = sizeof(T) == 4 ? 1 : 2;  // pieces that a thread keeps
        S8Piece<T> held[HELD], v;
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < HELD; ++i) held[i].load(x + at(i), p.K - at(i), p.x_aligned);
#pragma unroll
        for (int i = 0; i < HELD; ++i) amax = held[i].largest(amax);
        for (int i = HELD; i < pieces; ++i) {
            v.load(x + at(i), p.K - at(i), p.x_aligned);
            amax = v.largest(amax);
        }
        amax = warp_max_u32(S8Piece<T>::bits(amax));
        if (lane == 0) red_max[warp] = amax;
        __syncthreads();
        amax = warp_max_u32(red_max[lane & (kGemvWarps - 1)]);
        const float s = s8_scale(amax, kRowScaleFloor), r = s8_inverse(s);
        if (threadIdx.x == 0) token_scale[0] = s;
        auto store = [&](int i, const S8Piece<T>& w) {
            if (at(i) >= 64 * blocks) return;
            float f[8];
            w.values(f);
            store_codes(reinterpret_cast<int8_t*>(codes) + at(i), f, r);
        };
#pragma unroll
        for (int i = 0; i < HELD; ++i) store(i, held[i]);
        for (int i = HELD; i < pieces; ++i) {
            v.load(x + at(i), p.K - at(i), p.x_aligned);
            store(i, v);
        }
        __syncthreads();
    } else {
        if (threadIdx.x < p.M) token_scale[threadIdx.x] = p.sa[threadIdx.x];
    }

    int total[4] = {0, 0, 0, 0};
    for (int b0 = warp; b0 < blocks; b0 += kGemvBatch * kGemvWarps) {
        if (b0 != warp) load(b0);
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kGemvBatch; ++j) {
            const int b = b0 + j * kGemvWarps;
            if (b >= blocks) break;
            uint4 x;
            if constexpr (QUANT)
                x = g == 0 ? *reinterpret_cast<const uint4*>(codes + 64 * b + 16 * t) : make_uint4(0, 0, 0, 0);
            else
                x = xc[j];
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            const uint32_t r0[4] = {a[j][0].x, a[j][0].y, a[j][0].z, a[j][0].w};
            const uint32_t r1[4] = {a[j][1].x, a[j][1].y, a[j][1].z, a[j][1].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t a0, a1, a2, a3, b0h, b1h;
                s8_to_f16(r0[c], a0, a2);
                s8_to_f16(r1[c], a1, a3);
                s8_to_f16(xw[c], b0h, b1h);
                mma_f16(acc, a0, a1, a2, a3, b0h, b1h);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) total[i] += __float2int_rn(acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][i][lane] = total[i];
    __syncthreads();
    // accumulator element e of lane 4 g + t: weight row g + 8 (e / 2), token 2 t + e % 2
    if (threadIdx.x < 128) {
        const int e = threadIdx.x >> 5, row = g + 8 * (e >> 1), m = 2 * t + (e & 1);
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kGemvWarps; ++w) sum += sums[w][e][lane];
        const int n = n0 + row;
        if (m < p.M && n < p.N) {
            const float b = p.bias ? to_f32<T>(static_cast<const T*>(p.bias)[n]) : 0.f;
            static_cast<T*>(p.Y)[m * p.ldy + n] =
                from_f32<T>(s8_scaled(sum, token_scale[m], p.sb[n], b));
        }
    }
}

template <class T, bool QUANT>
static int launch_gemv(const GemvParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.N + 15) / 16));
    if constexpr (QUANT) {
        struct Tag;
        const int rc = raise_smem<Tag>(k_s8_gemv<T, true>);
        if (rc) return rc;
        return launch_serialized(k_s8_gemv<T, true>, grid, kGemvThreads,
                                 static_cast<size_t>(gemv_token_bytes(p.ldq)), 1, s, p);
    } else {
        return launch_serialized(k_s8_gemv<T, false>, grid, kGemvThreads, 0, 1, s, p);
    }
}

// ------------------------------------------------------------ which kernel

static bool takes_gemv(int64_t M) { return M <= kGemvTokens; }

// Tokens a tile (32, 64, 128) and CTAs of a cluster that share K.
struct SomeForm {
    int tile, splits;
};

// A CTA's accumulators hold 1024 values of K each.
static bool some_holds(const SomeForm& f, int64_t K) {
    const int64_t stages = (K + kS8Bk - 1) / kS8Bk;
    return (stages + f.splits - 1) / f.splits <= 512 / f.tile * kS8Exact;
}

// The form with the least estimated time, in cycles of an SM, as measured: a CTA's start, its
// stages (the bytes that they bring from the L2, and turning codes into fp16), its epilogue and
// the exchange of sums; whole rounds of CTAs, of which clusters of 8 leave SMs out.  Estimates
// were within 10% of 4 to 250 us at 36 problems; the best form of each was chosen, or one at most
// 8% slower.
static int64_t some_cycles(const SomeForm& f, int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = (N + 127) / 128 * ((M + f.tile - 1) / f.tile);
    const int64_t stages = ((K + kS8Bk - 1) / kS8Bk + f.splits - 1) / f.splits;
    const int64_t cta = 5700 + 20 * f.tile + stages * (500 + 6 * f.tile) + (f.splits > 1 ? 2500 + 32 * f.tile : 0);
    const int64_t sms = f.splits == 8 ? 104 : 148;
    return (tiles * f.splits + sms - 1) / sms * cta;
}
static SomeForm some_form(int64_t M, int64_t N, int64_t K, int64_t* cycles) {
    SomeForm best = {32, 8};
    int64_t least = INT64_MAX;
    for (int tile = 32; tile <= 128; tile *= 2) {
        if (tile > 32 && tile >= 2 * M) break;
        for (int splits = 1; splits <= 8; splits *= 2) {
            const SomeForm f = {tile, splits};
            if (!some_holds(f, K) || (splits > 1 && K < 256 * splits)) continue;
            const int64_t time = some_cycles(f, M, N, K);
            if (time < least) least = time, best = f;
        }
    }
    *cycles = least;
    return best;
}

// Does that kernel take the problem, or the one on CTA pairs, behind a pass that writes the
// weights as fp16?  The latter's estimate: that pass at 6.2 TB/s (3.3 kB a cycle) and rounds of
// 256 x 256 tiles, 630 cycles a step of 64 values of K.  Measured, linear of 4096 x 4096, this kernel and
// pairs: 128 tokens 16.3 and 33.6 us, 512 27.8 and 35.7, 777 49.5 and 36.6, 2048 98 and 60; of
// 1024 x 8192: 777 tokens 33 and 53, 2048 62 and 60; of 8192 x 8192: 256 tokens 57.5 and 80.6, 512 113
// and 83.  The choice was within 3% of the better one at 45 sizes.  4096 x 8192 x 8192 by pairs 335 to
// 350 us, 1.6 PFLOP/s, of which the product takes 289 (1.9), the weights' pass 28 and the quantizer 19.
static int64_t pairs_cycles(int64_t M, int64_t N, int64_t K) {
    const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256);
    return 5700 + 3 * N * K / 3300 + (tiles + 75) / 76 * ((K + 63) / 64 * 630 + 7600);
}
static bool takes_some(int64_t M, int64_t N, int64_t K) {
    if (M > 4096 || !some_holds(SomeForm{32, 8}, K)) return false;
    int64_t cycles = 0;
    some_form(M, N, K, &cycles);
    return cycles <= pairs_cycles(M, N, K);
}

// May a product of up to M tokens be one on pairs?  Whole rounds of CTAs let the choice go back and forth
// as M grows, but a workspace for M tokens has to do for fewer, so it has the weights' place from
// the first such M on, or a little earlier.  In each 256 tokens the pairs' estimate is one number, and the
// other kernel's grows with M as long as it chooses among the same tiles (up to 32 tokens, up to 64, above).
static bool may_take_pairs(int64_t M, int64_t N, int64_t K) {
    if (M > 4096 || !some_holds(SomeForm{32, 8}, K)) return true;
    int64_t most = 0;  // of the other kernel, up to `end` tokens
    for (int64_t end = 32;; end = end < 64 ? 64 : end < 256 ? 256 : end + 256) {
        const int64_t m = M < end ? M : end;
        int64_t cycles = 0;
        some_form(m, N, K, &cycles);
        most = cycles > most ? cycles : most;
        if (most > pairs_cycles(m, N, K)) return true;
        if (end >= M) return false;
    }
}

// ------------------------------------------------------------ workspaces and calls

static size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// The tokens' codes (a few tokens: 8 bits, more: fp16) and scales and, where they may be turned
// into fp16 in memory, the weights.
struct S8Workspace {
    size_t a, b, sa, total;
};
static S8Workspace s8_workspace(int64_t M, int64_t N, int64_t K) {
    const size_t ld = static_cast<size_t>(s8_codes_ld(K)), m = static_cast<size_t>(M);
    S8Workspace w;
    w.a = 0;
    w.b = up256((takes_gemv(M) ? 1 : 2) * ld * m);
    w.sa = w.b + (takes_gemv(M) || !may_take_pairs(M, N, K) ? 0 : up256(2 * ld * static_cast<size_t>(N)));
    w.total = w.sa + up256(4 * m);
    return w;
}
size_t s8_linear_workspace(int64_t M, int64_t N, int64_t K) {
    return gemv_quantizes(M, K) ? 0 : s8_workspace(M, N, K).total;
}

constexpr int64_t kMaxRows = int64_t(1) << 27, kMaxK = 131072;

static int check_s8(int dtype, int64_t M, int64_t N, int64_t K) {
    if (!dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0 || M > kMaxRows || N > kMaxRows || K >= kMaxK) return QG_ERR_INVALID_ARG;
    return QG_OK;
}

static int check_out(int dtype, int64_t N, const float* sb, const void* bias, const void* Y, int64_t ldy, int64_t M) {
    if (!Y || (M > 1 && ldy < N)) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(Y) % dtype_bytes(dtype) || reinterpret_cast<uintptr_t>(bias) % dtype_bytes(dtype) ||
        reinterpret_cast<uintptr_t>(sb) % 4)
        return QG_ERR_MISALIGNED;
    return QG_OK;
}

static int check_workspace(const void* ws, size_t bytes, size_t want) {
    if (want == 0) return QG_OK;
    if (!ws || bytes < want) return QG_ERR_WORKSPACE;
    return reinterpret_cast<uintptr_t>(ws) % 256 ? QG_ERR_MISALIGNED : QG_OK;
}

__global__ void __launch_bounds__(256) k_s8_only_bias(int64_t M, int64_t N, const void* bias, void* Y, int64_t ldy,
                                                      int dtype) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    for (int64_t i = blockIdx.x * 256 + threadIdx.x; i < M * N; i += gridDim.x * int64_t(256)) {
        const int64_t m = i / N, n = i % N;
        if (dtype == QG_F32)
            static_cast<float*>(Y)[m * ldy + n] = bias ? static_cast<const float*>(bias)[n] : 0.f;
        else  // 16-bit types: 0 has the same bits in both
            static_cast<uint16_t*>(Y)[m * ldy + n] = bias ? static_cast<const uint16_t*>(bias)[n] : uint16_t(0);
    }
}

static int only_bias(int dtype, int64_t M, int64_t N, const void* bias, void* Y, int64_t ldy, cudaStream_t s) {
    return launch_serialized(k_s8_only_bias, dim3(static_cast<unsigned>(conv_grid(current_device(), M * N))), 256, 0, 1,
                             s, M, N, bias, Y, ldy, dtype);
}

// Sums of fp16 operands, scaled: the exact chunked GEMM of qgemm_s8 with another epilogue.
static int tensor_product(int dtype, int64_t M, int64_t N, int64_t K, const __half* A, const float* sa, const __half* B,
                          const float* sb, const void* bias, void* Y, int64_t ldy, const Ctl& ctl, cudaStream_t s) {
    S8Scales e;
    e.sa = sa;
    e.sb = sb;
    e.bias = bias;
    e.dtype = dtype;
    return run_gemm_s8_scaled(A, B, M, N, K, s8_codes_ld(K), Y, ldy, e, ctl, s);
}

// ------------------------------------------------------------ some tokens

template <int NT>
static int launch_some(const int8_t* W, const __half* X, const S8Params& p, int splits, cudaStream_t s) {
    using Cfg = S8Cfg<NT>;
    struct Tag;
    int rc = raise_smem<Tag>(s8_gemm_kernel<Cfg>);
    if (rc) return rc;
    const int64_t ld = s8_codes_ld(p.K);
    CUtensorMap tw, tx;
    rc = make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, W, p.K, p.N, ld, kS8Bk, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!rc) rc = make_tmap_kmajor(&tx, true, X, p.K, p.M, 2 * ld, 64, NT);
    if (rc) return rc;
    return launch_serialized(s8_gemm_kernel<Cfg>,
                             dim3(static_cast<unsigned>((p.N + 127) / 128 * splits), static_cast<unsigned>((p.M + NT - 1) / NT)),
                             kS8Threads, Cfg::SMEM, splits, s, tw, tx, p);
}

static int some_product(int dtype, int64_t M, int64_t N, int64_t K, const __half* A, const float* sa,
                        const int8_t* W, const float* sb, const void* bias, void* Y, int64_t ldy, const Ctl& ctl,
                        cudaStream_t s) {
    S8Params p = {};
    p.M = static_cast<int>(M); p.N = static_cast<int>(N); p.K = static_cast<int>(K);
    int64_t cycles = 0;
    const SomeForm f = some_form(M, N, K, &cycles);
    while ((1 << p.log_splits) < f.splits) ++p.log_splits;
    p.sa = sa; p.sb = sb; p.bias = bias; p.Y = Y; p.ldy = ldy; p.dtype = dtype; p.ctl = ctl;
    if (f.tile == 32) return launch_some<32>(W, A, p, f.splits, s);
    if (f.tile == 64) return launch_some<64>(W, A, p, f.splits, s);
    return launch_some<128>(W, A, p, f.splits, s);
}

#define QG_S8_SOME(NT)                                                                                              \
    QG_BLOCK_KERNEL_BUDGET("s8_gemm_kernel<" #NT ">", (reinterpret_cast<const void*>(s8_gemm_kernel<S8Cfg<NT>>)),   \
                           kS8Threads, S8Cfg<NT>::SMEM, 512, 8, 1)
QG_S8_SOME(32);
QG_S8_SOME(64);
QG_S8_SOME(128);

#define QG_S8_QUANT(T, NAME, OUT, ONAME, TPR, CHUNKS)                                                \
    QG_BLOCK_KERNEL_BUDGET("k_s8_quantize<" NAME "," ONAME "," #TPR "," #CHUNKS ">",                 \
                           (reinterpret_cast<const void*>(k_s8_quantize<T, OUT, TPR, CHUNKS>)),      \
                           TPR < 128 ? 128 : TPR, 0, 0, 1, 1)
#define QG_S8_QUANT_SIZES(T, NAME, OUT, ONAME)  \
    QG_S8_QUANT(T, NAME, OUT, ONAME, 32, 4);    \
    QG_S8_QUANT(T, NAME, OUT, ONAME, 128, 4);   \
    QG_S8_QUANT(T, NAME, OUT, ONAME, 128, 8);   \
    QG_S8_QUANT(T, NAME, OUT, ONAME, 512, 4);   \
    QG_S8_QUANT(T, NAME, OUT, ONAME, 512, 0)
#define QG_S8_GEMV(T, NAME, QUANT)                                                                \
    QG_BLOCK_KERNEL_BUDGET("k_s8_gemv<" NAME "," #QUANT ">"       ,                              \
                           (reinterpret_cast<const void*>(k_s8_gemv<T, QUANT>)), kGemvThreads,     \
                           QUANT ? static_cast<int>(kGemvSmem) : 0, 0, 1, 2)
#define QG_S8_BUDGETS(T, NAME)                    \
    QG_S8_QUANT_SIZES(T, NAME, int8_t, "s8");     \
    QG_S8_QUANT_SIZES(T, NAME, __half, "codes");  \
    QG_S8_GEMV(T, NAME, true);                    \
    QG_S8_GEMV(T, NAME, false)
QG_S8_BUDGETS(__half, "f16");
QG_S8_BUDGETS(__nv_bfloat16, "bf16");
QG_S8_BUDGETS(float, "f32");

}  // namespace qg

using namespace qg;

extern "C" {

int64_t qg_s8_codes_ld(int64_t K) { return K > 0 ? s8_codes_ld(K) : 0; }

int s8_quantize(int dtype, int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q, float* S, void* stream) {
    const NvtxRange nvtx_range("s8_quantize");
    int rc = check_s8(dtype, M, 0, K);
    if (rc) return rc;
    if (M == 0 || K == 0) return QG_OK;
    if (!X || !Q || !S || (M > 1 && ldx < K)) return QG_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype) || !aligned16(Q) || reinterpret_cast<uintptr_t>(S) % 4)
        return QG_ERR_MISALIGNED;
    if (current_device() < 0) return QG_ERR_CUDA;
    return by_dtype(dtype, [&](auto t) {
        return launch_quantize<decltype(t), int8_t>(M, K, X, ldx, Q, S, static_cast<cudaStream_t>(stream));
    });
}

int s8_gemm(int dtype, int64_t M, int64_t N, int64_t K, const int8_t* Aq, const float* As, const int8_t* Bq,
            const float* Bs, const void* bias, void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("s8_gemm");
    int rc = check_s8(dtype, M, N, K);
    if (rc) return rc;
    if (M == 0 || N == 0) return QG_OK;
    if (K > 0 && (!Aq || !As || !Bq || !Bs)) return QG_ERR_INVALID_ARG;
    rc = check_out(dtype, N, Bs, bias, Y, ldy, M);
    if (rc) return rc;
    if (!aligned16(Aq) || !aligned16(Bq) || reinterpret_cast<uintptr_t>(As) % 4) return QG_ERR_MISALIGNED;
    if (K > 0 && !takes_gemv(M)) rc = check_workspace(ws, ws_bytes, s8_linear_workspace(M, N, K));
    if (rc) return rc;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return only_bias(dtype, M, N, bias, Y, ldy, s);
    const int64_t ld = s8_codes_ld(K);
    if (takes_gemv(M)) {
        GemvParams p = {};
        p.M = static_cast<int>(M); p.N = static_cast<int>(N); p.K = static_cast<int>(K); p.ldq = static_cast<int>(ld);
        p.X = Aq; p.sa = As; p.W = Bq; p.sb = Bs; p.bias = bias; p.Y = Y; p.ldy = ldy;
        return by_dtype(dtype, [&](auto t) { return launch_gemv<decltype(t), false>(p, s); });
    }
    const Ctl ctl = host_ctl(dev);
    if (!ctl.status) return QG_ERR_CUDA;
    const S8Workspace w = s8_workspace(M, N, K);
    uint8_t* base = static_cast<uint8_t*>(ws);
    __half *a = reinterpret_cast<__half*>(base + w.a), *b = reinterpret_cast<__half*>(base + w.b);
    rc = s8_to_f16_rows(Aq, M, ld, a, ld, dev, s);
    if (!rc && takes_some(M, N, K)) return some_product(dtype, M, N, K, a, As, Bq, Bs, bias, Y, ldy, ctl, s);
    if (!rc) rc = s8_to_f16_rows(Bq, N, ld, b, ld, dev, s);
    return rc ? rc : tensor_product(dtype, M, N, K, a, As, b, Bs, bias, Y, ldy, ctl, s);
}

int s8_linear(int dtype, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const int8_t* Wq,
              const float* Ws, const void* bias, void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("s8_linear");
    int rc = check_s8(dtype, M, N, K);
    if (rc) return rc;
    if (M == 0 || N == 0) return QG_OK;
    if (K > 0 && (!X || !Wq || !Ws || (M > 1 && ldx < K))) return QG_ERR_INVALID_ARG;
    rc = check_out(dtype, N, Ws, bias, Y, ldy, M);
    if (rc) return rc;
    if (!aligned16(Wq) || reinterpret_cast<uintptr_t>(X) % dtype_bytes(dtype)) return QG_ERR_MISALIGNED;
    if (K > 0) rc = check_workspace(ws, ws_bytes, s8_linear_workspace(M, N, K));
    if (rc) return rc;
    const int dev = current_device();
    if (dev < 0) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return only_bias(dtype, M, N, bias, Y, ldy, s);
    const int64_t ld = s8_codes_ld(K);
    const S8Workspace w = s8_workspace(M, N, K);
    uint8_t* base = static_cast<uint8_t*>(ws);
    if (takes_gemv(M)) {
        GemvParams p = {};
        p.M = static_cast<int>(M); p.N = static_cast<int>(N); p.K = static_cast<int>(K); p.ldq = static_cast<int>(ld);
        p.W = Wq; p.sb = Ws; p.bias = bias; p.Y = Y; p.ldy = ldy;
        if (gemv_quantizes(M, K)) {
            p.X = X; p.ldx = ldx; p.x_aligned = aligned16(X) && (M == 1 || ldx * dtype_bytes(dtype) % 16 == 0);
            return by_dtype(dtype, [&](auto t) { return launch_gemv<decltype(t), true>(p, s); });
        }
        float* sa = reinterpret_cast<float*>(base + w.sa);
        p.X = base + w.a;
        p.sa = sa;
        return by_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            const int rc = launch_quantize<T, int8_t>(M, K, X, ldx, reinterpret_cast<int8_t*>(base + w.a), sa, s);
            return rc ? rc : launch_gemv<T, false>(p, s);
        });
    }
    const Ctl ctl = host_ctl(dev);
    if (!ctl.status) return QG_ERR_CUDA;
    __half *a = reinterpret_cast<__half*>(base + w.a), *b = reinterpret_cast<__half*>(base + w.b);
    float* sa = reinterpret_cast<float*>(base + w.sa);
    rc = by_dtype(dtype, [&](auto t) { return launch_quantize<decltype(t), __half>(M, K, X, ldx, a, sa, s); });
    if (!rc && takes_some(M, N, K)) return some_product(dtype, M, N, K, a, sa, Wq, Ws, bias, Y, ldy, ctl, s);
    if (!rc) rc = s8_to_f16_rows(Wq, N, ld, b, ld, dev, s);
    return rc ? rc : tensor_product(dtype, M, N, K, a, sa, b, Ws, bias, Y, ldy, ctl, s);
}

}  // extern "C"
