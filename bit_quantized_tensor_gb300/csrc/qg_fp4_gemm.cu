// Products of microscaled 4-bit operands: fp4_gemm (both packed), fp4_linear
// (activations quantized in the call) and fp4_linear_backward (gradients of
// the activations, the weights and the bias).  Kernels: fp4_gemm.cuh
// (one CTA a tile) and fp4_gemm2.cuh (CTA pairs).
#include <mutex>

#include "fp4_gemm2.cuh"

namespace qg {

struct Fp4Operand {
    const uint8_t *codes, *scales;
    int64_t rows;
    const float* ts;
};

// Lifts the kernel's dynamic shared-memory limit, once per device.  Cfg keeps
// the flags of different kernels apart.
template <class Cfg, class F>
static int raise_smem(F* kernel) {
    static std::mutex mu;
    static bool done[64] = {};
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return QG_ERR_CUDA;
    std::lock_guard<std::mutex> g(mu);
    if (done[dev]) return QG_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES);
    if (e != cudaSuccess) return map_cuda(e);
    done[dev] = true;
    return QG_OK;
}

static int codes_map(CUtensorMap* map, const Fp4Operand& o, int64_t K, int box_rows) {
    return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.codes, fp4_codes_ld(K), o.rows, fp4_codes_ld(K), 128,
                        box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles as rows of 128 32-bit words.
static int scales_map(CUtensorMap* map, const Fp4Operand& o, int fmt, int64_t K, int atoms) {
    return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, o.scales, 128, fp4_scale_bytes(fmt, o.rows, K) / 512,
                        512, 128, atoms, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <class Cfg>
static int launch_fp4(const Fp4Operand& x, const Fp4Operand& w, const Fp4Params& p, int splits, cudaStream_t s) {
    CUtensorMap tw, tx, tsw, tsx;
    int rc = codes_map(&tw, w, p.K, 128);
    if (!rc) rc = codes_map(&tx, x, p.K, Cfg::NT);
    if (!rc) rc = scales_map(&tsw, w, Cfg::FMT, p.K, Cfg::ATOMS);
    if (!rc) rc = scales_map(&tsx, x, Cfg::FMT, p.K, Cfg::ATOMS);
    if (!rc) rc = raise_smem<Cfg>(fp4_gemm_kernel<Cfg>);
    if (rc) return rc;
    const int64_t gy = (p.N + 127) / 128, gz = (p.M + Cfg::NT - 1) / Cfg::NT;
    if (gy > 65535 || gz > 65535) return QG_ERR_UNSUPPORTED;
    return launch_serialized(fp4_gemm_kernel<Cfg>,
                             dim3(static_cast<unsigned>(splits), static_cast<unsigned>(gy), static_cast<unsigned>(gz)),
                             kFp4Threads, Cfg::SMEM_BYTES, splits, s, tw, tx, tsw, tsx, p);
}

template <class Cfg>
static int launch_fp4_pair(const Fp4Operand& x, const Fp4Operand& w, const Fp4Params& p, int dev, cudaStream_t s) {
    CUtensorMap tw, tx, tsw, tsx;
    int rc = codes_map(&tw, w, p.K, 128);
    if (!rc) rc = codes_map(&tx, x, p.K, 128);
    if (!rc) rc = scales_map(&tsw, w, Cfg::FMT, p.K, Cfg::ATOMS);
    if (!rc) rc = scales_map(&tsx, x, Cfg::FMT, p.K, Cfg::ATOMS);
    if (!rc) rc = raise_smem<Cfg>(fp4_gemm2_kernel<Cfg>);
    if (rc) return rc;
    const int64_t tiles = (int64_t(p.M) + 255) / 256 * ((int64_t(p.N) + 255) / 256);
    if (tiles > INT32_MAX) return QG_ERR_UNSUPPORTED;
    const int64_t pairs = num_sms(dev) / 2;
    return launch_serialized(fp4_gemm2_kernel<Cfg>, dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs))),
                             Cfg::THREADS, Cfg::SMEM_BYTES, 1, s, tx, tw, tsx, tsw, p);
}

// Splits of K over a cluster: doubled while the tiles alone leave half of the
// SMs without work and each split keeps at least two K blocks.
static int choose_splits(int64_t tiles, int64_t num_kb, int sms) {
    int s = 1;
    while (s < 8 && tiles * s * 2 <= sms && num_kb >= 4 * s) s *= 2;
    return s;
}

template <int FMT>
static int run_fmt(const Fp4Operand& x, const Fp4Operand& w, const Fp4Params& p, int dev, cudaStream_t s) {
    if (p.M > 128 && p.N > 128 && (p.M > 256 || p.N > 2048)) return launch_fp4_pair<Fp4PairCfg<FMT>>(x, w, p, dev, s);
    const int nt = p.M <= 16 ? 16 : p.M <= 32 ? 32 : p.M <= 64 ? 64 : 128;
    const int64_t tiles = (int64_t(p.N) + 127) / 128 * ((int64_t(p.M) + nt - 1) / nt);
    const int splits = choose_splits(tiles, (p.K + kFp4Bk - 1) / kFp4Bk, num_sms(dev));
    switch (nt) {
        case 16: return launch_fp4<Fp4Cfg<FMT, 16>>(x, w, p, splits, s);
        case 32: return launch_fp4<Fp4Cfg<FMT, 32>>(x, w, p, splits, s);
        case 64: return launch_fp4<Fp4Cfg<FMT, 64>>(x, w, p, splits, s);
        default: return launch_fp4<Fp4Cfg<FMT, 128>>(x, w, p, splits, s);
    }
}

// Y (M x N) = alpha X . W^T + bias, K >= 0.
static int fp4_gemm_run(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const Fp4Operand& x,
                        const Fp4Operand& w, const void* bias, void* Y, int64_t ldy, bool weights_ready, int dev,
                        cudaStream_t s) {
    Fp4Params p = {};
    p.M = static_cast<int>(M); p.N = static_cast<int>(N); p.K = static_cast<int>(K);
    p.ts_a = x.ts; p.ts_b = w.ts; p.bias = bias; p.Y = Y; p.ldy = ldy; p.dtype = dtype;
    p.weights_ready = weights_ready;
    p.ctl = host_ctl(dev);
    if (!p.ctl.status) return QG_ERR_CUDA;
    return fmt == kNv ? run_fmt<kNv>(x, w, p, dev, s) : run_fmt<kMx>(x, w, p, dev, s);
}

// Products over nothing: every output is its bias (or 0).
__global__ void __launch_bounds__(256) k_fp4_only_bias(int64_t M, int64_t N, const void* bias, void* Y, int64_t ldy,
                                                       int dtype) {
    pdl_wait_prior_grid();
    pdl_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < M * N;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t m = i / N, n = i - m * N;
        typed_store(Y, dtype, m * ldy + n, bias ? typed_at(bias, dtype, n) : 0.f);
    }
}

static int only_bias(int dtype, int64_t M, int64_t N, const void* bias, void* Y, int64_t ldy, cudaStream_t s) {
    if (M == 0 || N == 0) return QG_OK;
    const int64_t want = (M * N + 255) / 256;
    return launch_serialized(k_fp4_only_bias, dim3(static_cast<unsigned>(want > 4096 ? 4096 : want)), 256, 0, 1, s, M,
                             N, bias, Y, ldy, dtype);
}

static size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Bytes of a packed operand inside a workspace; the larger format's.
static size_t packed_codes(int64_t rows, int64_t K) { return up256(static_cast<size_t>(rows * fp4_codes_ld(K))); }
static size_t packed_scales(int64_t rows, int64_t K) {
    return up256(static_cast<size_t>(fp4_scale_bytes(kNv, rows, K)));
}

size_t fp4_linear_workspace(int64_t M, int64_t K) { return packed_codes(M, K) + packed_scales(M, K); }

size_t fp4_linear_backward_workspace(int64_t M, int64_t N, int64_t K) {
    return packed_codes(M, N) + packed_scales(M, N) + packed_codes(N, M) + packed_scales(N, M) +
           packed_codes(K, M) + packed_scales(K, M) +
           up256(static_cast<size_t>((M + 127) / 128 * N) * sizeof(float));
}

// Carves consecutive pieces out of a workspace.
struct Carver {
    uint8_t* at;
    uint8_t* take(size_t bytes) {
        uint8_t* p = at;
        at += bytes;
        return p;
    }
};

#define QG_FP4_GEMM_BUDGET(FMT, FNAME, NT)                                                     \
    QG_BLOCK_KERNEL_BUDGET("fp4_gemm_kernel<" FNAME "," #NT ">",                               \
                           (reinterpret_cast<const void*>(fp4_gemm_kernel<Fp4Cfg<FMT, NT>>)),  \
                           kFp4Threads, (Fp4Cfg<FMT, NT>::SMEM_BYTES), (Fp4Cfg<FMT, NT>::TMEM_COLS), 8, 1)
QG_FP4_GEMM_BUDGET(kNv, "nv", 16); QG_FP4_GEMM_BUDGET(kNv, "nv", 32);
QG_FP4_GEMM_BUDGET(kNv, "nv", 64); QG_FP4_GEMM_BUDGET(kNv, "nv", 128);
QG_FP4_GEMM_BUDGET(kMx, "mx", 16); QG_FP4_GEMM_BUDGET(kMx, "mx", 32);
QG_FP4_GEMM_BUDGET(kMx, "mx", 64); QG_FP4_GEMM_BUDGET(kMx, "mx", 128);
QG_BLOCK_KERNEL_BUDGET("fp4_gemm2_kernel<nv>", reinterpret_cast<const void*>(fp4_gemm2_kernel<Fp4PairCfg<kNv>>),
                       Fp4PairCfg<kNv>::THREADS, Fp4PairCfg<kNv>::SMEM_BYTES, 512, 2, 1);
QG_BLOCK_KERNEL_BUDGET("fp4_gemm2_kernel<mx>", reinterpret_cast<const void*>(fp4_gemm2_kernel<Fp4PairCfg<kMx>>),
                       Fp4PairCfg<kMx>::THREADS, Fp4PairCfg<kMx>::SMEM_BYTES, 512, 2, 1);
QG_BLOCK_KERNEL_BUDGET("k_fp4_only_bias", reinterpret_cast<const void*>(k_fp4_only_bias), 256, 0, 0, 1, 4);

// Checks shared by the three calls.
static int check_product(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const float* ta, const float* tb) {
    if (!fmt_ok(fmt) || !dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0 || M > (1 << 30) || N > (1 << 30) || K > (1 << 30)) return QG_ERR_INVALID_ARG;
    if (fmt == kMx && (ta || tb)) return QG_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(ta) % 4 || reinterpret_cast<uintptr_t>(tb) % 4) return QG_ERR_MISALIGNED;
    return QG_OK;
}

static int check_typed(const void* v, int dtype) {
    return reinterpret_cast<uintptr_t>(v) % dtype_bytes(dtype) ? QG_ERR_MISALIGNED : QG_OK;
}

}  // namespace qg

using namespace qg;

extern "C" {

int fp4_gemm(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const uint8_t* Aq, const uint8_t* As,
             const float* a_tscale, const uint8_t* Bq, const uint8_t* Bs, const float* b_tscale, const void* bias,
             void* Y, int64_t ldy, void* stream) {
    const NvtxRange nvtx_range("fp4_gemm");
    int rc = check_product(fmt, dtype, M, N, K, a_tscale, b_tscale);
    if (!rc) rc = check_typed(bias, dtype);
    if (!rc) rc = check_typed(Y, dtype);
    if (rc) return rc;
    if (M == 0 || N == 0) return QG_OK;
    if (!Y || (M > 1 && ldy < N) || (K > 0 && (!Aq || !As || !Bq || !Bs))) return QG_ERR_INVALID_ARG;
    if (!aligned16(Aq) || !aligned16(As) || !aligned16(Bq) || !aligned16(Bs)) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return only_bias(dtype, M, N, bias, Y, ldy, s);
    return fp4_gemm_run(fmt, dtype, M, N, K, {Aq, As, M, a_tscale}, {Bq, Bs, N, b_tscale}, bias, Y, ldy, false, dev,
                        s);
}

int fp4_linear(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
               const float* x_tscale, const uint8_t* Wq, const uint8_t* Ws, const float* w_tscale, const void* bias,
               void* Y, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("fp4_linear");
    int rc = check_product(fmt, dtype, M, N, K, x_tscale, w_tscale);
    if (!rc) rc = check_typed(X, dtype);
    if (!rc) rc = check_typed(bias, dtype);
    if (!rc) rc = check_typed(Y, dtype);
    if (rc) return rc;
    if (M == 0 || N == 0) return QG_OK;
    if (!Y || (M > 1 && (ldy < N || ldx < K)) || (K > 0 && (!X || !Wq || !Ws))) return QG_ERR_INVALID_ARG;
    if (!aligned16(Wq) || !aligned16(Ws)) return QG_ERR_MISALIGNED;
    if (K > 0 && (!ws || ws_bytes < fp4_linear_workspace(M, K))) return QG_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return only_bias(dtype, M, N, bias, Y, ldy, s);
    Carver c{static_cast<uint8_t*>(ws)};
    uint8_t* xq = c.take(packed_codes(M, K));
    uint8_t* xs = c.take(packed_scales(M, K));
    rc = fp4_quantize_run(fmt, dtype, M, K, X, ldx, x_tscale, xq, xs, false, s);
    if (rc) return rc;
    return fp4_gemm_run(fmt, dtype, M, N, K, {xq, xs, M, x_tscale}, {Wq, Ws, N, w_tscale}, bias, Y, ldy, true, dev,
                        s);
}

int fp4_linear_backward(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy,
                        const float* dy_tscale, const void* X, int64_t ldx, const float* x_tscale,
                        const uint8_t* Wtq, const uint8_t* Wts, const float* w_tscale, void* dX, int64_t lddx,
                        void* dW, int64_t lddw, float* db, void* ws, size_t ws_bytes, void* stream) {
    const NvtxRange nvtx_range("fp4_linear_backward");
    int rc = check_product(fmt, dtype, M, N, K, dy_tscale, x_tscale);
    if (!rc) rc = check_product(fmt, dtype, M, N, K, w_tscale, nullptr);
    for (const void* v : {dY, X, static_cast<const void*>(dX), static_cast<const void*>(dW)})
        if (!rc) rc = check_typed(v, dtype);
    if (!rc) rc = check_typed(db, QG_F32);
    if (rc) return rc;
    if (!dX && !dW && !db) return QG_ERR_INVALID_ARG;
    const bool some = M > 0 && N > 0;
    if (some && (!dY || (M > 1 && lddy < N))) return QG_ERR_INVALID_ARG;
    if (dX && M > 1 && lddx < K) return QG_ERR_INVALID_ARG;
    if (dW && ((N > 1 && lddw < K) || (M > 1 && ldx < K) || (some && K > 0 && !X))) return QG_ERR_INVALID_ARG;
    if (dX && some && K > 0 && (!Wtq || !Wts)) return QG_ERR_INVALID_ARG;
    if (!aligned16(Wtq) || !aligned16(Wts)) return QG_ERR_MISALIGNED;
    if (some && (!ws || ws_bytes < fp4_linear_backward_workspace(M, N, K))) return QG_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!some) {  // sums over nothing
        if (dX) rc = only_bias(dtype, M, K, nullptr, dX, lddx, s);
        if (!rc && dW) rc = only_bias(dtype, N, K, nullptr, dW, lddw, s);
        if (!rc && db) rc = only_bias(QG_F32, 1, N, nullptr, db, N, s);
        return rc;
    }
    Carver c{static_cast<uint8_t*>(ws)};
    uint8_t* yq = c.take(packed_codes(M, N));
    uint8_t* ys = c.take(packed_scales(M, N));
    uint8_t* ytq = c.take(packed_codes(N, M));
    uint8_t* yts = c.take(packed_scales(N, M));
    uint8_t* xtq = c.take(packed_codes(K, M));
    uint8_t* xts = c.take(packed_scales(K, M));
    float* partial = reinterpret_cast<float*>(c.at);
    rc = fp4_quantize_both_run(fmt, dtype, M, N, dY, lddy, dy_tscale, dX ? yq : nullptr, dX ? ys : nullptr,
                               dW ? ytq : nullptr, dW ? yts : nullptr, db, partial, s);
    if (rc || K == 0) return rc;
    if (dW) {
        rc = fp4_quantize_both_run(fmt, dtype, M, K, X, ldx, x_tscale, nullptr, nullptr, xtq, xts, nullptr, nullptr, s);
        if (rc) return rc;
    }
    if (dX) {
        rc = fp4_gemm_run(fmt, dtype, M, K, N, {yq, ys, M, dy_tscale}, {Wtq, Wts, K, w_tscale}, nullptr, dX, lddx,
                          false, dev, s);
        if (rc) return rc;
    }
    if (dW)
        rc = fp4_gemm_run(fmt, dtype, N, K, M, {ytq, yts, N, dy_tscale}, {xtq, xts, K, x_tscale}, nullptr, dW, lddw,
                          false, dev, s);
    return rc;
}

}  // extern "C"
