// Products of microscaled 4-bit operands: fp4_gemm (both packed), fp4_linear
// (activations quantized in the call) and fp4_linear_backward (gradients of
// the activations, the weights and the bias).  Kernels: fp4_gemm.cuh
// (one CTA a tile) and fp4_gemm2.cuh (CTA pairs).
#include <atomic>

#include "fp4_gemm2.cuh"

namespace qg {

struct Fp4Operand {
    const uint8_t *codes, *scales;
    int64_t rows;
    const float* ts;
};

static int codes_map(CUtensorMap* map, const Fp4Operand& o, int64_t K, int box_rows) {
    return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, o.codes, fp4_codes_ld(K), o.rows, fp4_codes_ld(K), 128,
                        box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles as rows of 128 32-bit words.
static int scales_map(CUtensorMap* map, const Fp4Operand& o, int fmt, int64_t K, int atoms) {
    return make_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, o.scales, 128, fp4_scale_bytes(fmt, o.rows, K) / 512,
                        512, 128, atoms, CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <class Cfg, class QUANT>
static int launch_fp4(const Fp4Operand& x, const Fp4Operand& w, Fp4Params p, int splits, cudaStream_t s) {
    struct Flags {};  // the kernel's own shared-memory flag below
    // a tile of fewer than 128 tokens holds all of them (plan_fp4 sees to it): another one
    // would begin inside 128 scale rows, at a column of tensor memory that is none of theirs
    if (Cfg::NT < 128 && p.M > Cfg::NT) return QG_ERR_UNSUPPORTED;
    CUtensorMap tw, tx, tsw, tsx;
    int rc = codes_map(&tw, w, p.K, 128);
    if (!rc) rc = scales_map(&tsw, w, Cfg::FMT, p.K, Cfg::ATOMS);
    if constexpr (std::is_void<QUANT>::value) {
        if (!rc) rc = codes_map(&tx, x, p.K, Cfg::NT);
        if (!rc) rc = scales_map(&tsx, x, Cfg::FMT, p.K, Cfg::ATOMS);
    } else {  // not used
        tx = tw;
        tsx = tsw;
    }
    if (!rc) rc = raise_smem<Flags>(fp4_gemm_kernel<Cfg, QUANT>);
    if (rc) return rc;
    const int64_t gx = (int64_t(p.N) + 127) / 128 * splits, gy = (int64_t(p.M) + Cfg::NT - 1) / Cfg::NT;
    if (gy > kMaxGridY) return QG_ERR_UNSUPPORTED;  // not by plan_fp4
    while ((1 << p.log_splits) < splits) ++p.log_splits;
    return launch_serialized(fp4_gemm_kernel<Cfg, QUANT>,
                             dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kFp4Threads,
                             splits > 1 ? Cfg::SMEM_JOIN_BYTES : Cfg::SMEM_BYTES, splits, s, tw, tx, tsw, tsx, p);
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

// How a product is cut (qg_set_fp4_path): 0 by the rule below, else the
// tokens of a tile (256: CTA pairs) and the splits of K (0: by the rule).
static std::atomic<int> g_fp4_nt{0}, g_fp4_splits{0};

struct Fp4Plan {
    int nt, splits;
};

// Splits of K over a cluster: doubled while a CTA an SM takes them and each keeps
// a K block, or, up to two CTAs an SM (16 tokens a tile: two fit), while each
// keeps eight.  Measured (us, a call in a chain): 1 x 4096 x 4096 4.2 with 4
// splits, 4.8 with 8; 16 x 8192 x 8192 7.7 with 4, 9.7 with 2; 8 x 1024 x 2048
// 3.0 with 8, 3.4 with 4.
static int choose_splits(int64_t tiles, int64_t num_kb, int nt, int sms) {
    int s = 1;
    while (s < 8 && 2 * s <= num_kb) {
        const int64_t ctas = tiles * s * 2;
        if (!(ctas <= (nt == 128 ? sms / 2 : sms) || (nt == 16 && ctas <= 2 * sms && num_kb >= 16 * s))) break;
        s *= 2;
    }
    return s;
}

// Estimates in microseconds, fitted to products of 64 to 2048 tokens: a pair's
// tile takes 0.30 a K block, a 128-token tile 0.37, and a cluster's join grows
// with the number of CTAs that exchange sums at once.
//   2048 x 2048 x 2048: pairs 8.2, single CTAs 18;  128 x 4096 x 4096: 10.5, 11.3;
//   100 x 300 x 8192: pairs 14, single CTAs with 8 splits 8.3.  Rows of Y that are
// not 32-byte aligned cost pairs 3 more: 777 x 1001 x 2304 11.8, single CTAs 10.2.
static double pair_time(int64_t M, int64_t N, int64_t kb, bool sectors, int sms) {
    const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256), pairs = sms > 1 ? sms / 2 : 1;
    return (sectors ? 3.6 : 6.6) +
           static_cast<double>((tiles + pairs - 1) / pairs) * (0.30 * static_cast<double>(kb) + 0.6);
}
static double single_time(int64_t M, int64_t N, int64_t kb, int splits, int sms) {
    const int64_t ctas = (M + 127) / 128 * ((N + 127) / 128) * splits;
    return 5.0 + static_cast<double>((ctas + sms - 1) / sms) * 0.37 * static_cast<double>(kb) / splits +
           (splits > 1 ? 2.0 + 0.06 * static_cast<double>(ctas) : 0.0);
}

static bool whole_sectors(const void* Y, int64_t ldy, int dtype) {
    return (reinterpret_cast<uintptr_t>(Y) & 31u) == 0 && static_cast<size_t>(ldy) * dtype_bytes(dtype) % 32 == 0;
}

static Fp4Plan plan_fp4(int64_t M, int64_t N, int64_t K, bool sectors, int sms) {
    Fp4Plan f{g_fp4_nt.load(), g_fp4_splits.load()};
    const int64_t kb = (K + kFp4Bk - 1) / kFp4Bk;
    if (f.nt < M && f.nt && f.nt < 128) f.nt = 128;  // smaller tiles hold all tokens
    const bool chosen = f.nt != 0;
    if (!chosen) f.nt = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    if (!f.splits) f.splits = choose_splits((N + 127) / 128 * ((M + f.nt - 1) / f.nt), kb, f.nt, sms);
    // a grid's y counts the single CTAs' tiles of tokens; pairs walk over any number
    if (f.nt == 128 && (M + 127) / 128 > kMaxGridY) f.nt = 256;
    if (!chosen && f.nt == 128 && pair_time(M, N, kb, sectors, sms) < single_time(M, N, kb, f.splits, sms)) f.nt = 256;
    if (f.nt == 256 || f.splits > kb) f.splits = 1;
    return f;
}

template <int FMT>
static int run_fmt(const Fp4Operand& x, const Fp4Operand& w, const Fp4Params& p, const Fp4Plan& f, int dev,
                   cudaStream_t s) {
    switch (f.nt) {
        case 16: return launch_fp4<Fp4Cfg<FMT, 16>, void>(x, w, p, f.splits, s);
        case 32: return launch_fp4<Fp4Cfg<FMT, 32>, void>(x, w, p, f.splits, s);
        case 64: return launch_fp4<Fp4Cfg<FMT, 64>, void>(x, w, p, f.splits, s);
        case 128: return launch_fp4<Fp4Cfg<FMT, 128>, void>(x, w, p, f.splits, s);
        default: return launch_fp4_pair<Fp4PairCfg<FMT>>(x, w, p, dev, s);
    }
}

static Fp4Params fp4_params(int dtype, int64_t M, int64_t N, int64_t K, const Fp4Operand& x, const Fp4Operand& w,
                            const void* bias, void* Y, int64_t ldy, bool weights_ready, int dev) {
    Fp4Params p = {};
    p.M = static_cast<int>(M); p.N = static_cast<int>(N); p.K = static_cast<int>(K);
    p.ts_a = x.ts; p.ts_b = w.ts; p.bias = bias; p.Y = Y; p.ldy = ldy; p.dtype = dtype;
    p.weights_ready = weights_ready;
    p.ctl = host_ctl(dev);
    return p;
}

// Y (M x N) = alpha X . W^T + bias, K >= 0.
static int fp4_gemm_run(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const Fp4Operand& x,
                        const Fp4Operand& w, const void* bias, void* Y, int64_t ldy, bool weights_ready, int dev,
                        cudaStream_t s) {
    const Fp4Params p = fp4_params(dtype, M, N, K, x, w, bias, Y, ldy, weights_ready, dev);
    if (!p.ctl.status) return QG_ERR_CUDA;
    const Fp4Plan f = plan_fp4(M, N, K, whole_sectors(Y, ldy, dtype), num_sms(dev));
    return fmt == kNv ? run_fmt<kNv>(x, w, p, f, dev, s) : run_fmt<kMx>(x, w, p, f, dev, s);
}

// The product of up to 16 tokens that are still values: one kernel.
static int fp4_linear_few(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                          const float* x_ts, const Fp4Operand& w, const void* bias, void* Y, int64_t ldy, int dev,
                          cudaStream_t s) {
    const Fp4Operand x{nullptr, nullptr, M, x_ts};
    Fp4Params p = fp4_params(dtype, M, N, K, x, w, bias, Y, ldy, false, dev);
    if (!p.ctl.status) return QG_ERR_CUDA;
    p.X = X;
    p.ldx = ldx;
    p.x_aligned = aligned16(X) && (M <= 1 || static_cast<size_t>(ldx) * dtype_bytes(dtype) % 16 == 0);
    const Fp4Plan f = plan_fp4(M, N, K, whole_sectors(Y, ldy, dtype), num_sms(dev));
    return by_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        return fmt == kNv ? launch_fp4<Fp4Cfg<kNv, 16>, T>(x, w, p, f.splits, s)
                          : launch_fp4<Fp4Cfg<kMx, 16>, T>(x, w, p, f.splits, s);
    });
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

// Are M tokens quantized inside the product's kernel?
static bool quantized_inside(int64_t M) {
    const int nt = g_fp4_nt.load();
    return M <= 16 && (nt == 0 || nt == 16);
}

size_t fp4_linear_workspace(int64_t M, int64_t K) {
    return quantized_inside(M) ? 0 : packed_codes(M, K) + packed_scales(M, K);
}

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

#define QG_FP4_GEMM_BUDGET(FMT, FNAME, NT, QUANT, QNAME)                                              \
    QG_BLOCK_KERNEL_BUDGET("fp4_gemm_kernel<" FNAME "," #NT "," QNAME ">",                            \
                           (reinterpret_cast<const void*>(fp4_gemm_kernel<Fp4Cfg<FMT, NT>, QUANT>)),  \
                           kFp4Threads, (Fp4Cfg<FMT, NT>::SMEM_JOIN_BYTES), (Fp4Cfg<FMT, NT>::TMEM_COLS), 8, \
                           1)
#define QG_FP4_GEMM_BUDGETS(FMT, FNAME)                                                               \
    QG_FP4_GEMM_BUDGET(FMT, FNAME, 16, void, "packed"); QG_FP4_GEMM_BUDGET(FMT, FNAME, 32, void, "packed"); \
    QG_FP4_GEMM_BUDGET(FMT, FNAME, 64, void, "packed"); QG_FP4_GEMM_BUDGET(FMT, FNAME, 128, void, "packed"); \
    QG_FP4_GEMM_BUDGET(FMT, FNAME, 16, __half, "f16"); QG_FP4_GEMM_BUDGET(FMT, FNAME, 16, float, "f32"); \
    QG_FP4_GEMM_BUDGET(FMT, FNAME, 16, __nv_bfloat16, "bf16")
QG_FP4_GEMM_BUDGETS(kNv, "nv");
QG_FP4_GEMM_BUDGETS(kMx, "mx");
QG_BLOCK_KERNEL_BUDGET("fp4_gemm2_kernel<nv>", reinterpret_cast<const void*>(fp4_gemm2_kernel<Fp4PairCfg<kNv>>),
                       Fp4PairCfg<kNv>::THREADS, Fp4PairCfg<kNv>::SMEM_BYTES, 512, 2, 1);
QG_BLOCK_KERNEL_BUDGET("fp4_gemm2_kernel<mx>", reinterpret_cast<const void*>(fp4_gemm2_kernel<Fp4PairCfg<kMx>>),
                       Fp4PairCfg<kMx>::THREADS, Fp4PairCfg<kMx>::SMEM_BYTES, 512, 2, 1);
QG_BLOCK_KERNEL_BUDGET("k_fp4_only_bias", reinterpret_cast<const void*>(k_fp4_only_bias), 256, 0, 0, 1, 4);

// Checks shared by the three calls.
static int check_product(int fmt, int dtype, int64_t M, int64_t N, int64_t K, const float* ta, const float* tb) {
    if (!fmt_ok(fmt) || !dtype_ok(dtype)) return QG_ERR_UNSUPPORTED;
    if (M < 0 || N < 0 || K < 0 || M > (1 << 27) || N > (1 << 27) || K > (1 << 27)) return QG_ERR_INVALID_ARG;
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

int qg_set_fp4_path(int tokens, int splits) {
    if (tokens != 0 && tokens != 16 && tokens != 32 && tokens != 64 && tokens != 128 && tokens != 256)
        return QG_ERR_INVALID_ARG;
    if (splits != 0 && splits != 1 && splits != 2 && splits != 4 && splits != 8) return QG_ERR_INVALID_ARG;
    g_fp4_nt.store(tokens);
    g_fp4_splits.store(splits);
    return QG_OK;
}

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
    const bool inside = quantized_inside(M);
    if (K > 0 && !inside && (!ws || ws_bytes < fp4_linear_workspace(M, K))) return QG_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return QG_ERR_MISALIGNED;
    const int dev = current_device();
    if (dev < 0 || dev >= 64) return QG_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) return only_bias(dtype, M, N, bias, Y, ldy, s);
    if (inside)
        return fp4_linear_few(fmt, dtype, M, N, K, X, ldx, x_tscale, {Wq, Ws, N, w_tscale}, bias, Y, ldy, dev, s);
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
