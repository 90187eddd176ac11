"""Run one operation of the library once (after one warm-up call) on seeded
synthetic inputs, for profilers such as Nsight Compute.

    python -m bit_quantized_tensor_gb300.profile_case OP [--m M] [--n N] [--k K]

OP is one of s8, s4, f16 (M x N x K GEMMs), w4a16 (M x N x K with group 128),
w4a4_quant (M x K activations with rank-32 projection) or w4a4_gemm
(M x N x K, rank 32, bias); of the microscaled 4-bit operators fp4_quant
(M x K bf16), fp4_both (both directions), fp4_gemm, fp4_linear and fp4_backward
(M x N x K); norm, norm_fp4 and norm_backward (M x K).  --fmt picks the 4-bit
format, --dtype the type of values (bf16, f16, f32).  Sizes default to 2048 each.  Prints one line
with the call's device time from CUDA events (a number taken under a
profiler is not a benchmark figure).
"""
import argparse
import sys

import numpy as np


def _block_case(qg, torch, a, dev):
    """The call of a microscaled 4-bit operator or of layer norm, as a function."""
    M, N, K, fmt = a.m, a.n, a.k, a.fmt
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[a.dtype]
    g = torch.Generator(device=dev).manual_seed(1005)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    def scale(v):
        return qg.fp4_tensor_scale(v) if fmt == "nv" else None

    X = normal(M, K)
    if a.op == "fp4_quant":
        xs = scale(X)
        return lambda: qg.fp4_quantize(X, fmt, scale=xs)
    if a.op == "fp4_both":
        xs = scale(X)
        return lambda: qg.fp4_quantize_both(X, fmt, scale=xs)
    if a.op.startswith("norm"):
        gamma, beta = normal(K), normal(K)
        if a.op == "norm":
            return lambda: qg.layer_norm(X, gamma, beta)
        if a.op == "norm_fp4":
            return lambda: qg.layer_norm_fp4(X, gamma, beta, fmt=fmt)
        dY = normal(M, K)
        _, mean, rstd = qg.layer_norm(X, gamma, beta)
        return lambda: qg.layer_norm_backward(dY, X, gamma, mean, rstd)
    W = normal(N, K)
    xs, ws = scale(X), scale(W)
    Wq, Ws, Wtq, Wts = qg.fp4_quantize_both(W, fmt, scale=ws)
    if a.op == "fp4_linear":
        return lambda: qg.fp4_linear(X, Wq, Ws, fmt, x_scale=xs, w_scale=ws)
    if a.op == "fp4_gemm":
        Xq, Xs = qg.fp4_quantize(X, fmt, scale=xs)
        return lambda: qg.fp4_gemm(Xq, Xs, Wq, Ws, K, fmt, a_scale=xs, b_scale=ws, dtype=dtype)
    dY = normal(M, N)
    return lambda: qg.fp4_linear_backward(dY, X, Wtq, Wts, fmt, dy_scale=scale(dY), x_scale=xs, w_scale=ws)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("op", choices=["s8", "s4", "f16", "w4a16", "w4a4_quant", "w4a4_gemm", "fp4_quant", "fp4_both", "fp4_gemm",
                                  "fp4_linear", "fp4_backward", "norm", "norm_fp4", "norm_backward"])
    ap.add_argument("--m", type=int, default=2048)
    ap.add_argument("--n", type=int, default=2048)
    ap.add_argument("--k", type=int, default=2048)
    ap.add_argument("--fmt", choices=["nv", "mx"], default="nv")
    ap.add_argument("--dtype", choices=["bf16", "f16", "f32"], default="bf16")
    a = ap.parse_args(argv)

    import torch

    import bit_quantized_tensor_gb300 as qg
    from bit_quantized_tensor_gb300 import inputs

    if not torch.cuda.is_available():
        sys.exit("profile_case needs a CUDA device")
    dev = torch.device("cuda:0")
    qg.lib()
    M, N, K = a.m, a.n, a.k

    def t(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(dev)

    if a.op == "s8":
        A, B = t(inputs.s8_uniform(M, K, 1000)), t(inputs.s8_uniform(N, K, 2000))
        run = lambda: qg.qgemm_s8(A, B)  # noqa: E731
    elif a.op == "s4":
        A, B = t(inputs.s4_packed_uniform(M, K, 1001)), t(inputs.s4_packed_uniform(N, K, 2001))
        run = lambda: qg.qgemm_s4(A, B, K)  # noqa: E731
    elif a.op == "f16":
        A, B = t(inputs.f16_normal(M, K, 1002)), t(inputs.f16_normal(N, K, 2002))
        run = lambda: qg.gemm_f16(A, B)  # noqa: E731
    elif a.op == "w4a16":
        X = t(inputs.f16_normal(M, K, 1003))
        Wq = t(inputs.s4_packed_uniform(N, K, 2003))
        S = t(inputs.f16_uniform(N, K // 128, 0.005, 0.02, 3003))
        run = lambda: qg.w4a16_gemm(X, Wq, S)  # noqa: E731
    elif a.op == "w4a4_quant":
        X = t(inputs.f32_normal(M, K, 1004))
        Ut = t(inputs.f16_normal(K, 32, 3004, sigma=0.02).T)
        run = lambda: qg.w4a4_quantize(X, Ut)  # noqa: E731
    elif a.op.startswith(("fp4", "norm")):
        run = _block_case(qg, torch, a, dev)
    else:
        X = t(inputs.f32_normal(M, K, 1004))
        W = t(inputs.f32_normal(N, K, 2004))
        Ut = t(inputs.f16_normal(K, 32, 3004, sigma=0.02).T)
        Vt = t(inputs.f16_normal(32, N, 3005, sigma=0.02).T)
        b = t(inputs.f16_normal(1, N, 3006, sigma=0.1)[0])
        qx, sx, xu = qg.w4a4_quantize(X, Ut)
        qw, sw, _ = qg.w4a4_quantize(W)
        del X, W
        run = lambda: qg.w4a4_gemm(qx, sx, qw, sw, K, XU=xu, Vt=Vt, bias=b)  # noqa: E731

    run()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    run()
    e1.record()
    torch.cuda.synchronize()
    assert qg.device_status() == qg.QG_OK
    print(f"{a.op} M={M} N={N} K={K}: {e0.elapsed_time(e1) * 1e3:.1f} us (one call)")


if __name__ == "__main__":
    main()
