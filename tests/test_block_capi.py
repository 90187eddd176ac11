"""CPU checks of the C ABI of the microscaled 4-bit operators and layer norm:
sizes, refusals before any GPU work, and the kernels' resource table."""
import pytest

import bit_quantized_tensor_gb300 as qg
from bit_quantized_tensor_gb300 import budget

P = 0x10000  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return qg.lib()


def test_packed_sizes(L):
    assert [L.qg_fp4_codes_ld(k) for k in (0, 1, 32, 33, 4096)] == [0, 16, 16, 32, 2048]
    assert L.qg_fp4_scale_bytes(0, 1, 1) == 512
    assert L.qg_fp4_scale_bytes(0, 129, 65) == 2 * 2 * 512   # 5 blocks of 16
    assert L.qg_fp4_scale_bytes(1, 129, 65) == 2 * 1 * 512   # 3 blocks of 32
    assert L.qg_fp4_scale_bytes(2, 1, 1) == 0 and L.qg_fp4_scale_bytes(0, 0, 5) == 0


def test_workspace_sizes(L):
    ws = L.qg_workspace_size
    assert ws(qg.QG_OP_FP4_LINEAR, 17, 4096, 4096) == 17 * 2048 + 64 * 512
    assert ws(qg.QG_OP_FP4_LINEAR, 16, 4096, 4096) == 0  # quantized inside the product
    assert ws(qg.QG_OP_LAYER_NORM_BACKWARD, 1, 1, 100) >= 2 * 100 * 4
    assert ws(qg.QG_OP_FP4_TENSOR_SCALE, 1, 1, 1) > 0
    assert ws(qg.QG_OP_FP4_LINEAR_BACKWARD, 64, 64, 64) > 0


def _quant(L, fmt=0, dt=1, M=4, K=64, X=P, ld=64, ts=None, q=P, s=P):
    return L.fp4_quantize(fmt, dt, M, K, X, ld, ts, q, s, None)


def test_quantize_refusals(L):
    assert _quant(L, fmt=2) == 2 and _quant(L, dt=3) == 2
    assert _quant(L, M=-1) == 1 and _quant(L, K=-1) == 1 and _quant(L, ld=63) == 1
    assert _quant(L, X=None) == 1 and _quant(L, q=None) == 1 and _quant(L, s=None) == 1
    assert _quant(L, fmt=1, ts=P) == 2                       # mx has no tensor scale
    assert _quant(L, X=P + 1) == 3 and _quant(L, q=P + 8) == 3 and _quant(L, ts=P + 2) == 3
    assert _quant(L, M=0) == 0 and _quant(L, K=0) == 0       # nothing to do
    assert L.fp4_quantize_both(0, 1, 4, 64, P, 64, None, P, None, P, P, None) == 1
    assert L.fp4_quantize_both(0, 1, 4, 64, P, 64, None, None, None, None, P, None) == 1
    assert L.fp4_dequantize(0, 1, 4, 64, P, None, None, P, 64, None) == 1
    assert L.fp4_dequantize(0, 1, 4, 64, P, P, None, P, 60, None) == 1
    assert L.fp4_tensor_scale(1, 4, 64, P, 64, None, P, 4096, None) == 1
    assert L.fp4_tensor_scale(1, 4, 64, P, 64, P, P, 100, None) == 4
    assert L.fp4_tensor_scale(1, 4, 64, P, 64, P, P + 4, 4096, None) == 3


def _gemm(L, fmt=0, dt=1, M=4, N=8, K=64, a=P, sa=P, ta=None, b=P, sb=P, tb=None, bias=None, Y=P, ldy=8):
    return L.fp4_gemm(fmt, dt, M, N, K, a, sa, ta, b, sb, tb, bias, Y, ldy, None)


def _linear(L, fmt=0, dt=1, M=40, N=8, K=64, X=P, ldx=64, w=P, sw=P, Y=P, ldy=8, ws=P, wsb=BIG):
    return L.fp4_linear(fmt, dt, M, N, K, X, ldx, None, w, sw, None, None, Y, ldy, ws, wsb, None)


def test_product_refusals(L):
    assert _gemm(L, fmt=7) == 2 and _gemm(L, dt=-1) == 2 and _gemm(L, fmt=1, ta=P) == 2 and _gemm(L, fmt=1, tb=P) == 2
    assert _gemm(L, M=-1) == 1 and _gemm(L, K=(1 << 27) + 1) == 1 and _gemm(L, ldy=7) == 1
    for name in ("a", "sa", "b", "sb", "Y"):
        assert _gemm(L, **{name: None}) == 1, name
    for name in ("a", "sa", "b", "sb"):
        assert _gemm(L, **{name: P + 8}) == 3, name
    assert _gemm(L, bias=P + 1) == 3 and _gemm(L, Y=P + 1) == 3
    assert _gemm(L, M=0) == 0 and _gemm(L, N=0) == 0
    assert _linear(L, ws=None) == 4 and _linear(L, wsb=16) == 4 and _linear(L, ws=P + 16) == 3
    assert _linear(L, ldx=60) == 1 and _linear(L, X=None) == 1 and _linear(L, w=P + 4) == 3
    assert _linear(L, M=0) == 0


def test_cut_refusals(L):
    for tokens, splits in ((8, 0), (-1, 0), (512, 0), (0, 3), (0, 16), (0, -1)):
        assert L.qg_set_fp4_path(tokens, splits) == 1
    assert L.qg_set_fp4_path(0, 0) == 0


def _backward(L, fmt=0, dt=1, M=4, N=8, K=64, dY=P, lddy=8, X=P, ldx=64, w=P, sw=P, dX=P, lddx=64, dW=P, lddw=64,
              db=P, ws=P, wsb=BIG):
    return L.fp4_linear_backward(fmt, dt, M, N, K, dY, lddy, None, X, ldx, None, w, sw, None, dX, lddx, dW, lddw, db,
                                 ws, wsb, None)


def test_backward_refusals(L):
    assert _backward(L, dX=None, dW=None, db=None) == 1
    assert _backward(L, dY=None) == 1 and _backward(L, X=None) == 1 and _backward(L, w=None) == 1
    assert _backward(L, lddy=7) == 1 and _backward(L, ldx=63) == 1 and _backward(L, lddx=63) == 1
    assert _backward(L, lddw=63) == 1 and _backward(L, db=P + 2) == 3 and _backward(L, dW=P + 1) == 3
    assert _backward(L, ws=None) == 4 and _backward(L, wsb=64) == 4 and _backward(L, ws=P + 32) == 3


def test_norm_refusals(L):
    f = lambda dt=1, M=4, D=64, X=P, ldx=64, g=P, wd=1, eps=1e-5, Y=P, ldy=64: L.layer_norm(  # noqa: E731
        dt, M, D, X, ldx, g, g, wd, eps, Y, ldy, None, None, None)
    assert f(dt=4) == 2 and f(wd=0) == 2 and f(D=0) == 1 and f(M=-1) == 1 and f(eps=-1e-9) == 1
    assert f(eps=float("nan")) == 1 and f(X=None) == 1 and f(Y=None) == 1 and f(ldx=63) == 1 and f(ldy=63) == 1
    assert f(X=P + 1) == 3 and f(g=P + 1) == 3 and f(Y=P + 1) == 3 and f(M=0) == 0
    g = lambda fmt=0, ts=None, q=P, s=P: L.layer_norm_fp4(  # noqa: E731
        fmt, 1, 4, 64, P, 64, None, None, 1, 1e-5, ts, q, s, None, None, None)
    assert g(fmt=3) == 2 and g(fmt=1, ts=P) == 2 and g(q=None) == 1 and g(s=P + 4) == 3
    h = lambda dY=P, X=P, mean=P, dX=P, dg=P, ws=P, wsb=BIG, D=64: L.layer_norm_backward(  # noqa: E731
        1, 4, D, dY, 64, X, 64, None, 1, mean, P, dX, 64, dg, P, ws, wsb, None)
    assert h(dY=None) == 1 and h(X=None) == 1 and h(mean=None) == 1 and h(dX=None) == 1 and h(dg=None) == 1
    assert h(ws=None) == 4 and h(wsb=8) == 4 and h(ws=P + 8) == 3 and h(D=0) == 1


def test_no_gpu_reports_cuda_error(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _quant(L) == _gemm(L) == _linear(L) == _backward(L) == qg.QG_ERR_CUDA


def test_kernel_table(L):
    rows = qg.kernel_budgets(table="block")
    names = [r["kernel"] for r in rows]
    assert len(names) == len(set(names))
    for stem in ("k_fp4_quantize<", "k_fp4_quantize_both<", "k_fp4_amax<", "k_fp4_scale_join", "k_fp4_dequantize<",
                 "fp4_gemm_kernel<", "k_layer_norm<", "k_layer_norm_backward<", "k_sum_partials"):
        assert any(n.startswith(stem) for n in names), stem
    bad = {r["kernel"]: budget.accounting_errors(r) for r in rows if budget.accounting_errors(r)}
    assert not bad, bad
    with pytest.raises(ValueError):
        qg.kernel_budgets(table="other")


@pytest.mark.gpu
def test_device_residency_matches_the_design(L):
    for r in qg.kernel_budgets(measure=True, table="block"):
        assert r["static_smem_bytes"] + r["smem_bytes"] <= budget.CTA_SMEM_LIMIT, r
        assert r["ctas_per_sm"] >= r["min_ctas_per_sm"], r
        assert r["ctas_per_sm"] * r["tmem_cols"] <= budget.TMEM_COLUMNS, r
