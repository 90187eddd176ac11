"""8-bit operands with a scale for each row, and their products, against 64 bits.

Bounds.  Codes and scales are the definition's, bit for bit.  A product's integer sum is
exact; it is rounded to fp32, multiplied by one scale (a rounding each, 2^-24) and in one
fused step by the other with the bias added (a rounding of the result), and rounded to its
type (half a unit).
"""
import numpy as np
import pytest

from tests import _attention_ref as ref
from tests.test_fp4_gpu import HALF_UNIT, as_np, on_gpu

pytestmark = pytest.mark.gpu
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -149}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a CUDA device"
    return t


@pytest.fixture(scope="module")
def qg():
    import bit_quantized_tensor_gb300 as q
    q.lib()
    return q


@pytest.fixture(autouse=True)
def _no_device_timeouts(qg):
    yield
    assert qg.device_status() == qg.QG_OK


def values(M, K, seed):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))).astype(np.float32)


def check_codes(got, X):
    q, s = ref.s8_quantize(as_np(X))
    assert np.array_equal(as_np(got[0]), q) and np.array_equal(as_np(got[1]).astype(np.float32), s, equal_nan=True)


def check_product(Y, qa, sa, qb, sb, bias, dtype):
    total = qa.astype(np.float64) @ qb.astype(np.float64).T
    size = np.abs(total) * sa[:, None].astype(np.float64) * sb[None, :].astype(np.float64)
    y = total * sa[:, None].astype(np.float64) * sb[None, :].astype(np.float64)
    if bias is not None:
        y = y + as_np(bias)
    bound = 2.02 * 2.0 ** -24 * size + (1.01 * 2.0 ** -24 + 1.01 * HALF_UNIT[dtype]) * np.abs(y) + TINY[dtype]
    err = np.abs(as_np(Y) - y)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("K", [1, 7, 8, 16, 17, 100, 1000, 1024, 1025, 4096, 4100, 16384, 16385, 40000])
@pytest.mark.parametrize("M", [1, 5, 130])
def test_quantize(torch, qg, M, K, dtype):
    X = on_gpu(torch, values(M, K, M + K), dtype)
    if M == 5:
        X[1] = 0
        X[3] = 2.0 ** -140 if dtype == "float32" else 0
    check_codes(qg.s8_quantize(X), X)
    wide = torch.empty((M, K + 7), dtype=X.dtype, device="cuda")
    wide[:, 3:K + 3] = X
    check_codes(qg.s8_quantize(wide[:, 3:K + 3]), X)


def test_quantize_marks_rows_that_are_not_finite(torch, qg):
    X = on_gpu(torch, values(4, 300, 1), "float32")
    X[1, 299], X[2, 0] = float("nan"), -float("inf")
    q, s = qg.s8_quantize(X)
    check_codes((q, s), X)
    assert as_np(torch.isnan(s)).tolist() == [False, True, True, False] and not bool(q[1:3].any())
    big = torch.full((2, 40), 3.3e38, device="cuda")
    check_codes(qg.s8_quantize(big), big)


SIZES = [(1, 1, 1), (1, 16, 16), (1, 17, 63), (1, 333, 4096), (3, 40, 65), (8, 100, 1000), (9, 64, 2049), (16, 129, 512),
         (17, 64, 64), (16, 48, 20000), (33, 1001, 2304), (128, 256, 1040), (130, 300, 777), (257, 515, 1100),
         (300, 260, 4097), (512, 512, 512), (4100, 261, 1100)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_products(torch, qg, M, N, K, dtype):
    X, W = on_gpu(torch, values(M, K, 1), dtype), on_gpu(torch, values(N, K, 2), "float32")
    bias = on_gpu(torch, np.random.default_rng(3).standard_normal(N).astype(np.float32), dtype)
    (qa, sa), (qb, sb) = ref.s8_quantize(as_np(X)), ref.s8_quantize(as_np(W))
    Wq, Ws = qg.s8_quantize(W)
    Y = qg.s8_linear(X, Wq, Ws, bias=bias)
    assert Y.dtype == X.dtype
    check_product(Y, qa, sa, qb, sb, bias, dtype)
    Xq, Xs = qg.s8_quantize(X)
    assert torch.equal(qg.s8_gemm(Xq, Xs, Wq, Ws, K, bias=bias, dtype=X.dtype), Y)
    check_product(qg.s8_gemm(Xq, Xs, Wq, Ws, K, dtype=X.dtype), qa, sa, qb, sb, None, dtype)
    # rows of another stride and alignment in and out; what lies between stays
    wide, out = torch.empty((M, K + 5), dtype=X.dtype, device="cuda"), torch.full((M, N + 3), 7.0, dtype=X.dtype, device="cuda")
    wide[:, 1:K + 1] = X
    qg.s8_linear(wide[:, 1:K + 1], Wq, Ws, bias=bias, Y=out[:, 2:N + 2])
    assert torch.equal(out[:, 2:N + 2], Y) and bool((out[:, :2] == 7).all()) and bool((out[:, N + 2:] == 7).all())


def test_sums_are_exact_at_their_largest(torch, qg):
    """Every code at its largest: sums of 2^30, far over what fp32 holds exactly."""
    for M, N, K in ((2, 20, 65536 + 48), (16, 16, 4096), (140, 270, 65536 + 48)):
        q, s = torch.full((M, K), 127, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
        w, t = torch.full((N, K), 127, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
        w[:, ::2] = -126
        w[0] = 127
        Y = qg.s8_gemm(q, s, w, t, K, dtype=torch.float32)
        want = 127 * w.double().sum(1)
        assert torch.equal(Y, want.float().expand(M, N))


@pytest.mark.parametrize("M,N,K", [(4200003, 24, 32), (1, 4200003, 32), (3, 4200003, 32), (40, 1100003, 32), (70001, 40, 16)])
def test_many_tokens_and_channels(torch, qg, M, N, K):
    """Grids and offsets far from small: the first, some middle and the last rows and columns."""
    gen = torch.Generator(device="cuda").manual_seed(M % 1000)
    X, W = (torch.randn(r, K, generator=gen, device="cuda").half() for r in (M, N))
    Wq, Ws = qg.s8_quantize(W)
    Xq, Xs = qg.s8_quantize(X)
    Y = qg.s8_linear(X, Wq, Ws)
    rows, cols = (torch.cat([torch.arange(n, device="cuda")[i:i + 40] for i in (0, n // 2, max(0, n - 40))]).unique() for n in (M, N))
    for t, q, scale, at in ((X, Xq, Xs, rows), (W, Wq, Ws, cols)):
        want, s = ref.s8_quantize(as_np(t[at]))
        assert np.array_equal(as_np(q[at]), want) and np.array_equal(as_np(scale[at]).astype(np.float32), s)
    qa, sa, qb, sb = (as_np(t) for t in (Xq[rows], Xs[rows], Wq[cols], Ws[cols]))
    check_product(Y[rows][:, cols], qa, sa.astype(np.float32), qb, sb.astype(np.float32), None, "float16")


def test_scales_whose_product_with_the_sum_alone_leaves_fp32(torch, qg):
    """Tokens near fp32's largest against weights near its smallest scales, in every kernel, and the other way round."""
    for M, N, K in ((1, 40, 512), (5, 40, 512), (60, 40, 512), (1500, 2100, 512)):
        for x, w in ((118, -90), (-90, 118)):
            X, W = (on_gpu(torch, values(r, K, r), "float32") * 2.0 ** f for r, f in ((M, x), (N, w)))
            Wq, Ws = qg.s8_quantize(W)
            (qa, sa), (qb, sb) = ref.s8_quantize(as_np(X)), ref.s8_quantize(as_np(W))
            Y = qg.s8_linear(X, Wq, Ws)
            assert bool(torch.isfinite(Y).all())
            check_product(Y, qa, sa, qb, sb, None, "float32")


def test_what_lies_behind_k_does_not_count(torch, qg):
    for M in (2, 40):
        X, W = on_gpu(torch, values(M, 100, 1), "bfloat16"), on_gpu(torch, values(50, 100, 2), "float32")
        Wq, Ws = qg.s8_quantize(W)
        Y = qg.s8_linear(X, Wq, Ws)
        Wq[:, 100:] = 99
        assert torch.equal(qg.s8_linear(X, Wq, Ws), Y)
        Xq, Xs = qg.s8_quantize(X)
        Xq[:, 100:] = -5
        assert torch.equal(qg.s8_gemm(Xq, Xs, qg.s8_quantize(W)[0], Ws, 100), Y)
        assert torch.equal(qg.s8_gemm(Xq, Xs, Wq, Ws, 100), Y)


def test_not_finite_stays_in_its_row_and_column(torch, qg):
    for M in (4, 40):
        X, W = on_gpu(torch, values(M, 96, 1), "float16"), on_gpu(torch, values(24, 96, 2), "float32")
        X[2, 5] = float("inf")
        W[7, 1] = float("nan")
        Y = qg.s8_linear(X, *qg.s8_quantize(W))
        nan = as_np(torch.isnan(Y))
        want = np.zeros((M, 24), bool)
        want[2], want[:, 7] = True, True
        assert np.array_equal(nan, want)


def test_empty(torch, qg):
    X, W = torch.zeros((0, 32), device="cuda"), torch.zeros((5, 32), device="cuda")
    Wq, Ws = qg.s8_quantize(W)
    assert qg.s8_linear(X, Wq, Ws).shape == (0, 5)
    bias = torch.arange(5.0, device="cuda")
    none = torch.zeros((3, 0), device="cuda")
    Y = qg.s8_linear(none, torch.zeros((5, 0), dtype=torch.int8, device="cuda"), Ws, bias=bias)
    assert torch.equal(Y, bias.expand(3, 5))
    assert qg.s8_quantize(none)[0].shape == (3, 0)


def test_streams_graph_and_repeats(torch, qg):
    for M in (2, 100):
        X, W = on_gpu(torch, values(M, 1000, 1), "bfloat16"), on_gpu(torch, values(200, 1000, 2), "float32")
        Wq, Ws = qg.s8_quantize(W)
        Y = qg.s8_linear(X, Wq, Ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        Z = qg.s8_linear(X, Wq, Ws, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q, s = qg.s8_quantize(W)  # written by the kernel just ahead of the product
            out = qg.s8_linear(X, q, s)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, Y)
