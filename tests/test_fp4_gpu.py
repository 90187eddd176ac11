"""Microscaled 4-bit quantizers and products on the GPU against the plain 64-bit forms.

Codes and scale bytes are compared bit for bit.  A product's bound: the tensor
core adds the sums of 64 products each, every addition off by at most 2^-22 of
what has been added so far, so |y - ref| <= (K / 64 + 8) 2^-22 sum |a b| plus
half a unit of the output type.
"""
import numpy as np
import pytest

from tests import _block_ref as ref

pytestmark = pytest.mark.gpu

HALF_UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}


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


def activations(rows, K, seed, big=1.0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1))) * big).astype(np.float32)


def on_gpu(torch, a, dtype="float32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", getattr(torch, dtype))


def as_np(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def packed(torch, X, fmt, ts=1.0):
    code, byte = ref.codes_and_bytes(X, fmt, ts)
    q, s = ref.pack(code, byte)
    return on_gpu(torch, q, "uint8"), on_gpu(torch, s, "uint8")


def one(torch, ts):
    return torch.full((1,), float(ts), dtype=torch.float32, device="cuda")


# ------------------------------------------------------------- quantizers

SHAPES = [(1, 1), (1, 16), (2, 31), (3, 33), (130, 47), (128, 64), (5, 129), (257, 500), (1, 4096), (33, 1000)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,K", SHAPES)
def test_quantize_bits(torch, qg, M, K, fmt, dtype):
    X = on_gpu(torch, activations(M, K, 100 + M + K), dtype)
    ts = 0.0123 if fmt == "nv" and M % 2 else 1.0
    scale = one(torch, ts) if ts != 1.0 else None
    ts = float(np.float32(ts))
    q, s = qg.fp4_quantize(X, fmt, scale=scale)
    q_ref, s_ref = ref.pack(*ref.codes_and_bytes(X.float().cpu().numpy(), fmt, ts))
    assert np.array_equal(as_np(s), s_ref)
    assert np.array_equal(as_np(q), q_ref)
    both = qg.fp4_quantize_both(X, fmt, scale=scale)
    t_ref = ref.pack(*ref.codes_and_bytes(X.t().float().cpu().numpy(), fmt, ts))
    for got, want in zip(both, (q_ref, s_ref) + t_ref):
        assert np.array_equal(as_np(got), want)
    # and back: fl(code d) with d = fl(s ts), rounded once more to the type
    code, byte = ref.codes_and_bytes(X.float().cpu().numpy(), fmt, ts)
    d = (ref.scale_values(byte, fmt).astype(np.float32) * np.float32(ts)).astype(np.float32)
    v = (ref.code_values(code).reshape(M, -1, ref.BLOCK[fmt]).astype(np.float32) * d[:, :, None]).astype(np.float32)
    want = torch.from_numpy(v.reshape(M, -1)[:, :K].copy()).to(getattr(torch, dtype))
    got = qg.fp4_dequantize(q, s, K, fmt, scale=scale, dtype=getattr(torch, dtype))
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_strided_and_misaligned_rows(torch, qg, fmt, dtype):
    for M, K, ld, off in [(5, 100, 128, 0), (5, 100, 104, 8), (7, 65, 67, 1), (130, 64, 71, 3), (1, 40, 41, 1)]:
        buf = on_gpu(torch, activations(1, M * ld + off + 8, 7 + K), dtype)[0]
        X = buf[off:off + M * ld].as_strided((M, K), (ld, 1))
        for got, want in zip(qg.fp4_quantize_both(X, fmt), qg.fp4_quantize_both(X.contiguous(), fmt)):
            assert torch.equal(got, want)
        want = qg.fp4_quantize(X.contiguous(), fmt)
        for got, w in zip(qg.fp4_quantize(X, fmt), want):
            assert torch.equal(got, w)
        # values back into strided, misaligned rows, the gaps untouched
        out = torch.full_like(buf, 7.0)
        Y = out[off:off + M * ld].as_strided((M, K), (ld, 1))
        qg.fp4_dequantize(*want, K, fmt, Y=Y)
        assert torch.equal(Y, qg.fp4_dequantize(*want, K, fmt, dtype=X.dtype))
        mask = torch.ones_like(out, dtype=torch.bool)
        mask[off:off + M * ld].as_strided((M, K), (ld, 1)).fill_(False)
        assert bool((out[mask] == 7.0).all())


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_ties_extremes_and_zeros(torch, qg, fmt):
    b = ref.BLOCK[fmt]
    rows = [np.zeros(b), -np.zeros(b), np.full(b, 1e-44), np.full(b, 6 * 2.0 ** -11), np.full(b, 6 * 2.0 ** -10),
            np.full(b, 6 * 2.0 ** -9), np.full(b, 2688.0), np.full(b, 1e6), np.full(b, -3.0e38),
            np.resize([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25, -0.75, -0.25, -6], b),
            np.resize([7.99, 6.5, 5.0001, 4.9999, 0.2500001, -7.9], b)]
    X = np.stack(rows).astype(np.float32)
    for ts in (1.0, 0.37) if fmt == "nv" else (1.0,):
        q, s = qg.fp4_quantize(on_gpu(torch, X), fmt, scale=one(torch, ts) if ts != 1 else None)
        q_ref, s_ref = ref.pack(*ref.codes_and_bytes(X, fmt, ts))
        assert np.array_equal(as_np(s), s_ref)
        assert np.array_equal(as_np(q), q_ref)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_not_finite_stays_in_its_block(torch, qg, fmt):
    b = ref.BLOCK[fmt]
    X = activations(40, 5 * b, 11)
    X[3, b] = np.nan
    X[4, 2 * b + 1] = np.inf
    X[5, 0] = -np.inf
    q, s, tq, ts = qg.fp4_quantize_both(on_gpu(torch, X), fmt)
    for K, rows, (c, y) in ((5 * b, X, (q, s)), (40, X.T, (tq, ts))):
        got = as_np(qg.fp4_dequantize(c, y, K, fmt))
        want = ref.quantized(rows, fmt)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])
    # a product with it: NaN in the rows that hold it, nowhere else
    w = activations(33, 5 * b, 12)
    y = as_np(qg.fp4_linear(on_gpu(torch, X), *packed(torch, w, fmt), fmt))
    assert np.array_equal(np.isnan(y).all(axis=1), np.isin(np.arange(40), (3, 4, 5)))
    assert np.array_equal(np.isnan(y).any(axis=1), np.isin(np.arange(40), (3, 4, 5)))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 33), (300, 1111), (1, 100000), (2048, 8)])
def test_tensor_scale(torch, qg, M, K, dtype):
    X = on_gpu(torch, activations(M, K, 13 + K, 1e-3), dtype)
    wide = torch.zeros((M, K + 3), dtype=X.dtype, device="cuda")
    wide[:, :K] = X
    wide[:, K:] = 100.0
    want = np.float32(float(X.float().abs().max())) * np.float32(1 / np.float32(2688))
    assert float(qg.fp4_tensor_scale(X)) == want
    assert float(qg.fp4_tensor_scale(wide[:, :K])) == want
    X[0, 0] = float("inf")
    X[-1, -1] = float("nan")
    rest = X[torch.isfinite(X)].float().abs()
    want = np.float32(float(rest.max()) if len(rest) else 0) * np.float32(1 / np.float32(2688)) or 1.0
    assert float(qg.fp4_tensor_scale(X)) == want
    assert float(qg.fp4_tensor_scale(torch.zeros_like(X))) == 1.0
    assert float(qg.fp4_tensor_scale(X[:0])) == 1.0


# ------------------------------------------------------------- products

def check_product(y, va, vb, alpha, bias, dtype):
    """y against alpha * va . vb^T + bias in 64 bits (bound: the module's docstring)."""
    want = alpha * (va @ vb.T)
    size = alpha * (np.abs(va) @ np.abs(vb).T)
    if bias is not None:
        want = want + bias
        size = size + np.abs(bias)
    bound = (va.shape[1] / 64 + 8) * 2.0 ** -22 * size + HALF_UNIT[dtype] * np.abs(want) * 1.01 + 2.0 ** -25
    err = np.abs(as_np(y) - want)
    assert err.shape == bound.shape
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])


PRODUCTS = [(1, 1, 1), (1, 130, 4096), (2, 64, 16), (15, 129, 65), (16, 128, 256), (17, 200, 257), (33, 7, 511),
            (64, 128, 1024), (65, 300, 63), (127, 128, 64), (128, 256, 512), (129, 131, 1000), (200, 1, 96),
            (257, 513, 320), (300, 640, 2048), (513, 1025, 700)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_gemm(torch, qg, M, N, K, fmt, dtype):
    a, b = activations(M, K, 20 + M), activations(N, K, 21 + N, 0.05)
    bias = on_gpu(torch, activations(1, N, 22)[0], dtype)
    ta, tb = (0.5, 0.0007) if fmt == "nv" else (1.0, 1.0)
    va, vb = ref.quantized(a, fmt, ta), ref.quantized(b, fmt, tb)
    sa, sb = (one(torch, ta), one(torch, tb)) if fmt == "nv" else (None, None)
    y = qg.fp4_gemm(*packed(torch, a, fmt, ta), *packed(torch, b, fmt, tb), K, fmt, a_scale=sa, b_scale=sb,
                    bias=bias, dtype=getattr(torch, dtype))
    alpha = float(np.float32(ta)) * float(np.float32(tb))
    check_product(y, va, vb, alpha, as_np(bias), dtype)
    # rows with a stride of their own, and no bias
    wide = torch.full((M, N + 5), 7.0, dtype=y.dtype, device="cuda")
    out = qg.fp4_gemm(*packed(torch, a, fmt, ta), *packed(torch, b, fmt, tb), K, fmt, a_scale=sa, b_scale=sb,
                      Y=wide[:, 3:N + 3])
    check_product(out, va, vb, alpha, None, dtype)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, N + 3:] == 7).all())


CUTS = [(16, 1), (16, 2), (16, 4), (16, 8), (32, 1), (32, 4), (64, 1), (64, 2), (128, 1), (128, 2), (128, 8), (256, 0)]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("tokens,splits", CUTS)
def test_every_cut_of_a_product(torch, qg, tokens, splits, fmt):
    """Each tile and split, with tokens that fill a tile, that leave some out and that need several."""
    try:
        assert qg.lib().qg_set_fp4_path(tokens, splits) == qg.QG_OK
        for M, N, K in [(1, 130, 2100), (tokens, 257, 2048), (min(tokens, 128) - 3, 128, 1057), (261, 300, 2111)]:
            a, b = activations(M, K, 70 + M), activations(N, K, 71 + N, 0.05)
            bias = on_gpu(torch, activations(1, N, 22)[0], "float16")
            pa, pb = packed(torch, a, fmt), packed(torch, b, fmt)
            want = ref.quantized(a, fmt), ref.quantized(b, fmt)
            y = qg.fp4_gemm(*pa, *pb, K, fmt, bias=bias, dtype=torch.float16)
            check_product(y, *want, 1.0, as_np(bias), "float16")
            assert torch.equal(y, qg.fp4_gemm(*pa, *pb, K, fmt, bias=bias, dtype=torch.float16))
            X = on_gpu(torch, a)
            check_product(qg.fp4_linear(X, *pb, fmt), *want, 1.0, None, "float32")
    finally:
        qg.lib().qg_set_fp4_path(0, 0)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_products_of_nothing(torch, qg, fmt, dtype):
    dt = getattr(torch, dtype)
    bias = on_gpu(torch, activations(1, 40, 3)[0], dtype)
    new = lambda r, k: qg.fp4_quantize(torch.ones((r, k), dtype=dt, device="cuda"), fmt)  # noqa: E731
    y = qg.fp4_gemm(*new(7, 0), *new(40, 0), 0, fmt, bias=bias, dtype=dt)
    assert torch.equal(y, bias.expand(7, 40))
    assert qg.fp4_gemm(*new(0, 32), *new(40, 32), 32, fmt, dtype=dt).shape == (0, 40)
    assert qg.fp4_linear(torch.ones((3, 0), dtype=dt, device="cuda"), *new(40, 0), fmt, bias=bias).equal(bias.expand(3, 40))
    assert qg.fp4_linear(torch.ones((3, 32), dtype=dt, device="cuda"), *new(0, 32), fmt).shape == (3, 0)
    # no tokens: no dX rows, the other gradients are sums over nothing
    dx, dw, db = qg.fp4_linear_backward(torch.ones((0, 40), dtype=dt, device="cuda"),
                                        torch.ones((0, 32), dtype=dt, device="cuda"), *new(32, 40), fmt)
    assert dx.shape == (0, 32) and not bool(dw.any()) and not bool(db.any()) and dw.shape == (40, 32)
    dx, dw, db = qg.fp4_linear_backward(torch.ones((3, 0), dtype=dt, device="cuda"),
                                        torch.ones((3, 32), dtype=dt, device="cuda"), *new(32, 0), fmt)
    assert dx.shape == (3, 32) and not bool(dx.any()) and dw.shape == (0, 32)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 1000, 777), (100, 260, 1030), (600, 512, 512)])
def test_linear_is_quantize_then_gemm(torch, qg, M, N, K, fmt):
    X = on_gpu(torch, activations(M, K, 30), "bfloat16")
    w = packed(torch, activations(N, K, 31, 0.02), fmt)
    bias = on_gpu(torch, activations(1, N, 32)[0], "bfloat16")
    xs = qg.fp4_tensor_scale(X) if fmt == "nv" else None
    q, s = qg.fp4_quantize(X, fmt, scale=xs)
    want = qg.fp4_gemm(q, s, *w, K, fmt, a_scale=xs, bias=bias)
    # (the same cut of K: one token to sixteen are quantized inside the product's kernel)
    assert torch.equal(qg.fp4_linear(X, *w, fmt, x_scale=xs, bias=bias), want)
    # strided activations, another stream, a workspace full of NaN bytes
    wide = torch.empty((M, K + 9), dtype=X.dtype, device="cuda")
    wide[:, 1:K + 1] = X
    ws = torch.full((max(256, qg.workspace_size(qg.QG_OP_FP4_LINEAR, M, N, K)),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = qg.fp4_linear(wide[:, 1:K + 1], *w, fmt, x_scale=xs, bias=bias, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_chain_in_a_graph_sees_new_inputs(torch, qg, fmt):
    """quantize, product and gradient captured once and replayed on other inputs."""
    M, N, K = 24, 384, 640
    X, dY = on_gpu(torch, activations(M, K, 40), "float16"), on_gpu(torch, activations(M, N, 41), "float16")
    w = on_gpu(torch, activations(N, K, 42, 0.05), "float16")
    wq, wsc, tq, tsc = qg.fp4_quantize_both(w, fmt)

    def step():
        return (qg.fp4_linear(X, wq, wsc, fmt),) + qg.fp4_linear_backward(dY, X, tq, tsc, fmt)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for seed in (43, 44):
        X.copy_(on_gpu(torch, activations(M, K, seed), "float16"))
        dY.copy_(on_gpu(torch, activations(M, N, seed + 10), "float16"))
        g.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, step()):
            assert torch.equal(got, want)


# ------------------------------------------------------------- gradients

@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 40, 70), (17, 129, 33), (130, 64, 256), (300, 257, 200),
                                   (515, 600, 640)])
def test_linear_backward(torch, qg, M, N, K, fmt, dtype):
    X = on_gpu(torch, activations(M, K, 50), dtype)
    dY = on_gpu(torch, activations(M, N, 51, 0.01), dtype)
    W = activations(N, K, 52, 0.1)
    tx, ty, tw = (0.011, 0.0003, 0.002) if fmt == "nv" else (1.0, 1.0, 1.0)
    kw = dict(dy_scale=one(torch, ty), x_scale=one(torch, tx), w_scale=one(torch, tw)) if fmt == "nv" else {}
    wt = packed(torch, W.T, fmt, tw)
    dx, dw, db = qg.fp4_linear_backward(dY, X, *wt, fmt, **kw)
    x, dy = X.float().cpu().numpy(), dY.float().cpu().numpy()
    f = lambda v: float(np.float32(v))  # noqa: E731
    check_product(dx, ref.quantized(dy, fmt, ty), ref.quantized(W.T, fmt, tw), f(ty) * f(tw), None, dtype)
    check_product(dw, ref.quantized(dy.T, fmt, ty), ref.quantized(x.T, fmt, tx), f(ty) * f(tx), None, dtype)
    # column sums: fp32 additions, at most 128 + M / 128 + 8 in a chain
    bound = (136 + M / 128) * 2.0 ** -24 * np.abs(dy.astype(np.float64)).sum(axis=0)
    assert np.all(np.abs(as_np(db) - dy.astype(np.float64).sum(axis=0)) <= bound)
    # each gradient alone is the same
    a = qg.fp4_linear_backward(dY, X, *wt, fmt, need_dw=False, need_db=False, **kw)
    b = qg.fp4_linear_backward(dY, X, *wt, fmt, need_dx=False, need_db=False, **kw)
    c = qg.fp4_linear_backward(dY, X, *wt, fmt, need_dx=False, need_dw=False, **kw)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert torch.equal(b[1], dw) and torch.equal(c[2], db) and c[0] is None


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_gradients_against_differences(torch, qg, fmt):
    """On operands that quantize exactly (every block holds a 6 and values of the
    grid) the layer is linear, and its gradients must match differences of it."""
    M, N, K = 32, 64, 96

    def exact(rows, cols, seed):
        rng = np.random.default_rng(seed)
        v = rng.choice(np.concatenate((ref.GRID, -ref.GRID)), size=(rows, cols))
        i, j = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
        return np.where((i + j) % 16 == 0, 6.0, v).astype(np.float32)

    X, W, dY = exact(M, K, 60), exact(N, K, 61), exact(M, N, 62)
    wt = packed(torch, W.T, fmt)
    dx, dw, db = (as_np(t) for t in qg.fp4_linear_backward(on_gpu(torch, dY), on_gpu(torch, X), *wt, fmt))

    def loss(X, W, bias):
        # exact in 64 bits: the kernel's own output for exact operands is compared in the other tests
        return float((dY.astype(np.float64) * (X.astype(np.float64) @ W.astype(np.float64).T + bias)).sum())

    y = as_np(qg.fp4_linear(on_gpu(torch, X), *packed(torch, W, fmt), fmt))
    assert np.array_equal(y, X.astype(np.float64) @ W.astype(np.float64).T)
    zero = np.zeros(N)
    rng = np.random.default_rng(63)
    for _ in range(40):
        i, j, n = rng.integers(M), rng.integers(K), rng.integers(N)
        e = np.zeros_like(X)
        e[i, j] = 1
        assert dx[i, j] == (loss(X + e, W, zero) - loss(X - e, W, zero)) / 2
        e = np.zeros_like(W)
        e[n, j] = 1
        assert dw[n, j] == (loss(X, W + e, zero) - loss(X, W - e, zero)) / 2
        e = np.zeros(N)
        e[n] = 1
        assert db[n] == (loss(X, W, e) - loss(X, W, -e)) / 2


# ------------------------------------------------------------- refusals

def test_refusals(torch, qg):
    X = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    q, s = qg.fp4_quantize(X, "nv")
    ts = one(torch, 1.0)
    with pytest.raises(ValueError, match="fmt"):
        qg.fp4_quantize(X, "fp4")
    with pytest.raises(TypeError, match="CUDA"):
        qg.fp4_quantize(X.cpu())
    with pytest.raises(TypeError, match="float16, bfloat16 or float32"):
        qg.fp4_quantize(X.double())
    with pytest.raises(ValueError, match="2-D"):
        qg.fp4_quantize(X[0])
    with pytest.raises(ValueError, match="contiguous last"):
        qg.fp4_quantize(X.t())
    with pytest.raises(ValueError, match="overlap"):
        qg.fp4_quantize(X[:1].expand(4, 64))
    with pytest.raises(ValueError, match="no tensor scale"):
        qg.fp4_quantize(X, "mx", scale=ts)
    with pytest.raises(TypeError, match="one float32"):
        qg.fp4_quantize(X, "nv", scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="bytes for K"):
        qg.fp4_gemm(q, s, q, s, 100, "nv")
    with pytest.raises(ValueError, match="scales do not match"):
        qg.fp4_gemm(q, s, q, s[..., :256].contiguous(), 64, "nv")
    wide, wide_s = qg.fp4_quantize(torch.ones((4, 128), dtype=torch.bfloat16, device="cuda"), "nv")
    with pytest.raises(ValueError, match="scales do not match"):
        qg.fp4_gemm(wide, wide_s, wide, wide_s, 128, "mx")  # packed as nv
    with pytest.raises(ValueError, match="bias"):
        qg.fp4_linear(X, q, s, "nv", bias=torch.ones(3, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError, match="bias"):
        qg.fp4_linear(X, q, s, "nv", bias=torch.ones(4, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="Y must be"):
        qg.fp4_linear(X, q, s, "nv", Y=torch.empty((4, 5), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(qg.QgError, match="QG_ERR_WORKSPACE"):
        qg.fp4_linear(X.repeat(10, 1), q, s, "nv", ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="W\\^T"):
        qg.fp4_linear_backward(torch.ones((4, 64), dtype=torch.bfloat16, device="cuda"), X, q, s, "nv")
    assert qg.fp4_linear(X, q, s, "nv").shape == (4, 4)  # and the context is intact
