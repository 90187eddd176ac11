"""Layer norm, forward, fused with the quantizer and backward, against 64 bits.

Bounds.  The statistics are fp32 sums over D values in trees of at most
32 + 10 additions a thread chain, so mean is off by at most 64 2^-24 of the
mean magnitude and rstd by at most 128 2^-24 of itself; y then by the sum of
these through (x - mean) rstd gamma + beta, and half a unit of its type.
"""
import numpy as np
import pytest

from tests import _block_ref as ref
from tests.test_fp4_gpu import HALF_UNIT, as_np, on_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5


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


def rows(M, D, seed, offset=0.5):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((M, D)) * np.exp(rng.standard_normal((M, 1))) + offset).astype(np.float32)


def params(torch, D, dtype, seed=9):
    rng = np.random.default_rng(seed)
    return (on_gpu(torch, (1 + 0.2 * rng.standard_normal(D)).astype(np.float32), dtype),
            on_gpu(torch, (0.3 * rng.standard_normal(D)).astype(np.float32), dtype))


def check_forward(got, X, gamma, beta, dtype):
    x = as_np(X)
    y, mean, rstd = ref.layer_norm(x, None if gamma is None else as_np(gamma), None if beta is None else as_np(beta), EPS)
    e_mean = 64 * 2.0 ** -24 * np.abs(x).mean(axis=1)
    # a shift of the mean by e changes the variance by e^2, and (x - mean) by e
    e_rstd = rstd * (128 * 2.0 ** -24 + (e_mean * rstd) ** 2 / 2)
    assert np.all(np.abs(as_np(got[1]) - mean) <= e_mean + 2.0 ** -149)
    assert np.all(np.abs(as_np(got[2]) - rstd) <= e_rstd)
    g = 1.0 if gamma is None else np.abs(as_np(gamma))
    b = 0.0 if beta is None else np.abs(as_np(beta))
    c = np.abs(x - mean[:, None])
    # the subtraction rounds at the size of its result only: x and mean are near each other or not
    e_y = g * (c * e_rstd[:, None] + (e_mean[:, None] + 2.0 ** -24 * c) * rstd[:, None]) + 4 * 2.0 ** -24 * (np.abs(y) + b)
    bound = e_y + HALF_UNIT[dtype] * np.abs(y) * 1.01 + (2.0 ** -25 if dtype == "float16" else 2.0 ** -149)
    err = np.abs(as_np(got[0]) - y)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])


LENGTHS = [1, 2, 7, 8, 31, 33, 128, 515, 1000, 1024, 1333, 2048, 4096, 4100, 8192, 10000, 33000]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("D", LENGTHS)
@pytest.mark.parametrize("M", [1, 3, 200])
def test_forward(torch, qg, M, D, dtype):
    X = on_gpu(torch, rows(M, D, M + D), dtype)
    g, b = params(torch, D, dtype)
    check_forward(qg.layer_norm(X, g, b, EPS), X, g, b, dtype)
    if M == 3:
        g, b = params(torch, D, "float32")
        check_forward(qg.layer_norm(X, g, None, EPS), X, g, None, dtype)
        check_forward(qg.layer_norm(X, None, b, EPS), X, None, b, dtype)
        # rows of another stride and alignment, in and out
        wide = torch.empty((M, D + 11), dtype=X.dtype, device="cuda")
        wide[:, 5:D + 5] = X
        out = torch.full_like(wide, 7.0)
        check_forward(qg.layer_norm(wide[:, 5:D + 5], g, b, EPS, Y=out[:, 2:D + 2]), X, g, b, dtype)
        assert bool((out[:, :2] == 7).all()) and bool((out[:, D + 2:] == 7).all())


def test_far_offset_and_constant_rows(torch, qg):
    X = on_gpu(torch, rows(5, 777, 3, offset=1000.0))
    check_forward(qg.layer_norm(X, None, None, EPS), X, None, None, "float32")
    flat = torch.full((3, 96), 2.5, device="cuda")
    y, mean, rstd = qg.layer_norm(flat, None, None, EPS)
    assert not bool(y.any()) and bool((mean == 2.5).all())
    assert np.allclose(as_np(rstd), 1 / np.sqrt(EPS), rtol=1e-6)


def test_not_finite_stays_in_its_row(torch, qg):
    X = on_gpu(torch, rows(6, 300, 5))
    X[1, 7] = float("nan")
    X[4, 0] = float("inf")
    y, _, _ = qg.layer_norm(X, None, None, EPS)
    assert as_np(torch.isnan(y).all(dim=1)).tolist() == [False, True, False, False, True, False]
    q, s, _, _ = qg.layer_norm_fp4(X, None, None, EPS)
    v = qg.fp4_dequantize(q, s, 300)
    assert as_np(torch.isnan(v).all(dim=1)).tolist() == [False, True, False, False, True, False]
    assert not bool(torch.isnan(v[[0, 2, 3, 5]]).any())


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,D", [(1, 1), (1, 4096), (3, 33), (130, 100), (200, 128), (5, 515), (129, 1000),
                                 (300, 2304), (3, 5000), (2, 9001), (2, 33000)])
def test_forward_to_codes(torch, qg, M, D, fmt, dtype):
    """The codes are those of y as fp32 (its values, not rounded to the type of x)."""
    X = on_gpu(torch, rows(M, D, 7 + D), dtype)
    g, b = params(torch, D, dtype)
    scale = torch.full((1,), 0.03, device="cuda") if fmt == "nv" and M % 2 else None
    q, s, mean, rstd = qg.layer_norm_fp4(X, g, b, EPS, fmt, scale=scale, stats=True)
    q2, s2, none, none2 = qg.layer_norm_fp4(X, g, b, EPS, fmt, scale=scale)
    assert torch.equal(q, q2) and torch.equal(s, s2) and none is None and none2 is None
    _, mean2, rstd2 = qg.layer_norm(X, g, b, EPS)
    # same statistics as the plain norm up to the order of the sums
    assert np.allclose(as_np(mean), as_np(mean2), rtol=1e-5, atol=1e-6) and np.allclose(as_np(rstd), as_np(rstd2), rtol=1e-5)
    # y rebuilt from those statistics in 64 bits: fp32 rounding may move a value across a
    # rounding boundary of its code or block scale, in one of 10^4 places at most (and one)
    x = as_np(X)
    y = ((x - as_np(mean)[:, None]) * as_np(rstd)[:, None] * as_np(g) + as_np(b)).astype(np.float32)
    code, byte = ref.codes_and_bytes(y, fmt, 0.03 if scale is not None else 1.0)
    q_ref, s_ref = ref.pack(code, byte)
    assert q.shape == q_ref.shape and s.shape == s_ref.shape
    assert np.count_nonzero(as_np(s) != s_ref) <= 1 + s_ref.size // 10000
    assert np.count_nonzero(as_np(q) != q_ref) <= 16 + q_ref.size // 5000


# ------------------------------------------------------------- backward

def check_backward(torch, got, dY, X, gamma, dtype):
    """fp32 sums over D (rows) and over M (columns), from statistics that are fp32 themselves."""
    x, dy = as_np(X), as_np(dY)
    g = None if gamma is None else as_np(gamma)
    dx, dg, db = ref.layer_norm_backward(dy, x, g, EPS)
    _, mean, rstd = ref.layer_norm(x, None, None, EPS)
    e_mean = 64 * 2.0 ** -24 * np.abs(x).mean(axis=1, keepdims=True)
    r = rstd[:, None]
    e_rel = 136 * 2.0 ** -24 + (e_mean * r) ** 2 / 2
    xh = (x - mean[:, None]) * r
    e_xh = np.abs(xh) * e_rel + e_mean * r
    d = np.abs(dy if g is None else dy * g)
    s1, s2 = d.mean(axis=1, keepdims=True), (d * np.abs(xh)).mean(axis=1, keepdims=True)
    e_s2 = 64 * 2.0 ** -24 * s2 + (d * e_xh).mean(axis=1, keepdims=True)
    total = d + s1 + np.abs(xh) * s2
    e_dx = r * (total * (e_rel + 8 * 2.0 ** -24) + 64 * 2.0 ** -24 * s1 + e_xh * s2 + np.abs(xh) * e_s2)
    bound = e_dx + HALF_UNIT[dtype] * np.abs(dx) * 1.01 + (2.0 ** -25 if dtype == "float16" else 2.0 ** -149)
    err = np.abs(as_np(got[0]) - dx)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])
    chain = 2.0 ** -24 * (64 + x.shape[0] / 8)
    e_dg = chain * (np.abs(dy) * np.abs(xh)).sum(axis=0) + (np.abs(dy) * e_xh).sum(axis=0)
    assert np.all(np.abs(as_np(got[1]) - dg) <= e_dg + 2.0 ** -149)
    assert np.all(np.abs(as_np(got[2]) - db) <= chain * np.abs(dy).sum(axis=0) + 2.0 ** -149)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("D", [1, 2, 7, 40, 256, 300, 515, 1000, 1024, 1333, 2048, 4096, 4100, 8192, 8200, 33000])
@pytest.mark.parametrize("M", [1, 3, 700])
def test_backward(torch, qg, M, D, dtype):
    if M == 700 and D > 9000:
        M = 150
    X = on_gpu(torch, rows(M, D, 2 * M + D), dtype)
    dY = on_gpu(torch, 0.1 * rows(M, D, 3 * M + D, offset=0.1), dtype)
    g, _ = params(torch, D, dtype)
    _, mean, rstd = qg.layer_norm(X, g, None, EPS)
    got = qg.layer_norm_backward(dY, X, g, mean, rstd)
    check_backward(torch, got, dY, X, g, dtype)
    again = qg.layer_norm_backward(dY, X, g, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    if M == 3:
        check_backward(torch, qg.layer_norm_backward(dY, X, None, mean, rstd), dY, X, None, dtype)
        g, _ = params(torch, D, "float32")
        wide, wide_y = (torch.zeros((M, D + 11), dtype=X.dtype, device="cuda") for _ in range(2))
        wide[:, 5:D + 5] = X
        wide_y[:, 1:D + 1] = dY
        out = torch.full_like(wide, 7.0)
        dg, db = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        got = qg.layer_norm_backward(wide_y[:, 1:D + 1], wide[:, 5:D + 5], g, mean, rstd, out=(out[:, 3:D + 3], dg, db))
        check_backward(torch, got, dY, X, g, dtype)
        assert bool((out[:, :3] == 7).all()) and bool((out[:, D + 3:] == 7).all())


def test_backward_against_differences(torch, qg):
    X, dY = rows(3, 10, 70).astype(np.float64), rows(3, 10, 71).astype(np.float64)
    g, b = (as_np(t) for t in params(torch, 10, "float32"))
    Xt = on_gpu(torch, X.astype(np.float32))
    gt = on_gpu(torch, g.astype(np.float32))
    _, mean, rstd = qg.layer_norm(Xt, gt, None, EPS)
    dx, dg, db = (as_np(t) for t in qg.layer_norm_backward(on_gpu(torch, dY.astype(np.float32)), Xt, gt, mean, rstd))
    X, dY = as_np(Xt), dY.astype(np.float32).astype(np.float64)
    h = 1e-5

    def loss(X, g, b):
        return float((ref.layer_norm(X, g, b, EPS)[0] * dY).sum())

    for i in range(3):
        for j in range(10):
            e = np.zeros_like(X)
            e[i, j] = h
            assert abs((loss(X + e, g, b) - loss(X - e, g, b)) / (2 * h) - dx[i, j]) < 1e-4
    for j in range(10):
        e = np.zeros(10)
        e[j] = h
        assert abs((loss(X, g + e, b) - loss(X, g - e, b)) / (2 * h) - dg[j]) < 1e-4
        assert abs((loss(X, g, b + e) - loss(X, g, b - e)) / (2 * h) - db[j]) < 1e-4


def test_no_rows(torch, qg):
    X = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = qg.layer_norm(X)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dg, db = qg.layer_norm_backward(X, X, None, mean, rstd)
    assert dx.shape == (0, 64) and not bool(dg.any()) and not bool(db.any())


def test_refusals(torch, qg):
    X = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    stats = torch.ones(4, device="cuda")
    with pytest.raises(TypeError, match="gamma"):
        qg.layer_norm(X, g.half())
    with pytest.raises(TypeError, match="same type"):
        qg.layer_norm(X, g, g.float())
    with pytest.raises(ValueError, match="gamma"):
        qg.layer_norm(X, g[:63])
    with pytest.raises(ValueError, match="contiguous last"):
        qg.layer_norm(X.t())
    with pytest.raises(TypeError, match="CUDA"):
        qg.layer_norm(X, g.cpu())
    with pytest.raises(qg.QgError, match="QG_ERR_INVALID_ARG"):
        qg.layer_norm(X, g, eps=-1.0)
    with pytest.raises(qg.QgError, match="QG_ERR_INVALID_ARG"):
        qg.layer_norm(X, g, eps=float("nan"))
    with pytest.raises(qg.QgError, match="QG_ERR_INVALID_ARG"):
        qg.layer_norm(X[:, :0])
    with pytest.raises(TypeError, match="dY"):
        qg.layer_norm_backward(X.half(), X, g, stats, stats)
    with pytest.raises(ValueError, match="mean"):
        qg.layer_norm_backward(X, X, g, stats[:3], stats)
    with pytest.raises(qg.QgError, match="QG_ERR_WORKSPACE"):
        qg.layer_norm_backward(X, X, g, stats, stats, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_after_measuring_the_table(torch, qg):
    """Measuring the kernels' residency leaves them launchable with more shared memory
    than the table's entry (which is that of the longest row, not of the fullest ring)."""
    qg.kernel_budgets(measure=True, table="block")
    for D in (1000, 1333, 2048, 4100):
        X = on_gpu(torch, rows(200, D, D), "float32")
        g, b = params(torch, D, "float32")
        check_forward(qg.layer_norm(X, g, b, EPS), X, g, b, "float32")
        qg.layer_norm_backward(X, X, g, *qg.layer_norm(X, g, b, EPS)[1:])
