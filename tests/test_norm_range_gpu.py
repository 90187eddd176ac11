"""Layer norm at the ends of its range: rows that are not finite, sizes of the
values far from 1, against 64 bits."""
import numpy as np
import pytest

from tests import _block_ref as ref
from tests.test_fp4_gpu import HALF_UNIT, as_np, on_gpu
from tests.test_norm_gpu import EPS, params, qg, rows, torch, _no_device_timeouts  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- codes behind the row

def scale_rows(s, rows_, fmt):
    """Scale bytes of the packed layout as (row, block), with the blocks behind the last one."""
    s = as_np(s)
    tr, tc, _ = s.shape
    return s.reshape(tr, tc, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(tr * 128, tc * 4)[:rows_]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,D", [(3, 100), (200, 100), (200, 33), (300, 515), (200, 1064), (200, 4100), (160, 8200)])
def test_codes_behind_rows_that_are_not_finite(torch, qg, M, D, fmt, dtype):
    """A NaN or an infinity makes all of its row NaN, but what lies behind the row stays 0."""
    X = on_gpu(torch, rows(M, D, 5 + D), dtype)
    X[1, D // 2] = float("nan")
    X[M - 1, 0] = float("inf")
    q, s, _, _ = qg.layer_norm_fp4(X, None, None, EPS, fmt)
    blocks = -(-D // ref.BLOCK[fmt])
    byte = scale_rows(s, M, fmt)
    assert not byte[:, blocks:].any()
    nan_scale = 0x7F if fmt == "nv" else 0xFF
    assert ((byte[:, :blocks] == nan_scale).all(axis=1) == np.isin(np.arange(M), (1, M - 1))).all()
    codes = as_np(q)
    codes = np.stack((codes & 15, codes >> 4), axis=2).reshape(M, -1)
    assert not codes[:, D:].any()


# ------------------------------------------------------------- gradients of large and small rows

def check_gradient(got, dY, X, gamma, eps, dtype):
    """As test_norm_gpu.check_backward, with eps given: fp32 sums over D (rows) and over M (columns), from
    statistics that are fp32 themselves; results near the smallest numbers round to multiples of 2^-149."""
    x, dy, g = as_np(X), as_np(dY), as_np(gamma)
    dx, dg, db = ref.layer_norm_backward(dy, x, g, eps)
    _, mean, rstd = ref.layer_norm(x, None, None, eps)
    r = rstd[:, None]
    e_mean = 64 * 2.0 ** -24 * np.abs(x).mean(axis=1, keepdims=True)
    e_rel = 136 * 2.0 ** -24 + (e_mean * r) ** 2 / 2
    xh = (x - mean[:, None]) * r
    e_xh = np.abs(xh) * e_rel + e_mean * r
    d = np.abs(dy * g)
    s1, s2 = d.mean(axis=1, keepdims=True), (d * np.abs(xh)).mean(axis=1, keepdims=True)
    e_s2 = 64 * 2.0 ** -24 * s2 + (d * e_xh).mean(axis=1, keepdims=True)
    total = d + s1 + np.abs(xh) * s2
    e_dx = r * (total * (e_rel + 8 * 2.0 ** -24) + 64 * 2.0 ** -24 * s1 + e_xh * s2 + np.abs(xh) * e_s2)
    least = 2.0 ** -133 if dtype == "bfloat16" else 2.0 ** -149
    bound = e_dx + HALF_UNIT[dtype] * np.abs(dx) * 1.01 + least
    err = np.abs(as_np(got[0]) - dx)
    assert np.all(err <= bound), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:4])
    chain = 2.0 ** -24 * (64 + x.shape[0] / 8)
    e_dg = chain * (np.abs(dy) * np.abs(xh)).sum(axis=0) + (np.abs(dy) * e_xh).sum(axis=0)
    assert np.all(np.abs(as_np(got[1]) - dg) <= e_dg + 2.0 ** -149 * x.shape[0])
    assert np.all(np.abs(as_np(got[2]) - db) <= chain * np.abs(dy).sum(axis=0) + 2.0 ** -149)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D", [64, 515, 1333, 5000, 8200])
@pytest.mark.parametrize("x_size,dy_size", [(2.0 ** 55, 2.0 ** -30), (2.0 ** -61, 2.0 ** 10), (2.0 ** -40, 2.0 ** -100),
                                            (2.0 ** 40, 2.0 ** -70)])
def test_gradient_far_from_one(torch, qg, D, x_size, dy_size, dtype):
    """rstd^2 and products of dy and x - mean leave fp32's range here; xh and the gradient do not."""
    M = 7
    X = on_gpu(torch, rows(M, D, D) * np.float32(x_size), dtype)
    dY = on_gpu(torch, rows(M, D, D + 1, offset=0.1) * np.float32(dy_size), dtype)
    g, _ = params(torch, D, "float32")
    _, mean, rstd = (on_gpu(torch, v) for v in ref.layer_norm(as_np(X), None, None, 0.0))
    check_gradient(qg.layer_norm_backward(dY, X, g, mean, rstd), dY, X, g, 0.0, dtype)
