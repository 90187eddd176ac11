"""Layer norm of many rows at any place in a 16-byte piece, shorter than one,
against 64 bits.

Bounds as in test_norm_gpu (fp32 sums over D values in trees of at most 64 additions
a chain), with the 64-bit forms in torch on the GPU, since the matrices are large.
"""
import pytest

from tests.test_fp4_gpu import HALF_UNIT
from tests.test_norm_gpu import EPS, qg, torch, _no_device_timeouts  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def matrix(torch, M, D, dtype, seed, shift=None, size=1.0):
    """Values of spread row sizes; shift: a view that starts `shift` columns into rows of D + 11,
    with NaN around it."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn((M, D), device="cuda", generator=g) * torch.exp(torch.randn((M, 1), device="cuda", generator=g))
    x = ((x + 0.5) * size).to(getattr(torch, dtype))
    if shift is None:
        return x
    wide = torch.full((M, D + 11), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, shift:shift + D] = x
    return wide[:, shift:shift + D]


def vector(torch, D, dtype, seed, around):
    g = torch.Generator("cuda").manual_seed(seed)
    return (around + 0.2 * torch.randn(D, device="cuda", generator=g)).to(getattr(torch, dtype))


def exact_stats(x):
    mean = x.mean(1, keepdim=True)
    return mean, (((x - mean) ** 2).mean(1, keepdim=True) + EPS) ** -0.5


def least(dtype):
    return {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -149}[dtype]


def check_forward(torch, got, X, gamma, beta, dtype):
    x, g, b = X.double(), gamma.double(), beta.double()
    mean, rstd = exact_stats(x)
    y = (x - mean) * rstd * g + b
    e_mean = 64 * 2.0 ** -24 * x.abs().mean(1, keepdim=True)
    e_rstd = rstd * (128 * 2.0 ** -24 + (e_mean * rstd) ** 2 / 2)
    assert bool(((got[1].double() - mean[:, 0]).abs() <= e_mean[:, 0] + 2.0 ** -149).all())
    assert bool(((got[2].double() - rstd[:, 0]).abs() <= e_rstd[:, 0]).all())
    c = (x - mean).abs()
    e_y = g.abs() * (c * e_rstd + (e_mean + 2.0 ** -24 * c) * rstd) + 4 * 2.0 ** -24 * (y.abs() + b.abs())
    bound = e_y + HALF_UNIT[dtype] * y.abs() * 1.01 + least(dtype)
    bad = ~((got[0].double() - y).abs() <= bound)
    assert not bool(bad.any()), bad.nonzero()[:4]


def check_backward(torch, got, dY, X, gamma, dtype):
    x, dy, g = X.double(), dY.double(), gamma.double()
    mean, r = exact_stats(x)
    xh = (x - mean) * r
    d = dy * g
    dx = r * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
    e_mean = 64 * 2.0 ** -24 * x.abs().mean(1, keepdim=True)
    e_rel = 136 * 2.0 ** -24 + (e_mean * r) ** 2 / 2
    e_xh = xh.abs() * e_rel + e_mean * r
    d = d.abs()
    s1, s2 = d.mean(1, keepdim=True), (d * xh.abs()).mean(1, keepdim=True)
    e_s2 = 64 * 2.0 ** -24 * s2 + (d * e_xh).mean(1, keepdim=True)
    total = d + s1 + xh.abs() * s2
    e_dx = r * (total * (e_rel + 8 * 2.0 ** -24) + 64 * 2.0 ** -24 * s1 + e_xh * s2 + xh.abs() * e_s2)
    bad = ~((got[0].double() - dx).abs() <= e_dx + HALF_UNIT[dtype] * dx.abs() * 1.01 + least(dtype))
    assert not bool(bad.any()), bad.nonzero()[:4]
    chain = 2.0 ** -24 * (64 + x.shape[0] / 8)
    e_dg = chain * (dy * xh).abs().sum(0) + (dy.abs() * e_xh).sum(0)
    assert bool(((got[1].double() - (dy * xh).sum(0)).abs() <= e_dg + 2.0 ** -149).all())
    assert bool(((got[2].double() - dy.sum(0)).abs() <= chain * dy.abs().sum(0) + 2.0 ** -149).all())


# ------------------------------------------------------------- rows shorter than a piece

@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("off", [0, 1, 2, 3, 5, 7])
def test_short_rows_at_any_place(torch, qg, off, D, dtype):
    """Packed rows of a few bytes that begin anywhere in a piece, NaN before and behind them."""
    for M in (153, 1002, 20011):
        def placed(seed, size, shift):
            buf = torch.full((M * D + shift + 9,), float("nan"), dtype=getattr(torch, dtype), device="cuda")
            v = buf[shift:shift + M * D].view(M, D)
            v.copy_(matrix(torch, M, D, dtype, seed, size=size))
            return v

        X, dY, dY2 = placed(6 + M, 1.0, off), placed(7 + M, 0.1, off), placed(8 + M, 0.1, off // 2)
        gamma, beta = vector(torch, D, dtype, 8, 1.0), vector(torch, D, dtype, 9, 0.0)
        got = qg.layer_norm(X, gamma, beta, EPS)
        check_forward(torch, got, X, gamma, beta, dtype)
        for dy in (dY, dY2):  # at the same place as x, and at another
            check_backward(torch, qg.layer_norm_backward(dy, X, gamma, *got[1:]), dy, X, gamma, dtype)
        for fmt in ("nv", "mx"):
            q, s, mean, rstd = qg.layer_norm_fp4(X, gamma, beta, EPS, fmt, stats=True)
            y = ((X.double() - mean.double()[:, None]) * rstd.double()[:, None] * gamma.double() + beta.double()).float()
            q_ref, s_ref = qg.fp4_quantize(y, fmt)
            assert int((s != s_ref).sum()) <= 1 + s_ref.numel() // 10000
            assert int((q != q_ref).sum()) <= 16 + q_ref.numel() // 5000
