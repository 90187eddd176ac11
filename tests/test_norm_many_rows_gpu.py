"""Layer norm with more rows than the rings in shared memory hold at once: every
thread count a row at both ends of its range of lengths, rows at any place in a
16-byte piece, and rows shorter than one, against 64 bits.

Bounds as in test_norm_gpu (fp32 sums over D values in trees of at most 64 additions
a chain), with the 64-bit forms in torch on the GPU, since the matrices are large.
"""
import pytest

from tests.test_fp4_gpu import HALF_UNIT
from tests.test_norm_gpu import EPS, qg, torch, _no_device_timeouts  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def rows_for(D, elem, groups, slots_bytes):
    """Rows that walk every ring around more than once: groups, each with up to 8 slots."""
    slots = max(3, min(8, slots_bytes // (D * elem)))
    return groups * (slots + 1) + 37


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


def alike(a, b):
    """Equal bits (a row's NaN included)."""
    return all(bool(((u == v) | (u.isnan() & v.isnan())).all()) for u, v in zip(a, b))


# ------------------------------------------------------------- forward

FORWARD = [8, 33, 515, 1016, 1017, 1024, 1025, 4088, 4089, 4096, 4097, 8184, 8185, 8192, 8193, 16376, 16377, 16384]


@pytest.mark.parametrize("x_shift,y_shift", [(None, None), (5, 5), (5, 2), (None, 3)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D", FORWARD)
def test_forward(torch, qg, D, dtype, x_shift, y_shift):
    elem = 2 if dtype == "bfloat16" else 4
    groups, smem = (2432, 10240) if D <= 1024 else (608, 40960) if D <= 4096 else (304, 81920) if D <= 8192 else (152, 163840)
    M = rows_for(D, elem, groups, smem)
    X = matrix(torch, M, D, dtype, D, x_shift)
    wdtype = "float32" if x_shift is None else dtype  # fp32 weights beside 16-bit rows, too
    gamma, beta = vector(torch, D, wdtype, 1, 1.0), vector(torch, D, wdtype, 2, 0.0)
    if y_shift is None:
        got = qg.layer_norm(X, gamma, beta, EPS)
    else:
        wide = torch.full((M, D + 11), 7.0, dtype=X.dtype, device="cuda")
        got = qg.layer_norm(X, gamma, beta, EPS, Y=wide[:, y_shift:y_shift + D])
        assert bool((wide[:, :y_shift] == 7).all()) and bool((wide[:, y_shift + D:] == 7).all())
    check_forward(torch, got, X, gamma, beta, dtype)


# ------------------------------------------------------------- forward to codes

@pytest.mark.parametrize("shift", [None, 5])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("M,D", [(20011, 33), (20011, 64), (6001, 515), (5003, 1333), (2600, 2304), (1501, 5001), (1501, 8192),
                                 (700, 10001), (700, 16368)])
def test_forward_to_codes(torch, qg, M, D, fmt, dtype, shift):
    """The codes are those of y as fp32 with the statistics that the call gives."""
    X = matrix(torch, M, D, dtype, D + 1, shift)
    gamma, beta = vector(torch, D, dtype, 3, 1.0), vector(torch, D, dtype, 4, 0.0)
    scale = torch.full((1,), 0.03, device="cuda") if fmt == "nv" else None
    q, s, mean, rstd = qg.layer_norm_fp4(X, gamma, beta, EPS, fmt, scale=scale, stats=True)
    e_mean = 64 * 2.0 ** -24 * X.double().abs().mean(1)
    m, r = exact_stats(X.double())
    assert bool(((mean.double() - m[:, 0]).abs() <= e_mean + 2.0 ** -149).all())
    assert bool(((rstd.double() - r[:, 0]).abs() <= r[:, 0] * (128 * 2.0 ** -24 + (e_mean * r[:, 0]) ** 2 / 2)).all())
    y = ((X.double() - mean.double()[:, None]) * rstd.double()[:, None] * gamma.double() + beta.double()).float()
    q_ref, s_ref = qg.fp4_quantize(y, fmt, scale=scale)  # bit for bit the plain form's, see test_fp4_gpu
    # fp32 rounding of y may move a value across a rounding boundary of its code or block
    # scale, in one of 10^4 places at most (and one); a moved scale moves its block's codes
    assert int((s != s_ref).sum()) <= 1 + s_ref.numel() // 10000
    assert int((q != q_ref).sum()) <= 16 + q_ref.numel() // 5000


# ------------------------------------------------------------- backward

BACKWARD = [8, 33, 248, 249, 256, 257, 504, 512, 513, 760, 761, 768, 769, 1016, 1024, 1025, 2040, 2048, 2049, 4088, 4096, 4097,
            8184, 8185, 8191, 8192]


@pytest.mark.parametrize("x_shift,dy_shift,dx_shift", [(None, None, None), (5, 5, 5), (5, 1, 3), (None, 2, None)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D", BACKWARD)
def test_backward(torch, qg, D, dtype, x_shift, dy_shift, dx_shift):
    elem = 2 if dtype == "bfloat16" else 4
    groups = 152 * (16 if D <= 768 else 4 if D <= 2048 else 2 if D <= 4096 else 1)
    M = rows_for(D, elem, groups, 200 * 1024 * 152 // groups // 2)
    X, dY = matrix(torch, M, D, dtype, D + 2, x_shift), matrix(torch, M, D, dtype, D + 3, dy_shift, 0.1)
    gamma = vector(torch, D, "float32" if x_shift is None else dtype, 5, 1.0)
    _, mean, rstd = qg.layer_norm(X, gamma, None, EPS)

    def call():
        if dx_shift is None:
            return qg.layer_norm_backward(dY, X, gamma, mean, rstd)
        wide = torch.full((M, D + 11), 7.0, dtype=X.dtype, device="cuda")
        out = (wide[:, dx_shift:dx_shift + D], torch.empty(D, device="cuda"), torch.empty(D, device="cuda"))
        got = qg.layer_norm_backward(dY, X, gamma, mean, rstd, out=out)
        assert bool((wide[:, :dx_shift] == 7).all()) and bool((wide[:, dx_shift + D:] == 7).all())
        return got

    got = call()
    check_backward(torch, got, dY, X, gamma, dtype)
    assert alike(got, call())  # the same bits on every run


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
