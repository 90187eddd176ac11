"""Microscaled 4-bit products at the ends of their range: tensor scales whose product
leaves fp32's normal range."""
import numpy as np
import pytest

from tests import _block_ref as ref
from tests.test_fp4_gpu import activations, as_np, on_gpu, one, packed, qg, torch, _no_device_timeouts  # noqa: F401

pytestmark = pytest.mark.gpu

CUTS = [(16, 1), (16, 4), (64, 2), (128, 1), (128, 4), (256, 0)]


@pytest.mark.parametrize("tokens,splits", CUTS)
@pytest.mark.parametrize("ta,tb,big", [(1.37 * 2.0 ** -72, 1.59 * 2.0 ** -72, 1000.0), (1.37 * 2.0 ** -100, 1.1 * 2.0 ** -30, 1000.0),
                                       (1.37 * 2.0 ** 100, 1.59 * 2.0 ** 28, 0.02), (1.37 * 2.0 ** 28, 1.59 * 2.0 ** 100, 0.02)])
def test_products_of_extreme_tensor_scales(torch, qg, ta, tb, big, tokens, splits):
    """The result is in range though ta tb is not (subnormal, or infinite).  Bound: the
    accumulation's, two more roundings, and half of the smallest subnormal twice."""
    M, N, K = 16, 160, 1024
    ta, tb = float(np.float32(ta)), float(np.float32(tb))
    rng = np.random.default_rng(80)
    a, b = ((rng.standard_normal((rows, K)) * big * t).astype(np.float32) for rows, t in ((M, ta), (N, tb)))
    a[3] = 0
    va, vb = ref.quantized(a, "nv", ta), ref.quantized(b, "nv", tb)
    want = (va @ vb.T) * ta * tb
    assert np.isfinite(want).all() and np.abs(want).max() < 1e38 and np.abs(want).max() > 1e-37
    bound = (K / 64 + 12) * 2.0 ** -22 * (np.abs(va) @ np.abs(vb).T) * ta * tb + 2.0 ** -149
    try:
        assert qg.lib().qg_set_fp4_path(tokens, splits) == qg.QG_OK
        outs = [qg.fp4_gemm(*packed(torch, a, "nv", ta), *packed(torch, b, "nv", tb), K, "nv", a_scale=one(torch, ta),
                            b_scale=one(torch, tb), dtype=torch.float32),
                qg.fp4_linear(on_gpu(torch, a), *packed(torch, b, "nv", tb), "nv", x_scale=one(torch, ta),
                              w_scale=one(torch, tb))]
    finally:
        qg.lib().qg_set_fp4_path(0, 0)
    for y in outs:
        err = np.abs(as_np(y) - want)
        assert np.all(err <= bound), (float(np.nanmax(err / bound)), np.argwhere(~(err <= bound))[:4])


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_one_rounding_behind_the_sum(torch, qg, fmt):
    """With sums that are exact in fp32 every cut gives the same bits: alpha sum + bias is rounded once."""
    M, N, K = 16, 320, 256
    rng = np.random.default_rng(90)
    a, b = (rng.choice(np.concatenate((ref.GRID, -ref.GRID)), size=(n, K)).astype(np.float32) for n in (M, N))
    a[:, ::16], b[:, ::16] = 6, 6  # every block's scale is a power of two
    scales = dict(a_scale=one(torch, 0.337), b_scale=one(torch, 1.0)) if fmt == "nv" else {}
    pa, pb = packed(torch, a, fmt), packed(torch, b, fmt)
    bias = on_gpu(torch, activations(1, N, 91)[0])
    outs = []
    try:
        for tokens, splits in CUTS:
            assert qg.lib().qg_set_fp4_path(tokens, splits) == qg.QG_OK
            outs.append(qg.fp4_gemm(*pa, *pb, K, fmt, bias=bias, dtype=torch.float32, **scales))
    finally:
        qg.lib().qg_set_fp4_path(0, 0)
    alpha = np.float32(0.337) if fmt == "nv" else np.float32(1)
    exact = (ref.quantized(a, fmt) @ ref.quantized(b, fmt).T).astype(np.longdouble) * np.longdouble(alpha)
    want = (exact + as_np(bias).astype(np.longdouble)).astype(np.float32)
    for y, cut in zip(outs, CUTS):
        assert np.array_equal(y.cpu().numpy(), want), cut
