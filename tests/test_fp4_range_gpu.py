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
