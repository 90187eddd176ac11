"""The scales of 8-bit operands where they are least ordinary.

A product's sum is rounded to fp32, multiplied by either scale and rounded to its type: three roundings of 2^-24."""
import numpy as np
import pytest

from tests.test_fp4_gpu import as_np

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("M", [1, 6, 60, 1500])
def test_scales_of_either_sign(torch, qg, M):
    """Scales that a caller brings may be negative: the one of the smaller magnitude comes first then, too."""
    N, K = (2100, 512) if M == 1500 else (40, 512)
    rng = np.random.default_rng(M)
    qa, qb = (rng.integers(-127, 128, (r, K)).astype(np.int8) for r in (M, N))
    sa = (-2.0 ** 118 * rng.uniform(1, 2, M)).astype(np.float32)
    sb = (rng.choice([-1, 1], N) * 2.0 ** -90 * rng.uniform(1, 2, N)).astype(np.float32)
    for a, b in ((sa, sb), (np.abs(sa), -np.abs(sb)), (sb[0] * np.ones(M, np.float32), np.resize(sa, N))):
        Y = qg.s8_gemm(*(torch.from_numpy(t).cuda() for t in (qa, a, qb, b)), K, dtype=torch.float32)
        total = qa.astype(np.float64) @ qb.astype(np.float64).T
        want = total * a[:, None].astype(np.float64) * b[None, :].astype(np.float64)
        assert np.all(np.abs(as_np(Y) - want) <= 4.04 * 2.0 ** -24 * np.abs(want))


def test_scales_of_rows_without_values(torch, qg):
    """K = 0: there is no code, and the scale is the smallest, as of a row of zeros."""
    for dtype in (torch.float16, torch.float32):
        out = torch.empty((3, 0), dtype=torch.int8, device="cuda"), torch.full((3,), 7.0, device="cuda")
        X = torch.zeros((3, 0), dtype=dtype, device="cuda")
        assert qg.s8_quantize(X, out=out)[1].tolist() == [2.0 ** -100] * 3
        assert qg.s8_quantize(X)[1].tolist() == [2.0 ** -100] * 3
