"""The scales of 8-bit operands where they are least ordinary."""
import pytest

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


def test_scales_of_rows_without_values(torch, qg):
    """K = 0: there is no code, and the scale is the smallest, as of a row of zeros."""
    for dtype in (torch.float16, torch.float32):
        out = torch.empty((3, 0), dtype=torch.int8, device="cuda"), torch.full((3,), 7.0, device="cuda")
        X = torch.zeros((3, 0), dtype=dtype, device="cuda")
        assert qg.s8_quantize(X, out=out)[1].tolist() == [2.0 ** -100] * 3
        assert qg.s8_quantize(X)[1].tolist() == [2.0 ** -100] * 3
