"""Every form of the scaled 8-bit products that the estimates choose, against 64 bits; bounds as in test_s8_gpu.py."""
import numpy as np
import pytest

from tests import _attention_ref as ref
from tests.test_fp4_gpu import as_np, on_gpu
from tests.test_s8_gpu import check_product, values

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


@pytest.fixture(autouse=True)
def _no_device_timeouts(qg):
    yield
    assert qg.device_status() == qg.QG_OK


# tokens a tile and CTAs that share K as the estimates choose them; several accumulators a CTA where K is long
FORMS = [
    (9, 4933, 1159),     # 32, 1
    (10, 4823, 1457),    # 32, 2
    (90, 1003, 8200),    # 32, 4
    (40, 300, 9000),     # 32, 8
    (250, 4099, 4100),   # 64, 1
    (777, 1001, 2304),   # 64, 1
    (35, 4749, 2723),    # 64, 2
    (64, 4096, 4096),    # 64, 4
    (595, 129, 1889),    # 64, 4
    (33, 871, 3701),     # 64, 8
    (300, 140, 20000),   # 64, 8
    (70, 9481, 1197),    # 128, 1
    (512, 4096, 4096),   # 128, 1
    (2692, 129, 4337),   # 128, 2
    (100, 4096, 4096),   # 128, 4
    (300, 1024, 8192),   # 128, 4
    (606, 135, 7071),    # 128, 8
    # a lone token: values that are read again, more than one round of weights, codes from a kernel ahead
    (1, 70, 4104), (1, 70, 8200), (1, 133, 14336), (1, 40, 102336), (1, 40, 102400), (1, 40, 131071), (8, 40, 131071),
]


def check_large_product(torch, Y, qa, sa, qb, sb, bias, dtype):
    """check_product; sums of 65520 and more round to fp16's infinity (those within 2^-20 of it, to either)."""
    if dtype == "float16":
        y = (qa.astype(np.float64) @ qb.astype(np.float64).T) * sa[:, None].astype(np.float64) * sb[None, :].astype(np.float64)
        y = torch.from_numpy(y + as_np(bias)).cuda()
        over = y.abs() >= 65520 * (1 - 2.0 ** -20)
        assert bool((torch.isinf(Y) | ~(y.abs() >= 65520 * (1 + 2.0 ** -20))).all())
        assert bool((torch.sign(Y.double()) == torch.sign(y))[over].all())
        Y = torch.where(over, y, Y.double())
    check_product(Y, qa, sa, qb, sb, bias, dtype)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("M,N,K", FORMS)
def test_forms_of_the_products(torch, qg, M, N, K, dtype):
    X, W = on_gpu(torch, values(M, K, 1), dtype), on_gpu(torch, values(N, K, 2), "float32")
    bias = on_gpu(torch, np.random.default_rng(3).standard_normal(N).astype(np.float32), dtype)
    (qa, sa), (qb, sb) = ref.s8_quantize(as_np(X)), ref.s8_quantize(as_np(W))
    Wq, Ws = qg.s8_quantize(W)
    Y = qg.s8_linear(X, Wq, Ws, bias=bias)
    check_large_product(torch, Y, qa, sa, qb, sb, bias, dtype)
    Xq, Xs = qg.s8_quantize(X)
    assert torch.equal(qg.s8_gemm(Xq, Xs, Wq, Ws, K, bias=bias, dtype=X.dtype), Y)
    assert torch.equal(qg.s8_linear(X, Wq, Ws, bias=bias), Y)
