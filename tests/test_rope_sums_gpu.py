"""Head norm with rotation: heads that are not there."""
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


@pytest.mark.parametrize("D", [64, 63])
def test_gains_without_heads_have_gradients_of_zero(torch, qg, D):
    T, table = 5, torch.rand(5, 32, device="cuda")
    X, none = torch.randn(T, 2, D, device="cuda").half(), torch.zeros(T, 0, D, device="cuda").half()
    for q, k in ((X, none), (none, X), (none, none)):
        _, _, rq, rk = qg.qk_norm_rope(q, k, None, None, None, table)
        out = (torch.empty_like(q), torch.empty_like(k)) + tuple(torch.full((D,), 7.0, device="cuda") for _ in range(2))
        _, _, dgq, dgk = qg.qk_norm_rope_backward(q, k, q, k, None, None, None, table, rq, rk, out=out)
        for heads, dg in ((q, dgq), (k, dgk)):
            assert bool(dg.any()) == (heads is X)
