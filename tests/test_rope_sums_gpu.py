"""Head norm with rotation: long sums of the gains' gradients, against 64 bits, and heads that are not there."""
import numpy as np
import pytest

from tests import _attention_ref as ref
from tests.test_fp4_gpu import as_np, on_gpu
from tests.test_rope_gpu import EPS, U, case, check_backward, check_forward

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


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("D,R", [(128, 128), (80, 32), (66, 66)])
def test_gradients_of_gains_over_many_tokens(torch, qg, D, R, dtype, style):
    """Warps that take several tokens, and more heads of each than they have lanes for at a time.

    6000 tokens of 8 + 2 heads by 4 CTAs of 4 warps on each of 148 SMs and more, 4/5 of them Q's.  Heads of 128 and 80: a
    warp of Q adds up 4 tokens of 8 heads or 7 halves of a token (fp32) in at most 14 steps, one of K 13 tokens in 13; the
    CTA then at most 16 sums of warps and lanes, the last kernel 16 of a slice of CTAs and 32 slices.  Heads of 66: 26
    heads a warp, 4 warps, 16 and 32.  No chain of additions is longer than 80, and a term has 4 roundings.
    """
    T, Hq, Hk = 6000, 8, 2
    Q, K, gq, gk, pos, table = case(torch, T, Hq, Hk, D, R, dtype)
    yq, yk, rq, rk = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS, style=style)
    check_forward(yq, rq, Q, gq, pos, table, style, dtype)
    check_forward(yk, rk, K, gk, pos, table, style, dtype)
    rng = np.random.default_rng(7)
    dq, dk = (on_gpu(torch, rng.standard_normal((T, h * D)).astype(np.float32), dtype).view(T, h, D) for h in (Hq, Hk))
    dxq, dxk, dgq, dgk = qg.qk_norm_rope_backward(dq, dk, Q, K, gq, gk, pos, table, rq, rk, style=style)
    check_backward(dxq, dgq, dq, Q, gq, pos, table, rq, style, dtype)
    check_backward(dxk, dgk, dk, K, gk, pos, table, rk, style, dtype)
    rows = as_np(table)[as_np(pos).astype(int)]
    c, s = rows[:, :R // 2], rows[:, R // 2:]
    for dg, dy, x, r in ((dgq, dq, Q, rq), (dgk, dk, K, rk)):
        dz, size = ref.turn(as_np(dy), c, -s, R, style), ref.turn_size(as_np(dy), c, s, R, style)
        xh = as_np(x) * as_np(r)[..., None]
        bound = (80 + 8) * U * (size * np.abs(xh)).sum(axis=(0, 1))
        assert np.all(np.abs(as_np(dg) - (dz * xh).sum(axis=(0, 1))) <= bound)


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
