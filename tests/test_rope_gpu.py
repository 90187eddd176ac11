"""RMS norm of heads with rotation, forward and backward, against 64 bits.

Bounds.  The sum of squares of a head is an fp32 chain of at most 64 fused additions and a
tree of 5, all of one sign: 72 2^-24 of itself, so 1 / rms is off by at most 40 2^-24 with
the square root and the division.  A value goes through at most 4 more roundings on its way
to y, relative to the magnitudes that the rotation adds up, and half a unit of its type.
"""
import numpy as np
import pytest

from tests import _attention_ref as ref
from tests.test_fp4_gpu import HALF_UNIT, as_np, on_gpu
from tests.test_s8_gpu import TINY

pytestmark = pytest.mark.gpu
EPS = 1e-6
U = 2.0 ** -24


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


def angles(T, R, seed, rows=97):
    rng = np.random.default_rng(seed)
    a = rng.uniform(-4, 4, (rows, R // 2))
    table = np.concatenate((np.cos(a), np.sin(a)), axis=1).astype(np.float32)
    return table, rng.integers(0, rows, T).astype(np.int32)


def case(torch, T, Hq, Hk, D, R, dtype, seed=1):
    rng = np.random.default_rng(seed)
    X = on_gpu(torch, (rng.standard_normal((T, (Hq + 2 * Hk) * D)) * np.exp(rng.standard_normal((T, 1)))).astype(np.float32), dtype)
    Q, K = X[:, :Hq * D].unflatten(1, (Hq, D)), X[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    g = [on_gpu(torch, (1 + 0.2 * rng.standard_normal(D)).astype(np.float32), dtype) for _ in range(2)]
    table, pos = angles(T, R, seed)
    return Q, K, g[0], g[1], torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda()


def check_forward(y, r, X, gain, pos, table, style, dtype):
    x = as_np(X)
    g = 1.0 if gain is None else as_np(gain)
    inv = ref.rms(x, EPS)
    assert np.all(np.abs(as_np(r) - inv) <= 40 * U * inv)
    rows = as_np(table)[as_np(pos).astype(int)]
    R = rows.shape[1]
    z = x * inv[..., None] * g
    want = ref.turn(z, rows[:, :R // 2], rows[:, R // 2:], R, style)
    size = ref.turn_size(z, rows[:, :R // 2], rows[:, R // 2:], R, style)
    bound = 48 * U * size + 1.01 * HALF_UNIT[dtype] * np.abs(want) + TINY[dtype]
    err = np.abs(as_np(y) - want)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])


def check_backward(dx, dgain, dY, X, gain, pos, table, inv, style, dtype):
    x, dy, r = as_np(X), as_np(dY), as_np(inv)[..., None]
    g = np.ones(x.shape[2]) if gain is None else as_np(gain)
    rows = as_np(table)[as_np(pos).astype(int)]
    R = rows.shape[1]
    c, s = rows[:, :R // 2], rows[:, R // 2:]
    dz, size = ref.turn(dy, c, -s, R, style), ref.turn_size(dy, c, s, R, style)
    xh = x * r
    dot = (dz * g * xh).mean(axis=2, keepdims=True)
    want = r * (dz * g - xh * dot)
    # the sum over a head is a chain of at most 64 and a tree of 5, of terms with 4 roundings each
    e_dot = 80 * U * (size * np.abs(g * xh)).mean(axis=2, keepdims=True)
    bound = r * (8 * U * size * np.abs(g) + np.abs(xh) * (e_dot + 4 * U * np.abs(dot)))
    bound = bound + 1.01 * HALF_UNIT[dtype] * np.abs(want) + TINY[dtype]
    err = np.abs(as_np(dx) - want)
    assert np.all(err <= bound), (float((err / bound).max()), np.argwhere(err > bound)[:4])
    terms = x.shape[0] * x.shape[1] + 64  # no chain of additions is longer
    err = np.abs(as_np(dgain) - (dz * xh).sum(axis=(0, 1)))
    assert np.all(err <= (terms + 4) * U * (size * np.abs(xh)).sum(axis=(0, 1)) + 2.0 ** -149)


# pieces of 16 bytes: every number of lanes; others: heads that have none
SHAPES = [(1, 1, 1, 64, 64), (5, 12, 4, 64, 64), (3, 4, 2, 128, 128), (7, 5, 1, 256, 256), (4, 3, 3, 80, 80), (9, 2, 2, 96, 96),
          (6, 4, 4, 80, 32), (5, 4, 2, 128, 64), (2, 3, 1, 16, 16), (3, 2, 2, 512, 512), (200, 8, 2, 128, 128),
          (4, 3, 2, 66, 66), (3, 2, 1, 7, 6), (5, 2, 2, 1, 0), (4, 2, 1, 100, 50), (3, 2, 2, 1024, 1000), (3, 3, 1, 128, 0),
          (2, 1, 1, 90, 2), (333, 20, 4, 64, 64)]


@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
def test_forward_and_backward(torch, qg, T, Hq, Hk, D, R, dtype, style):
    Q, K, gq, gk, pos, table = case(torch, T, Hq, Hk, D, R, dtype)
    yq, yk, rq, rk = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS, style=style)
    check_forward(yq, rq, Q, gq, pos, table, style, dtype)
    check_forward(yk, rk, K, gk, pos, table, style, dtype)
    rng = np.random.default_rng(7)
    dq = on_gpu(torch, rng.standard_normal((T, Hq * D)).astype(np.float32), dtype).view(T, Hq, D)
    dk = on_gpu(torch, rng.standard_normal((T, Hk * D)).astype(np.float32), dtype).view(T, Hk, D)
    dxq, dxk, dgq, dgk = qg.qk_norm_rope_backward(dq, dk, Q, K, gq, gk, pos, table, rq, rk, style=style)
    check_backward(dxq, dgq, dq, Q, gq, pos, table, rq, style, dtype)
    check_backward(dxk, dgk, dk, K, gk, pos, table, rk, style, dtype)
    again = qg.qk_norm_rope_backward(dq, dk, Q, K, gq, gk, pos, table, rq, rk, style=style)
    assert all(torch.equal(a, b) for a, b in zip((dxq, dxk, dgq, dgk), again))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gains_positions_and_places(torch, qg, dtype):
    """No gains, fp32 gains, no positions, no K, rows at odd places, outputs in place and in a packed matrix."""
    T, Hq, Hk, D = 9, 4, 2, 64
    Q, K, gq, gk, pos, table = case(torch, T, Hq, Hk, D, D, dtype)
    count = torch.arange(T, dtype=torch.int32, device="cuda")
    yq, yk, rq, rk = qg.qk_norm_rope(Q, K, None, None, None, table, EPS)
    check_forward(yq, rq, Q, None, count, table, "half", dtype)
    check_forward(yk, rk, K, None, count, table, "half", dtype)
    yq, _, rq, _ = qg.qk_norm_rope(Q, K, gq.float(), None, pos, table, EPS)
    check_forward(yq, rq, Q, gq, pos, table, "half", dtype)
    y, none, r, none2 = qg.qk_norm_rope(Q, None, gq, None, pos, table, EPS)
    assert none is None and none2 is None and torch.equal(y, yq) and torch.equal(r, rq)
    plain, _, _, _ = qg.qk_norm_rope(Q, K, gq, gk, None, None, EPS)
    check_forward(plain, rq, Q, gq, pos, table[:, :0], "half", dtype)
    # an odd place: other kernels
    want = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS)
    odd = torch.full((T, (Hq + Hk) * D + 13), 7.0, dtype=Q.dtype, device="cuda")
    oq, ok = odd[:, 3:3 + Hq * D].unflatten(1, (Hq, D)), odd[:, 5 + Hq * D:5 + (Hq + Hk) * D].unflatten(1, (Hk, D))
    oq.copy_(Q), ok.copy_(K)
    got = qg.qk_norm_rope(oq, ok, gq, gk, pos, table, EPS, out=(oq, ok))  # in place
    check_forward(oq, got[2], Q, gq, pos, table, "half", dtype)
    check_forward(ok, got[3], K, gk, pos, table, "half", dtype)
    assert bool((odd[:, :3] == 7).all()) and bool((odd[:, 3 + Hq * D:5 + Hq * D] == 7).all())
    assert bool((odd[:, 5 + (Hq + Hk) * D:] == 7).all())
    X = torch.cat((Q.flatten(1), K.flatten(1)), 1)
    xq, xk = X[:, :Hq * D].unflatten(1, (Hq, D)), X[:, Hq * D:].unflatten(1, (Hk, D))
    qg.qk_norm_rope(xq, xk, gq, gk, pos, table, EPS, out=(xq, xk))
    assert torch.equal(xq, want[0]) and torch.equal(xk, want[1])
    # gradients into a packed matrix, and over dY itself
    dq, dk = torch.randn_like(want[0]), torch.randn_like(want[1])
    grads = qg.qk_norm_rope_backward(dq, dk, Q, K, gq, gk, pos, table, want[2], want[3])
    P = torch.empty_like(X)
    pq, pk = P[:, :Hq * D].unflatten(1, (Hq, D)), P[:, Hq * D:].unflatten(1, (Hk, D))
    got = qg.qk_norm_rope_backward(dq, dk, Q, K, gq, gk, pos, table, want[2], want[3],
                                   out=(pq, pk, torch.empty(D, device="cuda"), torch.empty(D, device="cuda")))
    assert all(torch.equal(a, b) for a, b in zip(got, grads))
    qg.qk_norm_rope_backward(dq, dk, Q, K, gq, gk, pos, table, want[2], want[3], out=(dq, dk, got[2], got[3]))
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])


def test_gradients_against_differences(torch, qg):
    """The formula's gradient is the function's: fp32 calls differenced along random directions.

    f is a sum of n = 3 x 4 x 32 products of size about 1, each off by about 50 2^-24, so a
    difference over 2 h with h = 2^-8 is off by at most n 50 2^-24 / h = 0.3 at worst and some
    hundredths in fact; the third derivative's share is h^2 of values of the gradient's size.
    """
    T, H, D = 3, 2, 32
    Q, K, gq, gk, pos, table = case(torch, T, H, H, D, D, "float32")
    Q, K = Q.contiguous(), K.contiguous()
    Q /= Q.pow(2).mean().sqrt()
    K /= K.pow(2).mean().sqrt()
    gen = torch.Generator(device="cuda").manual_seed(3)
    wq, wk = (torch.randn(T, H, D, generator=gen, device="cuda") for _ in range(2))

    def f(q, k, a, b):
        yq, yk, _, _ = qg.qk_norm_rope(q, k, a, b, pos, table, EPS, style="pairs")
        return float((yq.double() * wq).sum() + (yk.double() * wk).sum())
    _, _, rq, rk = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS, style="pairs")
    grads = qg.qk_norm_rope_backward(wq, wk, Q, K, gq, gk, pos, table, rq, rk, style="pairs")
    at, h = (Q, K, gq, gk), 2.0 ** -8
    for _ in range(4):
        d = [torch.randn(t.shape, generator=gen, device="cuda") for t in at]
        up, down = ([t + s * h * e for t, e in zip(at, d)] for s in (1, -1))
        slope = (f(*up) - f(*down)) / (2 * h)
        want = sum(float((g.double() * e).sum()) for g, e in zip(grads, d))
        assert abs(slope - want) <= 0.3


def test_positions_outside_the_table_and_not_finite(torch, qg):
    Q, K, gq, gk, pos, table = case(torch, 6, 2, 2, 64, 32, "float16")
    pos[1], pos[4] = -1, table.shape[0]
    Q[3, 1, 5] = float("nan")
    for d in (64, 63):  # heads of 16-byte pieces, and not
        q, k = Q[:, :, :d].contiguous(), K[:, :, :d].contiguous()
        y, yk, _, _ = qg.qk_norm_rope(q, k, gq[:d], gk[:d], pos, table, EPS)
        for t in range(6):
            lost = t in (1, 4)
            assert bool(torch.isnan(yk[t, :, :32]).all()) == lost and not bool(torch.isnan(yk[t, :, 32:]).any())
            assert bool(torch.isnan(y[t, 1]).all()) == (t == 3)


@pytest.mark.parametrize("D,Hq,Hk", [(16, 3, 1), (24, 1, 2)])
def test_many_tokens(torch, qg, D, Hq, Hk):
    """Far more items than CTAs: the first, some middle and the last tokens are those of a short call."""
    T = 700001
    gen = torch.Generator(device="cuda").manual_seed(D)
    Q, K = (torch.randn(T, h, D, generator=gen, device="cuda").half() for h in (Hq, Hk))
    table = torch.rand(T, 8, generator=gen, device="cuda")
    got = qg.qk_norm_rope(Q, K, None, None, None, table, EPS)
    grads = qg.qk_norm_rope_backward(Q, K, Q, K, None, None, None, table, got[2], got[3])
    for i in (0, T // 2, T - 50):
        pos = torch.arange(i, i + 50, dtype=torch.int32, device="cuda")
        q, k = Q[i:i + 50].contiguous(), K[i:i + 50].contiguous()
        want = qg.qk_norm_rope(q, k, None, None, pos, table, EPS)
        assert all(torch.equal(a[i:i + 50], b) for a, b in zip(got, want))
        dq, dk, _, _ = qg.qk_norm_rope_backward(q, k, q, k, None, None, pos, table, want[2], want[3])
        assert torch.equal(grads[0][i:i + 50], dq) and torch.equal(grads[1][i:i + 50], dk)


def test_empty_and_graph(torch, qg):
    Q, K, gq, gk, pos, table = case(torch, 6, 2, 2, 64, 64, "bfloat16")
    yq, yk, rq, rk = qg.qk_norm_rope(Q[:0], K[:0], gq, gk, pos[:0], table, EPS)
    assert yq.shape == (0, 2, 64)
    _, _, dgq, dgk = qg.qk_norm_rope_backward(yq, yk, Q[:0], K[:0], gq, gk, pos[:0], table, rq, rk)
    assert not bool(dgq.any()) and not bool(dgk.any())
    want = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS)
    grads = qg.qk_norm_rope_backward(want[0], want[1], Q, K, gq, gk, pos, table, want[2], want[3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = qg.qk_norm_rope(Q, K, gq, gk, pos, table, EPS)
        dgot = qg.qk_norm_rope_backward(got[0], got[1], Q, K, gq, gk, pos, table, got[2], got[3])
    for _ in range(2):
        for t in got + dgot:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want + grads, got + dgot))
