"""Microscaled 4-bit products at the ends of their range: tensor scales whose product
leaves fp32's normal range, tensor scales at its ends, and as many rows as the calls take."""
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


# ------------------------------------------------------------- tensor scales at the ends of fp32

def plain_nv(X, ts):
    """Codes and scale bytes by the formula, each step rounded to 32 bits; r = fl(1 / d), at most the largest fp32."""
    f = np.float32
    x = X.reshape(X.shape[0], -1, 16)
    with np.errstate(all="ignore"):
        q = (np.abs(x).max(axis=2) / (f(6) * f(ts))).astype(f)
        byte = ref._nearest_even(q.astype(np.float64), ref.E4M3)
        d = (ref.E4M3[byte].astype(f) * f(ts)).astype(f)
        r = np.where(byte > 0, np.minimum(f(1) / d, np.finfo(f).max), f(0)).astype(f)
        y = (x * r[:, :, None]).astype(f)
    code = ref._nearest_even(np.abs(y).astype(np.float64), ref.GRID) | np.where(np.signbit(y), 8, 0)
    return code.reshape(X.shape).astype(np.uint8), byte.astype(np.uint8)


@pytest.mark.parametrize("ts", [2.0 ** -149, 1.3 * 2.0 ** -140, 1.3 * 2.0 ** -131, 1.7 * 2.0 ** -127, 1.9 * 2.0 ** -119, 1.7 * 2.0 ** 110,
                                1.3 * 2.0 ** 124, 1.9 * 2.0 ** 125, 3e38])
def test_tensor_scales_at_the_ends_of_fp32(torch, qg, ts):
    ts = float(np.float32(ts))
    rng = np.random.default_rng(101)
    for K in (256, 250):  # 250: rows that are not 16-byte aligned
        X = np.zeros((40, 256), dtype=np.float32)
        size = np.minimum(np.exp(rng.uniform(-6, 9, (40, 1))) * ts, 1e38)
        X[:, :K] = np.clip(rng.standard_normal((40, K)) * size, -3e38, 3e38).astype(np.float32)
        X[:, :K][rng.random((40, K)) < 0.2] = 0
        code, byte = plain_nv(X, ts)
        q_ref, s_ref = ref.pack(code, byte)
        x = on_gpu(torch, X[:, :K])
        for got in (qg.fp4_quantize(x, "nv", scale=one(torch, ts)), qg.fp4_quantize_both(x, "nv", scale=one(torch, ts))[:2]):
            assert np.array_equal(as_np(got[1]), s_ref)
            assert np.array_equal(as_np(got[0]), q_ref)
        # what was 0 stands for 0
        v = as_np(qg.fp4_dequantize(*qg.fp4_quantize(x, "nv", scale=one(torch, ts)), K, "nv", scale=one(torch, ts)))
        assert not v[X[:, :K] == 0].any()


# ------------------------------------------------------------- as many rows as the calls take

ROWS = 65536 * 128 + 1  # one more tile of 128 rows than a grid's y or z counts


def test_products_of_very_many_rows(torch, qg):
    K, few = 32, 8
    a, w = activations(few, K, 95), activations(128, K, 96)
    pick = torch.arange(ROWS, device="cuda") * 7 % 128
    wq, ws = packed(torch, w, "mx")
    many_q = wq[pick]
    # scales of many rows: the bytes of w's rows in their new places (one block a row)
    byte = torch.from_numpy(ref.codes_and_bytes(w, "mx")[1][:, 0].copy()).cuda()[pick]
    tiles = -(-ROWS // 128)
    at = torch.arange(ROWS, device="cuda")
    many_s = torch.zeros((tiles, 1, 512), dtype=torch.uint8, device="cuda")
    many_s.view(-1)[at // 128 * 512 + at % 32 * 16 + at % 128 // 32 * 4] = byte
    aq, as_ = packed(torch, a, "mx")
    small = qg.fp4_gemm(aq, as_, wq, ws, K, "mx", dtype=torch.float32)
    y = qg.fp4_gemm(aq, as_, many_q, many_s, K, "mx", dtype=torch.float32)       # as weights
    assert torch.equal(y, small[:, pick])
    del y
    y = qg.fp4_gemm(many_q, many_s, aq, as_, K, "mx", dtype=torch.float32)       # as tokens
    assert torch.equal(y, small.t()[pick])


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_both_directions_of_very_many_rows(torch, qg, fmt):
    K = 16
    X = torch.randn((ROWS, K), device="cuda", generator=torch.Generator("cuda").manual_seed(97)).to(torch.bfloat16)
    q, s, tq, ts = qg.fp4_quantize_both(X, fmt)
    for got, want in zip((q, s, tq, ts), qg.fp4_quantize(X, fmt) + qg.fp4_quantize(X.t().contiguous(), fmt)):
        assert torch.equal(got, want)


def test_gradients_of_very_many_rows(torch, qg):
    """dX row by row, dW and db over all of them."""
    N, K = 16, 32
    g = torch.Generator("cuda").manual_seed(98)
    dY = (torch.randint(-3, 4, (ROWS, N), device="cuda", generator=g)).to(torch.bfloat16)
    X = (torch.randint(-1, 2, (ROWS, K), device="cuda", generator=g)).to(torch.bfloat16)
    wt = activations(K, N, 99)
    dx, dw, db = qg.fp4_linear_backward(dY, X, *packed(torch, wt, "mx"), "mx")
    q, s = qg.fp4_quantize(dY, "mx")
    v = qg.fp4_dequantize(q, s, N, "mx").double()
    want = v @ torch.from_numpy(ref.quantized(wt, "mx").T.copy()).cuda()
    size = v.abs() @ torch.from_numpy(np.abs(ref.quantized(wt, "mx")).T.copy()).cuda()
    assert bool(((dx.double() - want).abs() <= 9 * 2.0 ** -22 * size + 1.01 * 2.0 ** -8 * want.abs() + 2.0 ** -133).all())
    del v, want, size
    # whole numbers: 128 rows' sums are exact in fp32, and so are their sums up to 2^24
    assert torch.equal(db.double(), dY.double().sum(0))
    vt = qg.fp4_dequantize(*qg.fp4_quantize(dY.t().contiguous(), "mx"), ROWS, "mx").double()
    xt = qg.fp4_dequantize(*qg.fp4_quantize(X.t().contiguous(), "mx"), ROWS, "mx").double()
    size = (vt.abs() @ xt.abs().t())
    bound = (ROWS / 64 + 8) * 2.0 ** -22 * size + 1.01 * 2.0 ** -8 * (vt @ xt.t()).abs() + 2.0 ** -133
    assert bool(((dw.double() - vt @ xt.t()).abs() <= bound).all())
