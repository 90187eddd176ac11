"""CPU checks of the C ABI of the scaled 8-bit products, the head norm with rotation and the
paged 8-bit cache: sizes, refusals before any GPU work, and the kernels' resource table."""
import pytest

import bit_quantized_tensor_gb300 as qg

P = 0x10000  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 40
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build_library()
    return qg.lib()


def test_sizes(L):
    assert [L.qg_s8_codes_ld(k) for k in (-3, 0, 1, 16, 17, 4096)] == [0, 0, 16, 16, 32, 4096]
    ws = L.qg_workspace_size
    assert ws(qg.QG_OP_S8_LINEAR, 1, 4096, 4096) == 0  # quantized inside the product
    assert ws(qg.QG_OP_S8_LINEAR, 100, 50, 33) >= 100 * 48 * 2 + 100 * 4      # the tokens as fp16
    assert ws(qg.QG_OP_S8_LINEAR, 5000, 50, 33) >= 5050 * 48 * 2 + 5000 * 4   # and the weights
    assert ws(qg.QG_OP_QK_NORM_ROPE_BACKWARD, 1, 1, 128) > 0
    assert ws(qg.QG_OP_KV8_ATTENTION, 4, 8, 128) > 0


def _quant(L, dt=1, M=4, K=64, X=P, ld=64, q=P, s=P):
    return L.s8_quantize(dt, M, K, X, ld, q, s, None)


def _linear(L, dt=1, M=40, N=8, K=64, X=P, ldx=64, w=P, sw=P, bias=None, Y=P, ldy=8, ws=P, wsb=BIG):
    return L.s8_linear(dt, M, N, K, X, ldx, w, sw, bias, Y, ldy, ws, wsb, None)


def _gemm(L, dt=1, M=40, N=8, K=64, a=P, sa=P, b=P, sb=P, bias=None, Y=P, ldy=8, ws=P, wsb=BIG):
    return L.s8_gemm(dt, M, N, K, a, sa, b, sb, bias, Y, ldy, ws, wsb, None)


def test_product_refusals(L):
    assert _quant(L, dt=3) == UNSUPPORTED and _quant(L, M=-1) == INVALID and _quant(L, K=131072) == INVALID
    assert _quant(L, ld=63) == INVALID and _quant(L, X=None) == INVALID and _quant(L, q=None) == INVALID
    assert _quant(L, X=P + 1) == MISALIGNED and _quant(L, q=P + 8) == MISALIGNED and _quant(L, s=P + 2) == MISALIGNED
    assert _quant(L, M=0) == OK and _quant(L, K=0) == OK
    for f in (_linear, _gemm):
        assert f(L, dt=7) == UNSUPPORTED and f(L, M=-1) == INVALID and f(L, N=(1 << 27) + 1) == INVALID
        assert f(L, K=131072) == INVALID and f(L, ldy=7) == INVALID and f(L, Y=None) == INVALID
        assert f(L, Y=P + 1) == MISALIGNED and f(L, bias=P + 1) == MISALIGNED and f(L, ws=P + 16) == MISALIGNED
        assert f(L, ws=None) == WORKSPACE and f(L, wsb=64) == WORKSPACE
        assert f(L, M=0) == OK and f(L, N=0) == OK
    assert _linear(L, X=None) == INVALID and _linear(L, w=None) == INVALID and _linear(L, sw=None) == INVALID
    assert _linear(L, ldx=63) == INVALID and _linear(L, w=P + 4) == MISALIGNED and _linear(L, X=P + 1) == MISALIGNED
    assert _gemm(L, a=None) == INVALID and _gemm(L, sb=None) == INVALID and _gemm(L, sa=P + 1) == MISALIGNED
    assert _gemm(L, b=P + 8) == MISALIGNED


def _rope(L, dt=1, style=0, T=4, Hq=2, Hk=1, D=64, R=64, Q=P, ldq=128, K=P, ldk=64, g=P, wd=1, pos=P, table=P, rows=10,
          eps=1e-6, Yq=P, ldyq=128, Yk=P, ldyk=64, rq=P, rk=P):
    return L.qk_norm_rope(dt, style, T, Hq, Hk, D, R, Q, ldq, K, ldk, g, g, wd, pos, table, rows, eps, Yq, ldyq, Yk, ldyk,
                          rq, rk, None)


def _rope_backward(L, T=4, Hq=2, Hk=1, D=64, dYq=P, lddyq=128, dYk=P, Q=P, K=P, rq=P, rk=P, dQ=P, dK=P, dgq=P, dgk=P, ws=P,
                   wsb=BIG, R=64):
    return L.qk_norm_rope_backward(1, 0, T, Hq, Hk, D, R, dYq, lddyq, dYk, 64, Q, 128, K, 64, P, P, 1, P, P, 10, rq, rk, dQ,
                                   128, dK, 64, dgq, dgk, ws, wsb, None)


def test_rope_refusals(L):
    assert _rope(L, dt=3) == UNSUPPORTED and _rope(L, wd=0) == UNSUPPORTED and _rope(L, style=2) == UNSUPPORTED
    assert _rope(L, D=1026, ldq=BIG, ldk=BIG, ldyq=BIG, ldyk=BIG) == UNSUPPORTED
    for bad in ({"T": -1}, {"Hq": -1}, {"Hk": -1}, {"D": 0}, {"R": 65}, {"R": 63}, {"R": -2}, {"Q": None}, {"K": None},
                {"Yq": None}, {"Yk": None}, {"ldq": 127}, {"ldk": 63}, {"ldyq": 127}, {"ldyk": 63}, {"table": None},
                {"rows": 0}, {"eps": -1e-9}, {"eps": float("nan")}):
        assert _rope(L, **bad) == INVALID, bad
    for name in ("Q", "K", "Yq", "Yk"):
        assert _rope(L, **{name: P + 1}) == MISALIGNED, name
    for name in ("pos", "table", "rq", "rk"):
        assert _rope(L, **{name: P + 2}) == MISALIGNED, name
    assert _rope(L, g=P + 1) == MISALIGNED and _rope(L, T=0) == OK and _rope(L, Hq=0, Hk=0) == OK
    for bad in ({"dYq": None}, {"dYk": None}, {"Q": None}, {"K": None}, {"rq": None}, {"rk": None}, {"dQ": None}, {"dK": None},
                {"dgq": None}, {"dgk": None}, {"lddyq": 100}, {"R": 66}):
        assert _rope_backward(L, **bad) == INVALID, bad
    assert _rope_backward(L, ws=None) == WORKSPACE and _rope_backward(L, wsb=100) == WORKSPACE
    assert _rope_backward(L, ws=P + 8) == MISALIGNED and _rope_backward(L, dgq=P + 1) == MISALIGNED


def _cache(B=2, rows=4, heads=2, D=64, kq=P, vq=P, ks=P, vs=P, pages=8, page=16, table=P, cols=4, starts=P, lengths=P):
    return B, rows, heads, D, kq, vq, ks, vs, pages, page, table, cols, starts, lengths


def _append(L, dt=1, K=P, ldk=128, V=P, ldv=128, **kw):
    B, rows, heads, D, *rest = _cache(**kw)
    return L.kv8_append(dt, B, rows, heads, D, K, ldk, V, ldv, *rest, None)


def _gather(L, dt=1, K=P, ldk=128, V=P, ldv=128, **kw):
    B, rows, heads, D, *rest = _cache(**kw)
    return L.kv8_gather(dt, B, rows, heads, D, *rest, K, ldk, V, ldv, None)


def _attention(L, dt=1, q_heads=4, K=P, ldk=256, V=P, ldv=256, scale=0.1, ws=P, wsb=BIG, **kw):
    B, rows, heads, D, *rest = _cache(**kw)
    return L.kv8_attention(dt, B, rows, q_heads, heads, D, K, ldk, *rest, scale, 1, V, ldv, ws, wsb, None)


def test_cache_refusals(L):
    for f in (_append, _gather, _attention):
        assert f(L, dt=5) == UNSUPPORTED
        for bad in ({"page": 8}, {"page": 24}, {"page": 256}, {"D": 32}, {"D": 96}, {"D": 512}):
            assert f(L, **bad) == UNSUPPORTED, bad
        for bad in ({"B": -1}, {"rows": -1}, {"heads": 0}, {"pages": 0}, {"pages": -1}, {"cols": 0}, {"page": 0}, {"D": 0},
                    {"kq": None}, {"vq": None}, {"ks": None}, {"vs": None}, {"table": None}, {"starts": None},
                    {"lengths": None}, {"K": None}, {"V": None}, {"cols": 1 << 30}, {"pages": BIG}, {"rows": 1 << 30}):
            assert f(L, **bad) == INVALID, bad
        for name in ("kq", "vq"):
            assert f(L, **{name: P + 8}) == MISALIGNED, name
        for name in ("ks", "vs", "table", "starts", "lengths"):
            assert f(L, **{name: P + 2}) == MISALIGNED, name
        assert f(L, K=P + 1) == MISALIGNED and f(L, V=P + 1) == MISALIGNED
        assert f(L, ldk=100) == INVALID and f(L, ldv=100) == INVALID
        assert f(L, B=0) == OK and f(L, rows=0) == OK
    assert _attention(L, dt=qg.QG_F32) == UNSUPPORTED
    assert _attention(L, q_heads=3) == INVALID and _attention(L, q_heads=0) == INVALID
    for scale in (float("nan"), float("inf")):
        assert _attention(L, scale=scale) == INVALID
    assert _attention(L, ws=None) == WORKSPACE and _attention(L, wsb=64) == WORKSPACE and _attention(L, ws=P + 16) == MISALIGNED


def test_no_gpu_reports_cuda_error(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for f in (_quant, _linear, _gemm, _rope, _rope_backward, _append, _gather, _attention):
        assert f(L) == CUDA, f.__name__


def test_kernel_table(L):
    names = [r["kernel"] for r in qg.kernel_budgets(table="block")]
    for stem in ("k_s8_quantize<", "k_s8_gemv<", "tc_gemm_kernel<F16,S8>", "tc_gemm2_kernel<F16,S8>", "k_qk_norm_rope<",
                 "k_qk_norm_rope_backward<", "k_qk_norm_rope_any<", "k_rope_gains", "k_kv8_append<", "k_kv8_gather<",
                 "k_kv8_attention<", "k_kv8_attention_join<"):
        assert any(n.startswith(stem) for n in names), stem
