"""Attention over the 8-bit cache at the ends of its range: scores that are -inf throughout, weights far
below the largest.  Bounds as in test_kv8_gpu.py where none is derived here."""
import math

import pytest

from tests.test_fp4_gpu import HALF_UNIT
from tests.test_kv8_gpu import check_attention, filled, int32, starts_of
from tests.test_s8_gpu import TINY

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


# few rows, whole units and joined ones; many rows (128 and more), whole and joined; both in a batch; rows ahead of
# their sequence's first token
ONE_SIGN = [([1], [1]), ([1, 2], [1, 40]), ([1], [3000]), ([3], [2]), ([40], [40]), ([70], [300]), ([40], [2500]),
            ([60], [50]), ([90], [1500]), ([1, 300, 2], [1500, 300, 2]), ([1, 300, 2], [1, 280, 1]), ([200], [3])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news,lengths", ONE_SIGN)
def test_scores_that_are_all_minus_infinity(torch, qg, news, lengths, D, causal):
    """An infinity in a query against a channel of keys that makes every score -inf: the softmax is 0 / 0, not 0."""
    heads, group, page = 2, 4, 16
    for sign, scale in ((1, D ** -0.5), (-1, D ** -0.5), (1, -0.1)):
        cache, table = filled(torch, lengths, heads, D, page, 19)
        cache[0][..., 5] = sign * (cache[0][..., 5].int().abs().clamp(1, 127)).to(torch.int8)
        gen = torch.Generator(device="cuda").manual_seed(sum(news))
        good = torch.randn(sum(news), heads * group, D, generator=gen, device="cuda").half()
        bad, infinite = good.clone(), -math.inf if sign * scale > 0 else math.inf
        places, row = [], 0
        for n in news:
            places += [(row, 1, 0), (row + n // 2, 6, 0), (row + n - 1, 3, 0)]
            row += n
        for r, h, _ in places:
            bad[r, h, 5] = infinite
            good[r, h] = 0
        args = (cache, table, int32(torch, starts_of(news)), int32(torch, lengths), scale, causal)
        O, want = qg.kv8_attention(bad, *args), qg.kv8_attention(good, *args)
        row = 0
        for n, m in zip(news, lengths):
            for i in {0, n // 2, n - 1}:
                sees = m - n + i >= 0 if causal else m > 0
                for h in (j for r, j, _ in places if r == row + i):
                    got = O[row + i, h]
                    assert bool(torch.isnan(got).all()) if sees else not bool(got.any()), (n, m, i, h)
                    O[row + i, h] = want[row + i, h]
            row += n
        check_attention(torch, O, good, cache, table, news, lengths, scale, causal, "float16")


@pytest.mark.parametrize("page,D", [(16, 64), (64, 128), (32, 256)])
@pytest.mark.parametrize("B,new,length", [(1, 1, 131072), (1, 40, 131072), (700, 1, 8192), (40, 40, 8192)])
@pytest.mark.parametrize("below", [17.0, 18.0, 22.0])
def test_many_small_weights_next_to_large_ones(torch, qg, below, B, new, length, page, D):
    """Four tokens that hold nearly all of the weight but whose values are 0, as a sink's are, before thousands whose
    weights are e^-below of theirs each: the result is what the thousands make.  (B sequences on the same pages.)

    A weight is rounded to fp16 in units in which the largest is at least 2^9: by half of 2^-10 of itself, or by half
    of 2^-24 below the normal range, which is 2^-34 of the largest.  The rest of the bound is that of check_attention.
    """
    heads, group = 1, 4
    cache, table = filled(torch, [length], heads, D, page, 23, spread=0.0)
    kq, vq, ks, vs = cache
    kq[..., 0] = 0
    vq.copy_(vq.int().abs().clamp(60, 127).to(torch.int8))
    for at in (3, 35, 67, 99):
        sink = int(table[0, at // page]), 0, at % page
        kq[sink] = 0
        vq[sink] = 0
        kq[sink][0] = 100
    gen = torch.Generator(device="cuda").manual_seed(new)
    # scores of the others are normal with 0.1 (codes have a mean square of about 73^2), the sinks' are `below`
    Q = (0.1 / (73 * 0.01 * D ** 0.5) * torch.randn(B * new, heads * group, D, generator=gen, device="cuda")).half()
    Q[..., 0] = below / (100 * 0.01)
    starts, lengths = int32(torch, starts_of([new] * B)), int32(torch, [length] * B)
    O = qg.kv8_attention(Q, cache, table.expand(B, -1).contiguous(), starts, lengths, 1.0).double()
    k8, v8 = (c[table[0].long(), 0].double().reshape(-1, D)[:length] for c in (kq, vq))
    sk, sv = (s[table[0].long(), 0].double().repeat_interleave(page)[:length, None] for s in (ks, vs))
    last = torch.arange(length - new, length, device="cuda").repeat(B)
    hide = torch.arange(length, device="cuda")[None, :] > last[:, None]
    for h in range(group):
        q = Q[:, h].double()
        x = (q @ (k8 * sk).t()).masked_fill(hide, -math.inf)
        w = torch.softmax(x, 1)
        want = w @ (v8 * sv)
        e = D * 2.0 ** -23 * (q.abs() @ (k8.abs() * sk).t()).amax(1) + 10 * 2.0 ** -24 * (x.amax(1) + 8) + 2.0 ** -21
        joined = (length / 16 + 64) * 2.0 ** -23
        bulk, low = w @ (v8.abs() * sv), 2.0 ** -34 * w.amax(1, keepdim=True) * (v8.abs() * sv).sum(0)
        bound = bulk * (1.01 * 2.0 ** -11 + 2 * e[:, None] + joined) + low
        bound = bound + 1.01 * HALF_UNIT["float16"] * want.abs() + TINY["float16"]
        err = (O[:, h] - want).abs()
        assert bool((err <= bound).all()), (h, float((err / bound).max()), float((err / want).max()))


def kernels_of(torch, call):
    """Names of the kernels that a call launches."""
    from torch.profiler import ProfilerActivity, profile
    for _ in range(3):  # the first record of a process may be empty
        with profile(activities=[ProfilerActivity.CUDA]) as prof:
            call()
            torch.cuda.synchronize()
        names = [e.key for e in prof.key_averages()]
        if any("k_kv8_attention" in n for n in names):
            return names
    pytest.skip("no kernels were recorded")


@pytest.mark.parametrize("heads,page,D,news,lengths,cols", [
    (2, 16, 64, [300, 1, 2], [700, 800, 2], 33000), (1, 64, 128, [1, 900, 0, 2], [300, 900, 5, 3000], 12000),
    (8, 32, 64, [1200, 1, 1, 70, 3], [1300, 500, 1, 90, 2000], 4096)])
def test_large_prompts_next_to_single_tokens_of_long_sequences(torch, qg, heads, page, D, news, lengths, cols):
    """On average many rows a sequence, and room in the table for so many tokens that single tokens count: both kernels."""
    cache, short = filled(torch, lengths, heads, D, page, 29)
    table = torch.full((len(news), cols), -1, dtype=torch.int32, device="cuda")
    table[:, :short.shape[1]] = short
    gen = torch.Generator(device="cuda").manual_seed(heads)
    Q = torch.randn(sum(news), heads * 4, D, generator=gen, device="cuda").bfloat16()
    starts, length = int32(torch, starts_of(news)), int32(torch, lengths)
    O = qg.kv8_attention(Q, cache, table, starts, length)
    check_attention(torch, O, Q, cache, table, news, lengths, D ** -0.5, True, "bfloat16")
    names = kernels_of(torch, lambda: qg.kv8_attention(Q, cache, table, starts, length))
    assert any("k_kv8_attention_rows<" in n for n in names) and any("k_kv8_attention<" in n for n in names)
    # with little room the kernel for many rows takes them all
    names = kernels_of(torch, lambda: qg.kv8_attention(Q, cache, short, starts, length))
    assert any("k_kv8_attention_rows<" in n for n in names) and not any("k_kv8_attention<" in n for n in names)
