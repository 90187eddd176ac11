"""Attention over the 8-bit cache at the ends of its range: scores that are -inf throughout."""
import math

import pytest

from tests.test_kv8_gpu import check_attention, filled, int32, starts_of

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
