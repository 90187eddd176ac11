"""The paged cache in 8 bits and the attention over it, against 64 bits.

Bounds of the attention.  The exponent of token j, in base 2, is scale log2(e) sk (q . kq) + log2 sv
less the running maximum: the dot product is off by at most D 2^-23 of the sum of its magnitudes,
the rest is 6 roundings of the exponent and its parts (2^-24 each, log2 2^-22), and 2^e itself
is good to 2^-22; together a factor 1 + e_j of the weight.  Weights are rounded to fp16 for the
product with V (2^-11, or 2^-25 of the largest below the normal range), whose fp32 sums have
a rounding for every 16 tokens and every time that parts are joined.  The result is rounded
once (half a unit).
"""
import math

import numpy as np
import pytest

from tests import _attention_ref as ref
from tests.test_fp4_gpu import HALF_UNIT, as_np, on_gpu
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


def int32(torch, v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(news):
    return [0] + np.cumsum(news).tolist()


def filled(torch, lengths, heads, D, page, seed, extra=2, spread=1.0):
    """A cache with pages of many scales; what no sequence holds is codes of -128 under scales that are NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cols = max(1, max(-(-n // page) for n in lengths))
    pages = len(lengths) * cols + extra
    table = torch.randperm(pages, generator=gen, device="cuda")[:len(lengths) * cols].view(len(lengths), cols).int()
    kq, vq = (torch.randint(-127, 128, (pages, heads, page, D), generator=gen, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (0.01 * torch.exp(spread * torch.randn((pages, heads), generator=gen, device="cuda")) for _ in range(2))
    used = torch.zeros(pages, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lengths):
        full, rest = divmod(n, page)
        used[table[b, :full + (rest > 0)].long()] = True
        if rest:
            kq[table[b, full], :, rest:] = -128
            vq[table[b, full], :, rest:] = -128
    kq[~used], vq[~used], ks[~used], vs[~used] = -128, -128, float("nan"), float("nan")
    return (kq, vq, ks, vs), table.contiguous()


def check_attention(torch, O, Q, cache, table, news, lengths, scale, causal, dtype):
    """Sequence by sequence and head by head, in 64 bits on the device."""
    kq, vq, ks, vs = cache
    page, D = kq.shape[2:]
    heads, group = kq.shape[1], Q.shape[1] // kq.shape[1]
    row = 0
    for b, (n, m) in enumerate(zip(news, lengths)):
        if n == 0:
            continue
        q = Q[row:row + n].double()
        got = O[row:row + n].double()
        row += n
        used = table[b, :-(-m // page)].long()
        pos = torch.arange(n, device="cuda") + m - n
        sees = torch.arange(m, device="cuda")[None, :] <= (pos[:, None] if causal else torch.full_like(pos, m)[:, None])
        for h in range(heads):
            sk, sv = (s[used, h].double().repeat_interleave(page)[:m] for s in (ks, vs))
            k8, v8 = (c[used, h].double().reshape(-1, D)[:m] for c in (kq, vq))
            qh = q[:, h * group:(h + 1) * group]
            x = torch.einsum("ngd,md->ngm", qh, k8) * sk * scale
            size = torch.einsum("ngd,md->ngm", qh.abs(), k8.abs()) * sk * abs(scale)
            hide = ~sees[:, None, :]
            x = x.masked_fill(hide, -math.inf)
            any_seen = sees.any(1)
            w = torch.softmax(x, 2).masked_fill(hide, 0.0)
            w[~any_seen] = 0
            want = torch.einsum("ngm,md->ngd", w, v8 * sv[:, None])
            # exponents in base 2 are log2(e) x: as a factor of the weight, ln 2 times their error
            largest = (x.masked_fill(hide, 0.0).abs() + 0.7 * torch.log2(sv).abs()).amax(2) if m else torch.zeros(n, group, device="cuda").double()
            most = size.masked_fill(hide, 0.0).amax(2) if m else largest
            e = D * 2.0 ** -23 * most + 10 * 2.0 ** -24 * (largest + 1) + 2.0 ** -21
            joined = (m / 16 + 64) * 2.0 ** -23
            bulk = torch.einsum("ngm,md->ngd", w, v8.abs() * sv[:, None])
            low = 2.0 ** -25 * (sv.max() if m else 0.0) * torch.einsum("nm,md->nd", sees.double(), v8.abs())[:, None, :]
            bound = bulk * (1.01 * 2.0 ** -11 + 2 * e[..., None] + joined) + low
            bound = bound + 1.01 * HALF_UNIT[dtype] * want.abs() + TINY[dtype]
            err = (got[:, h * group:(h + 1) * group] - want).abs()
            assert bool((err <= bound).all()), (b, h, float((err / bound).max()))


# ------------------------------------------------------------- append, gather

def random_cache(torch, qg, pages, heads, page, D, seed):
    cache = qg.kv8_cache(pages, heads, page, D)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for c in cache[:2]:
        c.copy_(torch.randint(-127, 128, c.shape, generator=gen, device="cuda", dtype=torch.int8))
    for s in cache[2:]:
        s.copy_(0.02 * torch.exp(torch.randn(s.shape, generator=gen, device="cuda")))
    return cache


APPENDS = [(16, 64, 2, [1], [1]), (16, 64, 1, [20], [20]), (32, 128, 2, [1, 1, 1], [33, 64, 7]), (64, 256, 1, [70, 3], [130, 3]),
           (128, 64, 3, [5, 0, 300, 1], [5, 77, 301, 129]), (16, 128, 4, [17, 16, 15, 1, 0], [17, 48, 31, 16, 0]),
           (16, 64, 1, [5, 3], [3, 3]), (64, 128, 8, [1] * 9, [1, 2, 64, 65, 127, 128, 129, 300, 5])]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("page,D,heads,news,lengths", APPENDS)
def test_append_and_gather(torch, qg, page, D, heads, news, lengths, dtype):
    """Codes and scales are the definition's bit for bit, and nothing else changes; twice in a row."""
    B, cols = len(news), max(1, max(-(-n // page) for n in lengths)) + 1
    cache = random_cache(torch, qg, B * cols + 3, heads, page, D, 5)
    plain = ref.Cache(*(as_np(t).astype(np.int8 if t.dtype is torch.int8 else np.float32) for t in cache))
    order = np.random.default_rng(2).permutation(B * cols + 3)[:B * cols].reshape(B, cols).astype(np.int32)
    table, starts = torch.from_numpy(order).cuda(), starts_of(news)
    rng = np.random.default_rng(4)
    for step in range(2):
        rows = starts[-1] + 2  # two rows that are no sequence's
        kv = [(rng.standard_normal((rows, heads, D)) * np.exp(rng.standard_normal((rows, 1, 1)))).astype(np.float32) for _ in range(2)]
        K, V = (on_gpu(torch, x, dtype) for x in kv)
        if step:  # rows at an odd place
            wide = torch.empty((rows, heads * D + 9), dtype=K.dtype, device="cuda")
            wide[:, 3:3 + heads * D] = K.flatten(1)
            K = wide[:, 3:3 + heads * D].unflatten(1, (heads, D))
        args = (table, int32(torch, starts), int32(torch, lengths))
        qg.kv8_append(K, V, cache, *args)
        plain.append("k", as_np(K), order, starts, lengths)
        plain.append("v", as_np(V), order, starts, lengths)
        for got, want in zip(cache, (plain.q["k"], plain.q["v"], plain.s["k"], plain.s["v"])):
            assert np.array_equal(as_np(got).astype(want.dtype), want)
        out = torch.full((2, rows, heads, D), 7.0, dtype=K.dtype, device="cuda")
        gk, gv = qg.kv8_gather(cache, *args, rows, out=(out[0], out[1]))
        for which, got in (("k", gk), ("v", gv)):
            for b, n in enumerate(news):
                m, r = lengths[b], starts[b]
                v, _ = plain.tokens(which, order, b, m)
                missing = max(0, n - m)
                want = torch.from_numpy(v[max(0, m - n):].astype(np.float32)).to(K.dtype)
                assert torch.equal(got[r + missing:r + n].cpu(), want)
                assert bool(torch.isnan(got[r:r + missing]).all())
            assert bool((got[starts[-1]:] == 7).all())
    assert qg.kv8_gather(cache, *args, rows)[0].dtype == torch.bfloat16


def test_append_of_values_that_are_not_finite(torch, qg):
    cache = qg.kv8_cache(4, 2, 16, 64)
    table, x = int32(torch, [[2, 0], [1, 3]]), torch.randn(12, 2, 64, device="cuda")
    x[3, 1, 5], x[9, 0, 0] = float("inf"), float("nan")
    qg.kv8_append(x, x, cache, table, int32(torch, [0, 8, 12]), int32(torch, [8, 4]))
    for s in cache[2:]:
        assert as_np(torch.isnan(s)).tolist() == [[False, False], [True, False], [False, True], [False, False]]
    # the page keeps it; the next page and a fresh start do not
    y = torch.randn(20, 2, 64, device="cuda")
    qg.kv8_append(y, y, cache, table, int32(torch, [0, 10, 20]), int32(torch, [18, 10]))
    assert as_np(torch.isnan(cache[2])).tolist() == [[False, False], [False, False], [False, True], [False, False]]
    k, _ = qg.kv8_gather(cache, table, int32(torch, [0, 18, 18]), int32(torch, [18, 10]), 18, dtype=torch.float32)
    assert bool(torch.isnan(k[:16, 1]).all()) and not bool(torch.isnan(k[:, 0]).any()) and not bool(torch.isnan(k[16:]).any())


def test_scale_and_codes_of_tiny_and_large_values(torch, qg):
    cache = qg.kv8_cache(3, 1, 16, 64)
    table = int32(torch, [[0], [1], [2]])
    x = torch.zeros(3, 1, 64, device="cuda")
    x[1], x[2] = 2.0 ** -90, 3e38
    qg.kv8_append(x, -x, cache, table, int32(torch, [0, 1, 2, 3]), int32(torch, [1, 1, 1]))
    assert as_np(cache[2])[:, 0].tolist() == [2.0 ** -64, 2.0 ** -64, float(np.float32(3e38) / np.float32(127))]
    k, v = qg.kv8_gather(cache, table, int32(torch, [0, 1, 2, 3]), int32(torch, [1, 1, 1]), 3, dtype=torch.float32)
    assert not bool(k[:2].any()) and torch.allclose(k[2], x[2], rtol=1e-6) and torch.equal(v, -k)


def test_pages_and_rows_that_do_not_exist(torch, qg):
    """Wrong entries of the table, starts and lengths: nothing is written for them, they read as NaN, the rest is right."""
    heads, page, D = 2, 16, 64
    cache = random_cache(torch, qg, 6, heads, page, D, 1)
    before = [t.clone() for t in cache]
    table = int32(torch, [[0, -1], [6, 1], [2, 3], [4, 5], [2 ** 31 - 1, -2 ** 31]])
    x = torch.randn(40, heads, D, device="cuda").half()
    # sequence 2 has more tokens than its table; 3's rows leave the tensor; 4 has only bad pages
    starts, lengths = int32(torch, [0, 20, 22, 24, 41, 41]), int32(torch, [20, 18, 40, 17, 9])
    qg.kv8_append(x, x, cache, table, starts, lengths)
    changed = [bool((a != b).flatten(1).any(1)[p]) for a, b in zip(cache[:1], before[:1]) for p in range(6)]
    assert changed == [True, True, False, False, False, False]
    k, _ = qg.kv8_gather(cache, table, starts, lengths, 40)
    nan = as_np(torch.isnan(k).flatten(1).all(1)).tolist()
    assert nan[:24] == [False] * 16 + [True] * 4 + [False] * 2 + [True] * 2
    q = torch.randn(40, 4, D, device="cuda").half()
    O = torch.full_like(q, 7.0)
    qg.kv8_attention(q, cache, table, starts, lengths, O=O)
    nan = as_np(torch.isnan(O).flatten(1).all(1)).tolist()
    # rows 16 .. 19 see page 1 of sequence 0, which is bad; sequence 1's first page is
    assert nan[:24] == [False] * 16 + [True] * 8 and bool((O[24:] == 7).all())
    check_attention(torch, O[:16], q[:16], cache, table, [16], [16], D ** -0.5, True, "float16")
    for s, n in ((int32(torch, [5, 3, 3, 3, 3, 3]), lengths), (int32(torch, [-4, 2, 2, 2, 2, 2]), lengths),
                 (starts, int32(torch, [-5, -2 ** 31, 2 ** 31 - 1, 0, 0]))):
        held = [t.clone() for t in cache]
        qg.kv8_append(x, x, cache, table, s, n)
        assert all(torch.equal(a, b) for a, b in zip(held, cache)) or n is not lengths
        qg.kv8_gather(cache, table, s, n, 40)
        qg.kv8_attention(q, cache, table, s, n)


# ------------------------------------------------------------- attention

BATCHES = [
    ([1], [1]), ([1], [17]), ([1], [1000]), ([1, 1, 1], [5, 64, 129]), ([3], [3]), ([70], [70]), ([33], [200]),
    ([1, 40, 0, 7], [300, 40, 9, 77]), ([2, 1], [0, 3]), ([6, 4], [2, 4]), ([1], [3001]), ([1] * 20, list(range(3, 403, 20))),
    ([130, 1], [130, 1]), ([300], [777]),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("D,page", [(64, 16), (64, 128), (128, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("news,lengths", BATCHES)
def test_attention(torch, qg, news, lengths, D, page, dtype):
    gen = torch.Generator(device="cuda").manual_seed(len(news) + D)
    for heads, group, causal in ((2, 1, True), (1, 4, True), (2, 5, False), (1, 16, True)):
        cache, table = filled(torch, lengths, heads, D, page, 3)
        Q = torch.randn((sum(news) + 1, heads * group, D), generator=gen, device="cuda").to(getattr(torch, dtype))
        args = (table, int32(torch, starts_of(news)), int32(torch, lengths))
        O = torch.full_like(Q, 7.0)
        qg.kv8_attention(Q, cache, *args, causal=causal, O=O)
        check_attention(torch, O, Q, cache, table, news, lengths, D ** -0.5, causal, dtype)
        assert bool((O[sum(news):] == 7).all())
        again = qg.kv8_attention(Q, cache, *args, causal=causal)
        assert torch.equal(again[:sum(news)], O[:sum(news)])


@pytest.mark.parametrize("group", [3, 7, 8, 20, 33])
def test_attention_head_groups_and_views(torch, qg, group):
    """Groups that fill no tile or several; queries and outputs inside wider rows; another scale."""
    news, lengths, heads, D = [5, 1], [90, 200], 2, 128
    cache, table = filled(torch, lengths, heads, D, 32, 8)
    wide = torch.randn(6, heads * group * D + 11, device="cuda").bfloat16()
    Q = wide[:, 3:3 + heads * group * D].unflatten(1, (heads * group, D))
    out = torch.full_like(wide, 7.0)
    O = out[:, 5:5 + heads * group * D].unflatten(1, (heads * group, D))
    args = (table, int32(torch, starts_of(news)), int32(torch, lengths))
    for scale in (0.05, 0.0, -0.1):
        qg.kv8_attention(Q, cache, *args, scale, O=O)
        check_attention(torch, O, Q, cache, table, news, lengths, scale, True, "bfloat16")
    assert bool((out[:, :5] == 7).all()) and bool((out[:, 5 + heads * group * D:] == 7).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,page,D,news,lengths", [
    (2, 16, 64, [64], [2500]), (1, 64, 128, [40, 0, 33], [1030, 50, 2047]), (2, 32, 128, [100, 64], [70, 1500]),
    (1, 128, 64, [300], [1153]), (1, 64, 128, [32], [5000]), (3, 64, 64, [128, 1, 70], [128, 4097, 3000])])
def test_attention_of_few_units_shares_out_their_tokens(torch, qg, heads, page, D, news, lengths, causal):
    """Units whose tokens several CTAs take: odd shares, sequences shorter than the others, rows that see nothing."""
    cache, table = filled(torch, lengths, heads, D, page, len(news) + D)
    gen = torch.Generator(device="cuda").manual_seed(sum(lengths))
    Q = torch.randn(sum(news), heads * 4, D, generator=gen, device="cuda").half()
    args = (table, int32(torch, starts_of(news)), int32(torch, lengths))
    O = qg.kv8_attention(Q, cache, *args, causal=causal)
    check_attention(torch, O, Q, cache, table, news, lengths, D ** -0.5, causal, "float16")
    assert torch.equal(O, qg.kv8_attention(Q, cache, *args, causal=causal))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("heads,D,group,causal", [(2, 64, 4, True), (1, 128, 8, True), (2, 128, 1, False), (1, 64, 20, True)])
def test_prompts_next_to_single_tokens(torch, qg, heads, D, group, causal, dtype):
    """Sequences for either kernel in one batch, with some at the border between them and some without rows."""
    news = [1, 300, 0, 16, 15, 1, 33, 128, 2, 0, 127, 1]
    lengths = [700, 300, 50, 16, 1030, 1, 33, 2000, 5, 0, 1500, 0]
    cache, table = filled(torch, lengths, heads, D, 32, 11)
    gen = torch.Generator(device="cuda").manual_seed(group)
    Q = torch.randn(sum(news), heads * group, D, generator=gen, device="cuda").to(getattr(torch, dtype))
    args = (table, int32(torch, starts_of(news)), int32(torch, lengths))
    O = qg.kv8_attention(Q, cache, *args, causal=causal)
    check_attention(torch, O, Q, cache, table, news, lengths, D ** -0.5, causal, dtype)


def test_attention_of_few_units_keeps_what_is_not_finite_to_those_that_see_it(torch, qg):
    heads, D, page, length, new = 1, 64, 16, 2048, 64
    cache, table = filled(torch, [length], heads, D, page, 3)
    Q = torch.randn(new, 4, D, device="cuda").half()
    args = (table, int32(torch, [0, new]), int32(torch, [length]))
    want = qg.kv8_attention(Q, cache, *args)
    for which in (2, 3):
        for block, first in ((5, 0), (length // page - 2, new - 2 * page)):
            spoilt = [t.clone() for t in cache]
            spoilt[which][table[0, block].long()] = float("nan")
            O = qg.kv8_attention(Q, tuple(spoilt), *args)
            assert bool(torch.isnan(O[first:]).all()) and torch.equal(O[:first], want[:first])
    O = qg.kv8_attention(Q, cache, table[:, :-1].contiguous(), *args[1:])
    assert bool(torch.isnan(O).all())  # longer than its table


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_attention_over_pages_of_very_different_scales(torch, qg, dtype):
    """V scales over 2^-60 .. 2^60 next to each other: the weights' range does not depend on them."""
    news, lengths, heads, D, page = [1, 40], [200, 333], 2, 64, 16
    cache, table = filled(torch, lengths, heads, D, page, 5)
    e = torch.randint(-60, 61 if dtype == "bfloat16" else -20, cache[3].shape, device="cuda")
    cache[3].copy_(torch.where(torch.isnan(cache[3]), cache[3], torch.exp2(e.float())))
    Q = torch.randn(41, heads * 4, D, device="cuda").to(getattr(torch, dtype))
    args = (table, int32(torch, starts_of(news)), int32(torch, lengths))
    O = qg.kv8_attention(Q, cache, *args)
    check_attention(torch, O, Q, cache, table, news, lengths, D ** -0.5, True, dtype)


@pytest.mark.parametrize("small,large", [(-60, 60), (-64, 80), (-40, 115)])
@pytest.mark.parametrize("news", [1, 80])
def test_attention_counts_tokens_of_small_scales_next_to_large_ones(torch, qg, news, small, large):
    """Most of a row's weight on pages whose V scale is 2^small, some on pages of 2^large."""
    heads, D, page, length = 2, 64, 16, 180
    cache, table = filled(torch, [length], heads, D, page, 7)
    used = table[0, :-(-length // page)].long()
    for j, p in enumerate(used):
        cache[3][p] = 2.0 ** (large if j % 5 == 2 else small)
    gen = torch.Generator(device="cuda").manual_seed(news)
    for sharp in (0.1, 1.0, 4.0):
        Q = (sharp * torch.randn(news, heads * 4, D, generator=gen, device="cuda")).bfloat16()
        O = qg.kv8_attention(Q, cache, table, int32(torch, [0, news]), int32(torch, [length]))
        check_attention(torch, O, Q, cache, table, [news], [length], D ** -0.5, True, "bfloat16")


@pytest.mark.parametrize("new", [1, 64])
def test_tokens_that_nothing_was_written_to_are_zeros(torch, qg, new):
    heads, D, page, length = 1, 64, 16, 200
    cache = qg.kv8_cache(20, heads, page, D)
    table = torch.randperm(20, device="cuda")[:13].view(1, 13).int()
    kv = torch.randn(60, heads, D, device="cuda").half()
    qg.kv8_append(kv, kv, cache, table, int32(torch, [0, 60]), int32(torch, [100]))
    Q = torch.randn(new, 4, D, device="cuda").half()
    args = (table, int32(torch, [0, new]), int32(torch, [length]))
    O = qg.kv8_attention(Q, cache, *args)
    check_attention(torch, O, Q, cache, table, [new], [length], D ** -0.5, True, "float16")
    for s in cache[2:]:  # and so under scales of 0
        s[s == 2.0 ** -64] = 0
    assert torch.equal(qg.kv8_attention(Q, cache, *args), O)


def test_attention_with_large_and_small_queries(torch, qg):
    """bf16 queries far outside fp16's range, with keys to match, and sharp weights."""
    news, lengths, heads, D = [2, 20], [100, 150], 1, 128
    cache, table = filled(torch, lengths, heads, D, 64, 6)
    args = (table, int32(torch, starts_of(news)), int32(torch, lengths))
    for power in (-100, -20, 18, 60, 100):
        Q = (torch.randn(22, 2, D, device="cuda") * 2.0 ** power).bfloat16()
        scale = 2.0 ** -power * 0.3
        O = qg.kv8_attention(Q, cache, *args, scale)
        check_attention(torch, O, Q, cache, table, news, lengths, scale, True, "bfloat16")


@pytest.mark.parametrize("new", [3, 80])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-30])
def test_scales_of_any_sign(torch, qg, new, scale):
    cache, table = filled(torch, [300], 2, 128, 32, 13)
    gen = torch.Generator(device="cuda").manual_seed(new)
    Q = torch.randn(new, 8, 128, generator=gen, device="cuda").half()
    O = qg.kv8_attention(Q, cache, table, int32(torch, [0, new]), int32(torch, [300]), scale)
    check_attention(torch, O, Q, cache, table, [new], [300], scale, True, "float16")


@pytest.mark.parametrize("new", [3, 80])
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_queries_that_are_not_finite_spoil_their_own_results(torch, qg, new, dtype):
    cache, table = filled(torch, [400], 2, 64, 16, 17)
    gen = torch.Generator(device="cuda").manual_seed(new)
    good = torch.randn(new, 8, 64, generator=gen, device="cuda").to(getattr(torch, dtype))
    bad, places = good.clone(), [(0, 2, float("inf")), (1, 7, float("nan")), (new - 1, 0, -float("inf"))]
    for row, head, value in places:
        good[row, head] = 0
        bad[row, head, 5] = value
    args = (cache, table, int32(torch, [0, new]), int32(torch, [400]))
    O, want = qg.kv8_attention(bad, *args), qg.kv8_attention(good, *args)
    for row, head, _ in places:
        assert bool(torch.isnan(O[row, head]).all())
        O[row, head] = want[row, head]
    check_attention(torch, O, good, cache, table, [new], [400], 64 ** -0.5, True, dtype)


def test_attention_keeps_what_is_not_finite_to_those_that_see_it(torch, qg):
    """A page that holds a NaN, or a bad key, reaches the rows that see one of its tokens and no others."""
    D, page = 64, 16
    cache, table = filled(torch, [64], 1, D, page, 9)
    for which in (2, 3):
        spoilt = [t.clone() for t in cache]
        spoilt[which][table[0, 2].long()] = float("nan")
        Q = torch.randn(64, 2, D, device="cuda").half()
        O = qg.kv8_attention(Q, tuple(spoilt), table, int32(torch, [0, 64]), int32(torch, [64]))
        nan = as_np(torch.isnan(O).flatten(1).all(1))
        assert nan.tolist() == [False] * 32 + [True] * 32 and not bool(torch.isnan(O[:32]).any())
        check_attention(torch, O[:32], Q[:32], cache, table, [32], [32], D ** -0.5, True, "float16")
    Q[5, 1, 3] = float("nan")
    O = qg.kv8_attention(Q, cache, table, int32(torch, [0, 64]), int32(torch, [64]))
    nan = as_np(torch.isnan(O).all(2))
    assert nan[5].tolist() == [False, True] and nan.sum() == 1


def test_sequences_that_share_pages(torch, qg):
    cache, table = filled(torch, [160], 2, 128, 32, 4)
    shared = torch.cat((table, table, table)).contiguous()
    Q = torch.randn(6, 4, 128, device="cuda").half()
    news, lengths = [1, 2, 3], [160, 100, 33]
    O = qg.kv8_attention(Q, cache, shared, int32(torch, starts_of(news)), int32(torch, lengths))
    check_attention(torch, O, Q, cache, shared, news, lengths, 128 ** -0.5, True, "float16")


def test_attention_of_a_long_sequence(torch, qg):
    for D, page, n in ((128, 16, 1), (64, 64, 5)):
        cache, table = filled(torch, [70001], 1, D, page, 2, spread=0.2)
        Q = torch.randn(n, 4, D, device="cuda").half()
        O = qg.kv8_attention(Q, cache, table, int32(torch, [0, n]), int32(torch, [70001]))
        check_attention(torch, O, Q, cache, table, [n], [70001], D ** -0.5, True, "float16")


def test_many_sequences(torch, qg):
    rng = np.random.default_rng(3)
    lengths = rng.integers(0, 90, 1500).tolist()
    news = [int(min(n, rng.integers(0, 3))) for n in lengths]
    cache, table = filled(torch, lengths, 1, 64, 16, 2)
    Q = torch.randn(sum(news), 2, 64, device="cuda").bfloat16()
    O = qg.kv8_attention(Q, cache, table, int32(torch, starts_of(news)), int32(torch, lengths))
    check_attention(torch, O, Q, cache, table, news, lengths, 0.125, True, "bfloat16")


def test_empty(torch, qg):
    cache, table = filled(torch, [20], 1, 64, 16, 2)
    Q = torch.zeros(0, 2, 64, device="cuda").half()
    one = int32(torch, [0, 0]), int32(torch, [20])
    assert qg.kv8_attention(Q, cache, table, *one).shape == (0, 2, 64)
    qg.kv8_append(Q[:, :1], Q[:, :1], cache, table, *one)
    none = table[:0], int32(torch, [0]), int32(torch, [])
    out = torch.full((3, 2, 64), 7.0, device="cuda").half()
    qg.kv8_attention(out.clone(), cache, *none, O=out)
    assert bool((out == 7).all())


def test_streams_graphs_and_their_workspaces(torch, qg):
    """Other streams, two captured graphs that each keep a workspace, replayed in turn, and new lengths in place."""
    news, lengths = [1] * 5, [100, 900, 33, 4, 2000]
    cache, table = filled(torch, [n + 8 for n in lengths], 2, 128, 16, 2)
    starts, length = int32(torch, starts_of(news)), int32(torch, lengths)
    Qs = [torch.randn(5, 8, 128, device="cuda").half() for _ in range(2)]
    wants = [qg.kv8_attention(Q, cache, table, starts, length) for Q in Qs]
    sides = [torch.cuda.Stream() for _ in range(2)]
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
    outs = [qg.kv8_attention(Q, cache, table, starts, length, stream=s) for Q, s in zip(Qs, sides)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(wants, outs))
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, Q in zip(graphs, Qs):
        with torch.cuda.graph(g):
            outs.append(qg.kv8_attention(Q, cache, table, starts, length))
    for _ in range(2):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(wants, outs))
    length += 8
    graphs[1].replay()
    torch.cuda.synchronize()
    check_attention(torch, outs[1], Qs[1], cache, table, news, [n + 8 for n in lengths], 128 ** -0.5, True, "float16")


@pytest.mark.parametrize("group,news,lengths,later,grown", [
    (4, [64], [1500], [64], [1999]), (4, [60, 40], [1100, 90], [1, 70], [1999, 1500]),
    (8, [300, 1, 1, 0, 16], [400, 1300, 2, 9, 16], [1, 3, 0, 200, 90], [1, 1999, 7, 900, 1000])])
def test_a_graph_serves_other_rows_and_lengths(torch, qg, group, news, lengths, later, grown):
    """Shared units and batches for both kernels, captured; then other rows, lengths and rows of no sequence."""
    heads, D, page = 2, 128, 16
    cache, table = filled(torch, [1999] * len(news), heads, D, page, 21)
    gen = torch.Generator(device="cuda").manual_seed(group)
    Q = torch.randn(sum(news), heads * group, D, generator=gen, device="cuda").half()
    starts, length = int32(torch, starts_of(news)), int32(torch, lengths)
    graph = torch.cuda.CUDAGraph()
    qg.kv8_attention(Q, cache, table, starts, length)
    with torch.cuda.graph(graph):
        O = qg.kv8_attention(Q, cache, table, starts, length)
    for n, m in ((news, lengths), (later, grown), (news, lengths)):
        starts.copy_(int32(torch, starts_of(n)))
        length.copy_(int32(torch, m))
        O.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check_attention(torch, O, Q, cache, table, n, m, D ** -0.5, True, "float16")
        assert bool((O[sum(n):] == 7).all())


def test_a_layer_run_as_it_is_used(torch, qg):
    """Product, norm and rotation, append, attention, product: a prompt, then tokens one at a time, eagerly and as a graph.

    Each step is checked against its plain form on what the step before it gave.
    """
    dim, Hq, Hk, D, page = 256, 4, 2, 64, 16
    gen = torch.Generator(device="cuda").manual_seed(11)
    dt = torch.bfloat16
    Wqkv, Wo = (0.06 * torch.randn(s, generator=gen, device="cuda") for s in (((Hq + 2 * Hk) * D, dim), (dim, Hq * D)))
    qkv, so = qg.s8_quantize(Wqkv), qg.s8_quantize(Wo)
    gq, gk = (1 + 0.1 * torch.randn(D, generator=gen, device="cuda") for _ in range(2))
    turn = torch.arange(64, device="cuda").double()[:, None] * 1e4 ** (-torch.arange(0, D, 2, device="cuda").double() / D)
    angle = torch.cat((turn.cos(), turn.sin()), 1).float()
    cache, lengths = qg.kv8_cache(12, Hk, page, D), [17, 5]
    plain = ref.Cache(*(as_np(t).astype(np.int8 if t.dtype is torch.int8 else np.float32) for t in cache))
    table = int32(torch, [[3, 9, 1], [0, 7, 11]])

    def layer(X, positions, starts, length):
        P = qg.s8_linear(X, *qkv)
        Q, K, V = P.unflatten(1, (Hq + 2 * Hk, D)).split([Hq, Hk, Hk], 1)
        yq, yk, rq, rk = qg.qk_norm_rope(Q, K, gq, gk, positions, angle)
        qg.kv8_append(yk, V, cache, table, starts, length)
        O = qg.kv8_attention(yq, cache, table, starts, length)
        return P, yq, yk, V, O, qg.s8_linear(O.flatten(1), *so)

    def check(out, X, news, lengths, pos):
        from tests.test_rope_gpu import check_forward
        from tests.test_s8_gpu import check_product
        P, yq, yk, V, O, Y = out
        operand = lambda t: (as_np(t[0])[:, :], as_np(t[1]).astype(np.float32))  # noqa: E731
        check_product(P, *ref.s8_quantize(as_np(X)), *operand(qkv), None, "bfloat16")
        Q, K, _ = P.unflatten(1, (Hq + 2 * Hk, D)).split([Hq, Hk, Hk], 1)
        p = torch.tensor(pos)
        check_forward(yq, torch.from_numpy(ref.rms(as_np(Q), 1e-6)), Q, gq, p, angle, "half", "bfloat16")
        check_forward(yk, torch.from_numpy(ref.rms(as_np(K), 1e-6)), K, gk, p, angle, "half", "bfloat16")
        plain.append("k", as_np(yk), as_np(table), starts_of(news), lengths)
        plain.append("v", as_np(V), as_np(table), starts_of(news), lengths)
        for got, want in zip(cache, (plain.q["k"], plain.q["v"], plain.s["k"], plain.s["v"])):
            assert np.array_equal(as_np(got).astype(want.dtype), want)
        check_attention(torch, O, yq, cache, table, news, lengths, D ** -0.5, True, "bfloat16")
        check_product(Y, *ref.s8_quantize(as_np(O.flatten(1))), *operand(so), None, "bfloat16")

    X = torch.randn((22, dim), generator=gen, device="cuda").to(dt)
    pos = list(range(17)) + list(range(5))
    check(layer(X, int32(torch, pos), int32(torch, [0, 17, 22]), int32(torch, lengths)), X, lengths, lengths, pos)
    x, p, length, starts = X[:2].clone(), int32(torch, lengths), int32(torch, lengths), int32(torch, [0, 1, 2])
    graph = None
    for step in range(6):
        x.copy_(torch.randn((2, dim), generator=gen, device="cuda"))
        p.copy_(length)
        length += 1
        lengths = [n + 1 for n in lengths]
        if step < 2:
            out = layer(x, p, starts, length)
        else:
            if graph is None:
                held = [t.clone() for t in cache]
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out = layer(x, p, starts, length)
                for a, b in zip(cache, held):
                    a.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
        check(out, x, [1, 1], lengths, [n - 1 for n in lengths])
