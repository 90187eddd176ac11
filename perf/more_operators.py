"""Cases of the operators of an attention layer that works on 8-bit operands.

A case is one call, or one short chain of calls, of a program that runs or
trains the attention of transformer blocks:

  s8_linear      a linear layer in 8-bit integers: Y = Q(X) . Q(W)^T + bias, with a
                 scale for each token (found in the call) and each output channel
  qk_norm_rope   RMS norm of every head of Q and K and the rotation by position
  qk_norm_rope_backward   its gradients
  append         new tokens' K and V into a paged cache of 8-bit codes with a scale
                 for each page and head; the pages that this touches, read back
  attention      attention of new tokens over such a cache

Codes are round(x / s) in -127 .. 127 with s = amax / 127: over a row for
s8_linear, over the tokens of one page and head for the cache, where a page that
holds tokens already keeps the larger scale, its older codes rounded to it.
Cache: codes pages x heads x page x D, scales pages x heads, a table of pages
for every sequence.  New tokens of all sequences follow one another; sequence b has
rows starts[b] .. starts[b + 1], which are the last of its lengths[b] tokens.

`run` computes the plain form in 32 bits from elementary operations, or, where
`own` is true, calls bit_quantized_tensor_gb300.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6
ROW_FLOOR = 2.0 ** -100   # smallest scale of a row of codes
PAGE_FLOOR = 2.0 ** -64   # smallest scale of a page of the cache


def listed():
    return [
        # one new token against one layer's weights: latency and the weights' bytes
        {"name": "s8_linear 1x4096x4096", "op": "s8_linear", "dtype": "bf16", "m": 1, "n": 4096, "k": 4096},
        # a ragged prompt and an odd layer
        {"name": "s8_linear 777x1001x2304", "op": "s8_linear", "dtype": "f16", "m": 777, "n": 1001, "k": 2304},
        # a long prompt against the largest benchmark layer: tensor cores
        {"name": "s8_linear 4096x8192x8192", "op": "s8_linear", "dtype": "bf16", "m": 4096, "n": 8192, "k": 8192},
        # a batch of one new token for each of a few sequences: latency
        {"name": "qk_norm_rope f16 5 tokens", "op": "qk_norm_rope", "dtype": "f16", "t": 5, "hq": 12, "hk": 4, "d": 64,
         "r": 64, "style": "pairs"},
        # a long prompt's queries and keys: bandwidth
        {"name": "qk_norm_rope bf16 8192 tokens", "op": "qk_norm_rope", "dtype": "bf16", "t": 8192, "hq": 32, "hk": 8,
         "d": 128, "r": 128, "style": "half"},
        # the gradients of a training step of the same
        {"name": "qk_norm_rope_backward bf16 8192 tokens", "op": "qk_norm_rope_backward", "dtype": "bf16", "t": 8192,
         "hq": 32, "hk": 8, "d": 128, "r": 128, "style": "half"},
        # a ragged micro-batch of fp32 heads that rotate in part
        {"name": "qk_norm_rope_backward f32 1333 tokens", "op": "qk_norm_rope_backward", "dtype": "f32", "t": 1333,
         "hq": 12, "hk": 12, "d": 80, "r": 32, "style": "half"},
        # one new token for each sequence of a batch: latency
        {"name": "append 64 x 1", "op": "append", "dtype": "bf16", "b": 64, "most": 2048, "new": 1, "hk": 8, "d": 128, "page": 32},
        # ragged prompts into the cache
        {"name": "append 7 x 1333", "op": "append", "dtype": "f16", "b": 7, "most": 2304, "new": 1333, "hk": 4, "d": 64, "page": 16},
        # a batch of new tokens over caches of many lengths: the cache's bytes
        {"name": "attention 64 x 1 over 8192", "op": "attention", "dtype": "bf16", "b": 64, "most": 8192, "new": 1, "hq": 32,
         "hk": 8, "d": 128, "page": 64, "causal": True},
        # one sequence, very long, odd: the axis has to be split
        {"name": "attention 1 x 1 over 131071", "op": "attention", "dtype": "f16", "b": 1, "most": 131071, "new": 1, "hq": 32,
         "hk": 8, "d": 128, "page": 16, "causal": True},
        # pieces of long prompts over what is cached of them: tensor cores
        {"name": "attention 4 x 2048 over 8192", "op": "attention", "dtype": "bf16", "b": 4, "most": 8192, "new": 2048, "hq": 32,
         "hk": 8, "d": 128, "page": 64, "causal": True},
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm, as often odd as even."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["s8_linear", "qk_norm_rope", "qk_norm_rope_backward", "append", "attention", "attention"])
    if op == "s8_linear":
        m, n, k = _spread(rng, 1, 8192), _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        return {"op": op, "dtype": rng.choice(["f16", "bf16"]), "m": max(1, min(m, (1 << 38) // (n * k))), "n": n, "k": k}
    if op.startswith("qk_norm_rope"):
        hk, d = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 80, 96, 128, 256])
        hq = hk * rng.choice([1, 2, 3, 4, 8])
        t = min(_spread(rng, 1, 16384), (1 << 25) // ((hq + hk) * d))
        return {"op": op, "dtype": rng.choice(["f16", "bf16", "f32"]), "t": t, "hq": hq, "hk": hk, "d": d,
                "r": rng.choice([d, d, d // 2]), "style": rng.choice(["half", "pairs"])}
    hk, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "b": _spread(rng, 1, 64)}
    if op == "append":
        most = min(_spread(rng, 1, 8192), (1 << 17) // case["b"])
        return {**case, "most": most, "new": rng.choice([1, _spread(rng, 1, most)]), "hk": hk, "d": d, "page": page}
    case["most"] = min(_spread(rng, 1, 131072), (1 << 19) // case["b"])
    hq = hk * rng.choice([1, 2, 4, 5, 8])
    new = _spread(rng, 1, min(4096, case["most"])) if rng.random() < 0.5 else 1
    new = max(1, min(new, (1 << 31) // (case["b"] * case["most"] * hq)))
    return {**case, "new": new, "hq": hq, "hk": hk, "d": d, "page": page, "causal": rng.random() < 0.75}


# ------------------------------------------------------------------ the batch of a case

def _batch(case):
    """(new tokens, lengths) of every sequence: ragged, the first at the case's most."""
    rng = random.Random("%(b)d %(most)d %(new)d" % case)
    b, most, new = case["b"], case["most"], case["new"]
    lengths = [most] + [rng.randint((most + 3) // 4, most) for _ in range(b - 1)]
    news = [new] + [rng.randint((new + 1) // 2, new) for _ in range(b - 1)]
    return [min(n, m) for n, m in zip(news, lengths)], lengths


def _pages(case):
    page = case["page"]
    return (case["most"] + page - 1) // page


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return out


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plain forms

def _row_codes(x):
    """x (rows x K, 32 bits) -> whole codes as fp32, scales."""
    s = (x.abs().amax(1) / 127.0).clamp(min=ROW_FLOOR)
    return torch.round(x * (1.0 / s)[:, None]).clamp(-127, 127), s


def _turned(x, case, cos, sin, back=False):
    """The rotation of the first r values of every head (or its transpose)."""
    r, half = case["r"], case["r"] // 2
    cos, sin = cos[:, None, :], sin[:, None, :]
    if back:
        sin = -sin
    if case["style"] == "half":
        a, b = x[..., :half], x[..., half:r]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., r:]), 2)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    y = torch.stack((a * cos - b * sin, b * cos + a * sin), 3).flatten(2)
    return torch.cat((y, x[..., r:]), 2)


def _angles(s):
    rows = s["table"][s["positions"].long()]
    half = s["case"]["r"] // 2
    return rows[:, :half], rows[:, half:]


def _heads(s):
    """Views of Q and K in the packed rows of one product's output."""
    c, t = s["case"], s["x"].shape[0]
    nq, nk = c["hq"] * c["d"], c["hk"] * c["d"]
    return s["x"][:, :nq].view(t, c["hq"], c["d"]), s["x"][:, nq:nq + nk].view(t, c["hk"], c["d"])


def _rms(x):
    return 1.0 / torch.sqrt((x * x).mean(2) + EPS)


def _tokens(starts, lengths, rows):
    """Sequence and position of every row."""
    starts, lengths = starts.long(), lengths.long()
    i = torch.arange(rows, device=DEV)
    b = torch.bucketize(i, starts[1:], right=True)
    return b, lengths[b] - starts[b + 1] + i


def _gather_plain(codes, scales, page_of, offset, dt):
    return (codes[page_of, :, offset].float() * scales[page_of][:, :, None]).to(dt)


def _append_plain(x, codes, scales, table, starts, lengths):
    page = codes.shape[2]
    x = x.float()
    b, pos = _tokens(starts, lengths, x.shape[0])
    pages, offset = table.long()[b, pos // page], pos % page
    # only the first page that a sequence's new tokens touch holds tokens already
    n = (starts[1:] - starts[:-1]).long()
    at = lengths.long() - n
    first, kept = table.long().gather(1, (at // page)[:, None])[:, 0], at % page
    amax = torch.zeros_like(scales)
    amax.scatter_reduce_(0, pages[:, None].expand(-1, x.shape[1]), x.abs().amax(2), "amax")
    old = torch.where((kept > 0)[:, None], scales[first], torch.zeros_like(scales[first]))
    new = (amax / 127.0).clamp(min=PAGE_FLOOR)
    new[first] = torch.maximum(new[first], old)
    ratio = old / new[first]
    was = codes[first]
    keep = torch.arange(page, device=DEV)[None, :] < kept[:, None]
    now = torch.round(was.float() * ratio[:, :, None, None]).to(torch.int8)
    codes[first] = torch.where(keep[:, None, :, None], now, was)
    scales[pages] = new[pages]
    r = 1.0 / scales[pages]
    codes[pages, :, offset] = torch.round(x * r[:, :, None]).clamp(-127, 127).to(torch.int8)


def _attention_plain(s):
    c, q = s["case"], s["q"].float()
    page, hk, d, b = c["page"], c["hk"], c["d"], c["b"]
    g, n = c["hq"] // hk, c["new"]
    table = s["table"].long()
    span = table.shape[1] * page
    k = (s["kq"][table].float() * s["ks"][table][..., None, None]).transpose(1, 2).reshape(b, hk, span, d)
    seq, pos = _tokens(s["starts"], s["lengths"], q.shape[0])
    i = torch.arange(q.shape[0], device=DEV) - s["starts"].long()[seq]
    full = q.new_zeros(b, n, c["hq"], d)
    full[seq, i] = q
    full = full.view(b, n, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, n * g, d)
    w = (full @ k.transpose(2, 3)).mul_(s["scale"]).view(b, hk, n, g, span)
    del k
    # how many tokens each query sees
    lengths = s["lengths"].long()
    sees = lengths[:, None].expand(b, n)
    if c["causal"]:
        have = (s["starts"][1:] - s["starts"][:-1]).long()
        sees = (lengths - have + 1)[:, None] + torch.arange(n, device=DEV)[None, :]
    hide = torch.arange(span, device=DEV)[None, None, :] >= sees[:, :, None]
    w.masked_fill_(hide[:, None, :, None, :], -math.inf)
    w.sub_(w.amax(4, keepdim=True)).exp_()
    total = w.sum(4, keepdim=True)
    v = (s["vq"][table].float() * s["vs"][table][..., None, None]).transpose(1, 2).reshape(b, hk, span, d)
    o = (w.view(b, hk, n * g, span) @ v).view(b, hk, n, g, d) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(b, n, c["hq"], d)
    return o[seq, i].to(s["q"].dtype)


# ------------------------------------------------------------------ the cases

def _filled(x, page):
    """Codes and scales of full pages (pages x heads x page x D)."""
    s = (x.abs().amax((2, 3)) / 127.0).clamp(min=PAGE_FLOOR)
    return torch.round(x * (1.0 / s)[:, :, None, None]).clamp_(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    dt, op = DTYPES[case["dtype"]], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    state = {"case": case}
    if op == "s8_linear":
        m, n, k = case["m"], case["n"], case["k"]
        # activations: a spread of row sizes and a few loud channels
        loud = torch.where(torch.rand(k, generator=g, device=DEV) < 0.01, 8.0, 1.0)
        state["x"] = (normal(m, k) * loud * torch.exp(0.5 * normal(m, 1))).to(dt)
        w = normal(n, k) * torch.exp(0.3 * normal(n, 1)) / math.sqrt(k)
        codes, state["ws"] = _row_codes(w)
        # rows of codes are padded to 16 bytes
        state["wq"] = torch.nn.functional.pad(codes, (0, -k % 16)).to(torch.int8)
        state["bias"] = (0.1 * normal(n)).to(dt)
        return state
    if op.startswith("qk_norm_rope"):
        t, hq, hk, d, r = case["t"], case["hq"], case["hk"], case["d"], case["r"]
        # one product's output holds Q, K and V
        state["x"] = (normal(t, (hq + 2 * hk) * d) * torch.exp(0.5 * normal(t, 1)) + 0.1 * normal((hq + 2 * hk) * d)).to(dt)
        state["gq"], state["gk"] = (1.0 + 0.1 * normal(d)).to(dt), (1.0 + 0.1 * normal(d)).to(dt)
        most = 16384
        turn = torch.arange(most, device=DEV, dtype=torch.float64)[:, None] * 1e4 ** (
            -torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
        state["table"] = torch.cat((torch.cos(turn), torch.sin(turn)), 1).float()
        # several sequences of a batch, each from a place of its own
        first = int(torch.randint(0, 1000, (1,), generator=g, device=DEV))
        state["positions"] = ((torch.arange(t, device=DEV) * 7 // 4 + first) % most).to(torch.int32)
        if op == "qk_norm_rope_backward":
            q, k = _heads(state)
            state["rq"], state["rk"] = _rms(q.float()), _rms(k.float())
            state["dq"] = (1e-2 * normal(t, hq, d) * torch.exp(0.5 * normal(t, 1, 1))).to(dt)
            state["dk"] = (1e-2 * normal(t, hk, d) * torch.exp(0.5 * normal(t, 1, 1))).to(dt)
        return state
    b, hk, d, page = case["b"], case["hk"], case["d"], case["page"]
    news, lengths = _batch(case)
    per = _pages(case)
    pool = b * per + 3
    order = torch.randperm(pool, generator=g, device=DEV)[:b * per]
    state["table"] = order.view(b, per).to(torch.int32)
    # keys have loud channels; what a page holds differs in size from page to page
    loud = 1.0 + 3.0 * (torch.rand(hk, 1, d, generator=g, device=DEV) < 0.05)
    state["kq"], state["ks"] = _filled(normal(pool, hk, page, d) * loud * torch.exp(0.2 * normal(pool, 1, 1, 1)), page)
    state["vq"], state["vs"] = _filled(normal(pool, hk, page, d) * torch.exp(0.2 * normal(pool, 1, 1, 1)), page)
    state["starts"], state["lengths"] = _int32(_starts(news)), _int32(lengths)
    if op == "append":
        state["k"] = (normal(sum(news), hk, d) * loud.view(1, hk, d)).to(dt)
        state["v"] = normal(sum(news), hk, d).to(dt)
        # what is read back: all tokens of the pages that are touched
        count = [m - (m - n) // page * page for n, m in zip(news, lengths)]
        state["back"], state["rows"] = _int32(_starts(count)), sum(count)
        return state
    state["q"] = normal(sum(news), case["hq"], d).to(dt)
    state["scale"] = 1.0 / math.sqrt(d)
    return state


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import bit_quantized_tensor_gb300 as qg
    c = s["case"]
    op = c["op"]
    if op == "s8_linear":
        return qg.s8_linear(s["x"], s["wq"], s["ws"], bias=s["bias"])
    if op == "qk_norm_rope":
        q, k = _heads(s)
        return qg.qk_norm_rope(q, k, s["gq"], s["gk"], s["positions"], s["table"], EPS, style=c["style"])
    if op == "qk_norm_rope_backward":
        q, k = _heads(s)
        return qg.qk_norm_rope_backward(s["dq"], s["dk"], q, k, s["gq"], s["gk"], s["positions"], s["table"], s["rq"],
                                        s["rk"], style=c["style"])
    cache = (s["kq"], s["vq"], s["ks"], s["vs"])
    if op == "append":
        qg.kv8_append(s["k"], s["v"], cache, s["table"], s["starts"], s["lengths"])
        return qg.kv8_gather(cache, s["table"], s["back"], s["lengths"], s["rows"], dtype=s["k"].dtype)
    return qg.kv8_attention(s["q"], cache, s["table"], s["starts"], s["lengths"], s["scale"], causal=c["causal"])


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "s8_linear":
        xq, xs = _row_codes(s["x"].float())
        y = xq @ s["wq"][:, :c["k"]].float().t()
        return (y * xs[:, None] * s["ws"] + s["bias"].float()).to(s["x"].dtype)
    if op == "append":
        _append_plain(s["k"], s["kq"], s["ks"], s["table"], s["starts"], s["lengths"])
        _append_plain(s["v"], s["vq"], s["vs"], s["table"], s["starts"], s["lengths"])
        b, pos = _tokens(s["back"], s["lengths"], s["rows"])
        at = s["table"].long()[b, pos // c["page"]], pos % c["page"]
        return (_gather_plain(s["kq"], s["ks"], *at, s["k"].dtype), _gather_plain(s["vq"], s["vs"], *at, s["k"].dtype))
    if op == "attention":
        return _attention_plain(s)
    cos, sin = _angles(s)
    q, k = (x.float() for x in _heads(s))
    dt, gq, gk = s["x"].dtype, s["gq"].float(), s["gk"].float()
    if op == "qk_norm_rope":
        rq, rk = _rms(q), _rms(k)
        return (_turned(q * rq[:, :, None] * gq, c, cos, sin).to(dt),
                _turned(k * rk[:, :, None] * gk, c, cos, sin).to(dt), rq, rk)
    dzq, dzk = _turned(s["dq"].float(), c, cos, sin, True), _turned(s["dk"].float(), c, cos, sin, True)
    hq, hk = q * s["rq"][:, :, None], k * s["rk"][:, :, None]
    eq, ek = dzq * gq, dzk * gk
    dq = s["rq"][:, :, None] * (eq - hq * (eq * hq).mean(2, keepdim=True))
    dk = s["rk"][:, :, None] * (ek - hk * (ek * hk).mean(2, keepdim=True))
    return dq.to(dt), dk.to(dt), (dzq * hq).sum((0, 1)), (dzk * hk).sum((0, 1))


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op == "s8_linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * e + n * k + 4 * n + n * e + m * n * e, "flops": 2 * m * n * k}
    if op.startswith("qk_norm_rope"):
        heads, t, d = case["hq"] + case["hk"], case["t"], case["d"]
        fixed = 2 * d * e + t * (4 + 4 * case["r"]) + 4 * t * heads
        if op == "qk_norm_rope":
            return {"bytes": 2 * t * heads * d * e + fixed, "flops": 8 * t * heads * d}
        return {"bytes": 3 * t * heads * d * e + fixed + 8 * d, "flops": 16 * t * heads * d}
    news, lengths = _batch(case)
    hk, d, page = case["hk"], case["d"], case["page"]
    if op == "append":
        # the new tokens are read, their codes written, and what the touched pages hold read back
        back = sum(m - (m - n) // page * page for n, m in zip(news, lengths))
        return {"bytes": 2 * sum(news) * hk * d * (e + 1) + 2 * back * hk * d * (1 + e) + 16 * hk * back // page,
                "flops": 8 * sum(news) * hk * d}
    hq = case["hq"]
    if case["causal"]:
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(news, lengths))
    else:
        pairs = sum(n * m for n, m in zip(news, lengths))
    pages = sum((m + page - 1) // page for m in lengths)
    return {"bytes": 2 * sum(lengths) * hk * d + pages * (4 + 8 * hk) + 2 * sum(news) * hq * d * e,
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ in 64 bits

def _exact_turned(x, case, angles, sign):
    r = case["r"]
    i = torch.arange(r // 2, device=DEV)
    first, second = (i, i + r // 2) if case["style"] == "half" else (2 * i, 2 * i + 1)
    z = torch.complex(x[..., first], x[..., second])
    c, s = angles[:, :r // 2].double(), angles[:, r // 2:].double() * sign
    z = z * torch.complex(c, s)[:, None, :]
    out = x.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_append(x, codes, scales, table, news, lengths, page, dt):
    """Values of the touched pages after the append, sequence by sequence.  The steps that the format's
    definition takes in 32 bits (scale, its inverse, the scaled value) are rounded to 32 bits here too."""
    out, row = [], 0
    table = table.tolist()
    for b, (n, m) in enumerate(zip(news, lengths)):
        for j in range((m - n) // page, (m + page - 1) // page):
            lo, hi = max(m - n, j * page), min(m, (j + 1) * page)
            p, kept = table[b][j], lo - j * page
            v = x[row:row + hi - lo].double()
            row += hi - lo
            s = (v.abs().amax((0, 2)) / 127.0).float().double().clamp(min=PAGE_FLOOR)
            part = []
            if kept:
                s = torch.maximum(s, scales[p].double())
                f = (scales[p].double() / s).float().double()
                part.append(torch.round((codes[p, :, :kept].double() * f[:, None, None]).float().double()).transpose(0, 1))
            r = (1.0 / s).float().double()
            part.append(torch.round((v * r[:, None]).float().double()).clamp(-127, 127))
            out.append(torch.cat(part) * s[:, None])
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "s8_linear":
        x = s["x"].double()
        sx = torch.clamp((x.abs().max(1).values / 127.0).float().double(), min=ROW_FLOOR)
        inverse = (1.0 / sx).float().double()
        q = torch.round((x * inverse[:, None]).float().double())
        q = torch.minimum(torch.maximum(q, q.new_tensor(-127.0)), q.new_tensor(127.0))
        w = s["wq"].double()[:, :case["k"]] * s["ws"].double()[:, None]
        return (q * sx[:, None]) @ w.t() + s["bias"].double()
    if op in ("append", "attention"):
        news, lengths = _batch(case)
        page, hk = case["page"], case["hk"]
        if op == "append":
            if sum(lengths) > 200000 or sum((m + page - 1) // page for m in lengths) > 20000:
                return None
            return tuple(_exact_append(s[x], s[x + "q"], s[x + "s"], s["table"], news, lengths, page, None) for x in "kv")
        out, row, g = [], 0, case["hq"] // hk
        for b, (n, m) in enumerate(zip(news, lengths)):
            pages = s["table"][b, :(m + page - 1) // page].long()
            k, v = ((s[x + "q"][pages].double() * s[x + "s"][pages].double()[:, :, None, None]).permute(1, 0, 2, 3)
                    .flatten(1, 2)[:, :m] for x in "kv")
            q = s["q"][row:row + n].double()
            row += n
            seen = torch.arange(m, device=DEV)[None, :] <= (m - n + torch.arange(n, device=DEV))[:, None]
            heads = []
            for h in range(case["hq"]):
                a = torch.einsum("nd,md->nm", q[:, h], k[h // g]) * s["scale"]
                if case["causal"]:
                    a = torch.where(seen, a, torch.full_like(a, -math.inf))
                heads.append(torch.softmax(a, 1) @ v[h // g])
            out.append(torch.stack(heads, 1))
        return torch.cat(out)
    angles = s["table"][s["positions"].long()]
    q, k = (x.double() for x in _heads(s))
    gq, gk = s["gq"].double(), s["gk"].double()
    if op == "qk_norm_rope":
        rq, rk = ((torch.einsum("thd,thd->th", x, x) / case["d"] + EPS) ** -0.5 for x in (q, k))
        return (_exact_turned(q * rq[..., None] * gq, case, angles, 1.0),
                _exact_turned(k * rk[..., None] * gk, case, angles, 1.0), rq, rk)
    out, sums = [], []
    # the 1 / rms that the call is given
    for dy, x, gain, inv in ((s["dq"], q, gq, s["rq"]), (s["dk"], k, gk, s["rk"])):
        inv = inv.double()[..., None]
        dz = _exact_turned(dy.double(), case, angles, -1.0)
        xh = x * inv
        dot = torch.einsum("thd,thd->th", dz * gain, xh) / case["d"]
        out.append(inv * (dz * gain - xh * dot[..., None]))
        sums.append(torch.einsum("thd,thd->d", dz, xh))
    return out[0], out[1], sums[0], sums[1]
