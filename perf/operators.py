"""What is timed of the 4-bit key/value cache: writing it, reading it back, attending over it.

The cache is paged.  A page holds `page` tokens of every key/value head; a token's row of
`dim` channels is stored as `dim / 2` bytes of 4-bit codes (channel 2i in the low half of byte
i, channel 2i + 1 in the high half) and `dim / 32` bf16 scales, one for each 32 channels:

    m    = the value of largest magnitude in the group (the positive one of an equal pair)
    s    = -m / 8, rounded to 5 significant bits (ties to even)
    code = clamp(rint(x / s), -8, 7) + 8        and reads back as (code - 8) * s

Operators (the entry points of the library, called where `own` is true):

* "write":  fa_kv4_append quantises the new tokens' keys and values into the cache, and
            fa_kv4_read gives the same positions back as bf16;
* "read":   fa_kv4_read gives a span of the cache back as dense bf16;
* "attend": fa_fwd_kv4, O = softmax(scale * Q K^T + mask) V and its log-sum-exp over the cache.

A case: `batch` sequences, `heads` query heads on `kv_heads` key/value heads, up to `queries` new
tokens and up to `keys` keys a sequence (spread over the range where `ragged`), `dim` channels a
head, `page` tokens a page, `causal` (query i of a sequence stands at its key length - its query
length + i) and `window` (keys further back than that are hidden; -1: none).
"""
import math

import torch

own = False

GROUP = 32
LARGEST = 2.0 ** 120    # a group that holds more, or what is not finite, reads back as NaN
SMALLEST = 2.0 ** -107  # a group that holds less reads back as zeros


def _case(op, batch, heads, kv_heads, queries, keys, dim, page, ragged=False, causal=False, window=-1):
    return {"op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "queries": queries, "keys": keys,
            "dim": dim, "page": page, "ragged": ragged, "causal": causal, "window": window}


def listed():
    return [
        # the tokens of one decoding step of a batch, each behind its own sequence: latency counts
        {"name": "write_step", **_case("write", 24, 8, 8, 1, 2048, 128, 64, ragged=True)},
        # short prompts of a batch with 12 heads of 64, each of its own length
        {"name": "write_prompts_d64", **_case("write", 8, 12, 12, 1024, 1024, 64, 16, ragged=True)},
        # whole long prompts, with a length that fills neither tiles nor pages
        {"name": "write_prompts_d128", **_case("write", 2, 32, 32, 8000, 8000, 128, 64)},
        # a short prefix taken back for a prompt that continues it
        {"name": "read_prefix_d64", **_case("read", 16, 16, 16, 512, 512, 64, 32, ragged=True)},
        # a long context taken back whole
        {"name": "read_long_d128", **_case("read", 1, 8, 8, 65536, 65536, 128, 256)},
        # one sequence, one token, a short context: latency alone counts
        {"name": "attend_one_short", **_case("attend", 1, 8, 8, 1, 700, 128, 64)},
        # a small batch with 12 heads of 64 at the end of its context
        {"name": "attend_step_d64", **_case("attend", 8, 12, 12, 1, 1024, 64, 16, ragged=True)},
        # decoding one sequence with a very long context and few heads
        {"name": "attend_64k_h8", **_case("attend", 1, 8, 8, 1, 65536, 128, 64)},
        # decoding a batch of unlike lengths, four query heads to each key/value head
        {"name": "attend_batch_ragged", **_case("attend", 32, 32, 8, 1, 16384, 128, 64, ragged=True)},
        # a few proposed tokens checked at once, causal among themselves, with a window
        {"name": "attend_proposed_window", **_case("attend", 16, 16, 4, 5, 8000, 128, 32, ragged=True, causal=True, window=2048)},
        # every head its own keys, long contexts: the whole cache is streamed once
        {"name": "attend_16k_h32", **_case("attend", 4, 32, 32, 1, 16384, 128, 128)},
        # a piece of a prompt over what is cached before it: compute counts
        {"name": "attend_chunk", **_case("attend", 2, 32, 8, 512, 8000, 128, 64, causal=True)},
    ]


def _between(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 12, 16, 32])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    ragged = rng.random() < 0.6
    if op == "attend":
        group = rng.choice([1, 1, 2, 3, 4, 8])
        queries = rng.choice([1, 1, 1, rng.randint(2, 9), _between(rng, 10, 512)])
        keys = _between(rng, 1, 65536)
        most = 4 * 32 * 16384 // (kv_heads * keys)                 # no more cache than the largest listed case
        rows = int(2 * 32 * 512 * 8000 / (queries * keys * kv_heads * group))  # nor more products
        batch = _between(rng, 1, max(1, min(64, most, rows)))
        while batch * kv_heads * group * queries * keys > 2 * 32 * 512 * 8000 or batch * kv_heads * keys > 4 * 32 * 16384:
            keys = max(1, keys // 2)
        window = rng.choice([-1, -1, _between(rng, 1, 4096)])
        return _case(op, batch, kv_heads * group, kv_heads, queries, keys, dim, page, ragged, rng.random() < 0.6, window)
    keys = _between(rng, 1, 65536)
    queries = keys if op == "read" or rng.random() < 0.5 else _between(rng, 1, min(keys, 64))
    batch = _between(rng, 1, max(1, min(64, 2 * 32 * 8000 // (kv_heads * keys))))
    while batch * kv_heads * keys > 2 * 32 * 8000:
        keys = max(1, keys // 2)
        queries = min(queries, keys)
    return _case(op, batch, kv_heads, kv_heads, queries, keys, dim, page, ragged)


def _lengths(case):
    """(key lengths, query or new-token lengths) of the sequences, as lists; the order is for the seed to choose."""
    n, keys, queries = case["batch"], case["keys"], case["queries"]
    if not case["ragged"]:
        return [keys] * n, [queries] * n
    part = [(i * 0.6180339887498949) % 1.0 for i in range(n)]
    kl = [keys] + [max(1, int(keys * p)) for p in part[1:]]
    ql = [min(k, queries if case["op"] != "attend" else max(1, queries - i % 3)) for i, k in enumerate(kl)]
    return kl, ql


def _random(shape, gen, sigma=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sigma


def _tokens(case, count, gen):
    """Keys and values [batch, kv_heads, count, dim] in bf16: keys with channels of unlike size and an offset, values plain."""
    shape = (case["batch"], case["kv_heads"], count, case["dim"])
    per = (1, case["kv_heads"], 1, case["dim"])
    k = _random(shape, gen) * torch.exp(_random(per, gen, 0.5)) + _random(per, gen, 0.5)
    return k.to(torch.bfloat16), _random(shape, gen, 0.7).to(torch.bfloat16)


def _scales(x):
    """The groups' scales in 32 bits: x [..., groups, 32]."""
    high, low = x.amax(-1), x.amin(-1)
    m = torch.where(high >= -low, high, low)
    whole = torch.isfinite(m) & (m.abs() <= LARGEST)
    part, power = torch.frexp(torch.where(whole, m, torch.zeros_like(m)))
    s = -torch.ldexp(torch.round(part * 32.0), power - 8)
    s = torch.where(m.abs() < SMALLEST, torch.zeros_like(s), s)
    return torch.where(whole, s, torch.full_like(s, math.nan))


def _quantise(x):
    """bf16 [..., dim] to (bytes [..., dim/2], bf16 scales [..., dim/32])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    s = _scales(g)
    t = torch.where((s == 0)[..., None] | torch.isnan(s)[..., None], torch.zeros_like(g), g / s[..., None])
    c = (torch.round(t).clamp(-8, 7) + 8).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.to(torch.bfloat16)


def _values(codes, scales):
    """Bytes [..., dim/2] and scales [..., dim/32] to the values they stand for, 32 bits [..., dim]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, GROUP)) * scales.float()[..., None]).flatten(-2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    order = torch.randperm(case["batch"], generator=gen, device="cuda")
    kl, ql = (torch.tensor(x, dtype=torch.int32, device="cuda")[order] for x in _lengths(case))
    b, h, d, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    per_seq = -(-case["keys"] // page)
    pages = b * per_seq
    st = {"case": case, "key_lens": kl.contiguous(), "new_lens": ql.contiguous(), "max_pages": per_seq, "pages": pages,
          "table": torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).view(b, per_seq).contiguous()}
    for t in ("k", "v"):
        st[t + "_codes"] = torch.zeros((pages, h, page, d // 2), dtype=torch.uint8, device="cuda")
        st[t + "_scales"] = torch.zeros((pages, h, page, d // GROUP), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "write":
        st["k"], st["v"] = _tokens(case, case["queries"], gen)
        st["first"] = (st["key_lens"] - st["new_lens"]).contiguous()
        return st
    # a filled cache: the contents of the pages, page by page (their order is the table's, which is random)
    for t, x in zip("kv", _tokens({**case, "batch": 1}, pages * page, gen)):
        codes, scales = _quantise(x)
        for name, y in (("_codes", codes), ("_scales", scales)):
            st[t + name].copy_(y.view(h, pages, page, -1).transpose(0, 1))
    if case["op"] == "attend":
        st["q"] = _random((b, case["heads"], case["queries"], d), gen).to(torch.bfloat16)
    else:
        st["first"] = torch.zeros_like(st["key_lens"])
    return st


def _run_own(st):
    import io_aware_exact_24_b200 as fa
    c = st["case"]
    b, h, d, n = c["batch"], c["kv_heads"], c["dim"], c["queries"]
    cache = (st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["table"], st["key_lens"])
    sizes = (d, st["pages"], c["page"], st["max_pages"])
    if c["op"] == "attend":
        q = st["q"]
        if "workspace" not in st:  # a program keeps one for all its calls
            st["workspace"] = torch.empty(fa.fa_fwd_kv4_workspace_size(b, c["heads"], h, n, d), dtype=torch.uint8, device=q.device)
        ws = st["workspace"]
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        fa.fa_fwd_kv4(q, *cache, st["new_lens"], o, lse, b, c["heads"], h, n, *sizes, 1.0 / math.sqrt(d), c["causal"], c["window"],
                      ws, ws.numel())
        return {"o": o, "lse": lse}
    if c["op"] == "write":
        fa.fa_kv4_append(st["k"], st["v"], *cache, st["new_lens"], b, h, n, *sizes)
    k = torch.empty((b, h, n, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    fa.fa_kv4_read(*cache, st["first"], k, v, b, h, n, *sizes)
    return {"k": k, "v": v}


def _append(st):
    c = st["case"]
    n = torch.arange(c["queries"], device="cuda")
    pos = (st["key_lens"] - st["new_lens"])[:, None] + n
    seq, tok = ((n < st["new_lens"][:, None]) & (pos >= 0)).nonzero(as_tuple=True)
    at = pos[seq, tok].long()
    page, off = st["table"][seq, at // c["page"]].long(), at % c["page"]
    for t in ("k", "v"):
        codes, scales = _quantise(st[t])
        st[t + "_codes"][page, :, off] = codes[seq, :, tok]
        st[t + "_scales"][page, :, off] = scales[seq, :, tok]


def _read(st, t):
    c = st["case"]
    pos = st["first"][:, None].long() + torch.arange(c["queries"], device="cuda")
    there = (pos >= 0) & (pos < st["key_lens"][:, None])
    pos = torch.where(there, pos, torch.zeros_like(pos))
    page, off = st["table"].gather(1, pos // c["page"]).long(), pos % c["page"]
    x = _values(st[t + "_codes"][page, :, off], st[t + "_scales"][page, :, off])  # [batch, count, kv_heads, dim]
    x = torch.where(there[:, :, None, None], x, torch.zeros_like(x))
    return x.transpose(1, 2).to(torch.bfloat16).contiguous()


def _whole(st, t):
    """Every sequence's keys or values, [batch, kv_heads, positions, dim] in 32 bits."""
    at = st["table"].long()
    x = _values(st[t + "_codes"][at], st[t + "_scales"][at])  # [batch, pages, kv_heads, page, dim]
    return x.transpose(1, 2).flatten(2, 3)


def _seen(st, positions, kind):
    """[batch, queries, positions]: whether a query sees a position."""
    c = st["case"]
    kl, ql = (st[x][:, None, None].to(kind) for x in ("key_lens", "new_lens"))
    i = torch.arange(c["queries"], device="cuda", dtype=kind)[None, :, None]
    j = torch.arange(positions, device="cuda", dtype=kind)[None, None, :]
    at = kl - ql + i
    seen = (j < kl) & (i < ql)
    if c["causal"]:
        seen = seen & (j <= at)
    if c["window"] >= 0:
        seen = seen & (j >= at - c["window"])
    return seen


def _attend(st):
    c = st["case"]
    b, h, d, n = c["batch"], c["kv_heads"], c["dim"], c["queries"]
    k, v = _whole(st, "k"), _whole(st, "v")
    seen = _seen(st, k.shape[2], torch.int32)[:, None, None]
    q = st["q"].float().view(b, h, c["heads"] // h * n, d)
    s = (torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))).view(b, h, c["heads"] // h, n, -1)
    s = torch.where(seen, s, torch.full((), -math.inf, device="cuda"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h, -1, p.shape[-1]), v).view(b, h, c["heads"] // h, n, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (torch.log(total) + m)[..., 0]
    return {"o": o.view(b, c["heads"], n, d).to(torch.bfloat16), "lse": lse.view(b, c["heads"], n)}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attend":
        return _attend(state)
    if op == "write":
        _append(state)
    return {"k": _read(state, "k"), "v": _read(state, "v")}


def work(case):
    """What a pass cannot do without: new tokens or queries in, the visible part of the cache once, results out."""
    kl, ql = _lengths(case)
    d, h, hq, n = case["dim"], case["kv_heads"], case["heads"], case["queries"]
    row = 2 * h * (d // 2 + d // 16)  # a token's keys and values in the cache
    if case["op"] != "attend":
        spans = [min(n, k) for k in kl] if case["op"] == "read" else ql
        dense = 2 * case["batch"] * h * n * d * 2  # what is given back
        if case["op"] == "read":
            return {"bytes": sum(spans) * row + dense, "flops": 2 * sum(spans) * h * d * 2}
        # the write reads the new tokens and fills their rows; the read back takes them from there
        return {"bytes": sum(spans) * (2 * h * d * 2 + 2 * row) + dense, "flops": 8 * sum(spans) * h * d * 2}
    moved, pairs = 0, 0
    for k, q in zip(kl, ql):
        first, w = k - q, case["window"]
        low = max(0, first - w) if w >= 0 else 0
        moved += (k - low) * row
        for_each = [(first + i + 1 if case["causal"] else k) - (max(0, first + i - w) if w >= 0 else 0) for i in range(q)]
        pairs += sum(max(0, x) for x in for_each)
    moved += case["batch"] * hq * n * (d * 4 + 4)
    return {"bytes": moved, "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _exact_rows(x):
    """bf16 [..., dim] to the values their quantised groups stand for."""
    g = x.double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    top = g.abs().amax(-1, keepdim=True)
    m = torch.where((g == top).any(-1, keepdim=True), top, -top)
    step = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 7)  # |m| / 8 is 16 to 32 of these
    s = -torch.round(m / 8 / step) * step
    return torch.where(top < SMALLEST, torch.zeros_like(g), torch.round(g / s).clamp(-8, 7) * s).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    kl, ql = st["key_lens"].tolist(), st["new_lens"].tolist()
    b, h, d, n, page = case["batch"], case["kv_heads"], case["dim"], case["queries"], case["page"]
    if case["op"] == "write":
        out = {}
        for t in ("k", "v"):
            x = _exact_rows(st[t])
            for i, q in enumerate(ql):
                x[i, :, q:] = 0.0
            out[t] = x
        return out

    def sequence(t, i, low, high):
        """Positions [low, high) of sequence i: [kv_heads, high - low, dim] in 64 bits."""
        at = st["table"][i, low // page: -(-high // page)].long()
        byte = st[t + "_codes"][at].long()
        value = torch.empty((*byte.shape[:-1], d), dtype=torch.float64, device=byte.device)
        value[..., 0::2] = (byte % 16 - 8).double()
        value[..., 1::2] = (byte // 16 - 8).double()
        value *= st[t + "_scales"][at].double().repeat_interleave(GROUP, dim=-1)
        value = value.permute(1, 0, 2, 3).reshape(h, -1, d)
        return value[:, low % page: low % page + high - low]

    if case["op"] == "read":
        out = {t: torch.zeros((b, h, n, d), dtype=torch.float64, device="cuda") for t in "kv"}
        for t in "kv":
            for i, k in enumerate(kl):
                out[t][i, :, :min(n, k)] = sequence(t, i, 0, min(n, k))
        return out
    hq, group = case["heads"], case["heads"] // h
    o = torch.zeros((b, hq, n, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq, n), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(b):
        k, q = kl[i], ql[i]
        keys, values = sequence("k", i, 0, k), sequence("v", i, 0, k)
        j = torch.arange(k, device="cuda")
        at = torch.arange(k - q, k, device="cuda")[:, None]
        hidden = torch.zeros((q, k), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > at
        if case["window"] >= 0:
            hidden |= j < at - case["window"]
        for head in range(hq):
            s = st["q"][i, head, :q].double() @ keys[head // group].T / math.sqrt(d)
            s.masked_fill_(hidden, -math.inf)
            lse[i, head, :q] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[i, head, :q, None]).masked_fill(hidden, 0.0)  # a query that sees nothing: zeros
            o[i, head, :q] = p @ values[head // group]
    return {"o": o, "lse": lse}
