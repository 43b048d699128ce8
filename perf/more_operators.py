"""Serving operators of a cache in 8 bits and of prefixes that sequences share: cases, plain forms, 64-bit values.

Four operators are run one pass at a time: ``append`` (new keys and values quantised into the pages
of a cache: e4m3 values, one power-of-two scale for each token and key head), ``read`` (cached tokens
back to packed 16-bit rows), ``decode`` (attention of one new token per sequence over that cache) and
``shared`` (attention of one new token per sequence over a 16-bit cache in which groups of
sequences share the pages of a long prefix). With ``own`` false, ``run`` is elementary torch; with
``own`` true it makes the calls of ``pass_attention_gb300``.
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_E4M3_MAX = 448.0


def listed():
    return [
        # one user's chat a few hundred tokens in: a single decode step, latency only
        {"name": "decode_one", "op": "decode", "batch": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "page": 16, "min_len": 777, "max_len": 777, "dtype": "bf16"},
        # a serving batch in full flow: every sequence at a length of its own
        {"name": "decode_batch", "op": "decode", "batch": 64, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "page": 64, "min_len": 1, "max_len": 8192, "dtype": "bf16"},
        # long documents, a key head for every query head, small heads in half precision
        {"name": "decode_long_f16", "op": "decode", "batch": 6, "q_heads": 16, "kv_heads": 16, "head_dim": 64,
         "page": 128, "min_len": 20001, "max_len": 32768, "dtype": "f16"},
        # one new token of each sequence of a batch
        {"name": "append_step", "op": "append", "batch": 64, "kv_heads": 8, "head_dim": 128, "page": 16,
         "min_len": 1, "max_len": 700, "new": 1, "dtype": "bf16"},
        # whole prompts, of uneven lengths, into their pages
        {"name": "append_prompts", "op": "append", "batch": 12, "kv_heads": 8, "head_dim": 128, "page": 64,
         "min_len": 33, "max_len": 5000, "new": 0, "dtype": "bf16"},
        # the cached beginning of one prompt, before its next piece is attended to
        {"name": "read_one_f16", "op": "read", "batch": 1, "kv_heads": 2, "head_dim": 64, "page": 16,
         "min_len": 1001, "max_len": 1001, "dtype": "f16"},
        # the cached beginnings of a batch of prompts
        {"name": "read_prompts", "op": "read", "batch": 12, "kv_heads": 8, "head_dim": 128, "page": 64,
         "min_len": 33, "max_len": 5000, "dtype": "bf16"},
        # a few chats behind one system prompt
        {"name": "shared_few", "op": "shared", "groups": 1, "batch": 4, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 16, "prefix": 1000, "min_len": 1, "max_len": 77, "dtype": "bf16"},
        # a serving batch behind one long system prompt
        {"name": "shared_batch", "op": "shared", "groups": 1, "batch": 64, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 64, "prefix": 8192, "min_len": 1, "max_len": 1000, "dtype": "bf16"},
        # several prompts, each sampled a few times, small heads in half precision
        {"name": "shared_groups_f16", "op": "shared", "groups": 5, "batch": 37, "q_heads": 16, "kv_heads": 2,
         "head_dim": 64, "page": 32, "prefix": 5001, "min_len": 1, "max_len": 333, "dtype": "f16"},
        # many questions about one very long document
        {"name": "shared_long", "op": "shared", "groups": 1, "batch": 64, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 128, "prefix": 65536, "min_len": 16, "max_len": 2500, "dtype": "bf16"},
    ]


def _log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "append", "read", "shared", "shared"))
    c = {"op": op, "head_dim": rng.choice((64, 128, 128)), "dtype": rng.choice(("bf16", "bf16", "f16")),
         "page": rng.choice((16, 32, 64, 128, 256)), "kv_heads": rng.choice((1, 2, 4, 5, 8, 16))}
    c["batch"] = _log_between(rng, 1, 64)
    if op in ("decode", "shared"):
        c["q_heads"] = c["kv_heads"] * rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 12, 16) if g * c["kv_heads"] <= 64])
    if op == "shared":
        c["groups"] = rng.choice((1, 1, _log_between(rng, 1, c["batch"])))
        # the padded scores of all heads, and the prefixes side by side, stay within those of the longest listed one
        most = min(2 ** 27 // (c["groups"] * c["batch"] * c["q_heads"]), 2 ** 19 // (c["groups"] * c["kv_heads"]))
        c["prefix"] = _log_between(rng, 1, max(1, min(65536, most)))
        c["max_len"] = _log_between(rng, 1, max(1, min(4096, 2 ** 20 // (c["batch"] * c["kv_heads"]))))
    else:
        rows = 2 ** 21 // (c["batch"] * c["kv_heads"])
        c["max_len"] = _log_between(rng, 1, max(1, min(65536 if op == "decode" else 8192, rows)))
    if op == "append":
        c["new"] = rng.choice((0, 1, 1, _log_between(rng, 1, c["max_len"])))
    c["min_len"] = _log_between(rng, 1, c["max_len"])
    return c


def _lengths(case):
    """The case's sequence lengths: the longest first, the others spread over the range."""
    r = random.Random("%d %d %d" % (case["batch"], case["min_len"], case["max_len"]))
    return [case["max_len"]] + [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"] - 1)]


def _new_tokens(case):
    """Tokens each sequence appends: all of them for new = 0."""
    return [n if case["new"] == 0 else min(n, case["new"]) for n in _lengths(case)]


def _group_sizes(case):
    """Sequences of each group, at least one."""
    r = random.Random("groups %d %d" % (case["batch"], case["groups"]))
    at = [0] + sorted(r.sample(range(1, case["batch"]), case["groups"] - 1)) + [case["batch"]]
    return [b - a for a, b in zip(at, at[1:])]


def _prefixes(case):
    """Tokens of each group's prefix: the longest first, the others down to half of it."""
    r = random.Random("prefix %d %d" % (case["groups"], case["prefix"]))
    low = (case["prefix"] + 1) // 2
    return [case["prefix"]] + [r.randint(low, case["prefix"]) for _ in range(case["groups"] - 1)]


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(order, lengths, page, first):
    """Page tables over the pool's pages in random order, from number `first` of that order; -1 behind a sequence's last page."""
    need = [-(-n // page) for n in lengths]
    column = torch.arange(max(max(need), 1), device="cuda")[None]
    start = torch.tensor(_starts(need)[:-1], device="cuda")[:, None] + first
    used = column < torch.tensor(need, device="cuda")[:, None]
    return torch.where(used, order[(start + column).clamp(max=order.numel() - 1)], torch.full_like(order[:1], -1)).contiguous()


def _rows(gen, shape, dtype):
    """Keys or values: normal, the rows of different sizes, as projections of real tokens are."""
    x = _randn(gen, shape, torch.float32)
    return x.mul_(_randn(gen, shape[:-1] + (1,), torch.float32).mul_(0.3).exp_()).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype, d, heads, page = _DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"], case["page"]
    lengths = _lengths(case)
    pages = sum(-(-n // page) for n in lengths)
    s = {"op": case["op"], "kv_len": _ints(lengths), "dtype": dtype}
    before = 0
    if case["op"] == "shared":
        prefixes = _prefixes(case)
        before = sum(-(-n // page) for n in prefixes)
        pages += before
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    s["table"] = _table(order, lengths, page, before)
    shape = (pages, heads, page, d)
    if case["op"] == "shared":
        s["prefix_table"], s["prefix_len"] = _table(order, prefixes, page, 0), _ints(prefixes)
        s["cu_groups"], s["largest"] = _ints(_starts(_group_sizes(case))), max(_group_sizes(case))
        s["k_pages"], s["v_pages"] = _rows(gen, shape, dtype), _rows(gen, shape, dtype)
    else:
        for x in ("k", "v"):
            s[x + "_pages"], s[x + "_scales"] = _quantise(_rows(gen, shape, dtype))
    if case["op"] in ("decode", "shared"):
        s["q"] = _randn(gen, (len(lengths), case["q_heads"], d), dtype)
    if case["op"] == "append":
        new = _new_tokens(case)
        s["k"], s["v"] = _rows(gen, (sum(new), heads, d), dtype), _rows(gen, (sum(new), heads, d), dtype)
        s["cu"] = _ints(_starts(new))
    if case["op"] == "read":
        s["cu"], s["tokens"] = _ints(_starts(lengths)), sum(lengths)
    return s


def run(state):
    s = state
    if s["op"] == "decode":
        return _decode_own(s) if own else _decode_plain(s)
    if s["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    if s["op"] == "read":
        return _read_own(s) if own else _read_plain(s)
    return _shared_own(s) if own else _shared_plain(s)


# -- the framework's calls ------------------------------------------------------------------

def _decode_own(s):
    import pass_attention_gb300 as oss
    o, lse = oss.attention_decode_paged_fp8(s["q"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"],
                                            s["table"], s["kv_len"])
    return {"o": o, "lse": lse}


def _append_own(s):
    import pass_attention_gb300 as oss
    oss.kv_cache_append_fp8(s["k"], s["v"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                            s["kv_len"], s["cu"])
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}


def _read_own(s):
    import pass_attention_gb300 as oss
    k, v = oss.kv_cache_read_fp8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"], s["kv_len"],
                                 s["cu"], s["tokens"], s["dtype"])
    return {"k": k, "v": v}


def _shared_own(s):
    import pass_attention_gb300 as oss
    o, lse = oss.attention_decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"],
                                         s["table"], s["kv_len"], s["cu_groups"])
    return {"o": o, "lse": lse}


# -- the plain forms ------------------------------------------------------------------------

def _quantise(x):
    """Codes [..., D] in e4m3 and scales [...] in e8m0: the smallest power of two with which a row's values are at most 448."""
    y = x.float()
    largest = y.abs().amax(-1)
    # largest = part * 2^e with part in [0.5, 1), and 448 = 0.875 * 2^9
    part, e = torch.frexp(largest)
    e = torch.where(largest > 0, e - 9 + (part > 0.875).int(), -127).clamp(min=-127)
    down = ((127 - e) << 23).view(torch.float32)  # 2^-e
    codes = (y * down[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _values(codes, scales, at):
    """The values of the rows that the index `at` picks, in 32 bits."""
    c = codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    return c * scales.view(torch.uint8)[at].view(torch.float8_e8m0fnu).float()[..., None]


def _places(cu, kv_len, table, page, tokens):
    """Page and slot of packed token t: the tokens are the last ones of their sequences."""
    token = torch.arange(tokens, device=cu.device)
    seq = (token[:, None] >= cu[None, 1:]).sum(1)
    pos = kv_len[seq] - cu[seq + 1] + token
    return table[seq, pos // page].long(), pos % page


def _append_plain(s):
    where, slot = _places(s["cu"], s["kv_len"], s["table"], s["k_pages"].shape[2], s["k"].shape[0])
    for x in ("k", "v"):
        codes, scales = _quantise(s[x])
        s[x + "_pages"].view(torch.uint8)[where, :, slot] = codes.view(torch.uint8)
        s[x + "_scales"].view(torch.uint8)[where, :, slot] = scales.view(torch.uint8)
    return {x: s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}


def _read_plain(s):
    where, slot = _places(s["cu"], s["kv_len"], s["table"], s["k_pages"].shape[2], s["tokens"])
    at = (where, slice(None), slot)
    return {x: _values(s[x + "_pages"], s[x + "_scales"], at).to(s["dtype"]) for x in ("k", "v")}


def _in_one_piece(x):
    """Pages [B, n, Hkv, page, D] as [B, Hkv, n * page, D]."""
    b, n, heads, page, d = x.shape
    return x.transpose(1, 2).reshape(b, heads, n * page, d)


def _scores(q, k, lengths):
    """q [B, H, D] against k [B, Hkv, n, D]: [B, Hkv, G, n], -inf behind the lengths."""
    b, h, d = q.shape
    x = (q.float().reshape(b, k.shape[1], h // k.shape[1], d) @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    hidden = torch.arange(k.shape[2], device=q.device)[None, :] >= lengths[:, None]
    return x.masked_fill_(hidden[:, None, None, :], -math.inf)


def _decode_plain(s):
    q, table = s["q"], s["table"].long()
    k = _in_one_piece(_values(s["k_pages"], s["k_scales"], table))
    v = _in_one_piece(_values(s["v_pages"], s["v_scales"], table))
    # what lies behind a sequence's last token may be anything
    v = v.masked_fill_((torch.arange(v.shape[2], device=q.device) >= s["kv_len"][:, None])[:, None, :, None], 0.0)
    scores = _scores(q, k, s["kv_len"])
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    o = (p @ v) / total
    return {"o": o.reshape(q.shape).to(q.dtype), "lse": (m + torch.log(total)).reshape(q.shape[:2])}


def _shared_plain(s):
    q, cu, most = s["q"], s["cu_groups"], s["largest"]
    b, h, d = q.shape
    heads = s["k_pages"].shape[1]
    groups = cu.numel() - 1
    # the groups' queries side by side: [groups, Hkv, most * G, D]
    at = cu[:-1, None].long() + torch.arange(most, device=q.device)
    qg = q[at.clamp(max=b - 1)].reshape(groups, most, heads, h // heads, d).transpose(1, 2)
    qg = qg.reshape(groups, heads * most * (h // heads), d)
    prefix = s["prefix_table"].long()
    k0, v0 = (_in_one_piece(s[x][prefix]).float() for x in ("k_pages", "v_pages"))
    x0 = _scores(qg, k0, s["prefix_len"])
    m0 = x0.amax(-1, keepdim=True)
    p0 = x0.sub_(m0).exp_()
    l0, o0 = p0.sum(-1, keepdim=True), p0 @ v0
    # back to one row for each sequence: number b - cu[group] of its group
    token = torch.arange(b, device=q.device)
    group = (token[:, None] >= cu[None, 1:]).sum(1)
    row = token - cu[group]
    m0, l0, o0 = (x.reshape(groups, heads, most, h // heads, -1)[group, :, row] for x in (m0, l0, o0))
    table = s["table"].long()
    k1, v1 = (_in_one_piece(s[x][table]).float() for x in ("k_pages", "v_pages"))
    x1 = _scores(q, k1, s["kv_len"])
    m1 = x1.amax(-1, keepdim=True)
    p1 = x1.sub_(m1).exp_()
    l1, o1 = p1.sum(-1, keepdim=True), p1 @ v1
    m = torch.maximum(m0, m1)
    f0, f1 = torch.exp(m0 - m), torch.exp(m1 - m)
    total = l0 * f0 + l1 * f1
    o = (o0 * f0 + o1 * f1) / total
    return {"o": o.reshape(b, h, d).to(q.dtype), "lse": (m + torch.log(total)).reshape(b, h)}


# -- what a pass cannot do without ----------------------------------------------------------

def work(case):
    d, heads, total = case["head_dim"], case["kv_heads"], sum(_lengths(case))
    row16, row8 = heads * d * 2 * 2, heads * (d + 1) * 2  # K and V of one token
    if case["op"] == "append":
        return {"bytes": sum(_new_tokens(case)) * (row16 + row8), "flops": 0}
    if case["op"] == "read":
        return {"bytes": total * (row16 + row8), "flops": 0}
    h = case["q_heads"]
    ends = case["batch"] * h * (2 * d * 2 + 4)  # q, o and lse
    if case["op"] == "decode":
        return {"bytes": total * row8 + ends, "flops": 4 * total * h * d}
    pairs = total + sum(n * p for n, p in zip(_group_sizes(case), _prefixes(case)))
    return {"bytes": (total + sum(_prefixes(case))) * row16 + ends, "flops": 4 * pairs * h * d}


# -- the definitions in 64 bits -------------------------------------------------------------

def _exact_codes(x):
    """Values on the e4m3 grid and exponents of rows x, by the definition."""
    x = x.double()
    largest = x.abs().amax(-1)
    e = torch.full_like(largest, -127.0)
    guess = torch.log2(largest.clamp(min=1e-300) / _E4M3_MAX).round()
    for up in (1, 0, -1):  # the smallest exponent that is enough
        enough = largest <= _E4M3_MAX * torch.exp2(guess + up)
        e = torch.where(enough & (guess + up > -127), guess + up, e)
    y = x / torch.exp2(e)[..., None]
    # three binary places behind the leading one, down to 2^-6
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.exp2(e)


def _cached(s, i, n, table="table"):
    """K and V [n, Hkv, D] in 64 bits of the first n tokens of row i of a page table."""
    page = s["k_pages"].shape[2]
    t = torch.arange(n, device="cuda")
    at = s[table][i, torch.div(t, page, rounding_mode="floor")].long()
    out = []
    for x in ("k", "v"):
        if s["op"] == "shared":
            out.append(s[x + "_pages"][at, :, t % page].double())
        else:
            code = s[x + "_pages"].view(torch.uint8)[at, :, t % page].view(torch.float8_e4m3fn).double()
            e = s[x + "_scales"].view(torch.uint8)[at, :, t % page].double() - 127
            out.append(code * torch.exp2(e)[..., None])
    return out


def _exact_attention(q, k, v):
    """q [n, H, D] over k, v [m, Hkv, D], all in 64 bits and all seen: o and lse."""
    n, h, d = q.shape
    o, lse = torch.empty_like(q), torch.empty((n, h), dtype=torch.float64, device=q.device)
    for j in range(h):
        g = j * k.shape[1] // h
        x = torch.einsum("nd,md->nm", q[:, j], k[:, g]) / math.sqrt(d)
        lse[:, j] = torch.logsumexp(x, 1)
        o[:, j] = torch.einsum("nm,md->nd", torch.exp(x - lse[:, j:j + 1]), v[:, g])
    return o, lse


def _exact_decode(case, s):
    parts = [_exact_attention(s["q"][i:i + 1].double(), *_cached(s, i, n)) for i, n in enumerate(_lengths(case))]
    return {"o": torch.cat([p[0] for p in parts]), "lse": torch.cat([p[1] for p in parts])}


def _exact_shared(case, s):
    lengths, o, lse, b = _lengths(case), [], [], 0
    for g, (size, n) in enumerate(zip(_group_sizes(case), _prefixes(case))):
        k0, v0 = _cached(s, g, n, "prefix_table")
        for i in range(b, b + size):
            k1, v1 = _cached(s, i, lengths[i])
            oo, ll = _exact_attention(s["q"][i:i + 1].double(), torch.cat([k0, k1]), torch.cat([v0, v1]))
            o.append(oo)
            lse.append(ll)
        b += size
    return {"o": torch.cat(o), "lse": torch.cat(lse)}


def _exact_append(case, s):
    page, out = case["page"], {}
    for x in ("k", "v"):
        pages, scales = s[x + "_pages"].double(), torch.exp2(s[x + "_scales"].view(torch.uint8).double() - 127)
        at = 0
        for i, (n, new) in enumerate(zip(_lengths(case), _new_tokens(case))):
            t = torch.arange(n - new, n, device="cuda")
            where = s["table"][i][torch.div(t, page, rounding_mode="floor")].long()
            codes, scale = _exact_codes(s[x][at:at + new])
            pages[where, :, t % page] = codes
            scales[where, :, t % page] = scale
            at += new
        out[x + "_pages"], out[x + "_scales"] = pages, scales
    return out


def _exact_read(case, s):
    parts = [_cached(s, i, n) for i, n in enumerate(_lengths(case))]
    return {"k": torch.cat([p[0] for p in parts]), "v": torch.cat([p[1] for p in parts])}


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "read": _exact_read, "shared": _exact_shared}[case["op"]](case, s)
