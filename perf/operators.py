"""The serving operators of a paged key-value cache: their cases, plain forms and 64-bit values.

Four operators are run one pass at a time: ``append`` (new keys and values into the pages of a
cache), ``prompt`` (attention over packed sequences), ``decode`` (attention of one new token over
the paged cache, which may add up the weights each cached token received) and ``evict`` (keeping
the cached tokens with the most weight). With ``own`` false, ``run`` is elementary torch; with
``own`` true it makes the calls of ``pass_attention_gb300``.
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one user's chat a few hundred tokens in: a single decode step, latency only
        {"name": "decode_one_short", "op": "decode", "batch": 1, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 16, "min_len": 333, "max_len": 333, "weights": False, "dtype": "bf16"},
        # a serving batch in full flow: every sequence at a length of its own
        {"name": "decode_batch", "op": "decode", "batch": 64, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 64, "min_len": 1, "max_len": 8192, "weights": False, "dtype": "bf16"},
        # long documents, a key head for every query head, small heads in half precision
        {"name": "decode_long_f16", "op": "decode", "batch": 6, "q_heads": 16, "kv_heads": 16,
         "head_dim": 64, "page": 128, "min_len": 20001, "max_len": 32768, "weights": False, "dtype": "f16"},
        # decode steps between evictions: the weights of the cached tokens are added up
        {"name": "decode_weights", "op": "decode", "batch": 16, "q_heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 32, "min_len": 500, "max_len": 9000, "weights": True, "dtype": "bf16"},
        # many short prompts in one launch, from one token up
        {"name": "prompt_short", "op": "prompt", "batch": 48, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "min_len": 1, "max_len": 96, "prefix": 0, "causal": True, "dtype": "bf16"},
        # an ordinary batch of prompts
        {"name": "prompt_batch", "op": "prompt", "batch": 8, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "min_len": 77, "max_len": 2500, "prefix": 0, "causal": True, "dtype": "bf16"},
        # one long document
        {"name": "prompt_long", "op": "prompt", "batch": 1, "q_heads": 32, "kv_heads": 8, "head_dim": 128,
         "min_len": 16384, "max_len": 16384, "prefix": 0, "causal": True, "dtype": "bf16"},
        # the next pieces of prompts whose beginnings are done: more keys than queries
        {"name": "prompt_piece_f16", "op": "prompt", "batch": 4, "q_heads": 16, "kv_heads": 2, "head_dim": 64,
         "min_len": 300, "max_len": 1001, "prefix": 5000, "causal": True, "dtype": "f16"},
        # one new token of each sequence of a batch
        {"name": "append_step", "op": "append", "batch": 64, "kv_heads": 8, "head_dim": 128, "page": 16,
         "min_len": 1, "max_len": 700, "new": 1, "dtype": "bf16"},
        # whole prompts, of uneven lengths, into their pages
        {"name": "append_prompts", "op": "append", "batch": 12, "kv_heads": 8, "head_dim": 128, "page": 64,
         "min_len": 33, "max_len": 5000, "new": 0, "dtype": "bf16"},
        # a batch of caches cut to a quarter, some of them still short enough to stay whole
        {"name": "evict_batch", "op": "evict", "batch": 8, "kv_heads": 8, "head_dim": 128, "page": 32,
         "min_len": 1000, "max_len": 8192, "budget": 2048, "recent": 128, "dtype": "bf16"},
        # two very long caches cut to an eighth
        {"name": "evict_long", "op": "evict", "batch": 2, "kv_heads": 8, "head_dim": 128, "page": 64,
         "min_len": 100001, "max_len": 131072, "budget": 16384, "recent": 1000, "dtype": "bf16"},
    ]


def _log_between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "prompt", "prompt", "append", "evict"))
    c = {"op": op, "head_dim": rng.choice((64, 128, 128)), "dtype": rng.choice(("bf16", "bf16", "f16"))}
    if op in ("decode", "prompt"):
        c["kv_heads"] = rng.choice((1, 2, 4, 5, 8, 16))
        c["q_heads"] = c["kv_heads"] * rng.choice([g for g in (1, 2, 3, 4, 6, 7, 8, 12, 16) if g * c["kv_heads"] <= 64])
    else:
        c["kv_heads"] = rng.choice((1, 2, 4, 5, 8, 16))
    c["batch"] = _log_between(rng, 1, 64)
    if op == "prompt":
        # padded scores of all heads stay within those of the longest listed prompt
        most = 2 ** 28 * 32 // (c["q_heads"] * c["batch"])
        c["max_len"] = _log_between(rng, 1, max(1, min(8192, math.isqrt(most) // 2)))
        c["prefix"] = rng.choice((0, 0, _log_between(rng, 1, max(1, min(8192, most // (2 * c["max_len"]) - c["max_len"])))))
        c["causal"] = rng.random() < 0.8
    else:
        c["page"] = rng.choice((16, 32, 64, 128, 256))
        rows = 2 ** 21 // (c["batch"] * c["kv_heads"])
        c["max_len"] = _log_between(rng, 1, max(1, min(65536 if op in ("decode", "evict") else 8192, rows)))
        if op == "decode":
            c["weights"] = rng.random() < 0.3
        elif op == "append":
            c["new"] = rng.choice((0, 1, 1, _log_between(rng, 1, c["max_len"])))
        else:
            c["budget"] = _log_between(rng, 1, c["max_len"])
            c["recent"] = rng.randrange(0, c["budget"] + 1)
    c["min_len"] = _log_between(rng, 1, c["max_len"])
    return c


def _lengths(case):
    """The case's sequence lengths: the longest first, the others spread over the range."""
    r = random.Random("%d %d %d" % (case["batch"], case["min_len"], case["max_len"]))
    return [case["max_len"]] + [r.randint(case["min_len"], case["max_len"]) for _ in range(case["batch"] - 1)]


def _key_lengths(case):
    """Keys of each packed prompt: its own and those of its prefix."""
    r = random.Random("prefix %d %d" % (case["batch"], case["prefix"]))
    return [n + (r.randint(case["prefix"] // 2, case["prefix"]) if case["prefix"] else 0) for n in _lengths(case)]


def _new_tokens(case):
    """Tokens each sequence appends: all of them for new = 0."""
    return [n if case["new"] == 0 else min(n, case["new"]) for n in _lengths(case)]


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(gen, lengths, page, first, pages):
    """Page tables over the pool's pages in random order, from number `first` of that order; -1 behind a sequence's last page."""
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    need = [-(-n // page) for n in lengths]
    column = torch.arange(max(max(need), 1), device="cuda")[None]
    start = torch.tensor(_starts(need)[:-1], device="cuda")[:, None] + first
    used = column < torch.tensor(need, device="cuda")[:, None]
    return torch.where(used, order[(start + column).clamp(max=pages - 1)], torch.full_like(order[:1], -1)).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dtype, d, heads = _DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"]
    lengths = _lengths(case)
    s = {"op": case["op"]}
    if case["op"] == "prompt":
        keys = _key_lengths(case)
        s["q"] = _randn(gen, (sum(lengths), case["q_heads"], d), dtype)
        s["k"] = _randn(gen, (sum(keys), heads, d), dtype)
        s["v"] = _randn(gen, (sum(keys), heads, d), dtype)
        s["cu_q"], s["cu_k"] = _ints(_starts(lengths)), _ints(_starts(keys))
        s["max_q"], s["max_k"], s["causal"] = max(lengths), max(keys), case["causal"]
        return s
    page = case["page"]
    used = sum(-(-n // page) for n in lengths)
    if case["op"] == "evict":
        kept = [min(n, case["budget"]) for n in lengths]
        # the pages that the kept tokens move to have room for more of them
        room = [case["budget"]] * len(lengths)
        pages = used + sum(-(-n // page) for n in room)
        state = gen.get_state()
        s["table"] = _table(gen, lengths, page, 0, pages)
        gen.set_state(state)
        s["new_table"] = _table(gen, room, page, used, pages)
        s["budget"], s["recent"], s["max_kept"] = case["budget"], case["recent"], max(kept)
        weights = _randn(gen, (len(lengths), heads, s["table"].shape[1] * page), torch.float32)
        s["weights"] = weights.mul_(2.0).exp_()
    else:
        pages = used
        s["table"] = _table(gen, lengths, page, 0, pages)
    s["kv_len"] = _ints(lengths)
    s["k_pages"] = _randn(gen, (pages, heads, page, d), dtype)
    s["v_pages"] = _randn(gen, (pages, heads, page, d), dtype)
    if case["op"] == "decode":
        s["q"] = _randn(gen, (len(lengths), case["q_heads"], d), dtype)
        s["weights"] = None
        if case["weights"]:
            s["weights"] = _randn(gen, (len(lengths), heads, s["table"].shape[1] * page), torch.float32).exp_()
    if case["op"] == "append":
        new = _new_tokens(case)
        s["k"] = _randn(gen, (sum(new), heads, d), dtype)
        s["v"] = _randn(gen, (sum(new), heads, d), dtype)
        s["cu_new"] = _ints(_starts(new))
    return s


def run(state):
    s = state
    if s["op"] == "decode":
        return _decode_own(s) if own else _decode_plain(s)
    if s["op"] == "prompt":
        return _prompt_own(s) if own else _prompt_plain(s)
    if s["op"] == "append":
        return _append_own(s) if own else _append_plain(s)
    return _evict_own(s) if own else _evict_plain(s)


# -- the framework's calls ------------------------------------------------------------------

def _decode_own(s):
    import pass_attention_gb300 as oss
    o, lse = oss.attention_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"],
                                        weights=s["weights"])
    return {"o": o, "lse": lse} if s["weights"] is None else {"o": o, "lse": lse, "weights": s["weights"]}


def _prompt_own(s):
    import pass_attention_gb300 as oss
    o, lse = oss.attention_fwd_packed(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"])
    return {"o": o, "lse": lse}


def _append_own(s):
    import pass_attention_gb300 as oss
    oss.kv_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_len"], s["cu_new"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _evict_own(s):
    import pass_attention_gb300 as oss
    kept, new_len, new_weights = oss.kv_cache_evict(s["k_pages"], s["v_pages"], s["weights"], s["table"],
                                                    s["kv_len"], s["new_table"], s["budget"], s["recent"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "kept": kept, "new_len": new_len,
            "new_weights": new_weights}


# -- the plain forms ------------------------------------------------------------------------

def _decode_plain(s):
    q, table, kv_len = s["q"], s["table"].long(), s["kv_len"]
    pages, heads, page, d = s["k_pages"].shape
    b, h, _ = q.shape
    n = table.shape[1] * page
    # the cache of each sequence in one piece: [B, Hkv, n, D]
    k = s["k_pages"][table].transpose(1, 2).reshape(b, heads, n, d).float()
    v = s["v_pages"][table].transpose(1, 2).reshape(b, heads, n, d).float()
    qf = q.float().reshape(b, heads, h // heads, d)
    scores = (qf @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    hidden = torch.arange(n, device=q.device)[None, :] >= kv_len[:, None]
    hidden = hidden[:, None, None, :]
    scores = scores.masked_fill(hidden, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    p = p / total
    o = (p @ v).reshape(b, h, d).to(q.dtype)
    lse = (m + torch.log(total)).reshape(b, h)
    if s["weights"] is None:
        return {"o": o, "lse": lse}
    s["weights"] += p.sum(2)
    return {"o": o, "lse": lse, "weights": s["weights"]}


def _padded(x, cu, most):
    """The sequences of x [T, H, D] side by side: [B, H, most, D] in 32 bits, zeros behind each."""
    at = cu[:-1, None].long() + torch.arange(most, device=x.device)
    there = at < cu[1:, None]
    y = x[torch.where(there, at, 0)].float()
    return y.masked_fill_(~there[:, :, None, None], 0.0).permute(0, 2, 1, 3)


def _prompt_plain(s):
    q, k, v, cu_q, cu_k = s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"]
    tokens, h, d = q.shape
    heads = k.shape[1]
    b, mq, mk = cu_q.numel() - 1, s["max_q"], s["max_k"]
    qp = _padded(q, cu_q, mq).reshape(b, heads, (h // heads) * mq, d)
    kp, vp = _padded(k, cu_k, mk), _padded(v, cu_k, mk)
    scores = (qp @ kp.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).reshape(b, h, mq, mk)
    n_q, n_k = cu_q.diff()[:, None], cu_k.diff()[:, None]
    last = (n_k - 1).expand(b, mq)  # the last key that a query sees
    if s["causal"]:
        last = torch.arange(mq, device=q.device)[None, :] + (n_k - n_q)
    hidden = torch.arange(mk, device=q.device)[None, None, :] > last[:, :, None]
    scores.masked_fill_(hidden[:, None], -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(b, heads, (h // heads) * mq, mk) @ vp).reshape(b, h, mq, d) / total
    lse = (m + torch.log(total))[..., 0]
    # back to packed tokens: token t is number t - cu_q[sequence] of its sequence
    token = torch.arange(tokens, device=q.device)
    seq = (token[:, None] >= cu_q[None, 1:]).sum(1)
    pos = token - cu_q[seq]
    return {"o": o[seq, :, pos].to(q.dtype), "lse": lse[seq, :, pos]}


def _append_plain(s):
    k, cu, table, page = s["k"], s["cu_new"], s["table"], s["k_pages"].shape[2]
    token = torch.arange(k.shape[0], device=k.device)
    seq = (token[:, None] >= cu[None, 1:]).sum(1)
    # the new tokens are the last ones of their sequences
    pos = s["kv_len"][seq] - cu[seq + 1] + token
    where = table[seq, pos // page].long()
    s["k_pages"][where, :, pos % page] = k
    s["v_pages"][where, :, pos % page] = s["v"]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _evict_plain(s):
    weights, kv_len, budget = s["weights"], s["kv_len"], s["budget"]
    k_pages, v_pages = s["k_pages"], s["v_pages"]
    heads, page = k_pages.shape[1:3]
    b, _, n = weights.shape
    keep = kv_len.clamp(max=budget)
    recent = keep.clamp(max=s["recent"])
    slot = torch.arange(n, device=weights.device)
    older = slot[None, :] < (kv_len - recent)[:, None]
    newest = (slot[None, :] < kv_len[:, None]) & ~older
    # rank 0: the largest weight among the older tokens, the lowest slot among equal ones
    order = weights.masked_fill(~older[:, None], -1.0).sort(dim=-1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order))
    chosen = ((rank < (keep - recent)[:, None, None]) & older[:, None]) | newest[:, None]
    kept = torch.where(chosen, slot, n).sort(dim=-1)[0]
    kept = torch.nn.functional.pad(kept, (0, max(0, budget - n)), value=n)[:, :, :budget]
    there = kept < n
    kept = torch.where(there, kept, 0)
    # rows from the pages of the old table into those of the new one
    new = torch.arange(budget, device=weights.device)
    head = torch.arange(heads, device=weights.device)[None, :, None]
    src = s["table"].long()[:, None].expand(b, heads, -1).gather(2, kept // page)
    dst = s["new_table"].long()[:, new // page][:, None]
    for_pages = (dst, head, (new % page)[None, None])
    k_pages[for_pages] = torch.where(there[..., None], k_pages[src, head, kept % page], k_pages[for_pages])
    v_pages[for_pages] = torch.where(there[..., None], v_pages[src, head, kept % page], v_pages[for_pages])
    new_weights = torch.zeros((b, heads, s["new_table"].shape[1] * page), device=weights.device)
    new_weights[:, :, :budget] = torch.where(there, weights.gather(2, kept), 0.0)
    return {"k_pages": k_pages, "v_pages": v_pages, "kept": torch.where(there, kept, -1).to(torch.int32),
            "new_len": keep.to(torch.int32), "new_weights": new_weights}


# -- what a pass cannot do without ----------------------------------------------------------

def work(case):
    d, heads, lengths = case["head_dim"], case["kv_heads"], _lengths(case)
    row = heads * d * 2 * 2  # K and V of one token, 16 bits each
    if case["op"] == "prompt":
        h, tokens = case["q_heads"], sum(lengths)
        pairs = sum(n * (n + 1) // 2 + n * (k - n) if case["causal"] else n * k
                    for n, k in zip(lengths, _key_lengths(case)))
        return {"bytes": tokens * h * (2 * d * 2 + 4) + sum(_key_lengths(case)) * row, "flops": 4 * pairs * h * d}
    if case["op"] == "decode":
        h, total = case["q_heads"], sum(lengths)
        return {"bytes": total * row + len(lengths) * h * (2 * d * 2 + 4) + (8 * total * heads if case["weights"] else 0),
                "flops": 4 * total * h * d}
    if case["op"] == "append":
        return {"bytes": 2 * sum(_new_tokens(case)) * row, "flops": 0}
    kept = sum(min(n, case["budget"]) for n in lengths)
    room = case["batch"] * -(-case["budget"] // case["page"]) * case["page"]
    return {"bytes": 2 * kept * row + 4 * heads * (sum(lengths) + case["batch"] * case["budget"] + room), "flops": 0}


# -- the definitions in 64 bits -------------------------------------------------------------

def _one_exact(q, k, v, seen):
    """One head: q [n, D], k, v [m, D] in 64 bits, seen [n, m]. Returns o, lse and the weights."""
    x = torch.where(seen, torch.einsum("nd,md->nm", q, k) / math.sqrt(q.shape[1]), -math.inf)
    lse = torch.logsumexp(x, 1)
    w = torch.where(seen, torch.exp(x - lse[:, None]), 0.0)
    return torch.einsum("nm,md->nd", w, v), lse, w


def _exact_decode(case, s):
    b, h, d = s["q"].shape
    heads, page = s["k_pages"].shape[1:3]
    o = torch.zeros((b, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, h), -math.inf, dtype=torch.float64, device="cuda")
    weights = None if s["weights"] is None else s["weights"].double()
    for i, n in enumerate(_lengths(case)):
        t = torch.arange(n, device="cuda")
        at = s["table"][i, torch.div(t, page, rounding_mode="floor")].long()
        k = s["k_pages"][at, :, t % page].double()
        v = s["v_pages"][at, :, t % page].double()
        for j in range(h):
            g = j // (h // heads)
            seen = torch.ones((1, n), dtype=torch.bool, device="cuda")
            oo, ll, w = _one_exact(s["q"][i, j:j + 1].double(), k[:, g], v[:, g], seen)
            o[i, j], lse[i, j] = oo[0], ll[0]
            if weights is not None:
                weights[i, g, :n] += w[0]
    return {"o": o, "lse": lse} if weights is None else {"o": o, "lse": lse, "weights": weights}


def _exact_prompt(case, s):
    h, heads = case["q_heads"], case["kv_heads"]
    o, lse = [], []
    at_q = at_k = 0
    for n, m in zip(_lengths(case), _key_lengths(case)):
        i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")[None]
        seen = (j - m <= i - n) if case["causal"] else (j >= 0).expand(n, m)
        rows = [_one_exact(s["q"][at_q:at_q + n, x].double(), s["k"][at_k:at_k + m, x * heads // h].double(),
                           s["v"][at_k:at_k + m, x * heads // h].double(), seen)[:2] for x in range(h)]
        o.append(torch.stack([r[0] for r in rows], 1))
        lse.append(torch.stack([r[1] for r in rows], 1))
        at_q, at_k = at_q + n, at_k + m
    return {"o": torch.cat(o), "lse": torch.cat(lse)}


def _exact_append(case, s):
    k_pages, v_pages, page, at = s["k_pages"], s["v_pages"], case["page"], 0
    for i, (n, new) in enumerate(zip(_lengths(case), _new_tokens(case))):
        t = torch.arange(n - new, n, device="cuda")
        where = s["table"][i][torch.div(t, page, rounding_mode="floor")].long()
        k_pages[where, :, t % page] = s["k"][at:at + new]
        v_pages[where, :, t % page] = s["v"][at:at + new]
        at += new
    return {"k_pages": k_pages, "v_pages": v_pages}


def _exact_evict(case, s):
    page, budget, heads = case["page"], case["budget"], case["kv_heads"]
    k_pages, v_pages = s["k_pages"], s["v_pages"]
    kept = torch.full((case["batch"], heads, budget), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros((case["batch"], heads, s["new_table"].shape[1] * page), dtype=torch.float64, device="cuda")
    for i, n in enumerate(_lengths(case)):
        keep = min(n, budget)
        recent = min(keep, case["recent"])
        for g in range(heads):
            w = s["weights"][i, g, :n].double()
            by_weight = torch.argsort(-w[:n - recent], stable=True)[:keep - recent]
            slots = torch.cat([by_weight, torch.arange(n - recent, n, device="cuda")]).sort()[0]
            to = torch.arange(keep, device="cuda")
            new = s["new_table"][i][torch.div(to, page, rounding_mode="floor")].long()
            old = s["table"][i][torch.div(slots, page, rounding_mode="floor")].long()
            k_pages[new, g, to % page] = k_pages[old, g, slots % page]
            v_pages[new, g, to % page] = v_pages[old, g, slots % page]
            kept[i, g, :keep] = slots.to(torch.int32)
            weights[i, g, :keep] = w[slots]
    return {"k_pages": k_pages, "v_pages": v_pages, "kept": kept, "new_len": s["kv_len"].clamp(max=budget),
            "new_weights": weights}


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "prompt": _exact_prompt, "append": _exact_append,
            "evict": _exact_evict}[case["op"]](case, s)
