"""The definitions of the paged-cache operators in 64 bits, and their bars.

Every function works on CPU copies in float64 and follows include/oss.h's
formulas token by token; nothing here calls the library.

Bars. u = finfo(type).eps / 2 is one rounding to the inputs' type, U32 = 2^-24
one to fp32. The inputs are exact.

* Scores. s = scale * q.k sums D exact products in fp32: off by at most
  e_s = 2 D U32 scale sum_d |q_d k_d| (factor 2: any order and rounding mode).
  In base 2 the exponent is formed once more and subtracted from the maximum:
  4 U32 (|s| + max |s|) more, and 2^x itself is off by 2^-21. Together each
  weight exp(s - m) is off by a relative
      e_w = exp(2 e) - 1 ~ 2 e,  e = e_s + 4 U32 * 2 max |s| + 2^-21.
* lse: the sum of n such weights in fp32, n U32 relative at worst, the
  logarithm and its scaling 4 U32 (|lse| + 1):  e + n U32 + 4 U32 (|lse| + 2) + 2^-21.
* o = sum p_j v_j / l per element: rounding of o, u |o|; of each p_j, u A with
  A = sum p_j |v_j| / l; the sum over n keys, 2 n U32 A; the weights, 2 e_w A.
  An fp16 p_j below its smallest normal is off by 2^-25 of the largest weight:
  n 2^-25 max |v| more; and o likewise, 2^-25.
* summed weights: sum over the group of p (e_w + the lse's bar); G positive terms
  added in fp32 in any order round G - 1 times to at most the total, (G - 1) U32
  total; the addition to the old value rounds once more, U32 |new value|.
"""

import numpy as np
import torch

U32 = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def attend(q, k, v, seen, scale, u, f16):
    """One head: q [n, D], k, v [m, D], seen [n, m] bool. Returns o, lse, p
    and their bars (p's is relative)."""
    n, m = seen.shape
    D = q.shape[1]
    scale = float(np.float32(scale))
    o = np.zeros((n, D))
    lse = np.full(n, -np.inf)
    p = np.zeros((n, m))
    if m == 0 or n == 0:
        return o, lse, p, np.zeros((n, D)) , np.zeros(n), np.zeros(n)
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    mag = np.where(seen, scale * (np.abs(q) @ np.abs(k).T), 0.0).max(1)
    top = s.max(1)
    live = np.isfinite(top)
    safe = np.where(live, top, 0.0)
    w = np.exp(s - safe[:, None])
    l = w.sum(1)
    p = w / np.where(live, l, 1.0)[:, None]
    lse = np.where(live, safe + np.log(np.where(live, l, 1.0)), -np.inf)
    o = p @ v
    A = p @ np.abs(v)
    big = np.where(seen, np.abs(np.where(seen, s, 0.0)), 0.0).max(1)
    e = 2 * D * U32 * mag + 8 * U32 * big + 2.0 ** -21
    e_w = np.expm1(2 * e)
    keys = seen.sum(1)
    e_lse = e + keys * U32 + 4 * U32 * (np.abs(np.where(live, lse, 0.0)) + 2) + 2.0 ** -21
    e_o = u * np.abs(o) + (u + 2 * keys * U32 + 2 * e_w)[:, None] * A * 1.01
    if f16:
        e_o = e_o + (keys * 2.0 ** -25 * np.abs(v).max())[:, None] + 2.0 ** -25
    return o, lse, p, e_o + 1e-30, np.where(live, e_lse, 0.0), e_w + e_lse


def check(got, ref, bar, what):
    got, ref, bar = np.asarray(got, np.float64), np.asarray(ref), np.asarray(bar)
    same = (got == ref) | (np.isneginf(got) & np.isneginf(ref))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - ref) <= bar))
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, first at {at}: "
                             f"{got[at]} against {ref[at]}, bar {np.broadcast_to(bar, ref.shape)[at]}")


def check_packed(o, lse, q, k, v, lens_q, lens_k, scale, causal, at_q=0, at_k=0):
    """Every row of a packed forward; at_q, at_k: the first sequence's first rows."""
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    oh, lh, qh, kh, vh = (f64(t) for t in (o, lse, q, k, v))
    group = qh.shape[1] // kh.shape[1]
    for b, (n, m) in enumerate(zip(lens_q, lens_k)):
        i, j = np.arange(n)[:, None], np.arange(m)[None]
        seen = (j <= i + m - n) if causal else np.ones((n, m), bool)
        seen = np.broadcast_to(seen, (n, m))
        for h in range(qh.shape[1]):
            g = h // group
            ro, rl, _, bo, bl, _ = attend(qh[at_q:at_q + n, h], kh[at_k:at_k + m, g], vh[at_k:at_k + m, g],
                                          seen, scale, u, f16)
            check(lh[at_q:at_q + n, h], rl, bl, f"sequence {b} head {h} lse")
            check(oh[at_q:at_q + n, h], ro, bo, f"sequence {b} head {h} o")
        at_q, at_k = at_q + n, at_k + m


def gather(pages, table, n, g):
    """The first n rows of key head g of one sequence: [n, D] float64."""
    size = pages.shape[2]
    t = torch.arange(n)
    page = table.cpu().long()[t // size]
    return f64(pages[page.to(pages.device), g, (t % size).to(pages.device)])


def check_decode(o, lse, q, k_pages, v_pages, table, kv_len, scale, weights=None, before=None):
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    oh, lh, qh = f64(o), f64(lse), f64(q)
    heads = k_pages.shape[1]
    group = qh.shape[1] // heads
    for b, n in enumerate(int(x) for x in kv_len.cpu()):
        for g in range(heads):
            k, v = gather(k_pages, table[b], n, g), gather(v_pages, table[b], n, g)
            total, bar = np.zeros(n), np.zeros(n)
            for h in range(g * group, (g + 1) * group):
                ro, rl, p, bo, bl, ep = attend(qh[b, h:h + 1], k, v, np.ones((1, n), bool), scale, u, f16)
                check(lh[b, h:h + 1], rl, bl, f"sequence {b} head {h} lse")
                check(oh[b, h:h + 1], ro, bo, f"sequence {b} head {h} o")
                if n:
                    total += p[0]
                    bar += p[0] * ep[0]
            if weights is not None:
                was = f64(before[b, g])
                ref = was[:n] + total
                got = f64(weights[b, g])
                check(got[:n], ref, bar + U32 * (np.abs(ref) + group * total) + 2.0 ** -126, f"sequence {b} key head {g} weights")
                assert np.array_equal(got[n:], was[n:], equal_nan=True), "weights behind the sequence"


def evict(weights, n, budget, recent):
    """The kept positions of one (sequence, key head): weights [>= n] float32."""
    keep = min(n, budget)
    recent = min(recent, keep)
    w = weights[:n - recent].astype(np.float64)
    w = np.where(np.isnan(w), np.inf, w)
    nan = np.isnan(weights[:n - recent])
    order = np.lexsort((np.arange(n - recent), -w, ~nan))
    return np.sort(np.concatenate([order[:keep - recent], np.arange(n - recent, n)])).astype(np.int64)
