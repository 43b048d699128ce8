"""The definitions of the 8-bit cache and of attention behind shared prefixes in 64
bits, and their bars.

Every function works on CPU copies in float64 and follows include/oss.h's formulas;
nothing here calls the library.

The cache's codes and scales are exact: powers of two divide exactly, and the one
rounding, to e4m3, is to nearest even. So tests compare them bit for bit.

Bars of attention (u = finfo(type).eps / 2, one rounding to o's type; U32 = 2^-24; p = w /
l the weights, A = sum p |v|, n keys):

* Scores: as in paged_reference, 2 D U32 scale sum |q k| for the fp32 sum of exact
  products and 4 U32 (|s| + max |s|) for the exponent's forming. Over the 8-bit
  cache a bf16 q is held in fp16 relative to its head's largest element: elements
  below 2^-29 of it are off by up to 2^-40 of it, scale D 2^-40 max |q| max |k| in all.
* Each ex2 is off by 2^-21 relative. A weight passes through at most five: its own, and
  the factors with which its warp's (or tile's), its part's and its prefix's states
  meet: 5 * 2^-21 on each of w and l.  e = all of these; e_w = exp(2 e) - 1.
* lse: e + n U32 + 4 U32 (|lse| + 2) + 2^-21.
* o: u |o|, the rounding of o; p_round A, the weights' rounding for the product with V
  (u of the inputs' type, or 2^-11 where it runs in fp16); 2 n U32 A for the sums; 2 e_w A; and
  32 U32 A for the joins' multiplications. fp16 weights below the smallest
  normal are off by 2^-25 of a reference at most as large as the largest one, for each of the n
  keys: over 16-bit caches n 2^-25 max |v|. Over the 8-bit cache the reference is max_t p_t 2^ev_t and the
  product's other side a code of at most 448, with 2^ev_t <= amax_t / 224 (or 2^-127): n
  2^-25 448 max_t p_t (amax_t / 224 + 2^-127). An fp16 o below its smallest normal: 2^-25, a bf16 one 2^-133; a
  weight below fp32's smallest normal is flushed: n 2^-126 max |v|.
"""

import numpy as np
import torch

from paged_reference import U32, check, f64

E4M3_MAX = 448.0


def quantise(x):
    """Codes [..., D] and scales [...] (float64) of rows x, by the definition."""
    x = f64(x) if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    e = np.full(top.shape, -127.0)
    fine = ~bad & (top > 0)
    guess = np.floor(np.log2(np.where(fine, top, 1.0))) - 9
    for up in (2, 1, 0):  # the smallest exponent that is enough
        enough = np.where(fine, top, 0.0) <= E4M3_MAX * np.exp2(guess + up)
        e = np.where(fine & enough & (guess + up >= -127), guess + up, e)
    scale = np.where(bad, np.nan, np.exp2(e))
    y = np.where(bad[..., None], np.nan, x / np.exp2(e)[..., None])
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(np.where(np.isfinite(y), y, 0.0)), 2.0 ** -6))) - 3)
    return np.round(y / step) * step, scale


def codes(pages):
    """The e4m3 values of a pool as float64."""
    return pages.detach().float().cpu().double().numpy()


def scales(s):
    """The values of e8m0 scales as float64, formed from their bytes."""
    b = s.detach().view(torch.uint8).cpu().numpy().astype(np.int64)
    return np.where(b == 255, np.nan, np.exp2(b - 127.0))


def gather8(pages, scale, table, n, g):
    """Values of the first n rows of key head g of one sequence: [n, D] float64."""
    size = pages.shape[2]
    t = torch.arange(n)
    page = table.cpu().long()[t // size].to(pages.device)
    slot = (t % size).to(pages.device)
    c = pages.view(torch.uint8)[page, g, slot].view(torch.float8_e4m3fn)
    s = scale.view(torch.uint8)[page, g, slot].view(torch.float8_e8m0fnu)
    return codes(c) * scales(s)[:, None]


def attend_one(q, k, v, scale, u, p_round, f16_out, eight_bit=False, f16_weights=False):
    """One query q [D] over keys and values [n, D]: o, lse and their bars."""
    n, D = k.shape
    scale = float(np.float32(scale))
    if n == 0:
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    s = scale * (k @ q)
    top = s.max()
    w = np.exp(s - top)
    l = w.sum()
    p = w / l
    lse = top + np.log(l)
    o, A = p @ v, p @ np.abs(v)
    e = 2 * D * U32 * scale * (np.abs(k) @ np.abs(q)).max() + 8 * U32 * np.abs(s).max() + 5 * 2.0 ** -21
    if eight_bit:
        e += scale * D * 2.0 ** -40 * np.abs(q).max() * np.abs(k).max()
    e_w = np.expm1(2 * e)
    bar_lse = e + n * U32 + 4 * U32 * (abs(lse) + 2) + 2.0 ** -21
    bar_o = u * np.abs(o) + (p_round + 2 * n * U32 + 2 * e_w + 32 * U32) * A * 1.01
    bar_o = bar_o + n * 2.0 ** -126 * np.abs(v).max() + 2.0 ** -133
    if eight_bit:
        bar_o = bar_o + n * 2.0 ** -25 * 448 * (p * (np.abs(v).max(1) / 224 + 2.0 ** -127)).max()
    elif f16_weights:
        bar_o = bar_o + n * 2.0 ** -25 * np.abs(v).max()
    if f16_out:
        bar_o = bar_o + 2.0 ** -25
    return o, lse, bar_o, bar_lse


def check_decode_fp8(o, lse, q, k_pages, v_pages, k_scales, v_scales, table, kv_len, scale, heads=None):
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    oh, lh, qh = f64(o), f64(lse), f64(q)
    hkv = k_pages.shape[1]
    group = qh.shape[1] // hkv
    for b, n in enumerate(int(x) for x in kv_len.cpu()):
        for g in range(hkv):
            k, v = gather8(k_pages, k_scales, table[b], n, g), gather8(v_pages, v_scales, table[b], n, g)
            for h in range(g * group, (g + 1) * group):
                if heads is not None and h not in heads:
                    continue
                ro, rl, bo, bl = attend_one(qh[b, h], k, v, scale, u, 2.0 ** -11, f16, eight_bit=True)
                check(lh[b, h], rl, bl, f"sequence {b} head {h} lse")
                check(oh[b, h], ro, bo, f"sequence {b} head {h} o")


def check_shared(o, lse, q, keys, values, scale, rows=None):
    """keys(b, g), values(b, g): what sequence b sees in key head g, [n, D] float64."""
    u = torch.finfo(q.dtype).eps / 2
    f16 = q.dtype == torch.float16
    oh, lh, qh = f64(o), f64(lse), f64(q)
    hkv = keys.heads
    group = qh.shape[1] // hkv
    for b in range(qh.shape[0]) if rows is None else rows:
        for g in range(hkv):
            k, v = keys(b, g), values(b, g)
            for h in range(g * group, (g + 1) * group):
                ro, rl, bo, bl = attend_one(qh[b, h], k, v, scale, u, u, f16, f16_weights=f16)
                check(lh[b, h], rl, bl, f"sequence {b} head {h} lse")
                check(oh[b, h], ro, bo, f"sequence {b} head {h} o")
