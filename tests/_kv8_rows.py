"""Bounds of the 8-bit attention taken for every row, head and dimension by
itself: a large value in one page, head or dimension widens the bound of no
other."""
import math

import numpy as np

from _gpu import bits
from oracle import kv8
from oracle import paged_attention as pa


def row_bounds(layout, inp, cache, scale=None):
    """(exact output, how far a right one may be off), both [T, Hq, D], over
    the given cache (numpy: k, v, k_exp, v_exp).

    With p_t the weights (sum 1), o = sum p_t v_t and A = sum p_t |v_t|:
      * the output is rounded to bf16: 2^-8 |o|;
      * a score is a sum of D products in fp32 with three roundings more, its
        exponential good to 2^-22 and twice in the result (numerator and sum):
        e_t = (D + 3) 2^-24 scale sum_d |q_d k_td| + 2^-21 of p_t, so
        sum p_t e_t |v_t| + |o| sum p_t e_t;
      * a weight is rounded once in the products, and the sum may or may not
        hold the rounded ones: w (A + |o|), w = 2^-11 for decode rows (fp16),
        2^-8 for chunk rows (bf16);
      * an fp16 weight has no finer step than 2^-31 of the row's largest (the
        factors that it carries put the largest at 2^7 or more of 2^-24's
        steps): half of that times sum |v_t|;
      * the products are added up in fp32, at most all keys in a row:
        n 2^-23 A.
    Products of these terms are covered by a 2^-6 part more."""
    sh = layout.shape
    scale = 1.0 / math.sqrt(sh.head_dim) if scale is None else scale
    g = sh.num_q_heads // sh.num_kv_heads
    q = pa._as_f64(bits(inp.q))
    ref, tol = np.zeros_like(q), np.zeros_like(q)
    row = 0
    for s in range(layout.num_seqs):
        n, ctx = int(layout.q_len[s]), int(layout.context_len[s])
        if n == 0:
            continue
        w_round = 2.0 ** -11 if n == 1 else 2.0 ** -8
        low = max(0, ctx - n - sh.sliding_window + 1) // 16 if sh.sliding_window else 0
        pages = layout.block_table[s, low:-(-ctx // 16)]
        k = kv8.values(cache[0][pages], cache[2][pages]).reshape(-1, sh.num_kv_heads, sh.head_dim)[:ctx - 16 * low]
        v = kv8.values(cache[1][pages], cache[3][pages]).reshape(-1, sh.num_kv_heads, sh.head_dim)[:ctx - 16 * low]
        pos = np.arange(ctx - n, ctx)[:, None]
        key = np.arange(16 * low, ctx)[None, :]
        seen = (key <= pos) & ((key > pos - sh.sliding_window) if sh.sliding_window else True)
        some = seen.any(0)               # (what no row sees may be NaN)
        k, v, seen = k[some], v[some], seen[:, some]
        for h in range(sh.num_q_heads):
            qh, kh, vh = q[row:row + n, h], k[:, h // g], v[:, h // g]
            x = np.where(seen, scale * (qh @ kh.T), -np.inf)
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            e = (sh.head_dim + 3) * 2.0 ** -24 * scale * (np.abs(qh) @ np.abs(kh).T) + 2.0 ** -21
            o, a = p @ vh, p @ np.abs(vh)
            t = 2.0 ** -8 * np.abs(o) + (p * e) @ np.abs(vh) + np.abs(o) * (p * e).sum(1, keepdims=True)
            t += w_round * (a + np.abs(o)) + kh.shape[0] * 2.0 ** -23 * a
            if n == 1:
                t += 2.0 ** -32 * p.max(1, keepdims=True) * (seen @ np.abs(vh))
            ref[row:row + n, h], tol[row:row + n, h] = o, t * (1 + 2.0 ** -6)
        row += n
    return ref, tol
