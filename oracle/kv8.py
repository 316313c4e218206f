"""Oracle of the 8-bit KV cache (fp64, CPU): e4m3 values with one exponent per
(page, kv head).

TEST INFRASTRUCTURE, as oracle/paged_attention.py: one page and one head at a
time, from the definitions, sharing no code with the CUDA path.

An e4m3 byte is sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0 is
subnormal (step 2^-9), 0x7F / 0xFF is NaN, and there is no infinity: the
largest value is 0x7E = 448.  An element of page p and head h stands for
value * 2^exp[p, h], exponents held to [-64, 64].
"""
from __future__ import annotations

import numpy as np

from . import paged_attention as pa

E_MIN, E_MAX = -64, 64
MAX = 448.0


def _decode_table() -> np.ndarray:
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if (b & 0x7F) == 0x7F:
            v = np.nan
        t[b] = -v if b & 0x80 else v
    return t


DECODE = _decode_table()
_POSITIVE = DECODE[:0x7F]          # 0 .. 448, ascending with the byte


def decode(b) -> np.ndarray:
    return DECODE[np.asarray(b, np.uint8)]


def encode(x) -> np.ndarray:
    """Bytes of the nearest e4m3 values, ties to the even byte, held to +-448;
    NaN gives 0x7F."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=np.inf)), MAX)
    hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    b = np.where(take_lo, lo, hi).astype(np.uint8)
    b = b | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), b).astype(np.uint8)


def need_exp(x) -> int:
    """The smallest e in [-64, 64] with max |finite x| <= 448 * 2^e."""
    x = np.asarray(x, np.float64)
    a = np.abs(x[np.isfinite(x)])
    m = float(a.max()) if a.size else 0.0
    for e in range(E_MIN, E_MAX):
        if m <= MAX * 2.0 ** e:
            return e
    return E_MAX


def _held(e) -> int:
    return int(np.clip(int(e), E_MIN, E_MAX))


def append(k_cache, v_cache, k_exp, v_exp, k_new, v_new, q_len, context_len, block_table,
           page_size=16):
    """(k, v, k_exp, v_exp) after the append: caches uint8 [pages, P, Hkv, D],
    exponents int8 [pages, Hkv], new rows bf16 bits or floats [T, Hkv, D]."""
    out = [np.array(a) for a in (k_cache, v_cache, k_exp, v_exp)]
    new = [pa._as_f64(k_new), pa._as_f64(v_new)]
    cu = pa._cu(q_len)
    for s, (n, c) in enumerate(zip(q_len, context_len)):
        n, c = int(n), int(c)
        pos = c - n
        while pos < c:
            page, slot = int(block_table[s][pos // page_size]), pos % page_size
            m = min(page_size - slot, c - pos)
            tok = int(cu[s]) + pos - (c - n)
            for pool, exp, x in ((out[0], out[2], new[0]), (out[1], out[3], new[1])):
                for h in range(pool.shape[2]):
                    xs = x[tok:tok + m, h]
                    e = need_exp(xs)
                    if slot:
                        old = _held(exp[page, h])
                        e = max(e, old)
                        if e > old:
                            pool[page, :slot, h] = encode(decode(pool[page, :slot, h]) * 2.0 ** (old - e))
                    exp[page, h] = e
                    pool[page, slot:slot + m, h] = encode(
                        np.where(np.isfinite(xs), xs, np.nan) * 2.0 ** -e)
            pos += m
    return tuple(out)


def values(cache, exp) -> np.ndarray:
    """The numbers a cache stands for, [pages, P, Hkv, D]."""
    e = np.clip(np.asarray(exp).astype(np.int64), E_MIN, E_MAX)
    return decode(cache) * (2.0 ** e.astype(np.float64))[:, None, :, None]


def attention(q, k_cache, v_cache, k_exp, v_exp, q_len, context_len, block_table, page_size,
              num_q_heads, num_kv_heads, scale, tokens=None, window=0):
    """paged_attention.attention over the numbers the cache stands for."""
    return pa.attention(pa._as_f64(q), values(k_cache, k_exp), values(v_cache, v_exp), q_len,
                        context_len, block_table, page_size, num_q_heads, num_kv_heads, scale,
                        tokens=tokens, window=window)


def mean_abs(q, k_cache, v_cache, k_exp, v_exp, *args, **kw):
    """The same attention over |V|: sum_t p_t |v_t|, which rounding errors of
    the weights are relative to."""
    return pa.attention(pa._as_f64(q), values(k_cache, k_exp), np.abs(values(v_cache, v_exp)),
                        *args, **kw)
