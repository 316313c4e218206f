"""Helpers of the 8-bit cache's tests: seeded caches, the append and the
attention through the library, and the oracle's answers with bounds that
follow from the formats."""
import math

import numpy as np
import torch

from _gpu import sms
from _hbutil import lib
from chunked_prefill_decode_gb300 import workloads
from chunked_prefill_decode_gb300.device import from_layout
from oracle import kv8

bits = workloads.bf16_bits
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2     # 2^-8: half a step, relative


class Inputs:
    """q, k_new, v_new (bf16, CPU) and a cache that holds the layout's older
    tokens; every other byte of the pools is NaN (0x7F) and the exponents of
    pages without older tokens are junk."""

    def __init__(self, layout, seed, exps=(-9, -6)):
        sh = layout.shape
        g = torch.Generator().manual_seed(seed)
        T = layout.total_q
        normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q = normal(T, sh.num_q_heads, sh.head_dim).to(torch.bfloat16)
        self.k_new, self.v_new = (normal(T, sh.num_kv_heads, sh.head_dim)
                                  .mul_(torch.exp(0.5 * normal(T, sh.num_kv_heads, 1))).to(torch.bfloat16)
                                  for _ in range(2))
        mask = workloads.cached_slot_mask(layout)
        pool = (layout.num_pages, sh.page_size, sh.num_kv_heads, sh.head_dim)
        self.cache, self.exps = [], []
        held = mask.any(1)
        for _ in range(2):
            b = (normal(*pool) * 112).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            self.cache.append(np.where(mask[:, :, None, None], b, np.uint8(0x7F)))
            e = torch.randint(exps[0], exps[1] + 1, (pool[0], pool[2]), generator=g).numpy()
            self.exps.append(np.where(held[:, None], e, 99).astype(np.int8))

    def device(self, dev="cuda:0"):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        return (*(t(c).view(torch.float8_e4m3fn) for c in self.cache), *(t(e) for e in self.exps))

    def oracle_append(self, layout):
        return kv8.append(*self.cache, *self.exps, bits(self.k_new), bits(self.v_new), layout.q_len,
                          layout.context_len, layout.block_table, layout.shape.page_size)


def as_bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def same_bytes(got, want):
    """e4m3 bytes alike, any NaN being like any other."""
    nan_g, nan_w = (got & 0x7F) == 0x7F, (want & 0x7F) == 0x7F
    return np.array_equal(nan_g, nan_w) and np.array_equal(got[~nan_g], want[~nan_w])


def step(layout, inp, scale=None, repeats=1, check=True, append=True):
    """Append + plan + attention on cuda:0: (cache tensors after, out)."""
    hb = lib()
    scale = 1.0 / math.sqrt(layout.shape.head_dim) if scale is None else scale
    db = from_layout(layout, "cuda:0")
    q, kn, vn = (t.to("cuda:0") for t in (inp.q, inp.k_new, inp.v_new))
    cache = inp.device()
    out = torch.full_like(q, float("nan"))
    if append:
        hb.hb_kv8_append(db.batch, kn, vn, *cache)
    plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
    for _ in range(repeats):
        hb.hb_kv8_attention(db.batch, plan, q, *cache, scale, out, ws)
    if check:
        hb.hb_check()
    torch.cuda.synchronize()
    return cache, out


def bounds(layout, inp, cache, scale=None, tokens=None):
    """(exact output, how far a right one may be off) over the given cache
    (numpy: k, v, k_exp, v_exp).

    The output is rounded to bf16: 2^-8 |o|.  Each weight is rounded once to
    bf16 or finer: 2^-8 of its share, sum_t p_t |v_t| =: A in all, and the sum
    of the weights may or may not hold the rounded ones: 2^-8 |o| more.  A
    score is a sum of D products in fp32 and three roundings more, and its
    exponential is good to 2^-22: (D + 3) 2^-24 (sum_d |q_d k_d|) scale +
    2^-21 relative in each weight, taken twice (numerator and sum).  In fp16 a
    weight has no finer step than 2^-24, against a largest one of 2^7 or more
    (P carries that factor): a key far below the row's maximum is off by up to
    2^-25 / 2^7 = 2^-32 of the largest weight, hence of the sum, so the ctx
    keys of a row by 2^-32 ctx max |v| at most."""
    sh = layout.shape
    scale = 1.0 / math.sqrt(sh.head_dim) if scale is None else scale
    args = (layout.q_len, layout.context_len, layout.block_table, sh.page_size, sh.num_q_heads,
            sh.num_kv_heads, scale)
    kw = dict(tokens=tokens, window=sh.sliding_window)
    qb = bits(inp.q)
    ref = kv8.attention(qb, *cache, *args, **kw)
    a = kv8.mean_abs(qb, *cache, *args, **kw)
    k = np.abs(kv8.values(cache[0], cache[2]))
    k = k[np.isfinite(k)].max() if np.isfinite(k).any() else 0.0
    qmax = np.abs(inp.q.double().numpy()).sum(-1).max()
    score = (sh.head_dim + 3) * 2.0 ** -24 * qmax * k * scale + 2.0 ** -21
    v = np.abs(kv8.values(cache[1], cache[3]))
    v = v[np.isfinite(v)].max() if np.isfinite(v).any() else 0.0
    far = np.repeat(np.asarray(layout.context_len, np.float64), layout.q_len)[:, None, None] * 2.0 ** -32 * v
    return ref, HALF_BF16 * (2 * np.abs(ref) + a) + 2 * score * a + far


def check_out(out, ref, tol, tokens=None):
    got = out.float().cpu().numpy().astype(np.float64)
    if tokens is not None:
        got, ref, tol = got[tokens], ref[tokens], tol[tokens]
    assert np.isfinite(got).all(), "non-finite output"
    err = np.abs(got - ref)
    worst = float((err / tol).max()) if err.size else 0.0
    assert (err <= tol).all(), f"error up to {worst:.2f} of the bound (max-abs {err.max():.3e})"
    return worst
