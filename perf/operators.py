"""The operators of the 8-bit paged KV cache, as cases to measure.

Four operators, run in this order by a serving step:

  assign     block tables, slot maps and prefix sums from request lengths, with
             pages taken from a ring of free pages on the GPU
  append     the step's new K/V rows quantised into their cache pages: e4m3
             values with one power-of-two exponent per (page, kv head)
  attention  decode rows and prefill chunks over that cache
  release    the finished requests' pages back to the ring

`own = False` computes each in elementary torch operations in 32 bits; `own =
True` makes the library's calls.  The lengths of a case's sequences are drawn
from the case's own values, the tensors and page numbers from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
E_MIN, E_MAX = -64, 64      # exponents that the cache uses
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _attention(name, hq, hkv, d, decode, lo, hi, spread="uniform", median=0, chunks=0, chunk=0, offset=0,
               window=0):
    return {"name": name, "op": "attention", "hq": hq, "hkv": hkv, "d": d, "decode": decode, "lo": lo, "hi": hi,
            "spread": spread, "median": median, "chunks": chunks, "chunk": chunk, "offset": offset,
            "window": window}


def _append(name, hkv, d, decode, lo, hi, chunks=0, chunk=0, offset=0):
    return {"name": name, "op": "append", "hkv": hkv, "d": d, "decode": decode, "lo": lo, "hi": hi,
            "spread": "uniform", "median": 0, "chunks": chunks, "chunk": chunk, "offset": offset}


def _pages(name, op, decode, lo, hi, chunks=0, chunk=0, offset=0):
    return {"name": name, "op": op, "decode": decode, "lo": lo, "hi": hi, "spread": "uniform", "median": 0,
            "chunks": chunks, "chunk": chunk, "offset": offset}


def listed():
    return [
        # the smallest step: a few short decodes and a 64-token chunk, where latency counts
        _attention("attention-tiny", 8, 8, 64, 4, 100, 300, chunks=1, chunk=64, offset=64),
        # budget 512: 64 decodes over chat-length contexts and a ragged piece of a prompt, grouped heads
        _attention("attention-b512", 32, 8, 128, 64, 128, 8192, "lognormal", 2145, 1, 448, 1339),
        # budget 2048: long contexts, a large chunk far into its prompt, group of 7
        _attention("attention-b2048", 56, 8, 128, 32, 1, 16384, "lognormal", 7267, 1, 2016, 6048),
        # decodes only, the cache's largest read
        _attention("attention-decode256", 32, 8, 128, 256, 1024, 8192),
        # several prompts in flight, short chunks under a sliding window
        _attention("attention-window", 16, 2, 128, 37, 200, 6000, chunks=4, chunk=150, offset=2500, window=1024),
        # the append of the smallest step, of a decode-only step and of a large prefill
        _append("append-tiny", 8, 64, 4, 100, 300, 1, 64, 64),
        _append("append-decode256", 8, 128, 256, 1024, 8192),
        _append("append-prefill", 8, 128, 33, 1, 8192, 8, 2021, 1003),
        # pages of a decode-only step and of a burst of prompts
        _pages("assign-decode256", "assign", 256, 1024, 8192),
        _pages("assign-prefill", "assign", 1021, 1, 16384, 32, 4001, 7),
        # a few requests finish; a whole wave of them does
        _pages("release-few", "release", 5, 100, 3000),
        _pages("release-wave", "release", 2047, 1, 16384),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "append", "assign", "release"])
    if op == "attention":
        hq, hkv, d = rng.choice([(8, 8, 64), (32, 8, 128), (56, 8, 128), (16, 2, 128), (16, 1, 64), (32, 16, 128)])
        hi = _log_int(rng, 64, 16384)
        decode = min(_log_int(rng, 1, 200), (1 << 20) // hi)
        chunks = rng.choice([0, 1, 1, 2, 4])
        chunk = min(_log_int(rng, 2, 2016), 2048 // max(1, chunks)) if chunks else 0
        offset = _log_int(rng, 1, 6048) - 1 if chunks else 0
        case = _attention("", hq, hkv, d, decode, max(1, hi // 9), hi, chunks=chunks, chunk=chunk, offset=offset,
                          window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]))
    elif op == "append":
        hkv, d = rng.choice([(8, 64), (8, 128), (2, 128), (1, 64), (16, 128)])
        chunks = rng.choice([0, 1, 3, 8])
        case = _append("", hkv, d, _log_int(rng, 1, 256), 1, _log_int(rng, 16, 8192), chunks,
                       _log_int(rng, 2, 8000) // chunks + 1 if chunks else 0, rng.randrange(0, 1500) if chunks else 0)
    else:
        chunks = rng.choice([0, 1, 8, 32]) if op == "assign" else 0
        case = _pages("", op, _log_int(rng, 1, 2047 if op == "release" else 1000), 1, _log_int(rng, 16, 16384),
                      chunks, _log_int(rng, 2, 4000) if chunks else 0, rng.randrange(0, 200) if chunks else 0)
    del case["name"]
    return case


def _rows(case):
    """(q_len, context_len) of the case's sequences, decodes first, from the case's values alone."""
    r = random.Random("%s %s" % (case["decode"], [case[k] for k in ("lo", "hi", "spread", "median", "chunks", "chunk",
                                                                    "offset")]))
    rows = []
    for _ in range(case["decode"]):
        if case["spread"] == "lognormal":
            n = int(round(case["median"] * math.exp(0.6 * r.gauss(0, 1))))
        else:
            n = r.randint(case["lo"], case["hi"])
        rows.append((1, min(max(n, case["lo"]), case["hi"])))
    for i in range(case["chunks"]):
        off = case["offset"] + 5 * i          # prompts are not in step with one another
        rows.append((case["chunk"], off + case["chunk"]))
    return np.array(rows, np.int64).reshape(-1, 2)


def _pages_of(n):
    return -(-n // PAGE)


# ------------------------------------------------------------------ inputs
def _layout(case, gen, extra=0):
    """Descriptors on the GPU: rows, cu_q_len, context_len and a block table over a permutation of the pool."""
    rows = _rows(case)
    q, ctx = rows[:, 0], rows[:, 1]
    n = _pages_of(ctx)
    used, maxp = int(n.sum()), int(n.max())
    num_pages = used + max(4, used // 10) + extra
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    first = np.concatenate([[0], np.cumsum(n)[:-1]])
    at = torch.from_numpy(first[:, None] + np.arange(maxp)[None, :]).cuda()
    live = torch.from_numpy(np.arange(maxp)[None, :] < n[:, None]).cuda()
    table = torch.where(live, perm[at.clamp_(max=num_pages - 1)], -1).to(torch.int32).contiguous()
    cu = np.concatenate([[0], np.cumsum(q)])
    as32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    return {"q_len_h": q.astype(np.int32), "ctx_h": ctx.astype(np.int32), "q_len": as32(q), "ctx": as32(ctx),
            "cu": as32(cu), "table": table, "num_pages": num_pages, "total_q": int(q.sum()), "used": used}


def _pool(gen, num_pages, hkv, d):
    """A pool of e4m3 values that fill their range, and exponents that put them near a unit deviation."""
    pool = torch.empty(num_pages, PAGE, hkv, d, dtype=torch.float8_e4m3fn, device="cuda")
    step = max(1, (1 << 28) // (PAGE * hkv * d))
    for a in range(0, num_pages, step):
        x = torch.randn(min(step, num_pages - a), PAGE, hkv, d, generator=gen, device="cuda")
        pool[a:a + step] = x.mul_(112.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    exp = torch.randint(-9, -6, (num_pages, hkv), generator=gen, device="cuda", dtype=torch.int8)
    return pool, exp


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    if case["op"] in ("assign", "release"):
        s = _layout(case, gen, extra=64)
        s["op"], n = case["op"], s["num_pages"]
        ring = torch.randperm(n, generator=gen, device="cuda").to(torch.int32)
        head = int(torch.randint(0, n, (1,), generator=gen, device="cuda"))
        s["ring"] = ring
        if case["op"] == "assign":
            # rows stand before the step: no entry yet for the pages that its new tokens open
            fresh = torch.arange(s["table"].shape[1], device="cuda")[None, :] * PAGE >= (s["ctx"] - s["q_len"])[:, None]
            s["table"] = torch.where(fresh, -1, s["table"]).to(torch.int32)
            s["state"] = torch.tensor([head, head + n, 0, 0], device="cuda")
            s["cu_out"] = torch.zeros(len(s["q_len_h"]) + 1, dtype=torch.int32, device="cuda")
            s["slots"] = torch.zeros(s["total_q"], dtype=torch.int64, device="cuda")
        else:
            s["state"] = torch.tensor([head, head + n - s["used"], 0, 0], device="cuda")
        s["state_out"] = torch.zeros_like(s["state"])
        if own:
            from chunked_prefill_decode_gb300 import hb
            s["hb"] = hb
        return s
    s = _layout(case, gen)
    s["op"], hkv, d = case["op"], case["hkv"], case["d"]
    s["k"], s["ke"] = _pool(gen, s["num_pages"], hkv, d)
    s["v"], s["ve"] = _pool(gen, s["num_pages"], hkv, d)
    T = s["total_q"]
    if case["op"] == "append":
        # tokens differ in size, so that some pages outgrow the exponent they had
        size = torch.exp(0.7 * torch.randn(2, T, 1, 1, generator=gen, device="cuda"))
        new = torch.randn(2, T, hkv, d, generator=gen, device="cuda") * size
        s["k_new"], s["v_new"] = new[0].to(torch.bfloat16), new[1].to(torch.bfloat16)
    else:
        s["q"] = torch.randn(T, case["hq"], d, generator=gen, device="cuda").to(torch.bfloat16)
        s["scale"], s["window"], s["decode"] = 1.0 / math.sqrt(d), case["window"], case["decode"]
        # slots behind a sequence's last token were never written
        last = (s["ctx"].long() - 1) // PAGE
        page = s["table"].gather(1, last[:, None])[:, 0].long()
        hole = torch.arange(PAGE, device="cuda")[None, :] > ((s["ctx"].long() - 1) % PAGE)[:, None]
        for pool in (s["k"], s["v"]):
            byte = pool.view(torch.uint8)
            byte[page] = torch.where(hole[:, :, None, None], 0x7F, byte[page])
    if own:
        from chunked_prefill_decode_gb300 import hb
        s["hb"] = hb
        s["batch"] = hb.make_batch(len(s["q_len_h"]), T, s["table"].shape[1], s["num_pages"], case.get("hq", hkv), hkv,
                                   d, s["cu"], s["ctx"], s["table"], sliding_window=case.get("window", 0))
        if case["op"] == "attention":
            sms = torch.cuda.get_device_properties(0).multi_processor_count
            s["plan"], s["ws"] = hb.hb_kv8_plan(s["batch"], s["q_len_h"], s["ctx_h"], sms)
            s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"assign": _plain_assign, "release": _plain_release, "append": _plain_append,
            "attention": _plain_attention}[state["op"]](state)


def _run_own(s):
    hb = s["hb"]
    if s["op"] == "assign":
        hb.hb_pages_assign(s["q_len"], s["ctx"], s["ring"], s["state"], s["state_out"], s["table"], s["cu_out"],
                           s["slots"])
        return {"table": s["table"], "cu": s["cu_out"], "slots": s["slots"], "state": s["state_out"]}
    if s["op"] == "release":
        hb.hb_pages_release(s["ctx"], s["ring"], s["state"], s["state_out"], s["table"])
        return {"ring": s["ring"], "state": s["state_out"]}
    if s["op"] == "append":
        hb.hb_kv8_append(s["batch"], s["k_new"], s["v_new"], s["k"], s["v"], s["ke"], s["ve"])
        return {"k": s["k"], "v": s["v"], "ke": s["ke"], "ve": s["ve"]}
    hb.hb_kv8_attention(s["batch"], s["plan"], s["q"], s["k"], s["v"], s["ke"], s["ve"], s["scale"], s["out"], s["ws"])
    return {"out": s["out"]}


def _plain_assign(s):
    q, ctx, ring, state = s["q_len"].long(), s["ctx"].long(), s["ring"], s["state"]
    off = ctx - q
    first, last = (off + PAGE - 1) // PAGE, (ctx + PAGE - 1) // PAGE
    before = torch.cumsum(last - first, 0) - (last - first)
    cu = torch.cat([q.new_zeros(1), torch.cumsum(q, 0)])
    lp = torch.arange(s["table"].shape[1], device=q.device)[None, :]
    taken = ring[(state[0] + before[:, None] + lp - first[:, None]) % ring.numel()]
    table = torch.where((lp >= first[:, None]) & (lp < last[:, None]), taken, s["table"])
    tok = torch.arange(s["total_q"], device=q.device)
    row = torch.searchsorted(cu[1:], tok, right=True)
    pos = off[row] + tok - cu[row]
    slots = table[row, pos // PAGE].long() * PAGE + pos % PAGE
    head = state[0] + (last - first).sum()
    return {"table": table, "cu": cu.to(torch.int32), "slots": slots,
            "state": torch.stack([head, state[1], 0 * head, 0 * head])}


def _plain_release(s):
    n = (s["ctx"].long() + PAGE - 1) // PAGE
    after = torch.cumsum(n, 0)
    ring, state = s["ring"], s["state"]
    at = (torch.arange(ring.numel(), device=n.device) - state[1]) % ring.numel()
    row = torch.searchsorted(after, at, right=True).clamp(max=n.numel() - 1)
    lp = (at - after[row] + n[row]).clamp(0, s["table"].shape[1] - 1)
    ring = torch.where(at < after[-1], s["table"][row, lp], ring)
    tail = state[1] + after[-1]
    return {"ring": ring, "state": torch.stack([state[0], tail, 0 * tail, 0 * tail])}


def _pow2(e):
    """2^e of whole e, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _need(amax):
    """The smallest e with amax <= 448 * 2^e, within the cache's range."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e.clamp(E_MIN, E_MAX), E_MIN).to(torch.int32)


def _plain_append(s):
    ctx, cu = s["ctx"].long(), s["cu"].long()
    off = ctx - (cu[1:] - cu[:-1])
    tok = torch.arange(s["total_q"], device=ctx.device)
    row = torch.searchsorted(cu[1:], tok, right=True)
    pos = off[row] + tok - cu[row]
    page, slot = s["table"][row, pos // PAGE].long(), pos % PAGE
    opened = off % PAGE > 0                       # sequences whose first new token joins older ones on a page
    page0 = s["table"].gather(1, (off // PAGE).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].clamp(min=0).long()
    older = (torch.arange(PAGE, device=ctx.device)[None, :] < (off % PAGE)[:, None])[:, :, None, None]
    for pool, exp, new in ((s["k"], s["ke"], s["k_new"]), (s["v"], s["ve"], s["v_new"])):
        x = new.float()
        x = torch.where(torch.isfinite(x), x, torch.nan)
        amax = x.abs().nan_to_num(0.0).amax(-1)                                         # [T, Hkv]
        grown = torch.zeros(exp.shape, device=x.device)
        grown.scatter_reduce_(0, page[:, None].expand_as(amax), amax, "amax")
        need = _need(grown)                                                             # [num_pages, Hkv]
        was = exp[page0].int().clamp(E_MIN, E_MAX)
        e0 = torch.where(opened[:, None], torch.maximum(was, need[page0]), need[page0])
        shift = torch.where(opened[:, None], was - e0, 0).clamp(min=-126)
        byte = pool.view(torch.uint8)
        held = _pow2(shift)[:, None, :, None] * byte[page0].view(torch.float8_e4m3fn).float()
        held = torch.where(older, held.to(torch.float8_e4m3fn).view(torch.uint8), byte[page0])
        byte.index_put_((page0,), held)
        exp.index_put_((page,), need[page].to(torch.int8))
        exp.index_put_((page0,), e0.to(torch.int8))
        y = x * _pow2(-exp[page].int())[:, :, None]
        y = y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        byte.index_put_((page, slot), y.view(torch.uint8))
    return {"k": s["k"], "v": s["v"], "ke": s["ke"], "ve": s["ve"]}


def _gathered(pool, exp, table, ctx):
    """K or V of some sequences as [n, L, Hkv, D] in 32 bits, zeros behind their last tokens."""
    at = table.clamp(min=0).long()
    x = pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).float()
    x = x * _pow2(exp[at])[:, :, None, :, None]
    x = x.flatten(1, 2)
    live = torch.arange(x.shape[1], device=x.device)[None, :] < ctx[:, None]
    return torch.where(live[:, :, None, None], x, 0.0)


def _rows_attend(q, k, v, ctx, scale, window):
    """q [n, r, Hq, D], the last r positions of each sequence, over k, v [n, L, Hkv, D]."""
    n, r, hq, d = q.shape
    hkv = k.shape[2]
    q = q.float().view(n, r, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    x = (q * scale) @ k.permute(0, 2, 3, 1)
    pos = ctx[:, None] - r + torch.arange(r, device=q.device)[None, :]
    key = torch.arange(k.shape[1], device=q.device)
    seen = key[None, None, :] <= pos[:, :, None]
    if window:
        seen &= key[None, None, :] > pos[:, :, None] - window
    x = x.view(n, hkv, r, -1, k.shape[1]).masked_fill(~seen[:, None, :, None, :], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = (x / x.sum(-1, keepdim=True)).view(n, hkv, -1, k.shape[1])
    o = x @ v.permute(0, 2, 1, 3)
    return o.view(n, hkv, r, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, r, hq, d)


def _plain_attention(s):
    # the decodes come first, then chunks of one length
    dec, q, ctx = s["decode"], s["q"], s["ctx"].long()
    outs = []
    if dec:
        t = s["table"][:dec, :_pages_of(int(s["ctx_h"][:dec].max()))]
        k, v = (_gathered(s[p], s[p + "e"], t, ctx[:dec]) for p in "kv")
        outs.append(_rows_attend(q[:dec, None], k, v, ctx[:dec], s["scale"], s["window"]).flatten(0, 1))
    if dec < len(s["q_len_h"]):
        t = s["table"][dec:, :_pages_of(int(s["ctx_h"][dec:].max()))]
        k, v = (_gathered(s[p], s[p + "e"], t, ctx[dec:]) for p in "kv")
        qc = q[dec:].view(len(s["q_len_h"]) - dec, -1, *q.shape[1:])
        outs.append(_rows_attend(qc, k, v, ctx[dec:], s["scale"], s["window"]).flatten(0, 1))
    return {"out": torch.cat(outs).to(torch.bfloat16)}


# ------------------------------------------------------------------ work
def work(case):
    rows = _rows(case)
    q, ctx = rows[:, 0], rows[:, 1]
    T, S = int(q.sum()), len(rows)
    if case["op"] == "assign":
        new = int((_pages_of(ctx) - _pages_of(ctx - q)).sum())
        held = int(((ctx - q) % PAGE > 0).sum())
        return {"bytes": 8 * S + 4 * (S + 1) + 8 * new + 4 * held + 8 * T + 64, "flops": 0}
    if case["op"] == "release":
        return {"bytes": 4 * S + 8 * int(_pages_of(ctx).sum()) + 64, "flops": 0}
    if case["op"] == "append":
        touched = int((_pages_of(ctx) - (ctx - q) // PAGE).sum())
        return {"bytes": T * case["hkv"] * case["d"] * 2 * (2 + 1) + 2 * touched * (case["hkv"] + 4), "flops": 0}
    w = case["window"]
    first = np.maximum(0, ctx - q - w + 1) if w else np.zeros_like(ctx)   # first key that any row sees
    pages = int((_pages_of(ctx) - first // PAGE).sum())
    size = int((ctx - first).sum()) * case["hkv"] * case["d"] * 2 + pages * (2 * case["hkv"] + 4)
    seen = 0
    for n, c in rows:
        p = np.arange(c - n, c) + 1
        seen += int((np.minimum(p, w) if w else p).sum())
    return {"bytes": size + 2 * T * case["hq"] * case["d"] * 2, "flops": 4 * case["hq"] * case["d"] * seen}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_pow2(e):
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_round(y):
    """y rounded to the nearest e4m3 value, ties to even, held at the largest one."""
    a = y.abs().clamp(max=E4M3_MAX)
    step = _exact_pow2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.round(a / step) * step * torch.sign(y)


def _exact_append(s):
    out = {}
    table, cu = s["table"].cpu().numpy(), s["cu"].cpu().numpy()
    for p in "kv":
        pool, exp, new = s[p].double(), s[p + "e"].double(), s[p + "_new"].double()
        for i, (n, c) in enumerate(zip(s["q_len_h"], s["ctx_h"])):
            n, c = int(n), int(c)
            at = c - n
            while at < c:
                page, slot = int(table[i, at // PAGE]), at % PAGE
                m = min(PAGE - slot, c - at)
                x = new[cu[i] + at - (c - n):cu[i] + at - (c - n) + m]
                m_abs = x.abs().amax((0, 2))
                e = torch.ceil(torch.log2(m_abs / E4M3_MAX)).clamp(E_MIN, E_MAX)
                e = e + (m_abs > E4M3_MAX * _exact_pow2(e)).double()        # should the logarithm have rounded
                e = e - (m_abs <= E4M3_MAX * _exact_pow2(e - 1)).double()
                e = e.clamp(E_MIN, E_MAX)
                if slot:
                    e = torch.maximum(e, exp[page])
                    pool[page, :slot] = _exact_round(pool[page, :slot] * _exact_pow2(exp[page] - e)[None, :, None])
                exp[page] = e
                pool[page, slot:slot + m] = _exact_round(x * _exact_pow2(-e)[None, :, None])
                at += m
        out[p], out[p + "e"] = pool, exp.to(torch.int8)
    return out


def _exact_attention(s):
    q, table = s["q"].double(), s["table"].long()
    out = torch.empty_like(q)
    hkv = s["k"].shape[2]
    g = q.shape[1] // hkv
    row = 0
    for i, (n, c) in enumerate(zip(s["q_len_h"], s["ctx_h"])):
        n, c = int(n), int(c)
        pages = table[i, :_pages_of(c)]
        k, v = (s[p].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() for p in "kv")
        k = (k * _exact_pow2(s["ke"][pages])[:, None, :, None]).flatten(0, 1)[:c]
        v = (v * _exact_pow2(s["ve"][pages])[:, None, :, None]).flatten(0, 1)[:c]
        pos = torch.arange(c - n, c, device="cuda")[:, None]
        key = torch.arange(c, device="cuda")[None, :]
        hidden = (key > pos) | (key <= pos - s["window"] if s["window"] else key < 0)
        for h in range(q.shape[1]):
            x = q[row:row + n, h] @ k[:, h // g].T * s["scale"]
            out[row:row + n, h] = torch.softmax(x.masked_fill(hidden, -math.inf), -1) @ v[:, h // g]
        row += n
    return {"out": out}


def exact(case, seed):
    if case["op"] in ("assign", "release"):
        return None                     # whole numbers, which are compared as they are
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
