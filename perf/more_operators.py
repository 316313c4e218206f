"""The operators of a transformer block around the attention step, as cases to
measure.

Three operators, which a block calls between its linear layers and its
attention:

  norm      the norm after a branch, its gate and residual scale, the residual
            sum and the norm before the next branch, over rows of the residual
            stream
  rope      rotary positions of q and k (after head norms where the model has
            them), with k and v put into their cache pages
  adapters  low-rank adapters of many requests beside a shared projection

`own = False` computes each in elementary torch operations in 32 bits (angles
in 64); `own = True` makes the library's calls.  The lengths, adapters and ranks
of a case are drawn from the case's own values, the tensors from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
EPS = 1e-5


# ------------------------------------------------------------------ cases
def _norm(name, rows, width, form, gate="none", residual=1.0, branch=1.0, fp32=False, offset=0.0, spare=0):
    """form: first (the stream's first norm), add (residual sum, norm), both (norm, gate, scaled sum, norm),
    last (norm, gate, scaled sum).  spare: elements between rows that belong to something else."""
    return {"name": name, "op": "norm", "rows": rows, "width": width, "form": form, "gate": gate,
            "residual": residual, "branch": branch, "fp32": fp32, "offset": offset, "spare": spare}


def _rope(name, hq, hkv, d, decode, lo, hi, chunks=0, chunk=0, offset=0, rot=0, interleaved=False, headnorm=False,
          scaling="none", by=1.0, base=10000.0, fused=False, k_out=True):
    return {"name": name, "op": "rope", "hq": hq, "hkv": hkv, "d": d, "decode": decode, "lo": lo, "hi": hi,
            "chunks": chunks, "chunk": chunk, "offset": offset, "rot": rot or d, "interleaved": interleaved,
            "headnorm": headnorm, "scaling": scaling, "by": by, "base": base, "fused": fused, "k_out": k_out}


def _adapters(name, k, n0, n1, n2, decode, chunks, chunk, adapters, max_rank, low_rank, none=0.0):
    """none: the share of sequences without an adapter."""
    return {"name": name, "op": "adapters", "k": k, "n0": n0, "n1": n1, "n2": n2, "decode": decode,
            "chunks": chunks, "chunk": chunk, "adapters": adapters, "max_rank": max_rank, "low_rank": low_rank,
            "none": none}


def listed():
    return [
        # one token of a long model: latency alone
        _norm("norm-token", 1, 7168, "add"),
        # budget 512: the sum and the norm between attention and MLP
        _norm("norm-b512", 512, 4096, "add"),
        # budget 2048: norms on both sides, a gate per channel, a stream in 32 bits
        _norm("norm-b2048-both", 2048, 7168, "both", "channel", 0.9, 0.7, fp32=True),
        # an unchunked prompt, gates per token, branch and gates inside wider tensors
        _norm("norm-prompt-gated", 8191, 4096, "both", "row", 1.0, 0.5, offset=1.0, spare=1024),
        # the smallest step: a few short decodes and a 64-token chunk
        _rope("rope-tiny", 8, 8, 64, 4, 100, 300, 1, 64, 64),
        # budget 512: 64 decodes over chat-length contexts and a piece of a prompt, q, k and v in one tensor
        _rope("rope-b512", 32, 8, 128, 64, 128, 8192, 1, 448, 1339, fused=True, k_out=False, base=1e6),
        # budget 2048: a large chunk, head norms, half of each head rotated in neighbouring pairs
        _rope("rope-b2048-norms", 56, 8, 128, 32, 1, 16384, 1, 2016, 6048, rot=64, interleaved=True, headnorm=True),
        # prompts far into long contexts, frequencies scaled by parts
        _rope("rope-long", 32, 8, 128, 37, 9000, 1 << 20, 8, 2021, 120001, scaling="parts", by=16.0, base=5e5),
        # 64 decodes that share 48 adapters beside a fused QKV projection
        _adapters("adapters-decode64", 4096, 4096, 1024, 1024, 64, 0, 0, 48, 16, 16),
        # a few decodes and a 64-token chunk beside an output projection
        _adapters("adapters-few", 512, 512, 0, 0, 4, 1, 64, 3, 8, 8),
        # budget 512: decodes and a chunk beside the down projection, ranks that differ, some without an adapter
        _adapters("adapters-b512-down", 14336, 4096, 0, 0, 64, 1, 448, 33, 64, 8, none=0.2),
        # budget 2048 and more: prompts of several adapters beside a wide QKV projection
        _adapters("adapters-prompts", 7168, 7168, 1024, 1024, 61, 5, 1201, 20, 64, 16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "adapters"])
    if op == "norm":
        form = rng.choice(["first", "add", "add", "both", "last"])
        width = 8 * _log_int(rng, 16, 1536)
        rows = min(_log_int(rng, 1, 12000), (1 << 25) // width)
        scaled = form in ("both", "last")
        case = _norm("", rows, width, form, rng.choice(["none", "channel", "row"]) if scaled else "none",
                     rng.choice([1.0, 0.8]) if scaled else 1.0, rng.choice([1.0, 0.3]) if scaled else 1.0,
                     rng.choice([False, False, True]), rng.choice([0.0, 1.0]), rng.choice([0, 0, 8, 4096]))
    elif op == "rope":
        hq, hkv, d = rng.choice([(8, 8, 64), (32, 8, 128), (56, 8, 128), (16, 2, 128), (16, 1, 64), (32, 16, 128)])
        chunks = rng.choice([0, 1, 1, 3, 8])
        case = _rope("", hq, hkv, d, _log_int(rng, 1, 256), 1, _log_int(rng, 16, 1 << 20), chunks,
                     _log_int(rng, 2, 8000) // chunks + 1 if chunks else 0, rng.randrange(0, 100000) if chunks else 0,
                     rng.choice([d, d, d // 2, d // 4]), rng.choice([False, False, True]),
                     rng.choice([False, False, True]), rng.choice(["none", "none", "linear", "base", "parts"]),
                     rng.choice([2.0, 8.0, 32.0]), rng.choice([1e4, 5e5, 1e6]), rng.choice([False, True]),
                     rng.choice([False, True]))
    else:
        k, n = rng.choice([(4096, (4096, 1024, 1024)), (4096, (4096, 0, 0)), (7168, (7168, 1024, 1024)),
                           (14336, (4096, 0, 0)), (512, (512, 256, 256)), (1000, (776, 0, 0))])
        chunks = rng.choice([0, 0, 1, 3])
        max_rank = rng.choice([8, 16, 16, 32, 64, 128])
        tokens = min(_log_int(rng, 2, 4000), 200000 // max_rank)
        case = _adapters("", k, *n, _log_int(rng, 1, 256), chunks, tokens // chunks + 1 if chunks else 0,
                         _log_int(rng, 1, 64), max_rank,
                         rng.choice([max_rank, max(1, max_rank // 3), 1]), rng.choice([0.0, 0.0, 0.3]))
    del case["name"]
    return case


def _cases_own(case):
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _rows(case):
    """(q_len, context_len) of the case's sequences, decodes first, from the case's values alone."""
    r = _cases_own(case)
    rows = [(1, r.randint(case["lo"], case["hi"])) for _ in range(case["decode"])]
    for i in range(case["chunks"]):
        off = case["offset"] + 5 * i          # prompts are not in step with one another
        rows.append((case["chunk"], off + case["chunk"]))
    return np.array(rows, np.int64).reshape(-1, 2)


def _ranks(case):
    """(q_len, adapter of each sequence or -1, rank of each adapter)."""
    r = _cases_own(case)
    q = [1] * case["decode"] + [case["chunk"]] * case["chunks"]
    of = [-1 if r.random() < case["none"] else r.randrange(case["adapters"]) for _ in q]
    rank = [r.randint(case["low_rank"], case["max_rank"]) for _ in range(case["adapters"])]
    return np.array(q, np.int64), np.array(of, np.int64), np.array(rank, np.int64)


def _cols(case):
    return [n for n in (case["n0"], case["n1"], case["n2"]) if n]


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape, dtype=torch.bfloat16, size=1.0):
    return torch.randn(*shape, generator=gen, device="cuda").mul_(size).to(dtype)


def _as32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    s = {"norm": _prepare_norm, "rope": _prepare_rope, "adapters": _prepare_adapters}[case["op"]](case, gen)
    s["case"] = case
    return s


def _prepare_norm(case, gen):
    rows, width, form = case["rows"], case["width"], case["form"]
    dtype = torch.float32 if case["fp32"] else torch.bfloat16

    def wide(dtype=torch.bfloat16, size=1.0):
        return _normal(gen, rows, width + case["spare"], dtype=dtype, size=size)[:, :width]

    def weight():
        return (1.0 - case["offset"] + 0.2 * torch.randn(width, generator=gen, device="cuda")).to(torch.bfloat16)
    # the stream of a deep model is larger than a branch, and its rows differ
    s = {"x": torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda")) * 4}
    s["x"] = (s["x"] * wide(torch.float32)).to(dtype)
    s["y"] = wide(size=0.7) if form != "first" else None
    s["w_post"] = weight() if form in ("both", "last") else None
    s["w_pre"] = weight() if form != "last" else None
    s["gate"] = None
    if case["gate"] == "channel":
        s["gate"] = _normal(gen, 1, width, size=0.5)
    elif case["gate"] == "row":
        s["gate"] = wide(size=0.5)
    s["x_out"] = torch.empty(rows, width, dtype=dtype, device="cuda") if form != "first" else None
    s["z"] = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda") if form != "last" else None
    if own:
        from chunked_prefill_decode_gb300 import hb
        s["hb"] = hb
    return s


def _pages_of(n):
    return -(-n // PAGE)


def _prepare_rope(case, gen):
    rows = _rows(case)
    q, ctx = rows[:, 0], rows[:, 1]
    hq, hkv, d, T = case["hq"], case["hkv"], case["d"], int(q.sum())
    # the pages that the step writes are its own; entries before them are pages that the call does not touch
    first, last = (ctx - q) // PAGE, _pages_of(ctx)
    n = last - first
    used, maxp = int(n.sum()), int(last.max())
    num_pages = used + used // 8 + 8
    perm = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    start = torch.from_numpy(np.cumsum(n) - n).cuda()[:, None]
    lp = torch.arange(maxp, device="cuda")[None, :]
    first, last = torch.from_numpy(first).cuda()[:, None], torch.from_numpy(last).cuda()[:, None]
    mine = (lp >= first) & (lp < last)
    table = torch.where(mine, perm[(start + lp - first).clamp(0, num_pages - 1)], perm[used])
    s = {"table": torch.where(lp < last, table, -1).to(torch.int32).contiguous(), "num_pages": num_pages,
         "cu": _as32(np.concatenate([[0], np.cumsum(q)])), "ctx": _as32(ctx)}
    if case["fused"]:
        qkv = _normal(gen, T, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        s["q"], s["k"], s["v"] = _normal(gen, T, hq, d), _normal(gen, T, hkv, d), _normal(gen, T, hkv, d)
    s["q_weight"] = s["k_weight"] = None
    if case["headnorm"]:
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(torch.bfloat16)
                                        for _ in range(2))
    s["factor"] = 0.1 * math.log(case["by"]) + 1 if case["scaling"] == "parts" else 1.0
    s["k_cache"], s["v_cache"] = (_normal(gen, num_pages, PAGE, hkv, d) for _ in range(2))
    s["q_out"] = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.empty(T, hkv, d, dtype=torch.bfloat16, device="cuda") if case["k_out"] else None
    if own:
        from chunked_prefill_decode_gb300 import hb
        s["hb"] = hb
        s["batch"] = hb.make_batch(len(rows), T, maxp, num_pages, hq, hkv, d, s["cu"], s["ctx"], s["table"])
        s["rope"] = hb.make_rope(case["rot"], case["base"], scaling=case["scaling"], scale_by=case["by"],
                                 original_context=8192, parts=(1.0, 32.0), interleaved=case["interleaved"],
                                 factor=s["factor"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    return s


def _prepare_adapters(case, gen):
    q, of, rank = _ranks(case)
    cols, k, n, r = _cols(case), case["k"], case["adapters"], case["max_rank"]
    T = int(q.sum())
    live = torch.arange(r, device="cuda")[None, :] < torch.from_numpy(rank).cuda()[:, None]
    a = _normal(gen, n, len(cols), r, k, size=1 / math.sqrt(k))
    b = _normal(gen, n, sum(cols), r, size=1 / math.sqrt(r))
    # ranks that an adapter does not have hold nothing that may be used
    a.masked_fill_(~live[:, None, :, None], math.nan)
    b.masked_fill_(~live[:, None, :], math.nan)
    s = {"a": a, "b": b, "rank": _as32(rank), "rank_h": rank, "cols": cols, "q_len_h": q, "of_h": of,
         "scale": torch.rand(n, generator=gen, device="cuda") * 1.5 + 0.5, "x": _normal(gen, T, k),
         "y": [_normal(gen, T, c) for c in cols]}
    s["out"] = [torch.empty_like(y) for y in s["y"]]
    if own:
        from chunked_prefill_decode_gb300 import hb
        s["hb"] = hb
        s["pool"] = hb.make_adapters(a, b, s["rank"], s["scale"], cols)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        s["plan"], s["ws"] = hb.hb_adapters_plan(s["pool"], q, of, sms)
    else:
        # the tokens of each adapter
        token = np.repeat(of, q)
        s["tokens"] = {i: torch.from_numpy(np.flatnonzero(token == i)).cuda() for i in np.unique(token) if i >= 0}
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return {"norm": _own_norm, "rope": _own_rope, "adapters": _own_adapters}[state["case"]["op"]](state)
    return {"norm": _plain_norm, "rope": _plain_rope, "adapters": _plain_adapters}[state["case"]["op"]](state)


def _given(**outs):
    return {k: v for k, v in outs.items() if v is not None}


def _own_norm(s):
    c = s["case"]
    s["hb"].hb_norm(x=s["x"], y=s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"], x_out=s["x_out"],
                    z=s["z"], eps=EPS, residual_scale=c["residual"], branch_scale=c["branch"],
                    weight_offset=c["offset"])
    return _given(x=s["x_out"], z=s["z"])


def _own_rope(s):
    s["hb"].hb_rope(s["batch"], s["rope"], s["q"], s["k"], s["v"], s["q_out"], s["k_out"], s["k_cache"],
                    s["v_cache"])
    return _given(q=s["q_out"], k=s["k_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_adapters(s):
    s["hb"].hb_adapters(s["pool"], s["plan"], s["x"], s["y"], s["out"], s["ws"])
    return {"out": s["out"]}


def _rms(x, w, offset):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * (offset + w.float())


def _plain_norm(s):
    c = s["case"]
    x, z = s["x"].float(), None
    if s["y"] is not None:
        u = s["y"].float()
        if s["w_post"] is not None:
            u = _rms(u, s["w_post"], c["offset"])
        if s["gate"] is not None:
            u = u * s["gate"].float()
        x = x * c["residual"] + u * c["branch"]
    if s["w_pre"] is not None:
        z = _rms(x, s["w_pre"], c["offset"]).to(torch.bfloat16)
    return _given(x=x.to(s["x"].dtype) if s["y"] is not None else None, z=z)


def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    rot, by = case["rot"], case["by"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    base = case["base"] * (by ** (rot / (rot - 2)) if case["scaling"] == "base" else 1.0)
    f = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        f = f / by
    elif case["scaling"] == "parts":
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * (keep + (1 - keep) / by)
    return f


def _places(s):
    """Of each new token: its position, its page and its slot."""
    cu, ctx = s["cu"].long(), s["ctx"].long()
    tok = torch.arange(s["q"].shape[0], device=cu.device)
    row = torch.searchsorted(cu[1:], tok, right=True)
    pos = ctx[row] - cu[row + 1] + tok
    return pos, s["table"][row, pos // PAGE].long(), pos % PAGE


def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    pos, page, slot = _places(s)
    angle = pos.double()[:, None, None] * _frequencies(c)
    cos, sin = (f(angle).float() * s["factor"] for f in (torch.cos, torch.sin))

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = _rms(x, w, 0.0)
        y = x.clone()
        if c["interleaved"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
        return y.to(torch.bfloat16)
    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    s["k_cache"][page, slot] = k
    s["v_cache"][page, slot] = s["v"]
    return _given(q=q, k=k if c["k_out"] else None, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_adapters(s):
    outs = [y.clone() for y in s["y"]]
    for i, tok in s["tokens"].items():
        r = int(s["rank_h"][i])
        x, first = s["x"][tok].float(), 0
        for j, n in enumerate(s["cols"]):
            h = x @ s["a"][i, j, :r].float().T
            delta = h @ s["b"][i, first:first + n, :r].float().T
            outs[j][tok] = (s["y"][j][tok].float() + s["scale"][i] * delta).to(torch.bfloat16)
            first += n
    return {"out": outs}


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "norm":
        form, n = case["form"], case["rows"] * case["width"]
        wide = 4 if case["fp32"] else 2
        size = wide * n                                                  # x
        size += (2 + wide) * n if form != "first" else 0                 # y, the new stream
        size += 2 * n if form != "last" else 0                           # z
        size += 2 * {"none": 0, "channel": case["width"], "row": n}[case["gate"]]
        size += 2 * case["width"] * {"first": 1, "add": 1, "both": 2, "last": 1}[form]
        return {"bytes": size, "flops": {"first": 4, "add": 6, "both": 12, "last": 8}[form] * n}
    if case["op"] == "rope":
        rows = _rows(case)
        T, S, d = int(rows[:, 0].sum()), len(rows), case["d"]
        pages = int((_pages_of(rows[:, 1]) - (rows[:, 1] - rows[:, 0]) // PAGE).sum())
        vectors = 2 * case["hq"] + (4 + case["k_out"]) * case["hkv"]     # read or written, of a token
        flops = (case["hq"] + case["hkv"]) * (3 * case["rot"] + (4 * d if case["headnorm"] else 0))
        return {"bytes": 2 * T * vectors * d + 4 * (2 * S + 1 + pages) + 8 * (case["rot"] // 2), "flops": T * flops}
    q, of, rank = _ranks(case)
    k, n, slices = case["k"], sum(_cols(case)), len(_cols(case))
    T, have = int(q.sum()), of >= 0
    rows = int(q[have].sum())
    size = 2 * rows * k + 4 * T * n + 8 * len(q)
    size += 2 * int(rank[np.unique(of[have])].sum()) * (k * slices + n)
    return {"bytes": size, "flops": 2 * int((q[have] * rank[of[have]]).sum()) * (k * slices + n)}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_norm(s):
    c = s["case"]
    out = {}
    rows, width = s["x"].shape
    x = s["x"].double()

    def scaled(t, weight):
        size = torch.linalg.vector_norm(t, dim=1, keepdim=True)
        return t * (c["offset"] + weight.double()) * torch.rsqrt(size ** 2 / width + EPS)
    if s["y"] is not None:
        branch = s["y"].double()
        branch = scaled(branch, s["w_post"]) if s["w_post"] is not None else branch
        branch = branch * s["gate"].double().expand(rows, width) if s["gate"] is not None else branch
        x = c["residual"] * x + c["branch"] * branch
        out["x"] = x
    if s["w_pre"] is not None:
        out["z"] = scaled(x, s["w_pre"])
    return out


def _exact_rope(s):
    c = s["case"]
    rot, rows = c["rot"], _rows(c)
    # multiplication by a unit complex number, sequence by sequence
    exponent = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot
    log_base = math.log(c["base"]) + (rot / (rot - 2) * math.log(c["by"]) if c["scaling"] == "base" else 0.0)
    freq = torch.exp(-exponent * log_base)
    if c["scaling"] == "linear":
        freq = freq / c["by"]
    if c["scaling"] == "parts":
        wave = 2 * math.pi / freq
        ramp = torch.clamp((8192 / wave - 1.0) / 31.0, min=0.0, max=1.0)
        freq = (1 - ramp) * freq / c["by"] + ramp * freq
    out = {"q": s["q"].double(), "k": s["k"].double(), "k_cache": s["k_cache"].double(),
           "v_cache": s["v_cache"].double()}
    table, at = s["table"].cpu(), 0
    for i, (n, ctx) in enumerate(rows.tolist()):
        pos = torch.arange(ctx - n, ctx, device="cuda")
        unit = torch.polar(torch.full((n, 1, rot // 2), s["factor"], dtype=torch.float64, device="cuda"),
                           (pos[:, None].double() * freq)[:, None, :])
        for p in "qk":
            x = out[p][at:at + n]
            if s[p + "_weight"] is not None:
                x = x * torch.rsqrt((x ** 2).sum(-1, keepdim=True) / c["d"] + EPS) * s[p + "_weight"].double()
            y = x[..., :rot].unflatten(-1, (-1, 2) if c["interleaved"] else (2, -1))
            y = y if c["interleaved"] else y.transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(y.contiguous()) * unit)
            y = (y if c["interleaved"] else y.transpose(-1, -2)).flatten(-2)
            out[p][at:at + n] = torch.cat([y, x[..., rot:]], -1)
        page = table[i][(pos // PAGE).cpu()].long().cuda()
        out["k_cache"].index_put_((page, pos % PAGE), out["k"][at:at + n])
        out["v_cache"].index_put_((page, pos % PAGE), s["v"][at:at + n].double())
        at += n
    if not c["k_out"]:
        del out["k"]
    return out


def _exact_adapters(s):
    of, q = s["of_h"], s["q_len_h"]
    outs = [y.double() for y in s["y"]]
    at = 0
    for i, n in zip(of.tolist(), q.tolist()):
        if i >= 0:
            r, first = int(s["rank_h"][i]), 0
            x = s["x"][at:at + n].double()
            for j, (out, c) in enumerate(zip(outs, s["cols"])):
                low = torch.einsum("tk,rk->tr", x, s["a"][i, j, :r].double())
                up = torch.einsum("tr,nr->tn", low, s["b"][i, first:first + c, :r].double())
                out[at:at + n] += float(s["scale"][i]) * up
                first += c
        at += n
    return {"out": outs}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "adapters": _exact_adapters}[case["op"]](s)
