"""A transformer block with norms, rotary positions and adapters
(layer.HybridBlock with its options), checked stage by stage against the fp64
oracle fed with the GPU's own intermediates, as the plain block is.

Bars: linear layers and adapters 2^-8 relative (of each value that is rounded on
the way: the projection, then the sum) + 2e-3, norms and rotations 2^-8 relative
+ 1e-5 of the terms, attention max-abs 1e-2 / mean-abs 1e-3 of unit values."""
import math

import numpy as np
import pytest
import torch

from _gpu import compare
from _hbutil import lib
from chunked_prefill_decode_gb300 import workloads
from chunked_prefill_decode_gb300.device import from_layout
from chunked_prefill_decode_gb300.layer import BlockNorms, BlockShape, HybridBlock
from chunked_prefill_decode_gb300.workloads import Shape, layout_from_rows
from oracle import block as ob
from oracle import linear as ol
from oracle import paged_attention as pa

pytestmark = pytest.mark.gpu
bits = workloads.bf16_bits
BF = torch.bfloat16
HQ, HKV, D = 8, 2, 128
SHAPE = BlockShape(hidden=512, num_q_heads=HQ, num_kv_heads=HKV, head_dim=D, ffn=1024)
ROWS = [(1, 300), (1, 41), (150, 150), (1, 129), (33, 600)]
OF = [1, -1, 0, 1, 2]


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, atol, size=0.0, rtol=2.0 ** -8):
    got = f64(got)
    assert np.isfinite(got).all()
    excess = np.abs(got - want) - (rtol * (np.abs(want) + size) + atol)
    assert (excess <= 0).all(), f"worst excess {excess.max():.3e}"


def pools(g, n=3, r=16):
    hb = lib()
    out = {}
    for name, k, cols in (("qkv", 512, (1024, 256, 256)), ("o", 1024, (512,)), ("d", 1024, (512,))):
        a = (torch.randn(n, len(cols), r, k, generator=g, device="cuda") / k ** 0.5).to(BF)
        b = (torch.randn(n, sum(cols), r, generator=g, device="cuda") / r ** 0.5).to(BF)
        rank = torch.tensor([r, 5, 8], dtype=torch.int32, device="cuda")
        out[name] = hb.make_adapters(a, b, rank, torch.tensor([0.5, 1.0, -0.7], device="cuda"), cols)
    return out


class Run:
    def __init__(self, blk, seed=21, plan=True, dtype=BF):
        self.lay = layout_from_rows(Shape(HQ, HKV, D), ROWS, seed)
        ten = workloads.make_tensors(self.lay, seed, device="cuda")
        self.kc0, self.vc0 = ten.k_cache, ten.v_cache
        self.db = from_layout(self.lay)
        g = torch.Generator("cuda").manual_seed(5)
        self.x0 = torch.randn(self.lay.total_q, 512, generator=g, device="cuda").to(dtype)
        self.x, self.kc, self.vc = self.x0.clone(), ten.k_cache.clone(), ten.v_cache.clone()
        self.plan = blk.plan_adapters(self.lay.q_len, OF) if plan else None


def adapted(blk, name, x, ys):
    """Projection outputs with the adapters', and the sizes of what was rounded before."""
    p = blk.adapters[name]
    a, b, rank, scale = (f64(t) for t in p.tensors)
    outs, _ = ob.adapters(x, ys, [r[0] for r in ROWS], OF, a, b, rank, scale)
    return outs, [np.abs(y) for y in ys]


@pytest.mark.parametrize("post,fp32", [(False, False), (True, False), (True, True)])
def test_full_block_stage_by_stage(post, fp32):
    hb = lib()
    n = BlockNorms(post=post, gated=post, residual_scale=0.9 if post else 1.0, branch_scale=0.8 if post else 1.0,
                   weight_offset=1.0 if post else 0.0, stream_fp32=fp32)
    g = torch.Generator("cuda").manual_seed(3)
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g, device="cuda").to(BF) for _ in range(2))
    rope = hb.make_rope(D // 2, base=5e5, q_weight=qw, k_weight=kw, eps=1e-5)
    blk = HybridBlock(SHAPE, seed=7, norms=n, rope=rope, adapters=pools(g))
    r = Run(blk, dtype=torch.float32 if fp32 else BF)
    q_pre = {}
    # what goes into hb_rope is turned in place: keep a copy of it
    real = hb.hb_rope

    def keep(batch, rope_, q, k, v, *rest):
        q_pre.update(q=q.clone(), k=k.clone())
        real(batch, rope_, q, k, v, *rest)
    z_pre = {}
    real_linear = hb.hb_linear

    def keep_linear(x, w, outs, **kws):
        if w is blk.w_qkv:
            z_pre["z"] = x.clone()
        real_linear(x, w, outs, **kws)
        if w is blk.w_o:
            z_pre["o"] = outs[0].clone()
    import chunked_prefill_decode_gb300.layer as layer
    patched = type("Calls", (), {"__getattr__": lambda self, k: {"hb_rope": keep, "hb_linear": keep_linear}.get(k) or getattr(hb, k)})()
    layer.hb, was = patched, layer.hb
    try:
        b = blk.forward(r.x, r.db, r.kc, r.vc, snapshot=True, adapter_plan=r.plan)
    finally:
        layer.hb = was
    torch.cuda.synchronize()
    hb.hb_check()
    lay, T = r.lay, r.lay.total_q
    off = n.weight_offset
    rs, bs = n.residual_scale, n.branch_scale

    def normed(stream, i):
        return ob.rms_norm(f64(stream), f64(blk.w_pre[i]), n.eps, off)

    def summed(x0, y, i):
        return ob.norm(x=f64(x0), y=f64(y), gate=f64(blk.gates[i]), w_post=f64(blk.w_post[i]), eps=n.eps,
                       residual_scale=rs, branch_scale=bs, offset=off)[0]
    close(z_pre["z"], normed(r.x0, 0), 1e-5)
    # projection and adapters; then norms and rotation of the heads
    z = f64(z_pre["z"])
    qkv = ol.linear(bits(z_pre["z"]), bits(blk.w_qkv))
    outs, sizes = adapted(blk, "qkv", z, [qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:]])
    for got, want, size in zip((q_pre["q"].view(T, -1), q_pre["k"].view(T, -1), b["v"]), outs, sizes):
        close(got, want, 2e-3, size)
    pos = np.concatenate([np.arange(c - m, c) for m, c in ROWS])
    angle = pos[:, None, None] * ob.rope_frequencies(D // 2, 5e5).astype(np.float64)
    for name, w, heads in (("q", qw, HQ), ("k", kw, HKV)):
        want = ob.rotate(ob.rms_norm(f64(q_pre[name]), f64(w), 1e-5), angle)
        close(b[name].view(T, heads, D), want, 2e-5 * np.abs(want).max())
    # the cache holds them, and the attention is over it
    kp, vp = pa.kv_append(bits(r.kc0), bits(r.vc0), bits(b["k"]).reshape(T, HKV, D), bits(b["v"]).reshape(T, HKV, D),
                          lay.q_len, lay.context_len, lay.block_table, 16)
    assert np.array_equal(bits(r.kc), kp) and np.array_equal(bits(r.vc), vp)
    att = pa.attention(bits(b["q"]).reshape(T, HQ, D), kp, vp, lay.q_len, lay.context_len, lay.block_table, 16, HQ, HKV,
                       1 / math.sqrt(D))
    unit = max(1.0, np.abs(f64(b["v"])).max() / 4)        # (the bars are for values of unit deviation)
    compare(b["a"].view(T, HQ, D), att, max_abs=1e-2 * unit, mean_abs=1e-3 * unit)
    # the branch, its norm and gate, the sum, the next norm
    o = ol.linear(bits(b["a"]), bits(blk.w_o))
    close(z_pre["o"], o, 2e-3)
    branch, size = adapted(blk, "o", f64(b["a"]), [o])
    y = branch[0]
    got_h = f64(b["h"])
    # (bounded through the branch's roundings: what the norm and gate do to them)
    gain = bs * np.abs(1.0 if blk.gates[0] is None else f64(blk.gates[0]))
    if post:
        gain = gain * np.abs(off + f64(blk.w_post[0])) / np.sqrt(np.mean(y * y, -1, keepdims=True) + n.eps) * 1.02
    bound = gain * (2.0 ** -8 * (np.abs(y) + size[0]) + 2e-3) + np.abs(summed(r.x0, y_tensor(y), 0)) * (0 if fp32 else 2.0 ** -8) + 1e-4
    if post:                                              # the row's own size moves with its elements' roundings
        bound = bound + 2.0 ** -8 * np.abs(summed(r.x0, y_tensor(y), 0) - rs * f64(r.x0))
    assert (np.abs(got_h - summed(r.x0, y_tensor(y), 0)) <= bound).all()
    h = b["h"]
    # (z is the norm of the sum before its rounding: 2^-8 of each element more)
    close(b["z1"], normed(h, 1), 1e-4, 0.0 if fp32 else np.abs(normed(h, 1)), 2.0 ** -8 * 1.2)
    close(b["m"], ol.gated_mlp_up(bits(b["z1"]), bits(blk.w_gu)), 2e-3)
    d = ol.linear(bits(b["m"]), bits(blk.w_d))
    y, size = adapted(blk, "d", f64(b["m"]), [d])
    close(b["y"], y[0], 2e-3, size[0])
    close(r.x, summed(b["h"], b["y"], 1), 1e-4, rtol=0.0 if fp32 else 2.0 ** -8)


def y_tensor(y):
    return torch.from_numpy(y)


def test_options_off_are_the_plain_block():
    hb = lib()
    plain = HybridBlock(SHAPE, seed=7)
    g = torch.Generator("cuda").manual_seed(3)
    other = HybridBlock(SHAPE, seed=7, adapters=pools(g))
    a, b = Run(plain, plan=False), Run(other)
    plain.forward(a.x, a.db, a.kc, a.vc)
    other.forward(b.x, b.db, b.kc, b.vc)                 # no adapters in this step
    hb.hb_check()
    assert torch.equal(a.x, b.x) and torch.equal(a.kc.view(torch.int16), b.kc.view(torch.int16))   # (NaN in free slots)
    c = Run(other)
    c.plan = other.plan_adapters(c.lay.q_len, [-1] * len(ROWS))
    other.forward(c.x, c.db, c.kc, c.vc, adapter_plan=c.plan)
    assert torch.equal(c.x, a.x)


def test_adapters_in_the_plain_block_reach_the_stream():
    hb = lib()
    g = torch.Generator("cuda").manual_seed(3)
    blk = HybridBlock(SHAPE, seed=7, adapters=pools(g))
    a, b = Run(blk), Run(blk)
    blk.forward(a.x, a.db, a.kc, a.vc)
    bufs = blk.forward(b.x, b.db, b.kc, b.vc, adapter_plan=b.plan)
    hb.hb_check()
    cu = np.concatenate([[0], np.cumsum([r[0] for r in ROWS])])
    for i, of in enumerate(OF):
        rows = slice(cu[i], cu[i + 1])
        assert torch.equal(a.x[rows], b.x[rows]) == (of < 0)
    d = f64(bufs["m"])
    assert np.isfinite(d).all()


def test_blocks_in_a_row_share_their_norm():
    """Two blocks with the norm between them taken by the first one's last launch,
    and as a launch of its own: the same but for the norm of the sum before its
    rounding (none with an fp32 stream)."""
    hb = lib()
    n = BlockNorms(stream_fp32=True)
    blks = [HybridBlock(SHAPE, seed=s, norms=n, rope=hb.make_rope(D)) for s in (1, 2)]
    outs = []
    for fused in (True, False):
        r = Run(blks[0], plan=False, dtype=torch.float32)
        caches = [(r.kc.clone(), r.vc.clone()) for _ in blks]
        bufs = blks[0].buffers(r.lay.total_q)
        blks[0].forward(r.x, r.db, *caches[0], bufs=bufs, next_weight=blks[1].w_pre[0] if fused else None)
        blks[1].forward(r.x, r.db, *caches[1], bufs=bufs, normed=fused)
        outs.append((r.x, *caches[1]))
    hb.hb_check()
    for a, b in zip(*outs):
        assert torch.equal(a.nan_to_num(0.0), b.nan_to_num(0.0))


def test_what_does_not_fit_is_refused():
    hb = lib()
    g = torch.Generator("cuda").manual_seed(3)
    p = pools(g)
    for bad in ({"k": p["o"]}, {"o": p["qkv"]}, {"qkv": p["o"]}):
        with pytest.raises(ValueError, match="adapters"):
            HybridBlock(SHAPE, adapters=bad)
    blk = HybridBlock(SHAPE)
    r = Run(blk, plan=False)
    with pytest.raises(ValueError, match="norms"):
        blk.forward(r.x, r.db, r.kc, r.vc, normed=True)
    blk = HybridBlock(SHAPE, norms=BlockNorms(stream_fp32=True))
    with pytest.raises(ValueError, match="stream_fp32"):
        blk.forward(r.x, r.db, r.kc, r.vc)


def test_captured_block_follows_its_inputs():
    """The whole block in a graph, replayed with other inputs."""
    hb = lib()
    g = torch.Generator("cuda").manual_seed(3)
    blk = HybridBlock(SHAPE, seed=7, norms=BlockNorms(post=True), rope=hb.make_rope(D), adapters=pools(g))
    a, b = Run(blk), Run(blk)
    b.x0 = torch.randn_like(b.x0.float()).to(BF)
    b.x.copy_(b.x0)
    blk.forward(b.x, b.db, b.kc, b.vc, adapter_plan=b.plan)
    want = b.x.clone()
    bufs = blk.buffers(a.lay.total_q)
    blk.forward(a.x, a.db, a.kc, a.vc, bufs=bufs, adapter_plan=a.plan)   # (plans are made outside)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        blk.forward(a.x, a.db, a.kc, a.vc, bufs=bufs, adapter_plan=a.plan, plan=False)
    a.x.copy_(b.x0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.x, want)
    hb.hb_check()
