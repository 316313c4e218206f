"""One transformer block of a hybrid batch: the linear layers around the
attention step, every step in this library's kernels.

"Sarathi-Serve：以 chunked-prefills 与 stall-free batching 驯服 LLM 推理的吞吐—
延迟权衡", §问题背景 (两阶段天然不对称): besides attention, every token of a
hybrid batch passes through the model's linear layers, which take most of
the iteration; chunking a prefill lets its tokens share those weight reads
with the decode tokens of the same iteration.  The pages do not write the
block out; the plain GQA block is taken:

    q, k, v = split(x Wqkv^T)                    hb_linear, split epilogue
    append k, v to the paged cache               hb_kv_append
    a = attention(q, cache)                       hb_plan + hb_attention_new_kv
    x = x + a Wo^T                                hb_linear, residual epilogue
    m = silu(x Wg^T) * (x Wu^T)                   hb_linear, gated epilogue
    x = x + m Wd^T                                hb_linear, residual epilogue

What a model adds to it is on request (BlockNorms, hb.make_rope, hb.make_adapters):

    z = norm(x)  before each branch               hb_norm
    x = r x + s gate norm(branch)  after it       hb_norm (with the next z)
    q, k turned by their positions                hb_rope (in hb_kv_append's place)
    + scale (x A^T) B^T  with each request's      hb_adapters (q, k, v; the output
      own adapter                                 and down projections; not gate and
                                                  up, whose epilogue applies silu)

Weights are synthetic (seeded, N(0, 1/fan_in) in bf16): no trained weights
are needed to time or check the block.  The residual stream x is updated in
place.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import hb


@dataclass
class BlockShape:
    hidden: int = 4096          # model width H
    num_q_heads: int = 32
    num_kv_heads: int = 8
    head_dim: int = 128
    ffn: int = 14336            # gated-MLP width F
    page_size: int = 16

    @property
    def q_cols(self):
        return self.num_q_heads * self.head_dim

    @property
    def kv_cols(self):
        return self.num_kv_heads * self.head_dim

    def params(self) -> int:
        H = self.hidden
        return (self.q_cols + 2 * self.kv_cols) * H + H * self.q_cols + 2 * self.ffn * H + H * self.ffn


@dataclass
class BlockNorms:
    """Norms around a block's two branches.  post: also after a branch; gated: a
    gate per channel on its output; the stream is residual_scale * x +
    branch_scale * gate * branch.  stream_fp32: x is fp32."""
    eps: float = 1e-5
    post: bool = False
    gated: bool = False
    residual_scale: float = 1.0
    branch_scale: float = 1.0
    weight_offset: float = 0.0
    stream_fp32: bool = False


MISTRAL_7B = BlockShape()
YI_34B = BlockShape(hidden=7168, num_q_heads=56, num_kv_heads=8, head_dim=128, ffn=20480)


class HybridBlock:
    """Synthetic weights of one block on a device, and its forward step."""

    def __init__(self, shape: BlockShape = MISTRAL_7B, seed: int = 0, device="cuda", norms: BlockNorms | None = None,
                 rope=None, adapters=None):
        """norms: BlockNorms, or None for a block without; rope: hb.make_rope's
        parameters; adapters: pools (hb.make_adapters) by projection, of "qkv" (three
        destinations), "o" and "d"."""
        s = shape
        for name, v in (("hidden", s.hidden), ("q columns", s.q_cols), ("kv columns", s.kv_cols),
                        ("ffn", s.ffn)):
            if v % 256:
                raise ValueError(f"{name} ({v}) must be a multiple of 256 for the GEMM tiles")
        self.shape = s
        self.dev = torch.device(device)
        g = torch.Generator(device=self.dev).manual_seed(seed)

        def weight(n, k):
            return (torch.randn(n, k, generator=g, device=self.dev) / math.sqrt(k)).to(torch.bfloat16)
        H = s.hidden
        self.w_qkv = weight(s.q_cols + 2 * s.kv_cols, H)
        self.w_o = weight(H, s.q_cols)
        self.w_gu = weight(2 * s.ffn, H)
        self.w_d = weight(H, s.ffn)
        self.norms, self.rope, self.adapters = norms, rope, dict(adapters or {})
        want = {"qkv": (H, (s.q_cols, s.kv_cols, s.kv_cols)), "o": (s.q_cols, (H,)), "d": (s.ffn, (H,))}
        for name, pool in self.adapters.items():
            if name not in want or (pool.K, pool.cols) != want[name]:
                raise ValueError(f"adapters[{name!r}] must be of {sorted(want)} and fit its projection")
        if norms is not None:
            def gain(spread, mean):
                return (mean + spread * torch.randn(H, generator=g, device=self.dev)).to(torch.bfloat16)
            unit = 1.0 - norms.weight_offset
            self.w_pre = [gain(0.1, unit) for _ in range(2)]
            self.w_post = [gain(0.1, unit) if norms.post else None for _ in range(2)]
            self.gates = [gain(0.3, 1.0) if norms.gated else None for _ in range(2)]
        self.scale = 1.0 / math.sqrt(s.head_dim)
        self._plan = None
        self._ws = None
        self._sms = torch.cuda.get_device_properties(self.dev).multi_processor_count

    def buffers(self, tokens: int) -> dict:
        """Activation buffers for a batch of `tokens` new tokens."""
        s = self.shape
        e = dict(dtype=torch.bfloat16, device=self.dev)
        b = {"q": torch.empty(tokens, s.q_cols, **e),
             "k": torch.empty(tokens, s.kv_cols, **e),
             "v": torch.empty(tokens, s.kv_cols, **e),
             "a": torch.empty(tokens, s.q_cols, **e),
             "m": torch.empty(tokens, s.ffn, **e)}
        if self.norms is not None:
            b["z"] = torch.empty(tokens, s.hidden, **e)     # a branch's normed input
            b["y"] = torch.empty(tokens, s.hidden, **e)     # a branch's output
        return b

    def plan_adapters(self, q_len, adapter, total_q=None, plan=None, workspace=None):
        """The step's adapter plan, for forward (and every block of as many
        adapters): each sequence's q_len and adapter (-1: none)."""
        return hb.hb_adapters_plan(list(self.adapters.values()), q_len, adapter, self._sms, total_q=total_q, plan=plan,
                                   workspace=workspace)

    def _adapt(self, name, plan, x, ys):
        if name in self.adapters and plan is not None:
            hb.hb_adapters(self.adapters[name], plan[0], x, ys, ys, plan[1])

    def _norm(self, i, x, y, x_out, z, w_pre):
        """The norm after branch i and its residual sum (y given), and the next
        branch's norm (z given)."""
        n = self.norms
        more = {} if y is None else dict(w_post=self.w_post[i], gate=self.gates[i], residual_scale=n.residual_scale,
                                         branch_scale=n.branch_scale)
        hb.hb_norm(x=x, y=y, x_out=x_out, z=z, w_pre=w_pre, eps=n.eps, weight_offset=n.weight_offset, **more)

    def forward(self, x, batch, k_cache, v_cache, bufs=None, plan=True, snapshot=False, adapter_plan=None,
                normed=False, next_weight=None):
        """x: [T, H] residual stream (updated in place), bf16 (fp32 with
        norms.stream_fp32); batch: an hb_batch (device.device_batch) of the same
        T new tokens; k_cache, v_cache: the layer's page pools; adapter_plan:
        plan_adapters' result, or None for no adapters in this step.  Returns
        the buffers used; with snapshot=True they also hold a copy of the
        residual stream after the attention block ("h", for checking the stages
        one by one).  With norms, blocks in a row share a launch between them:
        next_weight (the next block's w_pre[0]) leaves its normed input in
        bufs["z"], and normed=True says that the block before did (in these bufs)."""
        T = x.shape[0]
        s = self.shape
        if self.norms is not None and (x.dtype is torch.float32) != self.norms.stream_fp32:
            raise ValueError(f"x is {x.dtype}, norms.stream_fp32 is {self.norms.stream_fp32}")
        if self.norms is None and (normed or next_weight is not None):
            raise ValueError("a block without norms takes no normed input and leaves none")
        if normed and bufs is None:
            raise ValueError("normed: the block before left its normed input in its buffers, so bufs must be given")
        b = bufs if bufs is not None else self.buffers(T)
        inp = x
        if self.norms is not None:
            inp = b["z"]
            if not normed:
                self._norm(0, x, None, None, b["z"], self.w_pre[0])
        hb.hb_linear(inp, self.w_qkv, [b["q"], b["k"], b["v"]])
        self._adapt("qkv", adapter_plan, inp, [b["q"], b["k"], b["v"]])
        if self.rope is not None:
            heads = {"q": s.num_q_heads, "k": s.num_kv_heads, "v": s.num_kv_heads}
            q, k, v = (b[n].view(T, heads[n], s.head_dim) for n in "qkv")
            hb.hb_rope(batch.batch, self.rope, q, k, v, q, k, k_cache, v_cache)
        else:
            hb.hb_kv_append(batch.batch, b["k"], b["v"], k_cache, v_cache)
        if plan or self._plan is None:
            self._plan, self._ws = hb.hb_plan(batch.batch, batch.q_len, batch.context_len,
                                              self._sms, workspace=self._ws, plan=self._plan)
        hb.hb_attention_new_kv(batch.batch, self._plan, b["q"], b["k"], b["v"], k_cache, v_cache,
                               self.scale, b["a"], self._ws)
        if self.norms is None:
            hb.hb_linear(b["a"], self.w_o, [x], epilogue=hb.LINEAR_RESIDUAL)
            self._adapt("o", adapter_plan, b["a"], [x])
        else:
            hb.hb_linear(b["a"], self.w_o, [b["y"]])
            self._adapt("o", adapter_plan, b["a"], [b["y"]])
            self._norm(0, x, b["y"], x, b["z"], self.w_pre[1])
        if snapshot:
            b["h"] = x.clone()
            if self.norms is not None:
                b["z1"] = b["z"].clone()
        hb.hb_linear(inp, self.w_gu, [b["m"]], epilogue=hb.LINEAR_GATED)
        if self.norms is None:
            hb.hb_linear(b["m"], self.w_d, [x], epilogue=hb.LINEAR_RESIDUAL)
            self._adapt("d", adapter_plan, b["m"], [x])
        else:
            hb.hb_linear(b["m"], self.w_d, [b["y"]])
            self._adapt("d", adapter_plan, b["m"], [b["y"]])
            self._norm(1, x, b["y"], x, b["z"] if next_weight is not None else None, next_weight)
        return b

    def flops(self, tokens: int) -> float:
        """Linear-layer FLOPs of the block for `tokens` new tokens."""
        return 2.0 * self.shape.params() * tokens
