"""HybridBlock.forward's refusals on the host (no GPU): they come before any launch."""
import pytest
import torch

from chunked_prefill_decode_gb300 import layer
from chunked_prefill_decode_gb300.layer import BlockNorms, BlockShape, HybridBlock


def block(norms):
    b = HybridBlock.__new__(HybridBlock)      # (the constructor asks for a GPU)
    b.shape = BlockShape(hidden=512, num_q_heads=8, num_kv_heads=2, head_dim=64, ffn=1024)
    b.dev, b.norms, b.rope, b.adapters = torch.device("cpu"), norms, None, {}
    b.w_qkv = torch.zeros(768, 512, dtype=torch.bfloat16)
    return b


def test_a_normed_input_is_asked_for_with_the_buffers_that_hold_it(monkeypatch):
    class Launched(Exception):
        pass

    def launch(*args, **kw):
        raise Launched
    monkeypatch.setattr(layer.hb, "hb_linear", launch)
    b, x = block(BlockNorms()), torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bufs must be given"):
        b.forward(x, None, None, None, normed=True)
    with pytest.raises(Launched):             # with them it goes on to the first launch
        b.forward(x, None, None, None, normed=True, bufs=b.buffers(4))


def test_a_block_without_norms_takes_none():
    b, x = block(None), torch.zeros(4, 512, dtype=torch.bfloat16)
    for kw in (dict(normed=True), dict(next_weight=x[0])):
        with pytest.raises(ValueError, match="without norms"):
            b.forward(x, None, None, None, **kw)
