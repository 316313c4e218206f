"""hb_rope without a cache before the 8-bit cache's append and attention: a step's
q and k turned, the new rows quantised, the attention over them; each against its
definition, eagerly and replayed from a graph."""
import math

import numpy as np
import pytest
import torch

from _gpu import sms
from _hbutil import lib
from _kv8 import Inputs, as_bytes, bounds, check_out, same_bytes
from chunked_prefill_decode_gb300.device import from_layout
from chunked_prefill_decode_gb300.workloads import Shape, layout_from_rows
from test_gpu_rope import EPS, angles, check, expected

pytestmark = pytest.mark.gpu
ROWS = [(1, 300), (1, 33), (130, 1000), (1, 16), (40, 40), (1, 1)]


@pytest.mark.parametrize("geom,norms", [((8, 8, 64), False), ((32, 8, 128), True)])
def test_rotated_rows_into_the_8_bit_cache_and_the_attention(geom, norms):
    hb = lib()
    hq, hkv, d = geom
    lay = layout_from_rows(Shape(*geom), ROWS, 31)
    inp = Inputs(lay, 32)
    db = from_layout(lay, "cuda:0")
    T = lay.total_q
    # the projection's output: q, k and v in one tensor
    qkv = torch.cat([inp.q, inp.k_new, inp.v_new], 1).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], inp.v_new.cuda()
    g = torch.Generator("cuda").manual_seed(33)
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(torch.bfloat16) if norms else None for _ in range(2)]
    rope = hb.make_rope(d, q_weight=w[0], k_weight=w[1], eps=EPS)
    plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
    scale = 1.0 / math.sqrt(d)
    qo, ko = torch.empty_like(inp.q, device="cuda"), torch.empty_like(inp.k_new, device="cuda")
    out = torch.full_like(qo, float("nan"))
    cache = inp.device()

    def step():
        hb.hb_rope(db.batch, rope, q, k, None, qo, ko, None, None)
        hb.hb_kv8_append(db.batch, ko, v, *cache)
        hb.hb_kv8_attention(db.batch, plan, qo, *cache, scale, out, ws)
    step()
    hb.hb_check()
    angle = angles(d, np.concatenate([np.arange(c - n, c) for n, c in ROWS]))
    check(qo, expected(inp.q, w[0], angle, False, 1.0))
    check(ko, expected(inp.k_new, w[1], angle, False, 1.0))
    inp.q, inp.k_new = qo.cpu(), ko.cpu()
    want = inp.oracle_append(lay)
    for got, x in zip(cache[:2], want[:2]):
        assert same_bytes(as_bytes(got), x)
    for got, x in zip(cache[2:], want[2:]):
        assert np.array_equal(got.cpu().numpy(), x)
    check_out(out, *bounds(lay, inp, want))
    # the same step from a graph, into a cache without its rows
    first, filled = out.clone(), [as_bytes(c) for c in cache]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for c, was in zip(cache, inp.device()):
            c.view(torch.uint8).copy_(was.view(torch.uint8))
        qo.zero_(), ko.zero_(), out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and all(np.array_equal(as_bytes(c), f) for c, f in zip(cache, filled))
    hb.hb_check()
    assert T == sum(n for n, _ in ROWS)
