"""Rows that stand still (no new token: waiting, finished, empty) in the whole
step over the 8-bit cache: pages, append, plan, attention, release."""
import math

import numpy as np
import pytest
import torch

from _gpu import sms
from _hbutil import lib
from _kv8 import as_bytes, bits, check_out, same_bytes
from _kv8_rows import row_bounds
from chunked_prefill_decode_gb300 import workloads
from oracle import kv8, pages
from test_gpu_pages import Ring, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("geom,window", [((8, 2, 64), 0), ((14, 2, 128), 50), ((32, 8, 128), 0)])
def test_a_run_with_rows_that_stand_still(geom, window):
    """Every step some rows have no token, some are empty, and in one step none
    has any; tables, caches and outputs against the oracles after each."""
    hb = lib()
    hq, hkv, d = geom
    rng = np.random.default_rng(90)
    num_pages, maxp, S = 160, 24, 8
    ring = Ring(num_pages, head=21, seed=91)
    cache = hb.kv8_cache(num_pages, hkv, d)
    o_cache = [as_bytes(c).copy() for c in cache[:2]] + [e.cpu().numpy().copy() for e in cache[2:]]
    table, order = np.full((S, maxp), -1, np.int32), ring.order.copy()
    d_table, cu = dev(table), dev(np.zeros(S + 1))
    ctx = np.zeros(S, np.int64)
    for n_step in range(10):
        gone = np.where((ctx > 200) | ((rng.random(S) < 0.1) & (ctx > 0)), ctx, 0)
        order, ring.tail = pages.release(gone, order, ring.head, ring.tail, table)
        hb.hb_pages_release(dev(gone), ring.pages, ring.state, ring.state, d_table)
        ctx[gone > 0] = 0
        kind = rng.random(S)
        q = np.where(kind < 0.4, 0, np.where((kind < 0.7) & (ctx > 0), 1, rng.integers(1, 70, S)))
        if n_step == 5:
            q[:] = 0
        ctx = ctx + q
        T = int(q.sum())
        w_cu, table, w_slots, ring.head = pages.assign(q, ctx, order, ring.head, ring.tail, table)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        d_ctx = dev(ctx)
        hb.hb_pages_assign(dev(q), d_ctx, ring.pages, ring.state, ring.state, d_table, cu, slots)
        batch = hb.make_batch(S, T, maxp, num_pages, hq, hkv, d, cu, d_ctx, d_table, sliding_window=window)
        kn, vn = (torch.randn(T, hkv, d, generator=torch.Generator().manual_seed(10 * n_step + i)).to(torch.bfloat16)
                  for i in range(2))
        qt = torch.randn(T, hq, d, generator=torch.Generator().manual_seed(10 * n_step + 2)).to(torch.bfloat16)
        out = torch.full_like(qt, float("nan"), device="cuda")
        hb.hb_kv8_append(batch, kn.cuda(), vn.cuda(), *cache)
        plan, ws = hb.hb_kv8_plan(batch, q, ctx, sms())
        hb.hb_kv8_attention(batch, plan, qt.cuda(), *cache, 1.0 / math.sqrt(d), out, ws)
        hb.hb_check()
        assert np.array_equal(cu.cpu().numpy(), w_cu) and np.array_equal(slots.cpu().numpy(), w_slots)
        assert np.array_equal(d_table.cpu().numpy(), table)
        assert ring.state.tolist() == [ring.head, ring.tail, 0, 0]
        o_cache = kv8.append(*o_cache, bits(kn), bits(vn), q, ctx, table)
        assert all(same_bytes(as_bytes(c), w) for c, w in zip(cache[:2], o_cache[:2]))
        assert all(np.array_equal(e.cpu().numpy(), w) for e, w in zip(cache[2:], o_cache[2:]))
        layout = workloads.BatchLayout(workloads.Shape(hq, hkv, d, sliding_window=window), q.astype(np.int32),
                                       ctx.astype(np.int32), table, num_pages)

        class Inp:
            pass
        inp = Inp()
        inp.q = qt
        check_out(out, *row_bounds(layout, inp, o_cache))
