"""Page bookkeeping on the GPU against the loops of oracle/pages.py, and the
whole run: pages, append, attention and release over many steps."""
import math

import numpy as np
import pytest
import torch

from _gpu import sms
from _hbutil import lib
from _kv8 import Inputs, as_bytes, bits, bounds, check_out, same_bytes
from chunked_prefill_decode_gb300 import workloads
from oracle import kv8, pages

pytestmark = pytest.mark.gpu


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(dtype).cuda()


class Ring:
    def __init__(self, num_pages, head=0, taken=0, seed=0):
        self.order = np.random.default_rng(seed).permutation(num_pages).astype(np.int32)
        self.pages, self.n = dev(self.order), num_pages
        self.head, self.tail = head, head + num_pages - taken
        self.state = torch.tensor([self.head, self.tail, 0, 0], dtype=torch.int64, device="cuda")


def table_for(q, ctx, maxp, num_pages, seed=1):
    """A table whose rows hold pages of another range (num_pages ..) for what
    is cached already, and -7 elsewhere."""
    t = np.full((len(q), maxp), -7, np.int32)
    k = 0
    for s in range(len(q)):
        n = -(-(ctx[s] - q[s]) // 16)
        t[s, :n] = (np.arange(k, k + n) * 7 + seed) % num_pages
        k += n
    return t


def check_assign(q, ctx, maxp, ring, in_place=True, extra=3):
    hb = lib()
    q, ctx = np.asarray(q, np.int32), np.asarray(ctx, np.int32)
    T = int(q.sum())
    table = table_for(q, ctx, maxp, ring.n)
    want = pages.assign(q, ctx, ring.order, ring.head, ring.tail, table)
    d_table, cu = dev(table), torch.full((len(q) + 1,), -5, dtype=torch.int32, device="cuda")
    slots = torch.full((T + extra,), -9, dtype=torch.int64, device="cuda")
    out = ring.state if in_place else torch.zeros(4, dtype=torch.int64, device="cuda")
    before = ring.state.clone()
    hb.hb_pages_assign(dev(q), dev(ctx), ring.pages, ring.state, out, d_table, cu, slots)
    torch.cuda.synchronize()
    assert torch.equal(ring.pages.cpu(), torch.from_numpy(ring.order))
    assert (slots[T:] == -9).all()                 # behind the last token: as it was
    if not in_place:
        assert torch.equal(ring.state, before)
    assert cu.cpu().tolist() == [0] + np.cumsum(q).tolist()
    if want is None:
        with pytest.raises(hb.HbError) as e:
            hb.hb_check()
        assert e.value.status == 8
        assert torch.equal(d_table.cpu(), torch.from_numpy(table)) and (slots[:T] == -1).all()
        assert out.tolist() == [ring.head, ring.tail, 0, 0]
        return None
    hb.hb_check()
    w_cu, w_table, w_slots, w_head = want
    assert np.array_equal(cu.cpu().numpy(), w_cu) and np.array_equal(d_table.cpu().numpy(), w_table)
    assert np.array_equal(slots[:T].cpu().numpy(), w_slots)
    assert out.tolist() == [w_head, ring.tail, 0, 0]
    ring.head = w_head
    return w_table


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("rows", [
    [(1, 1)], [(1, 16)], [(1, 17)], [(0, 0)], [(0, 40), (1, 33), (0, 0), (0, 16)], [(16, 16), (17, 33), (1, 32)],
    [(0, 5), (100, 100), (1, 1), (31, 47), (0, 0)], [(1, c) for c in range(1, 70)]])
def test_assign(rows, in_place):
    q, ctx = zip(*rows)
    check_assign(q, ctx, 12, Ring(64, head=50), in_place)


@pytest.mark.parametrize("n", [511, 512, 513, 1024, 5000, 16384])
def test_assign_many_sequences(n):
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, 200, n)
    q = np.where(rng.random(n) < 0.7, np.minimum(1, ctx), rng.integers(0, ctx + 1))
    check_assign(q, ctx, 13, Ring(16 * n, head=5 * n + 3))


def test_assign_long_prompts():
    check_assign([40000, 1, 33333, 0, 7], [40000, 9, 50000, 8, 7], 3200, Ring(6000, head=10 ** 12))


def test_no_sequences():
    ring = Ring(8)
    check_assign([], [], 4, ring)


@pytest.mark.parametrize("free", [0, 1, 5, 6])
def test_too_few_pages_changes_nothing(free):
    ring = Ring(64, head=7, taken=64 - free)
    got = check_assign([1, 40, 33, 1], [17, 40, 64, 5], 8, ring)     # 1 + 3 + 2 + 0 new pages
    assert (got is None) == (free < 6)


def test_without_slots():
    hb = lib()
    ring = Ring(32)
    table, cu = dev(np.full((2, 4), -1)), dev(np.zeros(3))
    hb.hb_pages_assign(dev([20, 1]), dev([20, 1]), ring.pages, ring.state, ring.state, table, cu)
    hb.hb_check()
    assert table.tolist() == [[int(ring.order[0]), int(ring.order[1]), -1, -1], [int(ring.order[2]), -1, -1, -1]]
    assert ring.state.tolist() == [3, 32, 0, 0]


@pytest.mark.parametrize("q,ctx,state", [
    ([2, 1], [1, 1], None), ([-1, 1], [5, 5], None), ([1, 1], [5, 65], None), ([1, 2 ** 31 - 1], [1, 2 ** 31 - 1], None),
    ([40, 41], [40, 41], None),                      # 81 tokens, 80 slots
    ([1, 1], [1, 1], [-1, 5, 0, 0]), ([1, 1], [1, 1], [5, 4, 0, 0]), ([1, 1], [1, 1], [0, 33, 0, 0])])
def test_bad_lengths_change_nothing(q, ctx, state):
    hb = lib()
    ring = Ring(32)
    if state:
        ring.state = torch.tensor(state, dtype=torch.int64, device="cuda")
    before = ring.state.clone()
    table, cu = dev(np.full((2, 4), -1)), dev(np.full(3, -5))
    slots = torch.full((80,), -9, dtype=torch.int64, device="cuda")
    hb.hb_pages_assign(dev(q), dev(ctx), ring.pages, ring.state, ring.state, table, cu, slots)
    with pytest.raises(hb.HbError) as e:
        hb.hb_check()
    assert e.value.status == 2
    assert torch.equal(ring.state, before) and (table == -1).all() and (cu == -5).all() and (slots == -9).all()
    hb.hb_check()


def test_bad_pages_are_reported():
    hb = lib()
    for bad in (-1, 32):
        ring = Ring(32)
        ring.pages[1] = bad
        table, cu = dev(np.full((2, 4), -1)), dev(np.zeros(3))
        slots = torch.zeros(50, dtype=torch.int64, device="cuda")
        hb.hb_pages_assign(dev([40, 1]), dev([40, 20]), ring.pages, ring.state, ring.state, table, cu, slots)
        with pytest.raises(hb.HbError) as e:       # ring entry 1 and table entry [1, 1]
            hb.hb_check()
        assert e.value.status == 6
        s = slots.tolist()
        assert s[16:32] == [-1] * 16 and s[40] == -1 and s[0] == int(ring.order[0]) * 16 and table[0, 1] == -1
        d_table = dev(np.array([[3, bad, 5, 0]]))
        ring = Ring(32, taken=10)
        hb.hb_pages_release(dev([33]), ring.pages, ring.state, ring.state, d_table)
        with pytest.raises(hb.HbError) as e:
            hb.hb_check()
        assert e.value.status == 6
        assert ring.pages.tolist()[22:25] == [3, -1, 5]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lengths,maxp", [
    ([1], 1), ([0], 1), ([16, 17, 0, 32, 1], 3), ([0, 0, 160], 10), (list(range(0, 300)), 19), ([], 4)])
def test_release(lengths, maxp, in_place):
    hb = lib()
    n = sum(-(-x // 16) for x in lengths)
    ring = Ring(n + 9, head=n + 2, taken=n + 5)
    rng = np.random.default_rng(3)
    table = rng.integers(0, n + 9, (len(lengths), maxp)).astype(np.int32)
    want, w_tail = pages.release(lengths, ring.order, ring.head, ring.tail, table)
    out = ring.state if in_place else torch.zeros(4, dtype=torch.int64, device="cuda")
    hb.hb_pages_release(dev(lengths), ring.pages, ring.state, out, dev(table))
    hb.hb_check()
    assert np.array_equal(ring.pages.cpu().numpy(), want) and out.tolist() == [ring.head, w_tail, 0, 0]


def test_release_of_more_than_was_taken_changes_nothing():
    hb = lib()
    ring = Ring(20, taken=3)
    table = dev(np.zeros((2, 2)))
    for lengths in ([32, 32], [-1, 5], [33, 0]):
        before = ring.state.clone()
        hb.hb_pages_release(dev(lengths), ring.pages, ring.state, ring.state, table)
        with pytest.raises(hb.HbError) as e:
            hb.hb_check()
        assert e.value.status == 2
        assert torch.equal(ring.state, before) and np.array_equal(ring.pages.cpu().numpy(), ring.order)


def test_captured_assignments_advance_the_ring():
    """A captured assignment replayed: each replay takes the next pages."""
    hb = lib()
    ring = Ring(100, head=90)
    q, ctx = dev([32, 5]), dev([32, 5])
    table, cu = dev(np.full((2, 4), -1)), dev(np.zeros(3))
    slots = torch.zeros(37, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        hb.hb_pages_assign(q, ctx, ring.pages, ring.state, ring.state, table, cu, slots)
    for i in range(5):
        graph.replay()
        torch.cuda.synchronize()
        got = table[:, :2].flatten().tolist()
        want = [int(ring.order[(90 + 3 * i + k) % 100]) for k in range(3)]
        assert got == want + [-1] and ring.state.tolist() == [93 + 3 * i, 190, 0, 0]
    hb.hb_check()


@pytest.mark.parametrize("geom,window", [((8, 2, 64), 0), ((14, 2, 128), 50)])
def test_a_run_of_steps(geom, window):
    """Requests come, grow by chunks and single tokens and go, for 12 steps:
    pages from the ring, append, attention, pages back -- with tables, caches
    and outputs against the oracles after every step."""
    hb = lib()
    hq, hkv, d = geom
    rng = np.random.default_rng(60)
    num_pages, maxp, S = 120, 24, 6
    ring = Ring(num_pages, head=33, seed=61)
    cache = hb.kv8_cache(num_pages, hkv, d)
    o_cache = [as_bytes(c).copy() for c in cache[:2]] + [e.cpu().numpy().copy() for e in cache[2:]]
    table = np.full((S, maxp), -1, np.int32)
    d_table = dev(table)
    cu = dev(np.zeros(S + 1))
    ctx = np.zeros(S, np.int64)
    order = ring.order.copy()
    scale = 1.0 / math.sqrt(d)
    for n_step in range(12):
        gone = np.where((ctx > 150) | ((rng.random(S) < 0.15) & (ctx > 0)), ctx, 0)
        if gone.any():
            order, ring.tail = pages.release(gone, order, ring.head, ring.tail, table)
            hb.hb_pages_release(dev(gone), ring.pages, ring.state, ring.state, d_table)
            ctx[gone > 0] = 0
        q = np.where(ctx == 0, rng.integers(1, 60, S), np.where(rng.random(S) < 0.6, 1, rng.integers(1, 40, S)))
        ctx = ctx + q
        T = int(q.sum())
        w_cu, table, w_slots, ring.head = pages.assign(q, ctx, order, ring.head, ring.tail, table)
        slots = torch.empty(T, dtype=torch.int64, device="cuda")
        d_ctx = dev(ctx)
        hb.hb_pages_assign(dev(q), d_ctx, ring.pages, ring.state, ring.state, d_table, cu, slots)
        batch = hb.make_batch(S, T, maxp, num_pages, hq, hkv, d, cu, d_ctx, d_table, sliding_window=window)
        kn, vn = (torch.randn(T, hkv, d).mul_(2.0 ** float(rng.integers(-3, 4))).to(torch.bfloat16) for _ in range(2))
        qt = torch.randn(T, hq, d).to(torch.bfloat16)
        out = torch.full_like(qt, float("nan"), device="cuda")
        hb.hb_kv8_append(batch, kn.cuda(), vn.cuda(), *cache)
        plan, ws = hb.hb_kv8_plan(batch, q, ctx, sms())
        hb.hb_kv8_attention(batch, plan, qt.cuda(), *cache, scale, out, ws)
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
        check_out(out, *bounds(layout, inp, o_cache))


def test_state_out_may_hold_anything():
    """Many CTAs; the state written to an array of its own, whatever that held."""
    hb = lib()
    n, pages_, maxp = 700, 9000, 12
    ring, state = hb.pages_ring(pages_)
    q = torch.full((n,), 150, dtype=torch.int32, device="cuda")
    table = torch.full((n, maxp), -1, dtype=torch.int32, device="cuda")
    cu = torch.empty(n + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(n * 150, dtype=torch.int64, device="cuda")
    after, back = (torch.full((4,), 77, dtype=torch.int64, device="cuda") for _ in range(2))
    hb.hb_pages_assign(q, q, ring, state, after, table, cu, slots)
    hb.hb_pages_release(q, ring, after, back, table)
    hb.hb_check()
    assert state.tolist() == [0, pages_, 0, 0]
    assert after.tolist() == [7000, pages_, 0, 0] and back.tolist() == [7000, pages_ + 7000, 0, 0]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("rows,maxp", [(16384, 3), (15000, 2), (1, 9000), (2, 70000), (455, 300), (457, 300)])
def test_release_of_many_rows_and_of_wide_ones(rows, maxp, in_place):
    """More rows in a CTA than a warp has lanes; several CTAs for one row."""
    hb = lib()
    rng = np.random.default_rng(rows)
    lengths = np.where(rng.random(rows) < 0.2, 0, rng.integers(1, maxp * 16 + 1, rows)).astype(np.int32)
    lengths[0] = maxp * 16
    n = int((-(-lengths // 16)).sum())
    ring = Ring(n + 100, head=3 * n, taken=n, seed=rows)
    table = rng.integers(0, n + 100, (rows, maxp)).astype(np.int32)
    want, w_tail = pages.release(lengths, ring.order, ring.head, ring.tail, table)
    out = ring.state if in_place else torch.full((4,), 5, dtype=torch.int64, device="cuda")
    hb.hb_pages_release(dev(lengths), ring.pages, ring.state, out, dev(table))
    hb.hb_check()
    assert np.array_equal(ring.pages.cpu().numpy(), want)
    assert out.tolist() == [ring.head, w_tail, 0, 0]
