"""After a page assignment that failed, the calls that follow it in the same
stream: no page of another sequence is written, and the error that hb_check
gives is the assignment's."""
import numpy as np
import pytest
import torch

from _hbutil import lib
from test_gpu_pages import Ring, dev

pytestmark = pytest.mark.gpu

HKV, D, PAGES = 2, 64, 16


class Caches:
    """A bf16 and an 8-bit cache that hold known bytes everywhere."""

    def __init__(self, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        shape = (PAGES, 16, HKV, D)
        self.bf16 = [torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
        self.kv8 = [(torch.randn(shape, generator=g, device="cuda") * 100).to(torch.float8_e4m3fn) for _ in range(2)]
        self.kv8 += [torch.full((PAGES, HKV), -8, dtype=torch.int8, device="cuda") for _ in range(2)]

    def append(self, batch, total):
        hb = lib()
        g = torch.Generator("cuda").manual_seed(total)
        kn, vn = ((9 * torch.randn(total, HKV, D, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2))
        hb.hb_kv_append(batch, kn, vn, *self.bf16)
        hb.hb_kv8_append(batch, kn, vn, *self.kv8)

    def pages(self):
        """Each page's bytes, all caches together: [PAGES, n] uint8."""
        torch.cuda.synchronize()
        return torch.cat([c.reshape(PAGES, -1).view(torch.uint8) for c in self.bf16 + self.kv8], 1).cpu().numpy()


def changed(a, b):
    return np.flatnonzero((a != b).any(1)).tolist()


def stale_table(rows, maxp, live):
    """Rows of the live sequence's page ids, as finished requests leave them."""
    return np.resize(np.asarray(live, np.int32), (rows, maxp)).copy()


@pytest.mark.parametrize("free", [0, 1, 2])
def test_too_few_pages_and_an_append_behind_it(free):
    """Row 0 stands still on pages 0 and 1; row 1 is new, row 2 goes on to its
    next page, and the entries that they would fill still name row 0's pages."""
    hb = lib()
    ring = Ring(PAGES, head=5, taken=PAGES - free)
    table = stale_table(3, 4, [0, 1])
    table[0, :2], table[2, 0] = [0, 1], 7
    q, ctx = [0, 40, 1], [32, 40, 17]
    d_table, cu, d_ctx = dev(table), dev([0, 0, 1, 2]), dev(ctx)
    slots = torch.zeros(41, dtype=torch.int64, device="cuda")
    hb.hb_pages_assign(dev(q), d_ctx, ring.pages, ring.state, ring.state, d_table, cu, slots)
    caches = Caches(1)
    before = caches.pages()
    batch = hb.make_batch(3, 41, 4, PAGES, HKV, HKV, D, cu, d_ctx, d_table)
    caches.append(batch, 41)
    assert changed(before, caches.pages()) == []
    with pytest.raises(hb.HbError):
        hb.hb_check()
    hb.hb_check()
    # rows that ask for no page keep theirs, and no entry to be opened names a page
    got = d_table.cpu().numpy()
    assert got[0].tolist() == table[0].tolist() and got[2, 0] == 7
    assert not ((got[1, :3] >= 0) & (got[1, :3] < PAGES)).any() and not 0 <= got[2, 1] < PAGES
    assert got[1, 3] == table[1, 3] and got[2, 2:].tolist() == table[2, 2:].tolist()
    assert ring.state.tolist() == [5, 5 + free, 0, 0] and (slots == -1).all()
    # with pages back in the ring the same call gives what it would have given
    hb.hb_pages_release(dev([64]), ring.pages, ring.state, ring.state, dev([[9, 10, 11, 12]]))
    want = [int(x) for x in torch.roll(ring.pages, -5).tolist()[:4]]
    hb.hb_pages_assign(dev(q), d_ctx, ring.pages, ring.state, ring.state, d_table, cu, slots)
    hb.hb_check()
    got = d_table.cpu().numpy()
    assert got[1, :3].tolist() == want[:3] and got[2].tolist() == [7, want[3], table[2, 2], table[2, 3]]


def test_too_few_pages_for_many_rows():
    """More pages to open than a CTA has threads; only entries that name a page
    are cleared."""
    hb = lib()
    n, maxp = 900, 5
    ring = Ring(3000, head=1, taken=1000)
    rng = np.random.default_rng(2)
    q = rng.integers(0, 80, n)
    ctx = q + rng.integers(0, 80 - q + 1)
    table = rng.integers(-5, 3010, (n, maxp)).astype(np.int32)
    d_table, cu = dev(table), dev(np.zeros(n + 1))
    hb.hb_pages_assign(dev(q), dev(ctx), ring.pages, ring.state, ring.state, d_table, cu)
    with pytest.raises(hb.HbError) as e:
        hb.hb_check()
    assert e.value.status == 8
    lp = np.arange(maxp)[None, :]
    opened = (lp >= -(-(ctx - q) // 16)[:, None]) & (lp < -(-ctx // 16)[:, None])
    assert opened.sum() > 2000
    want = np.where(opened & (table >= 0) & (table < 3000), -1, table)
    assert np.array_equal(d_table.cpu().numpy(), want)
    assert cu.cpu().tolist() == [0] + np.cumsum(q).tolist()


@pytest.mark.parametrize("q,ctx", [([1, 3], [17, 2]), ([17, -1], [33, 5]), ([1, 1], [17, 65])])
def test_bad_lengths_and_an_append_behind_it(q, ctx):
    """The step before had one token per row; the entries beyond name another
    sequence's pages: nothing is written anywhere."""
    hb = lib()
    ring = Ring(PAGES)
    d_table, cu, d_ctx = dev(stale_table(2, 4, [3, 4, 5])), dev([0, 1, 2]), dev(ctx)
    slots = dev([48, 0, -9, 7], torch.int64)
    hb.hb_pages_assign(dev(q), d_ctx, ring.pages, ring.state, ring.state, d_table, cu, slots)
    caches = Caches(3)
    before = caches.pages()
    caches.append(hb.make_batch(2, 2, 4, PAGES, HKV, HKV, D, cu, d_ctx, d_table), 2)
    assert changed(before, caches.pages()) == []
    with pytest.raises(hb.HbError) as e:
        hb.hb_check()
    assert e.value.status == 2
    assert len(set(cu.tolist())) == 1          # a batch without tokens
    assert slots.tolist() == [-1, -1, -9, -1]
    assert np.array_equal(d_table.cpu().numpy(), stale_table(2, 4, [3, 4, 5]))


def test_captured_assign_and_append_until_the_ring_is_empty():
    """Each replay takes three pages; when they run out, replays go on and write
    to no page at all."""
    hb = lib()
    ring = Ring(PAGES, head=3, taken=PAGES - 7, seed=5)
    q, ctx, cu = dev([32, 5]), dev([32, 5]), dev([0, 0, 0])
    d_table, slots = dev(stale_table(2, 3, [1, 2])), torch.zeros(37, dtype=torch.int64, device="cuda")
    caches = Caches(6)
    kn, vn = (torch.randn(37, HKV, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    batch = hb.make_batch(2, 37, 3, PAGES, HKV, HKV, D, cu, ctx, d_table)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        hb.hb_pages_assign(q, ctx, ring.pages, ring.state, ring.state, d_table, cu, slots)
        hb.hb_kv_append(batch, kn, vn, *caches.bf16)
        hb.hb_kv8_append(batch, kn, vn, *caches.kv8)
    seen = [caches.pages()]
    for n in range(4):
        graph.replay()
        seen.append(caches.pages())
        taken = sorted(int(ring.order[(3 + 3 * n + k) % PAGES]) for k in range(3)) if n < 2 else []
        assert changed(seen[-2], seen[-1]) == taken
        assert ring.state.tolist() == [3 + 3 * min(n + 1, 2), 10, 0, 0]
        if n < 2:
            hb.hb_check()
        else:
            with pytest.raises(hb.HbError) as e:
                hb.hb_check()
            assert e.value.status == 8


def test_the_assignments_error_comes_before_what_follows_from_it():
    hb = lib()
    for q, ctx, status in (([1], [17], 8), ([3], [2], 2)):
        ring = Ring(PAGES, taken=PAGES)
        d_table, cu, d_ctx = dev([[-1, -1]]), dev([0, 1]), dev(ctx)
        hb.hb_pages_assign(dev(q), d_ctx, ring.pages, ring.state, ring.state, d_table, cu)
        cu, d_ctx = dev([0, 1]), dev([17])
        Caches(4).append(hb.make_batch(1, 1, 2, PAGES, HKV, HKV, D, cu, d_ctx, d_table), 1)   # reports a page index
        with pytest.raises(hb.HbError) as e:
            hb.hb_check()
        assert e.value.status == status
        hb.hb_check()


@pytest.mark.parametrize("rows", [[(1, 20), (1, 33), (1, 16)], [(1, 3 + i % 40) for i in range(300)],
                                  [(30, 40), (5, 5), (17, 100)]])
def test_bf16_append_with_tokens_of_no_sequence(rows):
    """New rows before the first sequence's and behind the last one's are
    written nowhere, as by hb_kv8_append."""
    from _gpu import bits
    from chunked_prefill_decode_gb300 import workloads
    from chunked_prefill_decode_gb300.device import from_layout
    from oracle import paged_attention as pa
    hb = lib()
    layout = workloads.layout_from_rows(workloads.Shape(4, 4, 64), rows, 61)
    g = torch.Generator().manual_seed(62)
    first, behind, T = 20, 9, layout.total_q
    kc, vc = (torch.randn(layout.num_pages, 16, 4, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    kn, vn = (torch.randn(first + T + behind, 4, 64, generator=g).to(torch.bfloat16) for _ in range(2))
    db = from_layout(layout, "cuda:0")
    # the rows may still grow: their tables name pages past the context too
    db.block_table.copy_(torch.where(db.block_table < 0, 0, db.block_table))
    db.cu_q_len.add_(first)
    db.batch.total_q = first + T + behind
    dk, dv = kc.cuda(), vc.cuda()
    hb.hb_kv_append(db.batch, kn.cuda(), vn.cuda(), dk, dv)
    hb.hb_check()
    wk, wv = pa.kv_append(bits(kc), bits(vc), bits(kn[first:first + T]), bits(vn[first:first + T]), layout.q_len,
                          layout.context_len, layout.block_table, 16)
    assert np.array_equal(bits(dk.cpu()), wk) and np.array_equal(bits(dv.cpu()), wv)
