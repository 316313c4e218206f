"""The 8-bit cache on the GPU: the quantising append byte for byte, and the
attention over it against fp64 with bounds derived from the formats."""
import math

import numpy as np
import pytest
import torch

from _gpu import sms
from _hbutil import lib
from _kv8 import Inputs, as_bytes, bits, bounds, check_out, same_bytes, step
from chunked_prefill_decode_gb300 import workloads
from chunked_prefill_decode_gb300.device import device_batch, from_layout
from chunked_prefill_decode_gb300.workloads import Shape, layout_from_rows
from oracle import kv8

pytestmark = pytest.mark.gpu

GEOMS = [(8, 8, 64), (32, 8, 128), (56, 8, 128)]
MORE_GEOMS = [(4, 4, 128), (16, 2, 64), (64, 16, 128), (32, 32, 128), (16, 1, 128), (8, 1, 64), (14, 2, 128)]


def check_append(layout, inp, cache):
    want = inp.oracle_append(layout)
    for got, w in zip(cache[:2], want[:2]):
        assert same_bytes(as_bytes(got), w)
    for got, w in zip(cache[2:], want[2:]):
        assert np.array_equal(got.cpu().numpy(), w)
    return want


def full_check(layout, seed=0, repeats=1, exps=(-9, -6), scale=None):
    inp = Inputs(layout, seed, exps)
    cache, out = step(layout, inp, scale=scale, repeats=repeats)
    want = check_append(layout, inp, cache)
    return check_out(out, *bounds(layout, inp, want, scale=scale))


# ------------------------------------------------------------------ append
ROWS = [[(1, 1)], [(1, 16)], [(1, 17), (1, 31), (1, 32)], [(2, 2), (15, 15), (16, 16), (17, 17)],
        [(16, 32), (17, 40), (33, 64), (5, 21)], [(1, 300), (130, 1000), (1, 5), (64, 64), (1, 2)]]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("geom", GEOMS + MORE_GEOMS)
def test_append(rows, geom):
    layout = layout_from_rows(Shape(*geom), rows, 3)
    inp = Inputs(layout, 5)
    hb = lib()
    db = from_layout(layout, "cuda:0")
    cache = inp.device()
    kn, vn = inp.k_new.cuda(), inp.v_new.cuda()
    hb.hb_kv8_append(db.batch, kn, vn, *cache)
    hb.hb_check()
    check_append(layout, inp, cache)
    # the same rows again change nothing
    before = [as_bytes(c) for c in cache]
    hb.hb_kv8_append(db.batch, kn, vn, *cache)
    hb.hb_check()
    assert all(np.array_equal(a, as_bytes(c)) for a, c in zip(before, cache))


def test_append_scales_that_grow_shrink_and_saturate():
    """Old exponents far above and below what the new tokens need; zeros,
    subnormal, huge and non-finite elements; the ends of the exponents' range."""
    layout = layout_from_rows(Shape(8, 4, 64), [(3, 10), (20, 37), (1, 16), (40, 40), (1, 9), (5, 5)], 4)
    for case, size in enumerate([1.0, 2.0 ** 40, 2.0 ** -40, 2.0 ** 100, 2.0 ** -120, 0.0]):
        inp = Inputs(layout, 10 + case, exps=(-30, 30))
        for x in (inp.k_new, inp.v_new):
            x.copy_((x.float() * size).to(torch.bfloat16))
            if case == 0:
                x[0, 0, 0], x[1, 1, 3], x[2, 2, 63] = float("inf"), float("-inf"), float("nan")
                x[5, 3, :] = float("nan")
                x[30:34, 1] = 0.0
                x[40, 0, :] = 448.0 * 2.0 ** -6      # exactly the border of an exponent
                x[41, 0, 5] = 2.0 ** 127
        hb = lib()
        db = from_layout(layout, "cuda:0")
        cache = inp.device()
        hb.hb_kv8_append(db.batch, inp.k_new.cuda(), inp.v_new.cuda(), *cache)
        hb.hb_check()
        check_append(layout, inp, cache)


def test_append_every_bf16_value():
    """All 65536 bf16 patterns, 16 tokens to a page: every value and rounding."""
    layout = layout_from_rows(Shape(8, 8, 128), [(64, 64)], 6)
    inp = Inputs(layout, 7)
    x = torch.from_numpy(np.arange(65536, dtype=np.uint16).view(np.int16)).view(torch.bfloat16)
    inp.k_new = x.view(64, 8, 128).clone()
    inp.v_new = x[torch.randperm(65536, generator=torch.Generator().manual_seed(1))].view(64, 8, 128).clone()
    # (near values share a page and head in k_new; v_new mixes all magnitudes)
    hb = lib()
    db = from_layout(layout, "cuda:0")
    cache = inp.device()
    hb.hb_kv8_append(db.batch, inp.k_new.cuda(), inp.v_new.cuda(), *cache)
    hb.hb_check()
    check_append(layout, inp, cache)


@pytest.mark.parametrize("n_seqs", [6143, 6144, 7000])
def test_append_with_many_sequences(n_seqs):
    layout = layout_from_rows(Shape(1, 1, 64), [(1 + i % 3, 3 + i % 50) for i in range(n_seqs)], 8)
    inp = Inputs(layout, 9)
    hb = lib()
    db = from_layout(layout, "cuda:0")
    cache = inp.device()
    hb.hb_kv8_append(db.batch, inp.k_new.cuda(), inp.v_new.cuda(), *cache)
    hb.hb_check()
    check_append(layout, inp, cache)


def test_append_reports_a_bad_page_and_writes_the_others():
    layout = layout_from_rows(Shape(8, 8, 64), [(1, 20), (5, 40), (1, 33)], 11)
    inp = Inputs(layout, 12)
    hb = lib()
    db = from_layout(layout, "cuda:0")
    good = db.block_table.clone()
    for bad in (-1, layout.num_pages, 2 ** 31 - 1):
        db.block_table.copy_(good)
        db.block_table[1, 2] = bad         # tokens 35 .. 39 of row 1: page 2 only
        cache = inp.device()
        hb.hb_kv8_append(db.batch, inp.k_new.cuda(), inp.v_new.cuda(), *cache)
        with pytest.raises(hb.HbError) as e:
            hb.hb_check()
        assert e.value.status == 6
        hb.hb_check()
        want = inp.oracle_append(layout)
        page = int(layout.block_table[1, 2])
        for got, w, old in zip(cache, want, inp.cache + inp.exps):
            w = np.array(w)
            w[page] = old[page]
            g = as_bytes(got) if got.dtype != torch.int8 else got.cpu().numpy()
            assert same_bytes(g, w) if got.dtype != torch.int8 else np.array_equal(g, w)


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("rows", [
    [(1, 1)], [(1, 16), (1, 17)], [(1, 128), (1, 129), (1, 2047)], [(2, 2), (15, 15), (17, 17)],
    [(127, 127), (128, 128), (129, 129)], [(257, 300), (16, 500)],
    [(1, 900), (64, 128), (1, 3), (5, 2000), (1, 1700)], [(3, 2051), (2, 9), (300, 1500)]])
@pytest.mark.parametrize("geom", GEOMS)
def test_rows(rows, geom):
    full_check(layout_from_rows(Shape(*geom), rows, 21), seed=22)


@pytest.mark.parametrize("geom", MORE_GEOMS)
def test_other_head_geometries(geom):
    full_check(layout_from_rows(Shape(*geom), [(1, 700), (1, 33), (40, 400), (130, 130), (1, 2500)], 23), seed=24)


@pytest.mark.parametrize("window", [1, 7, 16, 100, 1000, 5000])
@pytest.mark.parametrize("geom", GEOMS)
def test_sliding_window(window, geom):
    sh = Shape(*geom, sliding_window=window)
    full_check(layout_from_rows(sh, [(1, 1500), (1, 15), (70, 900), (1, 2049), (33, 33)], 25), seed=26)


def test_window_never_reads_pages_below_it():
    """Table entries and pages below every window may be stale."""
    sh = Shape(32, 8, 128, sliding_window=100)
    layout = layout_from_rows(sh, [(1, 1000), (40, 777), (1, 116)], 27)
    inp = Inputs(layout, 28)
    want = inp.oracle_append(layout)
    ref, tol = bounds(layout, inp, want)
    for s in range(3):
        low = int(layout.context_len[s]) - int(layout.q_len[s]) - 100 + 1
        layout.block_table[s, :max(0, low // 16)] = -1
    _, out = step(layout, inp)
    check_out(out, ref, tol)


@pytest.mark.parametrize("exps", [(-64, -60), (-20, 8), (30, 34), (-3, -3)])
def test_spread_of_scales(exps):
    """Pages whose scales differ by many powers of two, in K (one page takes
    the softmax over) and in V (a page of tiny values holds the weight)."""
    layout = layout_from_rows(Shape(16, 4, 128), [(1, 400), (1, 33), (30, 200), (1, 1200)], 29)
    inp = Inputs(layout, 30)
    g = np.random.default_rng(31)
    held = workloads.cached_slot_mask(layout).any(1)
    shape = (layout.num_pages, 4)
    inp.exps[1] = np.where(held[:, None], g.integers(exps[0], exps[1] + 1, shape), 99).astype(np.int8)
    inp.exps[0] = np.where(held[:, None], g.integers(-14, -5, shape), 99).astype(np.int8)
    inp.v_new = (inp.v_new.float() * 2.0 ** ((exps[0] + exps[1]) / 2 + 8)).to(torch.bfloat16)
    cache, out = step(layout, inp)
    want = check_append(layout, inp, cache)
    check_out(out, *bounds(layout, inp, want))


def test_exponents_outside_the_range_are_held_to_it():
    layout = layout_from_rows(Shape(8, 2, 64), [(1, 100), (20, 60)], 32)
    inp = Inputs(layout, 33)
    cache = inp.oracle_append(layout)
    cache[2][:, 0], cache[3][:, 1] = -128, 127
    inp.cache, inp.exps = list(cache[:2]), list(cache[2:])
    inp.q = (inp.q.float() * 2.0 ** -6).to(torch.bfloat16)
    _, out = step(layout, inp, append=False)
    check_out(out, *bounds(layout, inp, cache))


def test_constant_v_returns_it():
    """Every V element 0.75: a weighted mean of it is 0.75."""
    layout = layout_from_rows(Shape(32, 8, 128), [(1, 500), (1, 3000), (200, 900), (17, 17)], 34)
    inp = Inputs(layout, 35)
    cache = list(inp.oracle_append(layout))
    mask = np.zeros((layout.num_pages, 16), bool)
    for s in range(4):
        for p in range(int(layout.context_len[s])):
            mask[layout.block_table[s, p // 16], p % 16] = True
    cache[1] = np.where(mask[:, :, None, None], np.full_like(cache[1], kv8.encode(0.75 * 2.0 ** 8)), np.uint8(0x7F))
    cache[3] = np.full_like(cache[3], -8)
    inp.cache, inp.exps = cache[:2], cache[2:]
    _, out = step(layout, inp, append=False)
    # exact 0.75; weights and their sum round apart by 2^-8 at most, the output by half a step
    assert (out.float() - 0.75).abs().max() <= 0.75 * 2 * 2.0 ** -8


@pytest.mark.parametrize("geom", [(3, 3, 128), (6, 3, 64), (48, 3, 128), (5, 5, 64), (12, 6, 128), (14, 7, 64),
                                  (64, 4, 128), (32, 2, 128), (16, 1, 64), (128, 8, 128), (64, 32, 64)])
def test_any_number_of_kv_heads(geom):
    """Heads that do not divide the eight consumer warps, and groups of more
    than 8 q heads, alone and shared by several pages of a stage."""
    full_check(layout_from_rows(Shape(*geom), [(1, 1), (1, 17), (1, 530), (1, 1600), (33, 200)], 51), seed=52)


@pytest.mark.parametrize("geom", [(32, 8, 128), (8, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("rows", [1, 2, 3, 5, 9, 40, 150])
def test_few_and_many_decode_rows(geom, rows):
    """The plan gives few rows blocks of fewer kv heads, cut into many pieces."""
    full_check(layout_from_rows(Shape(*geom), [(1, 900 + 37 * i % 400) for i in range(rows)], 53), seed=rows)


def test_what_a_row_may_not_see_may_be_nan():
    """NaN values below a decode row's window, and q rows of NaN and infinity:
    no other row, head or sequence changes."""
    sh = Shape(8, 2, 128, sliding_window=40)
    layout = layout_from_rows(sh, [(1, 100), (1, 70), (20, 64)], 54)
    inp = Inputs(layout, 55)
    cache = list(inp.oracle_append(layout))
    inp.cache, inp.exps = cache[:2], cache[2:]
    ref, tol = bounds(layout, inp, cache)
    for s, low in ((0, 60), (1, 30)):
        for pos in range(low):
            cache[0][layout.block_table[s, pos // 16], pos % 16] = 0x7F
            cache[1][layout.block_table[s, pos // 16], pos % 16] = 0xFF
    inp.cache = cache[:2]
    _, out = step(layout, inp, append=False)
    check_out(out, ref, tol)
    inp.q[0, 3], inp.q[5, 1, 7] = float("nan"), float("inf")
    _, out = step(layout, inp, append=False)
    hit = np.zeros(out.shape[:2], bool)
    hit[0, 3] = hit[5, 1] = True
    got = out.float().cpu().numpy()
    assert np.isnan(got[0, 3]).all() and not np.isfinite(got[5, 1]).any()
    check_out(torch.from_numpy(np.where(hit[:, :, None], 0.0, got)), np.where(hit[:, :, None], 0.0, ref), tol)


def test_one_workspace_for_batches_in_turn():
    """A workspace sized for the larger of two batches, planned for each in
    turn: nothing of one batch's plan, counters or pages stays for the other."""
    hb = lib()
    work, ws = [], None
    for s, rows in ((56, [(1, 1500), (90, 700), (1, 33), (40, 40)]), (57, [(200, 1000), (1, 2000), (1, 5), (1, 900)])):
        layout = layout_from_rows(Shape(32, 8, 128), rows, s)
        inp = Inputs(layout, s)
        work.append((layout, inp, from_layout(layout, "cuda:0"), inp.device(), inp.q.cuda(), inp.k_new.cuda(),
                     inp.v_new.cuda(), []))
    for layout, _, db, *_ in work:
        need = hb.hb_plan_sizes(db.batch, db.q_len, db.context_len, sms(), kv8=True)[1]
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if ws is None or ws.numel() < need else ws
    for _ in range(15):
        for _, _, db, cache, q, kn, vn, outs in work:
            out = torch.empty_like(q)
            plan, w = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms(), workspace=ws)
            assert w is ws
            hb.hb_kv8_append(db.batch, kn, vn, *cache)
            hb.hb_kv8_attention(db.batch, plan, q, *cache, 1.0 / math.sqrt(128), out, ws)
            outs.append(out)
    hb.hb_check()
    for layout, inp, _, cache, _, _, _, outs in work:
        ref, tol = bounds(layout, inp, check_append(layout, inp, cache))
        for out in outs:
            check_out(out, ref, tol)


def test_plan_is_reused_and_results_repeat():
    layout = layout_from_rows(Shape(32, 8, 128), [(1, 3000), (100, 700), (1, 40)], 36)
    inp = Inputs(layout, 37)
    _, a = step(layout, inp)
    _, b = step(layout, inp, repeats=4)
    ref, tol = bounds(layout, inp, inp.oracle_append(layout))
    check_out(a, ref, tol)
    check_out(b, ref, tol)


def test_bad_page_is_reported():
    layout = layout_from_rows(Shape(32, 8, 128), [(1, 200), (40, 300)], 40)
    inp = Inputs(layout, 41)
    hb = lib()
    for row, col in ((0, 3), (1, 5)):
        bad = layout.block_table.copy()
        bad[row, col] = layout.num_pages
        lay = workloads.BatchLayout(layout.shape, layout.q_len, layout.context_len, bad, layout.num_pages)
        step(lay, inp, check=False, append=False)
        with pytest.raises(hb.HbError) as e:
            hb.hb_check()
        assert e.value.status == 6
        hb.hb_check()


def test_captured_and_replayed():
    layout = layout_from_rows(Shape(32, 8, 128), [(1, 3000)] * 5 + [(1, 700), (40, 300)], 42)
    inp = Inputs(layout, 43)
    hb = lib()
    db = from_layout(layout, "cuda:0")
    q, kn, vn = inp.q.cuda(), inp.k_new.cuda(), inp.v_new.cuda()
    cache, scale = inp.device(), 1.0 / math.sqrt(128)
    plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
    out = torch.full_like(q, float("nan"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        hb.hb_kv8_append(db.batch, kn, vn, *cache)
        hb.hb_kv8_attention(db.batch, plan, q, *cache, scale, out, ws)
    ref, tol = bounds(layout, inp, inp.oracle_append(layout))
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        hb.hb_check()
        check_out(out, ref, tol)
    check_append(layout, inp, cache)


def test_two_streams_at_once():
    """Two batches over one cache, each with its own workspace and stream."""
    hb = lib()
    layouts = [layout_from_rows(Shape(32, 8, 128), [(1, 2000), (60, 500), (1, 900)], s) for s in (44, 45)]
    work = []
    for i, layout in enumerate(layouts):
        inp = Inputs(layout, 46 + i)
        db = from_layout(layout, "cuda:0")
        cache = inp.device()
        plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
        work.append((layout, inp, db, cache, plan, ws, inp.q.cuda(), inp.k_new.cuda(), inp.v_new.cuda(),
                     torch.empty_like(inp.q, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, db, cache, plan, ws, q, kn, vn, out, st in work:
            with torch.cuda.stream(st):
                hb.hb_kv8_append(db.batch, kn, vn, *cache)
                hb.hb_kv8_attention(db.batch, plan, q, *cache, 1.0 / math.sqrt(128), out, ws)
    torch.cuda.synchronize()
    hb.hb_check()
    for layout, inp, _, cache, _, _, _, _, _, out, _ in work:
        check_out(out, *bounds(layout, inp, check_append(layout, inp, cache)))


@pytest.mark.parametrize("seed", range(10))
def test_random_batches(seed):
    rng = np.random.default_rng(500 + seed)
    geom = (GEOMS + MORE_GEOMS)[seed]
    rows = [(1, int(rng.integers(1, 2500))) for _ in range(int(rng.integers(0, 12)))]
    for _ in range(int(rng.integers(1, 4))):
        q = int(rng.integers(2, 300))
        rows.append((q, q + int(rng.integers(0, 1500))))
    rng.shuffle(rows)
    window = int(rng.choice([0, 0, 5, 300]))
    full_check(layout_from_rows(Shape(*geom, sliding_window=window), [tuple(r) for r in rows], 500 + seed),
               seed=seed)


def test_long_context_and_a_pool_past_32_bits():
    """A context of 70000 tokens in pages at the far end of a pool of more than
    2^31 elements (and bytes), decode row and chunk."""
    hb = lib()
    shape, page_elems = Shape(8, 8, 128), 16 * 8 * 128
    num_pages = 2 ** 31 // page_elems + 9000
    n = -(-70000 // 16)
    rows = [(1, 70000), (20, 30000)]
    ctx = np.array([c for _, c in rows], np.int32)
    table = np.full((2, n), -1, np.int32)
    table[0] = num_pages - 1 - np.arange(n)
    table[1, :1875] = num_pages - 1 - n - np.arange(1875)
    db = device_batch(np.array([1, 20], np.int32), ctx, table, num_pages, 8, 8, 128, 16, "cuda:0")
    g = torch.Generator("cuda").manual_seed(48)
    cache = hb.kv8_cache(num_pages, 8, 128)
    first = num_pages - n - 1875 - 8
    for c in cache[:2]:
        x = torch.randn(num_pages - first, 16, 8, 128, generator=g, device="cuda") * 100
        c[first:] = x.clamp_(-448, 448).to(torch.float8_e4m3fn)
    for e in cache[2:]:
        e.fill_(-8)
    q = torch.randn(21, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    kn, vn = (torch.randn(21, 8, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    hb.hb_kv8_append(db.batch, kn, vn, *cache)
    plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
    out = torch.empty_like(q)
    hb.hb_kv8_attention(db.batch, plan, q, *cache, 1.0 / math.sqrt(128), out, ws)
    hb.hb_check()
    # the oracle on the far pages alone, renumbered
    small = [as_bytes(c[first:]) for c in cache[:2]] + [e[first:].cpu().numpy() for e in cache[2:]]
    layout = workloads.BatchLayout(shape, np.array([1, 20], np.int32), ctx,
                                   np.where(table >= 0, table - first, -1).astype(np.int32), num_pages - first)

    class Inp:
        pass
    inp = Inp()
    inp.q = q.cpu()
    check_out(out, *bounds(layout, inp, small))
    # the appended tokens landed there
    last = kv8.values(small[0], small[2])[table[0, 69999 // 16] - first, 69999 % 16]
    new = kn[0].double().cpu().numpy()
    assert np.abs(last - new).max() <= 2.0 ** -4 * np.abs(new).max()


@pytest.mark.parametrize("name", ["mistral_b512", "yi_b2048", "decode_only"])
def test_full_size_workloads(name):
    """The benchmark batches: sampled sequences and tokens against fp64."""
    hb = lib()
    layout = workloads.WORKLOADS[name]()
    sh = layout.shape
    g = torch.Generator("cuda").manual_seed(49)
    db = from_layout(layout, "cuda:0")
    cache = hb.kv8_cache(layout.num_pages, sh.num_kv_heads, sh.head_dim)
    for c in cache[:2]:
        for a in range(0, layout.num_pages, 8192):
            x = torch.randn(min(8192, layout.num_pages - a), 16, sh.num_kv_heads, sh.head_dim, generator=g,
                            device="cuda")
            c[a:a + 8192] = (x * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    for e in cache[2:]:
        e.copy_(torch.randint(-9, -6, e.shape, generator=g, device="cuda"))
    T = layout.total_q
    q = torch.randn(T, sh.num_q_heads, sh.head_dim, generator=g, device="cuda").to(torch.bfloat16)
    kn, vn = (torch.randn(T, sh.num_kv_heads, sh.head_dim, generator=g, device="cuda").to(torch.bfloat16)
              for _ in range(2))
    scale = 1.0 / math.sqrt(sh.head_dim)
    hb.hb_kv8_append(db.batch, kn, vn, *cache)
    plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
    out = torch.full_like(q, float("nan"))
    hb.hb_kv8_attention(db.batch, plan, q, *cache, scale, out, ws)
    hb.hb_check()
    assert torch.isfinite(out.float()).all()
    rng = np.random.default_rng(50)
    seqs = sorted(set(rng.choice(layout.num_seqs, 5, replace=False)) | {layout.num_seqs - 1})
    cu = layout.cu_q_len
    for s in seqs:
        n, c = int(layout.q_len[s]), int(layout.context_len[s])
        pages = torch.from_numpy(layout.block_table[s, :-(-c // 16)].astype(np.int64)).cuda()
        small = [as_bytes(x.view(torch.uint8)[pages]) for x in cache[:2]] + [e[pages].cpu().numpy() for e in cache[2:]]
        sub = workloads.BatchLayout(sh, layout.q_len[s:s + 1], layout.context_len[s:s + 1],
                                    np.arange(len(pages), dtype=np.int32)[None], len(pages))

        class Inp:
            pass
        inp = Inp()
        inp.q = q[cu[s]:cu[s] + n].cpu()
        tok = None if n == 1 else np.unique(np.concatenate([[0, n - 1], rng.choice(n, 12)]))
        ref, tol = bounds(sub, inp, small, tokens=tok)
        check_out(out[cu[s]:cu[s] + n], ref, tol, tokens=tok)


@pytest.mark.parametrize("geom", [(16, 4, 128), (8, 1, 64)])
def test_scales_at_both_ends_of_the_range(geom):
    """Pages whose V scales are 2^64 and 2^-64: the values of the latter vanish
    beside the former's, their weights do not.  (Those come as 2^(x - M) down to
    2^-136, 13 bits of a number below 2^-126, so they are good to 2^-14, which
    lies inside the 2^-8 - 2^-11 that `bounds` grants fp16 weights too much.)"""
    layout = layout_from_rows(Shape(*geom), [(1, 400), (1, 33), (30, 200), (1, 3000), (1, 1200)], 58)
    inp = Inputs(layout, 59)
    cache = list(inp.oracle_append(layout))
    g = np.random.default_rng(60)
    cache[3] = g.choice([-64, 64], cache[3].shape).astype(np.int8)
    inp.cache, inp.exps = cache[:2], cache[2:]
    _, out = step(layout, inp, append=False)
    check_out(out, *bounds(layout, inp, cache))


@pytest.mark.parametrize("rows", [[(1, 20), (1, 33), (1, 16)], [(1, 3 + i) for i in range(40)],
                                  [(30, 40), (5, 5), (17, 100)]])
def test_append_with_tokens_of_no_sequence(rows):
    """New rows before the first sequence's and behind the last one's: not read,
    whatever they hold, and written nowhere."""
    layout = layout_from_rows(Shape(8, 4, 64), rows, 61)
    inp = Inputs(layout, 62)
    hb = lib()
    db = from_layout(layout, "cuda:0")
    cache = inp.device()
    first, behind = 20, 9
    new = [torch.cat([torch.full((first, 4, 64), float("inf")), x.float(), torch.full((behind, 4, 64), 1e30)])
           .to(torch.bfloat16).cuda() for x in (inp.k_new, inp.v_new)]
    db.cu_q_len.add_(first)
    db.batch.total_q = layout.total_q + first + behind
    hb.hb_kv8_append(db.batch, *new, *cache)
    hb.hb_check()
    check_append(layout, inp, cache)


def test_a_plan_that_is_read_only():
    hb = lib()
    layout = layout_from_rows(Shape(8, 8, 64), [(1, 40), (20, 60)], 63)
    inp = Inputs(layout, 64)
    cache = inp.oracle_append(layout)
    inp.cache, inp.exps = list(cache[:2]), list(cache[2:])
    db = from_layout(layout, "cuda:0")
    plan, ws = hb.hb_kv8_plan(db.batch, db.q_len, db.context_len, sms())
    plan.flags.writeable = False
    ref, tol = bounds(layout, inp, cache)
    out = torch.full_like(inp.q, float("nan"), device="cuda")
    hb.hb_kv8_attention(db.batch, plan, inp.q.cuda(), *inp.device(), 1.0 / math.sqrt(64), out, ws)
    hb.hb_check()
    check_out(out, ref, tol)
