"""The 8-bit attention under scales that lie far apart, held to bounds of each
row, head and dimension by itself (_kv8_rows.py)."""
import numpy as np
import pytest
import torch

from _kv8 import Inputs, check_out, step
from _kv8_rows import row_bounds
from chunked_prefill_decode_gb300 import workloads
from chunked_prefill_decode_gb300.workloads import Shape, layout_from_rows
from oracle import kv8

pytestmark = pytest.mark.gpu

ROWS = [(1, 400), (1, 33), (30, 200), (1, 3000), (1, 1200)]


def cached(layout, inp):
    """The input's cache with the new tokens in it."""
    cache = [np.array(a) for a in inp.oracle_append(layout)]
    inp.cache, inp.exps = cache[:2], cache[2:]
    return cache


def attend(layout, inp, cache):
    _, out = step(layout, inp, append=False)
    ref, tol = row_bounds(layout, inp, cache)
    return check_out(out, ref, tol)


@pytest.mark.parametrize("above", [0, 12, 20, 24, 28, 40, 60])
@pytest.mark.parametrize("geom,window", [((16, 4, 128), 0), ((8, 1, 64), 0), ((56, 8, 128), 0), ((16, 4, 128), 1000)])
def test_one_large_value_costs_the_other_dimensions_nothing(geom, window, above):
    """One page of each row and head whose V scale one element has driven up
    2^above times (the others of that page are zero under it): the element's
    own key has next to no weight, or has left the window, its neighbours have
    theirs.  Every other dimension stays as exact as without it."""
    layout = layout_from_rows(Shape(*geom, sliding_window=window), ROWS, 70)
    inp = Inputs(layout, 71)
    cache = cached(layout, inp)
    g = geom[0] // geom[1]
    q = inp.q.double().numpy()
    tok = 0
    for s in range(layout.num_seqs):
        n, ctx = int(layout.q_len[s]), int(layout.context_len[s])
        # the last page whose first slot lies below the window of the last row, or a middle one
        lp = (ctx - window) // 16 if window and ctx > window else ctx // 32
        page, slot = layout.block_table[s, lp], 0
        for h in range(geom[1]):
            cache[1][page, :, h] = 0
            cache[1][page, slot, h, 5] = kv8.encode(448.0)
            cache[3][page, h] = -8 + above
            # (a key that points away from the mean of the heads' queries)
            away = -q[tok + n - 1, h * g:(h + 1) * g].mean(0)
            cache[0][page, slot, h] = kv8.encode(np.clip(away * 400, -448, 448))
        tok += n
    inp.cache, inp.exps = cache[:2], cache[2:]
    attend(layout, inp, cache)


@pytest.mark.parametrize("lo,hi", [(-9, -6), (-20, 8), (-60, -30), (0, 60)])
@pytest.mark.parametrize("geom", [(16, 4, 128), (8, 1, 64), (8, 8, 64), (64, 4, 128), (32, 8, 128)])
def test_scales_of_all_sizes(geom, lo, hi):
    layout = layout_from_rows(Shape(*geom), ROWS, 72)
    inp = Inputs(layout, 73)
    cache = cached(layout, inp)
    g = np.random.default_rng(74)
    cache[3] = g.integers(lo, hi + 1, cache[3].shape).astype(np.int8)
    inp.exps[1] = cache[3]
    attend(layout, inp, cache)


@pytest.mark.parametrize("step_", [-3, -1, 1, 3])
@pytest.mark.parametrize("geom", [(16, 4, 128), (8, 1, 64)])
def test_scales_that_rise_or_fall_along_a_row(geom, step_):
    """Page after page's V scale 2^step_ times the one before (up to 2^60
    apart), with V zero in every second dimension of every second page."""
    layout = layout_from_rows(Shape(*geom), [(1, 330), (1, 700), (1, 20), (20, 300)], 75)
    inp = Inputs(layout, 76)
    cache = cached(layout, inp)
    for s in range(layout.num_seqs):
        for lp in range(-(-int(layout.context_len[s]) // 16)):
            page = layout.block_table[s, lp]
            cache[3][page] = (-30 if step_ > 0 else 30) + step_ * (lp % 20)
            if lp % 2:
                cache[1][page, :, :, ::2] = 0
    inp.cache, inp.exps = cache[:2], cache[2:]
    attend(layout, inp, cache)


def test_a_key_that_takes_nearly_all_the_weight():
    """One key per head that points along one of its queries, first, last or in
    the middle of the row: the others' weights lie far below its own."""
    layout = layout_from_rows(Shape(16, 4, 128), [(1, 500), (1, 500), (1, 500), (1, 1100)], 77)
    inp = Inputs(layout, 78)
    cache = cached(layout, inp)
    q = inp.q.double().numpy()
    for s, pos in enumerate((3, 250, 498, 700)):
        page = layout.block_table[s, pos // 16]
        for h in range(4):
            cache[0][page, pos % 16, h] = kv8.encode(np.clip(q[s, 4 * h + h] * 100 * (1 + s), -448, 448))
    inp.cache, inp.exps = cache[:2], cache[2:]
    attend(layout, inp, cache)


def test_each_exponent_outside_the_range_is_held_to_it():
    """K and V exponents of -128 and 127, a head each, with queries sized so that
    2^64 and 2^127 (2^-64 and 2^-128) give other weights: every head held to a
    bound that is a small part of its own answer."""
    layout = layout_from_rows(Shape(8, 4, 64), [(1, 100), (20, 60), (1, 700)], 79)
    inp = Inputs(layout, 80)
    cache = cached(layout, inp)
    cache[2][:, 0], cache[2][:, 1], cache[3][:, 2], cache[3][:, 3] = 127, -128, 127, -128
    inp.exps = cache[2:]
    q = inp.q.float()
    q[:, 0:2] *= 2.0 ** -71
    q[:, 2:4] *= 2.0 ** 57
    inp.q = q.to(torch.bfloat16)
    ref, tol = row_bounds(layout, inp, cache)
    held = workloads.cached_slot_mask(layout)
    for h in range(4):
        v = np.abs(kv8.values(cache[1], cache[3]))[held][:, h].mean()
        assert tol[:, 2 * h:2 * h + 2].max() < 0.05 * v
    # what other readings of the exponents would give lies outside the bound
    for which, head in ((2, 0), (2, 1)):
        e = cache[which].astype(np.int64)
        x = kv8.decode(cache[0]) * 2.0 ** e[:, None, :, None].astype(np.float64)
        other = kv8.pa.attention(inp.q.double().numpy(), x, kv8.values(cache[1], cache[3]), layout.q_len,
                                 layout.context_len, layout.block_table, 16, 8, 4, 0.125)
        off = np.abs(other - ref)[:, 2 * head:2 * head + 2] > 4 * tol[:, 2 * head:2 * head + 2]
        assert off.mean() > 0.5
    _, out = step(layout, inp, append=False)
    check_out(out, ref, tol)
