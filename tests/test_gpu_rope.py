"""hb_rope on the GPU against its definition in 64 bits.

Tolerance: one rounding to bf16 (2^-8 of the value).  Before it, in fp32 and
relative to 2^-24 (|a| + |b|) factor of a pair's members after their norm: the
angle (32 bits turned into a float, half a turn: pi), the sine and cosine (4),
products, sum and factor (6); a head norm adds a chain of 16 squares, a tree
and a root (20, halved, and 5).  40 covers them."""
import math

import numpy as np
import pytest
import torch

from _hbutil import lib
from _turns import exact_angles, exact_turns
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ULP = 2.0 ** -24
EPS = 1e-5


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


class Step:
    """A batch of rows (q_len, context_len) with `spare` token rows behind it."""

    def __init__(self, rows, hq, hkv, d, seed=0, spare=0, fused=False, extra_pages=3):
        hb = lib()
        g = torch.Generator("cuda").manual_seed(seed)
        self.rows, self.shape = rows, (hq, hkv, d)
        q = np.array([r[0] for r in rows])
        ctx = np.array([r[1] for r in rows])
        self.cu = np.concatenate([[0], np.cumsum(q)])
        T = self.T = int(q.sum()) + spare
        # only the pages that new tokens stand on are in the pool; the table names nothing else
        first, last = (ctx - q) // 16, -(-ctx // 16)
        n = np.where(q > 0, last - first, 0)
        self.num_pages = int(n.sum()) + extra_pages
        perm = np.random.default_rng(seed).permutation(self.num_pages)
        self.table = np.full((len(rows), max(1, int(last.max()))), -1, np.int32)
        at = 0
        for i in range(len(rows)):
            self.table[i, first[i]:first[i] + n[i]] = perm[at:at + n[i]]
            at += n[i]
        if fused:
            qkv = randn(g, T, hq + 2 * hkv, d)
            self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            self.q, self.k, self.v = randn(g, T, hq, d), randn(g, T, hkv, d), randn(g, T, hkv, d)
        self.kc, self.vc = (randn(g, self.num_pages, 16, hkv, d) for _ in range(2))
        self.dev = [torch.from_numpy(a.astype(np.int32)).cuda() for a in (self.cu, ctx, self.table)]
        self.batch = hb.make_batch(len(rows), T, self.table.shape[1], self.num_pages, hq, hkv, d, *self.dev)
        self.weights = [1 + 0.3 * randn(g, d) for _ in range(2)]

    def positions(self):
        """(token, position, row) of every token that belongs to a sequence."""
        tok, pos, row = [], [], []
        for i, (n, c) in enumerate(self.rows):
            tok += range(self.cu[i], self.cu[i] + n)
            pos += range(c - n, c)
            row += [i] * n
        return np.array(tok, np.int64), np.array(pos, np.int64), np.array(row, np.int64)


def f64(t):
    return t.double().cpu().numpy()


def angles(rot, pos, **kw):
    """Exact: position times phase, modulo a turn."""
    phases = lib().rope_phases(rot, **kw)
    return np.array([[(int(p) * int(f) % 2 ** 64) / 2 ** 64 * 2 * math.pi for f in phases] for p in pos]).reshape(
        len(pos), rot // 2)


def expected(x, w, angle, interleaved, factor):
    """(value, bound) of heads x [n, h, d]."""
    x = f64(x)
    if w is not None:
        x = ob.rms_norm(x, f64(w), EPS)
    want = ob.rotate(x, angle[:, None, :], interleaved, factor)
    rot, size = 2 * angle.shape[-1], np.abs(x)
    pair = np.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    pair[..., a] = pair[..., b] = (size[..., a] + size[..., b]) * abs(factor)
    if w is not None:
        pair[..., rot:] = size[..., rot:]
    return want, 2.0 ** -8 * np.abs(want) + 40 * ULP * (1 + 2.0 ** -8) * pair


def check(got, want):
    want, bound = want
    got = f64(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), f"worst excess {(np.abs(got - want) - bound).max():.3e}"


def run(st, rot, interleaved=False, factor=1.0, norms=(True, True), cached=True, k_out="new", q_out="new", stream=None,
        **kw):
    hb = lib()
    rope = hb.make_rope(rot, interleaved=interleaved, factor=factor, eps=EPS, q_weight=st.weights[0] if norms[0] else None,
                        k_weight=st.weights[1] if norms[1] else None, **kw)
    outs = [{"new": torch.full(x.shape, 7.0, dtype=BF, device="cuda"), "same": x, "none": None}[how]
            for how, x in ((q_out, st.q), (k_out, st.k))]
    hb.hb_rope(st.batch, rope, st.q, st.k, st.v if cached else None, *outs, st.kc if cached else None,
               st.vc if cached else None, stream=stream)
    return outs


def check_step(st, rot, interleaved=False, factor=1.0, norms=(True, True), **kw):
    """A call into new arrays and the cache, against the definition."""
    hb = lib()
    kc0, vc0 = st.kc.clone(), st.vc.clone()
    q, k = run(st, rot, interleaved, factor, norms, **kw)
    hb.hb_check()
    tok, pos, row = st.positions()
    angle = angles(rot, pos, **kw) if rot else np.zeros((len(pos), 0))
    t = torch.from_numpy(tok).cuda()
    check(q[t], expected(st.q[t], st.weights[0] if norms[0] else None, angle, interleaved, factor))
    check(k[t], expected(st.k[t], st.weights[1] if norms[1] else None, angle, interleaved, factor))
    # tokens of no sequence: as they were
    rest = torch.ones(st.T, dtype=torch.bool, device="cuda")
    rest[t] = False
    assert (q[rest] == 7).all() and (k[rest] == 7).all()
    # the pages: k as in k_out, v as given, nothing else
    page = torch.from_numpy(st.table[row, pos // 16].astype(np.int64)).cuda()
    slot = torch.from_numpy(pos % 16).cuda()
    kc0[page, slot], vc0[page, slot] = k[t], st.v[t]
    assert torch.equal(st.kc, kc0) and torch.equal(st.vc, vc0)
    return q, k


ROWS = [(1, 1), (1, 16), (1, 17), (5, 5), (17, 40), (1, 100000), (33, 1001), (2, 1 << 20)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (32, 8, 128), (7, 1, 128), (16, 1, 64), (56, 8, 128), (32, 16, 128), (128, 16, 128)])
def test_against_the_definition(hq, hkv, d, interleaved):
    for i, rot in enumerate((d, d // 2, 16, 48, 0)):
        st = Step(ROWS, hq, hkv, d, seed=i, spare=i % 3, fused=bool(i % 2))
        check_step(st, rot, interleaved, [1.0, 1.3, -0.5][i % 3], [(False, False), (True, True), (True, False), (False, True)][i % 4])


@pytest.mark.parametrize("kw", [dict(base=1e6), dict(scaling="linear", scale_by=8.0), dict(scaling="base", scale_by=4.0),
                                dict(scaling="parts", scale_by=16.0, original_context=8192)])
def test_scaled_frequencies(kw):
    check_step(Step(ROWS, 8, 2, 128, seed=3), 128, norms=(False, False), **kw)


@pytest.mark.parametrize("rows", [[(1, 3)], [(2, 2)], [(1, 50)] * 300, [(700, 700), (1, 9), (650, 2000)], [(0, 5), (1, 5), (0, 0), (3, 20), (0, 7)]])
def test_few_and_many_rows(rows):
    check_step(Step(rows, 8, 2, 64, seed=4, spare=2), 64)
    check_step(Step(rows, 32, 8, 128, seed=5), 64, True, norms=(False, False))


def test_more_sequences_than_shared_memory_holds():
    for n in (5500, 5501, 9000):
        check_step(Step([(1, 1 + i % 40) for i in range(n)], 2, 1, 64, seed=6), 32, norms=(False, False))


@pytest.mark.parametrize("pos", [(1 << 24) + 1, (1 << 31) - 20])
def test_far_positions_lose_nothing(pos):
    """The angle is position times phase modulo a turn, whatever the position.
    (The table would have 2^27 entries: the call has no cache.)"""
    hb = lib()
    d, n = 64, 5
    st = Step([(n, 40)], 4, 2, d, seed=7)
    st.dev[1].fill_(pos + n)
    q, k = run(st, d, norms=(False, False), cached=False)
    hb.hb_check()
    angle = angles(d, range(pos, pos + n))
    check(q, expected(st.q, None, angle, False, 1.0))
    check(k, expected(st.k, None, angle, False, 1.0))


@pytest.mark.parametrize("norms", [(False, False), (True, True)])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("rot", [128, 32, 0])
def test_in_place_and_without_k_out_gives_the_same_bits(rot, fused, norms):
    hb = lib()
    make = lambda: Step(ROWS, 8, 2, 128, seed=8, spare=1, fused=fused)  # noqa: E731
    st = make()
    q, k = run(st, rot, norms=norms)
    tok = torch.from_numpy(st.positions()[0]).cuda()
    for q_out, k_out, cached in (("same", "same", True), ("same", "none", True), ("new", "same", False), ("same", "new", True)):
        b = make()
        q_was, k_was, v_was = b.q.clone(), b.k.clone(), b.v.clone()
        qb, kb = run(b, rot, norms=norms, q_out=q_out, k_out=k_out, cached=cached)
        assert torch.equal(qb[tok], q[tok]) and (kb is None or torch.equal(kb[tok], k[tok]))
        if cached:
            assert torch.equal(b.kc, st.kc) and torch.equal(b.vc, st.vc)
        # the last row belongs to no sequence
        assert torch.equal(b.q[-1], q_was[-1]) and torch.equal(b.k[-1], k_was[-1]) and torch.equal(b.v, v_was)
        if q_out == "new":
            assert torch.equal(b.q, q_was)
        if k_out != "same":
            assert torch.equal(b.k, k_was)
    hb.hb_check()


def test_pages_that_do_not_exist_are_skipped_and_reported():
    hb = lib()
    st = Step([(20, 40), (1, 33)], 8, 2, 64, seed=9)
    want = run(Step([(20, 40), (1, 33)], 8, 2, 64, seed=9), 64)
    kc0 = st.kc.clone()
    st.dev[2][0, 1] = -1
    st.dev[2][1, 2] = st.num_pages
    q, k = run(st, 64)
    with pytest.raises(hb.HbError) as e:
        hb.hb_check()
    assert e.value.status == 6
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    gone = st.table[[0, 1], [1, 2]]
    assert torch.equal(st.kc[gone.tolist()], kc0[gone.tolist()])
    hb.hb_check()


def test_positions_below_zero_are_reported():
    """(A context length that the device holds wrong.)"""
    hb = lib()
    st = Step([(20, 40), (1, 33)], 8, 2, 64, seed=9)
    st.dev[1][0] = 3
    q, _ = run(st, 64)
    with pytest.raises(hb.HbError) as e:
        hb.hb_check()
    assert e.value.status == 6
    assert (q[:17] == 7).all() and (q[17:] != 7).any()


def test_values_that_are_not_finite_stay_in_their_pair():
    st = Step([(3, 30)], 8, 2, 64, seed=10)
    st.q[1, 2, 5] = float("inf")
    st.k[0, 1, 40] = float("nan")
    q, k = run(st, 64, norms=(False, False))
    bad = (~torch.isfinite(q)).nonzero().tolist()
    assert bad and all(i[:2] == [1, 2] and i[2] in (5, 37) for i in bad)
    bad = (~torch.isfinite(k)).nonzero().tolist()
    assert bad and all(i[:2] == [0, 1] and i[2] in (8, 40) for i in bad)


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 and tokens 2^31 elements apart."""
    hb = lib()
    hkv, d, pages = 1, 64, (1 << 21) + 70000
    st = Step([(20, 40)], 2, hkv, d, seed=11)
    st.kc, st.vc = (torch.zeros(pages, 16, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    at = torch.tensor([pages - 1, 3, pages - 60000], dtype=torch.int32, device="cuda")
    st.dev[2][0] = at
    st.batch.num_pages = pages
    q, k = run(st, 64)
    hb.hb_check()
    for i, p in enumerate(range(20, 40)):
        assert torch.equal(st.kc[at[p // 16], p % 16], k[i]) and torch.equal(st.vc[at[p // 16], p % 16], st.v[i])
    gap = (1 << 31) + 64
    big = torch.empty(2 * gap + 128, dtype=BF, device="cuda").as_strided((3, 2, 64), (gap, 64, 1))
    st = Step([(3, 9)], 2, 1, 64, seed=12)
    want = run(st, 64)[0]
    big.copy_(st.q)
    st.q = big
    got = run(st, 64, q_out="same")[0]
    assert torch.equal(got, want)


def test_captured_replayed_and_on_another_stream():
    hb = lib()
    st = Step(ROWS, 8, 2, 128, seed=13)
    rope = hb.make_rope(128, q_weight=st.weights[0], k_weight=st.weights[1], eps=EPS)
    q, k = torch.empty_like(st.q), torch.empty_like(st.k)
    call = lambda **kw: hb.hb_rope(st.batch, rope, st.q, st.k, st.v, q, k, st.kc, st.vc, **kw)  # noqa: E731
    call()
    want = q.clone(), k.clone(), st.kc.clone()
    side = torch.cuda.Stream()
    q.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    assert torch.equal(q, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        q.zero_(), k.zero_(), st.kc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # replayed for the step after: the lengths are read on the device
    st.dev[1][5] -= 1
    graph.replay()
    torch.cuda.synchronize()
    row = int(st.cu[5])
    assert not torch.equal(q[row], want[0][row]) and torch.equal(q[:row], want[0][:row])
    hb.hb_check()


def test_rotated_cache_feeds_the_attention():
    """hb_rope into the cache, then the attention over it: as with rows that were
    rotated before and appended."""
    hb = lib()
    hq, hkv, d = 8, 2, 128
    rows = [(1, 40), (21, 21), (1, 7), (40, 90)]
    st = Step(rows, hq, hkv, d, seed=14)
    # every page of a context is needed here
    maxp = max(-(-c // 16) for _, c in rows)
    n = maxp * len(rows)
    table = torch.randperm(n, device="cuda").to(torch.int32).view(len(rows), maxp).contiguous()
    g = torch.Generator("cuda").manual_seed(15)
    kc, vc = randn(g, n, 16, hkv, d), randn(g, n, 16, hkv, d)
    batch = hb.make_batch(len(rows), st.T, maxp, n, hq, hkv, d, st.dev[0], st.dev[1], table)
    rope = hb.make_rope(d)
    ql, cl = np.array([r[0] for r in rows], np.int32), np.array([r[1] for r in rows], np.int32)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan, ws = hb.hb_plan(batch, ql, cl, sms)
    outs = []
    for fused in (True, False):
        k2, v2 = kc.clone(), vc.clone()
        q, k = torch.empty_like(st.q), torch.empty_like(st.k)
        o = torch.empty_like(st.q)
        if fused:
            hb.hb_rope(batch, rope, st.q, st.k, st.v, q, k, k2, v2)
            hb.hb_attention_new_kv(batch, plan, q, k, st.v, k2, v2, 1 / math.sqrt(d), o, ws)
        else:
            hb.hb_rope(batch, rope, st.q, st.k, None, q, k, None, None)
            hb.hb_kv_append(batch, k, st.v, k2, v2)
            hb.hb_attention(batch, plan, q, k2, v2, 1 / math.sqrt(d), o, ws)
        outs.append((o, k2, v2))
    hb.hb_check()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("size", [1e30, 1e36, 1e-18, 1e-22, 1e-38, 1e-40])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,d", [(9, 128), (9, 64), (2000, 128), (2000, 64)])
def test_head_norms_of_squares_outside_of_fp32(tokens, d, interleaved, size):
    """A head of large or tiny values, between ordinary ones, is normed as well."""
    hb = lib()
    st = Step([(tokens, tokens + 20)], 8, 2, d, seed=16)
    for x, heads in ((st.q, (0, 5)), (st.k, (1,))):
        for h in heads:
            x[1::3, h] = (x[1::3, h].float() * size).to(BF)
    rope = hb.make_rope(d // 2, interleaved=interleaved, eps=0.0, q_weight=st.weights[0], k_weight=st.weights[1])
    q, k = torch.empty_like(st.q), torch.empty_like(st.k)
    hb.hb_rope(st.batch, rope, st.q, st.k, st.v, q, k, st.kc, st.vc)
    hb.hb_check()
    angle = angles(d // 2, range(20, 20 + tokens))
    for got, x, w in ((q, st.q, st.weights[0]), (k, st.k, st.weights[1])):
        normed = torch.from_numpy(ob.rms_norm(f64(x), f64(w), 0.0))
        check(got, expected(normed, None, angle, interleaved, 1.0))
    slot = torch.arange(20, 20 + tokens)
    page = torch.from_numpy(st.table[0, slot.numpy() // 16].astype(np.int64)).cuda()
    assert torch.equal(st.kc[page, (slot % 16).cuda()], k)


def test_head_norms_of_zeros_and_of_values_that_are_not_finite():
    """As by the formula, and in their own head alone: with eps zeros stay zeros, without 0 / 0."""
    hb = lib()
    for eps in (1e-6, 0.0):
        st = Step([(6, 20)], 8, 2, 64, seed=17)
        st.q[2, 3] = 0
        st.q[4, 1, 7] = float("inf")
        st.k[1, 0, 9] = float("nan")
        rope = hb.make_rope(64, eps=eps, q_weight=st.weights[0], k_weight=st.weights[1])
        q, k = torch.empty_like(st.q), torch.empty_like(st.k)
        hb.hb_rope(st.batch, rope, st.q, st.k, st.v, q, k, st.kc, st.vc)
        assert q[2, 3].isnan().all() if eps == 0.0 else not q[2, 3].any()
        # inf / inf in its pair, finite values over an infinite root: zeros
        bad = (~torch.isfinite(q[4, 1])).nonzero().flatten().tolist()
        assert bad == [7, 39] and not q[4, 1][[i for i in range(64) if i not in bad]].any()
        assert k[1, 0].isnan().all()
        q[2, 3] = q[4, 1] = 0
        k[1, 0] = 0
        assert torch.isfinite(q).all() and torch.isfinite(k).all()


@pytest.mark.parametrize("pos", [5, 1 << 20, (1 << 24) + 1, (1 << 31) - 20])
@pytest.mark.parametrize("scaling,by", [("none", 1.0), ("parts", 16.0), ("base", 4.0)])
def test_far_positions_against_exact_angles(pos, scaling, by):
    """The phases themselves are off by less than 2^-51 of a turn (test_rope_host.py), times the position."""
    hb = lib()
    d, n = 128, 5
    st = Step([(n, 40)], 4, 2, d, seed=18)
    st.dev[1].fill_(pos + n)
    kw = dict(base=5e5, scaling=scaling)
    q, k = run(st, d, norms=(False, False), cached=False, scale_by=by, original_context=8192, **kw)
    hb.hb_check()
    angle = np.array(exact_angles(exact_turns(d, by=by, **kw), range(pos, pos + n)))
    for got, x in ((q, st.q), (k, st.k)):
        want, bound = expected(x, None, angle, False, 1.0)
        size = np.abs(f64(x))
        size = np.concatenate([size[..., :d // 2] + size[..., d // 2:]] * 2, -1)
        check(got, (want, bound + 2 * math.pi * (pos + n) * 2.0 ** -51 * (1 + 2.0 ** -8) * size))
