"""The 8-bit cache and the page bookkeeping on the host (no GPU): refusals
through the C ABI and the binding, the plan, and pins of their oracles."""
import ctypes

import numpy as np
import pytest
import torch

from _hbutil import host_batch, lib
from oracle import kv8, pages
from oracle import paged_attention as pa

FAKE = 0x1000     # an address that is never dereferenced


def test_e4m3_table_agrees_with_torch():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(kv8.decode(b)))
    ok = ~np.isnan(t)
    assert np.array_equal(t[ok], kv8.decode(b)[ok])
    assert np.array_equal(kv8.encode(kv8.decode(b))[ok], b[ok])


def test_encode_rounds_like_torch_within_the_range():
    x = np.concatenate([np.linspace(-448, 448, 20011), 2.0 ** np.linspace(-14, 8, 4001), [0.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.encode(x), want)
    assert kv8.encode([1e9, -1e9, np.nan]).tolist() == [0x7E, 0xFE, 0x7F]


def test_need_exp_is_the_smallest_that_holds():
    rng = np.random.default_rng(0)
    for x in list(2.0 ** rng.uniform(-50, 50, 200)) + [448.0, 449.0, 448.0 * 2 ** -7, 1.75, 1.7500001]:
        e = kv8.need_exp([x, -x / 3, np.inf, np.nan])
        assert x <= 448 * 2.0 ** e and x > 448 * 2.0 ** (e - 1)
    assert kv8.need_exp([0.0]) == -64 and kv8.need_exp([1e30]) == 64 and kv8.need_exp([np.nan]) == -64


def test_oracle_append_keeps_the_new_values_to_half_a_step():
    rng = np.random.default_rng(1)
    k = np.zeros((6, 16, 2, 64), np.uint8)
    e = np.zeros((6, 2), np.int8)
    table = np.array([[3, 1, 4]])
    x = rng.standard_normal((40, 2, 64)) * 3
    out = kv8.append(k, k, e, e, x, -x, [40], [40], table)
    got = kv8.values(out[0], out[2])[table[0]].reshape(48, 2, 64)[:40]
    top = np.abs(x).reshape(-1, 2, 64)
    for p in range(3):
        rows = slice(16 * p, min(40, 16 * p + 16))
        m = top[rows].max((0, 2))
        # half a step of a normal value, or of the subnormal range under the scale that holds m
        tol = np.maximum(np.abs(x[rows]) * 2.0 ** -4, (m * 2 / 448 * 2.0 ** -10)[None, :, None])
        assert (np.abs(got[rows] - x[rows]) <= tol).all()
    assert np.array_equal(kv8.decode(out[1]), -kv8.decode(out[0]))


def test_oracle_append_grows_a_page_without_losing_normal_values():
    k = np.zeros((1, 16, 1, 64), np.uint8)
    e = np.zeros((1, 1), np.int8)
    old = np.full((3, 1, 64), 1.125)
    a = kv8.append(k, k, e, e, old, old, [3], [3], [[0]])
    b = kv8.append(*a, np.full((1, 1, 64), 1000.0), np.full((1, 1, 64), 0.001), [1], [4], [[0]])
    assert b[2][0, 0] == 2 and b[3][0, 0] == a[3][0, 0]
    assert (kv8.values(b[0], b[2])[0, :3] == 1.125).all() and (kv8.values(b[1], b[3])[0, :3] == 1.125).all()


def test_oracle_attention_is_the_bf16_oracle_on_the_values():
    """Caches whose values are exact in bf16 give the bf16 oracle's answer."""
    rng = np.random.default_rng(2)
    x = kv8.decode(kv8.encode(rng.standard_normal((3, 16, 2, 64)) * 100))
    enc, e = kv8.encode(x), np.full((3, 2), -7, np.int8)
    q = rng.standard_normal((5, 4, 64))
    args = ([5], [40], np.array([[2, 0, 1]]), 16, 4, 2, 0.1)
    assert np.array_equal(kv8.attention(q, enc, enc[::-1], e, e, *args), pa.attention(q, x / 128, x[::-1] / 128, *args))


def test_oracle_pages_by_hand():
    table = np.array([[9, -1, -1], [-1, -1, -1]])
    cu, t, slots, head = pages.assign([2, 17], [17, 17], [4, 5, 6, 7], 3, 7, table)
    # row 0: token 15 on page 9, token 16 opens ring[3] = 7; row 1: ring[0], ring[1]
    assert cu.tolist() == [0, 2, 19] and head == 6
    assert t.tolist() == [[9, 7, -1], [4, 5, -1]]
    assert slots.tolist() == [9 * 16 + 15, 7 * 16] + list(range(64, 80)) + [80]
    assert pages.assign([2, 17], [17, 17], [4, 5, 6, 7], 3, 5, table) is None
    ring, tail = pages.release([17, 0], [4, 5, 6, 7], 6, 7, t)
    assert ring.tolist() == [7, 5, 6, 9] and tail == 9


# ------------------------------------------------------------------ refusals
def batch(hb, **kw):
    b, ql, cl = host_batch(hb, [(1, 40), (5, 9)], **kw)
    return b, ql, cl


@pytest.mark.parametrize("field,value,status", [
    ("page_size", 8, 3), ("head_dim", 96, 3), ("num_kv_heads", 3, 2), ("num_pages", 0, 2), ("reserved", 1, 1),
    ("max_pages_per_seq", 0, 2), ("num_seqs", -1, 2), ("total_q", -5, 2), ("sliding_window", -1, 2)])
def test_bad_batches_are_refused(field, value, status):
    hb = lib()
    L = hb.load()
    b, ql, cl = batch(hb)
    setattr(b, field, value)
    assert L.hb_kv8_append(ctypes.byref(b), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None) == status
    with pytest.raises(hb.HbError) as e:
        hb.hb_plan_sizes(b, ql, cl, 152, kv8=True)
    assert e.value.status == status


def test_bad_pointers_are_refused():
    hb = lib()
    L = hb.load()
    b, ql, cl = batch(hb)
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    p = hb._ptr(plan)
    for i in range(6):
        for bad in (None, FAKE + 8):
            if bad and i >= 4:
                continue                     # exponents have no alignment
            a = [FAKE] * 6
            a[i] = bad
            assert L.hb_kv8_append(ctypes.byref(b), *a, None) == 1
    for i in range(7):
        for bad in (None, FAKE + 8):
            if bad and i in (3, 4):
                continue
            a = [FAKE] * 7                   # q, k, v, k_exp, v_exp, out, workspace
            a[i] = bad
            assert L.hb_kv8_attention(ctypes.byref(b), p, *a[:5], 1.0, a[5], a[6], None) == 1, (i, bad)
    for scale in (float("nan"), 0.0, -0.1, float("inf")):
        assert L.hb_kv8_attention(ctypes.byref(b), p, *[FAKE] * 5, scale, FAKE, FAKE, None) == 1
    assert L.hb_kv8_attention(ctypes.byref(b), None, *[FAKE] * 5, 1.0, FAKE, FAKE, None) == 1


def test_append_of_too_many_pieces_is_refused():
    hb = lib()
    b, _, _ = batch(hb)
    b.num_seqs = b.total_q = 2 ** 30
    assert hb.load().hb_kv8_append(ctypes.byref(b), *[FAKE] * 6, None) == 3


def test_plans_of_the_two_caches_are_told_apart():
    hb = lib()
    L = hb.load()
    b, ql, cl = batch(hb)
    p8, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    p16, _ = hb.hb_plan(b, ql, cl, 152, upload=False)
    assert L.hb_kv8_attention(ctypes.byref(b), hb._ptr(p16), *[FAKE] * 5, 1.0, FAKE, FAKE, None) == 4
    assert L.hb_attention(ctypes.byref(b), hb._ptr(p8), FAKE, FAKE, FAKE, 1.0, FAKE, FAKE, None) == 4
    other, _, _ = host_batch(hb, [(1, 40), (6, 9)])
    assert L.hb_kv8_attention(ctypes.byref(other), hb._ptr(p8), *[FAKE] * 5, 1.0, FAKE, FAKE, None) == 4
    # the same work items
    for a, c in zip(hb.plan_items(p8)[:2], hb.plan_items(p16)[:2]):
        assert a.shape[1] == c.shape[1]


def test_plan_sizes_and_short_buffers():
    hb = lib()
    L = hb.load()
    b, ql, cl = batch(hb)
    need_p, need_w = hb.hb_plan_sizes(b, ql, cl, 152, kv8=True)
    plan = np.zeros(need_p - 1, np.uint8)
    pb, wb = ctypes.c_size_t(plan.nbytes), ctypes.c_size_t(0)
    assert L.hb_kv8_plan(ctypes.byref(b), hb._ptr(ql), hb._ptr(cl), 152, hb._ptr(plan), ctypes.byref(pb), None,
                         ctypes.byref(wb), None) == 4
    assert (pb.value, wb.value) == (need_p, need_w)
    plan = np.zeros(need_p, np.uint8)
    pb, wb = ctypes.c_size_t(plan.nbytes), ctypes.c_size_t(need_w - 1)
    assert L.hb_kv8_plan(ctypes.byref(b), hb._ptr(ql), hb._ptr(cl), 152, hb._ptr(plan), ctypes.byref(pb), FAKE,
                         ctypes.byref(wb), None) == 4


def test_empty_batch_is_nothing_to_do():
    hb = lib()
    L = hb.load()
    b, ql, cl = host_batch(hb, [])
    assert L.hb_kv8_append(ctypes.byref(b), None, None, None, None, None, None, None) == 0
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    assert L.hb_kv8_attention(ctypes.byref(b), hb._ptr(plan), None, None, None, None, None, 1.0, None, None, None) == 0


def assign_args(**kw):
    a = dict(num_seqs=2, max_tokens=8, max_pages=4, num_pages=16, page_size=16, q_len=FAKE, ctx=FAKE, ring=FAKE,
             state_in=FAKE, state_out=FAKE, table=FAKE, cu=FAKE, slots=FAKE, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 2), (dict(num_seqs=16385), 3), (dict(max_tokens=-1), 2), (dict(max_pages=0), 2),
    (dict(num_pages=0), 2), (dict(num_pages=2 ** 28), 3), (dict(max_pages=2 ** 28), 3), (dict(page_size=32), 3),
    (dict(q_len=None), 1), (dict(ctx=None), 1), (dict(ring=None), 1), (dict(state_in=None), 1),
    (dict(state_out=None), 1), (dict(table=None), 1), (dict(cu=None), 1), (dict(q_len=FAKE + 2), 1),
    (dict(cu=FAKE + 1), 1), (dict(ring=FAKE + 2), 1), (dict(table=FAKE + 2), 1), (dict(state_in=FAKE + 4), 1),
    (dict(state_out=FAKE + 4), 1), (dict(slots=FAKE + 4), 1)])
def test_assign_refusals(kw, status):
    assert lib().load().hb_pages_assign(*assign_args(**kw)) == status


@pytest.mark.parametrize("i,value,status", [
    (0, -1, 2), (0, 16385, 3), (1, 0, 2), (2, 0, 2), (3, 8, 3), (4, None, 1), (5, None, 1), (6, None, 1),
    (7, None, 1), (8, None, 1), (4, FAKE + 2, 1), (7, FAKE + 4, 1), (8, FAKE + 4, 1)])
def test_release_refusals(i, value, status):
    a = [2, 4, 16, 16, FAKE, FAKE, FAKE, FAKE, FAKE, None]
    a[i] = value
    assert lib().load().hb_pages_release(*a) == status


def test_binding_refuses_tensors_that_do_not_fit():
    hb = lib()
    b, ql, cl = batch(hb, num_pages=8)
    k = torch.zeros(8, 16, 8, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros(8, 8, dtype=torch.int8)
    new = torch.zeros(6, 8, 128, dtype=torch.bfloat16)
    for args, what in [
            ((new.float(), new, k, k, e, e), "k_new"), ((new[:5], new, k, k, e, e), "k_new"),
            ((new.transpose(0, 1), new, k, k, e, e), "k_new"), ((new, new, k, k, e, e), "CUDA")]:
        with pytest.raises(ValueError, match=what):
            hb.hb_kv8_append(b, *args)
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    q = torch.zeros(6, 32, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        hb.hb_kv8_attention(b, plan, q, k, k, e, e, 1.0, q, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        hb.hb_kv8_attention(b, plan, q, k, k, e, e, 1.0, q, None)
    i32 = torch.zeros(2, dtype=torch.int32)
    st = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="q_len"):
        hb.hb_pages_assign(i32.long(), i32, i32, st, st, i32.view(2, 1), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        hb.hb_pages_release(i32, i32, st, st, i32.view(2, 1))
    with pytest.raises(ValueError, match="every page"):
        hb.pages_ring(4, [0, 1], device="cpu")


def test_a_ring_state_that_overlaps_the_other_is_refused():
    L = lib().load()
    for d in (-24, -8, 8, 24):
        assert L.hb_pages_assign(*assign_args(state_out=FAKE + d)) == 1
        assert L.hb_pages_release(2, 4, 16, 16, FAKE, FAKE, FAKE, FAKE, FAKE + d, None) == 1


@pytest.mark.parametrize("seed", range(60))
def test_the_decode_rows_of_a_plan_are_covered_once(seed):
    """Every page of a row and head in one item, the pieces of a row numbered,
    their slots and counters their own, no more CTAs than SMs."""
    hb = lib()
    rng = np.random.default_rng(900 + seed)
    hq, hkv, d = [(8, 8, 64), (32, 8, 128), (56, 8, 128), (16, 2, 64), (16, 1, 128), (12, 6, 128), (64, 16, 128)][seed % 7]
    window = int(rng.choice([0, 0, 40, 1000]))
    sms = int(rng.choice([1, 7, 152]))
    n = int(rng.choice([1, 2, 5, 17, 40, 200]))
    rows = [(1, int(2 ** rng.uniform(0, 13))) for _ in range(n)] + [(int(rng.integers(2, 200)), 300)] * int(rng.integers(0, 2))
    rng.shuffle(rows)
    b, ql, cl = host_batch(hb, [tuple(int(x) for x in r) for r in rows], hq=hq, hkv=hkv, d=d, window=window)
    plan, _ = hb.hb_kv8_plan(b, ql, cl, sms, upload=False)
    h = hb.plan_header(plan)
    dec, _, offs = hb.plan_items(plan)
    kvhb, grid = h["decode_kvh_block"], h["decode_grid"]
    assert hkv % kvhb == 0 and 1 <= grid <= sms and h["num_decode_dynamic"] == 0
    assert offs[0] == 0 and offs[-1] == len(dec) and (np.diff(offs) >= 1).all()
    cu = np.concatenate([[0], np.cumsum(ql)])
    got = {}
    for seq, kvh0, pb, pe, split, ns, slot, mid, ctx, tok, _, _ in dec:
        assert ql[seq] == 1 and ctx == cl[seq] and tok == cu[seq] and kvh0 % kvhb == 0 and 0 <= kvh0 < hkv
        got.setdefault((seq, kvh0), []).append((pb, pe, split, ns, slot, mid))
    assert len(got) == int((ql == 1).sum()) * (hkv // kvhb)
    slots, mids = set(), set()
    for (seq, _), items in got.items():
        items.sort()
        first = (cl[seq] - window) // 16 if 0 < window < cl[seq] else 0
        assert items[0][0] == first and items[-1][1] == -(-cl[seq] // 16)
        assert all(a[1] == c[0] for a, c in zip(items, items[1:])) and all(a[0] < a[1] for a in items)
        assert [a[2] for a in items] == list(range(len(items))) and all(a[3] == len(items) for a in items)
        if len(items) > 1:
            assert len({a[4:] for a in items}) == 1
            mine = set(range(items[0][4], items[0][4] + len(items)))
            assert not mine & slots and items[0][5] not in mids
            slots |= mine
            mids.add(items[0][5])
    assert len(slots) == h["num_partial_slots"] and len(mids) == h["num_merge_counters"]
    assert not slots or max(slots) == len(slots) - 1


@pytest.mark.parametrize("geom,ctxs,pieces", [
    ((8, 8, 64), [16, 100, 300, 512, 40], [1, 1, 1, 1, 1]),        # short rows are not cut
    ((32, 8, 128), [16384], [19]),                                 # 8 blocks of one head on 152 CTAs
    ((32, 8, 128), [2000, 2000, 100], [8, 8, 1])])                 # 125 pages in stages of 16
def test_few_decode_rows_are_cut_each_by_itself(geom, ctxs, pieces):
    hb = lib()
    b, ql, cl = host_batch(hb, [(1, c) for c in ctxs], hq=geom[0], hkv=geom[1], d=geom[2])
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    dec, _, offs = hb.plan_items(plan)
    assert (np.diff(offs) == 1).all()
    for s, n in enumerate(pieces):
        mine = [d for d in dec if d[0] == s and d[1] == 0]
        assert [d[5] for d in mine] == [n] * n
        lens = [d[3] - d[2] for d in mine]
        assert max(lens) - min(lens) <= 1
