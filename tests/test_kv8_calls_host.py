"""The 8-bit and page calls of the binding on the host (no GPU): arguments that
are not what they should be, plans that are cut short, rows that stand still."""
import numpy as np
import pytest
import torch

from _hbutil import host_batch, lib


@pytest.mark.parametrize("junk", [[1, 2], np.zeros(2, np.int32), None, 3])
@pytest.mark.parametrize("at", range(6))
def test_page_calls_refuse_what_is_no_tensor(at, junk):
    hb = lib()
    i32, st, table = torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(2, 3, dtype=torch.int32)
    args = [i32, i32, i32, st, st, table]
    names = ["q_len", "context_len", "free_pages", "state_in", "state_out", "block_table"]
    args[at] = junk
    with pytest.raises(ValueError, match=names[at]):
        hb.hb_pages_assign(*args, torch.zeros(3, dtype=torch.int32))
    if at != 1:
        with pytest.raises(ValueError, match="lengths" if at == 0 else names[at]):
            hb.hb_pages_release(args[0], *args[2:])


def test_page_calls_refuse_slots_that_are_no_tensor():
    hb = lib()
    i32, st, table = torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(2, 3, dtype=torch.int32)
    for junk in ([1, 2], np.zeros(2, np.int64), torch.zeros(2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int64)):
        with pytest.raises(ValueError, match="slot_map"):
            hb.hb_pages_assign(i32, i32, i32, st, st, table, torch.zeros(3, dtype=torch.int32), junk)


def test_page_calls_refuse_sizes_past_32_bits():
    """(They go to the library as 32-bit integers: 2^32 + 16 would pass as 16.)"""
    hb = lib()
    i32, st, table = torch.zeros(2, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(2, 3, dtype=torch.int32)
    ring = torch.empty(2 ** 32 + 16, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="free_pages.*2\\^31"):
        hb.hb_pages_assign(i32, i32, ring, st, st, table, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="free_pages.*2\\^31"):
        hb.hb_pages_release(i32, ring, st, st, table)


def test_attention_refuses_a_workspace_that_is_no_tensor():
    hb = lib()
    b, ql, cl = host_batch(hb, [(1, 40), (5, 9)], num_pages=8)
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    q = torch.zeros(6, 32, 128, dtype=torch.bfloat16)
    k = torch.zeros(8, 16, 8, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros(8, 8, dtype=torch.int8)
    for junk in ([1, 2], np.zeros(1 << 20, np.uint8), 7):
        with pytest.raises(ValueError, match="workspace"):
            hb.hb_kv8_attention(b, plan, q, k, k, e, e, 1.0, q, junk)


def test_a_plan_cut_short_or_strided_is_refused():
    """The library reads the plan at the places that its header gives."""
    hb = lib()
    b, ql, cl = host_batch(hb, [(1, 40), (5, 9)], num_pages=8)
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    q = torch.zeros(6, 32, 128, dtype=torch.bfloat16)
    k = torch.zeros(8, 16, 8, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros(8, 8, dtype=torch.int8)
    call = lambda p: hb.hb_kv8_attention(b, p, q, k, k, e, e, 1.0, q, None)  # noqa: E731
    twice = np.repeat(plan, 2)[::2]
    assert np.array_equal(twice, plan)
    for bad in (plan[:-1], plan[:hb.HEADER_BYTES], plan[:hb.HEADER_BYTES - 1], twice, plan.view(np.int8), plan.tobytes(), None):
        with pytest.raises(ValueError, match="plan"):
            call(bad)
    for good in (plan, np.concatenate([plan, np.zeros(100, np.uint8)])):
        with pytest.raises(ValueError, match="CUDA"):      # (gets as far as the tensors)
            call(good)


def plan_of(hb, rows, **kw):
    b, ql, cl = host_batch(hb, rows, **kw)
    plan, _ = hb.hb_kv8_plan(b, ql, cl, 152, upload=False)
    return plan, hb.hb_plan_sizes(b, ql, cl, 152, kv8=True)


@pytest.mark.parametrize("window", [0, 50])
def test_rows_that_stand_still_cost_nothing(window):
    """Rows without new tokens (waiting, finished, empty) add no work to a plan:
    it is the plan without them, at the rows' places."""
    hb = lib()
    rows = [(1, 700), (30, 200), (1, 33), (130, 130), (1, 5)]
    at = [1, 2, 4, 5, 7]
    still = [(0, 40), None, None, (0, 0), None, None, (0, 900), None, (0, 1)]
    both = list(still)
    for i, r in zip(at, rows):
        both[i] = r
    a, sizes_a = plan_of(hb, rows, max_pages=60, window=window)
    b, sizes_b = plan_of(hb, both, max_pages=60, window=window)
    for x, y, tok in zip(hb.plan_items(a)[:2], hb.plan_items(b)[:2], (9, 5)):
        want = x.copy()
        want[:, 0] = np.array(at)[x[:, 0]]
        assert np.array_equal(y, want)
    assert np.array_equal(hb.plan_items(a)[2], hb.plan_items(b)[2])
    assert sizes_a[0] == sizes_b[0]                  # as many items to upload


def test_a_step_in_which_every_row_stands_still():
    hb = lib()
    plan, _ = plan_of(hb, [(0, 5), (0, 0)])
    dec, chk, _ = hb.plan_items(plan)
    assert len(dec) == 0 and len(chk) == 0


@pytest.mark.parametrize("row", [(-1, 5), (6, 5), (0, -1), (0, 4000)])
def test_rows_that_break_the_rules_are_refused(row):
    hb = lib()
    b, ql, cl = host_batch(hb, [(1, 5), (1, 5)], max_pages=4)
    ql[1], cl[1] = row
    b.total_q = int(ql.sum())
    with pytest.raises(hb.HbError) as e:
        hb.hb_plan_sizes(b, ql, cl, 152, kv8=True)
    assert e.value.status == 2


def test_a_ring_lists_every_page_once():
    hb = lib()
    for bad in ([0, 0, 1, 2], [0, 1, 2, 4], [-1, 0, 1, 2], [0, 1, 2], [0, 1, 2, 3, 3], [[0, 1], [2, 3]]):
        with pytest.raises(ValueError, match="every page"):
            hb.pages_ring(4, bad, device="cpu")
    ring, state = hb.pages_ring(4, [3, 1, 0, 2], device="cpu")
    assert ring.tolist() == [3, 1, 0, 2] and state.tolist() == [0, 4, 0, 0]
    assert hb.pages_ring(3, device="cpu")[0].tolist() == [0, 1, 2]


def test_a_torch_without_its_private_shortcuts(monkeypatch):
    """The binding falls back to torch's public calls for the current device and
    stream."""
    import importlib.util
    from chunked_prefill_decode_gb300 import hb
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)

    class Stream:
        cuda_stream = 0x77
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream if dev == 3 else None)
    spec = importlib.util.spec_from_file_location("chunked_prefill_decode_gb300.hb_copy", hb.__file__)
    copy = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(copy)
    assert copy._current_device() == 3 and copy._raw_stream(None, 3) == 0x77 and copy._raw_stream(5, 3) == 5


@pytest.mark.parametrize("rows", [[(1, 40), (5, 9)], [(300, 2000), (1, 900), (17, 17)], [(64, 5000)] * 3,
                                  [(1, 100)] * 40 + [(2016, 8064)]])
@pytest.mark.parametrize("geom,window", [((32, 8, 128), 0), ((8, 8, 64), 0), ((56, 8, 128), 700)])
def test_both_caches_plans_cover_the_same_chunk_work(rows, geom, window):
    """Every (row, kv head, token, key tile) of the chunk rows once in each plan,
    however the two cut it into items."""
    hb = lib()
    b, ql, cl = host_batch(hb, rows, hq=geom[0], hkv=geom[1], d=geom[2], window=window)
    got = []
    for plan in (hb.hb_kv8_plan(b, ql, cl, 152, upload=False)[0], hb.hb_plan(b, ql, cl, 152, upload=False)[0]):
        _, chk, _ = hb.plan_items(plan)
        cover = {}
        for seq, kvh, tok0, ntok, end, q0, q_len, ctx, begin, *_ in chk.tolist():
            assert q_len == ql[seq] and ctx == cl[seq] and q0 == ql[:seq].sum()
            # (an item's range of key tiles is that of its last token; a token counts those that it sees)
            for t in range(tok0, tok0 + ntok):
                last = (ctx - q_len + t) // 128
                low = max(0, ctx - q_len + t - window + 1) // 128 if window else 0
                for j in range(max(begin, low), min(end, last + 1)):
                    key = (seq, kvh, t, j)
                    assert key not in cover
                    cover[key] = 1
        got.append(cover)
    assert got[0].keys() == got[1].keys()
    want = 0
    for q, c in zip(ql, cl):
        for t in range(q if q > 1 else 0):
            pos = c - q + t
            want += pos // 128 - (max(0, pos - window + 1) // 128 if window else 0) + 1
    assert len(got[0]) == want * geom[1]
