"""hb_adapters_plan and the refusals of hb_adapters on the host (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from _hbutil import lib

AT = 1 << 32      # device addresses that no call here follows


def pool(hb, n=5, slices=1, r=16, k=64, cols=(64,)):
    p = hb.HbAdapterPool()
    p.num_adapters, p.max_rank, p.K, p.N, p.slices = n, r, k, sum(cols), slices
    p.a, p.b, p.rank, p.scale = (AT + (i << 24) for i in range(4))
    return p


def plan_of(hb, q, of, n=5, total_q=None, **kw):
    return hb.hb_adapters_plan(pool(hb, n=n, **kw), q, of, 152, total_q=total_q, upload=False)[0]


@pytest.mark.parametrize("seed", range(6))
def test_a_plan_covers_every_token_once(seed):
    hb = lib()
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 40))
    q = rng.choice([0, 1, 1, 1, 3, 16, 63, 64, 65, 200], int(rng.integers(1, 80)))
    of = rng.integers(-1, n, len(q))
    plan = plan_of(hb, q, of, n=n, total_q=int(q.sum()) + 3)
    h = hb.adapters_plan_header(plan)
    segs, rows = hb.adapters_plan_items(plan)
    token = np.repeat(of, q)
    assert sorted(rows) == list(range(len(token)))
    assert h["total_q"] == len(token) + 3 and h["long_rows"] + h["short_rows"] == (token >= 0).sum()
    long, short, idle = np.split(segs, [h["num_long"], h["num_long"] + h["num_short"]])
    assert h["num_idle"] == len(idle) and (idle[:, 0] == -1).all() and (short[:, 0] >= 0).all()
    # segment after segment takes the row list
    assert (segs[:, 1] == np.cumsum(segs[:, 2]) - segs[:, 2]).all() and segs[:, 2].sum() == len(rows)
    for a, first, count, tok in segs:
        mine = rows[first:first + count]
        assert (token[mine] == a).all() and (np.diff(mine) > 0).all()
        assert 1 <= count <= (128 if tok >= 0 else 16)
        if tok >= 0:
            assert (mine == tok + np.arange(count)).all()
    # long tiles are the runs of 128 neighbours or more, short segments as few as can be
    edges = np.flatnonzero(np.diff(np.concatenate([[-2], token, [-2]])))
    runs = [(int(token[i]), j - i) for i, j in zip(edges, edges[1:])]
    assert sum(n for a, n in runs if a >= 0 and n >= 128) == h["long_rows"]
    assert sum(-(-n // 128) for a, n in runs if a >= 0 and n >= 128) == h["num_long"]
    for a in range(n):
        count = sum(m for b, m in runs if b == a and m < 128)
        assert (short[:, 0] == a).sum() == -(-count // 16)


def test_more_parts_of_k_where_rows_are_few():
    hb = lib()
    few, many, long = (hb.adapters_plan_header(plan_of(hb, q, np.arange(len(q)) % 2))
                       for q in ([1], [1] * 10000, [128]))
    assert few["short_pieces"] == 16 and many["short_pieces"] == 1 and long["num_long"] == 1
    for h in (few, many, long):
        assert h["ws_total"] >= (h["short_pieces"] * h["short_rows"] + 128 * h["num_long"]) * 16 * 4


def test_the_plan_serves_several_pools():
    hb = lib()
    pools = [pool(hb), pool(hb, slices=3, r=32, cols=(64, 32, 32))]
    assert hb.adapters_plan_header(hb.hb_adapters_plan(pools, [1], [0], 152, upload=False)[0])["max_ranks"] == 96
    with pytest.raises(ValueError, match="as many adapters"):
        hb.hb_adapters_plan([pool(hb), pool(hb, n=6)], [1], [0], 152, upload=False)
    with pytest.raises(ValueError, match="as many adapters"):
        hb.hb_adapters_plan([], [1], [0], 152, upload=False)


@pytest.mark.parametrize("q,of,total", [([1, 2], [0, 5], None), ([1, 2], [0, -2], None), ([1, -1], [0, 0], 9),
                                        ([1, 2], [0, 0], 2), ([1, 2], [0, 0], -1)])
def test_batches_that_break_the_rules_are_refused(q, of, total):
    hb = lib()
    with pytest.raises(hb.HbError) as e:
        plan_of(hb, q, of, total_q=total)
    assert e.value.status == 2


def test_plan_arguments():
    hb = lib()
    L = hb.load()
    one = np.ones(1, np.int32)
    pb, wb = ctypes.c_size_t(0), ctypes.c_size_t(0)

    def call(seqs=1, total=1, q=one, of=one, n=5, ranks=16, sms=152, plan=None, psize=pb, ws=None, wsize=wb):
        ptr = lambda a: a.ctypes.data if isinstance(a, np.ndarray) else a  # noqa: E731
        return L.hb_adapters_plan(seqs, total, ptr(q), ptr(of), n, ranks, sms, ptr(plan),
                                  ctypes.byref(psize) if psize is not None else None, ws,
                                  ctypes.byref(wsize) if wsize is not None else None, None)
    assert call() == 0 and pb.value > 0
    assert call(psize=None) == 1 and call(wsize=None) == 1 and call(q=None) == 1 and call(of=None) == 1
    assert call(seqs=-1) == 2 and call(n=0) == 2 and call(sms=0) == 2
    assert call(ranks=0) == 2 and call(ranks=12) == 2 and call(ranks=392) == 2
    buf = np.zeros(4096, np.uint8)
    assert call(plan=buf, psize=ctypes.c_size_t(8)) == 4
    assert call(plan=buf, psize=ctypes.c_size_t(4096), ws=AT, wsize=ctypes.c_size_t(8)) == 4
    assert call(plan=buf, psize=ctypes.c_size_t(4096), ws=AT + 16, wsize=ctypes.c_size_t(1 << 30)) == 1
    with pytest.raises(ValueError, match="q_len has shape"):
        plan_of(hb, [1, 2], [0])


def outs(hb, at, cols):
    o = hb.HbLinearOut()
    for i, c in enumerate(cols):
        o.cols[i] = c
        o.y[i] = at + (i << 20) if at else None
    return o


def call(hb, kw=None, q=(3, 4), of=(0, -1), x=AT + (8 << 24), y=AT + (9 << 24), out=AT + (10 << 24), ws=AT + (11 << 24),
         cols=(64,), out_cols=None, plan=None, plan_kw=None, **pool_kw):
    p = pool(hb, cols=cols, **pool_kw)
    for k, v in (kw or {}).items():
        setattr(p, k, v)
    if plan is None:
        plan = plan_of(hb, list(q), list(of), **(plan_kw or pool_kw))
    y, out = outs(hb, y, cols), outs(hb, out, out_cols or cols)
    return hb.load().hb_adapters(ctypes.byref(p), plan.ctypes.data, x, ctypes.byref(y), ctypes.byref(out), ws, None)


@pytest.mark.parametrize("want,kw", [
    (2, dict(kw=dict(num_adapters=0))), (2, dict(kw=dict(K=0))), (2, dict(kw=dict(slices=0))), (2, dict(kw=dict(slices=4))),
    (3, dict(kw=dict(max_rank=12))), (3, dict(kw=dict(max_rank=136))), (3, dict(kw=dict(max_rank=0))), (3, dict(kw=dict(K=12))),
    (4, dict(kw=dict(num_adapters=6))), (4, dict(kw=dict(max_rank=32))),
    (4, dict(plan=np.zeros(4096, np.uint8))), (2, dict(cols=(64, 8))), (2, dict(out_cols=(56,))), (2, dict(kw=dict(N=128))),
    (3, dict(cols=(60,))), (1, dict(kw=dict(a=None))), (1, dict(kw=dict(b=AT + 8))), (1, dict(kw=dict(rank=None))),
    (1, dict(kw=dict(scale=AT + 2))), (1, dict(x=None)), (1, dict(x=AT + 2)), (1, dict(y=None)), (1, dict(out=None)),
    (1, dict(out=AT + (10 << 24) + 8)), (1, dict(ws=None)), (1, dict(ws=AT + 128)),
])
def test_bad_arguments_are_refused(want, kw):
    assert call(lib(), **kw) == want


@pytest.mark.parametrize("kw", [
    dict(out=AT + (8 << 24)), dict(out=AT + (9 << 24) + 128), dict(out=AT + (9 << 24) - 128), dict(out=AT),
    dict(out=AT + (1 << 24)), dict(out=AT + (2 << 24)), dict(out=AT + (3 << 24)), dict(out=AT + (11 << 24)),
    dict(cols=(64, 64), slices=2, y=AT + (9 << 24), out=AT + (9 << 24) + (1 << 20)),   # one destination over another's
])
def test_operands_that_overlap_are_refused(kw):
    hb = lib()
    assert call(hb, **kw) == 1
    assert b"overlap" in hb.load().hb_last_error()


def test_no_tokens_are_no_work():
    assert call(lib(), q=(0, 0), of=(0, 1)) == 0


def test_tensors_are_checked_by_name():
    hb = lib()
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    a, b, rank, scale = z(5, 1, 16, 64), z(5, 64, 16), z(5, dtype=torch.int32), z(5, dtype=torch.float32)
    for at, junk, name in [(0, None, "a must be"), (0, z(5, 16, 64), "a must be"), (0, z(5, 2, 16, 64), "a has shape"),
                           (1, z(5, 32, 16), "b has shape"), (2, z(5), "rank must be"), (3, z(4, dtype=torch.float32), "scale has"),
                           (4, (32,), "b has shape"), (4, (), "cols"), (4, (64, 0), "cols"), (4, (8,) * 4, "cols"),
                           (1, z(5, 16, 64).transpose(1, 2), "b must be a contiguous")]:
        args = [a, b, rank, scale, (64,)]
        args[at] = junk
        with pytest.raises(ValueError, match=name):
            hb.make_adapters(*args)
    p = hb.make_adapters(a, b, rank, scale, (64,))
    plan, _ = hb.hb_adapters_plan(p, [3, 4], [0, -1], 152, upload=False)
    x, y = z(7, 64), z(7, 64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for at, junk, name in [(0, hb.HbAdapterPool(), "pool"), (1, plan[:-1], "plan"), (1, plan[:87], "plan"), (1, None, "plan"),
                           (1, np.repeat(plan, 2)[::2], "plan"), (2, z(6, 64), "x has shape"), (2, [1], "x must be"),
                           (3, y, "y must be a list"), (3, [y, y], "y must be a list"), (3, [z(7, 32)], "y.0. has shape"),
                           (4, [z(7, 64, dtype=torch.float32)], "out.0. must be"), (4, [], "out must be a list"),
                           (5, None, "workspace"), (5, ws[:8], "workspace has 8"), (5, [1], "workspace"), (2, x, "CUDA")]:
        args = [p, plan, x, [y], [z(7, 64)], ws]
        args[at] = junk
        with pytest.raises(ValueError, match=name):
            hb.hb_adapters(*args)


@pytest.mark.parametrize("kw", [dict(of=np.array([0, 1 << 32])), dict(of=np.array([0, (1 << 32) - 1], np.uint64)),
                                dict(of=np.array([0.0, 1.7])), dict(of=[0, 1 << 40]), dict(q=np.array([1, (1 << 32) + 2])),
                                dict(q=np.array([1, -(1 << 31) - 1])), dict(q=["1", "2"])])
def test_numbers_past_32_bits_are_refused(kw):
    """(Cut to 32 bits they would name another adapter, or another length.)"""
    with pytest.raises(ValueError, match="32 bits"):
        plan_of(lib(), **{"q": [1, 2], "of": [0, 1], **kw})


def test_host_numbers_of_any_width():
    hb = lib()
    want = plan_of(hb, [1, 2], [0, -1]).tobytes()
    for kind in (np.int8, np.int16, np.int64):
        assert plan_of(hb, np.array([1, 2], kind), np.array([0, -1], kind)).tobytes() == want
    assert plan_of(hb, np.array([1, 2], np.uint8), torch.tensor([0, -1])).tobytes() == want
    assert hb.adapters_plan_header(plan_of(hb, [], [], total_q=0))["total_q"] == 0


@pytest.mark.parametrize("kw", [dict(ws=AT + (8 << 24)), dict(ws=AT + (9 << 24) + 256), dict(ws=AT), dict(ws=AT + (1 << 24)),
                                dict(ws=AT + (2 << 24)), dict(ws=AT + (3 << 24)), dict(x=AT + (11 << 24) + 64)])
def test_a_workspace_over_an_operand_is_refused(kw):
    hb = lib()
    assert call(hb, **kw) == 1
    assert b"the workspace and" in hb.load().hb_last_error()
