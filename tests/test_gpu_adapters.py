"""hb_adapters on the GPU against its definition in 64 bits.

Tolerance: one rounding to bf16 (2^-8 of the value).  Before it, relative to s
= |scale| |x| |A|^T |B|^T (every product by its size): the sums over K and over
the ranks in fp32, one addition per 8 products at most (a tensor core adds 16
at a time, and may cut instead of round: 2^-23 each) and 100 more for the
joining of parts, the scale, the ranks and y: (K / 8 + 100) 2^-23; x A^T in two
bf16 terms: 2^-8 of 2^-8."""
import numpy as np
import pytest
import torch

from _hbutil import lib
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def f64(t):
    return t.double().cpu().numpy()


class Case:
    def __init__(self, q, of, k, cols, n, r, seed=0, spare=0, ranks=None):
        self.q, self.of, self.cols, self.k = list(q), list(of), list(cols), k
        g = torch.Generator("cuda").manual_seed(seed)
        self.live = int(sum(q))
        T = self.T = self.live + spare
        randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        rng = np.random.default_rng(seed)
        self.ranks = rng.integers(1, r + 1, n) if ranks is None else np.array(ranks)
        dead = torch.arange(r, device="cuda")[None, :] >= torch.from_numpy(self.ranks).cuda()[:, None]
        self.a = (randn(n, len(cols), r, k) / k ** 0.5).to(BF).masked_fill_(dead[:, None, :, None], float("nan"))
        self.b = randn(n, sum(cols), r).to(BF).masked_fill_(dead[:, None, :], float("nan"))
        self.scale = torch.from_numpy(rng.uniform(-2, 2, n).astype(np.float32)).cuda()
        self.rank = torch.from_numpy(self.ranks.astype(np.int32)).cuda()
        self.x = randn(T, k).to(BF)
        self.y = [randn(T, c).to(BF) for c in cols]
        self.pool = lib().make_adapters(self.a, self.b, self.rank, self.scale, cols)

    def plan(self, **kw):
        return lib().hb_adapters_plan(self.pool, self.q, self.of, sms(), total_q=self.T, **kw)

    def expected(self):
        a, b = f64(self.a), f64(self.b)
        return ob.adapters(f64(self.x), [f64(y) for y in self.y], self.q, self.of, a, b, self.ranks, f64(self.scale))

    def check(self, outs, y0=None):
        want, size = self.expected() if y0 is None else y0
        for out, w, s, y in zip(outs, want, size, self.y):
            got = f64(out)[:self.live]
            assert np.isfinite(got).all()
            w, s = w[:self.live], s[:self.live]
            bound = 2.0 ** -8 * np.abs(w) + (2.0 ** -16 + (self.k / 8 + 100) * 2.0 ** -23) * s * (1 + 2.0 ** -8)
            assert (np.abs(got - w) <= bound).all(), f"worst excess {(np.abs(got - w) - bound).max():.3e}"

    def run(self, how="new", **kw):
        """(outs after a call; with how='same' in place)"""
        hb = lib()
        plan, ws = self.plan()
        outs = [y.clone() for y in self.y] if how == "same" else [torch.full_like(y, 7.0) for y in self.y]
        hb.hb_adapters(self.pool, plan, self.x, outs if how == "same" else self.y, outs, ws, **kw)
        hb.hb_check()
        return outs

    def check_both(self):
        want = self.expected()
        outs = self.run()
        self.check(outs, want)
        token = np.concatenate([np.repeat(np.array(self.of, int), self.q), np.full(self.T - self.live, -2)])
        none, behind = (torch.from_numpy(token == v).cuda() for v in (-1, -2))
        for o, y in zip(outs, self.y):
            assert torch.equal(o[none], y[none]) and (o[behind] == 7).all()
        for o, p, y in zip(self.run("same"), outs, self.y):
            assert torch.equal(o[:self.live], p[:self.live]) and torch.equal(o[behind], y[behind])
        return outs


@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 104, 128])
@pytest.mark.parametrize("cols", [(256,), (40, 8), (512, 128, 128)])
def test_against_the_definition(cols, r):
    q = [1, 1, 5, 1, 70, 1, 0, 1, 33, 1, 131, 140, 1, 260]
    of = [0, 3, 1, 0, 2, -1, 1, 4, -1, 0, 4, -1, 2, 1]
    Case(q, of, 320, cols, 5, r, seed=r, spare=2).check_both()


@pytest.mark.parametrize("k,n", [(8, 8), (24, 16), (56, 264), (64, 32), (1000, 776), (72, 2056), (4096, 1024), (14336, 256)])
@pytest.mark.parametrize("rows", [[1], [1, 1, 1], [17, 1, 150], [128, 129]])
def test_widths(k, n, rows):
    Case(rows, [i % 2 for i in range(len(rows))], k, (n,), 2, 16, seed=k).check_both()


@pytest.mark.parametrize("ranks", [[0, 0, 0], [1, 2, 3], [8, 0, 16], [15, 16, 17], [31, 32, 33], [40, 47, 48]])
def test_ranks_of_every_kind(ranks):
    r = max(8, -(-max(ranks) // 8) * 8)
    for cols in ((96,), (96, 40)):
        Case([1, 20, 1, 4, 70], [0, 1, 2, 0, 2], 200, cols, 3, r, seed=sum(ranks), ranks=ranks).check_both()
        Case([150, 1, 140, 4, 128], [0, 1, 2, 0, 1], 200, cols, 3, r, seed=sum(ranks), ranks=ranks).check_both()


def test_ranks_outside_of_the_pool_are_held_to_it():
    hb = lib()
    for q in ([1, 3, 2], [130, 200, 128]):
        c = Case(q, [0, 1, 2], 64, (64,), 3, 16, ranks=[16, 16, 16])
        want = c.run()[0]
        c.rank.copy_(torch.tensor([17, 1 << 30, -5], dtype=torch.int32))
        got = c.run()[0]
        n = q[0] + q[1]
        assert torch.equal(got[:n], want[:n]) and torch.equal(got[n:], c.y[0][n:])


@pytest.mark.parametrize("seed", range(4))
def test_batches_of_many_requests(seed):
    rng = np.random.default_rng(seed)
    n = [1, 40, 3, 300][seed]
    q = [1] * int(rng.integers(60, 300)) + list(rng.integers(2, 400, int(rng.integers(0, 4))))
    rng.shuffle(q)
    of = rng.integers(-1 if seed % 2 else 0, n, len(q))
    Case(q, of, 512, (512, 256), n, 16, seed=seed).check_both()


def test_long_prompts_of_large_rank():
    Case([1500, 1, 700], [1, 0, 0], 1024, (1024,), 2, 128, ranks=[128, 100]).check_both()
    Case([1300, 1, 700], [1, 0, 0], 640, (256, 256, 256), 2, 64, ranks=[64, 50]).check_both()


def test_where_nothing_has_an_adapter():
    c = Case([3, 100], [-1, -1], 64, (64, 8), 2, 8, spare=1)
    c.check_both()


def test_one_request_does_not_change_another():
    """A row's bits do not depend on who else is in the batch's segment."""
    c = Case([1] * 20, [0, 1] * 10, 512, (256,), 2, 16, seed=5)
    full = c.run()[0]
    x = c.x.clone()
    c.x[6] = float("nan")
    c.x[9, 4] = float("inf")
    got = c.run()[0]
    keep = [i for i in range(20) if i not in (6, 9)]
    assert torch.equal(got[keep], full[keep])
    assert got[6].isnan().all() and not got[9].isfinite().any()


def test_a_row_of_a_tile_does_not_change_another():
    c = Case([150, 1, 135], [0, 1, 1], 512, (256, 64), 2, 24, seed=5)
    full = c.run()
    c.x[6] = float("nan")
    c.x[140, 4] = float("inf")
    c.x[200] = float("nan")
    bad = [6, 140, 200]
    keep = [i for i in range(286) if i not in bad]
    for got, want in zip(c.run(), full):
        assert torch.equal(got[keep], want[keep])
        assert got[[6, 200]].isnan().all() and not got[140].isfinite().any()


@pytest.mark.parametrize("n", [1, 140])
def test_infinities_come_through(n):
    """A rank-1 adapter, and one that has no rank, next to dead ranks."""
    c = Case([n, n], [0, 1], 64, (64,), 2, 8, ranks=[1, 0])
    c.a[0, 0, 0] = 1.0
    c.b[0, :, 0] = torch.where(torch.arange(64, device="cuda") % 2 == 0, 1.0, -1.0).to(BF)
    c.scale.fill_(1.0)
    c.x.fill_(0.5)
    c.x[:, 3] = float("inf")
    out = c.run()[0]
    assert (out[:n, ::2] == float("inf")).all() and (out[:n, 1::2] == float("-inf")).all()
    assert torch.equal(out[n:], c.y[0][n:])


def test_captured_replayed_and_on_another_stream():
    hb = lib()
    c = Case([1] * 30 + [100, 300], [i % 7 for i in range(32)], 512, (256, 64), 7, 16, seed=6)
    want = c.run()
    plan, ws = c.plan()
    outs = [torch.empty_like(y) for y in c.y]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hb.hb_adapters(c.pool, plan, c.x, c.y, outs, ws, stream=side)
    side.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    again = [torch.empty_like(y) for y in c.y]
    with torch.cuda.graph(graph):
        # two calls in a row share the workspace
        hb.hb_adapters(c.pool, plan, c.x, c.y, outs, ws)
        hb.hb_adapters(c.pool, plan, c.x, outs, again, ws)
    for o in outs + again:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    once = [a.clone() for a in again]
    c.y, y = want, c.y
    c.check(once)
    # adapters brought in afterwards count when it is replayed
    c.scale.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(again, y))


def test_a_plan_serves_the_projections_of_a_step():
    hb = lib()
    q, of = [1, 1, 40, 1, 260], [2, 0, 1, 2, 1]
    cases = [Case(q, of, 512, (512, 128, 128), 3, 16, seed=1), Case(q, of, 1024, (256,), 3, 64, seed=2)]
    plan, ws = hb.hb_adapters_plan([c.pool for c in cases], q, of, sms())
    for _ in range(2):
        for c in cases:
            outs = [torch.empty_like(y) for y in c.y]
            hb.hb_adapters(c.pool, plan, c.x, c.y, outs, ws)
            c.check(outs)
    # planned again into the same buffers
    plan2, ws2 = hb.hb_adapters_plan([c.pool for c in cases], q, [0] * 5, sms(), plan=plan, workspace=ws)
    assert ws2.data_ptr() == ws.data_ptr()
    c = cases[0]
    c.of = [0] * 5
    outs = [torch.empty_like(y) for y in c.y]
    hb.hb_adapters(c.pool, plan2, c.x, c.y, outs, ws2)
    c.check(outs)


def test_beside_the_projection():
    """hb_linear and the adapters in place: the tuned weights' product."""
    hb = lib()
    c = Case([1] * 9 + [50, 333], [0, 1, 2, -1, 0, 1, 2, 0, 1, 2, 1], 512, (512, 256, 256), 3, 16, seed=8)
    w = (torch.randn(1024, 512, device="cuda") / 512 ** 0.5).to(BF)
    hb.hb_linear(c.x, w, c.y)
    want, size = c.expected()
    plan, ws = c.plan()
    hb.hb_adapters(c.pool, plan, c.x, c.y, c.y, ws)
    c.check(c.y, (want, size))


def test_offsets_past_32_bits():
    """Adapters whose elements lie past 2^32 in the pool."""
    hb = lib()
    n, r, k, cols = 1100, 128, 16384, (256,)
    a = torch.zeros(n, 1, r, k, dtype=BF, device="cuda")          # 2.3 G elements
    b = torch.zeros(n, 256, r, dtype=BF, device="cuda")
    g = torch.Generator("cuda").manual_seed(9)
    a[n - 1] = (torch.randn(1, r, k, generator=g, device="cuda") / k ** 0.5).to(BF)
    b[n - 1] = torch.randn(256, r, generator=g, device="cuda").to(BF)
    pool = hb.make_adapters(a, b, torch.full((n,), r, dtype=torch.int32, device="cuda"), torch.ones(n, device="cuda"), cols)
    x, y = torch.randn(3, k, generator=g, device="cuda").to(BF), torch.zeros(3, 256, dtype=BF, device="cuda")
    plan, ws = hb.hb_adapters_plan(pool, [1, 2], [n - 1, n - 1], sms())
    out = torch.empty_like(y)
    hb.hb_adapters(pool, plan, x, [y], [out], ws)
    want = x.double() @ a[n - 1, 0].double().T @ b[n - 1].double().T
    assert torch.allclose(out.double(), want, rtol=2.0 ** -7, atol=2e-3)


def test_two_streams_with_workspaces_of_their_own():
    hb = lib()
    cases = [Case([1] * 20 + [400], [i % 5 for i in range(21)], 1024, (512, 128), 5, 32, seed=i) for i in (1, 2)]
    want = [c.run() for c in cases]
    plans = [c.plan() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.empty_like(y) for y in c.y] for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, (plan, ws), st, o in zip(cases, plans, streams, outs):
            hb.hb_adapters(c.pool, plan, c.x, c.y, o, ws, stream=st)
    torch.cuda.synchronize()
    hb.hb_check()
    assert all(torch.equal(a, b) for o, w in zip(outs, want) for a, b in zip(o, w))


def test_calls_that_follow_one_another_in_place():
    """Through one workspace, each on the last one's results, beside other launches."""
    hb = lib()
    c = Case([1] * 20 + [400, 7], [i % 5 for i in range(22)], 256, (256,), 5, 32, seed=3)
    plan, ws = c.plan()
    y = c.y[0].clone()
    apart = c.y[0]
    for _ in range(8):
        hb.hb_adapters(c.pool, plan, c.x, [y], [y], ws)
        hb.hb_norm(x=y, z=y)
        out = torch.empty_like(apart)
        hb.hb_adapters(c.pool, plan, c.x, [apart], [out], ws)
        torch.cuda.synchronize()
        apart = torch.empty_like(out)
        hb.hb_norm(x=out, z=apart)
        torch.cuda.synchronize()
    assert torch.equal(y, apart)


def test_long_prompts_over_many_columns():
    """Tiles for more than one round of clusters, over a long K."""
    for cols, r in (((256,), 24), ((128, 64, 64), 64)):
        Case([3200, 1, 3100], [0, 1, 1], 7168, cols, 2, r, seed=r, ranks=[r, r - 11]).check_both()
