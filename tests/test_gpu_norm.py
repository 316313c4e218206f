"""hb_norm on the GPU against its definition in 64 bits.

Tolerance: an output is rounded once (half a step: bf16 2^-8, fp32 2^-24 of
it).  Before that, in fp32: a mean of squares is a chain of at most 32 fused
products per thread and two trees of 5 sums (42 roundings, halved by the
root), the root itself 2 steps, the products and sums at most 8 more; each
2^-24 of terms no larger than |residual_scale x| + |branch_scale gate u|.  64
roundings cover the stream's, and as many more its norm's."""
import itertools

import numpy as np
import pytest
import torch

from _hbutil import lib
from oracle import block as ob

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -24


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def make(rows, width, seed, dtype=BF, gap=0, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, width + gap, generator=g, device="cuda") * size).to(dtype)[:, :width]


def case(rows, width, form, gate=None, dtype=BF, gap=0, seed=0):
    """The tensors of a call: form is a set of letters, x y p(ost) w(eights before) o(ut) z."""
    t = {"x": make(rows, width, seed, dtype, gap, 3.0) if "x" in form else None,
         "y": make(rows, width, seed + 1, BF, gap) if "y" in form else None,
         "w_post": 1 + 0.3 * make(1, width, seed + 2)[0] if "p" in form else None,
         "w_pre": 1 + 0.3 * make(1, width, seed + 3)[0] if "w" in form else None,
         "gate": None if gate is None else make(rows if gate == "row" else 1, width, seed + 4, BF, gap),
         "x_out": make(rows, width, seed + 5, dtype, gap) if "o" in form else None,
         "z": make(rows, width, seed + 6, BF, gap) if "z" in form else None}
    if gate == "vector":
        t["gate"] = t["gate"][0].contiguous()
    return t


def expected(t, **kw):
    names = dict(eps=kw.get("eps", 1e-6), residual_scale=kw.get("residual_scale", 1.0),
                 branch_scale=kw.get("branch_scale", 1.0), offset=kw.get("weight_offset", 0.0))
    ins = {k: f64(t[k]) for k in ("x", "y", "gate", "w_post", "w_pre")}
    new, z = ob.norm(**ins, **names)
    # the size of what the stream is summed from
    part = 0.0 if ins["x"] is None else np.abs(names["residual_scale"] * ins["x"])
    if ins["y"] is not None:
        zero = dict(ins, x=None, w_pre=None)
        part = part + np.abs(ob.norm(**zero, **names)[0])
    # what the norm multiplies the stream with
    gain = 1.0 if ins["w_pre"] is None else np.abs(names["offset"] + ins["w_pre"])
    with np.errstate(all="ignore"):
        gain = gain / np.sqrt(np.mean(new * new, -1, keepdims=True) + names["eps"])
    return new, z, part, gain


def close(got, want, parts, rounding):
    got = f64(got)
    assert np.isfinite(got).all()
    bound = np.abs(want) * rounding + parts
    assert (np.abs(got - want) <= bound).all(), f"worst excess {(np.abs(got - want) - bound).max():.3e}"


def check(t, want, dtype=BF):
    new, z, part, gain = want
    if t["x_out"] is not None:
        close(t["x_out"], new, 64 * ULP * part, 2.0 ** -8 if dtype is BF else ULP)
    if t["z"] is not None:
        close(t["z"], z, 128 * ULP * (part * gain + np.abs(z)) * (1 + 2.0 ** -8), 2.0 ** -8)


FORMS = ["xwz", "xz", "xyoz", "xywoz", "xyo", "xypo", "xypwoz", "yoz", "ypwz", "xywz"]


@pytest.mark.parametrize("rows,width", [(1, 8), (3, 16), (5, 248), (2, 256), (1, 1000), (700, 1024), (3, 4096),
                                        (331, 4104), (1100, 4096), (4100, 1032), (600, 8192), (1, 8192), (2, 8200), (310, 16384), (1500, 40), (1, 7168)])
def test_against_the_definition(rows, width):
    hb = lib()
    for i, (form, gate, dtype) in enumerate(itertools.product(FORMS, (None, "channel", "row"), (BF, F32))):
        if gate and "y" not in form:
            continue
        if rows * width > 1 << 21 and i % 5:
            continue
        kw = dict(eps=1e-5, residual_scale=[1.0, 0.7][i % 2], branch_scale=[1.0, -0.4][i % 3 == 0],
                  weight_offset=float(i % 2))
        t = case(rows, width, form, gate, dtype, seed=10 * i)
        want = expected(t, **kw)
        hb.hb_norm(**t, **kw)
        check(t, want, dtype)
    hb.hb_check()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [8, 1016])
def test_what_stands_between_rows_stays(gap, dtype):
    hb = lib()
    rows, width = (37, 520) if gap == 8 else (2500, 2056)
    t = case(rows, width, "xypwoz", "row", dtype, gap)
    for name in ("x", "y", "gate"):                          # and is not read
        t[name]._base[:, width:] = float("nan")
    outs = {n: t[n]._base.clone() for n in ("x_out", "z")}
    want = expected(t)
    hb.hb_norm(**t)
    check(t, want, dtype)
    for n, was in outs.items():
        assert torch.equal(t[n]._base[:, width:], was[:, width:])


@pytest.mark.parametrize("rows,width", [(3, 8192), (400, 640), (2100, 2056)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_gives_the_same_bits(rows, width, dtype):
    hb = lib()
    t = case(rows, width, "xypwoz", "row", dtype)
    hb.hb_norm(**t)
    for over in ([("x_out", "x")], [("x_out", "x"), ("z", "y")], [("x_out", "x"), ("z", "gate")]):
        u = {k: v if v is None else v.clone() for k, v in t.items()}
        for out, source in over:
            u[out] = u[source]
        hb.hb_norm(**u)
        assert torch.equal(u["x_out"], t["x_out"]) and torch.equal(u["z"], t["z"])


def test_one_row_of_gates_in_every_form():
    hb = lib()
    t = case(50, 264, "xyoz", "channel")
    hb.hb_norm(**t)
    for gate in (t["gate"][0], t["gate"].expand(50, 264), t["gate"].repeat(50, 1)):
        u = dict(t, gate=gate, x_out=torch.empty_like(t["x_out"]), z=torch.empty_like(t["z"]))
        hb.hb_norm(**u)
        assert torch.equal(u["z"], t["z"]) and torch.equal(u["x_out"], t["x_out"])


@pytest.mark.parametrize("size", [1e30, 1e-18, 1e-22])
def test_squares_outside_of_fp32(size):
    """A row of large or tiny values, between ordinary ones, is normed as well."""
    hb = lib()
    for width in (64, 4096):
        t = case(5, width, "xypwoz")
        for n in "xy":
            t[n][2] = (t[n][2].float() * size).to(BF)
        want = expected(t, eps=0.0)
        hb.hb_norm(**t, eps=0.0)
        check(t, want)


def test_rows_of_zeros():
    hb = lib()
    t = case(4, 512, "xypwoz")
    t["x"][1] = 0
    t["y"][1] = 0
    want = expected(t)
    hb.hb_norm(**t)
    check(t, want)
    assert not t["z"][1].any() and not t["x_out"][1].any()
    hb.hb_norm(**t, eps=0.0)                                  # 0 / 0, as by the formula
    assert t["z"][1].isnan().all() and t["z"][0].isfinite().all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_stay_in_their_row(bad):
    hb = lib()
    t = case(5, 1024, "xywoz", "row")
    t["x"][3, 77] = bad
    hb.hb_norm(**t)
    new, z = (torch.from_numpy(a) for a in expected(t)[:2])
    z[3, 77] = float("nan")                                   # (inf / inf)
    for got, want in ((t["x_out"], new), (t["z"], z)):
        got = got.double().cpu()
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got.isinf(), want.isinf())
        rows = torch.tensor([0, 1, 2, 4])
        assert torch.allclose(got[rows], want[rows], rtol=2.0 ** -7, atol=1e-6)


def test_captured_replayed_and_on_another_stream():
    hb = lib()
    t = case(64, 4096, "xywoz", "channel", F32)
    hb.hb_norm(**t)
    want = t["x_out"].clone(), t["z"].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    t["z"].zero_()
    side.wait_stream(torch.cuda.current_stream())
    hb.hb_norm(**t, stream=side)
    side.synchronize()
    assert torch.equal(t["z"], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hb.hb_norm(**t)
        hb.hb_norm(x=t["x_out"], x_out=t["x_out"], residual_scale=0.5)
    for _ in range(3):
        t["z"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(t["z"], want[1]) and torch.equal(t["x_out"], 0.5 * want[0])


def test_offsets_past_32_bits():
    """Rows whose elements lie more than 2^32 apart."""
    hb = lib()
    rows, width, gap = 3, 64, (1 << 31) + 64
    base = torch.empty(rows * gap, dtype=BF, device="cuda")
    x = base.as_strided((rows, width), (gap, 1))
    z = base.as_strided((rows, width), (gap, 1), 4096)
    x.copy_(make(rows, width, 1))
    want = ob.norm(x=f64(x))[1]
    hb.hb_norm(x=x, z=z)
    close(z, want, 64 * ULP * np.abs(want), 2.0 ** -8)


def walked(rows, width):
    """The rows that the CTAs of the row-walking kernel meet, CTA by CTA (rows, rows a grid apart, ..), for shapes that it
    takes: bf16 streams of 1024 to 8192 columns and 4 Mi elements or more."""
    assert 1024 <= width <= 8192 and rows * width >= 4 << 20
    threads = -(-(-(-width // 8 // 4)) // 32) * 32
    grid = min(rows, min(16, 512 // threads) * torch.cuda.get_device_properties(0).multi_processor_count)
    return [list(range(c, rows, grid)) for c in range(grid)]


WALKED = [(4200, 1032), (2600, 2056), (1300, 4096), (1100, 8192)]


@pytest.mark.parametrize("size", [1e30, 1e-18, 1e-22])
@pytest.mark.parametrize("rows,width", WALKED)
def test_squares_outside_of_fp32_in_walked_rows(rows, width, size):
    """All rows of one CTA (its sums in 64 bits one behind the other), the second ones of some, the last one of another,
    in y, in x, in both."""
    hb = lib()
    ctas = walked(rows, width)
    special = ctas[5] + [c[1] for c in ctas[10:14]] + [ctas[20][-1], rows - 1]
    assert len(ctas[5]) >= 2
    t = case(rows, width, "xypwoz", "row")
    for i, r in enumerate(special):
        for n in ("y", "x", "xy")[i % 3] if i >= len(ctas[5]) else "xy":
            t[n][r] = (t[n][r].float() * size).to(BF)
    want = expected(t, eps=0.0)
    hb.hb_norm(**t, eps=0.0)
    hb.hb_check()
    check(t, want)


@pytest.mark.parametrize("rows,width", WALKED)
def test_zeros_and_values_that_are_not_finite_stay_in_their_walked_row(rows, width):
    hb = lib()
    ctas = walked(rows, width)
    t = case(rows, width, "xypwoz", "row")
    plain = {k: v if v is None else v.clone() for k, v in t.items()}
    hb.hb_norm(**plain, eps=0.0)
    zeros, nans, infs = ctas[3], ctas[4][:1] + ctas[6][1:], [ctas[7][0], ctas[8][-1]]
    for n in "xy":
        t[n][zeros] = 0
    t["x"][nans, 77] = float("nan")
    t["y"][infs, width - 1] = float("-inf")
    hb.hb_norm(**t, eps=0.0)
    hb.hb_check()
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[zeros + nans + infs] = True
    for n in ("x_out", "z"):
        assert torch.equal(t[n][~bad], plain[n][~bad])
    # 0 / 0 as by the formula; a NaN in its element of the stream and all of its norm; inf / inf likewise
    assert t["x_out"][zeros].isnan().all() and t["z"][zeros].isnan().all()
    assert (t["x_out"][nans].isnan().sum(1) == 1).all() and t["z"][nans].isnan().all()
    assert t["x_out"][infs, -1].isnan().all() and t["x_out"][infs, :-1].isfinite().all() and t["z"][infs].isnan().all()
    # with an eps zeros stay zeros
    hb.hb_norm(**t, eps=1e-6)
    assert not t["x_out"][zeros].any() and not t["z"][zeros].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", ["xypwoz", "xywoz", "xwz", "ypwz", "ypoz"])
@pytest.mark.parametrize("rows,width", [(5, 64), (5, 1024), (5, 2048), (5, 16384), (2600, 2056)])
@pytest.mark.parametrize("size", [1e-34, 1e-38, 1e-40])
def test_rows_of_numbers_below_the_smallest_normal_one(rows, width, form, dtype, size):
    """The root of such a row has no inverse in fp32.  Below 2^-126 a number's step is fixed: each of the four
    operations that make the sum may be off by half of 2^-149, the stream's rounding to bf16 by half of 2^-133, and
    z's by as much (an element of an ordinary row may be as small)."""
    hb = lib()
    kw = dict(eps=0.0, residual_scale=0.7, branch_scale=-0.4)
    t = case(rows, width, form, None, dtype)
    special = [2] if rows == 5 else walked(rows, width)[5] + [rows - 1]
    for n in "xy":
        if t[n] is not None:
            t[n][special] = (t[n][special].double() * size).to(t[n].dtype)
    want = expected(t, **kw)
    hb.hb_norm(**t, **kw)
    hb.hb_check()
    new, z, part, gain = want
    step = 4 * 2.0 ** -150
    if t["x_out"] is not None:
        narrow = 2.0 ** -134 if dtype is BF else 2.0 ** -150
        close(t["x_out"], new, 64 * ULP * part + step + narrow, 2.0 ** -8 if dtype is BF else ULP)
    if t["z"] is not None:
        close(t["z"], z, 128 * ULP * (part * gain + np.abs(z)) * (1 + 2.0 ** -8) + step * gain * (1 + 2.0 ** -8) + 2.0 ** -134,
              2.0 ** -8)
