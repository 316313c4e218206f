"""hb_rope and hb_rope_phases on the host (no GPU): the phases against the
frequencies' definition, and the refusals."""
import ctypes
from decimal import Decimal

import numpy as np
import pytest
import torch

from _hbutil import host_batch, lib
from _turns import exact_turns
from oracle import block as ob

AT = 1 << 32      # device addresses that no call here follows


@pytest.mark.parametrize("scaling,by", [("none", 1.0), ("linear", 3.0), ("base", 8.0), ("parts", 16.0)])
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 5e5), (128, 1e6), (80, 1.5)])
def test_phases_are_the_frequencies_in_turns(rot, base, scaling, by):
    got = lib().rope_phases(rot, base, scaling, by, original_context=8192, parts=(1.0, 32.0))
    want = ob.rope_frequencies(rot, base, scaling, by, 8192) / (2 * np.longdouble(np.pi))
    # (computed in 64 bits: a power, a division and the turn, each to 2^-52 or so)
    got = got.astype(np.longdouble) / np.longdouble(2) ** 64
    assert got.shape == (rot // 2,) and (np.abs(got - want) <= want * 2.0 ** -49 + 2.0 ** -63).all()


@pytest.mark.parametrize("kw,status", [
    (dict(rotary_dim=0), 2), (dict(rotary_dim=24), 2), (dict(rotary_dim=-16), 2), (dict(base=1.0), 1),
    (dict(base=float("nan")), 1), (dict(base=float("inf")), 1), (dict(scaling="linear", scale_by=0.5), 1),
    (dict(scaling="base", scale_by=float("nan")), 1), (dict(scaling="parts", scale_by=2.0), 1),
    (dict(scaling="parts", scale_by=2.0, original_context=4096, parts=(4.0, 4.0)), 1),
    (dict(scaling="parts", scale_by=2.0, original_context=4096, parts=(-1.0, 4.0)), 1),
])
def test_phases_refuse(kw, status):
    hb = lib()
    with pytest.raises(hb.HbError) as e:
        hb.rope_phases(**{"rotary_dim": 64, **kw})
    assert e.value.status == status
    with pytest.raises(ValueError, match="scaling"):
        hb.rope_phases(64, scaling="log")
    assert hb.load().hb_rope_phases(64, 1e4, 4, 1.0, 0.0, 0.0, 0.0, None) == 1


def call(hb, batch=None, rope=None, **kw):
    b = host_batch(hb, [(1, 40), (5, 9)], hq=8, hkv=2, d=64, num_pages=8)[0]
    for k, v in (batch or {}).items():
        setattr(b, k, v)
    r = hb.HbRopeParams()
    r.rotary_dim, r.interleaved, r.factor, r.eps, r.phases = 64, 0, 1.0, 1e-6, AT + (9 << 24)
    for k, v in (rope or {}).items():
        setattr(r, k, v)
    a = dict(q=AT, qs=512, k=AT + (1 << 24), ks=128, v=AT + (2 << 24), vs=128, qo=AT + (3 << 24), ko=AT + (4 << 24),
             kc=AT + (5 << 24), vc=AT + (6 << 24))
    a.update(kw)
    return hb.load().hb_rope(ctypes.byref(b), ctypes.byref(r), a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                             a["qo"], a["ko"], a["kc"], a["vc"], None)


@pytest.mark.parametrize("want,kw", [
    (3, dict(batch=dict(head_dim=96))), (3, dict(batch=dict(page_size=8))), (2, dict(batch=dict(num_pages=0))),
    (2, dict(rope=dict(rotary_dim=72))), (2, dict(rope=dict(rotary_dim=80))), (2, dict(rope=dict(rotary_dim=-16))),
    (1, dict(rope=dict(interleaved=2))), (1, dict(rope=dict(factor=float("nan")))), (1, dict(rope=dict(eps=-1.0))),
    (1, dict(rope=dict(phases=None))), (1, dict(rope=dict(phases=AT + (9 << 24) + 8))),
    (1, dict(rope=dict(q_weight=AT + (9 << 24) + 514))),
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(kc=None)), (1, dict(vc=None)),
    (1, dict(qo=None)), (1, dict(ko=None, kc=None, vc=None, v=None)),
    (1, dict(q=AT + 4)), (1, dict(qs=516)), (2, dict(qs=504)), (2, dict(ks=0)), (2, dict(vs=-128)),
])
def test_bad_arguments_are_refused(want, kw):
    assert call(lib(), **kw) == want


@pytest.mark.parametrize("kw", [
    dict(qo=AT + 16), dict(ko=AT + (1 << 24) + 256), dict(qo=AT + (1 << 24)), dict(ko=AT + (2 << 24)),
    dict(ko=AT + (3 << 24)), dict(kc=AT), dict(vc=AT + (2 << 24) - 64), dict(kc=AT + (6 << 24)),
    dict(kc=AT + (4 << 24) + 16), dict(rope=dict(phases=AT + (3 << 24))), dict(rope=dict(k_weight=AT + (5 << 24))),
    dict(qs=768, ks=768, vs=768, k=AT + 1024, v=AT + 1280, qo=AT + 16),        # columns of one array
    dict(qs=768, ks=768, vs=768, k=AT + 1008, v=AT + 1280, qo=AT),
    dict(qs=768, ks=640, k=AT + 1024, qo=AT),                                  # two strides
])
def test_operands_that_overlap_are_refused(kw):
    hb = lib()
    assert call(hb, **kw) == 1
    assert b"overlap" in hb.load().hb_last_error()


def test_no_tokens_are_no_work():
    assert call(lib(), batch=dict(total_q=0, num_seqs=0)) == 0


def test_tensors_are_checked_by_name():
    hb = lib()
    b, _, _ = host_batch(hb, [(1, 40), (5, 9)], hq=8, hkv=2, d=64, num_pages=8)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    r = hb.make_rope(64, device="cpu")
    q, k, c = z(6, 8, 64), z(6, 2, 64), z(8, 16, 2, 64)
    good = [b, r, q, k, k, z(6, 8, 64), z(6, 2, 64), c, c]
    wide = z(6, 12, 64)
    for at, junk, name in [
            (1, None, "make_rope"), (1, hb.HbRopeParams(), "make_rope"), (2, [1], "q and k"), (2, z(6, 8, 32), "q has shape"),
            (3, z(5, 2, 64), "k has shape"), (3, z(6, 2, 64, dtype=torch.float16), "k must be"), (4, None, "go together"),
            (4, z(6, 2, 64, dtype=torch.float32), "v must be"), (5, None, "q_out must be"), (5, wide[:, :8], "q_out must be contig"),
            (6, wide[:, :2], "k_out must be contig"), (7, None, "go together"), (7, z(9, 16, 2, 64), "k_cache has shape"),
            (8, z(8, 32, 2, 64)[:, ::2], "v_cache must be contig"), (2, z(6, 8, 128)[:, :, ::2], "q: each row"),
            (1, hb.make_rope(64, q_weight=z(128), device="cpu"), "head norms"), (0, b, "CUDA")]:
        args = list(good)
        args[at] = junk
        with pytest.raises(ValueError, match=name):
            hb.hb_rope(*args)
    with pytest.raises(ValueError, match="go together"):
        hb.hb_rope(b, r, q, k, None, q, k, c, None)
    for bad in (z(64, dtype=torch.float32), z(2, 64), z(128)[::2]):
        with pytest.raises(ValueError, match="k_weight"):
            hb.make_rope(64, k_weight=bad, device="cpu")


class Weight:
    """A head norm's weight on a device that is not here."""
    dtype = torch.bfloat16

    def __init__(self, index):
        self.index, self.device = index, torch.device("cuda", index)

    dim = lambda self: 1  # noqa: E731
    is_contiguous = lambda self: True  # noqa: E731
    numel = lambda self: 64  # noqa: E731
    data_ptr = lambda self: AT + (self.index << 24)  # noqa: E731
    get_device = lambda self: self.index  # noqa: E731


def test_head_norms_are_on_one_device():
    hb = lib()
    assert hb.make_rope(0, q_weight=Weight(1), k_weight=Weight(1)).device_index == 1
    for q, k in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="k_weight is on cuda"):
            hb.make_rope(0, q_weight=Weight(q), k_weight=Weight(k))


@pytest.mark.parametrize("scaling,by", [("none", 1.0), ("linear", 3.0), ("base", 8.0), ("parts", 16.0), ("parts", 1.5)])
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 5e5), (128, 1e6), (80, 1.5), (48, 1e8), (112, 1e4)])
def test_phases_are_off_by_less_than_2_to_the_minus_51_of_a_turn(rot, base, scaling, by):
    """What far positions multiply.  f <= 1 is computed in 64 bits: with u = 2^-53, its
    exponent is off by u and the power's base by 4 u (a power and a product, by at most 8
    here), which moves f by at most |f ln f| u + 4 u (f ln f is at most 1 / e); the power
    itself rounds by 2 u, the share of the parts by 6 u, the division by a turn by 2 u, and
    the fixed point cuts 2^-64.  Under 16 u of f, over a turn of 6.28: less than 3 u, or 2^-51."""
    got = lib().rope_phases(rot, base, scaling, by, original_context=8192, parts=(1.0, 32.0))
    worst = max(abs(Decimal(int(p)) / 2 ** 64 - t) for p, t in zip(got, exact_turns(rot, base, scaling, by)))
    assert worst < Decimal(3) / 2 ** 53
