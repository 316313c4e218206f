"""hb_norm's refusals on the host (no GPU): nothing is launched for them."""
import ctypes

import pytest
import torch

from _hbutil import lib

AT = 1 << 32      # device addresses that no call here follows


def args(hb, **kw):
    a = hb.HbNormArgs()
    a.rows, a.width = 4, 64
    a.x, a.y, a.gate, a.w_post, a.w_pre, a.x_out, a.z = (AT + (i << 24) for i in range(7))
    a.x_stride = a.y_stride = a.gate_stride = a.x_out_stride = a.z_stride = 64
    a.eps, a.residual_scale, a.branch_scale = 1e-6, 1.0, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def status(hb, **kw):
    return hb.load().hb_norm(ctypes.byref(args(hb, **kw)), None)


@pytest.mark.parametrize("want,kw", [
    (1, dict(reserved=1)), (1, dict(stream_type=2)), (1, dict(stream_type=-1)),
    (2, dict(rows=-1)), (2, dict(width=0)), (3, dict(width=12)), (3, dict(width=16392)),
    (1, dict(x=None, y=None, gate=None, w_post=None)), (1, dict(x_out=None, z=None, w_pre=None)),
    (1, dict(y=None, w_post=None)), (1, dict(y=None, gate=None)), (1, dict(z=None)),
    (1, dict(eps=-1e-6)), (1, dict(eps=float("nan"))), (1, dict(eps=float("inf"))),
    (1, dict(residual_scale=float("nan"))), (1, dict(branch_scale=float("inf"))), (1, dict(weight_offset=float("nan"))),
    (1, dict(x=AT + 8)), (1, dict(z=AT + (6 << 24) + 2)), (1, dict(w_pre=AT + (4 << 24) + 4)),
    (1, dict(x_stride=68)), (2, dict(x_stride=56)), (2, dict(y_stride=0)), (2, dict(z_stride=-64)),
])
def test_bad_arguments_are_refused(want, kw):
    assert status(lib(), **kw) == want


def test_null_arguments_are_refused():
    assert lib().load().hb_norm(None, None) == 1


@pytest.mark.parametrize("kw", [
    dict(x_out=AT + 128), dict(x_out=AT + 16), dict(z=AT + (1 << 24) - 128), dict(x_out=AT + (6 << 24)),
    dict(z=AT + (3 << 24)), dict(x_out=AT + (4 << 24)),
    dict(gate_stride=0, z=AT + (2 << 24)),                     # one row of gates is read by all
    dict(stream_type=1, z=AT),                                 # fp32 rows are no place for bf16 ones
    dict(stream_type=1, x_out=AT + (1 << 24)),
    dict(x_stride=128, x_out=AT),                              # in place with another stride
    dict(x_stride=128, x_out_stride=128, x_out=AT + 64),       # side by side, but not apart
])
def test_operands_that_overlap_are_refused(kw):
    hb = lib()
    assert status(hb, **kw) == 1
    assert b"overlap" in hb.load().hb_last_error()


@pytest.mark.parametrize("kw", [
    dict(x_out=AT), dict(z=AT + (1 << 24)), dict(z=AT + (2 << 24)), dict(gate_stride=0),
    dict(x_stride=128, x_out_stride=128, x_out=AT + 128),      # columns of one array
    dict(y=None, gate=None, w_post=None), dict(x=None), dict(stream_type=1, x_out=AT),
])
def test_no_rows_are_no_work(kw):
    """(The checks that come before are passed, and no device is asked for.)"""
    assert status(lib(), rows=0, **kw) == 0


def test_tensors_are_checked_by_name():
    hb = lib()
    b = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    x = b(4, 64)
    for kw, name in [(dict(x=[1]), "x or y"), (dict(x=b(64)), "x or y"), (dict(x=x, z=b(4, 32)), "z has shape"),
                     (dict(x=x, y=b(4, 64, dtype=torch.float16), z=x), "y must be"),
                     (dict(x=b(4, 64, dtype=torch.float64), z=x), "x must be"),
                     (dict(x=x, x_out=b(4, 64, dtype=torch.float32)), "x_out must be"),
                     (dict(x=x, z=x, w_pre=b(32)), "w_pre has shape"), (dict(x=x, z=x, w_pre=3), "w_pre must be"),
                     (dict(x=x.expand(4, 64)[:, ::2], z=b(4, 32)), "contiguous"),
                     (dict(x=x, y=x, z=x, gate=b(2, 64)), "gate"), (dict(x=x, y=x, z=x, gate=b(4)), "gate"),
                     (dict(x=x, y=x, z=x, gate="g"), "gate"), (dict(x=x, z=x), "CUDA"), (dict(x=b(4, 0), z=b(4, 0)), "width|CUDA")]:
        with pytest.raises(ValueError, match=name):
            hb.hb_norm(**kw)
