"""The fp64 oracle of the block's norms, rotary positions and adapters, pinned
by closed forms and properties."""
import numpy as np

from oracle import block as ob


def test_norm_closed_forms():
    # a constant row has its own size as its rms
    x = np.full((2, 8), -3.0)
    new, z = ob.norm(x=x, eps=0.0)
    assert np.array_equal(new, x) and np.allclose(z, -1.0, rtol=1e-15)
    # 3, 4, 0, 0: rms 2.5
    y = np.array([[3.0, 4.0, 0.0, 0.0]])
    new, z = ob.norm(y=y, w_post=np.array([1.0, 2.0, 3.0, 4.0]), gate=np.array([0.5, 1.0, 1.0, 1.0]), eps=0.0,
                     branch_scale=10.0, offset=1.0)
    assert np.allclose(new, [[12.0, 48.0, 0.0, 0.0]], rtol=1e-15)
    assert np.allclose(ob.norm(x=y, eps=18.75)[1], y / 5.0, rtol=1e-15)


def test_norm_ignores_the_scale_of_a_row():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((3, 40)), rng.standard_normal(40)
    assert np.allclose(ob.norm(x=x, w_pre=w, eps=0.0)[1], ob.norm(x=7.0 * x, w_pre=w, eps=0.0)[1], rtol=1e-13)


def test_norm_sums_the_branches():
    rng = np.random.default_rng(1)
    x, y = rng.standard_normal((2, 3, 16))
    new, z = ob.norm(x=x, y=y, residual_scale=0.5, branch_scale=-2.0)
    assert np.allclose(new, 0.5 * x - 2 * y, rtol=1e-15)
    assert np.allclose(z, ob.norm(x=new)[1], rtol=1e-15)
