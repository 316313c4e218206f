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


def test_rotation_closed_forms():
    x = np.arange(1.0, 9.0)
    assert np.array_equal(ob.rotate(x, np.zeros(4)), x)
    quarter = ob.rotate(x, np.full(2, np.pi / 2))             # the first four dims, pairs (0, 2) and (1, 3)
    assert np.allclose(quarter, [-3, -4, 1, 2, 5, 6, 7, 8], atol=1e-15)
    quarter = ob.rotate(x, np.full(2, np.pi / 2), interleaved=True, factor=2.0)
    assert np.allclose(quarter, [-4, 2, -8, 6, 5, 6, 7, 8], atol=1e-15)


def test_rotated_products_depend_on_distances_alone():
    rng = np.random.default_rng(2)
    f = ob.rope_frequencies(16).astype(np.float64)
    q, k = rng.standard_normal((2, 16))
    for inter in (False, True):
        a = ob.rotate(q, 105 * f, inter) @ ob.rotate(k, 100 * f, inter)
        b = ob.rotate(q, 5 * f, inter) @ k
        assert np.isclose(a, b, rtol=1e-12)


def test_frequencies():
    assert np.allclose(ob.rope_frequencies(4, 100.0).astype(float), [1.0, 0.1])
    assert np.allclose(ob.rope_frequencies(4, 100.0, "linear", 4.0).astype(float), [0.25, 0.025])
    # the slowest pair of a scaled base is the slowest pair interpolated
    for n, by in ((32, 4.0), (128, 16.0)):
        assert np.isclose(float(ob.rope_frequencies(n, 1e4, "base", by)[-1]),
                          float(ob.rope_frequencies(n, 1e4, "linear", by)[-1]))
        plain, parts = (ob.rope_frequencies(n, 1e4, kind, by, 4096).astype(float) for kind in ("none", "parts"))
        turns = 4096 * plain / (2 * np.pi)
        assert np.allclose(parts[turns >= 32], plain[turns >= 32]) and np.allclose(parts[turns <= 1], plain[turns <= 1] / by)
        mid = (turns > 1) & (turns < 32)
        assert ((parts < plain) & (parts > plain / by))[mid].all() and mid.any()


def test_adapters_are_a_change_of_the_weights():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((7, 12)), rng.standard_normal((10, 12))
    a, b = rng.standard_normal((2, 2, 3, 12)), rng.standard_normal((2, 10, 3))
    y = x @ w.T
    outs, _ = ob.adapters(x, [y[:, :6], y[:, 6:]], [2, 1, 4], [1, -1, 0], a, b, [3, 2], [0.5, -2.0])
    got = np.concatenate(outs, 1)
    assert np.array_equal(got[2], y[2])
    for rows, i, r, s in ((slice(0, 2), 1, 2, -2.0), (slice(3, 7), 0, 3, 0.5)):
        for j, cols in enumerate((slice(0, 6), slice(6, 10))):
            tuned = w[cols] + s * b[i, cols, :r] @ a[i, j, :r]
            assert np.allclose(got[rows, cols], x[rows] @ tuned.T, rtol=1e-12, atol=1e-12)
