"""Oracle for what a transformer block does around its attention and linear
layers (fp64, CPU): norms, rotary positions, low-rank adapters.

TEST INFRASTRUCTURE, like the rest of `oracle/`: only tests import it; it
shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def rms_norm(v, w, eps, offset=0.0) -> np.ndarray:
    """v * (offset + w) / sqrt(mean(v^2) + eps) over the last axis; w None: ones."""
    v = np.asarray(v, np.float64)
    gain = 1.0 if w is None else offset + np.asarray(w, np.float64)
    with np.errstate(all="ignore"):
        return v / np.sqrt(np.mean(v * v, -1, keepdims=True) + eps) * gain


def norm(x=None, y=None, gate=None, w_post=None, w_pre=None, eps=1e-6, residual_scale=1.0, branch_scale=1.0,
         offset=0.0):
    """(new stream, its norm) of rows x, y [rows, width]."""
    new = 0.0
    if x is not None:
        new = residual_scale * np.asarray(x, np.float64)
    if y is not None:
        u = np.asarray(y, np.float64) if w_post is None else rms_norm(y, w_post, eps, offset)
        new = new + branch_scale * (u if gate is None else u * np.asarray(gate, np.float64))
    return new, rms_norm(new, w_pre, eps, offset)


def rope_frequencies(rotary_dim, base=10000.0, scaling="none", by=1.0, original=0.0, low=1.0, high=32.0) -> np.ndarray:
    """Radians per position of pairs 0 .. rotary_dim/2 - 1."""
    out = []
    for i in range(rotary_dim // 2):
        b = np.longdouble(base)
        if scaling == "base":
            b = b * np.longdouble(by) ** (np.longdouble(rotary_dim) / (rotary_dim - 2))
        f = b ** (-np.longdouble(2 * i) / rotary_dim)
        if scaling == "linear":
            f = f / by
        elif scaling == "parts":
            turns = original * f / (2 * np.longdouble(np.pi))
            if turns <= low:
                f = f / by
            elif turns < high:
                g = (turns - low) / (high - low)
                f = f * g + f / by * (1 - g)
        out.append(f)
    return np.array(out, np.longdouble)


def rotate(x, angle, interleaved=False, factor=1.0) -> np.ndarray:
    """Heads x [..., D] turned by angle [..., rotary_dim / 2] (radians)."""
    x = np.asarray(x, np.float64)
    out, half = x.copy(), angle.shape[-1]
    c, s = np.cos(angle) * factor, np.sin(angle) * factor
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        out[..., b] = x[..., a] * s[..., i] + x[..., b] * c[..., i]
    return out


def adapters(x, ys, q_len, adapter, a, b, rank, scale):
    """The outputs of a shared projection (ys, one array per destination) with
    each sequence's own low-rank product added: a [n, destinations, R, K], b [n,
    sum of columns, R].  Also the sums of the products' absolute values."""
    x = np.asarray(x, np.float64)
    outs = [np.asarray(y, np.float64).copy() for y in ys]
    sizes = [np.zeros_like(o) for o in outs]
    t = 0
    for n, i in zip(q_len, adapter):
        if i >= 0:
            r, col = int(rank[i]), 0
            for j, out in enumerate(outs):
                w = b[i, col:col + out.shape[1], :r].astype(np.float64)
                low = a[i, j, :r].astype(np.float64)
                out[t:t + n] += float(scale[i]) * ((x[t:t + n] @ low.T) @ w.T)
                sizes[j][t:t + n] = abs(float(scale[i])) * ((np.abs(x[t:t + n]) @ np.abs(low).T) @ np.abs(w).T)
                col += out.shape[1]
        t += n
    return outs, sizes
