"""Per-head RMS norms and rotary positions in float64.

Test infrastructure only (see ``oracle/__init__.py``).  The pages have no counterpart; a pair (a, b)
is turned as the complex number a + ib by exp(i position frequency).
"""

import numpy as np


def norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def pairs(rot, interleaved):
    """Element numbers (first, second) of every pair."""
    p = np.arange(rot // 2)
    return (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)


def rotate(x, positions, freqs, weight=None, eps=1e-6, interleaved=False, sections=None, scale=1.0):
    """x [B][H][S][D], positions [axes][B][S], freqs [rot / 2]: (y, size) in float64, size the sum of the
    absolute values of the two elements that make up each one of y, from which error bounds follow.
    `sections`: pairs per axis."""
    y = norm(x, weight, eps)
    size = np.abs(y)
    if freqs is None or len(freqs) == 0:
        return y, size
    rot = 2 * len(freqs)
    sections = [rot // 2] if sections is None else list(sections)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = positions[axis].astype(np.float64).transpose(1, 2, 0) * freqs.astype(np.float64)
    i, j = pairs(rot, interleaved)
    z = (y[..., i] + 1j * y[..., j]) * (np.exp(1j * angle) * scale)[:, None]
    both = scale * (np.abs(y[..., i]) + np.abs(y[..., j]))
    y = y.copy()
    y[..., i], y[..., j] = z.real, z.imag
    size[..., i] = size[..., j] = both
    return y, size
