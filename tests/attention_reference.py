"""64-bit definitions of the attention layer's operators (numpy).  No code is shared with the library; the tolerances of
ops_reference apply where a test states no others."""
import numpy as np


def rotate(x, positions, frequencies, pairs, back=False):
    """x [T, heads, d] with its first 2 len(frequencies) channels rotated by position (or back)."""
    r = 2 * len(frequencies)
    if r == 0:
        return x.copy()
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(frequencies, dtype=np.float64)[None, :]
    turn = np.exp((-1j if back else 1j) * a)[:, None, :]
    out = x.copy()
    if pairs == "adjacent":
        z = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * turn
        out[..., 0:r:2], out[..., 1:r:2] = z.real, z.imag
    else:
        z = (x[..., :r // 2] + 1j * x[..., r // 2:r]) * turn
        out[..., :r // 2], out[..., r // 2:r] = z.real, z.imag
    return out


def head_forward(x, norm, w, eps, positions, frequencies, pairs):
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    return rotate(x, positions, frequencies, pairs)


def head_backward(x, norm, w, eps, positions, frequencies, pairs, g):
    """dx and dw (None without a weight)."""
    g = rotate(g, positions, frequencies, pairs, back=True)
    if not norm:
        return g, None
    size = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    hat = x / size
    dw = None if w is None else (g * hat).sum((0, 1))
    e = g if w is None else g * w
    return (e - hat * (e * hat).mean(-1, keepdims=True)) / size, dw
