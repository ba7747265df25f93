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


def visible(n, window, sinks):
    """[n, n]: whether row i of a sequence of n tokens sees key j."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def window_forward(cu, q, k, v, scale, window, sinks):
    """o [T, H, d], lse [H, T] and sum p |v|, which the rounding of the probabilities goes by."""
    T, H, d = q.shape
    g = H // k.shape[1]
    o, size, lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros((H, T))
    for a, b in zip(cu[:-1], cu[1:]):
        seen = visible(b - a, window, sinks)
        for h in range(H):
            s = np.where(seen, scale * (q[a:b, h] @ k[a:b, h // g].T), -np.inf)
            m = s.max(-1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(-1, keepdims=True)
            lse[h, a:b] = (m + np.log(l))[:, 0]
            o[a:b, h], size[a:b, h] = p / l @ v[a:b, h // g], p / l @ np.abs(v[a:b, h // g])
    return o, lse, size


def window_backward(cu, q, k, v, scale, window, sinks, do):
    """dq, dk, dv, and for each the sum of the magnitudes that the rounding of p, of ds and of the output in D = do . o goes by
    (o is off by u of sum p |v| and of itself, so D by u of 'loose')."""
    H = q.shape[1]
    g = H // k.shape[1]
    out = [np.zeros(x.shape) for x in (q, k, v)]
    size = [np.zeros(x.shape) for x in (q, k, v)]
    for a, b in zip(cu[:-1], cu[1:]):
        seen = visible(b - a, window, sinks)
        for h in range(H):
            Q, K, V, D = q[a:b, h], k[a:b, h // g], v[a:b, h // g], do[a:b, h]
            s = np.where(seen, scale * (Q @ K.T), -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            dp = D @ V.T
            delta = (p * dp).sum(-1, keepdims=True)
            ds = scale * p * (dp - delta)
            loose = (np.abs(D) * (p @ np.abs(V) + np.abs(p @ V))).sum(-1, keepdims=True)
            mag = scale * p * (np.abs(dp - delta) + loose)
            for n, (x, m) in enumerate(((ds @ K, mag @ np.abs(K)), (ds.T @ Q, mag.T @ np.abs(Q)), (p.T @ D, p.T @ np.abs(D)))):
                at = (slice(a, b), h) if n == 0 else (slice(a, b), h // g)
                out[n][at] += x
                size[n][at] += m
    return (*out, *size)


def ring_row(p, window, sinks):
    return p if p < sinks else sinks + (p - sinks) % window


def cache_fill(cu, slots, k, v, window, sinks, cache_k, cache_v):
    cache_k, cache_v = cache_k.copy(), cache_v.copy()
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if 0 <= slots[n] < len(cache_k):
            for p in range(b - a):
                cache_k[slots[n], :, ring_row(p, window, sinks)] = k[a + p]
                cache_v[slots[n], :, ring_row(p, window, sinks)] = v[a + p]
    return cache_k, cache_v


def window_step(slots, lengths, q, k, v, scale, window, sinks, cache_k, cache_v):
    """o, sum p |v| and the caches after it; a padding row's o is zeros."""
    B, H, d = q.shape
    g = H // k.shape[1]
    cache_k, cache_v = cache_k.copy(), cache_v.copy()
    o, size = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        s, n = slots[b], lengths[b]
        if not 0 <= s < len(cache_k) or n < 0:
            continue
        cache_k[s, :, ring_row(n, window, sinks)], cache_v[s, :, ring_row(n, window, sinks)] = k[b], v[b]
        rows = min(n + 1, window + sinks)
        for h in range(H):
            x = scale * (cache_k[s, h // g, :rows] @ q[b, h])
            p = np.exp(x - x.max())
            p /= p.sum()
            o[b, h], size[b, h] = p @ cache_v[s, h // g, :rows], p @ np.abs(cache_v[s, h // g, :rows])
    return o, size, cache_k, cache_v
