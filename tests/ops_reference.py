"""64-bit definitions of the operators around the KDA layer (numpy, loops over tokens), and the
tolerances their GPU tests use.  No code is shared with the library.

Tolerances.  Everything is computed in fp32 and rounded once to the output's type:
  rounding  half a unit in the last place of the type, relative: 2^-24 (fp32), 2^-11 (fp16), 2^-8 (bf16, 8 bits),
            and for fp16 half its smallest subnormal, 2^-25;
  fp32      a value is reached through n fp32 operations of relative error 2^-24 each (an exponential,
            2^-23), whose errors add up as a random walk of at most a few hundred steps in these tests:
            sqrt(400) 2^-23 = 2.4e-6 of the sizes involved; the bar is eight times that, 2e-5, of the
            root mean square of the tensor (or of the value, where that is larger).
"""
import numpy as np

TOL32 = 2e-5
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def check(got, want, kind, what=""):
    """'got' (a torch tensor) against the 64-bit 'want' within the tolerances above."""
    x = got.double().cpu().numpy()
    y = np.asarray(want, dtype=np.float64)
    assert x.shape == y.shape, (what, x.shape, y.shape)
    if not y.size:
        return
    assert np.all(np.isfinite(x)), what
    rms = float(np.sqrt(np.mean(y * y)))
    bound = (ROUND[kind] * 1.001 + TOL32) * np.abs(y) + TOL32 * rms + (2.0 ** -25 if kind == "f16" else 0.0)
    worst = float(np.max(np.abs(x - y) / np.maximum(bound, 1e-300)))
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


def scan_forward(cu, x, i, g, h0):
    """h, final states and the state after every token, token by token."""
    T, D = x.shape
    u = x * (1.0 if i is None else i)
    a = np.exp(g)
    h, N = np.zeros((T, D)), len(cu) - 1
    final = np.zeros((N, D))
    for n in range(N):
        s = np.zeros(D) if h0 is None else h0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            s = a[t] * s + u[t]
            h[t] = s
        final[n] = s
    return h, final


def scan_backward(cu, x, i, g, h0, dh, dfinal):
    T, D = x.shape
    N = len(cu) - 1
    h, _ = scan_forward(cu, x, i, g, h0)
    one = np.ones((T, D)) if i is None else i
    a = np.exp(g)
    dx, di, dg, dh0 = np.zeros((T, D)), np.zeros((T, D)), np.zeros((T, D)), np.zeros((N, D))
    for n in range(N):
        G = np.zeros(D) if dfinal is None else dfinal[n].copy()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            G = G + dh[t]
            before = h[t - 1] if t > cu[n] else (np.zeros(D) if h0 is None else h0[n])
            dx[t], di[t], dg[t] = one[t] * G, x[t] * G, a[t] * before * G
            G = a[t] * G
        dh0[n] = G
    return dx, di, dg, dh0


def saved_states(h, tile=128):
    T, D = h.shape
    out = np.zeros((-(-T // tile), D))
    for j in range(1, out.shape[0]):
        out[j] = h[tile * j - 1]
    return out


def _gate(kind, z):
    if kind == "none":
        return 1.0, 0.0
    p = 1.0 / (1.0 + np.exp(-z))
    return (p, p * (1 - p)) if kind == "sigmoid" else (z * p, p * (1 + z * (1 - p)))


def _rms(v, G, eps):
    T, D = v.shape
    w = v.reshape(T, D // G, G)
    return np.broadcast_to(np.sqrt((w * w).mean(-1, keepdims=True) + eps), w.shape).reshape(T, D)


def norm_forward(r, o, z, gate, group, w_post, scale, ls, w_pre, eps):
    """r' and y (None without w_pre); absent parts are None."""
    shape = (r if r is not None else o).shape
    D = shape[1]
    out = np.zeros(shape) if r is None else r.copy()
    if o is not None:
        n = o
        if w_post is not None:
            G = group or D
            n = o / _rms(o, G, eps) * np.tile(w_post, D // G)
        out = out + scale * (1.0 if ls is None else ls) * _gate(gate, z)[0] * n
    y = None if w_pre is None else out / _rms(out, D, eps) * w_pre
    return out, y


def norm_backward(r_out, o, z, gate, group, w_post, scale, ls, w_pre, eps, dr_out, dy):
    """dr, do, dz, dw_post, dls, dw_pre (None where there is nothing to differentiate)."""
    shape = (dr_out if dr_out is not None else dy).shape
    D = shape[1]
    dr = np.zeros(shape) if dr_out is None else dr_out.copy()
    dw_pre = None
    if w_pre is not None:
        rms = _rms(r_out, D, eps)
        e = dy * w_pre
        dw_pre = (dy * r_out / rms).sum(0)
        dr = dr + e / rms - r_out * (e * r_out).mean(-1, keepdims=True) / rms ** 3
    if o is None:
        return dr, None, None, None, None, dw_pre
    G = group or D
    act, slope = _gate(gate, z)
    hat = o if w_post is None else o / _rms(o, G, eps)
    n = hat if w_post is None else hat * np.tile(w_post, D // G)
    dls = None if ls is None else (scale * dr * act * n).sum(0)
    du = scale * dr * (1.0 if ls is None else ls)
    dz = None if z is None else du * n * slope
    dn = du * act
    if w_post is None:
        return dr, dn, dz, None, dls, dw_pre
    dw_post = (dn * hat).reshape(-1, D // G, G).sum((0, 1))
    e = (dn * np.tile(w_post, D // G))
    mean = (e * hat).reshape(-1, D // G, G).mean(-1, keepdims=True)
    mean = np.broadcast_to(mean, (shape[0], D // G, G)).reshape(shape)
    return dr, (e - hat * mean) / _rms(o, G, eps), dz, dw_post, dls, dw_pre


def decode(state, slots, q, k, v, g, beta, scale):
    """o and the new pool of states; a negative slot's row is zeros."""
    B, H, K = q.shape
    state, o = state.copy(), np.zeros(q.shape)
    for b in range(B):
        s = slots[b]
        if s < 0 or s >= state.shape[0]:
            continue
        for h in range(H):
            S = np.exp(g[b, h])[:, None] * state[s, h]
            d = beta[b, h] * (v[b, h] - S.T @ k[b, h])
            S = S + np.outer(k[b, h], d)
            state[s, h] = S
            o[b, h] = scale * (S.T @ q[b, h])
    return o, state
