"""The 64-bit gradients the GPU tests compare with, against central differences of the 64-bit forward."""
import numpy as np
import pytest

import ops_reference as ref


def _difference(f, v, dv, eps=1e-6):
    return (f(v + eps * dv) - f(v - eps * dv)) / (2 * eps)


@pytest.mark.parametrize("with_i,with_h0", [(True, True), (False, True), (True, False)])
def test_scan_gradients_against_differences(with_i, with_h0):
    rng = np.random.default_rng(1)
    cu, D = [0, 5, 6, 17], 3
    T, N = cu[-1], len(cu) - 1
    x, g = rng.standard_normal((T, D)), -rng.uniform(0.01, 1.0, (T, D))
    i = rng.uniform(size=(T, D)) if with_i else None
    h0 = rng.standard_normal((N, D)) if with_h0 else None
    dh, dfinal = rng.standard_normal((T, D)), rng.standard_normal((N, D))

    def loss(x, i, g, h0):
        h, final = ref.scan_forward(cu, x, i, g, h0)
        return (h * dh).sum() + (final * dfinal).sum()

    dx, di, dg, dh0 = ref.scan_backward(cu, x, i, g, h0, dh, dfinal)
    d = rng.standard_normal((T, D))
    # central differences of a smooth loss: relative error of order eps^2 plus rounding 1e-16 / eps
    np.testing.assert_allclose(_difference(lambda v: loss(v, i, g, h0), x, d), (dx * d).sum(), rtol=1e-6)
    np.testing.assert_allclose(_difference(lambda v: loss(x, i, v, h0), g, d), (dg * d).sum(), rtol=1e-6)
    if with_i:
        np.testing.assert_allclose(_difference(lambda v: loss(x, v, g, h0), i, d), (di * d).sum(), rtol=1e-6)
    e = rng.standard_normal((N, D))
    base = np.zeros((N, D)) if h0 is None else h0
    np.testing.assert_allclose(_difference(lambda v: loss(x, i, g, v), base, e), (dh0 * e).sum(), rtol=1e-6)


@pytest.mark.parametrize("gate", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("group,post,ls,pre", [(0, True, True, True), (4, True, False, True), (4, True, True, False),
                                               (0, False, True, True)])
def test_norm_gradients_against_differences(gate, group, post, ls, pre):
    rng = np.random.default_rng(2)
    T, D, eps = 5, 12, 1e-3
    G = group or D
    v = {"r": rng.standard_normal((T, D)), "o": rng.standard_normal((T, D)),
         "z": None if gate == "none" else rng.standard_normal((T, D)),
         "w_post": 1 + 0.3 * rng.standard_normal(G) if post else None,
         "ls": 1 + 0.3 * rng.standard_normal(D) if ls else None,
         "w_pre": 1 + 0.3 * rng.standard_normal(D) if pre else None}
    dr_out, dy = rng.standard_normal((T, D)), rng.standard_normal((T, D)) if pre else None

    def forward(v):
        return ref.norm_forward(v["r"], v["o"], v["z"], gate, group, v["w_post"], 0.7, v["ls"], v["w_pre"], eps)

    def loss(v):
        r, y = forward(v)
        return (r * dr_out).sum() + (0.0 if y is None else (y * dy).sum())

    grads = ref.norm_backward(forward(v)[0], v["o"], v["z"], gate, group, v["w_post"], 0.7, v["ls"], v["w_pre"], eps,
                              dr_out, dy)
    for name, grad in zip(("r", "o", "z", "w_post", "ls", "w_pre"), grads):
        if v[name] is None:
            assert grad is None
            continue
        d = rng.standard_normal(v[name].shape)
        got = _difference(lambda w: loss({**v, name: w}), v[name], d)
        np.testing.assert_allclose(got, (grad * d).sum(), rtol=1e-5, atol=1e-8)


def test_decode_is_the_oracles_token_step():
    import oracle
    oracle.build()
    rng = np.random.default_rng(3)
    T, H, K = 5, 2, 128
    unit = lambda v: v / np.linalg.norm(v, axis=-1, keepdims=True)
    q, k = (unit(rng.standard_normal((T, H, K))).astype(np.float32) for _ in range(2))
    v = rng.standard_normal((T, H, K)).astype(np.float32)
    g = -rng.uniform(0.001, 0.2, (T, H, K)).astype(np.float32)
    beta = rng.uniform(size=(T, H)).astype(np.float32)
    h0 = rng.standard_normal((1, H, K, K)).astype(np.float32)
    want, final = oracle.forward([0, T], q, k, v, g, beta, h0=h0, scale=0.5)
    state = h0.astype(np.float64)
    for t in range(T):
        o, state = ref.decode(state, [0], *(a[t:t + 1].astype(np.float64) for a in (q, k, v, g, beta)), 0.5)
        np.testing.assert_allclose(o[0], want[t], rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(state, final, rtol=1e-9, atol=1e-12)
