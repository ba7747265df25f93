"""GPU tests of the window attention where scores are extreme.  Tolerances of test_gpu_window_attention.py; where they differ, the reason
stands with the test."""
import numpy as np
import pytest

import attention_reference as ref
from ops_reference import ROUND, TOL32, torch_type
from test_gpu_window_attention import BIG, _check_forward, _cu, _draw, _forward, _plan, _within
from test_gpu_window_gradients import _backward
from test_gpu_window_step import _check as _check_step, _draw as _draw_step, _step

pytestmark = pytest.mark.gpu


def _values(x):
    return x.double().cpu().numpy()


def _hide(dev, keys, how):
    """The score of every query with the given keys becomes minus infinity, by an infinite entry or by finite ones whose product passes
    fp32 (bf16 only); all other scores stay finite."""
    dev["q"][..., 0] = 1.0 if how == "infinite" else 2e19
    dev["k"][..., 0] = 0.0
    dev["k"][keys, :, 0] = float("-inf") if how == "infinite" else -3e19


@pytest.mark.parametrize("kind,how", [("bf16", "infinite"), ("bf16", "finite"), ("f16", "infinite")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1)])
@pytest.mark.parametrize("window,sinks", [(BIG, 0), (100, 3)])
def test_a_visible_score_of_minus_infinity(window, sinks, H, Hk, d, kind, how):
    """Its probability is zero and the row's others are as without it: also where it is the only key of its tile that a row sees (128, 256),
    and where it is all that a warp's rows see in their first tile."""
    lengths = (300, 150)
    dev, _ = _draw(lengths, H, Hk, d, kind)
    _hide(dev, [5, 128, 129, 130, 140, 256, 299, 301, 428], how)
    w = {n: _values(dev[n]) for n in ("q", "k", "v")}
    o, lse = _forward(_plan(lengths), dev, 0.125, window, sinks)
    _check_forward(o, lse, lengths, w, kind, 0.125, window, sinks)


def test_a_row_whose_scores_are_all_minus_infinity():
    """0 / 0, as the formula has it, in that row alone."""
    import torch
    dev, _ = _draw((300,), 1, 1, 64, "bf16")
    _hide(dev, [0], "infinite")
    o, lse = _forward(_plan((300,)), dev, 0.125, BIG, 0)
    assert bool(torch.isnan(o[0]).all()) and float(lse[0, 0]) == float("-inf")
    assert bool(torch.isfinite(o[1:].float()).all()) and bool(torch.isfinite(lse[0, 1:]).all())


def test_gradients_beside_scores_of_minus_infinity():
    """Finite entries whose products pass fp32 hide their keys; the gradients of all other channels are those of the formula."""
    lengths, window, sinks = (300, 150), 100, 3
    dev, _ = _draw(lengths, 2, 1, 64, "bf16", names=("q", "k", "v", "do"))
    _hide(dev, [5, 128, 129, 130, 140, 256, 299, 301, 428], "finite")
    w = {n: _values(x) for n, x in dev.items()}
    outs = _backward(_plan(lengths), dev, 0.125, window, sinks)
    want = ref.window_backward(_cu(lengths), w["q"], w["k"], w["v"], 0.125, window, sinks, w["do"])
    for n, got, x, size in zip(("dq", "dk", "dv"), outs, want[:3], want[3:]):
        x, size = x[..., 1:], size[..., 1:]
        _within(got[..., 1:], x, ROUND["bf16"] * 1.001 * (size + np.abs(x)) + TOL32 * (size + 1e-2 * np.abs(x).max() + 1e-3), n)


@pytest.mark.parametrize("kind,how", [("bf16", "infinite"), ("bf16", "finite"), ("f16", "infinite")])
@pytest.mark.parametrize("B,H,Hk,d", [(2, 4, 1, 64), (1, 2, 2, 128), (1, 20, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(20, 1), (900, 2)])
def test_a_visible_score_of_minus_infinity_in_the_step(window, sinks, B, H, Hk, d, kind, how):
    """Whole groups of 16 rows, a warp's first ones among them, and single rows."""
    cap = window + sinks
    dev, _ = _draw_step(B, H, Hk, d, kind, window, sinks, B)
    dev["k"][..., 0] = dev["cache_k"][..., 0] = 0.0
    dev["q"][..., 0] = 1.0 if how == "infinite" else 2e19
    hidden = list(range(0, 16)) + [17] + list(range(64, min(cap, 96))) + list(range(128, min(cap, 800)))
    dev["cache_k"][:, :, [r for r in hidden if r < cap], 0] = float("-inf") if how == "infinite" else -3e19
    w = {n: _values(x) for n, x in dev.items()}
    for n in (cap - 1, 3 * cap):
        d2 = {m: x.clone() for m, x in dev.items()}
        o = _step(d2, None, [n] * B, 0.125, window, sinks)
        _check_step(o, d2, w, list(range(B)), [n] * B, 0.125, window, sinks, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2)])
def test_a_row_keeps_its_bits_beside_any_other(H, Hk, kind):
    """Rows share a warp with rows of their own sequence and, in its last tile, of the next one.  Those rows' scores, here grown
    thirty times, have no part in a row's, whatever they do to their own maxima."""
    import torch
    lengths, d = (333, 333), 64
    dev, _ = _draw(lengths, H, Hk, d, kind)
    alone, lse1 = _forward(_plan(lengths[:1]), {n: x[:333].contiguous() for n, x in dev.items()}, 0.125, BIG, 0)
    packed, lse2 = _forward(_plan(lengths), dev, 0.125, BIG, 0)
    assert torch.equal(alone, packed[:333]) and torch.equal(lse1, lse2[:, :333])
    for rows in (slice(333, 666), slice(300, 333, 2), slice(130, 256, 3)):
        q = dev["q"].clone()
        q[rows] *= 30
        got, lse = _forward(_plan(lengths), dict(dev, q=q), 0.125, BIG, 0)
        keep = torch.ones(666, dtype=torch.bool)
        keep[rows] = False
        assert torch.equal(got[keep], packed[keep]) and torch.equal(lse[:, keep], lse2[:, keep]), rows


@pytest.mark.parametrize("kind,gain,scale", [("bf16", 1e6, 1.0), ("bf16", 6e17, 8.0), ("f16", 100.0, 64.0), ("f16", 1000.0, 1.0)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 1)])
def test_far_scores(H, Hk, kind, gain, scale):
    """Scores from 2^24 on, where an exponent of two in fp32 is off by one and more: o is the winner's value all the same.  Only rows whose
    two largest scores are further apart than 64 additions in fp32 are off (64 2^-24 of the largest) have a winner."""
    import torch
    lengths, d, window = (300,), 64, 40
    dev, _ = _draw(lengths, H, Hk, d, kind, seed=11)
    t = torch_type(kind)
    gen = torch.Generator().manual_seed(3)
    sign = lambda shape: torch.randint(0, 2, shape, generator=gen) * 2.0 - 1
    dev["q"] = (sign(dev["q"].shape) * gain).to(t).cuda()
    dev["k"] = (sign(dev["k"].shape) * gain * (1 + torch.arange(300).view(-1, 1, 1) % 61 / 64.0)).to(t).cuda()      # a size a key
    w = {n: _values(dev[n]) for n in ("q", "k", "v")}
    seen = ref.visible(300, window, 0)
    far = 0
    o, lse = _forward(_plan(lengths), dev, scale, window, 0)
    o_ref, lse_ref, size = ref.window_forward(_cu(lengths), w["q"], w["k"], w["v"], scale, window, 0)
    clear = np.zeros((300, H), dtype=bool)
    for h in range(H):
        s = w["q"][:, h] @ w["k"][:, h * Hk // H].T
        for i in range(300):
            x = np.sort(s[i, seen[i]])
            clear[i, h] = len(x) == 1 or x[-1] - x[-2] > 64 * 2.0 ** -24 * 4 * np.abs(s[i]).max()
        far = max(far, scale * np.abs(s).max())
    assert far > 2.0 ** 24 and clear.mean() > 0.8
    assert bool(torch.isfinite(o.float()).all()) and bool(torch.isfinite(lse).all())
    got = _values(o)
    bound = ROUND[kind] * 1.001 * (size + np.abs(o_ref)) + TOL32 * (size + 1e-3)
    assert np.all(np.abs(got - o_ref)[clear] <= bound[clear])
    got, want = lse.double().cpu().numpy().T[clear], lse_ref.T[clear]
    assert np.all(np.abs(got - want) <= TOL32 * (1 + np.abs(want)))


@pytest.mark.parametrize("kind,gain,scale", [("bf16", 1e6, 1.0), ("bf16", 2e18, 8.0), ("f16", 4000.0, 4.0), ("f16", 6000.0, 1.0)])
@pytest.mark.parametrize("H", [2, 12])
def test_far_scores_in_the_step(H, kind, gain, scale):
    """Every score is one product; the largest times scale log2(e) passes fp32 in the second case."""
    import torch
    window, sinks, d, n = 700, 2, 64, 702
    dev, _ = _draw_step(1, H, 1, d, kind, window, sinks, 1)
    t = torch_type(kind)
    order = torch.randperm(n, generator=torch.Generator().manual_seed(4))
    dev["q"].zero_()
    dev["q"][..., 3] = gain
    dev["k"][..., 3] = 0.0
    dev["cache_k"][0, 0, :, 3] = (gain * 8 * (0.25 + order / n)).to(t).cuda()
    dev["cache_k"][0, 0, int(order.argmax()), 3] = gain * 10.5      # above all others, which may be equal
    w = {m: _values(x) for m, x in dev.items()}
    o = _step(dev, None, [n - 1], scale, window, sinks)
    _check_step(o, dev, w, [0], [n - 1], scale, window, sinks, kind)


def test_very_many_small_probabilities_in_fp16():
    """One key 17.5 nats above 65,535 others whose values are all that counts.  A probability of 2^-25.2 is below fp16's numbers; the
    kernel keeps probabilities times a power of two, 2^7 at least: each is off by 2^-25 2^-7 of the largest at most."""
    import torch
    T, d = 65536, 64
    q = torch.zeros(T, 1, d, dtype=torch.float16, device="cuda")
    k, v = torch.zeros_like(q), torch.full_like(q, 8.0)
    q[..., 0], k[T - 100, 0, 0], v[T - 100] = 4.0, 4.375, 0.0
    o, lse = _forward(_plan((T,)), dict(q=q, k=k, v=v), 1.0, BIG, 0)
    rows = np.arange(T - 99, T)
    small = rows * np.exp(-17.5)                 # of all others together
    want = 8 * small / (1 + small)
    got = _values(o)[rows, 0]
    bound = 2 * ROUND["f16"] * want + TOL32 * want + 2.0 ** -32 * 8 * T
    assert np.all(np.abs(got - want[:, None]) <= bound[:, None])
    assert np.all(np.abs(_values(lse)[0, rows] - (17.5 + np.log1p(small))) <= TOL32 * 18)


@pytest.mark.parametrize("H", [1, 12])
def test_very_many_small_probabilities_in_fp16_in_the_step(H):
    """The same in a cache; the step keeps probabilities times 2^14 at least."""
    import torch
    n, d = 65536, 64
    ck = torch.zeros(1, 1, n, d, dtype=torch.float16, device="cuda")
    cv = torch.full_like(ck, 64.0)
    q = torch.zeros(1, H, d, dtype=torch.float16, device="cuda")
    q[..., 0], ck[0, 0, 0, 0], cv[0, 0, 0] = 4.0, 4.375, 0.0
    k, v = torch.zeros(1, 1, d, dtype=torch.float16, device="cuda"), torch.full((1, 1, d), 64.0, dtype=torch.float16, device="cuda")
    o = _step(dict(q=q, k=k, v=v, cache_k=ck, cache_v=cv), None, [n - 1], 1.0, n, 0)
    small = (n - 1) * np.exp(-17.5)
    want = 64 * small / (1 + small)
    assert np.all(np.abs(_values(o) - want) <= 2 * ROUND["f16"] * want + TOL32 * want + 2.0 ** -39 * 64 * n)
