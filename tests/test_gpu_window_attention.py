"""GPU tests of the window attention against its 64-bit definition (tests/attention_reference.py).

Tolerances.  u is half a step of the type (2^-8, fp16 2^-11).
  o     the probabilities are rounded to the type, u of each, and the output once more: u (sum p |v| + |o|); everything
        else is fp32 (scores, maxima, sums, exponentials; the bar of ops_reference, 2e-5 of the sizes involved).
        fp16 below its normal numbers rounds probabilities by up to 2^-25 of the row's largest: that times the number of keys and the
        largest value.
  lse   fp32: 2e-5 of its size, and of one.
"""
import numpy as np
import pytest

import attention_reference as ref
from ops_reference import ROUND, TOL32, torch_type

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1


def _cu(lengths):
    return [0] + list(np.cumsum(lengths))


def _draw(lengths, H, Hk, d, kind, seed=0, names=("q", "k", "v"), pad=0):
    """Tensors on the GPU (column ranges of wider rows where pad is given) and their 64-bit values."""
    import torch
    gen = torch.Generator().manual_seed(seed + sum(lengths) * 7 + H)
    t, T = torch_type(kind), sum(lengths)
    dev, wide = {}, {}
    for n in names:
        h = H if n in ("q", "do") else Hk
        x = torch.randn(T, h, d, generator=gen).to(t)
        wide[n] = x.double().numpy()
        if pad:
            rows = torch.full((T, h * d + pad), float("nan"), dtype=t, device="cuda")
            rows[:, pad // 2 // 8 * 8:][:, :h * d] = x.flatten(1).cuda()
            dev[n] = rows[:, pad // 2 // 8 * 8:][:, :h * d].unflatten(1, (h, d))
        else:
            dev[n] = x.cuda()
    return dev, wide


def _plan(lengths):
    from context_kda_gb300 import binding as kda
    plan = kda.kda_plan_segments(_cu(lengths), 1)
    return plan, kda.upload_plan(plan)


def _forward(plan, dev, scale, window, sinks, o=None):
    import torch
    from context_kda_gb300 import binding as kda
    T, H, d = dev["q"].shape
    o = torch.full((T, H, d), float("nan"), dtype=dev["q"].dtype, device="cuda") if o is None else o
    lse = torch.full((H, T), float("nan"), device="cuda")
    kda.kda_window_attention_forward(*plan, dev["q"], dev["k"], dev["v"], scale, window, sinks, o, lse)
    return o, lse


def _within(got, want, bound, what):
    x = got.double().cpu().numpy()
    assert np.all(np.isfinite(x)), what
    worst = float(np.max(np.abs(x - want) / bound))
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


def _check_forward(o, lse, lengths, w, kind, scale, window, sinks):
    o_ref, lse_ref, size = ref.window_forward(_cu(lengths), w["q"], w["k"], w["v"], scale, window, sinks)
    u = ROUND[kind] * 1.001
    tiny = 2.0 ** -25 * (1 + min(max(lengths), window + sinks)) * np.abs(w["v"]).max() if kind == "f16" else 0.0
    _within(o, o_ref, u * (size + np.abs(o_ref)) + TOL32 * (size + 1e-3) + tiny, "o")
    _within(lse, lse_ref, TOL32 * (1 + np.abs(lse_ref)), "lse")


def _case(lengths, H, Hk, d, kind, window, sinks, scale=None, pad=0, gain=1.0):
    import torch
    dev, w = _draw(lengths, H, Hk, d, kind, pad=pad)
    if gain != 1.0:
        dev["q"], w["q"] = dev["q"] * gain, (torch.from_numpy(w["q"]) * gain).numpy()
    scale = d ** -0.5 if scale is None else scale
    o, lse = _forward(_plan(lengths), dev, scale, window, sinks)
    _check_forward(o, lse, lengths, w, kind, scale, window, sinks)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [(1,), (5,), (128,), (129,), (256,), (700,), (300, 1, 77, 200), (1, 1, 1), (127, 128, 129, 257)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2)])
def test_everything_visible(lengths, H, Hk, d, kind):
    _case(lengths, H, Hk, d, kind, BIG, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (3, 1), (6, 1), (8, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (7, 0), (100, 4), (127, 17), (128, 1), (129, 128), (200, 33), (256, 5), (600, 4), (BIG, 128)])
def test_windows_and_sinks(window, sinks, H, Hk, d):
    _case((520, 1, 90, 333), H, Hk, d, "bf16", window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 2), (1000, 4)])
def test_long_sequence(window, sinks):
    _case((3001,), 2, 1, 128, "bf16", window, sinks)
    _case((2050,), 1, 1, 64, "f16", window, sinks)


@pytest.mark.parametrize("gain,scale", [(30.0, None), (1.0, 8.0), (1e-3, None), (1.0, 1e-30)])
def test_scores_of_any_size(gain, scale):
    """Scores of a hundred and more (maxima that grow along the row, probabilities of zero), and of next to nothing.  The scores'
    own error grows with them: 2^-24 sqrt(d) of sizes up to 300 is 2e-4, ten times the bar, so those get fp32 room: the
    comparison is with scores rounded nowhere, and p moves by that much relatively."""
    import torch
    lengths, d = (400, 150), 64
    dev, w = _draw(lengths, 2, 1, d, "bf16")
    dev["q"] = (dev["q"].float() * gain).to(torch.bfloat16)
    w["q"] = dev["q"].double().cpu().numpy()
    scale = d ** -0.5 if scale is None else scale
    o, lse = _forward(_plan(lengths), dev, scale, 200, 2)
    o_ref, lse_ref, size = ref.window_forward(_cu(lengths), w["q"], w["k"], w["v"], scale, 200, 2)
    most = scale * np.abs(w["q"]).max() * np.abs(w["k"]).max() * d
    moved = TOL32 + 2.0 ** -24 * 4 * most
    _within(o, o_ref, ROUND["bf16"] * 1.001 * (size + np.abs(o_ref)) + moved * (size + 1e-3), "o")
    _within(lse, lse_ref, moved * (1 + np.abs(lse_ref)), "lse")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rows_of_a_wider_matrix(kind):
    _case((140, 260), 4, 2, 128, kind, 150, 3, pad=72)
    _case((140, 260), 3, 3, 64, kind, 90, 1, pad=8)


def test_one_projection():
    """q, k, v as column ranges of one tensor, the output into a range of another; what lies between stays as it was."""
    import torch
    lengths, H, Hk, d = (333, 100), 4, 2, 64
    dev, w = _draw(lengths, H, Hk, d, "bf16")
    rows = torch.cat([dev[n].flatten(1) for n in ("q", "k", "v")], 1)
    cut = rows.split([H * d, Hk * d, Hk * d], dim=1)
    fused = {n: c.unflatten(1, (-1, d)) for n, c in zip(("q", "k", "v"), cut)}
    out = torch.full((433, H * d + 64), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = _forward(_plan(lengths), fused, 0.1, 64, 2, o=out[:, 32:32 + H * d].unflatten(1, (H, d)))
    _check_forward(o, lse, lengths, w, "bf16", 0.1, 64, 2)
    assert bool((out[:, :32] == 7).all()) and bool((out[:, 32 + H * d:] == 7).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window,sinks", [(BIG, 0), (40, 0), (40, 3), (150, 2)])
@pytest.mark.parametrize("H,Hk", [(2, 1), (1, 1)])
def test_bad_values_reach_only_the_rows_that_see_them(bad, window, sinks, H, Hk):
    """An infinite or NaN entry of v: every other row and channel keeps its bits, the rows that see it get it (or NaN)."""
    import torch
    lengths, d = (300, 130), 64
    plan = _plan(lengths)
    dev, _ = _draw(lengths, H, Hk, d, "bf16")
    want, lse = _forward(plan, dev, 0.125, window, sinks)
    seen = ref.visible(300, window, sinks)
    for at in (0, 2, 100, 127, 128, 299):
        v = dev["v"].clone()
        v[at, 0, 5] = bad
        got, lse2 = _forward(plan, dict(dev, v=v), 0.125, window, sinks)
        assert torch.equal(lse, lse2)
        same = (got.view(torch.int16) == want.view(torch.int16)).cpu().numpy()
        g = H // Hk
        hit = np.zeros(same.shape, dtype=bool)
        hit[:300, :g, 5] = seen[:, at, None]
        assert np.array_equal(~same, hit), at
        x = got.float().cpu().numpy()[hit]
        assert not np.any(np.isfinite(x))
        if np.isinf(bad):
            assert np.all(np.isnan(x) | (x == bad))


@pytest.mark.parametrize("name", ["q", "k"])
def test_bad_scores_reach_only_the_rows_that_see_them(name):
    import torch
    lengths, d = (300, 130), 64
    plan = _plan(lengths)
    dev, _ = _draw(lengths, 2, 1, d, "bf16")
    want, _ = _forward(plan, dev, 0.125, 70, 2)
    seen = ref.visible(300, 70, 2)
    for at in (1, 130, 299):
        x = dev[name].clone()
        x[at, 0] = float("nan")
        got, _ = _forward(plan, dict(dev, **{name: x}), 0.125, 70, 2)
        changed = (got.view(torch.int16) != want.view(torch.int16)).any(-1).cpu().numpy()
        hit = np.zeros(changed.shape, dtype=bool)
        if name == "q":
            hit[at, 0] = True
        else:
            hit[:300] = seen[:, at, None]
        assert np.array_equal(changed, hit), at


def test_a_sequence_sees_no_other():
    """NaN and infinities all over a neighbour change no bit."""
    import torch
    lengths, d = (77, 200, 130), 128
    plan = _plan(lengths)
    dev, _ = _draw(lengths, 2, 1, d, "bf16")
    want, lse = _forward(plan, dev, 0.1, 100, 4)
    for first, last in ((0, 77), (277, 407)):
        bad = {n: x.clone() for n, x in dev.items()}
        for n in bad:
            bad[n][first:last] = float("nan")
        bad["v"][first] = float("inf")
        got, lse2 = _forward(plan, bad, 0.1, 100, 4)
        keep = [i for i in range(407) if not first <= i < last]
        assert torch.equal(got[keep].view(torch.int16), want[keep].view(torch.int16))
        assert torch.equal(lse2[:, keep], lse[:, keep])


def test_without_lse_on_another_stream_and_in_a_graph():
    import torch
    from context_kda_gb300 import binding as kda
    lengths = (600, 300)
    plan = _plan(lengths)
    dev, _ = _draw(lengths, 4, 2, 128, "bf16")
    want, _ = _forward(plan, dev, 0.1, 150, 4)
    outs = [torch.empty_like(dev["q"]) for _ in range(2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kda.kda_window_attention_forward(*plan, dev["q"], dev["k"], dev["v"], 0.1, 150, 4, outs[0], None, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_window_attention_forward(*plan, dev["q"], dev["k"], dev["v"], 0.1, 150, 4, outs[1], None)
    outs[1].zero_()
    graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))
    assert kda.kda_device_status() == kda.KDA_OK


def test_many_short_sequences():
    """More sequences than one step of the search over them looks at."""
    lengths = [1 + (i * 7) % 40 for i in range(1500)]
    _case(lengths, 1, 1, 64, "bf16", 9, 1)


@pytest.mark.parametrize("count", [31, 32, 33, 64, 65])
def test_sequences_around_the_number_whose_starts_come_with_the_launch(count):
    lengths = [1 + (i * 37) % 300 for i in range(count)]
    _case(lengths, 2, 1, 64, "bf16", 100, 2)
    _case(lengths, 1, 1, 128, "f16", BIG, 0)


def test_a_device_plan_of_another_launch_is_refused():
    import torch
    from context_kda_gb300 import binding as kda
    dev, _ = _draw((200,), 1, 1, 64, "bf16")
    plan, other = _plan((200,)), _plan((90, 110))
    o = torch.full((200, 1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    assert kda.kda_device_status() == kda.KDA_OK
    kda.kda_window_attention_forward(plan[0], other[1], dev["q"], dev["k"], dev["v"], 0.1, 50, 0, o, None)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert bool((o == 3).all())
