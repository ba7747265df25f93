"""GPU tests of the window attention's gradients against the 64-bit formulas (tests/attention_reference.py) and differences.

Tolerances.  u is half a step of the type.  p is rounded once for dv, ds = p (dp - D) once for dq and dk.  D = sum_c do_c o_c comes from an o
that is off by u (sum p |v_c| + |o_c|) in channel c, from the rounding of its probabilities and its own, so D is off by up to
u sum_c |do_c| (sum p |v_c| + |o_c|), which is no part of |dp| or |D|: terms of both signs cancel in those.  'size' is the sum
over p (|dp - D| + that) times the other factor's magnitude, and the bar u (size + |gradient|), and fp32's, 2e-5 of the sizes.  fp16: ds is kept in range
by a factor and p times 2^10, whose smallest steps are 2^-25 2^-10 of one."""
import numpy as np
import pytest

import attention_reference as ref
from ops_reference import ROUND, TOL32
from test_gpu_window_attention import BIG, _cu, _draw, _forward, _plan, _within

pytestmark = pytest.mark.gpu


def _backward(plan, dev, scale, window, sinks, outs=None, ws=None):
    import torch
    from context_kda_gb300 import binding as kda
    T, H, d = dev["q"].shape
    Hk = dev["k"].shape[1]
    o, lse = _forward(plan, dev, scale, window, sinks)
    outs = outs or [torch.full(dev[n].shape, float("nan"), dtype=dev[n].dtype, device="cuda") for n in ("q", "k", "v")]
    need = kda.kda_window_attention_workspace_bytes(plan[0], H, Hk, d, window, sinks)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
    kda.kda_window_attention_backward(*plan, dev["q"], dev["k"], dev["v"], scale, window, sinks, o, lse, dev["do"], *outs, ws)
    return outs


def _check(outs, lengths, w, kind, scale, window, sinks):
    want = ref.window_backward(_cu(lengths), w["q"], w["k"], w["v"], scale, window, sinks, w["do"])
    u = ROUND[kind] * 1.001
    for n, (got, x, size) in enumerate(zip(outs, want[:3], want[3:])):
        tiny = 2.0 ** -25 * max(1.0, np.abs(x).max()) if kind == "f16" else 0.0
        _within(got, x, u * (size + np.abs(x)) + TOL32 * (size + 1e-2 * np.abs(x).max() + 1e-3) + tiny, ("dq", "dk", "dv")[n])


def _case(lengths, H, Hk, d, kind, window, sinks, scale=None, pad=0, gain=1.0):
    import torch
    dev, w = _draw(lengths, H, Hk, d, kind, names=("q", "k", "v", "do"), pad=pad)
    if gain != 1.0:
        dev["do"], w["do"] = dev["do"] * gain, w["do"] * gain       # a power of two
    scale = d ** -0.5 if scale is None else scale
    outs = _backward(_plan(lengths), dev, scale, window, sinks)
    if gain != 1.0:
        outs, w = [x.double() / gain for x in outs], dict(w, do=w["do"] / gain)
    _check(outs, lengths, w, kind, scale, window, sinks)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths", [(1,), (5,), (64,), (65,), (128,), (129,), (700,), (300, 1, 77, 200), (1, 1, 1), (127, 128, 129, 257)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 2)])
def test_everything_visible(lengths, H, Hk, d, kind):
    _case(lengths, H, Hk, d, kind, BIG, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (3, 1), (8, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (7, 0), (63, 1), (64, 70), (100, 4), (127, 17), (128, 1), (129, 128), (200, 33), (600, 4), (BIG, 128)])
def test_windows_and_sinks(window, sinks, H, Hk, d):
    _case((520, 1, 90, 333), H, Hk, d, "bf16", window, sinks)


@pytest.mark.parametrize("window,sinks", [(33, 2), (1000, 4), (1024, 65), (1025, 1), (1, 128)])
def test_long_sequences(window, sinks):
    """More than one piece of the sinks' queries."""
    _case((3001, 40, 1100), 2, 1, 128, "bf16", window, sinks)
    _case((2050,), 1, 1, 64, "f16", window, sinks)


@pytest.mark.parametrize("gain", [2.0 ** -20, 2.0 ** -10, 2.0 ** 9])
def test_fp16_gradients_of_any_size(gain):
    """do over the range of a scaled loss (fp16's own smallest steps, 2^-25 of one, are in do already where it is small; it is multiplied up
    for the check, so its bar grows by them): relative accuracy stays as long as the outputs are normal numbers."""
    import torch
    lengths, H, Hk, d = (400, 150), 2, 1, 64
    dev, w = _draw(lengths, H, Hk, d, "f16", names=("q", "k", "v", "do"))
    dev["do"] = (dev["do"].float() * gain).half()
    w["do"] = dev["do"].double().cpu().numpy()
    outs = _backward(_plan(lengths), dev, 0.125, 130, 2)
    want = ref.window_backward(_cu(lengths), w["q"], w["k"], w["v"], 0.125, 130, 2, w["do"])
    for got, x, size in zip(outs, want[:3], want[3:]):
        _within(got, x, ROUND["f16"] * 1.001 * (size + np.abs(x)) + TOL32 * (size + 1e-2 * np.abs(x).max()) + 2.0 ** -25, "gradient")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rows_of_a_wider_matrix(kind):
    _case((140, 260), 4, 2, 128, kind, 150, 3, pad=72)
    _case((140, 260), 3, 3, 64, kind, 90, 1, pad=8)


def test_outputs_into_ranges_of_one_matrix():
    import torch
    lengths, H, Hk, d = (333, 100), 4, 2, 64
    dev, w = _draw(lengths, H, Hk, d, "bf16", names=("q", "k", "v", "do"))
    rows = torch.full((433, (H + 2 * Hk) * d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    cut = rows[:, 8:-8].split([H * d, Hk * d, Hk * d], dim=1)
    outs = _backward(_plan(lengths), dev, 0.1, 64, 2, outs=[c.unflatten(1, (-1, d)) for c in cut])
    _check(outs, lengths, w, "bf16", 0.1, 64, 2)
    assert bool((rows[:, :8] == 7).all()) and bool((rows[:, -8:] == 7).all())


def test_a_sequence_sees_no_other():
    import torch
    lengths, d = (77, 200, 130), 128
    plan = _plan(lengths)
    for kind in ("bf16", "f16"):
        dev, _ = _draw(lengths, 2, 1, d, kind, names=("q", "k", "v", "do"))
        want = _backward(plan, dev, 0.1, 100, 4)
        for first, last in ((0, 77), (277, 407)):
            bad = {n: x.clone() for n, x in dev.items()}
            for n in bad:
                bad[n][first:last] = float("nan")
            got = _backward(plan, bad, 0.1, 100, 4)
            keep = [i for i in range(407) if not first <= i < last]
            for a, b in zip(got, want):
                if kind == "bf16":
                    assert torch.equal(a[keep].view(torch.int16), b[keep].view(torch.int16))
                else:      # the factor of ds goes by the finite rows of all sequences: the same value up to a rounding
                    assert torch.allclose(a[keep].float(), b[keep].float(), rtol=2 ** -9, atol=2e-3)


def test_same_bits_on_another_stream_and_in_a_graph():
    import torch
    lengths = (1500, 300)
    plan = _plan(lengths)
    for kind in ("bf16", "f16"):
        dev, _ = _draw(lengths, 4, 2, 64, kind, names=("q", "k", "v", "do"))
        want = _backward(plan, dev, 0.1, 150, 4)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = _backward(plan, dev, 0.1, 150, 4)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = _backward(plan, dev, 0.1, 150, 4)
        for x in held:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, held):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_many_short_sequences():
    lengths = [1 + (i * 7) % 40 for i in range(700)]
    _case(lengths, 1, 1, 64, "bf16", 9, 1)


@pytest.mark.parametrize("count", [32, 33])
def test_sequences_around_the_number_whose_starts_come_with_the_launch(count):
    lengths = [1 + (i * 37) % 300 for i in range(count)]
    _case(lengths, 2, 1, 64, "bf16", 100, 2)


def test_the_same_bits_many_times():
    """The roles of a CTA meet at barriers only: whatever their timing, every run gives the same bits."""
    import torch
    for lengths, H, Hk, d, kind, window, sinks in (((2050,), 1, 1, 64, "f16", 1025, 1), ((900, 333, 64), 4, 2, 128, "bf16", 200, 3)):
        plan = _plan(lengths)
        dev, _ = _draw(lengths, H, Hk, d, kind, names=("q", "k", "v", "do"))
        want = _backward(plan, dev, 0.1, window, sinks)
        for _ in range(30):
            for a, b in zip(_backward(plan, dev, 0.1, window, sinks), want):
                assert torch.equal(a, b)


def test_against_differences():
    """The formula in 64 bits against central differences of the 64-bit forward, step 1e-4: error of order 1e-8 and 1e-16 / 1e-4.  (The
    kernel is compared with that formula above.)"""
    lengths, window, sinks = (40, 9), 11, 2
    rng = np.random.RandomState(0)
    w = {n: rng.randn(49, h, 8) for n, h in (("q", 4), ("k", 2), ("v", 2), ("do", 4))}
    grads = ref.window_backward(_cu(lengths), w["q"], w["k"], w["v"], 0.3, window, sinks, w["do"])
    for n, g in zip(("q", "k", "v"), grads):
        e = rng.randn(*w[n].shape)
        f = [(ref.window_forward(_cu(lengths), *(dict(w, **{n: w[n] + s * 1e-4 * e})[m] for m in ("q", "k", "v")), 0.3, window, sinks)[0] * w["do"]).sum()
             for s in (1, -1)]
        want = (f[0] - f[1]) / 2e-4
        assert abs((g * e).sum() - want) <= 1e-6 * (1 + abs(want))


def test_a_device_plan_of_another_launch_is_refused():
    import torch
    from context_kda_gb300 import binding as kda
    dev, _ = _draw((200,), 1, 1, 64, "bf16", names=("q", "k", "v", "do"))
    plan, other = _plan((200,)), _plan((90, 110))
    o, lse = _forward(plan, dev, 0.1, 50, 3)
    outs = [torch.full_like(dev["q"], 3.0) for _ in range(3)]
    ws = torch.empty(kda.kda_window_attention_workspace_bytes(plan[0], 1, 1, 64, 50, 3), dtype=torch.uint8, device="cuda")
    assert kda.kda_device_status() == kda.KDA_OK
    kda.kda_window_attention_backward(plan[0], other[1], dev["q"], dev["k"], dev["v"], 0.1, 50, 3, o, lse, dev["do"], *outs, ws)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert all(bool((x == 3).all()) for x in outs)
