"""GPU tests of the window attention's gradients where ds is small beside what it is made from; tolerances of
test_gpu_window_gradients.py."""
import numpy as np
import pytest

import attention_reference as ref
from ops_reference import ROUND, TOL32
from test_gpu_window_attention import BIG, _cu, _draw, _plan, _within
from test_gpu_window_gradients import _backward

pytestmark = pytest.mark.gpu


def test_fp16_keeps_the_bits_of_ds_from_2_to_the_minus_27_of_its_bound():
    """One sequence's rows of do and v make the longest |do| |v|, 2^15, a power of two, which leaves ds the least room; the others are pairs
    of tokens with p = 1/2 each, whose ds = do (v_0 - v_1) / 4 are 1 to 2 times 2^-27 of that, and dq = 2 ds: rounded twice."""
    import torch
    n, d = 500, 64
    gen = torch.Generator().manual_seed(0)
    host = {m: torch.zeros(2 * n + 2, 1, d, dtype=torch.float16) for m in ("q", "k", "v", "do")}
    host["do"][:2], host["v"][:2] = 512.0, 1.0
    x = 1 + torch.rand(n, generator=gen)
    host["do"][3::2, 0, 0] = (2.0 ** -12 * x).half()
    host["v"][2::2, 0, 0], host["v"][3::2, 0, 0] = (2 + 0.1 * x).half(), -2.0
    host["k"][2::2, 0, 1], host["k"][3::2, 0, 1] = 1.0, -1.0
    w = {m: t.double().numpy() for m, t in host.items()}
    lengths = [2] * (n + 1)
    dq, _, _ = _backward(_plan(lengths), {m: t.cuda() for m, t in host.items()}, 1.0, BIG, 0)
    ds = w["do"][3::2, 0, 0] * (w["v"][2::2, 0, 0] - w["v"][3::2, 0, 0]) / 4
    assert np.all(ds >= 2.0 ** -12)
    got, want = dq.double().cpu().numpy()[3::2, 0, 1], 2 * ds
    assert np.all(np.abs(got - want) <= (2 * ROUND["f16"] * 1.001 + TOL32) * want)
    full = ref.window_backward(_cu(lengths), w["q"], w["k"], w["v"], 1.0, BIG, 0, w["do"])[0]
    assert np.allclose(full[3::2, 0, 1], want, rtol=1e-12)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("window,sinks", [(BIG, 0), (200, 3), (20, 1)])
@pytest.mark.parametrize("gain", [4.0, 12.0])
def test_rows_that_put_their_weight_on_few_keys(gain, window, sinks, kind):
    """Scores four and twelve times as wide: of most rows a key or two have all the weight, ds is next to nothing, and D's rounding is what its
    bar goes by ('loose' in the reference).  The scores' own error grows with them, 2^-24 of the sum of 64 products' sizes: p and ds move by
    that much relatively."""
    import torch
    lengths, d, scale = (700, 150), 64, 0.125
    dev, w = _draw(lengths, 4, 2, d, kind, names=("q", "k", "v", "do"))
    dev["q"] = dev["q"] * gain
    w["q"] = dev["q"].double().cpu().numpy()
    outs = _backward(_plan(lengths), dev, scale, window, sinks)
    want = ref.window_backward(_cu(lengths), w["q"], w["k"], w["v"], scale, window, sinks, w["do"])
    moved = TOL32 + 2.0 ** -24 * 4 * scale * np.abs(w["q"]).max() * np.abs(w["k"]).max() * d
    for n, got, x, size in zip(("dq", "dk", "dv"), outs, want[:3], want[3:]):
        tiny = 2.0 ** -25 * max(1.0, np.abs(x).max()) if kind == "f16" else 0.0
        _within(got, x, ROUND[kind] * 1.001 * (size + np.abs(x)) + moved * (size + 1e-2 * np.abs(x).max() + 1e-3) + tiny, n)
