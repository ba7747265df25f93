"""GPU tests: a device plan of another launch, with more sequences than come with the launch."""
import pytest

from test_gpu_window_attention import _draw, _forward, _plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_nothing_is_written(kind):
    import torch
    from context_kda_gb300 import binding as kda
    lengths, window, sinks = [5 + i % 7 for i in range(50)], 4, 2
    dev, _ = _draw(lengths, 2, 1, 64, kind, names=("q", "k", "v", "do"))
    plan, other = _plan(lengths), _plan(lengths[::-1])
    want, lse = _forward(plan, dev, 0.1, window, sinks)
    o = torch.full_like(want, 3.0)
    assert kda.kda_device_status() == kda.KDA_OK
    kda.kda_window_attention_forward(plan[0], other[1], dev["q"], dev["k"], dev["v"], 0.1, window, sinks, o, None)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert bool((o == 3).all())
    outs = [torch.full_like(dev[n], 3.0) for n in ("q", "k", "v")]
    ws = torch.empty(kda.kda_window_attention_workspace_bytes(plan[0], 2, 1, 64, window, sinks), dtype=torch.uint8, device="cuda")
    kda.kda_window_attention_backward(plan[0], other[1], dev["q"], dev["k"], dev["v"], 0.1, window, sinks, want, lse, dev["do"], *outs, ws)
    ws.fill_(7)      # the workspace is the caller's again behind the call
    torch.cuda.synchronize()
    assert bool((ws == 7).all())
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert all(bool((x == 3).all()) for x in outs)
