"""GPU tests of what the Python calls check of their tensors."""
import pytest

pytestmark = pytest.mark.gpu


def test_tensors_of_another_device_are_refused():
    """The work goes to the current device.  Tensors of a second one without data stand in for real ones: a call that took
    them would find null pointers and refuse those, with another message."""
    import torch
    from context_kda_gb300 import binding as kda

    class Elsewhere(torch.Tensor):
        @classmethod
        def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
            raise NotImplementedError("no data")

        @staticmethod
        def __new__(cls, *shape):
            return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=torch.float32, device="cuda:1")

    assert torch.cuda.current_device() == 0
    real = torch.zeros(4, 128, device="cuda")
    other = Elsewhere(4, 128)
    heads = lambda t: t[:, None] if t is not other else Elsewhere(4, 1, 128)
    flat = torch.ones(128, device="cuda")
    plan = kda.kda_plan_segments([0, 4], 1)
    plan_dev = kda.upload_plan(plan)
    calls = [lambda t: kda.kda_gated_scan_step(None, t, None, real, real.clone(), real.clone()),
             lambda t: kda.kda_gated_scan_step(None, real, t, real, real.clone(), real.clone()),
             lambda t: kda.kda_gated_scan_step(None, real, None, real, t, real.clone()),
             lambda t: kda.kda_gated_scan_forward(plan, plan_dev, real, t, real, None, real.clone(), None, None, None),
             lambda t: kda.kda_gated_scan_backward(plan, plan_dev, real, None, real, None, real[:1].contiguous(), t, None, real.clone(), None,
                                                   real.clone(), None, None),
             lambda t: kda.kda_block_norm_forward(t, real, None, "none", 0, flat, 1.0, None, flat, 1e-6, real.clone(), real.clone()),
             lambda t: kda.kda_block_norm_backward(real, real, None, "none", 0, flat, 1.0, None, flat, 1e-6, real, real, real.clone(), t, None,
                                                   None, None, None, torch.empty(kda.kda_block_norm_workspace_bytes(128), dtype=torch.uint8,
                                                                                 device="cuda")),
             lambda t: kda.kda_decode_step(None, heads(real), heads(real), heads(real), heads(t), real[:, :1], 1.0,
                                           torch.zeros(4, 1, 128, 128, device="cuda"), heads(real).clone())]
    for n, call in enumerate(calls):
        call(real if n != 2 else real.clone())
        with pytest.raises(kda.KDAError, match="another device") as e:
            call(other)
        assert e.value.status == kda.KDA_ERR_INVALID_ARG, n
    torch.cuda.synchronize()
    assert kda.kda_device_status() == kda.KDA_OK
