"""GPU tests of the KDA single-token step against its 64-bit definition (tests/ops_reference.py, whose
tolerances apply) and against the chunked forward it continues."""
import numpy as np
import pytest

import ops_reference as ref
from ops_reference import check, torch_type

pytestmark = pytest.mark.gpu

K = 128


def _draw(B, H, kind, pool=None, seed=0, fused=False):
    import torch
    gen = torch.Generator().manual_seed(seed + 100 * B + H)
    t = torch_type(kind)
    unit = lambda v: v / v.norm(dim=-1, keepdim=True)
    normal = lambda *s: torch.randn(*s, generator=gen)
    q, k, v = unit(normal(B, H, K)).to(t), unit(normal(B, H, K)).to(t), normal(B, H, K).to(t)
    g, beta = -0.2 * torch.rand(B, H, K, generator=gen), torch.rand(B, H, generator=gen)
    pool = B if pool is None else pool
    state = 0.3 * normal(pool, H, K, K)
    host = dict(q=q, k=k, v=v, g=g, beta=beta, state=state)
    dev = {n: x.cuda() for n, x in host.items()}
    if fused:      # q, k, v as column ranges of one projection, at an odd offset
        wide = torch.zeros(B, 3 * H * K + 5, dtype=t)
        for j, n in enumerate("qkv"):
            wide[:, 1 + j * H * K:1 + (j + 1) * H * K] = host[n].reshape(B, -1)
        wide = wide.cuda()
        for j, n in enumerate("qkv"):
            dev[n] = wide[:, 1 + j * H * K:1 + (j + 1) * H * K].unflatten(1, (H, K))
    return dev, {n: x.double().numpy() for n, x in host.items()}


def _step(dev, slots, scale=K ** -0.5):
    import torch
    from context_kda_gb300 import binding as kda
    o = torch.full(dev["v"].shape, float("nan"), dtype=dev["v"].dtype, device="cuda")
    s = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    kda.kda_decode_step(s, dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], scale, dev["state"], o)
    return o


def _want(w, slots, scale=K ** -0.5):
    return ref.decode(w["state"], slots, w["q"], w["k"], w["v"], w["g"], w["beta"], scale)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 16), (2, 3), (7, 4), (33, 2), (40, 16), (150, 5)])
def test_step(B, H, kind):
    dev, w = _draw(B, H, kind)
    o = _step(dev, None)
    o_ref, s_ref = _want(w, list(range(B)))
    check(o, o_ref, kind, "o")
    check(dev["state"], s_ref, "f32", "state")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_slots_and_padding(kind):
    import torch
    dev, w = _draw(9, 3, kind, pool=12)
    slots = [11, -1, 0, 5, 7, -1, 2, 3, 9]
    before = dev["state"].clone()
    o = _step(dev, slots)
    o_ref, s_ref = _want(w, slots)
    check(o, o_ref, kind, "o")
    check(dev["state"], s_ref, "f32", "state")
    for s in (1, 4, 6, 8, 10):
        assert torch.equal(before[s], dev["state"][s])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_fused_projection_rows(kind):
    dev, w = _draw(6, 3, kind, fused=True)
    o = _step(dev, None)
    o_ref, s_ref = _want(w, list(range(6)))
    check(o, o_ref, kind, "o")
    check(dev["state"], s_ref, "f32", "state")


def test_bad_values_stay_in_their_row():
    import torch
    a, _ = _draw(6, 3, "bf16")
    b, _ = _draw(6, 3, "bf16")
    oa = _step(a, None)
    b["v"][2], b["state"][4] = float("nan"), float("inf")
    ob = _step(b, None)
    for n in (0, 1, 3, 5):
        assert torch.equal(oa[n].view(torch.int16), ob[n].view(torch.int16))
        assert torch.equal(a["state"][n].view(torch.int32), b["state"][n].view(torch.int32))


def test_decay_of_minus_infinity_and_zero_beta():
    dev, w = _draw(3, 2, "f32")
    dev["g"][0], w["g"][0] = float("-inf"), -np.inf
    dev["beta"][1], w["beta"][1] = 0.0, 0.0
    o = _step(dev, None)
    o_ref, s_ref = _want(w, [0, 1, 2])
    check(o, o_ref, "f32", "o")
    check(dev["state"], s_ref, "f32", "state")


def test_a_slot_out_of_range_is_recorded():
    import torch
    from context_kda_gb300 import binding as kda
    assert kda.kda_device_status() == kda.KDA_OK
    dev, w = _draw(3, 2, "bf16")
    o = _step(dev, [0, 3, 2])
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert kda.kda_device_status() == kda.KDA_OK
    o_ref, s_ref = _want(w, [0, -1, 2])
    check(o, o_ref, "bf16", "o")
    check(dev["state"], s_ref, "f32", "state")


def test_decoding_continues_the_chunked_forward():
    """Prefill of n tokens and m steps give the outputs and states of the chunked forward over n + m, within
    that forward's own bars (2e-2 on outputs, 1e-4 relative on states)."""
    import torch
    from context_kda_gb300 import binding as kda
    from context_kda_gb300.inputs import make_inputs
    from harness import O_TOL, REL_TOL, gpu_forward, oracle_forward, rel_err, to_device
    n, m, H = 200, 9, 3
    inp = make_inputs([n + m], heads=H, segments=1, h0_std=0.1, seed=12)
    d = to_device(inp)
    o_ref, f_ref = oracle_forward(inp)
    plan = kda.kda_plan_segments([0, n], 2)
    plan_dev = kda.upload_plan(plan)
    ws = torch.empty(kda.kda_workspace_bytes(plan, H), dtype=torch.uint8, device="cuda")
    o = torch.empty(n, H, K, dtype=torch.bfloat16, device="cuda")
    state = torch.empty(1, H, K, K, device="cuda")
    kda.kda_forward_segmented(plan, plan_dev, H, *(d[x][:n].contiguous() for x in ("q", "k", "v", "g", "beta")), d["h0"], 1.0, o,
                              state, ws)
    for t in range(n, n + m):
        row = {x: d[x][t:t + 1] for x in ("q", "k", "v", "g", "beta")}
        out = torch.empty(1, H, K, dtype=torch.bfloat16, device="cuda")
        kda.kda_decode_step(None, row["q"], row["k"], row["v"], row["g"], row["beta"], 1.0, state, out)
        assert float(np.max(np.abs(out[0].float().cpu().numpy() - o_ref[t]))) <= O_TOL
    assert rel_err(state.cpu().numpy(), f_ref) <= REL_TOL


def test_another_stream():
    import torch
    dev, w = _draw(5, 4, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o = _step(dev, None)
    side.synchronize()
    check(o, _want(w, list(range(5)))[0], "bf16", "o")


def test_state_offsets_beyond_32_bits():
    """A pool of 2^17 + 5 slots of one head: element offsets pass 2^31."""
    import torch
    from context_kda_gb300 import binding as kda
    pool = 2 ** 17 + 5
    dev, w = _draw(3, 1, "bf16")
    state = torch.zeros(pool, 1, K, K, device="cuda")
    slots = [pool - 1, 0, 2 ** 17]
    state[slots] = dev["state"]
    small = dict(dev, state=state)
    o = _step(small, slots)
    o_ref, s_ref = _want(w, [0, 1, 2])
    check(o, o_ref, "bf16", "o")
    check(state[slots], s_ref, "f32", "state")
