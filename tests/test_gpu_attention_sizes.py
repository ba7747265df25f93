"""GPU tests of the attention layer's operators at the sizes of prompts: more tokens than one round of a kernel's warps, several batches of
heads, parts and tasks of a warp.  The head norms are compared with plain torch operations in 64 bits on the GPU (the definition of
tests/attention_reference.py, whose numpy would take minutes), the cache's fill with copies of rows, bit by bit."""
import numpy as np
import pytest

from ops_reference import check, torch_type
from test_gpu_head_rotary import EPS, _nan
from test_gpu_window_attention import _cu
from test_gpu_window_gradients import _case as _check_gradients

pytestmark = pytest.mark.gpu


def _turn(x, angle, pairs, back=False):
    """The first channels of x in 64 bits, rotated by the angles [T, pairs of channels]."""
    import torch
    r = 2 * angle.shape[1]
    if r == 0:
        return x
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None] * (-1 if back else 1)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs == "adjacent" else (x[..., :r // 2], x[..., r // 2:r])
    y = [a * c - b * s, a * s + b * c]
    y = torch.stack(y, -1).flatten(-2) if pairs == "adjacent" else torch.cat(y, -1)
    return torch.cat([y, x[..., r:]], -1)


# tokens x heads: two parts of several steps and several tasks of a warp; a warp a token with batches of steps, the last ones cut short;
# one channel fewer than 16 bytes further on; rounds of few wide heads
@pytest.mark.parametrize("kind,T,H,Hk,d,rot,pairs,offset", [
    ("bf16", 9000, 12, 4, 128, 128, "halves", 0), ("bf16", 22000, 9, 3, 128, 96, "halves", 0), ("f16", 5000, 22, 0, 128, 128, "adjacent", 0),
    ("f32", 23000, 5, 2, 256, 128, "halves", 0), ("f32", 15001, 13, 1, 64, 64, "adjacent", 0), ("bf16", 22000, 40, 8, 32, 32, "halves", 0),
    ("f16", 7001, 11, 6, 64, 48, "halves", 7), ("f32", 4000, 33, 7, 32, 0, "halves", 3), ("bf16", 16000, 3, 17, 128, 16, "adjacent", 1)])
def test_head_norms_of_prompts(kind, T, H, Hk, d, rot, pairs, offset):
    import torch
    from context_kda_gb300 import binding as kda
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    t = torch_type(kind)
    rows = lambda: torch.randn(T, (H + Hk) * d + offset, generator=gen, device="cuda").mul_(1.5).to(t)[:, offset:]
    split = lambda x: [y.unflatten(1, (-1, d)) if y.shape[1] else None for y in x.split([H * d, Hk * d], 1)]
    x, g = split(rows()), split(rows())
    w = [1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if y is not None else None for y in x]
    freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    pos = torch.randint(0, 200000, (T,), generator=gen, device="cuda").int()
    phases = torch.from_numpy(kda.kda_rotary_phases(freq)).cuda() if rot else None
    out, dx = ([None if y is None else _nan(*y.shape, dtype=t) for y in x] for _ in range(2))
    dw = [None if y is None else _nan(d, dtype=torch.float32) for y in x]
    ws = torch.empty(kda.kda_head_norm_rotary_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    kda.kda_head_norm_rotary_forward(*x, True, *w, EPS, pos, phases, pairs, *out)
    kda.kda_head_norm_rotary_backward(*x, True, *w, EPS, pos, phases, pairs, *g, *dx, *dw, ws)
    angle = pos.double()[:, None] * torch.from_numpy(freq).cuda()
    for n in range(2):
        if x[n] is None:
            continue
        v, weight = x[n].double(), w[n].double()
        size = (v.square().mean(-1, keepdim=True) + EPS).sqrt()
        hat = v / size
        check(out[n], _turn(hat * weight, angle, pairs).cpu().numpy(), kind, "qk"[n])
        e = _turn(g[n].double(), angle, pairs, back=True)
        check(dw[n], (e * hat).sum((0, 1)).cpu().numpy(), "f32", "dw")
        e = e * weight
        check(dx[n], ((e - hat * (e * hat).mean(-1, keepdim=True)) / size).cpu().numpy(), kind, "dx")


@pytest.mark.parametrize("kind,H,Hk,d", [("bf16", 2, 2, 128), ("f16", 4, 2, 64)])
def test_gradients_of_more_rows_than_one_round(kind, H, Hk, d):
    """D of all heads' rows in more than one round of the device's warps; more sequences than come with the launch."""
    _check_gradients((420,) * 100, H, Hk, d, kind, 200, 2)


def _fill(lengths, slots, Hk, d, window, sinks, pool, seed=0):
    """The arguments of a fill, and the caches as copies of rows make them."""
    import torch
    from context_kda_gb300 import binding as kda
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lengths)
    k, v = (torch.randn(T, Hk, d, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    got = [torch.full((pool, Hk, window + sinks, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = [x.clone() for x in got]
    plan = kda.kda_plan_segments(_cu(lengths), 1)
    s = torch.tensor(slots, dtype=torch.int32, device="cuda")
    for n, start in enumerate(_cu(lengths)[:-1]):
        if slots[n] < 0:
            continue
        p = torch.arange(lengths[n])
        p = p[(p < sinks) | (p >= lengths[n] - window)]
        row = torch.where(p < sinks, p, sinks + (p - sinks) % window).cuda()
        for x, y in ((k, want[0]), (v, want[1])):
            y[slots[n]][:, row] = x[start + p.cuda()].transpose(0, 1)
    return plan, kda.upload_plan(plan), s, k, v, got, want


@pytest.mark.parametrize("lengths,window,sinks", [((7000, 1, 12000), 1000, 3), ((30001,), 4096, 0), ([1 + i * 13 % 40 for i in range(700)], 9, 2)])
def test_fill_of_prompts(lengths, window, sinks):
    import torch
    from context_kda_gb300 import binding as kda
    slots = np.random.RandomState(1).permutation(len(lengths) + 1)[:len(lengths)].tolist()
    plan, plan_dev, s, k, v, got, want = _fill(lengths, slots, 3, 128, window, sinks, len(lengths) + 1)
    kda.kda_window_cache_fill(plan, plan_dev, s, k, v, window, sinks, *got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_fill_on_another_stream_and_in_a_graph():
    import torch
    from context_kda_gb300 import binding as kda
    plan, plan_dev, s, k, v, got, want = _fill((300, 40, 77), [2, -1, 0], 2, 64, 50, 4, 3)
    empty = [x.clone() for x in got]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kda.kda_window_cache_fill(plan, plan_dev, s, k, v, 50, 4, *got, side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    held = [x.clone() for x in empty]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_window_cache_fill(plan, plan_dev, s, k, v, 50, 4, *held)
    for x in held:
        x.copy_(empty[0])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_fill_refuses_a_device_plan_of_another_launch():
    import torch
    from context_kda_gb300 import binding as kda
    plan, _, s, k, v, got, _ = _fill((90, 110), [1, 0], 2, 64, 50, 4, 2)
    other = kda.upload_plan(kda.kda_plan_segments([0, 110, 200], 1))
    empty = [x.clone() for x in got]
    assert kda.kda_device_status() == kda.KDA_OK
    kda.kda_window_cache_fill(plan, other, s, k, v, 50, 4, *got)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(got, empty))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rows_whose_offsets_pass_32_bits(kind):
    """Every tensor a column range of rows 2^24 elements apart: the last ones start behind 2^31 elements."""
    import torch
    from context_kda_gb300 import binding as kda
    lengths, H, Hk, d, window, sinks = (100, 41), 4, 2, 64, 50, 3
    T = sum(lengths)
    t = torch_type(kind)
    gen = torch.Generator(device="cuda").manual_seed(0)
    wide = torch.empty(T, 2 ** 24, dtype=t, device="cuda")
    shapes = dict(q=H, k=Hk, v=Hk, o=H, do=H, dq=H, dk=Hk, dv=Hk)
    far = {n: wide[:, 4096 * i:4096 * i + h * d].unflatten(1, (h, d)) for i, (n, h) in enumerate(shapes.items())}
    near = {n: torch.randn(T, h, d, generator=gen, device="cuda").to(t) for n, h in shapes.items()}
    for n in ("q", "k", "v", "do"):
        far[n].copy_(near[n])
    plan = kda.kda_plan_segments(_cu(lengths), 1)
    plan_dev = kda.upload_plan(plan)
    ws = torch.empty(kda.kda_window_attention_workspace_bytes(plan, H, Hk, d, window, sinks), dtype=torch.uint8, device="cuda")
    for x in (near, far):
        lse = torch.empty(H, T, device="cuda")
        kda.kda_window_attention_forward(plan, plan_dev, x["q"], x["k"], x["v"], 0.125, window, sinks, x["o"], lse)
        kda.kda_window_attention_backward(plan, plan_dev, x["q"], x["k"], x["v"], 0.125, window, sinks, x["o"], lse, x["do"],
                                          x["dq"], x["dk"], x["dv"], ws)
        x["cache"] = [torch.zeros(2, Hk, window + sinks, d, dtype=t, device="cuda") for _ in range(2)]
        kda.kda_window_cache_fill(plan, plan_dev, None, x["k"], x["v"], window, sinks, *x["cache"])
    for n in ("o", "dq", "dk", "dv"):
        assert torch.equal(near[n], far[n]), n
    assert all(torch.equal(a, b) for a, b in zip(near["cache"], far["cache"]))
