"""The example decoder with attention layers: prefill, caches and steps together, and the attention layer under autograd against
differences."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_decoder", os.path.join(ROOT, "examples", "hybrid_decoder.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kinds", [("window",), ("kda", "window", "scan", "window")])
def test_decoding_continues_a_prefill(example, kinds):
    """Outputs of unit size in bf16 after four layers: every layer rounds its activations (and probabilities) a few times, 2^-8
    each, and the two paths round at different places; 16 roundings of independent sign and values up to 4 give
    4 * sqrt(16) * 2^-8 = 0.06.  (The prompts are longer than the window of 40, as long as one token, and pass it while decoding.)"""
    assert example.decode_error(lengths=(200, 1, 37), new=12, kinds=kinds) <= 0.06


def test_the_layer_runs_in_a_captured_step(example):
    """A decoding step captured once and replayed with other lengths, slots and rows gives what eager steps give."""
    import torch
    kinds = ("window", "scan", "kda")
    model = example.Decoder(seed=3, kinds=kinds, layers=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows = torch.randn(60, 3, model.width, generator=gen, device="cuda")
    states = [model.new_states(4) for _ in range(2)]
    for pool in states:
        for s in pool:
            for x in s if isinstance(s, tuple) else (s,):
                x.zero_()
    slots = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    want = [model.step(rows[t], states[0], slots, torch.full((3,), t, dtype=torch.int32, device="cuda")) for t in range(60)]
    row, had = rows[0].clone(), torch.zeros(3, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    spare = model.new_states(4)
    with torch.cuda.stream(side):
        model.step(row, spare, slots, had)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = model.step(row, states[1], slots, had)
    for t in range(60):
        row.copy_(rows[t])
        had.fill_(t)
        graph.replay()
        assert torch.equal(y, want[t]), t


def test_gradients_under_autograd(example):
    """The attention layer's loss in 64 bits through plain torch, and the gradients of the library's chain: each of the two
    operators rounds its outputs, probabilities and ds to bf16, 2^-8 each, so the norm of the difference is within a few times 2^-8 /
    sqrt(3) of the gradient's: 2e-2 covers eight of them."""
    import torch
    from context_kda_gb300 import binding as kda
    gen = torch.Generator(device="cuda").manual_seed(5)
    lengths, H, Hk, d, window, sinks = (150, 90), 4, 2, 64, 60, 2
    T, cu = sum(lengths), [0, 150, 240]
    plan = kda.kda_plan_segments(cu, 1)
    plan_dev = kda.upload_plan(plan)
    positions = torch.cat([torch.arange(n) for n in lengths]).cuda()
    freq = 10000.0 ** (-torch.arange(0, d, 2).double() / d)
    phases = torch.from_numpy(kda.kda_rotary_phases(freq)).cuda()
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    rows = normal(T, (H + 2 * Hk) * d).to(torch.bfloat16)
    w = {"w_q": 1 + 0.1 * normal(d), "w_k": 1 + 0.1 * normal(d)}
    c = normal(T, H, d)

    def split(x):
        return (y.unflatten(1, (-1, d)) for y in x.split([H * d, Hk * d, Hk * d], dim=1))

    own = {"rows": rows.clone().requires_grad_(), **{n: x.clone().requires_grad_() for n, x in w.items()}}
    q, k, v = split(own["rows"])
    q, k = example.HeadNormRotary.apply(positions.int(), phases, "halves", q, k, own["w_q"], own["w_k"])
    o = example.WindowAttention.apply(plan, plan_dev, d ** -0.5, window, sinks, q, k, v)
    (o.double() * c).sum().backward()

    wide = {"rows": rows.double().requires_grad_(), **{n: x.double().requires_grad_() for n, x in w.items()}}
    q, k, v = split(wide["rows"])
    a = positions.double()[:, None] * freq.cuda()
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]

    def turned(x, weight):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + example.EPS) * weight
        x, y = x.chunk(2, -1)
        return torch.cat([x * cos - y * sin, x * sin + y * cos], -1)

    q, k = turned(q, wide["w_q"]), turned(k, wide["w_k"])
    i, j = torch.arange(T, device="cuda")[:, None], torch.arange(T, device="cuda")[None]
    start = torch.where(i >= 150, 150, 0)
    seen = (j <= i) & (j >= start) & ((i - j < window) | (j - start < sinks))
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(H // Hk, 1)) * d ** -0.5
    p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
    (torch.einsum("hij,jhd->ihd", p, v.repeat_interleave(H // Hk, 1)) * c.double()).sum().backward()
    for n in own:
        got, want = own[n].grad.double(), wide[n].grad
        assert float((got - want).norm()) <= 2e-2 * float(want.norm()), n


def test_a_graph_of_the_backward_beside_an_eager_one(example):
    """A backward pass captured into a graph while an eager graph of the same leaves lives.  (Both on one stream other than the
    default one: autograd remembers the stream of a leaf's first use and orders later ones behind it, which a capture may not do
    with the default stream, whatever the operators.)"""
    import torch
    from context_kda_gb300 import binding as kda
    gen = torch.Generator(device="cuda").manual_seed(6)
    plan = kda.kda_plan_segments([0, 200, 333], 1)
    plan_dev = kda.upload_plan(plan)
    data = [torch.randn(333, h, 64, generator=gen, device="cuda").to(torch.bfloat16) for h in (4, 2, 2)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        leaves = [x.clone().requires_grad_() for x in data]
        run = lambda: example.WindowAttention.apply(plan, plan_dev, 0.125, 70, 1, *leaves)
        eager = run()
        want = torch.autograd.grad(eager.float().square().sum(), leaves, retain_graph=True)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = torch.autograd.grad(run().float().square().sum(), leaves)
    with torch.cuda.stream(side):
        graph.replay()
        again = torch.autograd.grad(eager.float().square().sum(), leaves)
    torch.cuda.synchronize()
    for a, b, c in zip(want, held, again):
        assert torch.equal(a, b) and torch.equal(a, c)
