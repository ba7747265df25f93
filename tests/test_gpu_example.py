"""The example decoder: decoding continues a prefill, training lowers the loss, and the operators' gradients
under autograd are those of the same layer in plain torch."""
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


def test_decoding_continues_a_prefill(example):
    """Outputs of unit size in bf16 after four layers: every layer rounds its activations a few times (2^-8 each),
    and the two paths round at different places; 16 roundings of independent sign and values up to 4 give
    4 * sqrt(16) * 2^-8 = 0.06."""
    assert example.decode_error() <= 0.06


def test_training_lowers_the_loss(example):
    losses = example.train()
    assert all(v == v for v in losses)
    assert losses[-1] < 0.5 * losses[0]


def test_gradients_under_autograd(example):
    """Central differences of the layer's loss in fp32 along random directions.  The difference of step 1e-2 has an error
    of order (1e-2)^2 and the fp32 losses round by 1e-7 of their size over 2e-2: one part in a hundred covers both."""
    import torch
    from context_kda_gb300 import binding as kda
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, D = 300, 64
    plan = kda.kda_plan_segments([0, 130, 300], 1)
    plan_dev, ws = kda.upload_plan(plan), torch.empty(16, dtype=torch.uint8, device="cuda")
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    leaves = {"x": normal(T, D), "i": torch.rand(T, D, generator=gen, device="cuda"), "g": -0.3 * torch.rand(T, D, generator=gen, device="cuda"),
              "r": normal(T, D), "z": normal(T, D), "w_post": 1 + 0.1 * normal(D), "ls": 1 + 0.1 * normal(D), "w_pre": 1 + 0.1 * normal(D)}
    c1, c2 = normal(T, D), normal(T, D)

    def loss(v):
        h = example.GatedScan.apply(plan, plan_dev, ws, v["x"], v["i"], v["g"])
        r, y = example.BlockNorm.apply("sigmoid", 32, 0.5, v["r"], h, v["z"], v["w_post"][:32].contiguous(), v["ls"], v["w_pre"])
        return (r.double() * c1).sum() + (y.double() * c2).sum()

    v = {k: a.clone().requires_grad_() for k, a in leaves.items()}
    loss(v).backward()
    for name, a in leaves.items():
        d = normal(*a.shape)
        eps = 1e-2
        with torch.no_grad():
            up, down = (loss({**leaves, name: a + s * eps * d}) for s in (1, -1))
        got, want = float((v[name].grad.double() * d).sum()), float((up - down) / (2 * eps))
        size = float((v[name].grad.double() * d).square().sum().sqrt())     # of a sum of terms of random sign
        assert abs(got - want) <= 1e-2 * max(abs(want), size), (name, got, want)


@pytest.mark.parametrize("absent", [("z",), ("r",), ("w_post",), ("ls",), ("w_pre",), ("r", "w_pre"), ("z", "r", "ls", "w_pre")], ids="-".join)
def test_block_norm_under_autograd_without_parts(example, absent):
    """Any part but o may be None: gradients against autograd through the definition in 64 bits, within the tolerances of the
    operators' own tests."""
    import torch
    import ops_reference as ref
    gen = torch.Generator(device="cuda").manual_seed(9)
    T, D, G = 37, 128, 32
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    parts = {"r": normal(T, D), "o": normal(T, D), "z": normal(T, D), "w_post": 1 + 0.1 * normal(G), "ls": 1 + 0.1 * normal(D), "w_pre": 1 + 0.1 * normal(D)}
    parts = {k: None if k in absent else v for k, v in parts.items()}
    gate = "none" if "z" in absent else "silu"
    c1, c2 = normal(T, D), normal(T, D)
    own = {k: None if v is None else v.clone().requires_grad_() for k, v in parts.items()}
    wide = {k: None if v is None else v.double().requires_grad_() for k, v in parts.items()}
    r, y = example.BlockNorm.apply(gate, G, 0.5, *own.values())
    assert (y is None) == ("w_pre" in absent)
    ((r * c1).sum() + (0 if y is None else (y * c2).sum())).backward()
    unit = lambda v, n: v * torch.rsqrt(v.unflatten(1, (-1, n)).square().mean(-1, keepdim=True) + example.EPS).expand(-1, -1, n).reshape(T, D)
    u = wide["o"] if wide["w_post"] is None else unit(wide["o"], G) * wide["w_post"].repeat(D // G)
    u = u if wide["z"] is None else u * torch.nn.functional.silu(wide["z"])
    r2 = (0 if wide["r"] is None else wide["r"]) + 0.5 * u * (1 if wide["ls"] is None else wide["ls"])
    loss = (r2 * c1.double()).sum()
    if wide["w_pre"] is not None:
        loss = loss + (unit(r2, D) * wide["w_pre"] * c2.double()).sum()
    loss.backward()
    for name, v in own.items():
        if v is not None:
            ref.check(v.grad, wide[name].grad.cpu().numpy(), "f32", name)
