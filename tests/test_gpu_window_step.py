"""GPU tests of the window attention's single-token step and of its cache against their 64-bit definitions
(tests/attention_reference.py); tolerances of test_gpu_window_attention.py (probabilities are rounded to the type there too)."""
import numpy as np
import pytest

import attention_reference as ref
from ops_reference import ROUND, TOL32, torch_type
from test_gpu_window_attention import _cu, _within

pytestmark = pytest.mark.gpu


def _draw(B, H, Hk, d, kind, window, sinks, pool, seed=0):
    import torch
    gen = torch.Generator().manual_seed(seed + B * 100 + window)
    t = torch_type(kind)
    host = {n: torch.randn(B, h, d, generator=gen).to(t) for n, h in (("q", H), ("k", Hk), ("v", Hk))}
    for n in ("cache_k", "cache_v"):
        host[n] = torch.randn(pool, Hk, window + sinks, d, generator=gen).to(t)
    return {n: x.cuda() for n, x in host.items()}, {n: x.double().numpy() for n, x in host.items()}


def _step(dev, slots, lengths, scale, window, sinks, stream=None):
    import torch
    from context_kda_gb300 import binding as kda
    o = torch.full(dev["q"].shape, float("nan"), dtype=dev["q"].dtype, device="cuda")
    s = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    kda.kda_window_attention_step(s, torch.tensor(lengths, dtype=torch.int32, device="cuda"), dev["q"], dev["k"], dev["v"], scale, window, sinks,
                                  dev["cache_k"], dev["cache_v"], o, stream)
    return o


def _check(o, dev, w, slots, lengths, scale, window, sinks, kind):
    o_ref, size, ck, cv = ref.window_step(slots, lengths, w["q"], w["k"], w["v"], scale, window, sinks, w["cache_k"], w["cache_v"])
    tiny = 2.0 ** -25 * (1 + window + sinks) * np.abs(w["v"]).max() if kind == "f16" else 0.0
    _within(o, o_ref, ROUND[kind] * 1.001 * (size + np.abs(o_ref)) + TOL32 * (size + 1e-3) + tiny, "o")
    for n, want in (("cache_k", ck), ("cache_v", cv)):
        assert np.array_equal(dev[n].double().cpu().numpy(), want), n


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hk", [(1, 1, 1), (2, 4, 1), (3, 8, 2), (2, 9, 1), (2, 12, 4), (1, 20, 1), (2, 34, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 1), (64, 4), (300, 0), (1100, 7)])
def test_step(window, sinks, B, H, Hk, d, kind):
    rng = np.random.RandomState(B * 7 + window)
    dev, w = _draw(B, H, Hk, d, kind, window, sinks, B + 1)
    slots = list(rng.permutation(B + 1)[:B])
    for lengths in (rng.randint(0, 2 * (window + sinks) + 1, B), [0] * B, [window + sinks - 1] * B, [window + sinks] * B):
        lengths = [int(x) for x in lengths]
        d2 = {n: x.clone() for n, x in dev.items()}
        o = _step(d2, slots, lengths, d ** -0.5, window, sinks)
        _check(o, d2, w, slots, lengths, d ** -0.5, window, sinks, kind)


@pytest.mark.parametrize("length", [15, 16, 17, 31, 63, 64, 127, 128, 129, 511, 512, 999])
def test_every_length_of_a_split_cache(length):
    dev, w = _draw(1, 4, 2, 128, "bf16", 1000, 3, 1)
    o = _step(dev, None, [length], 0.09, 1000, 3)
    _check(o, dev, w, [0], [length], 0.09, 1000, 3, "bf16")


def test_rows_without_a_token_are_not_read():
    import torch
    dev, w = _draw(2, 4, 2, 64, "bf16", 700, 2, 2)
    lengths = [40, 333]
    for s, n in enumerate(lengths):
        for c in ("cache_k", "cache_v"):
            dev[c][s, :, n:] = float("nan")
    o = _step(dev, None, lengths, 0.125, 700, 2)
    o_ref, size, _, _ = ref.window_step([0, 1], lengths, w["q"], w["k"], w["v"], 0.125, 700, 2, w["cache_k"], w["cache_v"])
    _within(o, o_ref, ROUND["bf16"] * 1.001 * (size + np.abs(o_ref)) + TOL32 * (size + 1e-3), "o")
    assert bool(torch.isnan(dev["cache_k"][0, :, 41:]).all()) and bool(torch.isfinite(dev["cache_k"][0, :, :41]).all())


def test_padding_and_bad_rows():
    import torch
    from context_kda_gb300 import binding as kda
    dev, w = _draw(6, 4, 2, 64, "bf16", 200, 2, 5)
    before = {n: dev[n].clone() for n in ("cache_k", "cache_v")}
    o = _step(dev, [3, -1, 0, -7, 4, 2], [10, 0, 500, 3, 0, 201], 0.125, 200, 2)
    _check(o, dev, w, [3, -1, 0, -7, 4, 2], [10, 0, 500, 3, 0, 201], 0.125, 200, 2, "bf16")
    assert bool((o[[1, 3]] == 0).all())
    assert torch.equal(before["cache_k"][1], dev["cache_k"][1])
    assert kda.kda_device_status() == kda.KDA_OK
    dev, w = _draw(4, 4, 2, 64, "bf16", 900, 2, 4)
    o = _step(dev, [3, 4, 0, 1], [10, 9, -1, 1000], 0.125, 900, 2)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert kda.kda_device_status() == kda.KDA_OK
    _check(o, dev, w, [3, 4, 0, 1], [10, 9, -1, 1000], 0.125, 900, 2, "bf16")


def test_bad_values_stay_in_their_row():
    import torch
    a, _ = _draw(4, 8, 2, 64, "bf16", 300, 2, 4)
    b, _ = _draw(4, 8, 2, 64, "bf16", 300, 2, 4)
    oa = _step(a, None, [400, 20, 350, 300], 0.125, 300, 2)
    b["cache_v"][1, 0, 5], b["cache_k"][2, 1, 7] = float("nan"), float("inf")
    ob = _step(b, None, [400, 20, 350, 300], 0.125, 300, 2)
    same = (oa.view(torch.int16) == ob.view(torch.int16)).all(-1).cpu().numpy()
    want = np.ones((4, 8), dtype=bool)
    want[1, :4] = want[2, 4:] = False
    assert np.array_equal(same, want)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (50, 3), (130, 0), (400, 128)])
def test_fill(window, sinks, kind):
    import torch
    from context_kda_gb300 import binding as kda
    lengths, slots, Hk, d = (1, 300, 77, 131, 2), [4, 0, -1, 2, 3], 3, 64
    dev, w = _draw(1, Hk, Hk, d, kind, window, sinks, 6)
    gen = torch.Generator().manual_seed(1)
    rows = torch.randn(sum(lengths), 2 * Hk * d + 8, generator=gen).to(torch_type(kind))
    k, v = (rows[:, i * Hk * d:(i + 1) * Hk * d].unflatten(1, (Hk, d)) for i in range(2))
    plan = kda.kda_plan_segments(_cu(lengths), 2)
    on = rows.cuda()
    kd, vd = (on[:, i * Hk * d:(i + 1) * Hk * d].unflatten(1, (Hk, d)) for i in range(2))
    kda.kda_window_cache_fill(plan, kda.upload_plan(plan), torch.tensor(slots, dtype=torch.int32, device="cuda"), kd, vd, window, sinks,
                              dev["cache_k"], dev["cache_v"])
    ck, cv = ref.cache_fill(_cu(lengths), slots, k.double().numpy(), v.double().numpy(), window, sinks, w["cache_k"], w["cache_v"])
    assert np.array_equal(dev["cache_k"].double().cpu().numpy(), ck) and np.array_equal(dev["cache_v"].double().cpu().numpy(), cv)
    assert kda.kda_device_status() == kda.KDA_OK
    kda.kda_window_cache_fill(plan, kda.upload_plan(plan), torch.tensor([0, 1, 2, 6, 3], dtype=torch.int32, device="cuda"), kd, vd, window, sinks,
                              dev["cache_k"], dev["cache_v"])
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("window,sinks", [(60, 4), (300, 0), (7, 1)])
def test_steps_continue_a_prefill(window, sinks):
    """A prefill of some tokens, its cache, and steps for the rest give the rows of a longer prefill: both round the probabilities and the
    output once, at different places, so they differ by twice the sum of the tolerances' two parts at most."""
    import torch
    from context_kda_gb300 import binding as kda
    H, Hk, d, new, prompts = 4, 2, 64, 40, (1, 100, 260)
    gen = torch.Generator().manual_seed(5)
    T = sum(prompts) + new * len(prompts)
    q, k, v = (torch.randn(T, h, d, generator=gen).to(torch.bfloat16).cuda() for h in (H, Hk, Hk))
    full = _cu([n + new for n in prompts])
    plan = kda.kda_plan_segments(full, 1)
    want, size = torch.empty_like(q), torch.empty_like(q)
    kda.kda_window_attention_forward(plan, kda.upload_plan(plan), q, k, v, 0.125, window, sinks, want, None)
    kda.kda_window_attention_forward(plan, kda.upload_plan(plan), q, k, v.abs(), 0.125, window, sinks, size, None)
    at = torch.cat([torch.arange(full[n], full[n] + p) for n, p in enumerate(prompts)]).cuda()
    plan = kda.kda_plan_segments(_cu(prompts), 1)
    caches = [torch.full((3, Hk, window + sinks, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    kda.kda_window_cache_fill(plan, kda.upload_plan(plan), slots, k[at], v[at], window, sinks, *caches)
    for t in range(new):
        rows = torch.tensor([full[n] + p + t for n, p in enumerate(prompts)], device="cuda")
        lengths = torch.tensor([p + t for p in prompts], dtype=torch.int32, device="cuda")
        o = torch.empty(3, H, d, dtype=torch.bfloat16, device="cuda")
        kda.kda_window_attention_step(slots, lengths, q[rows], k[rows], v[rows], 0.125, window, sinks, *caches, o)
        bound = 2 * (ROUND["bf16"] * 1.01 * (size[rows].double() + want[rows].double().abs()) + TOL32 * (size[rows].double() + 1e-3))
        assert bool(((o.double() - want[rows].double()).abs() <= bound).all()), t


def test_another_stream_a_graph_and_the_same_bits():
    import torch
    dev, _ = _draw(3, 8, 2, 128, "bf16", 800, 4, 3)
    lengths = [900, 100, 5000]
    want = _step(dev, None, lengths, 0.09, 800, 4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _step(dev, None, lengths, 0.09, 800, 4)
    side.synchronize()
    from context_kda_gb300 import binding as kda
    n, o = torch.tensor(lengths, dtype=torch.int32, device="cuda"), torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_window_attention_step(None, n, dev["q"], dev["k"], dev["v"], 0.09, 800, 4, dev["cache_k"], dev["cache_v"], o)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got) and torch.equal(want, o)


def test_cache_offsets_beyond_32_bits():
    """A pool whose last slot starts behind 2^31 elements."""
    import torch
    window, sinks, pool = 4092, 4, 4101
    dev, w = _draw(2, 2, 1, 128, "bf16", window, sinks, 1)
    big = {n: torch.zeros(pool, 1, window + sinks, 128, dtype=torch.bfloat16, device="cuda") for n in ("cache_k", "cache_v")}
    for n in big:
        big[n][pool - 1] = dev[n][0]
    got = _step(dict(dev, **big), [pool - 1, -1], [5000, 0], 0.09, window, sinks)
    want = _step(dev, [0, -1], [5000, 0], 0.09, window, sinks)
    assert torch.equal(got, want) and torch.equal(big["cache_v"][pool - 1], dev["cache_v"][0])


def test_no_tokens():
    import torch
    from context_kda_gb300 import binding as kda
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")
    kda.kda_window_attention_step(None, e(0, t=torch.int32), e(0, 4, 64), e(0, 2, 64), e(0, 2, 64), 0.1, 10, 0, e(3, 2, 10, 64), e(3, 2, 10, 64), e(0, 4, 64))
