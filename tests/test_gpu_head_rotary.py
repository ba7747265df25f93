"""GPU tests of the head norms with rotation against their 64-bit definitions (tests/attention_reference.py); tolerances of
ops_reference: everything in fp32, rounded once.  The angle is exact to 2^-32 of a turn, 1.5e-9, and sincospi to an ulp: they are
within the fp32 part of the bar (2e-5) at any position."""
import numpy as np
import pytest

import attention_reference as ref
from ops_reference import check, torch_type

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _draw(T, H, Hk, d, kind, weight=True, offset=None, seed=0):
    """q, k and their output gradients; offset: all of them at that column of wider rows."""
    import torch
    gen = torch.Generator().manual_seed(seed + 1000 * T + 10 * H + d)
    t = torch_type(kind)
    host = {n: (1.5 * torch.randn(T, h, d, generator=gen)).to(t) for n, h in (("q", H), ("k", Hk), ("gq", H), ("gk", Hk))}
    host["w_q"], host["w_k"] = (1 + 0.2 * torch.randn(d, generator=gen), 1 + 0.2 * torch.randn(d, generator=gen)) if weight else (None, None)
    dev = {n: None if x is None else x.cuda() for n, x in host.items()}
    if offset is not None:
        for n in ("q", "k", "gq", "gk"):
            h = host[n].shape[1]
            wide = torch.full((T, h * d + offset + 3), float("nan"), dtype=t)
            wide[:, offset:offset + h * d] = host[n].reshape(T, -1)
            dev[n] = wide.cuda()[:, offset:offset + h * d].unflatten(1, (h, d))
    return dev, {n: None if x is None else x.double().numpy() for n, x in host.items()}


def _rotation(T, rot, far=0, seed=0):
    import torch
    from context_kda_gb300 import binding as kda
    freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    pos = np.random.RandomState(seed + T).randint(0, 5000, T) + far
    if rot == 0:
        return np.zeros(T), freq, None, None
    return pos, freq, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.from_numpy(kda.kda_rotary_phases(freq)).cuda()


def _nan(*shape, dtype):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _both(T, H, Hk, d, rot, pairs, kind, norm=True, weight=True, far=0, offset=None):
    import torch
    from context_kda_gb300 import binding as kda
    dev, w = _draw(T, H, Hk, d, kind, weight and norm, offset)
    pos, freq, pos_dev, phases = _rotation(T, rot, far)
    t = torch_type(kind)
    has_k = Hk > 0
    qo, ko = _nan(T, H, d, dtype=t), _nan(T, Hk, d, dtype=t) if has_k else None
    k = dev["k"] if has_k else None
    kda.kda_head_norm_rotary_forward(dev["q"], k, norm, dev["w_q"], dev["w_k"] if has_k else None, EPS, pos_dev, phases, pairs, qo, ko)
    check(qo, ref.head_forward(w["q"], norm, w["w_q"], EPS, pos, freq, pairs), kind, "q")
    if has_k:
        check(ko, ref.head_forward(w["k"], norm, w["w_k"], EPS, pos, freq, pairs), kind, "k")
    dq, dk = _nan(T, H, d, dtype=t), _nan(T, Hk, d, dtype=t) if has_k else None
    grads = norm and weight
    dwq, dwk = (_nan(d, dtype=torch.float32), _nan(d, dtype=torch.float32) if has_k else None) if grads else (None, None)
    ws = torch.empty(kda.kda_head_norm_rotary_workspace_bytes(d), dtype=torch.uint8, device="cuda") if grads else None
    kda.kda_head_norm_rotary_backward(dev["q"] if norm else None, k if norm else None, norm, dev["w_q"], dev["w_k"] if has_k else None, EPS, pos_dev,
                                      phases, pairs, dev["gq"], dev["gk"] if has_k else None, dq, dk, dwq, dwk, ws)
    for n, dx, dw in (("q", dq, dwq), ("k", dk, dwk)):
        if dx is None:
            continue
        x_ref, w_ref = ref.head_backward(w[n], norm, w["w_" + n], EPS, pos, freq, pairs, w["g" + n])
        check(dx, x_ref, kind, "d" + n)
        if dw is not None:
            check(dw, w_ref, "f32", "dw_" + n)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,Hk,d", [(1, 1, 1, 32), (3, 5, 5, 64), (7, 16, 4, 128), (2, 3, 1, 256), (300, 8, 2, 64), (2500, 2, 1, 128)])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_heads(T, H, Hk, d, pairs, kind):
    _both(T, H, Hk, d, d, pairs, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(32, 0), (32, 16), (64, 48), (128, 16), (128, 112), (256, 64), (256, 256)])
@pytest.mark.parametrize("pairs", ["halves", "adjacent"])
def test_rotated_channels(d, rot, pairs, kind):
    _both(11, 3, 2, d, rot, pairs, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("norm,weight", [(False, False), (True, False)])
def test_absent_parts(norm, weight, kind):
    _both(13, 4, 2, 64, 32, "halves", kind, norm=norm, weight=weight)
    _both(13, 4, 0, 64, 64, "adjacent", kind, norm=norm, weight=weight)
    _both(13, 4, 0, 128, 0, "halves", kind, norm=norm, weight=True)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 2, 8])
def test_rows_of_a_wider_matrix(offset, kind):
    _both(29, 6, 3, 64, 64, "halves", kind, offset=offset)
    _both(29, 2, 1, 128, 32, "adjacent", kind, offset=offset)


@pytest.mark.parametrize("far", [1_000_000, 2 ** 31 - 5001, -(2 ** 31)])
def test_far_positions_keep_their_angles(far):
    """The reference's angle is position * frequency in 64 bits, 2^31 * 2^-53 = 2.4e-7 of a radian off at most."""
    _both(40, 2, 1, 64, 64, "halves", "f32", far=far)


def test_frequencies_of_any_size():
    from context_kda_gb300 import binding as kda
    f = np.array([0.0, 1e-9, 1.0, 6.283185307179586, 12.0, -0.5, -1e-30, 1e6])
    turns = kda.kda_rotary_phases(f).view(np.uint64).astype(np.float64) / 2.0 ** 64
    want = f / (2 * np.pi)
    gap = np.abs(turns - (want - np.floor(want)))
    assert np.all(np.minimum(gap, 1 - gap) <= 1e-15 * (1 + np.abs(want)))


def test_in_place():
    import torch
    from context_kda_gb300 import binding as kda
    dev, _ = _draw(50, 6, 2, 128, "bf16")
    pos, freq, pos_dev, phases = _rotation(50, 128)
    out = torch.empty_like(dev["q"]), torch.empty_like(dev["k"])
    args = (True, dev["w_q"], dev["w_k"], EPS, pos_dev, phases, "halves")
    kda.kda_head_norm_rotary_forward(dev["q"], dev["k"], *args, *out)
    q, k = dev["q"].clone(), dev["k"].clone()
    kda.kda_head_norm_rotary_forward(q, k, *args, q, k)
    assert torch.equal(q, out[0]) and torch.equal(k, out[1])
    grads = torch.empty_like(q), torch.empty_like(k)
    kda.kda_head_norm_rotary_backward(dev["q"], dev["k"], *args, dev["gq"], dev["gk"], *grads, None, None, None)
    gq, gk = dev["gq"].clone(), dev["gk"].clone()
    kda.kda_head_norm_rotary_backward(dev["q"], dev["k"], *args, gq, gk, gq, gk, None, None, None)
    assert torch.equal(gq, grads[0]) and torch.equal(gk, grads[1])


def test_bad_values_stay_in_their_head():
    """A NaN or infinity in one head leaves every other head's bits; without norm, channels that are not rotated keep theirs."""
    import torch
    from context_kda_gb300 import binding as kda
    dev, _ = _draw(9, 4, 2, 64, "bf16")
    pos, freq, pos_dev, phases = _rotation(9, 32)
    for bad in (float("nan"), float("inf")):
        outs = []
        for x in (dev["q"], dev["q"].clone()):
            if outs:
                x[3, 1, 5] = bad
                x[4, 2, 50] = bad
            o, ko = torch.empty_like(x), torch.empty_like(dev["k"])
            kda.kda_head_norm_rotary_forward(x, dev["k"], False, None, None, EPS, pos_dev, phases, "halves", o, ko)
            outs.append(o)
        same = outs[0].view(torch.int16) == outs[1].view(torch.int16)
        changed = {tuple(i) for i in (~same).nonzero().tolist()}
        assert changed == {(3, 1, 5), (3, 1, 21), (4, 2, 50)}


def test_positions_without_phases():
    """Nothing to rotate: positions are not looked at."""
    import torch
    from context_kda_gb300 import binding as kda
    dev, w = _draw(6, 2, 1, 64, "f32")
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(dev["q"]), torch.empty_like(dev["k"])
    kda.kda_head_norm_rotary_forward(dev["q"], dev["k"], True, None, None, EPS, pos, None, "halves", qo, ko)
    check(qo, ref.head_forward(w["q"], True, None, EPS, np.zeros(6), np.zeros(0), "halves"), "f32", "q")


def test_no_rows():
    import torch
    from context_kda_gb300 import binding as kda
    q, k = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    w, pos, phases = torch.ones(64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), torch.zeros(32, dtype=torch.int64, device="cuda")
    kda.kda_head_norm_rotary_forward(q, k, True, w, w, EPS, pos, phases, "halves", q, k)
    dw = _nan(64, dtype=torch.float32), _nan(64, dtype=torch.float32)
    ws = torch.empty(kda.kda_head_norm_rotary_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    kda.kda_head_norm_rotary_backward(q, k, True, w, w, EPS, pos, phases, "halves", q, k, q, k, *dw, ws)
    assert not dw[0].any() and not dw[1].any()


def test_same_bits_on_another_stream_and_in_a_graph():
    import torch
    from context_kda_gb300 import binding as kda
    dev, _ = _draw(700, 8, 2, 128, "bf16")
    pos, freq, pos_dev, phases = _rotation(700, 128)
    ws = torch.empty(kda.kda_head_norm_rotary_workspace_bytes(128), dtype=torch.uint8, device="cuda")

    def once():
        dq, dk, dw = torch.empty_like(dev["q"]), torch.empty_like(dev["k"]), torch.empty(2, 128, device="cuda")
        kda.kda_head_norm_rotary_backward(dev["q"], dev["k"], True, dev["w_q"], dev["w_k"], EPS, pos_dev, phases, "halves", dev["gq"], dev["gk"],
                                          dq, dk, dw[0], dw[1], ws)
        return dq, dk, dw

    want = once()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = once()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = once()
    for x in held:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, held):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_gradients_against_differences():
    """Central differences in fp32 along random directions, step 1e-2: error (1e-2)^2 of the third derivative and 1e-7 / 2e-2 from
    rounding; one part in a hundred of the directional derivative's size covers both."""
    import torch
    from context_kda_gb300 import binding as kda
    dev, _ = _draw(20, 3, 2, 64, "f32")
    pos, freq, pos_dev, phases = _rotation(20, 64)
    gen = torch.Generator(device="cuda").manual_seed(3)
    names = ("q", "k", "w_q", "w_k")

    def loss(v):
        qo, ko = torch.empty_like(v["q"]), torch.empty_like(v["k"])
        kda.kda_head_norm_rotary_forward(v["q"], v["k"], True, v["w_q"], v["w_k"], EPS, pos_dev, phases, "adjacent", qo, ko)
        return float((qo.double() * dev["gq"]).sum() + (ko.double() * dev["gk"]).sum())

    grads = {n: torch.empty_like(dev[n]) for n in names}
    ws = torch.empty(kda.kda_head_norm_rotary_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    kda.kda_head_norm_rotary_backward(dev["q"], dev["k"], True, dev["w_q"], dev["w_k"], EPS, pos_dev, phases, "adjacent", dev["gq"], dev["gk"],
                                      *(grads[n] for n in names), ws)
    for n in names:
        dirn = torch.randn(dev[n].shape, generator=gen, device="cuda")
        up, down = (loss({**{m: dev[m] for m in names}, n: dev[n] + s * 1e-2 * dirn}) for s in (1, -1))
        got, want = float((grads[n].double() * dirn).sum()), (up - down) / 2e-2
        size = float((grads[n].double() * dirn).square().sum().sqrt())
        assert abs(got - want) <= 1e-2 * max(abs(want), size), (n, got, want)


def test_row_offsets_beyond_32_bits():
    """Rows 2^30 elements apart: the third row's offset passes 2^31."""
    import torch
    from context_kda_gb300 import binding as kda
    wide = torch.empty(3, 2 ** 30, dtype=torch.bfloat16, device="cuda")
    q = wide[:, :4 * 64].unflatten(1, (4, 64))
    q.copy_(torch.randn(3, 4, 64, device="cuda"))
    want, got = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"), wide[:, 1024:1024 + 4 * 64].unflatten(1, (4, 64))
    kda.kda_head_norm_rotary_forward(q.contiguous(), None, True, None, None, EPS, None, None, "halves", want, None)
    kda.kda_head_norm_rotary_forward(q, None, True, None, None, EPS, None, None, "halves", got, None)
    assert torch.equal(got, want)
