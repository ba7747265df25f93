"""GPU tests of the gated linear recurrence (forward, gradients, one-token step) against its 64-bit
definition (tests/ops_reference.py, whose tolerances apply)."""
import numpy as np
import pytest

import ops_reference as ref
from ops_reference import check, torch_type

pytestmark = pytest.mark.gpu

LENGTHS = [[1], [2], [127], [128], [129], [1, 1, 1], [128, 128], [100, 1, 156, 300], [1500], [60, 1, 700, 64, 5, 128, 640, 3]]


def _draw(lens, D, kind, with_i=True, with_h0=True, split=False, seed=0, g_lo=-0.2, g_hi=-0.001):
    """Device tensors and their exact 64-bit values."""
    import torch
    t = torch_type(kind)
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    cu = [0] + [int(c) for c in np.cumsum(lens)]
    normal = lambda *s: torch.randn(*s, generator=gen)
    x, i, g = normal(T, D).to(t), torch.rand(T, D, generator=gen).to(t), g_lo + (g_hi - g_lo) * torch.rand(T, D, generator=gen)
    h0 = normal(N, D) if with_h0 else None
    dh, dfinal = normal(T, D).to(t), normal(N, D)
    if split:     # x, i and g as column ranges of wider rows, at an odd offset
        wide = torch.zeros(T, 2 * D + 3, dtype=t)
        wide[:, 1:D + 1], wide[:, D + 2:2 * D + 2] = x, i
        wide = wide.cuda()
        xd, idv = wide[:, 1:D + 1], wide[:, D + 2:2 * D + 2]
        gw = torch.zeros(T, D + 5)
        gw[:, 2:D + 2] = g
        gd = gw.cuda()[:, 2:D + 2]
    else:
        xd, idv, gd = x.cuda(), i.cuda(), g.cuda()
    dev = {"x": xd, "i": idv if with_i else None, "g": gd, "h0": None if h0 is None else h0.cuda(), "dh": dh.cuda(),
           "dfinal": dfinal.cuda()}
    f64 = lambda v: None if v is None else v.double().numpy()
    return cu, dev, {"x": f64(x), "i": f64(i) if with_i else None, "g": f64(g), "h0": f64(h0), "dh": f64(dh), "dfinal": f64(dfinal)}


def _forward(cu, dev, stream=None, plan=None):
    import torch
    from context_kda_gb300 import binding as kda
    x = dev["x"]
    T, D, N = cu[-1], x.shape[1], len(cu) - 1
    plan = kda.kda_plan_segments(cu, 1) if plan is None else plan
    plan_dev = kda.upload_plan(plan)
    nan = float("nan")
    h = torch.full((T, D), nan, dtype=x.dtype, device="cuda")
    final = torch.full((N, D), nan, device="cuda")
    states = torch.full((-(-T // 128), D), nan, device="cuda")
    ws = torch.full((kda.kda_gated_scan_workspace_bytes(plan, D) + 16,), 85, dtype=torch.uint8, device="cuda")[:-16]
    kda.kda_gated_scan_forward(plan, plan_dev, x, dev["i"], dev["g"], dev["h0"], h, final, states, ws, stream)
    return h, final, states


def _backward(cu, dev, states, with_dfinal=True):
    import torch
    from context_kda_gb300 import binding as kda
    x = dev["x"]
    T, D, N = cu[-1], x.shape[1], len(cu) - 1
    plan = kda.kda_plan_segments(cu, 1)
    plan_dev = kda.upload_plan(plan)
    nan = float("nan")
    dx = torch.full((T, D), nan, dtype=x.dtype, device="cuda")
    di = None if dev["i"] is None else torch.full((T, D), nan, dtype=x.dtype, device="cuda")
    dg, dh0 = torch.full((T, D), nan, device="cuda"), torch.full((N, D), nan, device="cuda")
    ws = torch.full((kda.kda_gated_scan_workspace_bytes(plan, D) + 16,), 85, dtype=torch.uint8, device="cuda")[:-16]
    kda.kda_gated_scan_backward(plan, plan_dev, x, dev["i"], dev["g"], dev["h0"], states, dev["dh"],
                                dev["dfinal"] if with_dfinal else None, dx, di, dg, dh0, ws)
    return dx, di, dg, dh0


def _check_all(lens, D, kind, with_dfinal=True, **how):
    import torch
    from context_kda_gb300 import binding as kda
    cu, dev, w = _draw(lens, D, kind, **how)
    h, final, states = _forward(cu, dev)
    got = _backward(cu, dev, states, with_dfinal)
    assert kda.kda_device_status() == kda.KDA_OK
    h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    check(h, h_ref, kind, "h")
    check(final, f_ref, "f32", "final")
    check(states, ref.saved_states(h_ref), "f32", "states")
    want = ref.scan_backward(cu, w["x"], w["i"], w["g"], w["h0"], w["dh"], w["dfinal"] if with_dfinal else None)
    for name, a, b, k in zip(("dx", "di", "dg", "dh0"), got, want, (kind, kind, "f32", "f32")):
        if a is not None:
            check(a, b, k, name)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", LENGTHS, ids=lambda v: "-".join(map(str, v)))
def test_lengths(lens, kind):
    _check_all(lens, 64, kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 3, 31, 33, 63, 65, 72, 128, 200, 1001, 2048])
def test_widths(D, kind):
    _check_all([90, 1, 300], D, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [64, 65, 320])
def test_column_ranges_of_wider_rows(D, kind):
    _check_all([200, 3, 180], D, kind, split=True)


@pytest.mark.parametrize("with_i,with_h0,with_dfinal", [(False, True, True), (True, False, True), (True, True, False), (False, False, False)])
def test_absent_tensors(with_i, with_h0, with_dfinal):
    for D in (64, 33):
        _check_all([70, 260, 1], D, "bf16", with_i=with_i, with_h0=with_h0, with_dfinal=with_dfinal)


def test_many_tiles_in_one_sequence():
    _check_all([128 * 45 + 17], 64, "bf16")
    _check_all([128 * 45 + 17], 200, "f32", seed=3)


def test_many_short_sequences():
    rng = np.random.default_rng(4)
    _check_all([int(n) for n in rng.integers(1, 9, 700)], 64, "bf16")
    _check_all([1] * 900, 40, "f16")


def test_long_memory():
    """Decays of 1 - 2^-12 to 1: sums over thousands of tokens; exp(g) is one rounding from exact, so
    n tokens of memory leave at most n 2^-24 relative, 4000 * 6e-8 = 2.4e-4, as a bound."""
    cu, dev, w = _draw([5000], 64, "f32", g_lo=-2.0 ** -12, g_hi=0.0)
    h, final, _ = _forward(cu, dev)
    h_ref, _ = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    x = h.double().cpu().numpy()
    assert np.linalg.norm(x - h_ref) <= 2.4e-4 * np.linalg.norm(h_ref)


def test_strong_and_total_decay():
    """g down to -200 (exp underflows) and minus infinity: h is then the token's own term."""
    import torch
    cu, dev, w = _draw([300, 40], 64, "f32", g_lo=-200.0, g_hi=0.0)
    dev["g"][::7] = float("-inf")
    w["g"][::7] = -np.inf
    h, final, states = _forward(cu, dev)
    h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    check(h, h_ref, "f32", "h")
    got = _backward(cu, dev, states)
    for name, a, b in zip(("dx", "di", "dg", "dh0"), got, ref.scan_backward(cu, w["x"], w["i"], w["g"], w["h0"], w["dh"], w["dfinal"])):
        check(a, b, "f32", name)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_sequences_do_not_see_each_other(bad):
    """Infinities and NaN in one sequence leave every other sequence's results as they were, bit for bit."""
    import torch
    lens = [130, 300, 5, 260]
    cu, dev, _ = _draw(lens, 72, "bf16")
    h, final, states = _forward(cu, dev)
    grads = _backward(cu, dev, states)
    dev["x"][cu[1] + 20, :] = bad
    dev["dh"][cu[1] + 20, :] = bad
    dev["h0"][1] = bad
    dev["dfinal"][1] = bad
    h2, final2, states2 = _forward(cu, dev)
    grads2 = _backward(cu, dev, states2)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for n in (0, 2, 3):
        rows = slice(cu[n], cu[n + 1])
        assert same(h[rows], h2[rows]) and same(final[n], final2[n])
        for a, b in zip(grads[:3], grads2[:3]):
            assert same(a[rows], b[rows])
        assert same(grads[3][n], grads2[3][n])
    assert not bool(torch.isfinite(h2[cu[1] + 20:cu[2]]).any())


def test_same_call_same_bits():
    import torch
    cu, dev, _ = _draw([4000, 100, 3000], 200, "bf16")
    a = _forward(cu, dev)
    ga = _backward(cu, dev, a[2])
    for _ in range(3):
        b = _forward(cu, dev)
        gb = _backward(cu, dev, b[2])
        for x, y in zip(a + ga, b + gb):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_another_stream():
    import torch
    cu, dev, w = _draw([700, 30], 64, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h, _, _ = _forward(cu, dev)
    side.synchronize()
    check(h, ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])[0], "bf16", "h")
    torch.cuda.synchronize()
    h, _, _ = _forward(cu, dev, stream=side)
    torch.cuda.synchronize()
    check(h, ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])[0], "bf16", "h")


def test_graph_capture_replays():
    """The calls can be captured: nothing is allocated or synchronised, and a replay redoes the work."""
    import torch
    from context_kda_gb300 import binding as kda
    cu, dev, w = _draw([1000, 200], 64, "bf16")
    plan = kda.kda_plan_segments(cu, 1)
    plan_dev = kda.upload_plan(plan)
    h = torch.zeros(cu[-1], 64, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kda.kda_gated_scan_workspace_bytes(plan, 64), dtype=torch.uint8, device="cuda")
    call = lambda: kda.kda_gated_scan_forward(plan, plan_dev, dev["x"], dev["i"], dev["g"], dev["h0"], h, None, None, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        h.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(h, ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])[0], "bf16", "h")


def test_offsets_beyond_32_bits():
    """Rows far apart: element offsets pass 2^31 and byte offsets 2^32."""
    import torch
    T, D, wide = 70000, 64, 40000
    cu, dev, w = _draw([T], D, "bf16", seed=9)
    big = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    x = big[:, wide - D:]
    x.copy_(dev["x"])
    assert (T - 1) * wide > 2 ** 31
    dev["x"] = x
    h, final, states = _forward(cu, dev)
    h_ref, _ = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    check(h, h_ref, "bf16", "h")
    got = _backward(cu, dev, states)
    want = ref.scan_backward(cu, w["x"], w["i"], w["g"], w["h0"], w["dh"], w["dfinal"])
    for name, a, b, k in zip(("dx", "di", "dg", "dh0"), got, want, ("bf16", "bf16", "f32", "f32")):
        check(a, b, k, name)


def test_a_device_plan_of_another_problem_is_refused():
    import torch
    from context_kda_gb300 import binding as kda
    assert kda.kda_device_status() == kda.KDA_OK
    cu, dev, _ = _draw([500], 64, "bf16")
    plan, other = kda.kda_plan_segments(cu, 1), kda.upload_plan(kda.kda_plan_segments([0, 100, 500], 1))
    h = torch.full((500, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(kda.kda_gated_scan_workspace_bytes(plan, 64), dtype=torch.uint8, device="cuda")
    kda.kda_gated_scan_forward(plan, other, dev["x"], dev["i"], dev["g"], dev["h0"], h, None, None, ws)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert kda.kda_device_status() == kda.KDA_OK
    assert bool((h == 7.0).all())


# ---- one token ------------------------------------------------------------------------------------------


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,D,with_i", [(1, 1, True), (1, 2048, True), (5, 33, False), (64, 2048, True), (300, 65, True), (70000, 8, True)])
def test_step(B, D, with_i, kind):
    import torch
    from context_kda_gb300 import binding as kda
    gen = torch.Generator().manual_seed(B + D)
    t = torch_type(kind)
    x, i = torch.randn(B, D, generator=gen).to(t), torch.rand(B, D, generator=gen).to(t)
    g, state = -0.2 * torch.rand(B, D, generator=gen), torch.randn(B + 4, D, generator=gen)
    slots = torch.randperm(B + 4, generator=gen)[:B].to(torch.int32)
    slots[::5] = -1                                  # padding rows
    got_state = state.cuda()
    h = torch.full((B, D), float("nan"), dtype=t, device="cuda")
    kda.kda_gated_scan_step(slots.cuda(), x.cuda(), i.cuda() if with_i else None, g.cuda(), got_state, h)
    live = (slots >= 0).numpy()
    sl = slots.numpy()[live]
    want = state.double().numpy()
    u = x.double().numpy() * (i.double().numpy() if with_i else 1.0)
    want[sl] = np.exp(g.double().numpy())[live] * want[sl] + u[live]
    out = np.zeros((B, D))
    out[live] = want[sl]
    check(got_state, want, "f32", "state")
    check(h, out, kind, "h")
    untouched = np.setdiff1d(np.arange(B + 4), sl)
    assert torch.equal(got_state.cpu()[untouched], state[untouched])
    assert bool((h.cpu()[~torch.from_numpy(live)] == 0).all())


def test_step_continues_a_forward():
    """A forward over n tokens equals a forward over n - 1 and one step, per sequence."""
    import torch
    from context_kda_gb300 import binding as kda
    lens = [130, 2, 257]
    cu, dev, w = _draw(lens, 72, "bf16")
    h, final, _ = _forward(cu, dev)
    keep = [t for n in range(3) for t in range(cu[n], cu[n + 1] - 1)]
    last = [cu[n + 1] - 1 for n in range(3)]
    cut = {k: (None if v is None else v[keep] if k in ("x", "i", "g", "dh") else v) for k, v in dev.items()}
    _, state, _ = _forward([0] + [int(c) for c in np.cumsum([n - 1 for n in lens])], cut)
    out = torch.empty(3, 72, dtype=torch.bfloat16, device="cuda")
    kda.kda_gated_scan_step(None, dev["x"][last], dev["i"][last], dev["g"][last], state, out)
    h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    check(state, f_ref, "f32", "state")
    check(out, h_ref[last], "bf16", "h")


def test_step_records_a_slot_out_of_range():
    import torch
    from context_kda_gb300 import binding as kda
    assert kda.kda_device_status() == kda.KDA_OK
    state = torch.ones(2, 8, device="cuda")
    h = torch.full((2, 8), 5.0, device="cuda")
    slots = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    kda.kda_gated_scan_step(slots, torch.ones(2, 8, device="cuda"), None, torch.zeros(2, 8, device="cuda"), state, h)
    assert kda.kda_device_status() == kda.KDA_ERR_INVALID_ARG
    assert kda.kda_device_status() == kda.KDA_OK
    assert state.tolist() == [[1.0] * 8, [2.0] * 8] and h.tolist() == [[2.0] * 8, [0.0] * 8]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [5, 34, 65, 130])
def test_every_alignment(D, kind):
    """Tensors that start at every element of 16 bytes, with rows of every length modulo 16 bytes; the values around
    them are NaN and stay out of the results."""
    import torch
    per = 128 // torch.finfo(torch_type(kind)).bits
    cu, dev, w = _draw([140, 20], D, kind, seed=D)
    h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    want = ref.scan_backward(cu, w["x"], w["i"], w["g"], w["h0"], w["dh"], w["dfinal"])
    for first in range(per):
        for pad in (0, 1, 2, 3):
            moved = dict(dev)
            for name in ("x", "i", "g", "dh"):
                ld = D + pad
                flat = torch.full((cu[-1] * ld + first + 8,), float("nan"), dtype=dev[name].dtype, device="cuda")
                rows = flat[first:first + cu[-1] * ld].view(cu[-1], ld)[:, :D]
                rows.copy_(dev[name])
                moved[name] = rows
            h, final, states = _forward(cu, moved)
            check(h, h_ref, kind, "h")
            check(final, f_ref, "f32", "final")
            for name, a, b, k in zip(("dx", "di", "dg", "dh0"), _backward(cu, moved, states), want, (kind, kind, "f32", "f32")):
                check(a, b, k, name)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths,D", [([300, 140], 34), ([300, 140], 65), ([900, 1, 320], 65), ([1290], 98)])
def test_alignment_inside(lengths, D, kind):
    """The same for tiles that have rows on both sides, which are copied in whole pieces of 16 bytes: by a cluster and
    by a chain of tiles."""
    import torch
    per = 128 // torch.finfo(torch_type(kind)).bits
    cu, dev, w = _draw(lengths, D, kind, seed=D)
    h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    want = ref.scan_backward(cu, w["x"], w["i"], w["g"], w["h0"], w["dh"], w["dfinal"])
    for first, pad in ((0, 1), (1, 0), (per - 1, 2), (2, 3)):
        moved = dict(dev)
        for name in ("x", "i", "g", "dh"):
            ld = D + pad
            flat = torch.full((cu[-1] * ld + first,), float("nan"), dtype=dev[name].dtype, device="cuda")
            rows = flat[first:first + cu[-1] * ld].view(cu[-1], ld)[:, :D]
            rows.copy_(dev[name])
            moved[name] = rows
        h, final, states = _forward(cu, moved)
        check(h, h_ref, kind, "h")
        check(final, f_ref, "f32", "final")
        for name, a, b, k in zip(("dx", "di", "dg", "dh0"), _backward(cu, moved, states), want, (kind, kind, "f32", "f32")):
            check(a, b, k, name)


@pytest.mark.parametrize("lengths", [[400, 300], [1400, 300], [5, 400, 1]])
def test_growing_decays_of_a_zero_state(lengths):
    """exp(g) = e: the decays' product passes fp32's range long before the sequence ends, the state is zero all along."""
    import torch
    D = 70
    cu, dev, _ = _draw(lengths, D, "bf16", seed=3, with_h0=False)
    a, b = cu[-3], cu[-2]
    dev["g"][a:b] = 1.0
    dev["x"][a:b] = 0.0
    dev["dh"][a:b] = 0.0
    dev["dfinal"][-2] = 0.0
    h, final, states = _forward(cu, dev)
    assert not h[a:b].any() and not final[-2].any() and torch.isfinite(h).all() and torch.isfinite(final).all()
    dx, di, dg, dh0 = _backward(cu, dev, states)
    for t in (dx, di, dg):
        assert not t[a:b].any() and torch.isfinite(t).all()
    assert not dh0[-2].any() and torch.isfinite(dh0).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [2048, 2049, 2050])
def test_groups_of_a_wide_input(D, kind):
    """Wide inputs pass their state on in shorter groups of tiles: several of them, boundaries at and within tiles."""
    _check_all([1500, 36, 1, 640], D, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,D", [(3, 511), (9, 513), (40, 1001), (7, 2046)])
def test_step_of_unaligned_rows(B, D, kind):
    test_step(B, D, True, kind)


def test_two_streams_at_once():
    """Chains of tiles on two streams of different priority share the device: neither needs its whole grid there at once."""
    import torch
    from context_kda_gb300 import binding as kda
    lens = [[9000, 40, 3000], [7000, 5000]]
    draws = [_draw(lens[0], 1100, "bf16", seed=5), _draw(lens[1], 1024, "bf16", seed=6)]
    want = [_forward(cu, dev) for cu, dev, _ in draws]
    want_grads = [_backward(cu, dev, w[2]) for (cu, dev, _), w in zip(draws, want)]
    for (cu, _, w), (h, final, _) in zip(draws, want):
        h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
        check(h, h_ref, "bf16", "h")
        check(final, f_ref, "f32", "final")
    streams = [torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for n, (cu, dev, _) in enumerate(draws):
            with torch.cuda.stream(streams[n]):
                f = _forward(cu, dev)
                got[n].append(f + _backward(cu, dev, f[2]))
    torch.cuda.synchronize()
    assert kda.kda_device_status() == kda.KDA_OK
    for n in range(2):
        for one in got[n]:
            for a, b in zip(one, want[n] + want_grads[n]):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _relative(got, want, bound, what):
    """Every value within a share of itself (and fp32's smallest numbers)."""
    x = got.double().cpu().numpy()
    assert x.shape == want.shape and np.all(np.isfinite(x)), what
    worst = float(np.max(np.abs(x - want) / (bound * np.abs(want) + 2.0 ** -126)))
    assert worst <= 1.0, f"{what}: {worst:.3g} times the tolerance"


# (lengths, (first token, tokens, log-decay) of the stretches whose decays are not one)
GROWING = {"within a run": ([40], [(0, 15, 8.0)]), "two runs": ([60], [(20, 15, 8.0)]), "within a tile": ([400], [(4, 120, 1.0)]),
           "over tiles": ([1000], [(100, 240, 0.5)]), "chain, a run": ([2500], [(200, 15, 8.0)]), "chain, over tiles": ([40, 2500, 7], [(300, 240, 0.5)]),
           "several boundaries in a run": ([5, 4, 12, 3, 30, 2], [(9, 12, 10.0)]), "before a boundary": ([19, 40], [(3, 14, 8.5)]),
           "and back": ([1500], [(16, 15, 8.0), (31, 60, -1.0)]), "and forgotten": ([300], [(16, 15, 8.0), (31, 1, -np.inf)])}


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 70])
@pytest.mark.parametrize("case", GROWING, ids=lambda c: c.replace(" ", "-"))
def test_growing_decays_of_a_small_state(case, D, kind):
    """A state of 1e-25 that grows by e^120: the product of the decays passes fp32's range, the state does not (nor do the
    gradients, whose last one is 1e-25 too, or 1e5 where they shrink before they grow).  Every decay is off by
    2^-22 (the exponential) and 1.5 |g| 2^-24 (its argument), every product by 2^-24 of itself; these add up.  Channels whose
    state is zero stay at zero next to it."""
    lens, stretches = GROWING[case]
    cu, dev, w = _draw(lens, D, kind, seed=D)
    for name in ("x", "dh"):
        dev[name].zero_()
        w[name][:] = 0
    steps = 60
    for v in (dev["g"], w["g"]):
        v[:] = 0
        for first, n, g in stretches:
            v[first:first + n] = g
    for first, n, g in stretches:
        steps += n * (4 + (1.5 * abs(g) if np.isfinite(g) else 0) + 2)
    for name, size in (("h0", 1e-25), ("dfinal", 1e5 if case == "and back" else 1e-25)):
        dev[name][:, ::3], w[name][:, ::3] = 0, 0
        dev[name][:, 1::3], w[name][:, 1::3] = size, float(np.float32(size))
        dev[name][:, 2::3], w[name][:, 2::3] = -size, -float(np.float32(size))
    bound = 2.0 ** -24 * steps
    h_ref, f_ref = ref.scan_forward(cu, w["x"], w["i"], w["g"], w["h0"])
    assert 1e26 < np.abs(h_ref).max() < 1e30
    h, final, states = _forward(cu, dev)
    _relative(h, h_ref, bound + ref.ROUND[kind], "h")
    _relative(final, f_ref, bound, "final")
    _relative(states, ref.saved_states(h_ref), bound, "states")
    assert not h[:, ::3].any() and not final[:, ::3].any()
    got = _backward(cu, dev, states)
    want = ref.scan_backward(cu, w["x"], w["i"], w["g"], w["h0"], w["dh"], w["dfinal"])
    for name, a, b, k in zip(("dx", "di", "dg", "dh0"), got, want, (kind, kind, "f32", "f32")):
        _relative(a, b, 2 * bound + 2 * ref.ROUND[k], name)


@pytest.mark.parametrize("lens", [[9, 400, 5, 260], [9, 1600, 3, 2, 300]], ids=["cluster", "chain"])
def test_growing_decays_of_one_channel_or_sequence(lens):
    """Other channels and other sequences keep their bits."""
    import torch
    D = 70
    cu, dev, _ = _draw(lens, D, "bf16", seed=11)
    a = _forward(cu, dev)
    ga = _backward(cu, dev, a[2])
    first, last = cu[1], cu[2]
    dev["g"][first:first + 20, 8] = 9.0
    dev["g"][last - 20:last, 8] = 9.0
    dev["g"][last - 40:last - 30, 9] = float("inf")
    b = _forward(cu, dev)
    gb = _backward(cu, dev, b[2])
    same = lambda x, y: torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    others = [c for c in range(D) if c not in (8, 9)]
    for x, y in zip(a + ga, b + gb):
        assert same(x[:, others], y[:, others])
    assert same(a[0][first + 20:last - 40, 9], b[0][first + 20:last - 40, 9])     # also what comes before an infinite decay
    for n in range(len(lens)):
        if n != 1:
            rows = slice(cu[n], cu[n + 1])
            for x, y in ((a[0], b[0]), *zip(ga[:3], gb[:3])):
                assert same(x[rows], y[rows])
            assert same(a[1][n], b[1][n]) and same(ga[3][n], gb[3][n])


def test_widths_beyond_2_to_the_29():
    """Bytes of a row that pass 2^31: h = exp(g) h0 + x with every value known, and its gradients."""
    import math

    import torch
    from context_kda_gb300 import binding as kda
    D = 2 ** 29 + 8
    full = lambda v: torch.full((1, D), v, device="cuda")
    plan = kda.kda_plan_segments([0, 1], 1)
    plan_dev = kda.upload_plan(plan)
    x, g, h0, h, final = full(1.0), full(math.log(0.5)), full(2.0), full(float("nan")), full(float("nan"))
    states = full(float("nan"))
    kda.kda_gated_scan_forward(plan, plan_dev, x, None, g, h0, h, final, states, None)
    off = lambda t, v: float(t.sub_(v).abs_().max())
    assert off(h, 2.0) <= 1e-5 and off(final, 2.0) <= 1e-5 and off(states, 0.0) == 0.0
    dx, dg, dh0 = full(float("nan")), full(float("nan")), full(float("nan"))
    kda.kda_gated_scan_backward(plan, plan_dev, x, None, g, h0, states, full(1.0), None, dx, None, dg, dh0, None)
    assert off(dx, 1.0) == 0.0 and off(dg, 1.0) <= 1e-5 and off(dh0, 0.5) <= 1e-5


def test_lengths_up_to_2_to_the_31():
    """The last tile of a stream of 2^31 - 100 tokens would end beyond 32 bits; its rows start anywhere."""
    import torch
    from context_kda_gb300 import binding as kda
    T, tail = 2 ** 31 - 100, 300
    plan = kda.kda_plan_segments([0, T], 1)
    plan_dev = kda.upload_plan(plan)
    x = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    g = torch.full((T, 1), -1.0, device="cuda")
    gen = torch.Generator().manual_seed(8)
    last = torch.randn(tail, 1, generator=gen).to(torch.bfloat16)
    x[T - tail:] = last.cuda()
    h = torch.empty_like(x)
    ws = torch.empty(kda.kda_gated_scan_workspace_bytes(plan, 1), dtype=torch.uint8, device="cuda")
    final = torch.empty(1, 1, device="cuda")
    kda.kda_gated_scan_forward(plan, plan_dev, x, None, g, None, h, final, None, ws)
    assert kda.kda_device_status() == kda.KDA_OK
    h_ref, f_ref = ref.scan_forward([0, tail], last.double().numpy(), None, np.full((tail, 1), -1.0), None)
    check(h[T - tail:], h_ref, "bf16", "h")
    check(final, f_ref, "f32", "final")
    assert not h[:T - tail].any()
