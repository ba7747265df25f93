"""GPU tests of the block norms (forward and gradients) against their 64-bit definition
(tests/ops_reference.py, whose tolerances apply)."""
import numpy as np
import pytest

import ops_reference as ref
from ops_reference import check, torch_type

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _draw(T, D, kind, res, gate="sigmoid", group=0, r=True, o=True, post=True, ls=True, pre=True, pad=0, seed=0):
    import torch
    gen = torch.Generator().manual_seed(seed + 7 * T + D)
    t, rt = torch_type(kind), torch_type(res)
    normal = lambda *s: torch.randn(*s, generator=gen)

    def rows(dtype, std=1.0):
        v = (std * normal(T, D)).to(dtype)
        if not pad:
            return v, v.cuda()
        wide = torch.zeros(T, D + pad, dtype=dtype)
        wide[:, pad // 2:pad // 2 + D] = v
        return v, wide.cuda()[:, pad // 2:pad // 2 + D]

    flat = lambda n: (lambda v: (v, v.cuda()))(1 + 0.3 * normal(n))
    none = (None, None)
    v = {"r": rows(rt, 2.0) if r else none, "o": rows(t, 0.5) if o else none,
         "z": rows(t) if o and gate != "none" else none, "w_post": flat(group or D) if o and post else none,
         "ls": flat(D) if o and ls else none, "w_pre": flat(D) if pre else none, "dr_out": rows(rt), "dy": rows(t) if pre else none}
    return {k: a[1] for k, a in v.items()}, {k: None if a[0] is None else a[0].double().numpy() for k, a in v.items()}


def _forward(d, T, D, kind, res, gate, group, in_place=False):
    import torch
    from context_kda_gb300 import binding as kda
    new = lambda name: torch.full((T, D), float("nan"), dtype=torch_type(name), device="cuda")
    r_out = d["r"] if in_place else new(res)
    y = new(kind) if d["w_pre"] is not None else None
    kda.kda_block_norm_forward(d["r"], d["o"], d["z"], gate, group, d["w_post"], 0.7, d["ls"], d["w_pre"], EPS, r_out, y)
    return r_out, y


def _backward(d, r_out, T, D, kind, res, gate, group):
    import torch
    from context_kda_gb300 import binding as kda
    new = lambda name: torch.full((T, D), float("nan"), dtype=torch_type(name), device="cuda")
    flat = lambda name, n: None if d[name] is None else torch.full((n,), float("nan"), device="cuda")
    dr, do = new(res), None if d["o"] is None else new(kind)
    dz = None if d["z"] is None else new(kind)
    dw = flat("w_post", group or D), flat("ls", D), flat("w_pre", D)
    ws = torch.full((kda.kda_block_norm_workspace_bytes(D),), 85, dtype=torch.uint8, device="cuda")
    kda.kda_block_norm_backward(r_out if d["w_pre"] is not None else None, d["o"], d["z"], gate, group, d["w_post"], 0.7, d["ls"],
                                d["w_pre"], EPS, d["dr_out"], d["dy"], dr, do, dz, *dw, ws)
    return (dr, do, dz) + dw


def _check_all(T, D, kind, res, gate="sigmoid", group=0, **how):
    d, w = _draw(T, D, kind, res, gate, group, **how)
    r_out, y = _forward(d, T, D, kind, res, gate, group)
    args = (w["o"], w["z"], gate, group, w["w_post"], 0.7, w["ls"], w["w_pre"], EPS)
    r_ref, y_ref = ref.norm_forward(w["r"], *args)
    check(r_out, r_ref, res, "r_out")
    if y is not None:
        check(y, y_ref, kind, "y")
    got = _backward(d, r_out, T, D, kind, res, gate, group)
    want = ref.norm_backward(r_out.double().cpu().numpy(), *args, w["dr_out"], w["dy"])
    kinds = (res, kind, kind, "f32", "f32", "f32")
    for name, a, b, k in zip(("dr", "do", "dz", "dw_post", "dls", "dw_pre"), got, want, kinds):
        assert (a is None) == (b is None), name
        if a is not None:
            check(a, b, k, name)


@pytest.mark.parametrize("kind,res", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("T,D,group", [(1, 128, 0), (5, 2048, 128), (3, 4096, 0), (77, 256, 32), (40, 512, 64), (9, 1024, 256)])
def test_types(T, D, group, kind, res):
    _check_all(T, D, kind, res, group=group)


@pytest.mark.parametrize("D", [1, 2, 7, 31, 33, 64, 100, 136, 384, 1000, 1001, 1536, 2056, 4104, 6144, 8192, 8200, 12288, 16384])
def test_widths(D):
    for kind, res in (("bf16", "f32"), ("f32", "f32")):
        _check_all(6, D, kind, res, gate="silu")


@pytest.mark.parametrize("T", [1, 2, 3, 151, 305, 1217, 5000])
def test_rows(T):
    _check_all(T, 256, "bf16", "bf16", group=128)
    _check_all(T, 129, "f16", "f32")


@pytest.mark.parametrize("gate", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("how", [dict(r=False), dict(post=False), dict(ls=False), dict(pre=False), dict(r=False, pre=False),
                                 dict(post=False, ls=False, pre=False)], ids=str)
def test_parts(how, gate):
    for D, group in ((512, 128), (515, 0)):
        _check_all(21, D, "bf16", "bf16", gate=gate, group=group, **how)
        _check_all(21, D, "f16", "f32", gate=gate, group=group, **how)


def test_first_norm_alone():
    import torch
    from context_kda_gb300 import binding as kda
    for D in (2048, 77):
        d, w = _draw(9, D, "bf16", "f32", gate="none", o=False)
        y = torch.full((9, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        kda.kda_block_norm_forward(d["r"], None, None, "none", 0, None, 1.0, None, d["w_pre"], EPS, None, y)
        _, y_ref = ref.norm_forward(w["r"], None, None, "none", 0, None, 1.0, None, w["w_pre"], EPS)
        check(y, y_ref, "bf16", "y")
        dr, dw = torch.full((9, D), float("nan"), device="cuda"), torch.full((D,), float("nan"), device="cuda")
        ws = torch.empty(kda.kda_block_norm_workspace_bytes(D), dtype=torch.uint8, device="cuda")
        kda.kda_block_norm_backward(d["r"], None, None, "none", 0, None, 1.0, None, d["w_pre"], EPS, None, d["dy"], dr, None, None,
                                    None, None, dw, ws)
        want = ref.norm_backward(w["r"], None, None, "none", 0, None, 1.0, None, w["w_pre"], EPS, None, w["dy"])
        check(dr, want[0], "f32", "dr")
        check(dw, want[5], "f32", "dw_pre")


@pytest.mark.parametrize("pad", [6, 16])
@pytest.mark.parametrize("kind,res", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32")])
def test_column_ranges_of_wider_rows(kind, res, pad):
    _check_all(13, 384, kind, res, group=128, pad=pad)
    _check_all(13, 385, kind, res, pad=pad)


def test_in_place_residual_and_gradient():
    import torch
    from context_kda_gb300 import binding as kda
    T, D = 33, 1024
    d, w = _draw(T, D, "bf16", "bf16")
    a, ya = _forward(d, T, D, "bf16", "bf16", "sigmoid", 0)
    b, yb = _forward(d, T, D, "bf16", "bf16", "sigmoid", 0, in_place=True)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(ya.view(torch.int16), yb.view(torch.int16))
    want = _backward(d, a, T, D, "bf16", "bf16", "sigmoid", 0)
    do, dz = torch.empty_like(want[1]), torch.empty_like(want[2])
    ws = torch.empty(kda.kda_block_norm_workspace_bytes(D), dtype=torch.uint8, device="cuda")
    kda.kda_block_norm_backward(a, d["o"], d["z"], "sigmoid", 0, d["w_post"], 0.7, d["ls"], d["w_pre"], EPS, d["dr_out"], d["dy"],
                                d["dr_out"], do, dz, None, None, None, ws)
    for x, y in ((d["dr_out"], want[0]), (do, want[1]), (dz, want[2])):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


def test_rows_of_zeros_and_large_gates():
    """A row of zeros norms to zeros (eps); gates saturate without infinities."""
    import torch
    for D in (512, 513):
        d, w = _draw(8, D, "f32", "f32", gate="silu")
        for name in ("r", "o"):
            d[name][2] = 0
            w[name][2] = 0
        d["z"][:, ::3], w["z"][:, ::3] = 120.0, 120.0
        d["z"][:, 1::3], w["z"][:, 1::3] = -120.0, -120.0
        r_out, y = _forward(d, 8, D, "f32", "f32", "silu", 0)
        r_ref, y_ref = ref.norm_forward(w["r"], w["o"], w["z"], "silu", 0, w["w_post"], 0.7, w["ls"], w["w_pre"], EPS)
        check(r_out, r_ref, "f32", "r_out")
        check(y, y_ref, "f32", "y")
        got = _backward(d, r_out, 8, D, "f32", "f32", "silu", 0)
        assert all(bool(torch.isfinite(v).all()) for v in got)


def test_a_bad_row_stays_alone():
    """Infinities and NaN in a row leave the other rows' results as they were, bit for bit."""
    import torch
    T, D = 40, 512
    d, _ = _draw(T, D, "bf16", "bf16", group=128)
    a = _forward(d, T, D, "bf16", "bf16", "sigmoid", 128)
    ga = _backward(d, a[0], T, D, "bf16", "bf16", "sigmoid", 128)
    d["o"][7, 3], d["r"][7, 9] = float("nan"), float("inf")
    b = _forward(d, T, D, "bf16", "bf16", "sigmoid", 128)
    gb = _backward(d, b[0], T, D, "bf16", "bf16", "sigmoid", 128)
    rows = [t for t in range(T) if t != 7]
    for x, y in zip(a + ga[:3], b + gb[:3]):
        assert torch.equal(x[rows].view(torch.int16), y[rows].view(torch.int16))


def test_same_call_same_bits():
    import torch
    T, D = 5000, 1024
    d, _ = _draw(T, D, "bf16", "bf16", group=128)
    a = _forward(d, T, D, "bf16", "bf16", "sigmoid", 128)
    ga = _backward(d, a[0], T, D, "bf16", "bf16", "sigmoid", 128)
    for _ in range(3):
        b = _forward(d, T, D, "bf16", "bf16", "sigmoid", 128)
        gb = _backward(d, b[0], T, D, "bf16", "bf16", "sigmoid", 128)
        for x, y in zip(a + ga, b + gb):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_no_rows():
    import torch
    from context_kda_gb300 import binding as kda
    d, _ = _draw(0, 64, "bf16", "bf16", group=32)
    r_out, y = _forward(d, 0, 64, "bf16", "bf16", "sigmoid", 32)
    got = _backward(d, r_out, 0, 64, "bf16", "bf16", "sigmoid", 32)
    assert all(bool((v == 0).all()) for v in got[3:])


def test_offsets_beyond_32_bits():
    import torch
    T, D, wide = 70000, 64, 40000
    d, w = _draw(T, D, "bf16", "bf16", group=32)
    big = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    o = big[:, wide - D:]
    o.copy_(d["o"])
    assert (T - 1) * wide > 2 ** 31
    d["o"] = o
    r_out, y = _forward(d, T, D, "bf16", "bf16", "sigmoid", 32)
    r_ref, y_ref = ref.norm_forward(w["r"], w["o"], w["z"], "sigmoid", 32, w["w_post"], 0.7, w["ls"], w["w_pre"], EPS)
    check(r_out, r_ref, "bf16", "r_out")
    check(y, y_ref, "bf16", "y")


def test_another_stream():
    import torch
    T, D = 300, 2048
    d, w = _draw(T, D, "bf16", "f32", group=128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r_out, y = _forward(d, T, D, "bf16", "f32", "sigmoid", 128)
        got = _backward(d, r_out, T, D, "bf16", "f32", "sigmoid", 128)
    side.synchronize()
    args = (w["o"], w["z"], "sigmoid", 128, w["w_post"], 0.7, w["ls"], w["w_pre"], EPS)
    check(y, ref.norm_forward(w["r"], *args)[1], "bf16", "y")
    check(got[1], ref.norm_backward(r_out.double().cpu().numpy(), *args, w["dr_out"], w["dy"])[1], "bf16", "do")


def test_no_eps():
    """eps = 0, with fewer rows than the CTAs take at once: rows that are not there leave nothing in the weights' gradients."""
    import torch
    from context_kda_gb300 import binding as kda
    for T, D, group in ((5, 128, 32), (3, 96, 0), (7, 33, 0)):
        d, w = _draw(T, D, "bf16", "bf16", group=group)
        r_out, y = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kda.kda_block_norm_forward(d["r"], d["o"], d["z"], "sigmoid", group, d["w_post"], 0.7, d["ls"], d["w_pre"], 0.0, r_out, y)
        args = (w["o"], w["z"], "sigmoid", group, w["w_post"], 0.7, w["ls"], w["w_pre"], 0.0)
        check(y, ref.norm_forward(w["r"], *args)[1], "bf16", "y")
        dr, do, dz = (torch.empty(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        dw = [torch.empty(n, device="cuda") for n in (group or D, D, D)]
        ws = torch.empty(kda.kda_block_norm_workspace_bytes(D), dtype=torch.uint8, device="cuda")
        kda.kda_block_norm_backward(r_out, d["o"], d["z"], "sigmoid", group, d["w_post"], 0.7, d["ls"], d["w_pre"], 0.0, d["dr_out"],
                                    d["dy"], dr, do, dz, *dw, ws)
        want = ref.norm_backward(r_out.double().cpu().numpy(), *args, w["dr_out"], w["dy"])
        for a, b, k in zip((dr, do, dz, *dw), want, ("bf16",) * 3 + ("f32",) * 3):
            check(a, b, k)


@pytest.mark.parametrize("kind,res", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("D,group", [(7, 0), (70, 0), (301, 0), (320, 64), (2050, 0)])
def test_every_alignment(D, group, kind, res):
    """Tensors that start at every element of 16 bytes, with rows of every length modulo 16 bytes; the values around
    them are NaN and stay out of the results."""
    import torch
    T = 11
    d, w = _draw(T, D, kind, res, group=group)
    args = (w["o"], w["z"], "sigmoid", group, w["w_post"], 0.7, w["ls"], w["w_pre"], EPS)
    r_ref, y_ref = ref.norm_forward(w["r"], *args)
    for first in range(0, 8, 1 if kind != "f32" else 3):
        for pad in (0, 1, 3):
            moved = dict(d)
            for name in ("r", "o", "z", "dr_out", "dy"):
                ld = D + pad
                flat = torch.full((T * ld + first + 8,), float("nan"), dtype=d[name].dtype, device="cuda")
                moved[name] = flat[first:first + T * ld].view(T, ld)[:, :D]
                moved[name].copy_(d[name])
            r_out, y = _forward(moved, T, D, kind, res, "sigmoid", group)
            check(r_out, r_ref, res, "r_out")
            check(y, y_ref, kind, "y")
            got = _backward(moved, r_out, T, D, kind, res, "sigmoid", group)
            want = ref.norm_backward(r_out.double().cpu().numpy(), *args, w["dr_out"], w["dy"])
            for name, a, b, k in zip(("dr", "do", "dz", "dw_post", "dls", "dw_pre"), got, want, (res, kind, kind, "f32", "f32", "f32")):
                check(a, b, k, name)


@pytest.mark.parametrize("kind,res", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("D,group", [(1, 0), (9, 0), (70, 0), (301, 0), (320, 64), (1002, 0)])
def test_alignment_inside(D, group, kind, res):
    """The same for rows that have 16 others on both sides, which are copied in whole pieces of 16 bytes."""
    import torch
    T = 70
    d, w = _draw(T, D, kind, res, group=group)
    args = (w["o"], w["z"], "sigmoid", group, w["w_post"], 0.7, w["ls"], w["w_pre"], EPS)
    r_ref, y_ref = ref.norm_forward(w["r"], *args)
    for first, pad in ((0, 1), (1, 0), (7, 2), (2, 2)):
        moved = dict(d)
        for name in ("r", "o", "z", "dr_out", "dy"):
            ld = D + pad
            flat = torch.full((T * ld + first,), float("nan"), dtype=d[name].dtype, device="cuda")
            moved[name] = flat[first:first + T * ld].view(T, ld)[:, :D]
            moved[name].copy_(d[name])
        r_out, y = _forward(moved, T, D, kind, res, "sigmoid", group)
        check(r_out, r_ref, res, "r_out")
        check(y, y_ref, kind, "y")
        got = _backward(moved, r_out, T, D, kind, res, "sigmoid", group)
        want = ref.norm_backward(r_out.double().cpu().numpy(), *args, w["dr_out"], w["dy"])
        for name, a, b, k in zip(("dr", "do", "dz", "dw_post", "dls", "dw_pre"), got, want, (res, kind, kind, "f32", "f32", "f32")):
            check(a, b, k, name)


@pytest.mark.parametrize("kind,res,D,T", [("bf16", "bf16", 512, 9001), ("bf16", "f32", 512, 9001), ("f32", "f32", 1024, 5001), ("bf16", "bf16", 2048, 2501),
                                          ("f16", "f32", 2048, 2501), ("bf16", "f32", 4096, 1301), ("bf16", "bf16", 8192, 901), ("f32", "f32", 8192, 701),
                                          ("bf16", "bf16", 12288, 601), ("f32", "f32", 12288, 601)])
@pytest.mark.parametrize("gate,r", [("sigmoid", False), ("none", True)], ids=["gated norm alone", "last residual"])
def test_whole_row_norm_without_the_next_norm(kind, res, D, T, gate, r):
    """w_pre absent: the sum of the norm after the block is the only one of a row and its barrier the only one.  Every CTA works
    many rows, one after the other: no row may be normed with sums of the next, and the same call gives the same bits."""
    import torch
    d, w = _draw(T, D, kind, res, gate, ls=r, r=r, pre=False)
    first, y = _forward(d, T, D, kind, res, gate, 0)
    assert y is None
    check(first, ref.norm_forward(w["r"], w["o"], w["z"], gate, 0, w["w_post"], 0.7, w["ls"], None, EPS)[0], res, "r_out")
    for _ in range(5):
        again, _ = _forward(d, T, D, kind, res, gate, 0)
        assert torch.equal(first.view(torch.uint8), again.view(torch.uint8))


def _steps(D):
    """Rows that keep every CTA of the widest launch (four CTAs of 256 threads an SM up to 2048 channels, two of 512 up to 4096,
    one above) at work for three steps and a bit."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    threads = 4
    while threads * 8 < D:
        threads *= 2
    per = 4 * max(1, 256 // threads) if D <= 2048 else 2 if D <= 4096 else 1
    return 3 * sms * per + 5


@pytest.mark.parametrize("how", [dict(), dict(pre=False), dict(r=False, pre=False), dict(post=False), dict(ls=False, r=False), dict(o=False, gate="none")], ids=str)
@pytest.mark.parametrize("D,group", [(96, 32), (300, 0), (301, 0), (384, 128), (1001, 0), (1024, 256), (2048, 0), (2048, 128), (2050, 0), (4096, 0), (4096, 128),
                                     (4098, 0), (4099, 0), (6144, 0), (6144, 128), (6146, 0), (8192, 256), (12288, 0), (12288, 128), (12289, 0)])
def test_many_rows_a_cta(D, group, how):
    """Slots of the ring are filled again, the buffers of the row sums alternate, weights are read again for every row."""
    pairs = (("bf16", "f32"), ("f32", "f32")) if how in (dict(), dict(pre=False)) else (("f16", "f16"),)
    for kind, res in pairs:
        _check_all(_steps(D), D, kind, res, group=group, **how)
