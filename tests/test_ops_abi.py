"""Host-side refusals of the operators around the KDA layer (no GPU needed): a rejected call returns before
it touches the device, so the addresses here are never used."""
import ctypes

import numpy as np
import pytest

F = 1 << 20          # an aligned address that is never dereferenced
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__
    __graft_entry__._load_build_module().build()
    from context_kda_gb300 import binding
    return binding


def _refusals(fn, names, good, bad, want):
    """Every change in 'bad' of the good arguments is answered with 'want'."""
    for change in bad:
        args = dict(good, **change)
        assert fn(*(args[n] for n in names)) == want, change


def test_gated_scan_refusals(kda):
    lib = kda._lib
    plan = kda.kda_plan_segments([0, 300], 1)
    pp = plan.ctypes.data_as(ctypes.c_void_p)
    need = kda.kda_gated_scan_workspace_bytes(plan, 64)
    names = "plan plan_dev D type x ldx i ldi g ldg h0 h ldh final states ws ws_bytes stream".split()
    good = dict(plan=pp, plan_dev=F, D=64, type=BF16, x=F, ldx=64, i=F, ldi=64, g=F, ldg=64, h0=F, h=F, ldh=64, final=F, states=F,
                ws=F, ws_bytes=need, stream=None)
    common = [dict(plan=None), dict(plan_dev=None), dict(D=0), dict(D=-3), dict(type=3), dict(type=-1), dict(x=None),
              dict(x=F + 1), dict(ldx=63), dict(i=F + 1), dict(ldi=63), dict(g=None), dict(g=F + 2), dict(ldg=0), dict(h0=F + 2)]
    _refusals(lib.kda_gated_scan_forward, names, good, common + [dict(h=None), dict(h=F + 1), dict(ldh=1), dict(final=F + 1),
                                                                 dict(states=F + 2)], kda.KDA_ERR_INVALID_ARG)
    _refusals(lib.kda_gated_scan_forward, names, dict(good, type=F32), [dict(x=F + 2), dict(h=F + 2)], kda.KDA_ERR_INVALID_ARG)
    names_b = ("plan plan_dev D type x ldx i ldi g ldg h0 states dh lddh dfinal dx lddx di lddi dg lddg dh0 ws ws_bytes "
               "stream").split()
    good_b = dict(good, dh=F, lddh=64, dfinal=F, dx=F, lddx=64, di=F, lddi=64, dg=F, lddg=64, dh0=F)
    _refusals(lib.kda_gated_scan_backward, names_b, good_b,
              common + [dict(states=None), dict(dh=None), dict(lddh=5), dict(dfinal=F + 1), dict(dx=None), dict(lddx=0),
                        dict(di=F + 1), dict(dg=None), dict(dg=F + 2), dict(lddg=63), dict(dh0=F + 2), dict(i=None)],
              kda.KDA_ERR_INVALID_ARG)
    if need:
        for fn, n, a in ((lib.kda_gated_scan_forward, names, good), (lib.kda_gated_scan_backward, names_b, good_b)):
            _refusals(fn, n, a, [dict(ws_bytes=need - 1)], kda.KDA_ERR_WORKSPACE)
            _refusals(fn, n, a, [dict(ws=None), dict(ws=F + 8)], kda.KDA_ERR_INVALID_ARG)
    assert kda.kda_gated_scan_workspace_bytes(plan, 0) == 0
    bad = plan.copy()
    bad[5] = 9
    assert kda.kda_gated_scan_workspace_bytes(bad, 64) == 0


def test_gated_scan_step_refusals(kda):
    names = "B D type slots num_slots x ldx i ldi g ldg state h ldh stream".split()
    good = dict(B=4, D=64, type=F16, slots=F, num_slots=9, x=F, ldx=64, i=F, ldi=64, g=F, ldg=64, state=F, h=F, ldh=64, stream=None)
    _refusals(kda._lib.kda_gated_scan_step, names, good,
              [dict(B=-1), dict(D=0), dict(type=7), dict(slots=F + 2), dict(num_slots=-1), dict(slots=None, num_slots=3),
               dict(x=None), dict(ldx=2), dict(i=F + 1), dict(g=None), dict(state=None), dict(state=F + 1), dict(h=None), dict(ldh=0)],
              kda.KDA_ERR_INVALID_ARG)
    _refusals(kda._lib.kda_gated_scan_step, names, good, [dict(B=0), dict(B=0, x=None, state=None)], kda.KDA_OK)


def test_block_norm_refusals(kda):
    lib = kda._lib
    names = ("T D res_type type r ldr o ldo z ldz gate group w_post scale ls w_pre eps r_out ldr_out y ldy stream").split()
    good = dict(T=4, D=256, res_type=BF16, type=BF16, r=F, ldr=256, o=F, ldo=256, z=F, ldz=256, gate=1, group=128, w_post=F,
                scale=1.0, ls=F, w_pre=F, eps=1e-6, r_out=F, ldr_out=256, y=F, ldy=256, stream=None)
    common = [dict(T=-1), dict(D=0), dict(res_type=3), dict(type=-1), dict(gate=0), dict(gate=3), dict(z=None), dict(ldz=1),
              dict(o=F + 1), dict(ldo=255), dict(w_post=F + 2), dict(ls=F + 1), dict(w_pre=F + 2), dict(eps=-1.0),
              dict(eps=float("nan")), dict(o=None)]
    unsupported = [dict(res_type=F16), dict(type=F16), dict(type=F32), dict(D=16385, group=0, ldr=16385, ldo=16385, ldz=16385),
                   dict(group=96), dict(group=512), dict(D=320, group=128), dict(group=-128), dict(group=16)]
    _refusals(lib.kda_block_norm_forward, names, good,
              common + [dict(r=F + 1), dict(ldr=3), dict(r_out=F + 1), dict(ldr_out=9), dict(y=None), dict(w_pre=None),
                        dict(ldy=9), dict(y=F + 1), dict(r=None, o=None, z=None, gate=0, w_post=None, ls=None),
                        dict(y=None, w_pre=None, r_out=None)], kda.KDA_ERR_INVALID_ARG)
    _refusals(lib.kda_block_norm_forward, names, good, unsupported, kda.KDA_ERR_UNSUPPORTED)
    _refusals(lib.kda_block_norm_forward, names, good, [dict(T=0)], kda.KDA_OK)
    names_b = ("T D res_type type r ldr o ldo z ldz gate group w_post scale ls w_pre eps dr_out lddr_out dy lddy dr lddr d_o lddo "
               "dz lddz dw_post dls dw_pre ws ws_bytes stream").split()
    need = kda.kda_block_norm_workspace_bytes(256)
    good_b = dict(good, dr_out=F, lddr_out=256, dy=F, lddy=256, dr=F, lddr=256, d_o=F, lddo=256, dz=F, lddz=256, dw_post=F, dls=F,
                  dw_pre=F, ws=F, ws_bytes=need)
    _refusals(lib.kda_block_norm_backward, names_b, good_b,
              common + [dict(r=None), dict(dy=None), dict(dr_out=F + 1), dict(lddr_out=2), dict(lddy=2), dict(d_o=None),
                        dict(lddo=2), dict(dr=F + 1), dict(lddr=2), dict(dz=F + 1), dict(dw_post=F + 1), dict(dls=F + 1),
                        dict(dw_pre=F + 1), dict(w_post=None), dict(ls=None), dict(w_pre=None), dict(ws=None), dict(ws=F + 4)],
              kda.KDA_ERR_INVALID_ARG)
    _refusals(lib.kda_block_norm_backward, names_b, good_b, unsupported, kda.KDA_ERR_UNSUPPORTED)
    _refusals(lib.kda_block_norm_backward, names_b, good_b, [dict(ws_bytes=need - 1)], kda.KDA_ERR_WORKSPACE)
    assert kda.kda_block_norm_workspace_bytes(0) == 0 and kda.kda_block_norm_workspace_bytes(16385) == 0


def test_decode_refusals(kda):
    names = "B H type slots num_slots q ldq k ldk v ldv g ldg beta ldb scale state o ldo stream".split()
    good = dict(B=2, H=3, type=BF16, slots=F, num_slots=4, q=F, ldq=384, k=F, ldk=384, v=F, ldv=384, g=F, ldg=384, beta=F, ldb=3,
                scale=1.0, state=F, o=F, ldo=384, stream=None)
    bad = [dict(B=-1), dict(H=0), dict(type=4), dict(slots=F + 1), dict(num_slots=-1), dict(slots=None, num_slots=1),
           dict(state=None), dict(state=F + 8), dict(ldb=2), dict(ldg=383)]
    for n in ("q", "k", "v", "g", "beta", "o"):
        bad += [{n: None}, {n: F + 1}]
    for n in ("ldq", "ldk", "ldv", "ldo"):
        bad.append({n: 383})
    _refusals(kda._lib.kda_decode_step, names, good, bad, kda.KDA_ERR_INVALID_ARG)
    _refusals(kda._lib.kda_decode_step, names, good, [dict(H=65536, ldq=1 << 24, ldk=1 << 24, ldv=1 << 24, ldg=1 << 24, ldb=1 << 17, ldo=1 << 24)],
              kda.KDA_ERR_UNSUPPORTED)
    _refusals(kda._lib.kda_decode_step, names, good, [dict(B=0)], kda.KDA_OK)


def test_binding_refuses_tensors_that_do_not_fit(kda):
    """Shapes, types and strides the C side cannot see; CPU tensors are refused too."""
    import torch
    plan = kda.kda_plan_segments([0, 8], 1)
    x, g = torch.zeros(8, 4), torch.zeros(8, 4)
    with pytest.raises(kda.KDAError) as e:
        kda.kda_gated_scan_forward(plan, g, x, None, g, None, x.clone(), None, None, None, 0)
    assert e.value.status == kda.KDA_ERR_INVALID_ARG
    with pytest.raises(kda.KDAError):
        kda.kda_block_norm_forward(x, None, None, "tanh", 0, None, 1.0, None, g[0], 1e-6, None, x.clone(), 0)
    with pytest.raises(kda.KDAError):
        kda.kda_decode_step(None, torch.zeros(1, 2, 128), torch.zeros(1, 2, 128), torch.zeros(1, 2, 128), torch.zeros(1, 2, 128),
                            torch.zeros(1, 2), 1.0, torch.zeros(1, 2, 128, 128), torch.zeros(1, 2, 128), 0)


def test_gated_scan_refuses_more_channels_than_its_indexes_hold(kda):
    lib, most = kda._lib, 2 ** 31 - 512
    for D in (most + 1, 2 ** 31 - 1):
        for cu in ([0, 1], [0, 3000]):
            plan = kda.kda_plan_segments(cu, 1)
            pp = plan.ctypes.data_as(ctypes.c_void_p)
            assert kda.kda_gated_scan_workspace_bytes(plan, D) == 0
            assert lib.kda_gated_scan_forward(pp, F, D, BF16, F, D, F, D, F, D, F, F, D, F, F, F, 1 << 62, None) == kda.KDA_ERR_UNSUPPORTED
            assert lib.kda_gated_scan_backward(pp, F, D, BF16, F, D, F, D, F, D, F, F, F, D, F, F, D, F, D, F, D, F, F, 1 << 62,
                                               None) == kda.KDA_ERR_UNSUPPORTED
        assert lib.kda_gated_scan_step(1, D, BF16, F, 4, F, D, F, D, F, D, F, F, D, None) == kda.KDA_ERR_UNSUPPORTED
    plan = kda.kda_plan_segments([0, 3000], 1)
    tiles, states = 24, 4                                        # one state every 8 tiles, one more
    assert kda.kda_gated_scan_workspace_bytes(plan, most) >= (tiles * 8 + states * 4) * most
