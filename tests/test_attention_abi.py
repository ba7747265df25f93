"""Host-side refusals of the attention layer's operators (no GPU needed): a rejected call returns before it touches the
device, so the addresses here are never used."""
import ctypes

import numpy as np
import pytest

from test_ops_abi import BF16, F, F16, F32, _refusals, kda  # noqa: F401  (kda: the fixture)


def test_head_norm_rotary_refusals(kda):  # noqa: F811
    lib = kda._lib
    shared = "T H Hk d type q ldq k ldk norm w_q w_k eps positions phases rot pairs".split()
    names = shared + "q_out ldq_out k_out ldk_out stream".split()
    good = dict(T=4, H=8, Hk=2, d=64, type=BF16, q=F, ldq=512, k=F, ldk=128, norm=1, w_q=F, w_k=F, eps=1e-6, positions=F, phases=F, rot=64,
                pairs=0, q_out=F, ldq_out=512, k_out=F, ldk_out=128, stream=None)
    common = [dict(T=-1), dict(H=0), dict(Hk=-1), dict(d=0), dict(type=3), dict(norm=2), dict(pairs=2), dict(pairs=-1), dict(rot=-16),
              dict(eps=-1.0), dict(eps=float("nan")), dict(norm=0), dict(w_q=F + 2), dict(w_k=F + 1), dict(positions=None),
              dict(positions=F + 2), dict(phases=None), dict(phases=F + 4), dict(q=None), dict(q=F + 1), dict(ldq=511), dict(k=None),
              dict(k=F + 1), dict(ldk=127), dict(Hk=0)]
    unsupported = [dict(d=48, rot=16), dict(d=512, rot=16), dict(rot=80), dict(rot=8), dict(rot=24)]
    _refusals(lib.kda_head_norm_rotary_forward, names, good,
              common + [dict(q_out=None), dict(q_out=F + 1), dict(ldq_out=511), dict(k_out=None), dict(ldk_out=5),
                        dict(Hk=0, k=None, w_k=None), dict(Hk=0, k=None, k_out=None)], kda.KDA_ERR_INVALID_ARG)
    _refusals(lib.kda_head_norm_rotary_forward, names, good, unsupported, kda.KDA_ERR_UNSUPPORTED)
    _refusals(lib.kda_head_norm_rotary_forward, names, good, [dict(T=0), dict(T=0, q=None, positions=None)], kda.KDA_OK)
    need = kda.kda_head_norm_rotary_workspace_bytes(64)
    names_b = shared + "gq ldgq gk ldgk dq lddq dk lddk dw_q dw_k ws ws_bytes stream".split()
    good_b = dict(good, gq=F, ldgq=512, gk=F, ldgk=128, dq=F, lddq=512, dk=F, lddk=128, dw_q=F, dw_k=F, ws=F, ws_bytes=need)
    _refusals(lib.kda_head_norm_rotary_backward, names_b, good_b,
              common + [dict(gq=None), dict(ldgq=1), dict(gk=None), dict(ldgk=1), dict(dq=None), dict(dq=F + 1), dict(lddq=1), dict(dk=None),
                        dict(lddk=1), dict(dw_q=F + 1), dict(dw_k=F + 2), dict(w_q=None), dict(w_k=None), dict(ws=None), dict(ws=F + 8)],
              kda.KDA_ERR_INVALID_ARG)
    _refusals(lib.kda_head_norm_rotary_backward, names_b, good_b, unsupported, kda.KDA_ERR_UNSUPPORTED)
    _refusals(lib.kda_head_norm_rotary_backward, names_b, good_b, [dict(ws_bytes=need - 1)], kda.KDA_ERR_WORKSPACE)
    assert kda.kda_head_norm_rotary_workspace_bytes(96) == 0


def test_rotary_phases(kda):  # noqa: F811
    f = np.array([np.pi, 0.0, -np.pi / 2, 2 * np.pi])
    got = kda.kda_rotary_phases(f).view(np.uint64)
    for word, turn in zip(got.tolist(), (0.5, 0.0, 0.75, 0.0)):
        gap = abs(word / 2 ** 64 - turn)
        assert min(gap, 1 - gap) < 1e-15
    for bad in (np.nan, np.inf):
        with pytest.raises(kda.KDAError):
            kda.kda_rotary_phases([1.0, bad])
    assert kda._lib.kda_rotary_phases(None, 3, None) == kda.KDA_ERR_INVALID_ARG
    assert kda._lib.kda_rotary_phases(ctypes.c_void_p(0), 0, None) == kda.KDA_OK


def test_binding_refuses_heads_that_do_not_fit(kda):  # noqa: F811
    import torch
    q, k = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64)
    with pytest.raises(kda.KDAError) as e:      # CPU tensors
        kda.kda_head_norm_rotary_forward(q, k, True, None, None, 1e-6, None, None, "halves", q, k, 0)
    assert e.value.status == kda.KDA_ERR_INVALID_ARG
    with pytest.raises(kda.KDAError):
        kda.kda_head_norm_rotary_forward(q[:, 0], None, True, None, None, 1e-6, None, None, "halves", q, None, 0)
