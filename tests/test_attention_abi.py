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
    unsupported = [dict(d=48, rot=16), dict(d=512, rot=16), dict(rot=80), dict(rot=8), dict(rot=24),
                   dict(H=2 ** 25, ldq=2 ** 40, ldq_out=2 ** 40, ldgq=2 ** 40, lddq=2 ** 40)]
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


WINDOW = "plan plan_dev H Hk d type q ldq k ldk v ldv scale window sinks".split()


def test_heads_of_a_row_that_32_bits_still_count(kda):  # noqa: F811
    """One head fewer than refused goes on to the next check (an output that is not there)."""
    names = "T H Hk d type q ldq k ldk norm w_q w_k eps positions phases rot pairs q_out ldq_out k_out ldk_out stream".split()
    good = dict(T=4, H=2 ** 25 - 1, Hk=0, d=64, type=BF16, q=F, ldq=2 ** 40, k=None, ldk=0, norm=0, w_q=None, w_k=None, eps=0.0, positions=None, phases=None,
                rot=0, pairs=0, q_out=None, ldq_out=2 ** 40, k_out=None, ldk_out=0, stream=None)
    assert kda._lib.kda_head_norm_rotary_forward(*(good[n] for n in names)) == kda.KDA_ERR_INVALID_ARG


def _window_good(kda):  # noqa: F811
    plan = kda.kda_plan_segments([0, 300, 333], 1)
    return plan, dict(plan=plan.ctypes.data_as(ctypes.c_void_p), plan_dev=F, H=8, Hk=2, d=64, type=BF16, q=F, ldq=512, k=F, ldk=128, v=F, ldv=128,
                      scale=0.125, window=100, sinks=4, stream=None)


WINDOW_BAD = [dict(plan=None), dict(plan_dev=None), dict(H=0), dict(Hk=0), dict(Hk=3), dict(d=0), dict(type=5), dict(q=None), dict(q=F + 8),
              dict(ldq=511), dict(ldq=516), dict(k=None), dict(k=F + 2), dict(ldk=120), dict(ldk=132), dict(v=None), dict(v=F + 4), dict(ldv=64),
              dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-39), dict(window=0),
              dict(window=-5), dict(sinks=-1)]
WINDOW_UNSUPPORTED = [dict(type=F32), dict(d=32), dict(d=256, ldq=2048, ldk=512, ldv=512), dict(d=96, ldq=768, ldk=192, ldv=192), dict(sinks=129),
                      dict(H=2 ** 25, Hk=1, ldq=2 ** 38), dict(ldq=2 ** 39), dict(ldk=2 ** 39), dict(ldv=2 ** 40)]


def test_window_forward_refusals(kda):  # noqa: F811
    plan, good = _window_good(kda)
    names = WINDOW + "o ldo lse stream".split()
    good.update(o=F, ldo=512, lse=F)
    _refusals(kda._lib.kda_window_attention_forward, names, good,
              WINDOW_BAD + [dict(o=None), dict(o=F + 8), dict(ldo=504), dict(ldo=514), dict(lse=F + 2)], kda.KDA_ERR_INVALID_ARG)
    _refusals(kda._lib.kda_window_attention_forward, names, good, WINDOW_UNSUPPORTED, kda.KDA_ERR_UNSUPPORTED)


def test_window_forward_refuses_more_tokens_than_its_rows_count(kda):  # noqa: F811
    """A plan that long has too many chunk records to be built here; its header alone would not pass the plan's check."""
    plan, good = _window_good(kda)
    bad = plan.copy()
    bad[3] = 2 ** 31 - 100
    good.update(o=F, ldo=512, lse=None, plan=bad.ctypes.data_as(ctypes.c_void_p))
    names = WINDOW + "o ldo lse stream".split()
    assert kda._lib.kda_window_attention_forward(*(good[n] for n in names)) == kda.KDA_ERR_INVALID_ARG


def test_window_step_refusals(kda):  # noqa: F811
    names = "B H Hk d type slots num_slots lengths q ldq k ldk v ldv scale window sinks ck cv o ldo stream".split()
    _, good = _window_good(kda)
    good.update(B=3, slots=F, num_slots=7, lengths=F, ck=F, cv=F, o=F, ldo=512)
    bad = [x for x in WINDOW_BAD if not set(x) & {"plan", "plan_dev"}]
    bad += [dict(B=-1), dict(num_slots=-1), dict(slots=F + 2), dict(slots=None, num_slots=2), dict(lengths=None), dict(lengths=F + 1), dict(ck=None),
            dict(ck=F + 8), dict(cv=None), dict(cv=F + 8), dict(o=None), dict(o=F + 8), dict(ldo=511), dict(window=2 ** 31 - 1, sinks=1), dict(window=2 ** 31 - 512, sinks=0)]
    step = kda._lib.kda_window_attention_step
    _refusals(step, names, good, bad, kda.KDA_ERR_INVALID_ARG)
    _refusals(step, names, good, WINDOW_UNSUPPORTED[:-4] + [dict(H=2 ** 25, Hk=1, ldq=2 ** 38, ldo=2 ** 38), dict(B=2 ** 30, num_slots=2 ** 30)], kda.KDA_ERR_UNSUPPORTED)
    _refusals(step, names, good, [dict(B=0), dict(B=0, q=None, lengths=None)], kda.KDA_OK)


def test_window_fill_refusals(kda):  # noqa: F811
    names = "plan plan_dev Hk d type slots num_slots k ldk v ldv window sinks ck cv stream".split()
    _, good = _window_good(kda)
    good.update(slots=F, num_slots=2, ck=F, cv=F)
    bad = [x for x in WINDOW_BAD if not set(x) & {"H", "q", "ldq", "scale"} and x != dict(Hk=3)]
    bad += [dict(num_slots=-1), dict(slots=F + 2), dict(slots=None, num_slots=1), dict(ck=None), dict(ck=F + 8), dict(cv=None), dict(cv=F + 8),
            dict(window=2 ** 31 - 1, sinks=1)]
    _refusals(kda._lib.kda_window_cache_fill, names, good, bad, kda.KDA_ERR_INVALID_ARG)
    _refusals(kda._lib.kda_window_cache_fill, names, good, [dict(type=F32), dict(d=32), dict(sinks=129)], kda.KDA_ERR_UNSUPPORTED)


def test_window_backward_refusals(kda):  # noqa: F811
    plan, good = _window_good(kda)
    names = WINDOW + "o ldo lse do lddo dq lddq dk lddk dv lddv ws ws_bytes stream".split()
    need = kda.kda_window_attention_workspace_bytes(plan, 8, 2, 64, 100, 4)
    good.update(o=F, ldo=512, lse=F, do=F, lddo=512, dq=F, lddq=512, dk=F, lddk=128, dv=F, lddv=128, ws=F, ws_bytes=need)
    bad = WINDOW_BAD + [dict(lse=None), dict(lse=F + 1), dict(ws=None), dict(ws=F + 8)]
    for n, ld in (("o", "ldo"), ("do", "lddo"), ("dq", "lddq"), ("dk", "lddk"), ("dv", "lddv")):
        bad += [{n: None}, {n: F + 8}, {ld: good[ld] - 8}, {ld: good[ld] + 4}]
    fn = kda._lib.kda_window_attention_backward
    _refusals(fn, names, good, bad, kda.KDA_ERR_INVALID_ARG)
    _refusals(fn, names, good, WINDOW_UNSUPPORTED[:-4] + WINDOW_UNSUPPORTED[-3:] + [dict(lddo=2 ** 39)], kda.KDA_ERR_UNSUPPORTED)
    _refusals(fn, names, good, [dict(ws_bytes=need - 1)], kda.KDA_ERR_WORKSPACE)
    size = lambda *a: kda.kda_window_attention_workspace_bytes(plan, *a)
    assert size(8, 3, 64, 100, 4) == size(8, 2, 32, 100, 4) == size(8, 2, 64, 0, 4) == size(8, 2, 64, 100, 129) == 0
    assert size(8, 2, 64, 333, 4) < need      # no sink leaves a window of that length
