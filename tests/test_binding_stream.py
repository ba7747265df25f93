"""How the binding finds the stream of a call (no GPU needed)."""
import ctypes
import types

import pytest


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__
    __graft_entry__._load_build_module().build()
    from context_kda_gb300 import binding
    return binding


def test_the_current_stream_is_torchs_public_one(kda, monkeypatch):
    """Without a stream a call takes what torch.cuda.current_stream() says, whatever stands behind it."""
    import torch
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: types.SimpleNamespace(cuda_stream=4711))
    value = kda._stream(None)
    assert isinstance(value, ctypes.c_void_p) and value.value == 4711


def test_a_given_stream_is_taken(kda):
    assert kda._stream(815).value == 815
    assert kda._stream(types.SimpleNamespace(cuda_stream=816)).value == 816
