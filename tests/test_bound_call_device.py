"""A bound call is launched on its tensors' device, so it refuses another one
that is current (no GPU: the current device is faked)."""

import pytest
import torch

from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import api, build


def test_bound_call_refuses_another_current_device(monkeypatch):
    build.build()
    current, calls = [0], []
    monkeypatch.setattr(api, "_current_device", lambda: current[0])
    monkeypatch.setattr(api, "_current_stream", lambda index: 100 + index)
    call = api.BoundCall("sv_chunk_windows", (None, 0, 2, None, None, None), torch.device("cuda", 0))
    call._f = lambda *a: calls.append(a[-1]) or N.SV_OK
    call()
    call(stream=7)
    assert calls == [100, 7]
    current[0] = 1
    for stream in (None, 7):
        with pytest.raises(N.SpecVerifyError, match="bound to cuda:0, the current device is cuda:1"):
            call(stream)
    assert calls == [100, 7]
