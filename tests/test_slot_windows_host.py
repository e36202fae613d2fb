"""What sv_slot_windows refuses on the host (no GPU)."""

import ctypes

import pytest
import torch

from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import api

A = 4096  # stands for a device pointer: nothing is enqueued before it is refused
BAD, SHAPE = N.SV_ERR_INVALID_ARGUMENT, N.SV_ERR_UNSUPPORTED_SHAPE


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_padding_gb300 import build
    build.build()
    return N.lib()


def test_slot_windows_refuses(lib):
    def call(kv=(A, A, 10, 16, 2, 64, A, 4, A), b=(2, 6, 4, A, A, A, None, None, None), slots=A, row_end=A):
        ref = lambda t, x: None if x is None else ctypes.byref(t(*x))  # noqa: E731
        return lib.sv_slot_windows(ref(N.SvPagedKV, kv), ref(N.SvBatch, b), slots, row_end, None)

    assert call(kv=None) == call(b=None) == call(slots=None) == call(row_end=None) == BAD
    assert call(kv=(A, A, -1, 16, 2, 64, A, 4, A)) == BAD
    assert call(kv=(A, A, 10, 32, 2, 64, A, 4, A)) == SHAPE
    assert call(b=(-1, 6, 4, A, A, A, None, None, None)) == call(b=(2, -1, 4, A, A, A, None, None, None)) == BAD
    assert call(b=(2, 6, 0, A, A, A, None, None, None)) == call(b=(2, 6, 4, None, A, A, None, None, None)) == BAD
    assert call(b=(2, 6, 129, A, A, A, None, None, None)) == SHAPE
    assert call(b=(0, 0, 4, None, None, None, None, None, None), slots=None, row_end=None) == N.SV_OK


def test_binding_refuses_short_and_wrong_tensors():
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    page = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    kv = api.PagedKV(page, page, i(1, 2), i(1))
    b = api.Batch(i(3), i(5), i(5), 3)
    for slots, row_end in ((i(4), i(2)), (i(5), i(1)), (i(5).long(), i(2)), (i(5), i(2).float()), (i(5), i(2))):
        with pytest.raises(N.SpecVerifyError):
            api.bind_slot_windows(kv, b, slots, row_end)
