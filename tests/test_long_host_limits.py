"""Host-side checks of the calls that read less of a long cache, at the ends of their
arguments' ranges (no GPU needed)."""

import ctypes

import pytest

from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import build
from test_long_host import A, INV, OUT, batch, kv

ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.lib()


@pytest.mark.parametrize("groups", [-1, -2 ** 31])
def test_no_workspace_for_a_negative_number_of_groups(lib, groups):
    shared = N.SvSharedPrefix(groups, A, A)
    for b in (batch(), batch(n_req=0), batch(n_req=0, total_rows=0)):
        assert lib.sv_prefix_attend_workspace(ref(b), ref(kv()), ref(shared), 8) == 0
        assert lib.sv_prefix_attend(ref(kv()), ref(b), ref(shared), A, 8, 0.1, OUT, A, 1 << 40, None, None) == INV
    none = N.SvSharedPrefix(0, A, A)  # an empty batch has no groups
    assert lib.sv_prefix_attend(ref(kv()), ref(batch(n_req=0)), ref(none), A, 8, 0.1, OUT, A, 0, None, None) == N.SV_OK
