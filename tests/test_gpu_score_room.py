"""Scores in arrays with room for more pages than any request has, up to the most."""

import pytest
import torch

from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_pages import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("room", [63, 49152, 2 ** 31 - 512, 2 ** 31 - 511, 2 ** 31 - 1])
def test_room_changes_no_score(room):
    s = Setup([1000], [1], 4, 1, 64)
    b = torch.zeros(s.blocks, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    api.sv_bound_pages(s.kv, b)
    want = torch.zeros(1, 1, 62, device="cuda")
    api.sv_score_pages(s.kv, s.batch, s.q, b, want)
    out = torch.empty(1, 1, room, device="cuda")
    out[..., :70] = 7.0
    api.sv_score_pages(s.kv, s.batch, s.q, b, out, s.status)
    assert s.status.item() == 0
    assert torch.equal(out[..., :62], want) and (out[0, 0, 62:70] == 7).all()
