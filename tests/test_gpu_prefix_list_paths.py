"""sv_prefix_attend at sizes where prefixes are read by lists of their own, along the
paths a served batch takes: graphs, several streams, offsets past 32 bits, whole steps.
Each test first sees to it that the call has such lists (the call's header, at the
start of its workspace, counts their stages)."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_prefix import Shared
from test_gpu_prefix_lists import check, own

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def workspace(s):
    return api.workspace(api.sv_prefix_attend_workspace(s.batch, s.kv, s.shared, s.H)).fill_(255)


def list_stages(ws):
    return int(ws[:20].view(torch.int32)[3])


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("dim", [64, 128])
def test_many_short_lists_a_cta(dim):
    # several lists of two stages a CTA, so that the barriers of a list are set up anew
    # at once: the same bits in every call
    rng = np.random.default_rng(dim)
    s = Shared([(144, own(rng, 600)), (256, own(rng, 600))], [4] * 1200, 32, 8, dim, seed=dim)
    ws = workspace(s)
    got = s.run(ws=ws)
    assert list_stages(ws) > 0
    check(s, got)
    for _ in range(40):
        assert torch.equal(bits(s.run(ws=ws)), bits(got))
    assert s.status.item() == 0
