"""The lists that sv_page_attend builds: every warp's entries are in them, however
the warps of a CTA fall apart."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_pages import Setup, attended, check_attend, listed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_lists_of_crowded_sms():
    # 1600 lists, many CTAs an SM, entries in all eight warps of each, two streams at
    # once: an entry left out would take a page away from its row.  Every call gives the
    # same bits, and they are right.
    rng = np.random.default_rng(6)
    n = 400
    s = Setup(rng.integers(0, 700, n).tolist(), rng.integers(1, 9, n).tolist(), 4, 4, 64, seed=6)
    pages = torch.from_numpy(s.lists(40)).cuda()
    first = attended(s, pages)
    streams = [torch.cuda.Stream() for _ in range(2)]
    size = api.sv_page_attend_workspace(s.batch, s.kv, s.H, 40)
    ws = [api.workspace(size).fill_(255) for _ in streams]
    outs = [[torch.full_like(s.q, 7.0) for _ in range(40)] for _ in streams]
    torch.cuda.synchronize()
    for k in range(40):
        for stream, w, out in zip(streams, ws, outs):
            with torch.cuda.stream(stream):
                attended(s, pages, w, out[k])
    torch.cuda.synchronize()
    assert s.status.item() == 0
    for out in outs:
        for y in out:
            assert torch.equal(y.view(torch.int16), first.view(torch.int16))
    check_attend(s, first, listed(s, pages.cpu().numpy()))
