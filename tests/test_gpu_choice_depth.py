"""The pages a draft row attends beside those it would attend with its path committed,
decoded alone under the same choice: the same while the path completes no page, and
from then on those and the pages that the path completed."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_pages import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def chosen(s, kv, batch, q, keep, first, last):
    bounds = torch.zeros(s.blocks, s.K, 2, s.D, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(q.shape[0], s.K, s.np_tables.shape[1], device="cuda")
    pages = torch.zeros(q.shape[0], s.K, keep, dtype=torch.int32, device="cuda")
    api.sv_bound_pages(kv, bounds, None, s.status)
    api.sv_score_pages(kv, batch, q, bounds, scores, s.status)
    api.sv_select_pages(kv, batch, scores, pages, first, last, s.status)
    return pages.cpu().numpy()


@pytest.mark.parametrize("keep,first,last", [(8, 1, 4), (6, 0, 1), (9, 2, 0), (200, 1, 2)])
@pytest.mark.parametrize("tree", [False, True])
def test_a_row_and_the_same_row_alone(keep, first, last, tree):
    ctx, rows = 60 * 16 + 11, 60
    s = Setup([ctx], [rows], 4, 2, 64, tree=tree, seed=keep)
    drafted = chosen(s, s.kv, s.batch, s.q, keep, first, last)
    exact = more = 0
    for r in range(rows):
        path = []
        j = r
        while s.np_parent[j] >= 0:
            j = int(s.np_parent[j])
            path.append(j)
        depth = len(path)
        # the path committed: its keys behind the context, then the row itself
        k = s.k.clone()
        slot = lambda n: (int(s.np_tables[0, n // 16]), n % 16)  # noqa: E731
        for at, j in enumerate(reversed(path)):
            (b, o), (c, p) = slot(ctx + at), slot(ctx + j)
            k[b, :, o] = s.k[c, :, p]
        kv = api.PagedKV(k, s.v, s.kv.block_tables, s.i32([ctx + depth]))
        one = api.Batch(s.i32([0, 1]), s.i32([-1]), s.i32([0]), 1)
        alone = chosen(s, kv, one, s.q[r:r + 1], keep, first, last)
        done = (ctx % 16 + depth) // 16  # pages that the path completed
        for g in range(s.K):
            a, d = set(alone[0, g]) - {-1}, set(drafted[r, g]) - {-1}
            if done == 0:
                exact += 1
                assert np.array_equal(alone[0, g], drafted[r, g])
            else:
                more += 1
                d |= set(range(ctx // 16, ctx // 16 + done))
                assert a <= d and len(d) - len(a) <= done
                assert keep > 60 or len(d) == keep + done
    assert exact > 0 and (more > 0 or tree)
    assert s.status.item() == 0
