"""Scores of pages whose keys hold infinities, by the formula of the header: a term is
max(q lo, q hi), 0 where q is 0; a head whose sum is no number counts for nothing."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_pages import Setup, f64

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def formula(q, bnd):
    """q [heads][dim], bnd [kv heads][2][dim] -> scores and sums of magnitudes [kv heads]."""
    group = q.shape[0] // bnd.shape[0]
    q = q.reshape(bnd.shape[0], group, -1)
    with np.errstate(invalid="ignore"):
        term = np.where(q == 0, 0.0, np.maximum(q * bnd[:, None, 0], q * bnd[:, None, 1]))
        total = term.sum(2)
    best = np.where(np.isnan(total), -np.inf, total).max(1)
    return np.where(np.isnan(total).all(1), np.nan, best), np.abs(np.where(np.isfinite(term), term, 0)).sum(2).max(1)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 64), (4, 2, 128), (10, 2, 128), (14, 2, 64), (16, 1, 128)])
@pytest.mark.parametrize("room", [64, 60000])  # pages a CTA: few, many
def test_scores_of_infinite_keys(heads, kv_heads, dim, room):
    ctx, rows = [700, 90, 1000], [5, 1, 19]
    s = Setup(ctx, rows, heads, kv_heads, dim, seed=heads)
    rng = np.random.default_rng(heads)
    s.q.masked_fill_(torch.rand(s.q.shape, generator=torch.Generator("cuda").manual_seed(3), device="cuda") < 0.2, 0.0)
    # of every third page one key, and of some every key, of a dimension or two
    for i, c in enumerate(ctx):
        for t in range(0, c // 16, 3):
            b, g = int(s.np_tables[i, t]), int(rng.integers(kv_heads))
            for x in (INF, -INF)[:int(rng.integers(1, 3))]:
                s.k[b, g, int(rng.integers(16)), int(rng.integers(dim))] = x
            if t % 2 == 0:
                s.k[b, g, :, int(rng.integers(dim))] = float(rng.choice([INF, -INF]))
    bounds = torch.zeros(s.blocks, kv_heads, 2, dim, dtype=torch.bfloat16, device="cuda")
    api.sv_bound_pages(s.kv, bounds)
    out = torch.full((25, kv_heads, room), 7.0, device="cuda")
    api.sv_score_pages(s.kv, s.batch, s.q, bounds, out, s.status)
    assert s.status.item() == 0
    bnd, q, got = f64(bounds), f64(s.q), out.cpu().double().numpy()
    seen = {"nan": 0, "inf": 0, "-inf": 0}
    for i, (c, m) in enumerate(zip(ctx, rows)):
        n = c // 16
        for r in range(s.cu[i], s.cu[i] + m):
            assert (got[r, :, n:] == 7).all()
            for t in range(n):
                want, mag = formula(q[r], bnd[s.np_tables[i, t]])
                for g in range(kv_heads):
                    x, y = got[r, g, t], want[g]
                    if np.isfinite(y):  # 2 D exact products added one by one in fp32
                        assert abs(x - y) <= 2 * dim * 2.0 ** -23 * mag[g], (r, g, t, x, y)
                    else:
                        seen[str(y)] += 1
                        assert np.isnan(x) if np.isnan(y) else x == y, (r, g, t, x, y)
    assert seen["inf"] > 0 and (heads > kv_heads or seen["-inf"] > 0)  # (a maximum of many hides -inf)


def test_a_page_of_infinite_keys_is_kept():
    # its bound is the greatest: selection keeps the page that holds it
    s = Setup([640], [3], 4, 1, 64)
    s.q.abs_()
    s.k[s.np_tables[0, 21], 0, 5, 9] = INF
    s.k[s.np_tables[0, 21], 0, 6, 10] = -INF
    bounds = torch.zeros(s.blocks, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(3, 1, 40, device="cuda")
    pages = torch.zeros(3, 1, 4, dtype=torch.int32, device="cuda")
    api.sv_bound_pages(s.kv, bounds)
    api.sv_score_pages(s.kv, s.batch, s.q, bounds, scores)
    api.sv_select_pages(s.kv, s.batch, scores, pages, 1, 1)
    assert (scores[:, 0, 21] == INF).all() and (pages == 21).any(2).all()


def test_bounds_that_are_no_numbers_rank_last():
    # a dimension whose keys are all NaN: no number is known, and no head has one
    s = Setup([320], [2], 4, 2, 128)
    s.k[s.np_tables[0, 7], 1, :, 100] = float("nan")
    bounds = torch.zeros(s.blocks, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(2, 2, 20, device="cuda")
    api.sv_bound_pages(s.kv, bounds)
    api.sv_score_pages(s.kv, s.batch, s.q, bounds, scores)
    assert torch.isnan(scores[:, 1, 7]).all() and torch.isnan(scores).sum() == 2
