"""Shared prefixes at sizes where a call reads them by lists of their own (many
requests, few rows each) and where it mixes these with requests that do not, against
64-bit attention on the GPU."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import build
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def check(s, got, missing=()):
    """missing: pages that are left out of the request's context, (request, page).
    Tolerance as check_attend's: 2^-8 of the output, 2^-8 + 2^-9 of the weighted
    magnitudes."""
    missing = set(missing)
    want = torch.full_like(got, 7.0).double()
    tol = torch.zeros_like(want)
    for i, (c, (b, e)) in enumerate(zip(s.ctx, s.windows)):
        if e <= b:
            continue
        m, r0 = s.rows[i], int(s.cu[i])
        t = torch.arange(c + m, device="cuda")
        block = torch.from_numpy(s.np_tables[i]).cuda().long()[t // 16]
        k, v = s.k[block, :, t % 16].double(), s.v[block, :, t % 16].double()  # [T][K][D]
        see = torch.ones(m, c + m, dtype=torch.bool)
        see[:, c:] = False
        for j in range(m):
            a = j
            while a >= 0:
                see[j, c + a] = True
                a = int(s.np_parent[r0 + a])
        for p in range(-(-c // 16)):
            if (i, p) in missing:
                see[:, 16 * p:16 * p + 16] = False
        see = see[b:e].cuda()
        q = s.q[r0 + b:r0 + e].double().view(e - b, s.K, -1, s.D)
        x = torch.einsum("rkgd,tkd->rkgt", q, k) * s.scale
        w = x.masked_fill(~see[:, None, None], -torch.inf).softmax(-1)
        out = torch.einsum("rkgt,tkd->rkgd", w, v).reshape(e - b, s.H, s.D)
        mag = torch.einsum("rkgt,tkd->rkgd", w, v.abs()).reshape(e - b, s.H, s.D)
        want[r0 + b:r0 + e] = out
        tol[r0 + b:r0 + e] = 2.0 ** -8 * out.abs() + (2.0 ** -8 + 2.0 ** -9) * mag
    assert torch.isfinite(got).all()
    err = (got.double() - want).abs()
    assert (err <= tol).all(), (err - tol).max().item()


def own(rng, n, top=30):
    return rng.integers(0, top, n).tolist()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 16])
@pytest.mark.parametrize("tree", [False, True])
def test_lists_of_head_groups(group, dim, tree):
    rng = np.random.default_rng(group)
    groups = [(320, own(rng, 70)), (0, own(rng, 5)), (16, own(rng, 3)), (1168, own(rng, 40)), (400, own(rng, 1))]
    s = Shared(groups, rng.integers(1, 4, 119).tolist(), 8 * group, 8, dim, tree=tree, seed=group)
    check(s, s.run())
    assert s.status.item() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("pages", [1, 7, 8, 9, 15, 16, 17, 24, 63, 130])
def test_list_lengths_around_a_stage(pages, dim):
    rng = np.random.default_rng(pages)
    s = Shared([(16 * pages, own(rng, 120)), (16 * pages + 16, own(rng, 20))], [1] * 140, 16, 8, dim, seed=pages)
    check(s, s.run())
    assert s.status.item() == 0


@pytest.mark.parametrize("n", [126, 127, 128, 129, 255, 256, 257, 384, 385])
def test_list_rows_around_a_tile(n):
    s = Shared([(160, [4] * n)], [1] * n, 8, 8, 64, seed=n)
    check(s, s.run())
    assert s.status.item() == 0


def test_lists_in_windows():
    rng = np.random.default_rng(5)
    rows = rng.integers(1, 6, 150).tolist()
    s = Shared([(256, own(rng, 100)), (640, own(rng, 50))], rows, 16, 8, 128)
    begin = [int(rng.integers(0, m + 1)) if rng.random() < 0.4 else 0 for m in rows]
    end = [int(rng.integers(b, m + 1)) for b, m in zip(begin, rows)]
    s.window(begin=begin, end=end, verify=rng.integers(0, 7, 150).tolist())
    check(s, s.run())
    assert s.status.item() == 0


@pytest.mark.parametrize("at", [0, 7, 8, 24, 25])
def test_list_page_outside_the_cache(at):
    rng = np.random.default_rng(at)
    s = Shared([(416, own(rng, 130)), (240, own(rng, 10))], [2] * 140, 16, 8, 64, seed=at)
    s.kv.block_tables[0, at] = -1
    got = s.run()
    assert s.status.item() == N.SV_DEV_BAD_BLOCK_ID
    check(s, got, [(i, at) for i in range(130)])


def test_list_findings():
    # requests that are left out, the first of their group among them, whose table is read
    rng = np.random.default_rng(0)
    s = Shared([(304, own(rng, 100)), (512, own(rng, 40)), (80, own(rng, 20))], [2] * 160, 16, 8, 128)
    s.shared.prefix_len[2] = 65
    s.kv.cache_lens[0] = 290
    s.kv.cache_lens[7] = 303
    s.batch.parent[2 * 30] = 1
    got = s.run()
    assert s.status.item() == N.SV_DEV_BAD_PARAM | N.SV_DEV_BAD_LENGTH | N.SV_DEV_BAD_PARENT
    for i in [0, 7, 30] + list(range(140, 160)):
        s.windows[i] = (0, 0)
    check(s, got)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("missing", [None, 124, 7])
def test_shares_of_several_lists(dim, missing):
    # about two lists a CTA: whole lists begin where the one before stopped, so that
    # the last, incomplete stage comes in their midst; other requests that do not share
    s = Shared([(2000, [3] * 30), (1808, [0, 20] * 10), (16, [9] * 3)], [40] * 30 + [38] * 20 + [3] * 3, 32, 8, dim,
               seed=dim)
    if missing is not None:
        s.kv.block_tables[0, missing] = -1
    got = s.run()
    assert s.status.item() == (0 if missing is None else N.SV_DEV_BAD_BLOCK_ID)
    check(s, got, [(i, missing) for i in range(30)])
    assert torch.equal(s.run().view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("dim", [64, 128])
def test_list_maxima_that_grow(dim):
    # keys that grow along the prefix: every stage moves the rows' maxima by more
    # than the rescaling allows to pass
    s = Shared([(1024, [3] * 60)], [2] * 60, 32, 8, dim, seed=2)
    s.q.copy_(s.q.abs())
    for t, b in enumerate(s.np_tables[0, :64]):
        s.k[int(b)] = (0.02 * t + 0.05 * s.k[int(b)].float()).bfloat16()
    check(s, s.run())


def test_lists_of_600_requests_in_300_groups():
    rng = np.random.default_rng(1)
    groups = [(16 * int(rng.integers(0, 40)), own(rng, 2, 60)) for _ in range(300)]
    s = Shared(groups, rng.integers(1, 4, 600).tolist(), 8, 4, 64, seed=1)
    check(s, s.run())
    assert s.status.item() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_a_group_of_both_kinds(dim):
    # one request of many rows reads the prefix with its own pages, the others together
    s = Shared([(320, [5] * 60 + [30] + [0] * 60)], [1] * 60 + [128] + [1] * 60, 64, 8, dim, tree=True)
    check(s, s.run())
    assert s.status.item() == 0
