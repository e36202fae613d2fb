"""Page choice and shared prefixes at the largest sizes they take, at offsets past 32
bits, and several calls at once."""

import numpy as np
import pytest
import torch

from oracle import pages as plain
from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_pages import Setup, attended, check_attend, check_scores, f64, listed
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_lists_of_1024_pages_for_128_rows():
    s = Setup([5000 * 16 + 3], [128], 1, 1, 64, tree=True)
    pages = torch.from_numpy(s.lists(1024)).cuda()
    got = attended(s, pages)
    assert s.status.item() == 0
    # the sums have 16384 weights: 16384 * 2^-23 of the magnitudes instead of 5000 * 2^-23,
    # 1.4e-3 more (of averages of |v|, which stay below 4.1)
    check_attend(s, got, listed(s, pages.cpu().numpy()), slack=1.4e-3 * 4.1)


def test_attention_of_many_requests():
    # more of them than threads that look for a tile's request at once
    rng = np.random.default_rng(3)
    n = 700
    s = Setup(rng.integers(0, 60, n).tolist(), rng.integers(1, 4, n).tolist(), 2, 1, 64)
    pages = torch.from_numpy(s.lists(2)).cuda()
    check_attend(s, attended(s, pages), listed(s, pages.cpu().numpy()))
    assert s.status.item() == 0


def _lengths_only(n_pages, rows=1):
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    kv = api.PagedKV(k, k.clone(), torch.zeros(1, n_pages + 1, dtype=torch.int32, device="cuda"), i32([n_pages * 16 + 5]))
    parent = list(range(-1, rows - 1))
    return kv, api.Batch(i32([0, rows]), i32(parent), i32([0] * rows), rows)


@pytest.mark.parametrize("keep", [1, 700, 1024])
@pytest.mark.parametrize("values", ["random", "few", "far"])
def test_selection_of_49152_pages(keep, values):
    kv, batch = _lengths_only(49152, rows=2)
    g = torch.Generator("cuda").manual_seed(keep)
    x = torch.randn(2, 1, 49152, generator=g, device="cuda")
    if values == "few":
        x = x.round()
    if values == "far":  # a narrow range far from zero: neighbours in fp32
        x = 1e6 + x.round() / 16
    out = torch.full((2, 1, keep), 7, dtype=torch.int32, device="cuda")
    first, last = (0, 0) if keep == 1 else (2, 3)
    api.sv_select_pages(kv, batch, x, out, first, last)
    for r in range(2):
        assert np.array_equal(out[r, 0].cpu().numpy(), plain.select(x[r, 0].cpu().numpy(), 49152, keep, first, last))


def test_bounds_of_8192_requests():
    n = 8192
    g = torch.Generator("cuda").manual_seed(0)
    k = torch.randn(n, 1, 16, 64, generator=g, device="cuda").bfloat16()
    ids = torch.randperm(n, generator=torch.Generator().manual_seed(0)).int().cuda()
    lens = torch.randint(0, 40, (n,), generator=g, device="cuda", dtype=torch.int32).clamp_(max=31)
    kv = api.PagedKV(k, k, ids[:, None].contiguous(), lens.clamp(max=16))
    b = torch.full((n, 1, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sv_bound_pages(kv, b, None, status)
    want = torch.full_like(b, 7.0)
    full = ids[kv.cache_lens == 16].long()
    want[full] = torch.stack([k[full].amin(2), k[full].amax(2)], 2)
    assert torch.equal(b, want) and status.item() == 0


def test_scores_of_65528_lists():
    n = 8191
    g = torch.Generator("cuda").manual_seed(1)
    bnd = torch.randn(n, 8, 2, 64, generator=g, device="cuda").sort(dim=2).values.bfloat16()
    k = torch.zeros(n, 8, 16, 64, dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: a.to(torch.int32).cuda().contiguous()  # noqa: E731
    kv = api.PagedKV(k, k, i32(torch.arange(n)[:, None]), i32(torch.full((n,), 16)))
    batch = api.Batch(i32(torch.arange(n + 1)), i32(torch.full((n,), -1)), i32(torch.zeros(n)), 1)
    q = torch.randn(n, 8, 64, generator=g, device="cuda").bfloat16()
    out = torch.full((n, 8, 1), 7.0, device="cuda")
    api.sv_score_pages(kv, batch, q, bnd, out)
    x = torch.maximum(q.double() * bnd[:, :, 0].double(), q.double() * bnd[:, :, 1].double())
    # 2 D exact products added one by one in fp32
    assert ((out[:, :, 0].double() - x.sum(2)).abs() <= 128 * 2.0 ** -23 * x.abs().sum(2)).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 11, 16])
@pytest.mark.parametrize("room", [30000, 60000])  # pages a CTA: 256, 512
def test_scores_of_large_calls(group, dim, room):
    ctx, rows = [9000, 40, 4200, 500], [2, 3, 1, 19]
    s = Setup(ctx, rows, 2 * group, 2, dim, seed=group)
    b = torch.empty(s.blocks, 2, 2, dim, dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    api.sv_bound_pages(s.kv, b)
    check_scores(s, b, torch.full((25, 2, room), 7.0, device="cuda"), ctx, dim)


def test_offsets_past_32_bits():
    # a cache of 2.3e9 elements: the same requests at its far end give the same bits
    near = Setup([900, 333], [5, 9], 16, 8, 128, seed=4)
    blocks = 140000
    shift = blocks - near.blocks
    far_k = torch.zeros(blocks, 8, 16, 128, dtype=torch.bfloat16, device="cuda")
    far_v = torch.zeros_like(far_k)
    far_k[shift:], far_v[shift:] = near.k, near.v
    tables = torch.where(near.kv.block_tables >= 0, near.kv.block_tables + shift, -1).int()
    kv = api.PagedKV(far_k, far_v, tables, near.kv.cache_lens)
    pages = torch.from_numpy(near.lists(20)).cuda()
    shared = api.SharedPrefix(near.i32([0, 1, 2]), near.i32([320, 160]))
    results = []
    for c in (near.kv, kv):
        b = torch.zeros(c.k_cache.shape[0], 8, 2, 128, dtype=torch.bfloat16, device="cuda")
        api.sv_bound_pages(c, b, None, near.status)
        scores = torch.zeros(14, 8, 60, device="cuda")
        api.sv_score_pages(c, near.batch, near.q, b, scores, near.status)
        ws = api.workspace(max(api.sv_page_attend_workspace(near.batch, c, 16, 20),
                               api.sv_prefix_attend_workspace(near.batch, c, shared, 16)))
        x, y = torch.zeros_like(near.q), torch.zeros_like(near.q)
        api.sv_page_attend(c, near.batch, near.q, near.scale, pages, x, ws, near.status)
        api.sv_prefix_attend(c, near.batch, shared, near.q, near.scale, y, ws, near.status)
        results.append((b[-near.blocks:], scores, x, y))
    assert near.status.item() == 0
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    check_attend(near, results[1][2], listed(near, pages.cpu().numpy()))


def test_scores_past_32_bits():
    # 6144 rows of 8 heads by 49152 pages: the last rows' scores lie past 2^31 elements
    rows = [128] * 48
    s = Setup([40] * 47 + [700], rows, 8, 8, 64)
    s.window(begin=[128] * 47 + [125], end=[128] * 48)
    b = torch.zeros(s.blocks, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
    api.sv_bound_pages(s.kv, b)
    scores = torch.empty(6144, 8, 49152, device="cuda")
    scores[-3:].fill_(7.0)
    pages = torch.full((6144, 8, 9), 7, dtype=torch.int32, device="cuda")
    api.sv_score_pages(s.kv, s.batch, s.q, b, scores, s.status)
    api.sv_select_pages(s.kv, s.batch, scores, pages, 1, 2, s.status)
    assert s.status.item() == 0
    bnd, q = f64(b), f64(s.q[-3:])
    got = scores[-3:].cpu().double().numpy()
    for r in range(3):
        want, mag = plain.scores(q[r], bnd, s.np_tables[47], 43)
        assert (np.abs(got[r, :, :43] - want) <= 128 * 2.0 ** -23 * mag).all() and (got[r, :, 43:] == 7).all()
        for g in range(8):
            assert np.array_equal(pages[6141 + r, g].cpu().numpy(), plain.select(got[r, g], 43, 9, 1, 2))
    assert (pages[:6141] == 7).all()


def test_calls_at_once_on_three_streams():
    # each with a workspace of its own; the same bits as one after the other
    a = Setup([3000, 90, 777], [9, 5, 3], 8, 2, 128, seed=1)
    pages = torch.from_numpy(a.lists(30)).cuda()
    b = Shared([(1024, [30, 5, 9]), (96, [5])], [40, 50, 10, 20], 8, 2, 64, seed=2)
    c = Setup([2000, 900], [64, 40], 8, 1, 128, tree=True, seed=3)  # tiles of tensor cores here too
    wa = api.workspace(api.sv_page_attend_workspace(a.batch, a.kv, a.H, 30))
    wb = api.workspace(api.sv_prefix_attend_workspace(b.batch, b.kv, b.shared, b.H))
    wc = api.workspace(api.sv_tree_attend_workspace(c.batch, c.kv, c.H))
    calls = [lambda out: api.sv_page_attend(a.kv, a.batch, a.q, a.scale, pages, out, wa, a.status),
             lambda out: api.sv_prefix_attend(b.kv, b.batch, b.shared, b.q, b.scale, out, wb, b.status),
             lambda out: api.sv_tree_attend(c.kv, c.batch, c.q, c.H, c.scale, out, wc, c.status)]
    alone = [torch.zeros_like(x.q) for x in (a, b, c)]
    for call, out in zip(calls, alone):
        call(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.zeros_like(x.q) for _ in range(20)] for x in (a, b, c)]
    torch.cuda.synchronize()
    for k in range(20):
        for call, stream, out in zip(calls, streams, outs):
            with torch.cuda.stream(stream):
                call(out[k])
    torch.cuda.synchronize()
    for x, want, got in zip((a, b, c), alone, outs):
        assert x.status.item() == 0
        for y in got:
            assert torch.equal(y.view(torch.int16), want.view(torch.int16))
    check_attend(a, alone[0], listed(a, pages.cpu().numpy()))
    b.check(alone[1])
