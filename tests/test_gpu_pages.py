"""Page bounds, scores, selection and attention over selected pages, against the
plain 64-bit forms, at the sizes and masks where they can go wrong."""

import numpy as np
import pytest
import torch

from oracle import pages as plain
from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def f64(t):
    return t.float().cpu().double().numpy()


class Setup:
    """A paged cache and a batch of drafts.  Every slot that no request has written
    holds NaN, in K and V, so that reading one shows."""

    def __init__(self, ctx, rows, heads=8, kv_heads=2, dim=128, tree=False, seed=0, spare=3, shared=0):
        g = torch.Generator("cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.rows, self.H, self.K, self.D = list(ctx), list(rows), heads, kv_heads, dim
        R = len(ctx)
        self.cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        n = [-(-(c + m) // 16) for c, m in zip(ctx, rows)]
        ids = rng.permutation(sum(n) + spare).astype(np.int32)
        self.np_tables = np.full((R, max(n) + 2), -1, dtype=np.int32)
        at = 0
        for i, m in enumerate(n):
            self.np_tables[i, :m] = ids[at:at + m]
            at += m
        if shared:
            self.np_tables[:, :shared] = self.np_tables[0, :shared]
        self.free_block = int(ids[-1])  # no request's
        self.blocks = len(ids)
        shape = (self.blocks, kv_heads, 16, dim)
        self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        for i, (c, m) in enumerate(zip(ctx, rows)):
            s = torch.arange(c + m, device="cuda")
            b = torch.from_numpy(self.np_tables[i]).cuda().long()[s // 16]
            for t in (self.k, self.v):
                t[b, :, s % 16] = torch.randn(c + m, kv_heads, dim, generator=g, device="cuda").bfloat16()
        parent = []
        for m in rows:
            parent += [-1] + [int(rng.integers(0, j)) if tree else j - 1 for j in range(1, m)]
        self.np_parent = np.array(parent, dtype=np.int32)
        i32 = lambda a: torch.tensor(np.asarray(a, dtype=np.int32), device="cuda")  # noqa: E731
        self.i32 = i32
        self.kv = api.PagedKV(self.k, self.v, i32(self.np_tables), i32(ctx))
        self.batch = api.Batch(i32(self.cu), i32(self.np_parent), i32(np.zeros(self.cu[-1])), max(rows))
        self.q = torch.randn(int(self.cu[-1]), heads, dim, generator=g, device="cuda").mul_(1.5).bfloat16()
        self.scale = dim ** -0.5
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.windows = [(0, m) for m in rows]

    def window(self, begin=None, end=None, verify=None):
        for name, v in (("row_begin", begin), ("row_end", end), ("verify_len", verify)):
            if v is not None:
                setattr(self.batch, name, self.i32(v))
        begin = begin or [0] * len(self.rows)
        self.windows = [(b, max(b, min(m if end is None else end[i], m if verify is None else verify[i] + 1)))
                        for i, (b, m) in enumerate(zip(begin, self.rows))]

    def numpy(self):
        return f64(self.k), f64(self.v), f64(self.q)

    def lists(self, keep, seed=1, overlap=0.5):
        """Ascending page lists of their own for every row and head, some short."""
        rng = np.random.default_rng(seed)
        out = np.full((int(self.cu[-1]), self.K, keep), -1, dtype=np.int32)
        for i, c in enumerate(self.ctx):
            n = c // 16
            for r in range(self.cu[i], self.cu[i + 1]):
                for g in range(self.K):
                    m = min(n, keep if rng.random() < 0.7 else int(rng.integers(0, keep + 1)))
                    out[r, g, :m] = np.sort(rng.permutation(n)[:m])
        return out


def attended(s, pages, ws=None, out=None, stream=None):
    if ws is None:
        # a workspace is not initialised: every bit of it set
        ws = api.workspace(api.sv_page_attend_workspace(s.batch, s.kv, s.H, pages.shape[2])).fill_(255)
    out = torch.full_like(s.q, 7.0) if out is None else out
    api.sv_page_attend(s.kv, s.batch, s.q, s.scale, pages, out, ws, s.status, stream)
    return out


def check_attend(s, got, cached, slack=0.0):
    """bf16 rounding of the output (2^-8 of it) and of the weights (2^-8 of each,
    in the sum of w |v|); fp32 scores, sums and exponentials stay below 2^-9 of
    that sum: a score's error is at most D 2^-23 sum |q k| scale < 128 * 2^-23 *
    (1.5 * 128 * 0.64 + tails < 200) * 0.09 < 3e-4, twice that in a weight; sums
    of at most 5000 weights add 5000 * 2^-23 < 6e-4; the exponential 2^-21."""
    k, v, q = s.numpy()
    ref, mag = plain.attend(q, k, v, s.np_tables, s.ctx, s.cu, s.np_parent, s.windows, s.scale, cached)
    got = f64(got)
    inside = ~np.isnan(ref)
    assert (got[~inside] == 7.0).all()  # rows outside the windows stay as they were
    assert np.isfinite(got).all()
    err, tol = np.abs(got - ref)[inside], (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * mag)[inside]
    assert (err <= tol + slack).all(), (err - tol).max()


def listed(s, pages):
    def cached(i, r, g):
        own = [t * 16 + o for t in pages[r, g] if t >= 0 for o in range(16)]
        return own + list(range(s.ctx[i] // 16 * 16, s.ctx[i]))
    return cached


# ----------------------------------------------------------------- bounds --

@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kv_heads", [1, 3, 8])
@pytest.mark.parametrize("ctx", [[0], [15, 16, 17, 1], [333, 0, 64, 1000]])
def test_bounds(dim, kv_heads, ctx):
    s = Setup(ctx, [1] * len(ctx), heads=kv_heads, kv_heads=kv_heads, dim=dim)
    for start in (None, [c // 2 for c in ctx], ctx, [c + 40 for c in ctx]):
        b = torch.full((s.blocks, kv_heads, 2, dim), 5.0, dtype=torch.bfloat16, device="cuda")
        api.sv_bound_pages(s.kv, b, None if start is None else s.i32(start), s.status)
        ref = plain.bounds(f64(s.k), s.np_tables, ctx, start, into=np.full(b.shape, 5.0))
        assert np.array_equal(f64(b), ref)
    assert s.status.item() == 0


def test_bounds_of_infinities_and_zeros():
    s = Setup([32], [1], heads=1, kv_heads=1, dim=64)
    s.k[s.np_tables[0, 0], 0, 3, 5] = float("inf")
    s.k[s.np_tables[0, 0], 0, 4, 6] = -float("inf")
    s.k[s.np_tables[0, 1]] = -0.0
    s.k[s.np_tables[0, 1], 0, 7] = 0.0
    s.k[s.np_tables[0, 1], 0, 9, 11] = float("nan")  # counts for nothing
    b = torch.zeros(s.blocks, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    api.sv_bound_pages(s.kv, b)
    first, second = f64(b)[s.np_tables[0, 0], 0], f64(b)[s.np_tables[0, 1], 0]
    assert first[1, 5] == np.inf and first[0, 6] == -np.inf and np.isfinite(first[0, 5])
    assert (second == 0).all()


def test_bounds_findings():
    s = Setup([100, 64, 48], [2, 2, 2])
    s.kv.cache_lens[1] = -1
    s.kv.block_tables[2, 1] = s.blocks
    b = torch.full((s.blocks, 2, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    api.sv_bound_pages(s.kv, b, None, s.status)
    assert s.status.item() == N.SV_DEV_BAD_LENGTH | N.SV_DEV_BAD_BLOCK_ID
    t = s.np_tables.copy()
    t[2, 1] = -1
    assert np.array_equal(f64(b), plain.bounds(f64(s.k), t, [100, 0, 48], into=np.full(b.shape, 5.0)))
    s.status.zero_()
    s.kv.cache_lens[1] = s.np_tables.shape[1] * 16 + 1  # more than the table
    api.sv_bound_pages(s.kv, b, s.i32([0, 0, 48]), s.status)
    assert s.status.item() == N.SV_DEV_BAD_LENGTH


# ----------------------------------------------------------------- scores --

@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 8, 128), (6, 3, 64), (6, 2, 128), (8, 2, 64), (10, 2, 128),
                                                (14, 2, 64), (8, 1, 128), (9, 1, 64), (32, 2, 128)])
@pytest.mark.parametrize("shape", ["one", "ragged", "tree"])
@pytest.mark.parametrize("wide", [False, True])  # room for many pages: larger parts a CTA
def test_scores(heads, kv_heads, dim, shape, wide):
    ctx, rows = {"one": ([300], [1]), "ragged": ([0, 15, 16, 1300, 257], [3, 2, 9, 1, 20]),
                 "tree": ([200, 90], [70, 33])}[shape]
    s = Setup(ctx, rows, heads, kv_heads, dim, tree=shape == "tree")
    if shape == "ragged":
        s.window(begin=[0, 1, 2, 0, 0], end=[3, 2, 9, 1, 20], verify=[5, 5, 5, 0, 18])
    b = torch.empty(s.blocks, kv_heads, 2, dim, dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    api.sv_bound_pages(s.kv, b)
    pages = 80000 // (len(ctx) * kv_heads) if wide else max(ctx) // 16 + 2
    check_scores(s, b, torch.full((int(s.cu[-1]), kv_heads, pages), 7.0, device="cuda"), ctx, dim)


@pytest.mark.parametrize("heads,kv_heads,dim,rows", [(10, 2, 128, [3, 1, 9]), (8, 2, 64, [1, 40, 2]), (32, 2, 128, [9, 1, 1])])
@pytest.mark.parametrize("ctx", [[8191, 17000, 8208], [40, 2048 * 16 + 3, 0]])
def test_scores_of_long_contexts(heads, kv_heads, dim, rows, ctx):
    # several tiles a CTA and several CTAs a request
    s = Setup(ctx, rows, heads, kv_heads, dim)
    b = torch.empty(s.blocks, kv_heads, 2, dim, dtype=torch.bfloat16, device="cuda").fill_(float("nan"))
    api.sv_bound_pages(s.kv, b)
    check_scores(s, b, torch.full((int(s.cu[-1]), kv_heads, 14001), 7.0, device="cuda"), ctx, dim)


def check_scores(s, b, out, ctx, dim):
    api.sv_score_pages(s.kv, s.batch, s.q, b, out, s.status)
    assert s.status.item() == 0
    bnd, q, got = f64(b), f64(s.q), out.cpu().double().numpy()
    ref = np.full(got.shape, 7.0)
    tol = np.zeros(got.shape)
    for i, (w0, w1) in enumerate(s.windows):
        n = ctx[i] // 16
        for r in range(s.cu[i] + w0, s.cu[i] + w1):
            ref[r, :, :n], mag = plain.scores(q[r], bnd, s.np_tables[i], n)
            # 2 D exact products added one by one in fp32, each sum off by at most 2^-23
            tol[r, :, :n] = 2 * dim * 2.0 ** -23 * mag
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) - tol).max()


def test_scores_bound_every_product():
    s = Setup([500], [4], 8, 2, 128)
    b = torch.zeros(s.blocks, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    api.sv_bound_pages(s.kv, b)
    out = torch.zeros(4, 2, 31, device="cuda")
    api.sv_score_pages(s.kv, s.batch, s.q, b, out)
    k = s.k[torch.from_numpy(s.np_tables[0, :31]).cuda().long()].double()  # [31][2][16][128]
    x = torch.einsum("rghd,tgsd->rghts", s.q.double().view(4, 2, 4, 128), k)
    assert (x.amax((2, 4)) <= out.double() + 1e-3).all()


@pytest.mark.parametrize("wide", [False, True])
def test_scores_findings(wide):
    s = Setup([100, 64, 48], [2, 2, 2])
    b = torch.ones(s.blocks, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full((6, 2, 4), 7.0, device="cuda")
    if wide:  # a length above the room of many pages
        s.kv.cache_lens[0] = 15000 * 16
        s.kv.block_tables = torch.nn.functional.pad(s.kv.block_tables, (0, 15010 - s.kv.block_tables.shape[1]), value=-1)
        out = torch.full((6, 2, 14000), 7.0, device="cuda")
    s.kv.block_tables[2, 1] = -1
    api.sv_score_pages(s.kv, s.batch, s.q, b, out, s.status)  # request 0 has 6 pages, room for 4
    assert s.status.item() == N.SV_DEV_BAD_LENGTH | N.SV_DEV_BAD_BLOCK_ID
    got = out.cpu().numpy()
    assert (got[:2] == 7).all() and (got[4:, :, 1] == 0).all() and (got[4:, :, 3:] == 7).all()
    s.status.zero_()
    s.batch.row_begin, s.batch.row_end = s.i32([0, 2, 0]), s.i32([0, 1, 0])
    api.sv_score_pages(s.kv, s.batch, s.q, b, out, s.status)
    assert s.status.item() == N.SV_DEV_BAD_WINDOW | N.SV_DEV_BAD_LENGTH  # request 0 is as long as it was


# -------------------------------------------------------------- selection --

def _selected(s, x, keep, first, last):
    out = torch.full((x.shape[0], x.shape[1], keep), 7, dtype=torch.int32, device="cuda")
    api.sv_select_pages(s.kv, s.batch, x, out, first, last, s.status)
    ref = np.full(out.shape, 7, dtype=np.int32)
    v = x.cpu().numpy()
    for i, (b, e) in enumerate(s.windows):
        for r in range(s.cu[i] + b, s.cu[i] + e):
            for g in range(x.shape[1]):
                ref[r, g] = plain.select(v[r, g], s.ctx[i] // 16, keep, first, last)
    assert np.array_equal(out.cpu().numpy(), ref)
    return out


@pytest.mark.parametrize("keep,first,last", [(1, 0, 0), (1, 1, 0), (2, 1, 1), (7, 1, 4), (64, 2, 5), (300, 0, 300),
                                             (1024, 3, 4)])
@pytest.mark.parametrize("values", ["random", "ties", "equal", "odd"])
def test_selection(keep, first, last, values):
    ctx = [0, 16, 7 * 16 + 3, 64 * 16 - 1, 1100 * 16 + 5, 5000 * 16]
    s = Setup([0] * 6, [1, 2, 3, 1, 2, 2], heads=2, kv_heads=2, dim=64)
    s.ctx = ctx  # only lengths and the tables' width are read
    s.kv = api.PagedKV(s.k, s.v, torch.zeros(6, 5000, dtype=torch.int32, device="cuda"), s.i32(ctx))
    g = torch.Generator("cuda").manual_seed(keep)
    x = torch.randn(int(s.cu[-1]), 2, 5003, generator=g, device="cuda")
    if values == "ties":
        x = (x * 2).round() / 2
    elif values == "equal":
        x = torch.full_like(x, -1.5)
    elif values == "odd":
        pick = torch.randint(0, 9, x.shape, generator=g, device="cuda")
        for k, v in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 3.4e38)):
            x[pick == k] = v
    _selected(s, x, keep, first, last)
    assert s.status.item() == 0


def test_selection_in_windows_and_findings():
    s = Setup([400, 300, 200], [4, 5, 6], heads=2, kv_heads=2, dim=64, tree=False)
    s.window(begin=[1, 0, 2], end=[4, 5, 6], verify=[9, 2, 9])
    x = torch.randn(15, 2, 25, device="cuda")
    _selected(s, x, 8, 1, 2)
    assert s.status.item() == 0
    s.kv.cache_lens[0] = 26 * 16
    s.ctx[0] = 0  # skipped
    s.windows[0] = (0, 0)
    _selected(s, x, 8, 1, 2)
    assert s.status.item() == N.SV_DEV_BAD_LENGTH


# -------------------------------------------------------------- attention --

@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 128), (4, 2, 64), (6, 2, 128), (8, 2, 64), (10, 2, 128),
                                                (14, 2, 64), (8, 1, 128), (16, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("shape", ["one", "ragged", "tree"])
def test_page_attention(heads, kv_heads, dim, shape):
    ctx, rows, keep = {"one": ([1000], [1], 9), "ragged": ([0, 15, 16, 700, 257, 33], [3, 2, 9, 1, 20, 1], 6),
                       "tree": ([200, 330], [70, 33], 5)}[shape]
    s = Setup(ctx, rows, heads, kv_heads, dim, tree=shape == "tree", seed=heads)
    pages = s.lists(keep)
    got = attended(s, s.i32(pages))
    assert s.status.item() == 0
    check_attend(s, got, listed(s, pages))


@pytest.mark.parametrize("dim", [64, 128])
def test_page_attention_reads_no_other_page(dim):
    # pages that no row of a request lists hold NaN
    s = Setup([640, 333], [5, 3], 8, 2, dim, seed=3)
    pages = np.full((8, 2, 4), -1, dtype=np.int32)
    pages[:5, :, :3] = [2, 11, 30]
    pages[5:, :, :2] = [0, 19]
    for i, used in ((0, [2, 11, 30]), (1, [0, 19])):
        for t in range(s.ctx[i] // 16):
            if t not in used:
                s.k[s.np_tables[i, t]] = s.v[s.np_tables[i, t]] = float("nan")
    got = attended(s, s.i32(pages))
    check_attend(s, got, listed(s, pages))


@pytest.mark.parametrize("keep", [0, 1, 64])
def test_page_attention_with_all_or_no_pages(keep):
    s = Setup([1000, 5, 160], [4, 4, 1], 8, 2, 128, seed=4)
    pages = np.full((9, 2, keep), -1, dtype=np.int32)
    if keep == 64:
        for i in range(3):
            pages[s.cu[i]:s.cu[i + 1], :, :s.ctx[i] // 16] = np.arange(s.ctx[i] // 16)
    got = attended(s, s.i32(pages))
    check_attend(s, got, listed(s, pages))
    if keep == 64:  # the whole context: what sv_tree_attend gives
        whole = torch.full_like(s.q, 7.0)
        ws = api.workspace(api.sv_tree_attend_workspace(s.batch, s.kv, s.H))
        api.sv_tree_attend(s.kv, s.batch, s.q, s.H, s.scale, whole, ws, s.status)
        check_attend(s, whole, lambda i, r, g: range(s.ctx[i]))
    assert s.status.item() == 0


def test_page_attention_in_windows():
    s = Setup([400, 300, 200, 100, 77], [4, 30, 6, 8, 9], 8, 2, 128)
    s.window(begin=[1, 0, 2, 3, 5], end=[4, 25, 2, 8, 9], verify=[9, 22, 9, 5, 3])  # the last begins behind its rows
    pages = s.lists(6)
    got = attended(s, s.i32(pages))
    assert s.status.item() == 0
    check_attend(s, got, listed(s, pages))


def test_page_attention_findings():
    s = Setup([400, 300, 200, 160, 90], [3, 3, 3, 3, 3], 8, 2, 128)
    pages = s.lists(6)
    pages[:] = np.arange(6)
    pages[1, 0] = [3, 5, 5, 7, 8, 9]     # does not ascend: ends behind 5
    pages[3, 1] = [0, 1, 18, 4, 5, 6]    # 18 is request 1's partly filled page: ends behind 1
    pages[4, 0] = [-2, 1, 2, 3, 4, 5]    # ends at once
    pages[12:, :, 5] = -1
    given = s.i32(pages)
    s.kv.block_tables[2, 3] = s.blocks + 5  # a listed page outside the cache
    s.batch.parent[10] = 2                  # request 3
    got = attended(s, given)
    assert s.status.item() == N.SV_DEV_BAD_PARAM | N.SV_DEV_BAD_BLOCK_ID | N.SV_DEV_BAD_PARENT
    pages[1, 0, 2:] = pages[3, 1, 2:] = pages[4, 0] = -1
    pages[6:9, :, 3] = -1  # left out
    s.windows[3] = (0, 0)
    check_attend(s, got, listed(s, pages))
    s.status.zero_()
    s.kv.cache_lens[4] = s.np_tables.shape[1] * 16 - 2
    attended(s, given)
    assert s.status.item() & N.SV_DEV_BAD_LENGTH


def test_page_attention_of_many_tiles():
    # more lists than CTAs, shares that end inside them, empty requests between
    rng = np.random.default_rng(0)
    rows = rng.integers(1, 12, 150).tolist()
    ctx = rng.integers(0, 300, 150).tolist()
    s = Setup(ctx, rows, 16, 4, 64, seed=5)
    s.window(end=[m if k % 5 else 0 for k, m in enumerate(rows)])
    pages = s.lists(7)
    given = s.i32(pages)
    got = attended(s, given)
    assert s.status.item() == 0
    check_attend(s, got, listed(s, pages))
    for _ in range(3):  # the same bits each time
        assert torch.equal(attended(s, given).view(torch.int16), got.view(torch.int16))


def test_page_calls_in_a_graph_and_on_another_stream():
    s = Setup([800, 333, 90], [4, 5, 1], 8, 2, 128)
    b = torch.zeros(s.blocks, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(10, 2, 52, device="cuda")
    pages = torch.zeros(10, 2, 9, dtype=torch.int32, device="cuda")
    out = torch.full_like(s.q, 7.0)
    ws = api.workspace(api.sv_page_attend_workspace(s.batch, s.kv, 8, 9))
    calls = [api.bind_bound_pages(s.kv, b, None, s.status), api.bind_score_pages(s.kv, s.batch, s.q, b, x, s.status),
             api.bind_select_pages(s.kv, s.batch, x, pages, 1, 2, s.status),
             api.bind_page_attend(s.kv, s.batch, s.q, s.scale, pages, out, ws, s.status)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for c in calls:
            c()
    torch.cuda.current_stream().wait_stream(stream)
    first = (x.clone(), pages.clone(), out.clone())
    check_attend(s, out, listed(s, pages.cpu().numpy()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for t in (b, x, pages):
        t.zero_()
    out.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(first, (x, pages, out)):
        assert torch.equal(a, c)
    # other queries, the same graph
    s.q.copy_(s.q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    check_attend(s, out, listed(s, pages.cpu().numpy()))
    assert s.status.item() == 0
