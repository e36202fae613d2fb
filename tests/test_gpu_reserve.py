"""sv_reserve_kv against the CPU oracle: table entries, free count, slots,
positions and counts equal, findings equal."""

import numpy as np
import pytest
import torch

from oracle import edges
from speculative_decoding_verification_padding_gb300 import api, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Case:
    """Requests with given rows and contexts, tables filled up to the context
    from a shuffled pool, `free` blocks left in it."""

    def __init__(self, rows, ctx, kind="chain", free=None, pad=0, seed=0, width=None, offset=True):
        rng = np.random.default_rng(seed)
        self.rows, self.ctx = np.asarray(rows), np.asarray(ctx, np.int32)
        R = len(rows)
        self.cu = np.zeros(R + 1, np.int32)
        self.cu[1:] = np.cumsum(rows)
        self.total = int(self.cu[-1]) + pad
        self.max_rows = int(max(rows, default=1))
        have, need = -(-self.ctx // 16), -(-(self.ctx + self.rows) // 16)
        new = int((need - have).sum())
        self.free = new + 3 if free is None else free if free >= 0 else max(0, new + free)
        self.blocks = int(have.sum()) + self.free + 2
        ids = rng.permutation(self.blocks).astype(np.int32)
        self.tables = np.full((R, width or int(need.max(initial=1)) + 2), -1, np.int32)
        at = 0
        for i in range(R):
            self.tables[i, :have[i]] = ids[at:at + have[i]]
            at += have[i]
        self.list = np.full(self.free + 5, -1, np.int32)
        self.list[:self.free] = ids[at:at + self.free]
        self.parent = None
        if kind != "prompt":
            up = [-1 if j == 0 else j - 1 if kind == "chain" else int(rng.integers(0, j))
                  for n in rows for j in range(n)]
            self.parent = np.array(up + [7] * pad, np.int32)
        self.offset = rng.integers(-3, 40, R).astype(np.int32) if offset else None

    def run(self, stream=None, times=1):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        dev = dict(tables=_i32(self.tables), count=_i32([self.free]), list=_i32(self.list),
                   ctx=_i32(self.ctx), slots=torch.full((self.total,), -7, dtype=torch.int32, device="cuda"),
                   positions=torch.full((self.total,), -7, dtype=torch.int32, device="cuda"),
                   taken=torch.full((len(self.rows),), -7, dtype=torch.int32, device="cuda"), status=st)
        pages = torch.empty((self.blocks, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
        batch = api.Batch(_i32(self.cu), None if self.parent is None else _i32(self.parent),
                          torch.zeros(self.total, dtype=torch.int32, device="cuda"), self.max_rows)
        self.call = api.bind_reserve_kv(
            api.PagedKV(pages, pages, dev["tables"], dev["ctx"]), batch,
            api.BlockPool(dev["list"], dev["count"]), dev["slots"], dev["positions"], dev["taken"],
            None if self.offset is None else _i32(self.offset), st)
        self.keep = (pages, batch, dev)
        torch.cuda.synchronize()
        for _ in range(times):
            self.call(stream)
        torch.cuda.synchronize()
        return dev

    def check(self, dev, err=0):
        e, ref = edges.reserve(self.cu, self.parent, self.ctx, self.tables, self.list, self.free,
                               self.blocks, self.max_rows, self.total, self.offset)
        assert e == err and dev["status"].item() == err
        for k in ("taken", "slots", "positions", "tables"):
            assert np.array_equal(dev[k].cpu().numpy(), ref[k]), k
        assert dev["count"].item() == ref["count"]
        assert np.array_equal(dev["list"].cpu().numpy(), self.list)  # ids are taken, not erased
        return ref


def _rng_case(R, hi, kind, seed, **kw):
    rng = np.random.default_rng(seed)
    return Case(rng.integers(1, hi + 1, R), rng.integers(0, 400, R), kind, seed=seed, **kw)


@pytest.mark.parametrize("kind", ["chain", "tree", "prompt"])
@pytest.mark.parametrize("R,hi", [(1, 1), (1, 6), (3, 128), (64, 9), (257, 17), (1300, 5), (90, 128)])
def test_matches_oracle(kind, R, hi):
    c = _rng_case(R, hi, kind, seed=R + hi)
    c.check(c.run())


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 17, 31, 32, 4096])
@pytest.mark.parametrize("rows", [1, 2, 16, 17, 128])
def test_page_borders(ctx, rows):
    c = Case([rows, 1, rows], [ctx, 16, ctx + 1], offset=False)
    c.check(c.run())


def test_long_prompts_of_ragged_lengths():
    c = Case([5001, 1, 16, 4097, 33, 12000], [0, 0, 48, 5, 0, 100], "prompt")
    c.check(c.run())


@pytest.mark.parametrize("free", [0, 1, -1, -4])
@pytest.mark.parametrize("R", [5, 700])
def test_short_pool_serves_a_prefix_whole(free, R):
    # contexts that end inside a page leave some requests that need no block:
    # those are served whatever the pool holds
    c = _rng_case(R, 40, "tree", seed=3, free=free)
    ref = c.check(c.run(), err=edges.POOL_EMPTY)
    assert (ref["taken"] == -1).any() and (free in (0, 1) or (ref["taken"] >= 0).any())


def test_exactly_enough_blocks():
    c = _rng_case(40, 30, "chain", seed=4, free=0)
    need = int((-(-(c.ctx + c.rows) // 16) - -(-c.ctx // 16)).sum())
    c = _rng_case(40, 30, "chain", seed=4, free=need)
    assert c.check(c.run())["count"] == 0


@pytest.mark.parametrize("R,hi", [(20, 9), (60, 128)])
def test_a_second_call_takes_nothing_and_answers_the_same(R, hi):
    c = _rng_case(R, hi, "tree", seed=9)
    once, twice = c.run(), c.run(times=2)
    for k in ("tables", "slots", "positions", "count"):
        assert torch.equal(once[k], twice[k]), k
    assert (twice["taken"] == 0).all()


@pytest.mark.parametrize("pad", [1, 50, 5000])
@pytest.mark.parametrize("kind", ["tree", "prompt"])
def test_rows_behind_the_last_request(pad, kind):
    c = _rng_case(9, 60, kind, seed=5, pad=pad)
    dev = c.run()
    c.check(dev)
    assert (dev["slots"][-pad:] == -1).all() and (dev["positions"][-pad:] == -1).all()


@pytest.mark.parametrize("big", [False, True])
def test_malformed_requests_are_left_alone(big):
    rng = np.random.default_rng(6)
    R = 200 if big else 12
    c = Case(rng.integers(20, 40, R), rng.integers(17, 300, R) // 16 * 16 + 3, "tree", seed=6)
    c.parent[c.cu[0]] = 0                      # a root with a parent
    c.parent[c.cu[1] + 5] = 5                  # its own parent
    c.parent[c.cu[2] + 3] = -1
    c.parent[c.cu[3] + 4] = 1 << 30
    c.ctx[4] = -1
    c.ctx[5] = c.tables.shape[1] * 16
    c.tables[6, c.ctx[6] // 16] = -1           # the page in use is missing
    c.tables[7, c.ctx[7] // 16] = c.blocks
    c.tables[8, (c.ctx[8] + c.rows[8] - 1) // 16] = 0  # in use behind new ones
    c.tables[9, c.ctx[9] // 16] = -2
    c.check(c.run(), err=edges.BAD_PARENT | edges.BAD_LENGTH | edges.BAD_BLOCK)


def test_bad_offsets():
    c = Case([3, 4, 9, 6], [10, 20, 30, 40])
    c.cu[2] = 3  # one request of no rows, one of more than the limit
    c.max_rows = 8
    c.check(c.run(), err=edges.BAD_WINDOW)
    c.cu[2] = 99  # one beyond the rows: its neighbours' rows are nobody's
    dev = c.run()
    assert dev["status"].item() == edges.BAD_WINDOW and (dev["taken"][1:3] == -1).all()
    assert (dev["slots"][:3] >= 0).all() and (dev["slots"][3:12] == -1).all()


def test_a_free_list_entry_that_is_no_block():
    c = Case([20, 20], [16, 32])
    c.list[c.free - 2] = c.blocks + 4
    c.check(c.run(), err=edges.BAD_BLOCK)
    c.list[c.free - 3] = -5
    c.check(c.run(), err=edges.BAD_BLOCK)


def test_no_requests_mark_every_row_as_padding():
    c = Case([], [], "prompt", pad=70)
    dev = c.run()
    assert (dev["slots"] == -1).all() and (dev["positions"] == -1).all()


def test_other_stream_and_graph_replay():
    c = _rng_case(30, 40, "tree", seed=11)
    s = torch.cuda.Stream()
    c.check(c.run(stream=s))
    dev = c.keep[2]
    start = {"tables": _i32(c.tables), "count": _i32([c.free])}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for k, v in start.items():
            dev[k].copy_(v)
        c.call()
    for _ in range(2):
        for k in ("slots", "positions", "taken"):
            dev[k].fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        c.check(dev)


def test_reserve_and_commit_conserve_the_pool():
    # everything rejected but the root: commit hands back what reserve took
    # beyond the one committed slot
    c = _rng_case(50, 60, "tree", seed=12)
    dev = c.run()
    pages, batch, _ = c.keep
    R = len(c.rows)
    al = torch.zeros(R, dtype=torch.int32, device="cuda")
    nodes = torch.full((R, c.max_rows), -1, dtype=torch.int32, device="cuda")
    nodes[:, 0] = 0
    kv = api.PagedKV(pages, pages.clone(), dev["tables"], dev["ctx"])
    pool = torch.full((c.blocks,), -1, dtype=torch.int32, device="cuda")
    pool[:c.list.size] = dev["list"]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.sv_commit_kv(kv, batch, al, nodes, api.BlockPool(pool, dev["count"]), st)
    torch.cuda.synchronize()
    assert st.item() == 0
    assert np.array_equal(dev["ctx"].cpu().numpy(), c.ctx + 1)
    tables, n = dev["tables"].cpu().numpy(), dev["count"].item()
    held = tables[tables >= 0].tolist() + pool[:n].cpu().tolist()
    assert len(held) == len(set(held)) == c.blocks - 2
    assert (tables >= 0).sum() == (-(-(c.ctx + 1) // 16)).sum()


def test_faults_found_anywhere_in_a_large_batch():
    # the rows of 300 trees are shared by several CTAs: each finds some faults
    rng = np.random.default_rng(13)
    c = Case(rng.integers(15, 40, 300), rng.integers(0, 300, 300), "tree", seed=13)
    bad = rng.choice(300, 40, replace=False)
    for i in bad:
        j = int(rng.integers(1, c.rows[i]))
        c.parent[c.cu[i] + j] = rng.choice([j, -1, 127, 1 << 20])
    ref = c.check(c.run(), err=edges.BAD_PARENT)
    assert (ref["taken"][bad] == -1).all() and (ref["taken"] >= 0).sum() == 260


def test_more_rows_than_shared_memory_holds():
    rng = np.random.default_rng(14)
    c = Case(rng.integers(120, 129, 1600), rng.integers(0, 100, 1600), "tree", seed=14, pad=77)
    c.parent[c.cu[700] + 9] = 9
    c.check(c.run(), err=edges.BAD_PARENT)
    c = Case([40000, 1, 3001, 29], [0, 31, 7, 0], "prompt", pad=3)
    c.check(c.run())


def test_two_batches_at_once_on_two_streams():
    cases = [_rng_case(200, 30, "tree", seed=20 + k) for k in range(2)]
    for c in cases:
        c.run()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for c, s in zip(cases, streams):
            d = c.keep[2]
            with torch.cuda.stream(s):
                d["tables"].copy_(torch.from_numpy(c.tables), non_blocking=False)
                d["count"].fill_(c.free)
                c.call()
    torch.cuda.synchronize()
    for c in cases:
        c.check(c.keep[2])


def test_without_positions_and_status():
    c = _rng_case(30, 20, "tree", seed=30)
    ref = c.run()
    fresh = c.run()
    d = c.keep[2]
    d["tables"].copy_(_i32(c.tables))
    d["count"].fill_(c.free)
    d["ctx"][3] = -5
    d["positions"].fill_(-3)
    pages, batch, _ = c.keep
    api.sv_reserve_kv(api.PagedKV(pages, pages, d["tables"], d["ctx"]), batch, api.BlockPool(d["list"], d["count"]),
                      d["slots"], None, d["taken"])
    torch.cuda.synchronize()
    assert d["status"].item() == 0 and (d["positions"] == -3).all() and d["taken"][3] == -1
    assert (d["slots"][c.cu[3]:c.cu[4]] == -1).all() and torch.equal(d["slots"][:c.cu[3]], ref["slots"][:c.cu[3]])
    del fresh


@pytest.mark.parametrize("count", [-7, 1 << 30])
def test_a_free_count_outside_the_list(count):
    c = _rng_case(6, 20, "chain", seed=31)
    c.list = np.arange(c.list.size, dtype=np.int32) % c.blocks
    c.free = count
    d = c.run()
    c.free = 0 if count < 0 else c.list.size
    e, ref = edges.reserve(c.cu, c.parent, c.ctx, c.tables, c.list, c.free, c.blocks, c.max_rows, c.total, c.offset)
    assert d["status"].item() == e
    for k in ("taken", "slots", "positions", "tables"):
        assert np.array_equal(d[k].cpu().numpy(), ref[k]), k
    taken = int(ref["taken"][ref["taken"] > 0].sum())
    assert d["count"].item() == (c.free - taken if taken else count)
