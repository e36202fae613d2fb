"""Attention of batches that share prefixes, against the plain 64-bit form."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_pages import Setup, check_attend

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


class Shared(Setup):
    """Groups of requests behind prefixes; the other requests' table entries of
    the prefix name a block of NaN, the plain form gets the first's."""

    def __init__(self, groups, rows, heads=8, kv_heads=2, dim=128, tree=False, seed=0):
        # groups: (prefix, [own lengths])
        ctx = [p + n for p, own in groups for n in own]
        super().__init__(ctx, rows, heads, kv_heads, dim, tree, seed)
        cu, first = [0], []
        for p, own in groups:
            a, b = cu[-1], cu[-1] + len(own)
            cu.append(b)
            if own:
                self.np_tables[a + 1:b, :p // 16] = self.np_tables[a, :p // 16]
            first.append(p)
        given = self.np_tables.copy()
        for (p, _), a, b in zip(groups, cu, cu[1:]):
            given[a + 1:b, :p // 16] = self.free_block
        self.kv.block_tables.copy_(self.i32(given))
        self.shared = api.SharedPrefix(self.i32(cu), self.i32(first))

    def run(self, out=None, ws=None):
        if ws is None:
            ws = api.workspace(api.sv_prefix_attend_workspace(self.batch, self.kv, self.shared, self.H)).fill_(255)
        out = torch.full_like(self.q, 7.0) if out is None else out
        api.sv_prefix_attend(self.kv, self.batch, self.shared, self.q, self.scale, out, ws, self.status)
        return out

    def check(self, got):
        check_attend(self, got, lambda i, r, g: range(self.ctx[i]))


@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 128), (4, 2, 64), (6, 2, 128), (8, 2, 64), (10, 2, 128),
                                                (14, 2, 64), (8, 1, 128), (16, 1, 64), (16, 1, 128)])
@pytest.mark.parametrize("shape", ["one", "page", "ragged", "tree"])
def test_prefix_attention(heads, kv_heads, dim, shape):
    groups, rows = {
        "one": ([(512, [3])], [1]),
        "page": ([(16, [0, 1, 16])], [2, 1, 3]),
        "ragged": ([(144, [0, 15, 200]), (0, [40, 0]), (1040, [7]), (128, [16, 1, 2, 3])],
                   [3, 2, 9, 1, 20, 4, 5, 1, 1, 8]),
        "tree": ([(272, [5, 60]), (400, [0])], [70, 33, 90])}[shape]
    s = Shared(groups, rows, heads, kv_heads, dim, tree=shape == "tree", seed=heads)
    got = s.run()
    assert s.status.item() == 0
    s.check(got)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65])
def test_prefix_rows_around_a_tile(n, dim):
    # n rows of eight heads: a tile is 16 rows, a unit 32
    s = Shared([(160, [4] * n)], [1] * n, 8, 1, dim, seed=n)
    s.check(s.run())
    assert s.status.item() == 0


@pytest.mark.parametrize("pages", [1, 7, 8, 9, 15, 16, 17, 24, 63, 130])
def test_prefix_lengths_around_a_stage(pages):
    s = Shared([(pages * 16, [0, 9]), (pages * 16 + 16, [30])], [3, 2, 6], 4, 1, 128, seed=pages)
    s.check(s.run())
    assert s.status.item() == 0


def test_prefix_in_windows():
    s = Shared([(256, [10, 20, 30]), (64, [5, 6, 7])], [4, 12, 6, 8, 3, 9], 8, 2, 128)
    s.window(begin=[4, 0, 2, 3, 0, 5], end=[4, 11, 6, 8, 3, 9], verify=[9, 7, 9, 5, 0, 3])
    s.check(s.run())
    assert s.status.item() == 0


def test_prefix_findings():
    s = Shared([(256, [10, 20, 30]), (64, [5, 6]), (48, [1])], [4, 12, 6, 8, 3, 2], 8, 2, 128)
    s.shared.prefix_len[1] = 65
    s.kv.cache_lens[1] = 255
    s.batch.parent[16] = 1  # the root of request 2
    got = s.run()
    assert s.status.item() == N.SV_DEV_BAD_PARAM | N.SV_DEV_BAD_LENGTH | N.SV_DEV_BAD_PARENT
    for i in (1, 2, 3, 4):
        s.windows[i] = (0, 0)
    s.check(got)
    for cu in ([0, 3, 5, 5], [1, 3, 5, 6], [0, 4, 3, 6], [0, 3, 7, 6]):  # groups that cut no runs: nothing is done
        s.status.zero_()
        s.shared.cu_groups.copy_(s.i32(cu))
        assert (s.run() == 7).all() and s.status.item() & N.SV_DEV_BAD_PARAM


@pytest.mark.parametrize("at", [0, 5, 15])
def test_prefix_page_outside_the_cache(at):
    # its slots are left out
    s = Shared([(256, [10, 20])], [4, 5], 8, 2, 128, seed=at)
    s.kv.block_tables[0, at] = -1
    got = s.run()
    assert s.status.item() == N.SV_DEV_BAD_BLOCK_ID
    check_attend(s, got, lambda i, r, g: [t for t in range(s.ctx[i]) if t // 16 != at])


def test_prefix_is_tree_attention():
    s = Shared([(640, [50, 3, 0]), (0, [77])], [5, 6, 1, 4], 16, 4, 128)
    whole = torch.full_like(s.q, 7.0)
    s.kv.block_tables.copy_(s.i32(s.np_tables))
    ws = api.workspace(api.sv_tree_attend_workspace(s.batch, s.kv, s.H))
    api.sv_tree_attend(s.kv, s.batch, s.q, s.H, s.scale, whole, ws, s.status)
    s.check(whole)
    s.check(s.run())


def test_prefix_of_many_units_and_the_same_bits():
    # units of unlike lengths, more than SMs; large scores that move the maximum about
    rng = np.random.default_rng(1)
    n = [7, 1, 12, 5]
    groups = [(16 * int(rng.integers(1, 80)), rng.integers(0, 90, k).tolist()) for k in n]
    s = Shared(groups, rng.integers(1, 14, sum(n)).tolist(), 64, 8, 64, seed=9)
    got = s.run()
    s.check(got)
    for _ in range(3):
        assert torch.equal(s.run().view(torch.int16), got.view(torch.int16))
    assert s.status.item() == 0


@pytest.mark.parametrize("dim", [64, 128])
def test_prefix_maxima_that_grow(dim):
    # keys that grow along the prefix: every stage moves the rows' maxima by more
    # than the rescaling allows to pass
    s = Shared([(1024, [3, 5])], [4, 9], 4, 1, dim, seed=2)
    ramp = torch.from_numpy(s.np_tables[0, :64]).cuda().long()
    s.q.copy_(s.q.abs())
    for t, b in enumerate(ramp):
        s.k[b] = (0.02 * t + 0.05 * s.k[b].float()).bfloat16()
    s.check(s.run())


def test_prefix_in_a_graph_and_on_another_stream():
    s = Shared([(512, [30, 5, 9]), (96, [5])], [4, 5, 1, 2], 8, 2, 128)
    ws = api.workspace(api.sv_prefix_attend_workspace(s.batch, s.kv, s.shared, 8))
    out = torch.full_like(s.q, 7.0)
    call = api.bind_prefix_attend(s.kv, s.batch, s.shared, s.q, s.scale, out, ws, s.status)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(stream)
    torch.cuda.current_stream().wait_stream(stream)
    s.check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    s.q.copy_(s.q.flip(0))
    s.kv.cache_lens[1] = s.ctx[1] = 515  # lengths are read when it runs
    out.fill_(7.0)
    graph.replay()
    s.check(out)
    assert s.status.item() == 0


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("missing", [None, 24, 7])
def test_prefix_shares_of_several_lists(dim, missing):
    # about three lists a CTA: whole lists begin where the one before stopped, so
    # that the last, incomplete stage (of one page) comes in their midst
    s = Shared([(400, [3] * 30), (208, [0, 20] * 10), (0, [9])], [40] * 30 + [38] * 20 + [3], 32, 8, dim, seed=dim)
    if missing is not None:
        s.kv.block_tables[0, missing] = -1
    got = s.run()
    assert s.status.item() == (0 if missing is None else N.SV_DEV_BAD_BLOCK_ID)
    check_attend(s, got, lambda i, r, g: [t for t in range(s.ctx[i]) if i >= 30 or t // 16 != missing])
    assert torch.equal(s.run().view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("n", [1, 40, 300])
def test_prefix_groups_of_one_and_of_none(n):
    # groups without requests, without rows and without a prefix among others
    rng = np.random.default_rng(n)
    groups = [(16 * int(rng.integers(0, 12)), rng.integers(0, 40, int(rng.integers(0, 5))).tolist()) for _ in range(n)]
    groups += [(144, [5, 0]), (32, []), (16, [1])]
    total = sum(len(own) for _, own in groups)
    rows = rng.integers(1, 4, total).tolist()
    s = Shared(groups, rows, 4, 2, 64, seed=n)
    keep = rng.random(total) > 0.3
    s.window(begin=[0] * total, end=[r if k else 0 for r, k in zip(rows, keep)], verify=rows)
    s.check(s.run())
    assert s.status.item() == 0
