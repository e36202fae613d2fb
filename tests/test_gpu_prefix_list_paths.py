"""sv_prefix_attend at sizes where prefixes are read by lists of their own, along the
paths a served batch takes: graphs, several streams, offsets past 32 bits, whole steps.
Each test first sees to it that the call has such lists (the call's header, at the
start of its workspace, counts their stages)."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep, EdgeStep
from test_gpu_pages import Setup, attended, check_attend, listed
from test_gpu_prefix import Shared
from test_gpu_prefix_lists import check, own

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


def workspace(s):
    return api.workspace(api.sv_prefix_attend_workspace(s.batch, s.kv, s.shared, s.H)).fill_(255)


def list_stages(ws):
    return int(ws[:20].view(torch.int32)[3])


def bits(t):
    return t.view(torch.int16)


def served(dim, seed, heads=32, kv_heads=8):
    rng = np.random.default_rng(seed)
    rows = rng.integers(1, 5, 100).tolist()
    return Shared([(512, own(rng, 60, 90)), (0, own(rng, 3)), (800, own(rng, 37, 200))], rows, heads, kv_heads, dim,
                  seed=seed)


@pytest.mark.parametrize("dim", [64, 128])
def test_list_path_in_a_graph(dim):
    s = served(dim, 1)
    s.kv.block_tables.copy_(s.i32(s.np_tables))  # (a shorter prefix is given below)
    ws, out = workspace(s), torch.full_like(s.q, 7.0)
    call = api.bind_prefix_attend(s.kv, s.batch, s.shared, s.q, s.scale, out, ws, s.status)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    call(stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert list_stages(ws) > 0
    check(s, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):  # queries, lengths and prefixes are read when it runs
        s.q.copy_(s.q.flip(0))
        if step:
            s.shared.prefix_len.copy_(s.i32([256, 0, 800] if step == 1 else [512, 0, 400]))
            for i in (5 * step, 50 + step, 80 + step):  # one token less, where there is one
                # (the last context slot becomes the first row's)
                if s.ctx[i] > (512 if i < 60 else 800):
                    s.ctx[i] -= 1
                    s.kv.cache_lens[i] -= 1
        out.fill_(7.0)
        graph.replay()
        assert list_stages(ws) > 0
        check(s, out)
    assert s.status.item() == 0


def test_list_path_beside_other_calls():
    # on three streams, each with a workspace of its own; the same bits as alone
    a = Setup([3000, 90, 777], [9, 5, 3], 8, 2, 128, seed=1)
    pages = torch.from_numpy(a.lists(30)).cuda()
    b = served(64, 2)
    c = Setup([2000, 900], [64, 40], 8, 1, 128, tree=True, seed=3)
    wa = api.workspace(api.sv_page_attend_workspace(a.batch, a.kv, a.H, 30))
    wb = [workspace(b) for _ in range(2)]
    wc = api.workspace(api.sv_tree_attend_workspace(c.batch, c.kv, c.H))
    calls = [lambda out: attended(a, pages, wa, out), lambda out: b.run(out, wb[0]), lambda out: b.run(out, wb[1]),
             lambda out: api.sv_tree_attend(c.kv, c.batch, c.q, c.H, c.scale, out, wc, c.status)]
    sets = (a, b, b, c)
    alone = [torch.full_like(x.q, 7.0) for x in sets]
    for call, out in zip(calls, alone):
        call(out)
    torch.cuda.synchronize()
    assert list_stages(wb[0]) > 0
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [[torch.full_like(x.q, 7.0) for _ in range(20)] for x in sets]
    torch.cuda.synchronize()
    for k in range(20):
        for call, stream, out in zip(calls, streams, outs):
            with torch.cuda.stream(stream):
                call(out[k])
    torch.cuda.synchronize()
    for x, want, got in zip(sets, alone, outs):
        assert x.status.item() == 0
        for y in got:
            assert torch.equal(bits(y), bits(want))
    check_attend(a, alone[0], listed(a, pages.cpu().numpy()))
    check(b, alone[1])


def test_list_path_past_32_bits():
    # the same requests at the far end of a cache of 2.3e9 elements: the same bits
    near = served(128, 4)
    blocks = 140000
    shift = blocks - near.blocks
    far = [torch.zeros(blocks, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    far[0][shift:], far[1][shift:] = near.k, near.v
    given = near.kv.block_tables
    kv = api.PagedKV(*far, torch.where(given >= 0, given + shift, -1).int(), near.kv.cache_lens)
    results = []
    for c in (near.kv, kv):
        ws = api.workspace(api.sv_prefix_attend_workspace(near.batch, c, near.shared, near.H)).fill_(255)
        out = torch.full_like(near.q, 7.0)
        api.sv_prefix_attend(c, near.batch, near.shared, near.q, near.scale, out, ws, near.status)
        assert list_stages(ws) > 0
        results.append(out)
    assert near.status.item() == 0
    assert torch.equal(bits(results[0]), bits(results[1]))
    check(near, results[1])


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


# ------------------------------------------------------------------- steps --

GROUPS = [(40, 640), (24, 320)]


def _workload():
    w = wl.make_workload(wl.config("batch64", ctx=("uniform", 700, 900)), vocab=512)
    cu, tables = [0], w.block_tables.copy()
    for n, p in GROUPS:
        a = cu[-1]
        cu.append(a + n)
        tables[a + 1:a + n, :p // 16] = tables[a, :p // 16]
    w.block_tables = tables
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return w, api.SharedPrefix(i32(cu), i32([p for _, p in GROUPS]))


def _check_step(s, lens, cache):
    """The step's attention, on the cache that it read (before the commit)."""
    w = s.w
    k, v, tables = cache
    for i, n in enumerate(lens):
        a, b = int(w.cu_rows[i]), int(w.cu_rows[i + 1])
        t = torch.arange(int(n) + b - a, device="cuda")
        block = tables[i].long()[t // 16]
        kk, vv = k[block, :, t % 16].double(), v[block, :, t % 16].double()
        see = torch.ones(b - a, len(t), dtype=torch.bool)
        see[:, int(n):] = False
        for j in range(b - a):
            x = j
            while x >= 0:
                see[j, int(n) + x] = True
                x = int(w.parent[a + x])
        q = s.q[a:b].double().view(b - a, k.shape[1], -1, k.shape[3])
        x = torch.einsum("rkgd,tkd->rkgt", q, kk) * w.softmax_scale
        p = x.masked_fill(~see.cuda()[:, None, None], -torch.inf).softmax(-1)
        want = torch.einsum("rkgt,tkd->rkgd", p, vv).flatten(1, 2)
        mag = torch.einsum("rkgt,tkd->rkgd", p, vv.abs()).flatten(1, 2)
        # the bound of test_gpu_pages.check_attend
        assert ((s.out[a:b].double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -9) * mag).all()


def _cache(s):
    return s.kv.k_cache.clone(), s.kv.v_cache.clone(), s.kv.block_tables.clone()


def test_list_path_in_a_step():
    w, shared = _workload()
    s, other = DeviceStep(w, mode="onepass", shared=shared), DeviceStep(w, mode="onepass")
    lens, cache = s.kv.cache_lens.tolist(), _cache(s)
    s.attend()
    assert list_stages(s.ws) > 0
    s.run()
    other.run()
    res, ref = s.results(), other.results()
    assert res["dev_status"] == 0
    _check_step(s, lens, cache)
    for name in ("accepted_len", "next_token"):  # the logits are given: the same decisions
        assert np.array_equal(res[name], ref[name])
    assert torch.equal(s.kv.cache_lens, other.kv.cache_lens)
    first = s.out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    s.out.zero_()
    graph.replay()
    assert s.results()["dev_status"] == 0 and torch.equal(bits(first), bits(s.out))


def test_list_path_in_an_edge_step():
    w, shared = _workload()
    g = torch.Generator("cuda").manual_seed(2)
    H, K, D, N = w.cfg.n_q_heads, w.cfg.n_kv_heads, w.cfg.head_dim, w.total_rows
    qkv = torch.randn(N, (H + 2 * K) * D, generator=g, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, K * D, K * D], 1))
    s = EdgeStep(w, q, k, v, shared=shared)
    s.restore_cache_state()
    lens = s.kv.cache_lens.tolist()
    s.reserve()
    s.stage()
    cache = _cache(s)
    s.attend()
    assert list_stages(s.ws) > 0
    _check_step(s, lens, cache)
    s.shape()
    s.accept_commit()
    assert s.results()["dev_status"] == 0
