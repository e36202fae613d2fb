"""Whole verification steps over long contexts: each row attends the pages that a
score selects for it, or the requests share a prefix; every call of the step
against the plain 64-bit forms on what the call before it left on the GPU."""

import numpy as np
import pytest
import torch

import oracle
from oracle import pages as plain
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep, EdgeStep, HostPipeline, PageChoice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


def f64(t):
    return t.float().cpu().double().numpy()


def _workload(name="batch64", **kw):
    kw = {**dict(n_req=7, ctx_scale=0.05, vocab=512), **kw}
    return wl.make_workload(wl.config(name), **kw)


def _lens(s):
    return s.kv.cache_lens.cpu().numpy()


def _check_choice(s, lens, windows, before_commit):
    """Scores, pages and attention of the step that ran, on the cache it read."""
    w, c = s.w, s.choice
    k, v, tables = before_commit
    q, bnd = f64(s.q), plain.bounds(k, tables, lens)
    scores, pages = s.scores.cpu().double().numpy(), s.pages.cpu().numpy()
    for i, (b, e) in enumerate(windows):
        n = int(lens[i]) // 16
        for r in range(w.cu_rows[i] + b, w.cu_rows[i] + e):
            ref, mag = plain.scores(q[r], bnd, tables[i], n)
            assert (np.abs(scores[r, :, :n] - ref) <= 2 * q.shape[2] * 2.0 ** -23 * mag).all()
            for g in range(k.shape[1]):
                got = plain.select(s.scores[r, g].cpu().numpy(), n, c.n_keep, c.n_first, c.n_last)
                assert np.array_equal(pages[r, g], got)
    _check_attention(s, lens, windows, before_commit, lambda i, r, g: (
        [t * 16 + o for t in pages[r, g] if t >= 0 for o in range(16)]
        + list(range(int(lens[i]) // 16 * 16, int(lens[i])))))


def _check_attention(s, lens, windows, before_commit, cached):
    w = s.w
    k, v, tables = before_commit
    ref, mag = plain.attend(f64(s.q), k, v, tables, lens, w.cu_rows, w.parent, windows, w.softmax_scale, cached)
    inside = ~np.isnan(ref)
    # the bound of test_gpu_pages.check_attend
    err, tol = np.abs(f64(s.out) - ref)[inside], (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * mag)[inside]
    assert inside.any() and (err <= tol).all(), (err - tol).max()


def _cache(s):
    return f64(s.kv.k_cache), f64(s.kv.v_cache), s.kv.block_tables.cpu().numpy()


@pytest.mark.parametrize("mode", ["onepass", "budget"])
def test_step_with_chosen_pages(mode):
    w = _workload("batch256" if mode == "budget" else "batch64")
    s = DeviceStep(w, mode=mode, choice=PageChoice(6, 1, 2))
    lens, cache = _lens(s).copy(), _cache(s)
    for _ in range(2):  # a step, and the same again
        s.run()
        res = s.results()
        assert res["dev_status"] == 0
        verify = s.verify_len.cpu().numpy() if mode == "budget" else np.diff(w.cu_rows) - 1
        _check_choice(s, lens, [(0, min(int(m), int(u) + 1)) for m, u in zip(np.diff(w.cu_rows), verify)], cache)
        # the pages that the commit filled are bounded
        after, now = _lens(s), _cache(s)
        assert np.array_equal(after, lens + 1 + res["accepted_len"])
        ref = plain.bounds(now[0], now[2], after)
        known = ~np.isnan(ref)
        assert np.array_equal(f64(s.bounds)[known], ref[known])


def test_edge_step_with_chosen_pages_over_several_steps():
    # blocks, queries and keys made by the step itself, three steps in a row
    w = _workload(n_req=5, temperature=0.7)
    g = torch.Generator("cuda").manual_seed(2)
    H, K, D, N = w.cfg.n_q_heads, w.cfg.n_kv_heads, w.cfg.head_dim, w.total_rows
    qkv = torch.randn(N, (H + 2 * K) * D, generator=g, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, K * D, K * D], 1))
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    s = EdgeStep(w, q, k, v, api.Rotary(freq, D), choice=PageChoice(5, 1, 1))
    s.restore_cache_state()
    rows = np.diff(w.cu_rows)
    for _ in range(3):
        lens = _lens(s).copy()
        s.reserve()
        s.stage()
        cache = _cache(s)
        s.attend()
        _check_choice(s, lens, [(0, int(m)) for m in rows], cache)
        s.shape()
        s.bounded.copy_(s.kv.cache_lens)
        s.accept_commit()
        s.bound_pages()
        res = s.results()
        assert res["dev_status"] == 0
        after, now = _lens(s), _cache(s)
        assert np.array_equal(after, lens + 1 + res["accepted_len"])
        ref = plain.bounds(now[0], now[2], after)
        known = ~np.isnan(ref)
        assert np.array_equal(f64(s.bounds)[known], ref[known])


def _share(w, groups):
    """The workload with the first pages of each group's requests shared: groups of
    (requests, prefix)."""
    cu, first = [0], []
    tables = w.block_tables.copy()
    for n, p in groups:
        a = cu[-1]
        cu.append(a + n)
        assert (w.cache_lens[a:a + n] >= p).all()
        tables[a + 1:a + n, :p // 16] = tables[a, :p // 16]
        first.append(p)
    w.block_tables = tables
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return api.SharedPrefix(i32(cu), i32(first))


@pytest.mark.parametrize("name", ["batch64", "tree70b"])
def test_step_with_a_shared_prefix(name):
    kw = {} if name == "batch64" else dict(n_req=1, ctx_scale=0.04)
    w = _workload(name, **kw)
    low = int(w.cache_lens.min()) // 16 * 16
    shared = _share(w, [(3, low), (4, 16)] if name == "batch64" else [(1, low)])
    s = DeviceStep(w, mode="onepass", shared=shared)
    plain_step = DeviceStep(w, mode="onepass")
    lens, cache = _lens(s).copy(), _cache(s)
    s.run()
    plain_step.run()
    res, ref = s.results(), plain_step.results()
    assert res["dev_status"] == 0
    _check_attention(s, lens, [(0, int(m)) for m in np.diff(w.cu_rows)], cache,
                     lambda i, r, g: range(int(lens[i])))
    for k in ("accepted_len", "next_token"):  # the logits are given: the same decisions
        assert np.array_equal(res[k], ref[k])
    assert np.array_equal(_lens(s), _lens(plain_step))


@pytest.mark.parametrize("kind", ["choice", "shared"])
def test_captured_step(kind):
    w = _workload()
    shared = _share(w, [(7, 16)]) if kind == "shared" else None
    s = DeviceStep(w, mode="onepass", shared=shared, choice=PageChoice(5, 1, 1) if kind == "choice" else None)
    s.run()
    first, lens = s.out.clone(), _lens(s).copy()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    s.out.zero_()
    graph.replay()
    assert s.results()["dev_status"] == 0
    assert torch.equal(first, s.out) and np.array_equal(lens, _lens(s))


def test_pipelined_step_with_chosen_pages():
    w = _workload()
    s = DeviceStep(w, mode="onepass", choice=PageChoice(5, 1, 1))
    s.run()
    want = [t.cpu().clone() for t in s.outputs()]
    host = [t.cpu().pin_memory() for t in s.inputs()]
    pipe = HostPipeline(s)
    for _ in range(3):
        out, ready = pipe.submit(host)
    ready.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_two_graphs_of_one_workspace():
    # captured one after the other on one workspace, replayed in turn on one stream
    w = _workload()
    s = DeviceStep(w, mode="onepass", choice=PageChoice(5, 1, 1))
    t = DeviceStep(w, mode="onepass", shared=_share(w, [(7, 16)]))
    t.ws = s.ws = s.ws if s.ws.numel() >= t.ws.numel() else t.ws
    graphs = []
    for x in (s, t):
        x.run()
        x.want = x.out.clone()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.run()
    for _ in range(2):
        for x, g in zip((s, t), graphs):
            x.out.zero_()
            g.replay()
    torch.cuda.synchronize()
    for x in (s, t):
        assert torch.equal(x.out, x.want)


def test_what_a_step_refuses():
    w = _workload()
    with pytest.raises(ValueError):
        DeviceStep(w, mode="chunked", choice=PageChoice(5))
    with pytest.raises(ValueError):
        DeviceStep(w, mode="onepass", choice=PageChoice(5), shared=_share(w, [(7, 16)]))
