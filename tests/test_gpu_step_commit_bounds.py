"""Steps with a page choice: whatever way a step commits, the pages that the commit
fills have bounds in the next step."""

import numpy as np
import pytest
import torch

import oracle
from oracle import pages as plain
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep, EdgeStep, PageChoice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


def f64(t):
    return t.float().cpu().double().numpy()


def _lens(s):
    return s.kv.cache_lens.cpu().numpy().copy()


def _forget(s):
    """Bounds of blocks that hold no complete page: what a former owner left."""
    known = set()
    for row, n in zip(s.kv.block_tables.cpu().tolist(), _lens(s)):
        known |= set(row[:n // 16])
    other = torch.tensor([b for b in range(s.bounds.shape[0]) if b not in known], device="cuda")
    s.bounds[other] = 1000.0


def _check(s, before):
    after = _lens(s)
    assert (after // 16 > before // 16).any()  # pages were filled
    ref = plain.bounds(f64(s.kv.k_cache), s.kv.block_tables.cpu().numpy(), after)
    known = ~np.isnan(ref)
    assert np.array_equal(f64(s.bounds)[known], ref[known])


def _workload(name, **kw):
    return wl.make_workload(wl.config(name), **{**dict(n_req=64, ctx_scale=0.05, vocab=512), **kw})


@pytest.mark.parametrize("mode", ["onepass", "budget"])
@pytest.mark.parametrize("way", ["commit", "accept_commit", "run"])
def test_commits_of_a_step(mode, way):
    s = DeviceStep(_workload("batch256" if mode == "budget" else "batch64"), mode=mode, choice=PageChoice(6, 1, 2))
    batch = s.batch_sel if mode == "budget" else s.batch
    _forget(s)
    s.restore_cache_state()
    before = _lens(s)
    if way == "run":
        s.run()
    else:
        s.run(commit=False, restore=False)
        if way == "commit":
            s.commit(batch)
        else:
            s.accept_commit(batch)
    _check(s, before)
    assert s.results()["dev_status"] == 0


@pytest.mark.parametrize("way", ["commit", "accept_commit", "run"])
def test_commits_of_an_edge_step(way):
    w = _workload("batch64", temperature=0.7)
    g = torch.Generator("cuda").manual_seed(2)
    H, K, D, N = w.cfg.n_q_heads, w.cfg.n_kv_heads, w.cfg.head_dim, w.total_rows
    qkv = torch.randn(N, (H + 2 * K) * D, generator=g, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, K * D, K * D], 1))
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    s = EdgeStep(w, q, k, v, api.Rotary(freq, D), choice=PageChoice(5, 1, 1))
    s.restore_cache_state()
    _forget(s)
    before = _lens(s)
    s.run(commit=way == "run", restore=False)
    if way != "run":
        getattr(s, way)()
    _check(s, before)
    assert s.results()["dev_status"] == 0


def test_a_captured_commit():
    s = DeviceStep(_workload("batch64"), mode="onepass", choice=PageChoice(6, 1, 2))
    s.run(commit=False)
    s.commit()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(commit=False)
        s.commit()
    s.restore_cache_state()
    before = _lens(s)
    _forget(s)
    graph.replay()
    _check(s, before)


def test_a_chunked_commit_in_between():
    # a step built for one pass offers the chunked call too (over the whole context)
    s = DeviceStep(_workload("batch64"), mode="onepass", choice=PageChoice(6, 1, 2))
    _forget(s)
    s.restore_cache_state()
    before = _lens(s)
    s.chunked_commit()
    _check(s, before)
    assert s.results()["dev_status"] == 0
