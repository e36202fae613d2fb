"""A verification step with its two edges, as a user runs it: blocks reserved,
Q / K / V staged, attention, logits under rules, accept and commit; every call
against the CPU oracle on what the call before it left on the GPU.  And the
acceptance of masked logits, which carry -inf."""

import numpy as np
import pytest
import torch

import oracle
from oracle import edges
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep, EdgeStep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


def _masked(w, seed, keep=0.4):
    """Bars most tokens of every target and draft row alike, the drafted ones
    and the rows' best excepted."""
    rng = np.random.default_rng(seed)
    for r in range(w.total_rows):
        bar = rng.random(w.target_logits.shape[1]) > keep
        bar[w.target_logits[r].argmax()] = bar[w.draft_logits[r].argmax()] = False
        bar[w.tokens] = False
        w.target_logits[r, bar] = -np.inf
        w.draft_logits[r, bar] = -np.inf
    return w


def _same_decisions(s, w, st):
    res = s.results()
    assert res["dev_status"] == 0
    sure = (st.ambiguous == 0) & (res["ambiguous"] == 0)
    assert sure.sum() >= len(sure) - 1
    for k, ref in (("accepted_len", st.accepted_len), ("next_token", st.next_token)):
        assert np.array_equal(res[k][sure], ref[sure]), k
    return res, sure


@pytest.mark.parametrize("T", [0.7, 1.0, 1.3, 0.0])
@pytest.mark.parametrize("case", ["chains", "tree", "odd"])
def test_accept_of_masked_logits(case, T):
    kw = dict(chains=dict(name="batch64", n_req=24, vocab=4096, draft_sigma=0.7),
              tree=dict(name="tree70b", vocab=1024, draft_sigma=0.7),
              odd=dict(name="batch64", n_req=9, vocab=1001, draft_sigma=1.5))[case]
    w = _masked(wl.make_workload(wl.config(kw.pop("name")), ctx_scale=0.01, temperature=T, **kw), 3)
    s = DeviceStep(w, mode="onepass")
    s.row_stats = torch.full((w.total_rows, 4), float("nan"), device="cuda")
    s.accept(row_stats=s.row_stats)
    err, st = oracle.accept(w.batch(), w.target_logits, w.draft_logits if T > 0 else None, T, w.seed)
    assert err == 0
    res, sure = _same_decisions(s, w, st)
    # no barred token is emitted
    for i in np.nonzero(sure)[0]:
        node = w.cu_rows[i] + res["accepted_nodes"][i, res["accepted_len"][i]]
        assert np.isfinite(w.target_logits[node, res["next_token"][i]])
    if T > 0 and case != "tree":
        assert torch.isfinite(s.row_stats[:, 0]).all()


def test_one_sided_masks_reject_and_fall_back():
    # the target bars a drafted token: rejected, and the residual is the
    # target's own where the draft bars what the target permits
    w = wl.make_workload(wl.config("batch64"), n_req=16, ctx_scale=0.01, vocab=512, temperature=0.7,
                         draft_sigma=0.3)
    rng = np.random.default_rng(0)
    for i in range(w.n_req):
        c0, n = w.cu_rows[i], w.cu_rows[i + 1] - w.cu_rows[i]
        j = int(rng.integers(1, n))
        w.target_logits[c0 + j - 1, w.tokens[c0 + j]] = -np.inf
        w.draft_logits[c0 + j - 1, rng.permutation(512)[:200]] = -np.inf
        w.draft_logits[c0 + j - 1, w.tokens[c0 + j]] = 5.0
    s = DeviceStep(w, mode="onepass")
    s.accept()
    err, st = oracle.accept(w.batch(), w.target_logits, w.draft_logits, 0.7, w.seed)
    assert err == 0
    _same_decisions(s, w, st)


def _edge_step(name="batch64", vocab=2048, temperature=0.7, **kw):
    w = wl.make_workload(wl.config(name), vocab=vocab, temperature=temperature, draft_sigma=0.5, **kw)
    g = torch.Generator("cuda").manual_seed(5)
    N, R, H, K, D, V = w.total_rows, w.n_req, w.cfg.n_q_heads, w.cfg.n_kv_heads, w.cfg.head_dim, vocab
    qkv = torch.randn(N, (H + 2 * K) * D, generator=g, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, K * D, K * D], 1))
    freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
    weights = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    ints = lambda lo, hi, *n: torch.randint(lo, hi, n, generator=g, device="cuda", dtype=torch.int32)  # noqa: E731
    length = ints(1, 300, R)
    # masks that bar the lower half here and there, never what was drafted
    let = torch.rand(N, V, generator=g, device="cuda") < 0.5
    let[:, torch.from_numpy(w.tokens).long().cuda()] = True
    words = (let.view(N, V // 32, 32).long() << torch.arange(32, device="cuda")).sum(-1)
    rules = api.LogitRules(
        history=ints(0, V, R, 300), history_len=length, prompt_len=length // 2,
        repetition=1 + 0.2 * torch.rand(R, generator=g, device="cuda"),
        frequency=0.3 * torch.rand(R, generator=g, device="cuda"),
        presence=0.3 * torch.rand(R, generator=g, device="cuda"),
        mask=torch.where(words >= 1 << 31, words - (1 << 32), words).int(),
        mask_row=torch.where(ints(0, 2, N) > 0, torch.arange(N, device="cuda").int(), -1))
    s = EdgeStep(w, q, k, v, api.Rotary(freq, D), rules if V % 32 == 0 else None, *weights, eps=1e-5)
    return s


def _arr(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def _state(s):
    return {"k_cache": _arr(s.kv.k_cache), "v_cache": _arr(s.kv.v_cache),
            "block_tables": _arr(s.kv.block_tables), "cache_lens": _arr(s.kv.cache_lens)}


def _check_step(s, before, free_before):
    """Every call of the step that just ran against the oracle, from the state
    before it; returns the accepted lengths."""
    w, T = s.w, s.T
    torch.cuda.synchronize()
    assert s.dev_status.item() == 0
    free, count = free_before
    err, r = edges.reserve(w.cu_rows, w.parent, before["cache_lens"], before["block_tables"], free, count,
                           s.kv.k_cache.shape[0], w.max_rows, w.total_rows)
    assert err == 0
    for k in ("slots", "positions", "taken"):
        assert np.array_equal(_arr(getattr(s, k)), r[k]), k
    # the turned queries, and the keys as they were staged (the commit moves
    # slots, so the cache is rebuilt from the oracle's slots)
    f64 = lambda t: t.float().cpu().double().numpy()  # noqa: E731
    args = (s.eps, r["positions"][None], _arr(s.rotary.inv_freq), s.rotary.rotary_dim)
    staged = {}
    for name, x, wt in (("q", s.qkv[0], s.weights[0]), ("k", s.qkv[1], s.weights[1])):
        y, mag = edges.stage(f64(x), _arr(wt), *args)
        staged[name] = y
        if name == "q":
            assert (np.abs(f64(s.q) - y) <= 2.0 ** -8 * np.abs(y) + 2.0 ** -16 * mag).all()
    kc, vc = before["k_cache"].copy(), before["v_cache"].copy()
    block, off = r["slots"] // 16, r["slots"] % 16
    kc[block, :, off] = wl.bf16_bits(staged["k"].astype(np.float32))
    vc[block, :, off] = _arr(s.qkv[2].contiguous())
    kv = {"k_cache": kc, "v_cache": vc, "block_tables": r["tables"], "cache_lens": before["cache_lens"]}
    err, _, ref = oracle.tree_attend(w.batch(), kv, _arr(s.q), w.cfg.n_q_heads, w.softmax_scale)
    assert err == 0
    np.testing.assert_allclose(f64(s.out), ref, atol=1e-2, rtol=1e-2)
    # the shaped logits, then the decision on them
    rules = {k: None if v is None else _arr(v) for k, v in vars(s.rules).items()}
    for raw, got in zip(s.raw, (s.target, s.draft)):
        if raw is None:
            continue
        want, mag = edges.shape_logits(w.cu_rows, w.parent, w.tokens, _arr(raw), **rules)
        g = _arr(got).astype(np.float64)
        assert np.array_equal(np.isinf(g), np.isinf(want))
        fin = np.isfinite(want)
        assert (np.abs(g[fin] - want[fin]) <= 6 * 2.0 ** -24 * mag[fin]).all()
    err, st = oracle.accept(w.batch(), _arr(s.target), None if s.draft is None else _arr(s.draft), T, w.seed)
    assert err == 0
    res, sure = _same_decisions(s, w, st)
    # the commit: lengths, and no block lost or held twice
    assert np.array_equal(_arr(s.kv.cache_lens), before["cache_lens"] + 1 + res["accepted_len"])
    tables, n = _arr(s.kv.block_tables), int(s.pool.free_count.item())
    held = tables[tables >= 0].tolist() + _arr(s.pool.free_list)[:n].tolist()
    assert len(held) == len(set(held)) == (before["block_tables"] >= 0).sum() + count
    return res


@pytest.mark.parametrize("name,T", [("batch64", 0.7), ("tree70b", 0.0), ("tree70b", 1.0), ("chain8b", 0.7)])
def test_two_steps_from_projections_to_commit(name, T):
    kw = dict(n_req=20) if name == "batch64" else {}
    s = _edge_step(name, temperature=T, ctx_scale=0.02, **kw)
    for step in range(2):
        before = _state(s)
        free = (_arr(s.pool.free_list).copy(), int(s.pool.free_count.item()))
        s.run(restore=step == 0)
        _check_step(s, before, free)


def test_a_captured_step_replays_as_it_ran():
    s = _edge_step(n_req=12, ctx_scale=0.01)
    kc, vc = s.kv.k_cache.clone(), s.kv.v_cache.clone()
    s.run()
    torch.cuda.synchronize()
    keep = lambda: [t.clone() for t in (*s.outputs(), s.target, s.draft, s._state, s.kv.k_cache, s.kv.v_cache)]  # noqa: E731
    first = keep()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for _ in range(2):
        s.kv.k_cache.copy_(kc)
        s.kv.v_cache.copy_(vc)
        for t in s.outputs():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(keep(), first):
            assert torch.equal(a, b)


def test_a_step_whose_pool_is_short_leaves_the_refused_request_alone():
    s = _edge_step(n_req=12, ctx_scale=0.01)
    need = _arr(s.pool.free_count).item()
    rows = np.diff(s.w.cu_rows)
    new = -(-(s.w.cache_lens + rows) // 16) - -(-s.w.cache_lens // 16)
    few = int(new.sum() - 1)
    assert few < need
    s.pool.free_count.fill_(few)
    s.q.fill_(7)
    s.reserve()
    s.stage()
    torch.cuda.synchronize()
    assert s.dev_status.item() == edges.POOL_EMPTY
    refused = np.nonzero(_arr(s.taken) < 0)[0]
    assert len(refused) >= 1 and (new[refused] > 0).all()
    for i in refused:
        part = s.q[s.w.cu_rows[i]:s.w.cu_rows[i + 1]]
        assert (part == 7).all()
