"""Acceptance of logits under masks that the drafts did not know: drafted tokens
barred in the target and the draft row alike are rejected and what is emitted is
permitted, against the CPU oracle (tests/test_oracle_barred.py pins its rule)."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


def _bar_drafts(w, seed, share, low=-np.inf):
    """Bars that share of the drafted tokens, and as many others, in their
    parents' target and draft rows; each row's best two others stay."""
    rng = np.random.default_rng(seed)
    V = w.target_logits.shape[1]
    for i in range(w.n_req):
        c0, c1 = w.cu_rows[i], w.cu_rows[i + 1]
        for r in range(c0, c1):
            kids = [c for c in range(c0 + 1, c1) if w.parent[c] == r - c0]
            bar = [w.tokens[c] for c in kids if rng.random() < share]
            keep = [v for v in np.argsort(w.target_logits[r])[::-1][:8] if v not in bar][:2]
            bar = np.setdiff1d(np.union1d(bar, rng.choice(V, V // 8)).astype(int), keep)
            w.target_logits[r, bar] = low
            w.draft_logits[r, bar] = low
    return w


def _check(w, T):
    """The step's decisions against the oracle; returns those of the requests
    that neither calls ambiguous."""
    s = DeviceStep(w, mode="onepass")
    s.accept()
    res = s.results()
    assert res["dev_status"] == 0
    err, st = oracle.accept(w.batch(), w.target_logits, w.draft_logits, T, w.seed)
    assert err == 0
    sure = (st.ambiguous == 0) & (res["ambiguous"] == 0)
    assert sure.sum() >= len(sure) - 1
    for k in ("accepted_len", "next_token", "accepted_nodes"):
        assert np.array_equal(res[k][sure], getattr(st, k)[sure]), k
    return res, sure


def _no_barred_token(w, res, sure):
    for i in np.nonzero(sure)[0]:
        c0, path = w.cu_rows[i], res["accepted_nodes"][i, :res["accepted_len"][i] + 1]
        for a, b in zip(path, path[1:]):
            assert w.target_logits[c0 + a, w.tokens[c0 + b]] > -1e30, i
        assert w.target_logits[c0 + path[-1], res["next_token"][i]] > -1e30, i


CASES = dict(chains=dict(name="batch64", n_req=40, vocab=4096, draft_sigma=0.3),
             odd=dict(name="batch64", n_req=40, vocab=1001, draft_sigma=0.3),
             one=dict(name="chain8b", vocab=4096, draft_sigma=0.3),
             tree=dict(name="tree70b", vocab=1024, draft_sigma=0.3),
             oddtree=dict(name="tree70b", vocab=777, draft_sigma=0.3))


@pytest.mark.parametrize("share", [0.3, 1.0])
@pytest.mark.parametrize("T", [0.7, 1.0, 1.3])
@pytest.mark.parametrize("case", list(CASES))
def test_drafts_barred_on_both_sides(case, T, share):
    kw = dict(CASES[case])
    w = wl.make_workload(wl.config(kw.pop("name")), ctx_scale=0.01, temperature=T, **kw)
    w = _bar_drafts(w, 3, share)
    res, sure = _check(w, T)
    _no_barred_token(w, res, sure)
    if share == 1.0:
        assert (res["accepted_len"][sure] == 0).all()


def test_a_long_chain_barred_behind_its_first_warp():
    # draft 40 of 60 is barred; the drafts before it are the draft's and the
    # target's own best, so they are accepted
    rows, V = 61, 512
    rng = np.random.default_rng(2)
    logits = rng.normal(0, 1, (rows, V)).astype(np.float32)
    tokens = np.zeros(rows, np.int32)
    tokens[1:] = rng.integers(0, V, rows - 1)
    logits[np.arange(rows - 1), tokens[1:]] = 30.0
    logits[39, tokens[40]] = -np.inf
    batch = {"cu_rows": np.array([0, rows], np.int32), "parent": np.arange(-1, rows - 1, dtype=np.int32),
             "tokens": tokens, "max_rows": rows}
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    b = api.Batch(dev(batch["cu_rows"]), dev(batch["parent"]), dev(tokens), rows)
    i32 = lambda *n: torch.full(n, -7, dtype=torch.int32, device="cuda")  # noqa: E731
    al, nodes, nxt, done, status = i32(1), i32(1, rows), i32(1), i32(1), torch.zeros(1, dtype=torch.int32, device="cuda")
    amb = torch.zeros(1, dtype=torch.uint8, device="cuda")
    x = dev(logits)
    api.sv_accept(b, x, x, V, 0.7, 9, al, nodes, nxt, amb, done, None,
                  api.workspace(api.sv_accept_workspace(b, V)), status)
    err, st = oracle.accept(batch, logits, logits, 0.7, 9)
    assert err == 0 and status.item() == 0
    assert al.item() == st.accepted_len[0] == 39
    assert nxt.item() == st.next_token[0] and np.isfinite(logits[39, nxt.item()])


LOWEST = float(np.finfo(np.float32).min)


def _grammar(w, seed, low, few=6):
    """Masks that permit a few tokens of the vocabulary, most of the row's
    drafted ones among them, as a grammar's do: everything else is at low."""
    rng = np.random.default_rng(seed)
    V = w.target_logits.shape[1]
    for i in range(w.n_req):
        c0, c1 = w.cu_rows[i], w.cu_rows[i + 1]
        for r in range(c0, c1):
            let = [w.tokens[c] for c in range(c0 + 1, c1) if w.parent[c] == r - c0 and rng.random() < 0.7]
            let = np.union1d(let, rng.choice(V, few, replace=False)).astype(int)
            for x in (w.target_logits[r], w.draft_logits[r]):
                kept = x[let].copy()
                x[:] = low
                x[let] = kept
            # drafts that p and q agree about
            w.target_logits[r, let] = w.draft_logits[r, let] + rng.normal(0, 0.3, len(let))
    return w


@pytest.mark.parametrize("case", list(CASES))
def test_masks_whose_quotient_is_below_the_range(case):
    # the lowest fp32 over T = 0.7 is -inf
    kw = dict(CASES[case])
    w = _grammar(wl.make_workload(wl.config(kw.pop("name")), ctx_scale=0.01, temperature=0.7, **kw), 4, LOWEST)
    _no_barred_token(w, *_check(w, 0.7))


@pytest.mark.parametrize("T,low", [(1.0, LOWEST), (1.3, LOWEST), (0.7, 0.69 * LOWEST), (1.0, -np.inf), (0.7, -np.inf)])
@pytest.mark.parametrize("case", list(CASES) + ["wide"])
def test_masks_that_permit_a_few_tokens(case, T, low):
    # whole spans of a row are barred, at -inf or at a value whose product with
    # log2 e is past the range
    kw = dict(CASES.get(case, dict(name="chain8b", vocab=128256, draft_sigma=0.3)))
    w = _grammar(wl.make_workload(wl.config(kw.pop("name")), ctx_scale=0.01, temperature=T, **kw), 6, low)
    _no_barred_token(w, *_check(w, T))


@pytest.mark.parametrize("share", [0.3, 1.0])
@pytest.mark.parametrize("T", [0.7, 1.0])
def test_barred_drafts_in_a_chunked_step(T, share):
    w = wl.make_workload(wl.config("batch64"), n_req=24, ctx_scale=0.01, vocab=2048, temperature=T, draft_sigma=0.3)
    w = _bar_drafts(w, 7, share)
    s = DeviceStep(w, mode="chunked", chunk=2)
    s.run()
    res = s.results()
    assert res["dev_status"] == 0
    err, st = oracle.verify_chunked(w.batch(), w.kv(), w.q, w.cfg.n_q_heads, w.softmax_scale, w.target_logits,
                                    w.draft_logits, T, w.seed, chunk=2)[:2]
    assert err == 0
    sure = (st.ambiguous == 0) & (res["ambiguous"] == 0)
    assert sure.sum() >= len(sure) - 1
    for k in ("accepted_len", "next_token"):
        assert np.array_equal(res[k][sure], getattr(st, k)[sure]), k
    _no_barred_token(w, res, sure)
    assert np.array_equal(s.kv.cache_lens.cpu().numpy(), w.cache_lens + 1 + res["accepted_len"])


def test_barred_drafts_under_a_budget():
    # verified prefixes only: a barred draft behind the prefix is never looked at
    w = wl.make_workload(wl.config("batch64"), n_req=24, ctx_scale=0.01, vocab=2048, temperature=0.7, draft_sigma=0.3)
    w = _bar_drafts(w, 9, 0.5)
    rng = np.random.default_rng(1)
    keep = np.array([rng.integers(0, n) for n in np.diff(w.cu_rows)], np.int32)
    s = DeviceStep(w, mode="onepass")
    b = api.Batch(s.batch.cu_rows, s.batch.parent, s.batch.tokens, s.batch.max_rows,
                  verify_len=torch.from_numpy(keep).cuda())
    s.accept(b)
    res = s.results()
    err, st = oracle.accept(dict(w.batch(), verify_len=keep), w.target_logits, w.draft_logits, 0.7, w.seed)
    assert err == 0 and res["dev_status"] == 0
    sure = (st.ambiguous == 0) & (res["ambiguous"] == 0)
    assert sure.sum() >= len(sure) - 1
    for k in ("accepted_len", "next_token"):
        assert np.array_equal(res[k][sure], getattr(st, k)[sure]), k
    _no_barred_token(w, res, sure)
