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
from speculative_decoding_verification_padding_gb300.step import DeviceStep

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
