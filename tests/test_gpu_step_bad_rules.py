"""A whole step in which some requests' logit rules are malformed: their logits
are not shaped, so they are neither decided nor committed; the others are as
the CPU oracle has them."""

import numpy as np
import pytest
import torch

import oracle
from oracle import edges
from speculative_decoding_verification_padding_gb300 import api, build
from test_gpu_step_edges import _arr, _edge_step, _state
from test_gpu_step_refused import RESULTS, _check_served, _prime

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


def _spoil(s, kind, i):
    r = s.rules
    {"penalty": lambda: r.repetition.__setitem__(i, float("nan")),
     "presence": lambda: r.presence.__setitem__(i, float("inf")),
     "history": lambda: r.history_len.__setitem__(i, r.history.shape[1] + 1),
     "prompt": lambda: r.prompt_len.__setitem__(i, -1)}[kind]()


FINDING = dict(penalty=edges.BAD_PARAM, presence=edges.BAD_PARAM, history=edges.BAD_LENGTH, prompt=edges.BAD_LENGTH)


@pytest.mark.parametrize("first", [True, False])  # the step's first run, or after a good one
@pytest.mark.parametrize("name,n,T,kind", [("batch64", 12, 0.7, "penalty"), ("batch64", 12, 0.0, "history"),
                                           ("tree70b", 3, 1.0, "prompt"), ("tree70b", 3, 0.0, "presence"),
                                           ("chain8b", 1, 0.7, "penalty")])
def test_malformed_rules_keep_their_request_undecided(name, n, T, kind, first):
    s = _edge_step(name, temperature=T, n_req=n, ctx_scale=0.02)
    if not first:
        s.run()
    out = [0] if n == 1 else [1, n - 1]
    keep = s.rules.repetition.clone(), s.rules.presence.clone(), s.rules.history_len.clone(), s.rules.prompt_len.clone()
    for i in out:
        _spoil(s, kind, i)
    _prime(s)
    s.restore_cache_state()
    before = _state(s)
    s.run(restore=False)
    torch.cuda.synchronize()
    assert s.dev_status.item() == FINDING[kind]
    lens = _arr(s.kv.cache_lens)
    for i in out:
        assert lens[i] == before["cache_lens"][i]
        for v, k in enumerate(RESULTS):
            assert (_arr(getattr(s, k))[i] == v + 1).all(), k
    served = np.setdiff1d(np.arange(n), out)
    rows = np.diff(s.w.cu_rows)
    rows[out] = 0
    assert np.array_equal(_arr(s.row_end), rows)
    for t, k in zip((s.rules.repetition, s.rules.presence, s.rules.history_len, s.rules.prompt_len), keep):
        t.copy_(k)
    if len(served):
        want, mag = edges.shape_logits(s.w.cu_rows, s.w.parent, s.w.tokens, _arr(s.raw[0]),
                                       **{k: None if v is None else _arr(v) for k, v in vars(s.rules).items()})
        at = np.concatenate([np.arange(s.w.cu_rows[i], s.w.cu_rows[i + 1]) for i in served])
        got, want, mag = _arr(s.target)[at].astype(np.float64), want[at], mag[at]
        fin = np.isfinite(want)
        assert np.array_equal(fin, np.isfinite(got)) and (np.abs(got[fin] - want[fin]) <= 6 * 2.0 ** -24 * mag[fin]).all()
        # what was not shaped may hold anything: the oracle is shown the raw rows there
        for raw, x in zip(s.raw, (s.target, s.draft)):
            if x is not None:
                for i in out:
                    x[s.w.cu_rows[i]:s.w.cu_rows[i + 1]] = raw[s.w.cu_rows[i]:s.w.cu_rows[i + 1]]
        _check_served(s, served, before)
    # with the rules put right the step decides everyone (blocks it took are still there)
    s.dev_status.zero_()
    before = _state(s)
    s.run(restore=False)
    torch.cuda.synchronize()
    assert s.dev_status.item() == 0 and np.array_equal(_arr(s.row_end), np.diff(s.w.cu_rows))
    assert np.array_equal(_arr(s.kv.cache_lens), before["cache_lens"] + 1 + _arr(s.accepted_len))


def test_rules_tell_malformed_requests_apart():
    # alone: row_end of the malformed is 0, of the others untouched, whether it
    # is the batch's own or another
    R, V = 5, 40
    dev = lambda a, t=torch.int32: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
    cu, parent = dev([0, 2, 4, 6, 8, 10]), dev([-1, 0, -1, 0, -1, 1, -1, 0, -1, 0])
    tokens = dev([1] * 10)
    x = torch.randn(10, V, device="cuda")
    rules = api.LogitRules(frequency=dev([0.5, float("nan"), 0.5, 0.5, 0.5], torch.float32))
    for own in (True, False):
        row_end, out = dev([2, 2, 2, 2, 0]), torch.full((10, V), 7.0, device="cuda")
        batch = api.Batch(cu, parent, tokens, 2, row_end=row_end if own else None)
        status = dev([0])
        api.sv_shape_logits(batch, x, rules, out, status, row_end=row_end)
        assert row_end.tolist() == [2, 0, 0, 2, 0]  # a parameter; a parent
        assert status.item() == edges.BAD_PARAM | edges.BAD_PARENT
        left = (out == 7).all(1).tolist()
        assert left == [False, False, True, True, True, True, False, False, own, own]
    with pytest.raises(api.N.SpecVerifyError):
        api.sv_shape_logits(batch, x, rules, out, status, row_end=row_end[:4].clone())
    with pytest.raises(api.N.SpecVerifyError):
        api.sv_shape_logits(batch, x, rules, out, status, row_end=row_end.long())
    assert R == batch.n_req
