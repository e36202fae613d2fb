"""Drafts that both sides bar (a logit of -inf in the target and the draft row
of the parent): proposed before the mask was known, so not draws from the masked
q.  The oracle's rule (no GPU): rejected on chains, passed over in trees, and
what is emitted is still distributed as the masked target."""

import numpy as np
import pytest
from scipy import stats

import oracle

V, T = 16, 0.7


def _softmax(x):
    e = np.exp(x - x.max())
    return e / e.sum()


def _rows(seed):
    """A target and a draft row, which tokens are barred, and the q that
    proposed: the draft's before the mask."""
    rng = np.random.default_rng(seed)
    target, draft = rng.normal(0, 1, (2, V)).astype(np.float32)
    proposed = _softmax(draft.astype(np.float64) / T)
    bar = np.zeros(V, bool)
    bar[[0, 3, 4, 9, 15]] = True
    target[bar] = draft[bar] = -np.inf
    return target, draft, bar, proposed


def _batch(n, parent, tokens):
    rows = len(parent)
    return {"cu_rows": np.arange(n + 1, dtype=np.int32) * rows, "parent": np.tile(np.int32(parent), n),
            "tokens": tokens.astype(np.int32).ravel(), "max_rows": rows}


def _first_tokens(parent, n, seed, same=False):
    """The first token that each of n requests emits."""
    target, draft, bar, proposed = _rows(seed)
    if same:
        draft = target
    rows = len(parent)
    tokens = np.random.default_rng(seed + 1).choice(V, (n, rows), p=proposed)
    if same:
        tokens[:] = np.nonzero(bar)[0][1]
    tl, dl = np.tile(target, (n * rows, 1)), np.tile(draft, (n * rows, 1))
    err, st = oracle.accept(_batch(n, parent, tokens), tl, dl, T, 77)
    assert err == 0
    node = st.accepted_nodes[:, 1] if rows > 1 else np.full(n, -1)
    first = np.where(st.accepted_len > 0, tokens[np.arange(n), np.maximum(node, 0)], st.next_token)
    return first, st, tokens, bar, _softmax(target.astype(np.float64) / T)


@pytest.mark.parametrize("parent", [[-1, 0], [-1, 0, 1, 2], [-1, 0, 0], [-1, 0, 0, 0, 1, 1]])
def test_no_barred_draft_is_accepted_and_the_target_is_kept(parent):
    n = 200000
    first, st, tokens, bar, p = _first_tokens(parent, n, 5)
    path = st.accepted_nodes[:, 1:]
    on = path >= 0
    taken = tokens[np.nonzero(on)[0], path[on]]
    assert not bar[taken].any() and not bar[st.next_token].any() and not bar[first].any()
    counts = np.bincount(first, minlength=V)[~bar]
    stat = ((counts - n * p[~bar]) ** 2 / (n * p[~bar])).sum()
    assert stat < stats.chi2.ppf(1 - 1e-3, (~bar).sum() - 1)


@pytest.mark.parametrize("parent", [[-1, 0], [-1, 0, 0]])
def test_the_same_masked_row_on_both_sides_leaves_the_target(parent):
    # p = q: max(0, p - q) is 0 everywhere, the token can only come from p
    n = 50000
    first, st, _, bar, p = _first_tokens(parent, n, 8, same=True)
    assert (st.accepted_len == 0).all()
    counts = np.bincount(first, minlength=V)
    assert counts[bar].sum() == 0
    stat = ((counts[~bar] - n * p[~bar]) ** 2 / (n * p[~bar])).sum()
    assert stat < stats.chi2.ppf(1 - 1e-3, (~bar).sum() - 1)
