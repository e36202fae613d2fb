"""A whole step in which some requests cannot be served: what the reservation
refuses is neither attended nor decided nor committed, the others are as the
CPU oracle has them, and the next step serves it."""

import numpy as np
import pytest
import torch

import oracle
from oracle import edges
from speculative_decoding_verification_padding_gb300 import api, build
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import DeviceStep
from test_gpu_step_edges import _arr, _check_step, _edge_step, _state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    oracle.build()


RESULTS = ("accepted_len", "accepted_nodes", "next_token", "ambiguous", "done")


def _prime(s):
    """Results of an earlier step that a request kept out still has."""
    for i, k in enumerate(RESULTS):
        getattr(s, k).fill_(i + 1)
    s.out.fill_(3)


def _page(s, i, tables, lens):
    """The K and V of request i's committed tokens."""
    t = np.arange(lens[i])
    at = tables[i, t // 16].astype(np.int64)
    return [_arr(c)[at, :, t % 16] for c in (s.kv.k_cache, s.kv.v_cache)]


def _check_kept_out(s, out, before):
    """The requests `out` are as they were before the step."""
    w = s.w
    for i in out:
        assert _arr(s.kv.cache_lens)[i] == before["cache_lens"][i]
        assert np.array_equal(_arr(s.kv.block_tables)[i], before["block_tables"][i])
        now, was = _page(s, i, _arr(s.kv.block_tables), _arr(s.kv.cache_lens)), before["pages"][i]
        assert all(np.array_equal(a, b) for a, b in zip(now, was))
        for v, k in enumerate(RESULTS):
            assert (_arr(getattr(s, k))[i] == v + 1).all(), k
        assert (s.out[w.cu_rows[i]:w.cu_rows[i + 1]] == 3).all()


def _before(s):
    b = _state(s)
    b["pages"] = [_page(s, i, b["block_tables"], b["cache_lens"]) for i in range(s.w.n_req)]
    return b


def _check_served(s, served, before):
    """The others' decisions and lengths are the oracle's on the shaped logits."""
    w = s.w
    err, st = oracle.accept(w.batch(), _arr(s.target), None if s.draft is None else _arr(s.draft), s.T, w.seed)
    assert err == 0
    amb = _arr(s.ambiguous)
    sure = [i for i in served if not (st.ambiguous[i] or amb[i])]
    assert len(sure) >= len(served) - 1
    for k in ("accepted_len", "next_token", "accepted_nodes"):
        assert np.array_equal(_arr(getattr(s, k))[sure], getattr(st, k)[sure]), k
    assert np.array_equal(_arr(s.kv.cache_lens)[served],
                          before["cache_lens"][served] + 1 + _arr(s.accepted_len)[served])


def _split(s):
    taken = _arr(s.taken)
    return np.nonzero(taken < 0)[0], np.nonzero(taken >= 0)[0]


def _blocks(s):
    """No block is lost or held twice."""
    tables, n = _arr(s.kv.block_tables), int(s.pool.free_count.item())
    held = tables[tables >= 0].tolist() + _arr(s.pool.free_list)[:n].tolist()
    assert len(held) == len(set(held))
    return len(held)


@pytest.mark.parametrize("commit", ["fused", "apart"])
@pytest.mark.parametrize("name,n,T", [("batch64", 12, 0.7), ("batch64", 12, 0.0), ("tree70b", 3, 0.0),
                                      ("tree70b", 3, 1.0)])
def test_a_short_pool_keeps_requests_out_of_the_whole_step(name, n, T, commit):
    s = _edge_step(name, temperature=T, n_req=n, ctx_scale=0.02)
    ctx, rows = s.w.cache_lens, np.diff(s.w.cu_rows)
    new = -(-(ctx + rows) // 16) - -(-ctx // 16)
    free, count = _arr(s.pool.free_list).copy(), int(s.pool.free_count.item())
    few = int(new.sum()) // 2  # some are served, some not
    s.pool.free_count.fill_(few)
    _prime(s)
    before = _before(s)
    s.run(commit=commit == "fused", restore=False)
    if commit == "apart":
        s.commit()
    torch.cuda.synchronize()
    out, served = _split(s)
    assert len(out) >= 1 and (new[out] > 0).all()
    # some could be committed: their accepted path lies in the page they have
    assert name != "batch64" or (ctx[out] % 16 > 0).any()
    assert s.dev_status.item() == edges.POOL_EMPTY | (0 if commit == "fused" else edges.BAD_WINDOW)
    assert np.array_equal(_arr(s.row_end), np.where(_arr(s.taken) < 0, 0, rows))
    _check_kept_out(s, out, before)
    _check_served(s, served, before)
    held = _blocks(s)
    # with blocks in the pool again, the next step serves everyone
    n0 = int(s.pool.free_count.item())
    back = free[few:count]
    s.pool.free_list[n0:n0 + len(back)] = torch.from_numpy(back).cuda()
    s.pool.free_count.fill_(n0 + len(back))
    assert _blocks(s) == held + len(back)
    s.dev_status.zero_()
    before, pool = _state(s), (_arr(s.pool.free_list).copy(), int(s.pool.free_count.item()))
    s.run(restore=False)
    _check_step(s, before, pool)


@pytest.mark.parametrize("name,T", [("chain8b", 0.7), ("tree70b", 0.0), ("tree70b", 1.0)])
def test_a_refused_request_alone_in_its_step(name, T):
    s = _edge_step(name, temperature=T, n_req=1, ctx_scale=0.0229)
    s.pool.free_count.fill_(0)
    # (a context that ends inside a page with too little room for the rows)
    assert s.w.cache_lens[0] % 16 + s.w.cu_rows[1] > 16
    _prime(s)
    before = _before(s)
    s.run(restore=False)
    torch.cuda.synchronize()
    assert s.dev_status.item() == edges.POOL_EMPTY and s.row_end.item() == 0
    _check_kept_out(s, [0], before)
    assert s.pool.free_count.item() == 0


def test_a_dropped_block_id_and_bad_parents_keep_their_requests_out():
    s = _edge_step(n_req=12, ctx_scale=0.01)
    n = int(s.pool.free_count.item())
    s.pool.free_list[n - 1] = 1 << 20  # the first block that the call takes
    s.batch.parent[int(s.w.cu_rows[7]) + 1] = 5
    _prime(s)
    before = _before(s)
    s.run(restore=False)
    torch.cuda.synchronize()
    first = int(np.nonzero(_arr(s.taken) > 0)[0][0])
    out = [first, 7]
    assert first != 7 and _arr(s.taken)[7] == -1
    rows = np.diff(s.w.cu_rows)
    assert np.array_equal(np.nonzero(_arr(s.row_end) != rows)[0], np.sort(out))
    assert s.dev_status.item() & edges.BAD_BLOCK and s.dev_status.item() & edges.BAD_PARENT
    _check_kept_out(s, [7], before)
    assert _arr(s.kv.cache_lens)[first] == before["cache_lens"][first]
    assert _arr(s.next_token)[first] == RESULTS.index("next_token") + 1
    served = np.setdiff1d(np.arange(12), out)
    assert np.array_equal(_arr(s.kv.cache_lens)[served],
                          before["cache_lens"][served] + 1 + _arr(s.accepted_len)[served])


def test_a_captured_step_sees_the_pool_of_each_replay():
    s = _edge_step(n_req=12, ctx_scale=0.01)
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run(restore=False)
    full = int(s._state0.view(-1)[-64].item())  # the free count, last of the state
    for count in (0, full, 0):
        s.restore_cache_state()
        s.pool.free_count.fill_(count)
        s.dev_status.zero_()
        _prime(s)
        before = _before(s)
        g.replay()
        torch.cuda.synchronize()
        out, served = _split(s)
        assert (len(out) > 0) == (count == 0)
        _check_kept_out(s, out, before)
        _check_served(s, served, before)


def test_a_chunked_step_leaves_out_what_has_no_slots():
    w = wl.make_workload(wl.config("batch64"), n_req=12, ctx_scale=0.01, vocab=1024, temperature=0.7)
    s = DeviceStep(w, mode="chunked", chunk=2)
    slots = torch.zeros(w.total_rows, dtype=torch.int32, device="cuda")
    out = [2, 9, 11]
    for i in out:
        slots[int(w.cu_rows[i + 1]) - 1] = -1
    row_end = torch.zeros(12, dtype=torch.int32, device="cuda")
    api.sv_slot_windows(s.kv, s.batch, slots, row_end)
    b = api.Batch(s.batch.cu_rows, s.batch.parent, s.batch.tokens, s.batch.max_rows, verify_len=row_end - 1)
    s.batch = b
    _prime(s)
    before = _before(s)
    s.run(restore=False)
    torch.cuda.synchronize()
    assert s.dev_status.item() == edges.BAD_WINDOW
    for i in out:
        assert _arr(s.kv.cache_lens)[i] == before["cache_lens"][i]
        assert np.array_equal(_arr(s.kv.block_tables)[i], before["block_tables"][i])
        assert _arr(s.next_token)[i] == RESULTS.index("next_token") + 1
    _check_served(s, np.setdiff1d(np.arange(12), out), before)


# ------------------------------------------------- sv_slot_windows alone --

def _windows(cu, slots, blocks, max_rows=128, verify_len=None, R=None):
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    page = torch.empty(blocks, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    kv = api.PagedKV(page, page, dev([[0]]), dev([0]))
    n = len(slots)
    b = api.Batch(dev(cu), torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"),
                  max_rows, verify_len=None if verify_len is None else dev(verify_len))
    row_end = torch.full((len(cu),), 99, dtype=torch.int32, device="cuda")
    api.sv_slot_windows(kv, b, dev(slots), row_end)
    assert row_end[-1].item() == 99  # nothing behind the requests is written
    return row_end[:-1].tolist()


def test_windows_of_slots():
    assert _windows([0, 3, 4, 6, 9], [0, 5, 31, 7, -1, 3, 4, 2, 32], 2) == [3, 1, 0, 0]
    # the last verified row decides: rows behind verify_len need no slot
    assert _windows([0, 3, 6], [1, 2, -1, 3, -1, -1], 2, verify_len=[1, 1]) == [2, 0]
    assert _windows([0, 3, 6], [1, 2, 3, 4, 5, 6], 2, verify_len=[9, -1]) == [3, 0]
    # malformed offsets; rows of no request
    assert _windows([0, 0, 5, 4, 6], [0] * 6, 1, max_rows=4) == [0, 0, 0, 2]
    assert _windows([2, 4], [-1, -1, 3, 4, -1], 1) == [2]
    assert _windows([0, 4], [1, 1], 1) == [0]
    assert _windows([0], [], 1) == []


@pytest.mark.parametrize("requests,rows", [(1, 128), (1000, 33), (9000, 1)])
def test_windows_of_many_requests(requests, rows):
    rng = np.random.default_rng(rows)
    n = rng.integers(1, rows + 1, requests)
    cu = np.concatenate([[0], np.cumsum(n)])
    slots = rng.integers(0, 64, cu[-1])
    slots[rng.random(cu[-1]) < 0.5 / rows] = -1
    want = [int(n[i]) if (slots[cu[i]:cu[i + 1]] >= 0).all() else 0 for i in range(requests)]
    assert _windows(cu.tolist(), slots.tolist(), 4) == want
