"""Host-side checks of the calls that read less of a long cache: refusals come back
before anything is enqueued (no GPU needed), workspaces, and the plain forms that
the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import pages as plain
from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import api, build

A = 256  # an aligned address that nothing reads
OUT = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return N.lib()


def kv(**over):
    f = dict(k_cache=A, v_cache=A, num_blocks=10, block_size=16, n_kv_heads=2, head_dim=128, block_tables=A,
             max_blocks_per_req=4, cache_lens=A)
    return N.SvPagedKV(*{**f, **over}.values())


def batch(**over):
    f = dict(n_req=2, total_rows=6, max_rows_per_req=4, cu_rows=A, parent=A, tokens=A, row_begin=None, row_end=None,
             verify_len=None)
    return N.SvBatch(*{**f, **over}.values())


ref = ctypes.byref
INV, SHAPE, WS = N.SV_ERR_INVALID_ARGUMENT, N.SV_ERR_UNSUPPORTED_SHAPE, N.SV_ERR_WORKSPACE_TOO_SMALL

BAD_KV = [(dict(block_size=32), SHAPE), (dict(head_dim=96), SHAPE), (dict(n_kv_heads=0), INV), (dict(num_blocks=-1), INV),
          (dict(max_blocks_per_req=-1), INV)]
BAD_BATCH = [(dict(n_req=-1), INV), (dict(total_rows=-1), INV), (dict(max_rows_per_req=0), INV),
             (dict(max_rows_per_req=129), SHAPE), (dict(cu_rows=None), INV)]


def test_bound_pages_refusals(lib):
    call = lambda k, n=2, b=A: lib.sv_bound_pages(None if k is None else ref(k), n, None, b, None, None)  # noqa: E731
    assert call(None) == INV
    for over, err in BAD_KV:
        assert call(kv(**over)) == err, over
    assert call(kv(), n=-1) == INV and call(kv(), n=8193) == SHAPE
    assert call(kv(), b=None) == INV and call(kv(), b=A + 8) == INV
    assert call(kv(k_cache=A + 2)) == INV and call(kv(cache_lens=None)) == INV
    assert call(kv(max_blocks_per_req=1 << 30)) == SHAPE
    assert call(kv(), n=0) == N.SV_OK


def test_score_pages_refusals(lib):
    def call(k=None, b=None, q=A, heads=8, bounds=A, scores=A, pages=4):
        return lib.sv_score_pages(ref(k or kv()), ref(b or batch()), q, heads, bounds, scores, pages, None, None)
    for over, err in BAD_KV:
        assert call(k=kv(**over)) == err, over
    for over, err in BAD_BATCH:
        assert call(b=batch(**over)) == err, over
    assert lib.sv_score_pages(ref(kv()), None, A, 8, A, A, 4, None, None) == INV
    assert call(heads=7) == INV and call(heads=0) == INV and call(heads=34) == SHAPE and call(pages=-1) == INV
    assert call(q=None) == INV and call(q=A + 2) == INV and call(bounds=A + 8) == INV and call(scores=A + 2) == INV
    assert call(b=batch(n_req=40000, total_rows=40000)) == SHAPE
    assert call(b=batch(n_req=0)) == N.SV_OK and call(b=batch(total_rows=0)) == N.SV_OK and call(pages=0) == N.SV_OK


def test_select_pages_refusals(lib):
    def call(k=None, b=None, scores=A, pages=4, first=0, last=0, keep=3, out=A):
        return lib.sv_select_pages(ref(k or kv()), ref(b or batch()), scores, pages, first, last, keep, out, None, None)
    for over, err in BAD_BATCH:
        assert call(b=batch(**over)) == err, over
    assert call(keep=0) == INV and call(keep=1025) == SHAPE and call(pages=-1) == INV and call(pages=49153) == SHAPE
    assert call(first=-1) == INV and call(last=-1) == INV and call(first=2, last=2) == INV
    assert call(first=(1 << 31) - 1, last=(1 << 31) - 1) == INV
    assert call(scores=None) == INV and call(out=None) == INV
    assert call(k=kv(cache_lens=None)) == INV
    assert call(b=batch(n_req=0)) == N.SV_OK


def test_page_attend_refusals(lib):
    need = lib.sv_page_attend_workspace(ref(batch()), ref(kv()), 8, 3)
    assert need > 0

    def call(k=None, b=None, q=A, heads=8, scale=0.1, pages=A, keep=3, out=OUT, ws=A, size=need):
        return lib.sv_page_attend(ref(k or kv()), ref(b or batch()), q, heads, scale, pages, keep, out, ws, size, None, None)
    for over, err in BAD_KV + [(dict(max_blocks_per_req=(1 << 18) + 1), SHAPE), (dict(num_blocks=1 << 27), SHAPE),
                               (dict(k_cache=A + 8), INV), (dict(v_cache=None), INV)]:
        assert call(k=kv(**over)) == err, over
        assert lib.sv_page_attend_workspace(ref(batch()), ref(kv(**over)), 8, 3) == 0
    for over, err in BAD_BATCH + [(dict(parent=None), INV)]:
        assert call(b=batch(**over)) == err, over
    assert call(heads=7) == INV and call(heads=34) == SHAPE and call(keep=-1) == INV and call(keep=1025) == SHAPE
    assert call(q=None) == INV and call(q=A + 8) == INV and call(out=OUT + 8) == INV and call(pages=None) == INV
    assert call(ws=A + 16) == INV and call(ws=None) == INV and call(size=need - 1) == WS
    assert call(out=A) == INV and call(out=A + 6 * 8 * 256 - 16) == INV  # over q
    assert call(b=batch(n_req=1 << 20, total_rows=1 << 27), k=kv(max_blocks_per_req=1 << 18)) == SHAPE
    for scale in (0.0, -1.0, float("nan")):
        assert call(scale=scale) == INV
    assert call(b=batch(n_req=0)) == N.SV_OK and call(b=batch(total_rows=0)) == N.SV_OK


def test_prefix_attend_refusals(lib):
    shared = N.SvSharedPrefix(1, A, A)
    need = lib.sv_prefix_attend_workspace(ref(batch()), ref(kv()), ref(shared), 8)
    assert need > 0

    def call(k=None, b=None, s=shared, q=A, heads=8, scale=0.1, out=OUT, ws=A, size=need):
        return lib.sv_prefix_attend(ref(k or kv()), ref(b or batch()), ref(s) if s else None, q, heads, scale, out, ws,
                                    size, None, None)
    for over, err in BAD_KV + [(dict(num_blocks=1 << 27), SHAPE), (dict(k_cache=A + 8), INV), (dict(v_cache=None), INV)]:
        assert call(k=kv(**over)) == err, over
    for over, err in BAD_BATCH + [(dict(parent=None), INV)]:
        assert call(b=batch(**over)) == err, over
    assert call(s=None) == INV
    for groups in (0, -1, 3):
        assert call(s=N.SvSharedPrefix(groups, A, A)) == INV
    assert call(s=N.SvSharedPrefix(1, None, A)) == INV and call(s=N.SvSharedPrefix(1, A, None)) == INV
    assert call(heads=7) == INV and call(heads=34) == SHAPE
    assert call(q=A + 8) == INV and call(out=OUT + 8) == INV and call(out=None) == INV
    assert call(ws=A + 16) == INV and call(size=need - 1) == WS
    assert call(out=A) == INV and call(out=A + 6 * 8 * 256 - 16) == INV  # over q
    assert call(b=batch(n_req=1 << 20, total_rows=1 << 27), k=kv(max_blocks_per_req=1 << 18)) == SHAPE
    for scale in (0.0, -1.0, float("nan")):
        assert call(scale=scale) == INV
    assert call(b=batch(n_req=0)) == N.SV_OK


def _tensors(rows=3, heads=4, kv_heads=2, dim=64, blocks=5):
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    page = torch.zeros(blocks, kv_heads, 16, dim, dtype=torch.bfloat16)
    return (api.PagedKV(page, page.clone(), i32(1, 4), i32(1)), api.Batch(i32(2), i32(rows), i32(rows), rows),
            torch.zeros(rows, heads, dim, dtype=torch.bfloat16))


def test_binding_refuses_wrong_tensors(lib):
    k, b, q = _tensors()
    f32 = lambda *n: torch.zeros(n)  # noqa: E731
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(1 << 10, dtype=torch.uint8)
    bad = [
        lambda: api.bind_bound_pages(k, bf(5, 2, 2, 32)),
        lambda: api.bind_bound_pages(k, f32(5, 2, 2, 64)),
        lambda: api.bind_bound_pages(k, bf(5, 2, 2, 64), i32(0)),
        lambda: api.bind_score_pages(k, b, q.float(), bf(5, 2, 2, 64), f32(3, 2, 4)),
        lambda: api.bind_score_pages(k, b, q[:2], bf(5, 2, 2, 64), f32(3, 2, 4)),
        lambda: api.bind_score_pages(k, b, q, bf(4, 2, 2, 64), f32(3, 2, 4)),
        lambda: api.bind_score_pages(k, b, q, bf(5, 2, 2, 64), f32(3, 3, 4)),
        lambda: api.bind_select_pages(k, b, f32(3, 2, 4), f32(3, 2, 4)),
        lambda: api.bind_select_pages(k, b, f32(3, 2, 4), i32(2, 2, 4)),
        lambda: api.bind_page_attend(k, b, q, 0.1, i32(3, 2), q.clone(), ws),
        lambda: api.bind_page_attend(k, b, q, 0.1, i32(3, 2, 4), q[:, :2].clone(), ws),
        lambda: api.bind_page_attend(k, b, q, 0.1, i32(3, 2, 4), q.float(), ws),
        lambda: api.bind_prefix_attend(k, b, api.SharedPrefix(i32(2), f32(1)), q, 0.1, q.clone(), ws),
        lambda: api.bind_prefix_attend(k, b, api.SharedPrefix(i32(3), i32(1)), q, 0.1, q.clone(), ws),
        # right shapes, but on the host
        lambda: api.bind_bound_pages(k, bf(5, 2, 2, 64)),
        lambda: api.bind_page_attend(k, b, q, 0.1, i32(3, 2, 4), q.clone(), ws),
        lambda: api.bind_prefix_attend(k, b, api.SharedPrefix(i32(2), i32(1)), q, 0.1, q.clone(), ws),
    ]
    for call in bad:
        with pytest.raises(N.SpecVerifyError):
            call()


# ------------------------------------------- pins of the plain forms themselves --

def test_plain_scores_bound_the_products():
    rng = np.random.default_rng(0)
    k = rng.standard_normal((3, 2, 16, 8))
    b = plain.bounds(k, np.array([[2, 0, 1]]), [48])
    q = rng.standard_normal((4, 8))
    s, _ = plain.scores(q, b, [2, 0, 1], 3)
    for g in range(2):
        for t, block in enumerate([2, 0, 1]):
            best = (q[2 * g:2 * g + 2] @ k[block, g].T).max()
            assert best <= s[g, t] + 1e-12
    one = plain.bounds(np.repeat(k[:, :, :1], 16, 2), np.array([[2, 0, 1]]), [48])  # pages of equal keys: no slack
    s, _ = plain.scores(q, one, [2, 0, 1], 3)
    assert np.allclose(s[0], [(q[:2] @ k[b, 0, 0]).max() for b in (2, 0, 1)])


def test_plain_selection():
    x = np.array([0.5, 3, 3, -1, 3, 2, 9], dtype=np.float32)
    assert plain.select(x, 7, 3, 0, 0).tolist() == [1, 2, 6]
    assert plain.select(x, 7, 4, 1, 1).tolist() == [0, 1, 2, 6]
    assert plain.select(x, 7, 3, 1, 2).tolist() == [0, 5, 6]
    assert plain.select(x, 3, 5, 1, 2).tolist() == [0, 1, 2, -1, -1]
    x[6] = np.nan
    assert plain.select(x, 7, 6, 0, 0).tolist() == [0, 1, 2, 3, 4, 5]
    x[:] = [0.0, -0.0, 0.0, -0.0, np.nan, -np.inf, np.nan]
    assert plain.select(x, 7, 2, 0, 0).tolist() == [0, 1]
    assert plain.select(x, 7, 5, 0, 0).tolist() == [0, 1, 2, 3, 5]


def test_plain_attention_is_a_softmax():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 4, 1, 16, 8))
    table = [3, 1, 0]
    out, mag = plain.attend_row(np.zeros((2, 8)), k, v, table, 0, [0, 17, 33], 0.5)
    assert np.allclose(out, np.mean([v[3, 0, 0], v[1, 0, 1], v[0, 0, 1]], 0)) and (mag >= np.abs(out)).all()
    assert plain.path([-1, 0, 0, 2, 3], 4) == [4, 3, 2, 0]


def test_attention_needs_a_cache(lib):
    shared = N.SvSharedPrefix(1, A, A)
    none = kv(num_blocks=0)
    assert lib.sv_page_attend_workspace(ref(batch()), ref(none), 8, 3) == 0
    assert lib.sv_prefix_attend_workspace(ref(batch()), ref(none), ref(shared), 8) == 0
    assert lib.sv_page_attend(ref(none), ref(batch()), A, 8, 0.1, A, 3, OUT, A, 1 << 40, None, None) == INV
    assert lib.sv_prefix_attend(ref(none), ref(batch()), ref(shared), A, 8, 0.1, OUT, A, 1 << 40, None, None) == INV
