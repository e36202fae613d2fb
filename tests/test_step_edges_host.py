"""The step's two edges without a GPU: what the host refuses, and pins of the
oracle that the GPU tests compare with."""

import ctypes
import math

import numpy as np
import pytest

from oracle import edges
from speculative_decoding_verification_padding_gb300 import _native as N
from speculative_decoding_verification_padding_gb300 import workloads as wl
from speculative_decoding_verification_padding_gb300.step import unstaged

BAD, SHAPE = N.SV_ERR_INVALID_ARGUMENT, N.SV_ERR_UNSUPPORTED_SHAPE
A = 4096  # stands for a device pointer: nothing is enqueued before it is refused


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_padding_gb300 import build
    build.build()
    return N.lib()


def _kv(**over):
    a = dict(k_cache=A, v_cache=A, num_blocks=10, block_size=16, n_kv_heads=2, head_dim=64, block_tables=A,
             max_blocks_per_req=4, cache_lens=A)
    a.update(over)
    return N.SvPagedKV(*(a[n] for n, _ in N.SvPagedKV._fields_))


def _batch(**over):
    a = dict(n_req=2, total_rows=6, max_rows_per_req=4, cu_rows=A, parent=A, tokens=A, row_begin=None,
             row_end=None, verify_len=None)
    a.update(over)
    return N.SvBatch(*(a[n] for n, _ in N.SvBatch._fields_))


def test_reserve_refuses(lib):
    pool = N.SvBlockPool(A, A, 10)

    def call(kv=_kv(), b=_batch(), p=pool, slots=A, taken=A):
        ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return lib.sv_reserve_kv(ref(kv), ref(b), ref(p), None, slots, A, taken, None, None)

    assert call(kv=None) == call(b=None) == call(p=None) == BAD
    assert call(slots=None) == call(taken=None) == BAD
    for kv in (dict(block_tables=None), dict(cache_lens=None), dict(num_blocks=-1), dict(max_blocks_per_req=-1)):
        assert call(kv=_kv(**kv)) == BAD, kv
    for kv in (dict(block_size=32), dict(num_blocks=1 << 28), dict(max_blocks_per_req=1 << 28)):
        assert call(kv=_kv(**kv)) == SHAPE, kv
    for b in (dict(n_req=-1), dict(total_rows=-1), dict(max_rows_per_req=0), dict(cu_rows=None)):
        assert call(b=_batch(**b)) == BAD, b
    assert call(b=_batch(max_rows_per_req=129)) == SHAPE  # a tree; without parents a chain may be longer
    assert call(b=_batch(n_req=8193)) == SHAPE
    for p in ((None, A, 10), (A, None, 10), (A, A, -1)):
        assert call(p=N.SvBlockPool(*p)) == BAD, p
    assert call(b=_batch(n_req=0, total_rows=0)) == N.SV_OK


def test_reserve_refuses_what_its_counts_cannot_hold(lib):
    # requests times the table entries that each may span: counted in 32 bits
    # (offsets that overlap could reach it, whatever the number of rows)
    def call(n_req, max_rows, entries):
        kv, b = _kv(max_blocks_per_req=entries), _batch(n_req=n_req, max_rows_per_req=max_rows, parent=None,
                                                        total_rows=1 << 30)
        return lib.sv_reserve_kv(ctypes.byref(kv), ctypes.byref(b), ctypes.byref(N.SvBlockPool(A, A, 10)), None,
                                 None, A, A, None, None)  # without slots it stops behind the check

    assert call(8192, 1 << 30, 1 << 26) == call(32, 1 << 30, (1 << 27) - 1) == call(8192, 1 << 23, 1 << 19) == SHAPE
    assert call(8192, 1 << 30, 1 << 17) == call(8192, 1 << 21, 1 << 26) == call(31, 1 << 30, (1 << 27) - 1) == BAD


def test_stage_refuses(lib):
    half = N.SvRotary(A, 64, 0, 1, None, 1.0)

    def call(kv=_kv(), rows=3, q=A, qs=256, k=1 << 20, ks=128, v=1 << 21, vs=128, heads=4, slots=A, pos=A,
             axis=0, rot=half, qw=A, kw=A, eps=1e-6, out=1 << 22):
        return lib.sv_stage_qkv(None if kv is None else ctypes.byref(kv), rows, q, qs, k, ks, v, vs, heads, slots,
                                pos, axis, None if rot is None else ctypes.byref(rot), qw, kw, eps, out, None, None)

    assert call(kv=None) == call(rows=-1) == call(heads=0) == call(kv=_kv(n_kv_heads=0)) == BAD
    assert call(kv=_kv(head_dim=96)) == call(kv=_kv(block_size=8)) == SHAPE
    for name in ("q", "k", "v", "slots", "pos", "out"):
        assert call(**{name: None}) == BAD, name
    assert call(kv=_kv(k_cache=None)) == call(kv=_kv(v_cache=None)) == BAD
    assert call(q=A + 8) == call(out=(1 << 22) + 4) == call(qw=A + 4) == call(kv=_kv(k_cache=A + 2)) == BAD
    assert call(qs=255) == call(qs=260) == call(ks=64) == call(vs=0) == call(axis=-1) == BAD
    assert call(eps=-1.0) == call(eps=math.nan) == BAD
    for rot, want in (((A, 24, 0, 1, None, 1.0), SHAPE), ((A, 80, 0, 1, None, 1.0), BAD),
                      ((A, -16, 0, 1, None, 1.0), BAD), ((None, 64, 0, 1, None, 1.0), BAD),
                      ((A, 64, 0, 0, None, 1.0), BAD), ((A, 64, 0, 3, None, 1.0), BAD),
                      ((A, 64, 0, 1, None, math.nan), BAD)):
        assert call(rot=N.SvRotary(*rot)) == want, rot
    assert call(out=A + 512) == call(out=1 << 20) == call(out=1 << 21) == BAD  # over q, k, v
    assert call(rows=0) == N.SV_OK


def test_shape_refuses(lib):
    def call(b=_batch(), x=1 << 20, kind=0, stride=100, V=100, out=1 << 24, rules=(), **r):
        ru = N.SvLogitRules(**{k: v for k, v in dict(rules, **r).items()})
        return lib.sv_shape_logits(None if b is None else ctypes.byref(b), x, kind, stride, V, ctypes.byref(ru), out,
                                   None, None)

    assert lib.sv_shape_logits(ctypes.byref(_batch()), A, 0, 100, 100, None, A, None, None) == BAD
    assert call(b=None) == call(V=0) == call(kind=2) == call(stride=99) == BAD
    assert call(x=None) == call(out=None) == call(b=_batch(cu_rows=None)) == BAD
    assert call(b=_batch(max_rows_per_req=129)) == SHAPE
    assert call(x=(1 << 20) + 2) == call(x=(1 << 20) + 1, kind=1) == call(out=(1 << 24) + 2) == BAD
    assert call(out=(1 << 20) + 400) == call(out=(1 << 20) - 4) == BAD  # overlap
    assert call(b=_batch(parent=None), repetition=A) == call(b=_batch(tokens=None), presence=A) == BAD
    assert call(history=A, max_history=4) == call(history=A, history_len=A, max_history=-1) == BAD
    assert call(bias_begin=A) == call(bias_begin=A, bias_token=A) == BAD
    assert call(bias_begin=A, bias_token=A, bias_value=A, n_bias=-1) == BAD
    assert call(mask=A, mask_stride=3, n_masks=6) == call(mask=A, mask_stride=4, n_masks=5) == BAD
    assert call(mask=A, mask_stride=4, n_masks=-1, mask_row=A) == BAD
    assert call(b=_batch(n_req=0)) == N.SV_OK


def test_binding_refuses_what_is_not_on_the_gpu():
    import torch
    from speculative_decoding_verification_padding_gb300 import api
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    page = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    kv = api.PagedKV(page, page.clone(), i(1, 2), i(1))
    b = api.Batch(i(2), torch.full((3,), -1, dtype=torch.int32), i(3), 3)
    x = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(N.SpecVerifyError):
        api.bind_reserve_kv(kv, b, api.BlockPool(i(4), i(1)), i(3), i(3), i(1))
    with pytest.raises(N.SpecVerifyError, match="at least"):
        api.bind_reserve_kv(kv, b, api.BlockPool(i(4), i(1)), i(2), i(3), i(1))
    with pytest.raises(N.SpecVerifyError):
        api.bind_stage_qkv(kv, x, x, x, i(3), None, None, x.clone())
    with pytest.raises(N.SpecVerifyError):
        api.bind_shape_logits(b, torch.zeros(3, 9), api.LogitRules(), torch.zeros(3, 9))
    assert api.Batch(i(2), None, i(5), 5).total_rows == 5


# ------------------------------------------------------------ oracle pins --

def test_oracle_reserve_by_hand():
    # 20 cached tokens and 13 rows: slots 20 .. 32, one entry there, one new
    tables = np.array([[4, 7, -1, -1], [1, -1, -1, -1], [-1, -1, -1, -1]], np.int32)
    err, s = edges.reserve([0, 13, 14, 47], [-1, 0, 0] + list(range(2, 12)) + [-1] + list(range(-1, 32)), [20, 5, 0],
                           tables, [9, 8, 6, 0], 3, 10, 40, 48, pos_offset=[100, 0, 0])
    assert err == edges.POOL_EMPTY  # request 2 asks for three blocks, two are left
    assert s["taken"].tolist() == [1, 0, -1] and s["count"] == 2
    assert s["tables"].tolist() == [[4, 7, 6, -1], [1, -1, -1, -1], [-1] * 4]
    assert s["slots"][:14].tolist() == list(range(7 * 16 + 4, 7 * 16 + 16)) + [6 * 16] + [16 + 5]
    assert s["positions"][:14].tolist() == [120, 121, 121] + list(range(122, 132)) + [5]
    assert (s["slots"][14:] == -1).all() and (s["positions"][14:] == -1).all()


def test_oracle_stage_turns_and_norms():
    x = np.zeros((1, 1, 8))
    x[0, 0] = [1, 0, 2, 0, 5, 6, 7, 8]
    y, _ = edges.stage(x, None, 0.0, np.array([[3]]), [math.pi / 6, math.pi / 12], 4)
    # pairs (0, 2) by 90 degrees, (1, 3) by 45; the rest as it was
    np.testing.assert_allclose(y[0, 0], [-2, 0, 1, 0, 5, 6, 7, 8], atol=1e-15)
    y, _ = edges.stage(x, None, 0.0, np.array([[3], [6]]), [math.pi / 6, math.pi / 12], 4, [0, 1], True, 2.0)
    np.testing.assert_allclose(y[0, 0], [0, 2, 0, 4, 5, 6, 7, 8], atol=1e-14)
    y, _ = edges.stage(x, np.full(8, 3.0), 1.0, np.array([[0]]), [], 0)
    np.testing.assert_allclose(y[0, 0], 3 * x[0, 0] / math.sqrt(179 / 8 + 1))


def test_oracle_shape_by_hand():
    logits = np.array([[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]])
    y, _ = edges.shape_logits([0, 2], [-1, 0], [3, 1], logits, history=[[0, 2, 2, 3, 9]], history_len=[4],
                              prompt_len=[1], repetition=[2.0], frequency=[0.5], presence=[0.25],
                              bias_begin=[0, 2], bias_token=[3, 3], bias_value=[1.0, 9.0],
                              mask=np.array([[0b1011], [0]], np.int32), mask_row=[0, 1])
    # token 0 asked for, 2 said twice, 3 once; row 1's path adds token 1
    np.testing.assert_allclose(y[0], [1.0, -2.0, -np.inf, 0.25 - 0.75 + 1.0])
    np.testing.assert_allclose(y[1], [1.0, -4.0 - 0.75, 0.5 - 1.25, 0.5])  # a mask of nothing is none


def test_unstaged_workload_holds_the_same_blocks():
    w = wl.make_workload(wl.config("batch64"), n_req=9, ctx_scale=0.01, vocab=64)
    u = unstaged(w)
    for i in range(w.n_req):
        have = -(-int(w.cache_lens[i]) // 16)
        assert (u.block_tables[i, :have] == w.block_tables[i, :have]).all() and (u.block_tables[i, have:] == -1).all()
    held = u.block_tables[u.block_tables >= 0].tolist() + u.free_list[:u.free_count].tolist()
    assert len(held) == len(set(held)) == (w.block_tables >= 0).sum() + w.free_count
    assert (w.block_tables >= 0).sum() > (u.block_tables >= 0).sum()  # the workload itself is as it was
