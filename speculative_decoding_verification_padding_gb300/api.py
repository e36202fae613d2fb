"""Python binding of libspecverify for torch tensors.

Every function has the name of the C call it marshals and runs nothing but
that call: torch provides device memory and the current stream.  Tensors
must live on the current CUDA device; results land in the tensors passed in.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _native as N


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise N.SpecVerifyError("libspecverify takes device tensors")
    if not t.is_contiguous():
        raise N.SpecVerifyError("libspecverify takes contiguous tensors")
    return t.data_ptr()


def _expect(t: Optional[torch.Tensor], dtype, name):
    if t is not None and t.dtype != dtype:
        raise N.SpecVerifyError(f"{name} must be {dtype}, got {t.dtype}")


def _at_least(t: Optional[torch.Tensor], n: int, name):
    if t is not None and t.numel() < n:
        raise N.SpecVerifyError(f"{name} must hold at least {n} elements, got {t.numel()}")


def _one_device(*tensors) -> torch.device:
    """The device of all the tensors, which must be the current one: a call
    is launched there."""
    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise N.SpecVerifyError(f"tensors of one call live on {sorted(map(str, devs))}")
    dev = devs.pop()
    if dev.type != "cuda":
        raise N.SpecVerifyError("libspecverify takes device tensors")
    if dev.index != torch.cuda.current_device():
        raise N.SpecVerifyError(f"tensors live on {dev}, the current device is "
                                f"cuda:{torch.cuda.current_device()}")
    return dev


def _rows_ptr(t: torch.Tensor, name):
    """Pointer and row stride of a [rows][heads][dim] or [rows][columns] tensor
    whose rows are dense and may lie apart (a view of a wider tensor)."""
    if not t.is_cuda:
        raise N.SpecVerifyError("libspecverify takes device tensors")
    dense = 1
    for size, step in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and step != dense:
            raise N.SpecVerifyError(f"{name}: the elements of a row must be dense")
        dense *= size
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else dense)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# The current stream's handle for a device index, without building a Stream
# object (a few microseconds less per call on the launch path).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _current_stream(device_index: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device_index)
    return torch.cuda.current_stream(device_index).cuda_stream


def _call(name: str, args: tuple, stream):
    N.check(getattr(N.lib(), name)(*args, _stream(stream)), name)


class BoundCall:
    """One library call with its arguments marshalled once: the dtypes
    checked, the structs built and the device pointers taken.  Calling it
    enqueues the call on the current stream of the bound tensors' device (or
    on `stream`).  The tensors it was bound to must stay allocated, and the
    Batch / PagedKV / BlockPool objects must keep the same tensors: the
    call reads their pointers as they were when it was bound."""

    __slots__ = ("_f", "_name", "_args", "_dev", "_keep")

    def __init__(self, name: str, args: tuple, device: torch.device, keep=None):
        self._f = getattr(N.lib(), name)
        self._name = name
        # Numbers become ctypes values once, not at every call; ctypes byref
        # objects keep their structs alive.
        self._args = tuple(t(a) if isinstance(a, (int, float)) else a
                           for t, a in zip(N.PROTOTYPES[name][1], args))
        self._keep = keep  # what the call's tensors belong to, where the binder hands it over
        self._dev = device.index if device.index is not None else torch.cuda.current_device()

    def __call__(self, stream=None):
        if _current_device() != self._dev:
            raise N.SpecVerifyError(f"{self._name} is bound to cuda:{self._dev}, the current device "
                                    f"is cuda:{_current_device()}")
        st = _current_stream(self._dev) if stream is None else _stream(stream)
        status = self._f(*self._args, st)
        if status != N.SV_OK:
            N.check(status, self._name)


@dataclass
class Batch:
    """sv_batch: packed draft chains / trees (int32 device tensors)."""
    cu_rows: torch.Tensor
    parent: Optional[torch.Tensor]
    tokens: torch.Tensor
    max_rows: int
    row_begin: Optional[torch.Tensor] = None
    row_end: Optional[torch.Tensor] = None
    verify_len: Optional[torch.Tensor] = None

    @property
    def n_req(self):
        return self.cu_rows.shape[0] - 1

    @property
    def total_rows(self):
        # sv_reserve_kv takes chains without parents
        return (self.tokens if self.parent is None else self.parent).shape[0]

    def c(self) -> N.SvBatch:
        for name in ("cu_rows", "parent", "tokens", "row_begin", "row_end", "verify_len"):
            _expect(getattr(self, name), torch.int32, name)
        return N.SvBatch(self.n_req, self.total_rows, self.max_rows, _ptr(self.cu_rows),
                         _ptr(self.parent), _ptr(self.tokens), _ptr(self.row_begin),
                         _ptr(self.row_end), _ptr(self.verify_len))


@dataclass
class PagedKV:
    """sv_paged_kv: bf16 [num_blocks][n_kv][16][d] caches, int32 tables."""
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    block_tables: torch.Tensor
    cache_lens: torch.Tensor

    def c(self) -> N.SvPagedKV:
        _expect(self.k_cache, torch.bfloat16, "k_cache")
        _expect(self.v_cache, torch.bfloat16, "v_cache")
        _expect(self.block_tables, torch.int32, "block_tables")
        _expect(self.cache_lens, torch.int32, "cache_lens")
        nb, hkv, bs, d = self.k_cache.shape
        return N.SvPagedKV(_ptr(self.k_cache), _ptr(self.v_cache), nb, bs, hkv, d,
                           _ptr(self.block_tables), self.block_tables.shape[1],
                           _ptr(self.cache_lens))


@dataclass
class BlockPool:
    """sv_block_pool: free list and its count (int32 device tensors)."""
    free_list: torch.Tensor
    free_count: torch.Tensor

    def c(self) -> N.SvBlockPool:
        _expect(self.free_list, torch.int32, "free_list")
        _expect(self.free_count, torch.int32, "free_count")
        return N.SvBlockPool(_ptr(self.free_list), _ptr(self.free_count), self.free_list.shape[0])


@dataclass
class Rotary:
    """sv_rotary: the rotation of Q and K heads.  inv_freq fp32
    [rotary_dim / 2]; freq_axis int32 [rotary_dim / 2] names the position axis
    of each pair (with positions of several axes)."""
    inv_freq: torch.Tensor
    rotary_dim: int
    freq_axis: Optional[torch.Tensor] = None
    interleaved: bool = False
    scale: float = 1.0

    def c(self, n_axes: int) -> N.SvRotary:
        _expect(self.inv_freq, torch.float32, "inv_freq")
        _expect(self.freq_axis, torch.int32, "freq_axis")
        half = self.rotary_dim // 2
        _at_least(self.inv_freq, half, "inv_freq")
        _at_least(self.freq_axis, half, "freq_axis")
        return N.SvRotary(_ptr(self.inv_freq), self.rotary_dim, int(self.interleaved), n_axes,
                          _ptr(self.freq_axis), float(self.scale))


@dataclass
class LogitRules:
    """sv_logit_rules: what shapes a request's logits; every part may be left
    out.  history int32 [n_req][max_history] with history_len / prompt_len
    int32 [n_req]; repetition, frequency, presence fp32 [n_req]; biases as one
    packed list with offsets bias_begin [n_req + 1]; mask int32 words
    [n_masks][words] with mask_row int32 [total_rows]."""
    history: Optional[torch.Tensor] = None
    history_len: Optional[torch.Tensor] = None
    prompt_len: Optional[torch.Tensor] = None
    repetition: Optional[torch.Tensor] = None
    frequency: Optional[torch.Tensor] = None
    presence: Optional[torch.Tensor] = None
    bias_begin: Optional[torch.Tensor] = None
    bias_token: Optional[torch.Tensor] = None
    bias_value: Optional[torch.Tensor] = None
    mask: Optional[torch.Tensor] = None
    mask_row: Optional[torch.Tensor] = None

    def c(self, n_req: int, total_rows: int,
          row_end: Optional[torch.Tensor] = None) -> N.SvLogitRules:
        for name in ("history", "history_len", "prompt_len", "bias_begin", "bias_token", "mask",
                     "mask_row"):
            _expect(getattr(self, name), torch.int32, name)
        for name in ("repetition", "frequency", "presence", "bias_value"):
            _expect(getattr(self, name), torch.float32, name)
        for name in ("history_len", "prompt_len", "repetition", "frequency", "presence"):
            _at_least(getattr(self, name), n_req, name)
        _at_least(self.bias_begin, n_req + 1, "bias_begin")
        _at_least(self.mask_row, total_rows, "mask_row")
        hist, mask = self.history, self.mask
        if hist is not None and (hist.dim() != 2 or hist.shape[0] < n_req):
            raise N.SpecVerifyError(f"history must be [{n_req}][max_history], got {tuple(hist.shape)}")
        if mask is not None and mask.dim() != 2:
            raise N.SpecVerifyError(f"mask must be [n_masks][words], got {tuple(mask.shape)}")
        if mask is not None and self.mask_row is None and mask.shape[0] < total_rows:
            raise N.SpecVerifyError(f"mask has {mask.shape[0]} rows for {total_rows} rows without mask_row")
        masks = _ptr(mask)
        if mask is not None and mask.shape[0] == 0 and self.mask_row is not None:
            masks = _ptr(self.mask_row)  # no address of its own; none of it is read
        n_bias = 0
        token, value = _ptr(self.bias_token), _ptr(self.bias_value)
        if self.bias_begin is not None and self.bias_token is not None:
            n_bias = self.bias_token.numel()
            _at_least(self.bias_value, n_bias, "bias_value")
            if n_bias == 0 and self.bias_value is not None:
                # an empty list has no address; none of it is read
                token = value = _ptr(self.bias_begin)
        return N.SvLogitRules(
            _ptr(hist), 0 if hist is None else hist.shape[1], _ptr(self.history_len),
            _ptr(self.prompt_len), _ptr(self.repetition), _ptr(self.frequency),
            _ptr(self.presence), _ptr(self.bias_begin), token, value, n_bias, masks,
            0 if mask is None else mask.shape[1], 0 if mask is None else mask.shape[0],
            _ptr(self.mask_row), _ptr(row_end))


@dataclass
class SharedPrefix:
    """sv_shared_prefix: requests cu_groups[k] .. cu_groups[k + 1] - 1 share their
    first prefix_len[k] cache slots (int32 device tensors)."""
    cu_groups: torch.Tensor
    prefix_len: torch.Tensor

    @property
    def n_groups(self):
        return self.cu_groups.shape[0] - 1

    def c(self) -> N.SvSharedPrefix:
        _expect(self.cu_groups, torch.int32, "cu_groups")
        _expect(self.prefix_len, torch.int32, "prefix_len")
        _at_least(self.prefix_len, self.n_groups, "prefix_len")
        return N.SvSharedPrefix(self.n_groups, _ptr(self.cu_groups), _ptr(self.prefix_len))


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A 256-byte aligned device buffer of at least nbytes (torch allocations are)."""
    return torch.empty(max(1, nbytes), dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------ calls --

def sv_tree_attend_workspace(batch: Batch, kv: PagedKV, n_q_heads: int) -> int:
    b, k = batch.c(), kv.c()
    return N.lib().sv_tree_attend_workspace(ctypes.byref(b), ctypes.byref(k), n_q_heads)


def _tree_attend_args(kv, batch, q, n_q_heads, softmax_scale, out, ws, dev_status):
    _expect(q, torch.bfloat16, "q")
    _expect(out, torch.bfloat16, "out")
    b, k = batch.c(), kv.c()
    return (ctypes.byref(k), ctypes.byref(b), _ptr(q), n_q_heads, softmax_scale, _ptr(out),
            _ptr(ws), ws.numel(), _ptr(dev_status))


def sv_tree_attend(kv: PagedKV, batch: Batch, q: torch.Tensor, n_q_heads: int,
                   softmax_scale: float, out: torch.Tensor, ws: torch.Tensor,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    _call("sv_tree_attend",
          _tree_attend_args(kv, batch, q, n_q_heads, softmax_scale, out, ws, dev_status), stream)


def bind_tree_attend(kv: PagedKV, batch: Batch, q: torch.Tensor, n_q_heads: int,
                     softmax_scale: float, out: torch.Tensor, ws: torch.Tensor,
                     dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_tree_attend with its arguments marshalled once (see BoundCall)."""
    return BoundCall("sv_tree_attend",
                     _tree_attend_args(kv, batch, q, n_q_heads, softmax_scale, out, ws,
                                       dev_status), q.device)


def sv_accept_workspace(batch: Batch, vocab: int) -> int:
    b = batch.c()
    return N.lib().sv_accept_workspace(ctypes.byref(b), vocab)


def sv_accept(batch: Batch, target_logits: torch.Tensor, draft_logits: Optional[torch.Tensor],
              vocab: int, temperature: float, seed: int, accepted_len: torch.Tensor,
              accepted_nodes: torch.Tensor, next_token: torch.Tensor, ambiguous: torch.Tensor,
              done: Optional[torch.Tensor], row_stats: Optional[torch.Tensor], ws: torch.Tensor,
              dev_status: Optional[torch.Tensor] = None, stream=None):
    _call("sv_accept",
          _accept_args(batch, target_logits, draft_logits, vocab, temperature, seed, accepted_len,
                       accepted_nodes, next_token, ambiguous, done, row_stats, ws, dev_status),
          stream)


def _accept_args(batch, target_logits, draft_logits, vocab, temperature, seed, accepted_len,
                 accepted_nodes, next_token, ambiguous, done, row_stats, ws, dev_status):
    _expect(target_logits, torch.float32, "target_logits")
    _expect(draft_logits, torch.float32, "draft_logits")
    _expect(ambiguous, torch.uint8, "ambiguous")
    _expect(row_stats, torch.float32, "row_stats")
    b = batch.c()
    return (ctypes.byref(b), _ptr(target_logits), _ptr(draft_logits), vocab, temperature,
            seed & 0xFFFFFFFFFFFFFFFF, _ptr(accepted_len), _ptr(accepted_nodes),
            _ptr(next_token), _ptr(ambiguous), _ptr(done), _ptr(row_stats), _ptr(ws), ws.numel(),
            _ptr(dev_status))


def bind_accept(batch: Batch, target_logits: torch.Tensor,
                draft_logits: Optional[torch.Tensor], vocab: int, temperature: float, seed: int,
                accepted_len: torch.Tensor, accepted_nodes: torch.Tensor,
                next_token: torch.Tensor, ambiguous: torch.Tensor, done: Optional[torch.Tensor],
                row_stats: Optional[torch.Tensor], ws: torch.Tensor,
                dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_accept with its arguments marshalled once (see BoundCall)."""
    return BoundCall("sv_accept",
                     _accept_args(batch, target_logits, draft_logits, vocab, temperature, seed,
                                  accepted_len, accepted_nodes, next_token, ambiguous, done,
                                  row_stats, ws, dev_status), target_logits.device)


def sv_accept_static(batch: Batch, target_logits: torch.Tensor,
                     draft_logits: Optional[torch.Tensor], vocab: int, temperature: float,
                     seed: int, accepted_len: torch.Tensor, accepted_nodes: torch.Tensor,
                     next_token: torch.Tensor, ambiguous: torch.Tensor,
                     done: Optional[torch.Tensor], row_stats: Optional[torch.Tensor],
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    """sv_accept for callers that cannot allocate a workspace: the scratch is
    a fixed device array inside the library (see the header for its limit
    and for why concurrent calls must not overlap)."""
    _expect(target_logits, torch.float32, "target_logits")
    _expect(draft_logits, torch.float32, "draft_logits")
    _expect(ambiguous, torch.uint8, "ambiguous")
    _expect(row_stats, torch.float32, "row_stats")
    b = batch.c()
    N.check(N.lib().sv_accept_static(ctypes.byref(b), _ptr(target_logits), _ptr(draft_logits),
                                     vocab, temperature, seed & 0xFFFFFFFFFFFFFFFF,
                                     _ptr(accepted_len), _ptr(accepted_nodes), _ptr(next_token),
                                     _ptr(ambiguous), _ptr(done), _ptr(row_stats),
                                     _ptr(dev_status), _stream(stream)), "sv_accept_static")


def sv_commit_kv(kv: PagedKV, batch: Batch, accepted_len: torch.Tensor,
                 accepted_nodes: torch.Tensor, pool: BlockPool,
                 dev_status: Optional[torch.Tensor] = None, stream=None):
    b, k, p = batch.c(), kv.c(), pool.c()
    N.check(N.lib().sv_commit_kv(ctypes.byref(k), ctypes.byref(b), _ptr(accepted_len),
                                 _ptr(accepted_nodes), ctypes.byref(p), _ptr(dev_status),
                                 _stream(stream)), "sv_commit_kv")


def sv_accept_commit_workspace(batch: Batch, vocab: int) -> int:
    b = batch.c()
    return N.lib().sv_accept_commit_workspace(ctypes.byref(b), vocab)


def sv_accept_commit(batch: Batch, target_logits: torch.Tensor,
                     draft_logits: Optional[torch.Tensor], vocab: int, temperature: float,
                     seed: int, accepted_len: torch.Tensor, accepted_nodes: torch.Tensor,
                     next_token: torch.Tensor, ambiguous: torch.Tensor,
                     done: Optional[torch.Tensor], row_stats: Optional[torch.Tensor],
                     kv: PagedKV, pool: BlockPool, ws: torch.Tensor,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    _call("sv_accept_commit",
          _accept_commit_args(batch, target_logits, draft_logits, vocab, temperature, seed,
                              accepted_len, accepted_nodes, next_token, ambiguous, done,
                              row_stats, kv, pool, ws, dev_status), stream)


def _accept_commit_args(batch, target_logits, draft_logits, vocab, temperature, seed,
                        accepted_len, accepted_nodes, next_token, ambiguous, done, row_stats, kv,
                        pool, ws, dev_status):
    _expect(target_logits, torch.float32, "target_logits")
    _expect(draft_logits, torch.float32, "draft_logits")
    _expect(ambiguous, torch.uint8, "ambiguous")
    _expect(row_stats, torch.float32, "row_stats")
    b, k, p = batch.c(), kv.c(), pool.c()
    return (ctypes.byref(b), _ptr(target_logits), _ptr(draft_logits), vocab, temperature,
            seed & 0xFFFFFFFFFFFFFFFF, _ptr(accepted_len), _ptr(accepted_nodes),
            _ptr(next_token), _ptr(ambiguous), _ptr(done), _ptr(row_stats), ctypes.byref(k),
            ctypes.byref(p), _ptr(ws), ws.numel(), _ptr(dev_status))


def bind_accept_commit(batch: Batch, target_logits: torch.Tensor,
                       draft_logits: Optional[torch.Tensor], vocab: int, temperature: float,
                       seed: int, accepted_len: torch.Tensor, accepted_nodes: torch.Tensor,
                       next_token: torch.Tensor, ambiguous: torch.Tensor,
                       done: Optional[torch.Tensor], row_stats: Optional[torch.Tensor],
                       kv: PagedKV, pool: BlockPool, ws: torch.Tensor,
                       dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_accept_commit with its arguments marshalled once (see BoundCall)."""
    return BoundCall("sv_accept_commit",
                     _accept_commit_args(batch, target_logits, draft_logits, vocab, temperature,
                                         seed, accepted_len, accepted_nodes, next_token,
                                         ambiguous, done, row_stats, kv, pool, ws, dev_status),
                     target_logits.device)


def sv_select_budget_workspace(n_req: int, gamma_max: int) -> int:
    return N.lib().sv_select_budget_workspace(n_req, gamma_max)


def sv_select_budget(cond_survival: torch.Tensor, gamma: Optional[torch.Tensor],
                     sps: torch.Tensor, verify_len: torch.Tensor, best_B: torch.Tensor,
                     best_theta: torch.Tensor, ws: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    _expect(cond_survival, torch.float32, "cond_survival")
    _expect(sps, torch.float32, "sps")
    _expect(best_theta, torch.float64, "best_theta")
    R, gmax = cond_survival.shape
    _call("sv_select_budget",
          (R, gmax, _ptr(cond_survival), _ptr(gamma), _ptr(sps), sps.shape[0] - 1,
           _ptr(verify_len), _ptr(best_B), _ptr(best_theta), _ptr(ws),
           0 if ws is None else ws.numel(), _ptr(dev_status)), stream)


def bind_select_budget(cond_survival: torch.Tensor, gamma: Optional[torch.Tensor],
                       sps: torch.Tensor, verify_len: torch.Tensor, best_B: torch.Tensor,
                       best_theta: torch.Tensor, ws: Optional[torch.Tensor] = None,
                       dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_select_budget with its arguments marshalled once (see BoundCall)."""
    _expect(cond_survival, torch.float32, "cond_survival")
    _expect(sps, torch.float32, "sps")
    _expect(best_theta, torch.float64, "best_theta")
    R, gmax = cond_survival.shape
    return BoundCall("sv_select_budget",
                     (R, gmax, _ptr(cond_survival), _ptr(gamma), _ptr(sps), sps.shape[0] - 1,
                      _ptr(verify_len), _ptr(best_B), _ptr(best_theta), _ptr(ws),
                      0 if ws is None else ws.numel(), _ptr(dev_status)), cond_survival.device)


def sv_adapt_gamma(accepted_len: torch.Tensor, verified: torch.Tensor, state: torch.Tensor,
                   gamma_next: torch.Tensor, decay: float = 0.7, overhead: float = 2.0,
                   gamma_min: int = 1, gamma_max: int = 8,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    _expect(accepted_len, torch.int32, "accepted_len")
    _expect(verified, torch.int32, "verified")
    _expect(state, torch.float64, "state")
    _expect(gamma_next, torch.int32, "gamma_next")
    N.check(N.lib().sv_adapt_gamma(accepted_len.numel(), _ptr(accepted_len), _ptr(verified),
                                   _ptr(state), _ptr(gamma_next), float(decay), float(overhead),
                                   int(gamma_min), int(gamma_max), _ptr(dev_status),
                                   _stream(stream)), "sv_adapt_gamma")


def sv_select_chunk(rows: torch.Tensor, ctx: torch.Tensor, state: torch.Tensor,
                    kv_bytes: float, row_bytes: float, chunk_bytes: int, chunk: torch.Tensor,
                    cost: torch.Tensor, costs: torch.Tensor,
                    dev_status: Optional[torch.Tensor] = None, stream=None):
    _expect(rows, torch.int32, "rows")
    _expect(ctx, torch.int32, "ctx")
    _expect(state, torch.float64, "state")
    _expect(chunk, torch.int32, "chunk")
    # cost and costs hold u64 values: any 8-byte integer tensor will do
    if cost.numel() < 1 or cost.element_size() != 8 or cost.is_floating_point():
        raise N.SpecVerifyError("cost: one 8-byte integer")
    if costs.numel() < 128 or costs.element_size() != 8 or costs.is_floating_point():
        raise N.SpecVerifyError("costs: 128 8-byte integers")
    N.check(N.lib().sv_select_chunk(rows.numel(), _ptr(rows), _ptr(ctx), _ptr(state),
                                    float(kv_bytes), float(row_bytes), int(chunk_bytes),
                                    _ptr(chunk), _ptr(cost), _ptr(costs), _ptr(dev_status),
                                    _stream(stream)), "sv_select_chunk")


def sv_selftest_bounded_wait(limit: int, dev_status: torch.Tensor, stream=None):
    _expect(dev_status, torch.int32, "dev_status")
    N.check(N.lib().sv_selftest_bounded_wait(int(limit), _ptr(dev_status), _stream(stream)),
            "sv_selftest_bounded_wait")


def sv_chunk_windows(batch: Batch, chunk_index: int, chunk_size: int,
                     done: Optional[torch.Tensor], row_begin: torch.Tensor,
                     row_end: torch.Tensor, stream=None):
    b = batch.c()
    N.check(N.lib().sv_chunk_windows(ctypes.byref(b), chunk_index, chunk_size, _ptr(done),
                                     _ptr(row_begin), _ptr(row_end), _stream(stream)),
            "sv_chunk_windows")


def sv_verify_chunked_workspace(batch: Batch, kv: PagedKV, n_q_heads: int, vocab: int) -> int:
    b, k = batch.c(), kv.c()
    return N.lib().sv_verify_chunked_workspace(ctypes.byref(b), ctypes.byref(k), n_q_heads, vocab)


def sv_verify_chunked(kv: PagedKV, batch: Batch, q: torch.Tensor, n_q_heads: int,
                      softmax_scale: float, out: torch.Tensor, target_logits: torch.Tensor,
                      draft_logits: Optional[torch.Tensor], vocab: int, temperature: float,
                      seed: int, chunk_size: int, accepted_len: torch.Tensor,
                      accepted_nodes: torch.Tensor, next_token: torch.Tensor,
                      ambiguous: torch.Tensor, done: torch.Tensor, ws: torch.Tensor,
                      dev_status: Optional[torch.Tensor] = None, stream=None):
    b, k = batch.c(), kv.c()
    _call("sv_verify_chunked",
          (ctypes.byref(k), ctypes.byref(b), _ptr(q), n_q_heads, softmax_scale, _ptr(out),
           _ptr(target_logits), _ptr(draft_logits), vocab, temperature,
           seed & 0xFFFFFFFFFFFFFFFF, chunk_size, _ptr(accepted_len), _ptr(accepted_nodes),
           _ptr(next_token), _ptr(ambiguous), _ptr(done), _ptr(ws), ws.numel(),
           _ptr(dev_status)), stream)


def sv_verify_chunked_commit(kv: PagedKV, batch: Batch, q: torch.Tensor, n_q_heads: int,
                             softmax_scale: float, out: torch.Tensor,
                             target_logits: torch.Tensor, draft_logits: Optional[torch.Tensor],
                             vocab: int, temperature: float, seed: int, chunk_size: int,
                             accepted_len: torch.Tensor, accepted_nodes: torch.Tensor,
                             next_token: torch.Tensor, ambiguous: torch.Tensor,
                             done: torch.Tensor, pool: BlockPool, ws: torch.Tensor,
                             dev_status: Optional[torch.Tensor] = None, stream=None):
    _call("sv_verify_chunked_commit",
          _chunked_commit_args(kv, batch, q, n_q_heads, softmax_scale, out, target_logits,
                               draft_logits, vocab, temperature, seed, chunk_size, accepted_len,
                               accepted_nodes, next_token, ambiguous, done, pool, ws,
                               dev_status), stream)


def _chunked_commit_args(kv, batch, q, n_q_heads, softmax_scale, out, target_logits,
                         draft_logits, vocab, temperature, seed, chunk_size, accepted_len,
                         accepted_nodes, next_token, ambiguous, done, pool, ws, dev_status):
    b, k, p = batch.c(), kv.c(), pool.c()
    return (ctypes.byref(k), ctypes.byref(b), _ptr(q), n_q_heads, softmax_scale, _ptr(out),
            _ptr(target_logits), _ptr(draft_logits), vocab, temperature,
            seed & 0xFFFFFFFFFFFFFFFF, chunk_size, _ptr(accepted_len), _ptr(accepted_nodes),
            _ptr(next_token), _ptr(ambiguous), _ptr(done), ctypes.byref(p), _ptr(ws), ws.numel(),
            _ptr(dev_status))


def bind_verify_chunked_commit(kv: PagedKV, batch: Batch, q: torch.Tensor, n_q_heads: int,
                               softmax_scale: float, out: torch.Tensor,
                               target_logits: torch.Tensor,
                               draft_logits: Optional[torch.Tensor], vocab: int,
                               temperature: float, seed: int, chunk_size: int,
                               accepted_len: torch.Tensor, accepted_nodes: torch.Tensor,
                               next_token: torch.Tensor, ambiguous: torch.Tensor,
                               done: torch.Tensor, pool: BlockPool, ws: torch.Tensor,
                               dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_verify_chunked_commit with its arguments marshalled once (see BoundCall)."""
    return BoundCall("sv_verify_chunked_commit",
                     _chunked_commit_args(kv, batch, q, n_q_heads, softmax_scale, out,
                                          target_logits, draft_logits, vocab, temperature, seed,
                                          chunk_size, accepted_len, accepted_nodes, next_token,
                                          ambiguous, done, pool, ws, dev_status), q.device)


# --------------------------------------------------- the step's two edges --

def _reserve_args(kv, batch, pool, slots, positions, taken, pos_offset, dev_status):
    for name, t in (("slots", slots), ("positions", positions), ("taken", taken),
                    ("pos_offset", pos_offset), ("dev_status", dev_status)):
        _expect(t, torch.int32, name)
    n, rows = batch.n_req, batch.total_rows
    _at_least(slots, rows, "slots")
    _at_least(positions, rows, "positions")
    _at_least(batch.tokens, rows, "tokens")
    for name, t in (("taken", taken), ("pos_offset", pos_offset), ("cache_lens", kv.cache_lens)):
        _at_least(t, n, name)
    if kv.block_tables.shape[0] < n:
        raise N.SpecVerifyError(f"block_tables has {kv.block_tables.shape[0]} rows for {n} requests")
    dev = _one_device(batch.cu_rows, batch.parent, kv.block_tables, kv.cache_lens, pool.free_list,
                      pool.free_count, slots, positions, taken, pos_offset, dev_status)
    b, k, p = batch.c(), kv.c(), pool.c()
    return (ctypes.byref(k), ctypes.byref(b), ctypes.byref(p), _ptr(pos_offset), _ptr(slots),
            _ptr(positions), _ptr(taken), _ptr(dev_status)), dev


def sv_reserve_kv(kv: PagedKV, batch: Batch, pool: BlockPool, slots: torch.Tensor,
                  positions: Optional[torch.Tensor], taken: torch.Tensor,
                  pos_offset: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None):
    """Blocks for the batch's rows out of the pool: table entries, cache slots
    and positions.  batch.parent None: chains of any length (prompts)."""
    args, _ = _reserve_args(kv, batch, pool, slots, positions, taken, pos_offset, dev_status)
    _call("sv_reserve_kv", args, stream)


def bind_reserve_kv(kv: PagedKV, batch: Batch, pool: BlockPool, slots: torch.Tensor,
                    positions: Optional[torch.Tensor], taken: torch.Tensor,
                    pos_offset: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_reserve_kv with its arguments marshalled once (see BoundCall)."""
    args, dev = _reserve_args(kv, batch, pool, slots, positions, taken, pos_offset, dev_status)
    return BoundCall("sv_reserve_kv", args, dev,
                     (kv, batch, pool, slots, positions, taken, pos_offset, dev_status))


def _slot_windows_args(kv, batch, slots, row_end):
    _expect(slots, torch.int32, "slots")
    _expect(row_end, torch.int32, "row_end")
    _at_least(slots, batch.total_rows, "slots")
    _at_least(row_end, batch.n_req, "row_end")
    _at_least(batch.verify_len, batch.n_req, "verify_len")
    dev = _one_device(batch.cu_rows, batch.verify_len, slots, row_end)
    b, k = batch.c(), kv.c()
    return (ctypes.byref(k), ctypes.byref(b), _ptr(slots), _ptr(row_end)), dev


def sv_slot_windows(kv: PagedKV, batch: Batch, slots: torch.Tensor, row_end: torch.Tensor,
                    stream=None):
    """row_end [n_req]: all rows of a request whose rows all have cache slots, 0
    for any other.  As the batch's row_end it keeps what was not served out of
    the rest of the step."""
    args, _ = _slot_windows_args(kv, batch, slots, row_end)
    _call("sv_slot_windows", args, stream)


def bind_slot_windows(kv: PagedKV, batch: Batch, slots: torch.Tensor,
                      row_end: torch.Tensor) -> BoundCall:
    """sv_slot_windows with its arguments marshalled once (see BoundCall)."""
    args, dev = _slot_windows_args(kv, batch, slots, row_end)
    return BoundCall("sv_slot_windows", args, dev, (kv, batch, slots, row_end))


def _stage_args(kv, q, k, v, slots, positions, rotary, q_out, q_weight, k_weight, eps, dev_status):
    for name, t in (("q", q), ("k", k), ("v", v), ("q_out", q_out)):
        _expect(t, torch.bfloat16, name)
    for name, t in (("slots", slots), ("positions", positions), ("dev_status", dev_status)):
        _expect(t, torch.int32, name)
    _expect(q_weight, torch.float32, "q_weight")
    _expect(k_weight, torch.float32, "k_weight")
    nb, hkv, bs, d = kv.k_cache.shape
    if kv.v_cache.shape != kv.k_cache.shape:
        raise N.SpecVerifyError("k_cache and v_cache differ in shape")
    if q.dim() != 3 or q.shape[2] != d:
        raise N.SpecVerifyError(f"q must be [rows][heads][{d}], got {tuple(q.shape)}")
    rows, heads = q.shape[:2]
    for name, t, want in (("k", k, (rows, hkv, d)), ("v", v, (rows, hkv, d)),
                          ("q_out", q_out, (rows, heads, d))):
        if tuple(t.shape) != want:
            raise N.SpecVerifyError(f"{name} must be {list(want)}, got {list(t.shape)}")
    if slots.dim() != 1 or slots.shape[0] != rows:
        raise N.SpecVerifyError(f"slots must be [{rows}], got {list(slots.shape)}")
    _at_least(q_weight, d, "q_weight")
    _at_least(k_weight, d, "k_weight")
    n_axes, axis_stride = 1, 0
    if positions is not None:
        if positions.shape[-1] != rows or positions.dim() not in (1, 2):
            raise N.SpecVerifyError(f"positions must be [{rows}] or [axes][{rows}], got "
                                    f"{list(positions.shape)}")
        if positions.dim() == 2:
            n_axes, axis_stride = positions.shape[0], positions.shape[1]
    if rotary is not None and rotary.freq_axis is not None and n_axes == 1:
        # one position for every axis: the pairs' axes make no difference
        rotary = Rotary(rotary.inv_freq, rotary.rotary_dim, None, rotary.interleaved, rotary.scale)
    dev = _one_device(kv.k_cache, kv.v_cache, q, k, v, slots, positions, q_out, q_weight, k_weight,
                      dev_status, *(() if rotary is None else (rotary.inv_freq, rotary.freq_axis)))
    c = N.SvPagedKV(_ptr(kv.k_cache), _ptr(kv.v_cache), nb, bs, hkv, d, None, 0, None)
    _expect(kv.k_cache, torch.bfloat16, "k_cache")
    _expect(kv.v_cache, torch.bfloat16, "v_cache")
    (qp, qs), (kp, ks), (vp, vs) = _rows_ptr(q, "q"), _rows_ptr(k, "k"), _rows_ptr(v, "v")
    r = None if rotary is None else ctypes.byref(rotary.c(n_axes))
    return (ctypes.byref(c), rows, qp, qs, kp, ks, vp, vs, heads, _ptr(slots), _ptr(positions),
            axis_stride, r, _ptr(q_weight), _ptr(k_weight), float(eps), _ptr(q_out),
            _ptr(dev_status)), dev


def sv_stage_qkv(kv: PagedKV, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 slots: torch.Tensor, positions: Optional[torch.Tensor],
                 rotary: Optional[Rotary], q_out: torch.Tensor,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, dev_status: Optional[torch.Tensor] = None, stream=None):
    """Head norms and rotation of q and k, q into q_out, k and v into the cache
    pages of slots.  q, k, v: [rows][heads][dim], views of one packed
    projection output will do; positions: [rows] or [axes][rows]."""
    args, _ = _stage_args(kv, q, k, v, slots, positions, rotary, q_out, q_weight, k_weight, eps,
                          dev_status)
    _call("sv_stage_qkv", args, stream)


def bind_stage_qkv(kv: PagedKV, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   slots: torch.Tensor, positions: Optional[torch.Tensor],
                   rotary: Optional[Rotary], q_out: torch.Tensor,
                   q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_stage_qkv with its arguments marshalled once (see BoundCall)."""
    args, dev = _stage_args(kv, q, k, v, slots, positions, rotary, q_out, q_weight, k_weight, eps,
                            dev_status)
    return BoundCall("sv_stage_qkv", args, dev,
                     (kv, q, k, v, slots, positions, rotary, q_out, q_weight, k_weight, dev_status))


_LOGIT_TYPES = {torch.float32: N.SV_LOGITS_F32, torch.bfloat16: N.SV_LOGITS_BF16}


def _shape_args(batch, logits, rules, out, dev_status, row_end):
    _expect(out, torch.float32, "out")
    _expect(dev_status, torch.int32, "dev_status")
    _expect(row_end, torch.int32, "row_end")
    if logits.dtype not in _LOGIT_TYPES:
        raise N.SpecVerifyError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    n, rows = batch.n_req, batch.total_rows
    if logits.dim() != 2 or logits.shape != out.shape or out.shape[0] != rows:
        raise N.SpecVerifyError(f"logits and out must be [{rows}][vocab], got {list(logits.shape)} "
                                f"and {list(out.shape)}")
    _at_least(batch.tokens, rows, "tokens")
    _at_least(row_end, n, "row_end")
    for name in ("row_begin", "row_end", "verify_len"):
        _at_least(getattr(batch, name), n, name)
    dev = _one_device(batch.cu_rows, batch.parent, batch.tokens, batch.row_begin, batch.row_end,
                      batch.verify_len, logits, out, dev_status, row_end, *vars(rules).values())
    b, r = batch.c(), rules.c(n, rows, row_end)
    lp, stride = _rows_ptr(logits, "logits")
    return (ctypes.byref(b), lp, _LOGIT_TYPES[logits.dtype], stride, out.shape[1], ctypes.byref(r),
            _ptr(out), _ptr(dev_status)), dev


def sv_shape_logits(batch: Batch, logits: torch.Tensor, rules: LogitRules, out: torch.Tensor,
                    dev_status: Optional[torch.Tensor] = None, stream=None,
                    row_end: Optional[torch.Tensor] = None):
    """The logits [rows][vocab] (fp32 or bf16; rows may lie apart) under each
    request's penalties, biases and masks, into out (fp32; may be logits).
    row_end [n_req] becomes 0 for a request whose rules are malformed, whose rows
    are left as they were."""
    args, _ = _shape_args(batch, logits, rules, out, dev_status, row_end)
    _call("sv_shape_logits", args, stream)


def bind_shape_logits(batch: Batch, logits: torch.Tensor, rules: LogitRules, out: torch.Tensor,
                      dev_status: Optional[torch.Tensor] = None,
                      row_end: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_shape_logits with its arguments marshalled once (see BoundCall)."""
    args, dev = _shape_args(batch, logits, rules, out, dev_status, row_end)
    return BoundCall("sv_shape_logits", args, dev,
                     (batch, logits, rules, out, dev_status, row_end))


# --------------------------------------------- less of a long cache is read --

def _cache_shape(kv, what):
    if kv.v_cache.shape != kv.k_cache.shape:
        raise N.SpecVerifyError(f"{what}: k_cache and v_cache differ in shape")
    return kv.k_cache.shape


def _batch_fits(kv, batch):
    n = batch.n_req
    _at_least(batch.tokens, batch.total_rows, "tokens")
    for name in ("row_begin", "row_end", "verify_len"):
        _at_least(getattr(batch, name), n, name)
    _at_least(kv.cache_lens, n, "cache_lens")
    if kv.block_tables.shape[0] < n:
        raise N.SpecVerifyError(f"block_tables has {kv.block_tables.shape[0]} rows for {n} requests")


def _batch_tensors(batch):
    return (batch.cu_rows, batch.parent, batch.row_begin, batch.row_end, batch.verify_len)


def _queries(kv, batch, q):
    """The query heads of q, [rows][heads][dim] for the batch and the cache."""
    _expect(q, torch.bfloat16, "q")
    d = kv.k_cache.shape[3]
    if q.dim() != 3 or q.shape[0] != batch.total_rows or q.shape[2] != d:
        raise N.SpecVerifyError(f"q must be [{batch.total_rows}][heads][{d}], got {list(q.shape)}")
    return q.shape[1]


def _bound_args(kv, bounds, from_len, dev_status):
    _expect(bounds, torch.bfloat16, "bounds")
    _expect(from_len, torch.int32, "from_len")
    _expect(dev_status, torch.int32, "dev_status")
    nb, hkv, _, d = _cache_shape(kv, "sv_bound_pages")
    if tuple(bounds.shape) != (nb, hkv, 2, d):
        raise N.SpecVerifyError(f"bounds must be {[nb, hkv, 2, d]}, got {list(bounds.shape)}")
    n = kv.cache_lens.shape[0]
    _at_least(from_len, n, "from_len")
    if kv.block_tables.shape[0] < n:
        raise N.SpecVerifyError(f"block_tables has {kv.block_tables.shape[0]} rows for {n} requests")
    dev = _one_device(kv.k_cache, kv.block_tables, kv.cache_lens, bounds, from_len, dev_status)
    k = kv.c()
    return (ctypes.byref(k), n, _ptr(from_len), _ptr(bounds), _ptr(dev_status)), dev


def sv_bound_pages(kv: PagedKV, bounds: torch.Tensor, from_len: Optional[torch.Tensor] = None,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    """Least and greatest key of the complete pages behind from_len (None: all) of
    every request of kv.cache_lens, into bounds [blocks][kv heads][2][dim]."""
    args, _ = _bound_args(kv, bounds, from_len, dev_status)
    _call("sv_bound_pages", args, stream)


def bind_bound_pages(kv: PagedKV, bounds: torch.Tensor, from_len: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_bound_pages with its arguments marshalled once (see BoundCall)."""
    args, dev = _bound_args(kv, bounds, from_len, dev_status)
    return BoundCall("sv_bound_pages", args, dev, (kv, bounds, from_len, dev_status))


def _scores(kv, batch, scores):
    _expect(scores, torch.float32, "scores")
    want = (batch.total_rows, kv.k_cache.shape[1])
    if scores.dim() != 3 or tuple(scores.shape[:2]) != want:
        raise N.SpecVerifyError(f"scores must be [{want[0]}][{want[1]}][pages], got {list(scores.shape)}")
    return scores.shape[2]


def _score_args(kv, batch, q, bounds, scores, dev_status):
    heads = _queries(kv, batch, q)
    _expect(bounds, torch.bfloat16, "bounds")
    _expect(dev_status, torch.int32, "dev_status")
    nb, hkv, _, d = _cache_shape(kv, "sv_score_pages")
    if tuple(bounds.shape) != (nb, hkv, 2, d):
        raise N.SpecVerifyError(f"bounds must be {[nb, hkv, 2, d]}, got {list(bounds.shape)}")
    max_pages = _scores(kv, batch, scores)
    _batch_fits(kv, batch)
    dev = _one_device(*_batch_tensors(batch), q, bounds, scores, kv.block_tables, kv.cache_lens,
                      dev_status)
    b, k = batch.c(), kv.c()
    return (ctypes.byref(k), ctypes.byref(b), _ptr(q), heads, _ptr(bounds), _ptr(scores), max_pages,
            _ptr(dev_status)), dev


def sv_score_pages(kv: PagedKV, batch: Batch, q: torch.Tensor, bounds: torch.Tensor,
                   scores: torch.Tensor, dev_status: Optional[torch.Tensor] = None, stream=None):
    """An upper bound of the products of each row's queries with the keys of each
    complete page, into scores [rows][kv heads][pages]."""
    args, _ = _score_args(kv, batch, q, bounds, scores, dev_status)
    _call("sv_score_pages", args, stream)


def bind_score_pages(kv: PagedKV, batch: Batch, q: torch.Tensor, bounds: torch.Tensor,
                     scores: torch.Tensor, dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_score_pages with its arguments marshalled once (see BoundCall)."""
    args, dev = _score_args(kv, batch, q, bounds, scores, dev_status)
    return BoundCall("sv_score_pages", args, dev, (kv, batch, q, bounds, scores, dev_status))


def _pages(kv, batch, pages):
    _expect(pages, torch.int32, "pages")
    want = (batch.total_rows, kv.k_cache.shape[1])
    if pages.dim() != 3 or tuple(pages.shape[:2]) != want:
        raise N.SpecVerifyError(f"pages must be [{want[0]}][{want[1]}][n_keep], got {list(pages.shape)}")
    return pages.shape[2]


def _select_args(kv, batch, scores, pages, n_first, n_last, dev_status):
    _expect(dev_status, torch.int32, "dev_status")
    max_pages, n_keep = _scores(kv, batch, scores), _pages(kv, batch, pages)
    _batch_fits(kv, batch)
    dev = _one_device(*_batch_tensors(batch), scores, pages, kv.cache_lens, dev_status)
    b, k = batch.c(), kv.c()
    return (ctypes.byref(k), ctypes.byref(b), _ptr(scores), max_pages, int(n_first), int(n_last),
            n_keep, _ptr(pages), _ptr(dev_status)), dev


def sv_select_pages(kv: PagedKV, batch: Batch, scores: torch.Tensor, pages: torch.Tensor,
                    n_first: int = 1, n_last: int = 4, dev_status: Optional[torch.Tensor] = None,
                    stream=None):
    """The pages each row attends, ascending, into pages [rows][kv heads][n_keep]:
    the first n_first, the last n_last and those of greatest score."""
    args, _ = _select_args(kv, batch, scores, pages, n_first, n_last, dev_status)
    _call("sv_select_pages", args, stream)


def bind_select_pages(kv: PagedKV, batch: Batch, scores: torch.Tensor, pages: torch.Tensor,
                      n_first: int = 1, n_last: int = 4,
                      dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_select_pages with its arguments marshalled once (see BoundCall)."""
    args, dev = _select_args(kv, batch, scores, pages, n_first, n_last, dev_status)
    return BoundCall("sv_select_pages", args, dev, (kv, batch, scores, pages, dev_status))


def sv_page_attend_workspace(batch: Batch, kv: PagedKV, n_q_heads: int, n_keep: int) -> int:
    b, k = batch.c(), kv.c()
    return N.lib().sv_page_attend_workspace(ctypes.byref(b), ctypes.byref(k), n_q_heads, n_keep)


def _attended(kv, batch, q, out, ws, dev_status, *others):
    """Query heads, batch and cache structs and device of an attention call."""
    heads = _queries(kv, batch, q)
    _expect(out, torch.bfloat16, "out")
    _expect(dev_status, torch.int32, "dev_status")
    if out.shape != q.shape:
        raise N.SpecVerifyError(f"out must be {list(q.shape)}, got {list(out.shape)}")
    _cache_shape(kv, "attention")
    _batch_fits(kv, batch)
    dev = _one_device(*_batch_tensors(batch), q, out, ws, kv.k_cache, kv.v_cache, kv.block_tables,
                      kv.cache_lens, dev_status, *others)
    return heads, batch.c(), kv.c(), dev


def _page_attend_args(kv, batch, q, softmax_scale, pages, out, ws, dev_status):
    n_keep = _pages(kv, batch, pages)
    heads, b, k, dev = _attended(kv, batch, q, out, ws, dev_status, pages)
    return (ctypes.byref(k), ctypes.byref(b), _ptr(q), heads, float(softmax_scale), _ptr(pages),
            n_keep, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status)), dev


def sv_page_attend(kv: PagedKV, batch: Batch, q: torch.Tensor, softmax_scale: float,
                   pages: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                   dev_status: Optional[torch.Tensor] = None, stream=None):
    """sv_tree_attend over the pages that sv_select_pages chose for each row and KV
    head, the slots behind the last complete page and the staged ancestors."""
    args, _ = _page_attend_args(kv, batch, q, softmax_scale, pages, out, ws, dev_status)
    _call("sv_page_attend", args, stream)


def bind_page_attend(kv: PagedKV, batch: Batch, q: torch.Tensor, softmax_scale: float,
                     pages: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                     dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_page_attend with its arguments marshalled once (see BoundCall)."""
    args, dev = _page_attend_args(kv, batch, q, softmax_scale, pages, out, ws, dev_status)
    return BoundCall("sv_page_attend", args, dev, (kv, batch, q, pages, out, ws, dev_status))


def sv_prefix_attend_workspace(batch: Batch, kv: PagedKV, shared: SharedPrefix,
                               n_q_heads: int) -> int:
    b, k, s = batch.c(), kv.c(), shared.c()
    return N.lib().sv_prefix_attend_workspace(ctypes.byref(b), ctypes.byref(k), ctypes.byref(s),
                                              n_q_heads)


def _prefix_attend_args(kv, batch, shared, q, softmax_scale, out, ws, dev_status):
    s = shared.c()
    heads, b, k, dev = _attended(kv, batch, q, out, ws, dev_status, shared.cu_groups,
                                 shared.prefix_len)
    return (ctypes.byref(k), ctypes.byref(b), ctypes.byref(s), _ptr(q), heads, float(softmax_scale),
            _ptr(out), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status)), dev


def sv_prefix_attend(kv: PagedKV, batch: Batch, shared: SharedPrefix, q: torch.Tensor,
                     softmax_scale: float, out: torch.Tensor, ws: torch.Tensor,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    """sv_tree_attend for requests that share prefixes, whose pages are read once
    for all rows of a group, from the table of its first request."""
    args, _ = _prefix_attend_args(kv, batch, shared, q, softmax_scale, out, ws, dev_status)
    _call("sv_prefix_attend", args, stream)


def bind_prefix_attend(kv: PagedKV, batch: Batch, shared: SharedPrefix, q: torch.Tensor,
                       softmax_scale: float, out: torch.Tensor, ws: torch.Tensor,
                       dev_status: Optional[torch.Tensor] = None) -> BoundCall:
    """sv_prefix_attend with its arguments marshalled once (see BoundCall)."""
    args, dev = _prefix_attend_args(kv, batch, shared, q, softmax_scale, out, ws, dev_status)
    return BoundCall("sv_prefix_attend", args, dev, (kv, batch, shared, q, out, ws, dev_status))
