"""Python binding of libsfi with the C ABI's names (argument marshalling only).

Each function takes torch CUDA tensors, checks their dtype, device and layout,
passes their device pointers to the C entry point of the same name on the given
(or current) stream, and raises SFIError on a non-zero status. No arithmetic of
the method happens here.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from fractions import Fraction
from typing import Optional

import torch

from . import _abi


SFI_ATTN_EARLY_KV_PREFETCH = _abi.SFI_ATTN_EARLY_KV_PREFETCH
SFI_MAX_QUERY_TOKENS = _abi.SFI_MAX_QUERY_TOKENS
SFI_MAX_PAGE_REQS = _abi.SFI_MAX_PAGE_REQS
SFI_MAX_COMPACT_PAGES = _abi.SFI_MAX_COMPACT_PAGES
SFI_MAX_VOCAB = _abi.SFI_MAX_VOCAB
SFI_ATTN_RAGGED = _abi.SFI_ATTN_RAGGED
SFI_ATTN_TEST_WITHHOLD = _abi.SFI_ATTN_TEST_WITHHOLD


class SFIError(RuntimeError):
    def __init__(self, status: int, where: str):
        name = _abi.lib().sfi_status_string(status).decode()
        super().__init__(f"{where}: {name}")
        self.status = status


@dataclass(frozen=True)
class AttnShape:
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    page_size: int = 16
    softmax_scale: float = 0.0  # <= 0: 1/sqrt(head_dim)

    @property
    def group(self) -> int:
        return self.num_q_heads // self.num_kv_heads

    def c(self) -> _abi.sfi_attn_shape:
        c = self.__dict__.get("_c")
        if c is None:  # the fields are frozen, so the C view is made once
            c = _abi.sfi_attn_shape(self.num_q_heads, self.num_kv_heads, self.head_dim, self.page_size,
                                    float(self.softmax_scale))
            object.__setattr__(self, "_c", c)
        return c


class _Handle:
    """Tensors that one C structure points to. The structure is checked and made when it is
    first needed, and again when a field has been assigned, a tensor's memory, shape or strides
    are no longer what they were (resize_, set_, .data = ...), or another device is the current
    one: a call that finds it ready saves itself the checks and the structure."""
    _tensors = ()

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_kept", None)  # with its references: a tensor that is let go is free

    def __getstate__(self):
        # a copy (copy, deepcopy, pickle) makes its own structure, of its own tensors
        return {k: v for k, v in self.__dict__.items() if not k.startswith("_")}

    def c(self, dev: Optional[int] = None):
        """The structure, for calls on device dev (None: the current one)."""
        if dev is None:
            dev = torch._C._cuda_getDevice()
        d = self.__dict__
        kept = d.get("_kept")
        if kept is not None and kept[1] == dev:
            for t, ptr, size, stride in kept[2]:
                if t.data_ptr() != ptr or t.shape != size or t.stride() != stride:
                    break
            else:
                return kept[0]
        d.pop("_kept", None)
        c = self._make(dev)
        at = [(t, t.data_ptr(), t.shape, t.stride()) for t in (d[n] for n in self._tensors)]
        d["_kept"] = (c, dev, at)
        return c


@dataclass
class PagedKV(_Handle):
    """Paged bf16 KV cache: pools [num_pages][Hkv][P][D], page_table int32 [B][max_pages], seq_lens int32 [B]."""
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor

    _tensors = ("k_pool", "v_pool", "page_table", "seq_lens")

    def _make(self, dev: int) -> _abi.sfi_paged_kv:
        for name, t, dt in (("k_pool", self.k_pool, torch.bfloat16), ("v_pool", self.v_pool, torch.bfloat16),
                            ("page_table", self.page_table, torch.int32), ("seq_lens", self.seq_lens, torch.int32)):
            _need(t, dt, name)
        return _abi.sfi_paged_kv(self.k_pool.data_ptr(), self.v_pool.data_ptr(), self.k_pool.shape[0],
                                 self.page_table.shape[1], self.page_table.data_ptr(), self.seq_lens.data_ptr())


@dataclass
class CompactKV:
    """Compact buffer: k, v bf16 [total_rows][D]; row_offset int64 [B]; capacity, count int32 [B]."""
    k: torch.Tensor
    v: torch.Tensor
    row_offset: torch.Tensor
    capacity: torch.Tensor
    count: torch.Tensor

    def c(self) -> _abi.sfi_compact_kv:
        _need(self.k, torch.bfloat16, "compact.k")
        _need(self.v, torch.bfloat16, "compact.v")
        _need(self.row_offset, torch.int64, "compact.row_offset")
        _need(self.capacity, torch.int32, "compact.capacity")
        _need(self.count, torch.int32, "compact.count")
        return _abi.sfi_compact_kv(self.k.data_ptr(), self.v.data_ptr(), self.k.shape[0],
                                   self.row_offset.data_ptr(), self.capacity.data_ptr(), self.count.data_ptr())


def _need(t: Optional[torch.Tensor], dtype, name: str):
    if t is not None and t.is_cuda and t.dtype is dtype and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor], dtype=None, name: str = "") -> Optional[int]:
    if t is None:
        return None
    if dtype is not None:
        _need(t, dtype, name)
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without the Stream object (3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _batch(batch, req_ids, seq_lens) -> int:
    if batch is not None:
        return int(batch)
    if req_ids is not None:
        return int(req_ids.numel())
    return int(seq_lens.numel())


def _check(status: int, where: str):
    if status != _abi.SFI_OK:
        raise SFIError(status, where)


def sfi_paged_kv_append(shape: AttnShape, kv: PagedKV, k_new: torch.Tensor, v_new: torch.Tensor,
                        req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                        dev_status: Optional[torch.Tensor] = None, stream=None):
    st = _abi.lib().sfi_paged_kv_append(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), _ptr(k_new, torch.bfloat16, "k_new"),
        _ptr(v_new, torch.bfloat16, "v_new"), _ptr(req_ids, torch.int32, "req_ids"),
        _batch(batch, req_ids, kv.seq_lens), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_paged_kv_append")


def sfi_fast_decode_attn(shape: AttnShape, kv: PagedKV, compact: CompactKV, sink: int, recent: int,
                         q: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                         req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None, max_tokens: int = 0,
                         num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                         dev_status: Optional[torch.Tensor] = None, stream=None,
                         k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                         flags: int = 0):
    ws = _ptr(workspace, torch.uint8, "workspace")
    st = _abi.lib().sfi_fast_decode_attn(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), ctypes.byref(compact.c()), int(sink), int(recent),
        _ptr(q, torch.bfloat16, "q"), _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"),
        _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, kv.seq_lens), int(max_tokens),
        int(num_splits), int(flags), ws, 0 if workspace is None else workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_fast_decode_attn")


def sfi_slow_dense_attn_with_scores(shape: AttnShape, kv: PagedKV, sink: int, recent: int, q: torch.Tensor,
                                    out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                                    scores: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                                    batch: Optional[int] = None, max_tokens: int = 0, num_splits: int = 0,
                                    workspace: Optional[torch.Tensor] = None,
                                    dev_status: Optional[torch.Tensor] = None, stream=None,
                                    k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                                    flags: int = 0):
    ws = _ptr(workspace, torch.uint8, "workspace")
    stride = 0 if scores is None else int(scores.shape[-1])
    st = _abi.lib().sfi_slow_dense_attn_with_scores(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), int(sink), int(recent), _ptr(q, torch.bfloat16, "q"),
        _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"), _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"), _ptr(scores, torch.float32, "scores"),
        stride, _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, kv.seq_lens), int(max_tokens),
        int(num_splits), int(flags), ws, 0 if workspace is None else workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_slow_dense_attn_with_scores")


def sfi_mixed_decode_attn(shape: AttnShape, kv: PagedKV, compact: Optional[CompactKV], sink: int, recent: int,
                          q: torch.Tensor, out: torch.Tensor, fast_ids: torch.Tensor, slow_ids: torch.Tensor,
                          lse: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                          k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                          max_fast_tokens: int = 0, max_dense_tokens: int = 0, flags: int = 0,
                          workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                          stream=None):
    ws = _ptr(workspace, torch.uint8, "workspace")
    n_fast, n_slow = int(fast_ids.numel()), int(slow_ids.numel())
    st = _abi.lib().sfi_mixed_decode_attn(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), None if compact is None else ctypes.byref(compact.c()),
        int(sink), int(recent), _ptr(q, torch.bfloat16, "q"), _ptr(k_new, torch.bfloat16, "k_new"),
        _ptr(v_new, torch.bfloat16, "v_new"), _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(scores, torch.float32, "scores"), 0 if scores is None else int(scores.shape[-1]),
        _ptr(fast_ids, torch.int32, "fast_ids") if n_fast else None, n_fast,
        _ptr(slow_ids, torch.int32, "slow_ids") if n_slow else None, n_slow, int(max_fast_tokens),
        int(max_dense_tokens), int(flags), ws, 0 if workspace is None else workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_mixed_decode_attn")


def sfi_mixed_workspace_size(shape: AttnShape, n_fast: int, n_slow: int, max_fast_tokens: int,
                             max_dense_tokens: int) -> int:
    return int(_abi.lib().sfi_mixed_workspace_size(ctypes.byref(shape.c()), int(n_fast), int(n_slow),
                                                   int(max_fast_tokens), int(max_dense_tokens)))


def alloc_mixed_workspace(shape: AttnShape, batch: int, max_fast_tokens: int, max_dense_tokens: int,
                          device="cuda") -> torch.Tensor:
    """A zero-filled workspace large enough for every split of `batch` requests into
    fast and slow subsets."""
    n = max([256] + [sfi_mixed_workspace_size(shape, batch - ns, ns, max_fast_tokens, max_dense_tokens)
                     for ns in range(batch + 1)])
    return torch.zeros(n, dtype=torch.uint8, device=device)


def alloc_ragged_workspace(shape: AttnShape, batch: int, max_tokens: int, dense: bool = False,
                           device="cuda") -> torch.Tensor:
    """A zero-filled workspace for sfi_fast_decode_attn (dense=False) or
    sfi_slow_dense_attn_with_scores (dense=True) with SFI_ATTN_RAGGED, valid for every
    batch size 1..batch."""
    n = max([256] + [sfi_mixed_workspace_size(shape, 0, b, 0, max_tokens) if dense
                     else sfi_mixed_workspace_size(shape, b, 0, max_tokens, 0) for b in range(1, batch + 1)])
    return torch.zeros(n, dtype=torch.uint8, device=device)


def sfi_paged_kv_append_tokens(shape: AttnShape, kv: PagedKV, k_new: torch.Tensor, v_new: torch.Tensor,
                               num_tokens: int, req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                               dev_status: Optional[torch.Tensor] = None, stream=None):
    st = _abi.lib().sfi_paged_kv_append_tokens(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), _ptr(k_new, torch.bfloat16, "k_new"),
        _ptr(v_new, torch.bfloat16, "v_new"), int(num_tokens), _ptr(req_ids, torch.int32, "req_ids"),
        _batch(batch, req_ids, kv.seq_lens), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_paged_kv_append_tokens")


def sfi_dense_verify_attn(shape: AttnShape, kv: PagedKV, sink: int, recent: int, q: torch.Tensor, num_tokens: int,
                          out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                          scores: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                          batch: Optional[int] = None, max_tokens: int = 0, num_splits: int = 0,
                          workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                          stream=None, flags: int = 0, k_new: Optional[torch.Tensor] = None,
                          v_new: Optional[torch.Tensor] = None):
    ws = _ptr(workspace, torch.uint8, "workspace")
    stride = 0 if scores is None else int(scores.shape[-1])
    st = _abi.lib().sfi_dense_verify_attn(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), int(sink), int(recent), _ptr(q, torch.bfloat16, "q"),
        int(num_tokens), _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"),
        _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(scores, torch.float32, "scores"), stride, _ptr(req_ids, torch.int32, "req_ids"),
        _batch(batch, req_ids, kv.seq_lens), int(max_tokens), int(num_splits), int(flags), ws,
        0 if workspace is None else workspace.numel(), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_dense_verify_attn")


def sfi_sparse_draft_attn(shape: AttnShape, kv: PagedKV, compact: CompactKV, sink: int, recent: int,
                          q: torch.Tensor, num_tokens: int, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                          req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None, max_tokens: int = 0,
                          num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                          dev_status: Optional[torch.Tensor] = None, stream=None, flags: int = 0,
                          k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None):
    ws = _ptr(workspace, torch.uint8, "workspace")
    st = _abi.lib().sfi_sparse_draft_attn(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), ctypes.byref(compact.c()), int(sink), int(recent),
        _ptr(q, torch.bfloat16, "q"), int(num_tokens), _ptr(k_new, torch.bfloat16, "k_new"),
        _ptr(v_new, torch.bfloat16, "v_new"), _ptr(out, torch.float32, "out"),
        _ptr(lse, torch.float32, "lse"), _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, kv.seq_lens),
        int(max_tokens), int(num_splits), int(flags), ws, 0 if workspace is None else workspace.numel(),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_sparse_draft_attn")


def sfi_multi_workspace_size(shape: AttnShape, batch: int, num_tokens: int, max_tokens: int,
                             num_splits: int = 0) -> int:
    return int(_abi.lib().sfi_multi_workspace_size(ctypes.byref(shape.c()), int(batch), int(num_tokens),
                                                   int(max_tokens), int(num_splits)))


def alloc_multi_workspace(shape: AttnShape, batch: int, num_tokens: int, max_tokens: int, num_splits: int = 0,
                          device="cuda") -> torch.Tensor:
    """A zero-filled workspace for the multi-token calls, valid for every batch size 1..batch."""
    n = max([256] + [sfi_multi_workspace_size(shape, b, num_tokens, max_tokens, num_splits)
                     for b in range(1, batch + 1)])
    return torch.zeros(n, dtype=torch.uint8, device=device)


def sfi_select_topk(scores: torch.Tensor, num_kv_heads: int, seq_lens: torch.Tensor, sink: int, recent: int,
                    k_per_req: torch.Tensor, idx_out: torch.Tensor, count_out: torch.Tensor,
                    req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None):
    st = _abi.lib().sfi_select_topk(
        _ptr(scores, torch.float32, "scores"), int(scores.shape[-1]), int(num_kv_heads),
        _ptr(seq_lens, torch.int32, "seq_lens"), int(sink), int(recent), _ptr(k_per_req, torch.int32, "k_per_req"),
        int(idx_out.shape[-1]), _ptr(idx_out, torch.int32, "idx_out"), _ptr(count_out, torch.int32, "count_out"),
        _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, seq_lens),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_select_topk")


def sfi_select_compact(shape: AttnShape, kv: PagedKV, scores: torch.Tensor, sink: int, recent: int,
                       k_per_req: torch.Tensor, idx_out: torch.Tensor, compact: CompactKV,
                       count_out: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                       batch: Optional[int] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """Selector + compaction in one launch; count_out defaults to compact.count."""
    count_out = compact.count if count_out is None else count_out
    st = _abi.lib().sfi_select_compact(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), _ptr(scores, torch.float32, "scores"), int(scores.shape[-1]),
        int(sink), int(recent), _ptr(k_per_req, torch.int32, "k_per_req"), int(idx_out.shape[-1]),
        _ptr(idx_out, torch.int32, "idx_out"), _ptr(count_out, torch.int32, "count_out"), ctypes.byref(compact.c()),
        _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, kv.seq_lens),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_select_compact")


def sfi_compact_gather(shape: AttnShape, kv: PagedKV, idx: torch.Tensor, count: torch.Tensor, sink: int,
                       compact: CompactKV, req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                       dev_status: Optional[torch.Tensor] = None, stream=None):
    st = _abi.lib().sfi_compact_gather(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), _ptr(idx, torch.int32, "idx"),
        _ptr(count, torch.int32, "count"), int(idx.shape[-1]), int(sink), ctypes.byref(compact.c()),
        _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, kv.seq_lens),
        _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_compact_gather")


def sfi_fast_decode_attn_noalloc(shape: AttnShape, kv: PagedKV, compact: CompactKV, sink: int, recent: int,
                                 q: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                                 req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                                 max_tokens: int = 0, num_splits: int = 0,
                                 dev_status: Optional[torch.Tensor] = None, stream=None,
                                 k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                                 flags: int = 0):
    """sfi_fast_decode_attn without a workspace argument, for callers that cannot
    allocate device memory: the split-KV scratch is a fixed array inside the library
    (SFI_NOALLOC_SCRATCH_BYTES per GPU). Calls that may overlap on the GPU share that
    array and race; order them on one stream."""
    st = _abi.lib().sfi_fast_decode_attn_noalloc(
        ctypes.byref(shape.c()), ctypes.byref(kv.c()), ctypes.byref(compact.c()), int(sink), int(recent),
        _ptr(q, torch.bfloat16, "q"), _ptr(k_new, torch.bfloat16, "k_new"), _ptr(v_new, torch.bfloat16, "v_new"),
        _ptr(out, torch.float32, "out"), _ptr(lse, torch.float32, "lse"),
        _ptr(req_ids, torch.int32, "req_ids"), _batch(batch, req_ids, kv.seq_lens), int(max_tokens),
        int(num_splits), int(flags), _ptr(dev_status, torch.int32, "dev_status"), _stream(stream))
    _check(st, "sfi_fast_decode_attn_noalloc")


# The launches go to the current device. The calls from here on take tensors of that device alone;
# dev is its index, asked for once a call.
def _on_current_device(t: torch.Tensor, name: str):
    if t.is_cuda and t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, not on the current device")


def _need_here(t: Optional[torch.Tensor], dtype, name: str, dev: int):
    if t is not None and t.get_device() == dev and t.dtype is dtype and t.is_contiguous():
        return
    _need(t, dtype, name)
    _on_current_device(t, name)


def _ptr_here(t: Optional[torch.Tensor], dtype, name: str, dev: int) -> Optional[int]:
    if t is None:
        return None
    _need_here(t, dtype, name, dev)
    return t.data_ptr()


def _stream_here(stream, dev: int) -> Optional[int]:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


@dataclass
class Rope(_Handle):
    """The position rotation of sfi_qk_norm_rope: turns int64 [rot_dim / 2] (rope_turns),
    axis uint8 [rot_dim / 2] or None, the number of position axes, and whether pairs are
    adjacent dims (interleaved) or dims rot_dim / 2 apart."""
    turns: torch.Tensor
    axis: Optional[torch.Tensor] = None
    num_axes: int = 1
    interleaved: bool = False

    @property
    def _tensors(self):
        return ("turns",) if self.axis is None else ("turns", "axis")

    def _make(self, dev: int) -> _abi.sfi_rope:
        _need_here(self.turns, torch.int64, "rope.turns", dev)
        axis = _ptr_here(self.axis, torch.uint8, "rope.axis", dev)
        if self.axis is not None and self.axis.numel() != self.turns.numel():
            raise ValueError("rope.axis needs one entry for each of rope.turns")
        return _abi.sfi_rope(self.turns.data_ptr(), axis, 2 * self.turns.numel(), int(self.num_axes),
                             int(bool(self.interleaved)))


# 2 pi to 40 decimals: positions are 32-bit, so 64-bit turns need more digits than a double has
_TWO_PI = Fraction(62831853071795864769252867665590057683943, 10 ** 40)


def rope_turns(inv_freq, device="cuda") -> torch.Tensor:
    """Rotation per position (inv_freq in radians, fp64) as 64-bit fixed-point turns modulo one turn."""
    freqs = [float(f) for f in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor) else inv_freq)]
    turns = [round(Fraction(f) * 2 ** 64 / _TWO_PI) % 2 ** 64 for f in freqs]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)


def _count(requests: int, batch, req_ids) -> int:
    """The number of requests a call takes out of `requests`."""
    n = requests if req_ids is None else req_ids.numel()
    if batch is None:
        return n
    if batch > n:
        raise ValueError(f"batch {batch} is beyond the {n} requests given")
    return int(batch)


def _indexed(t: Optional[torch.Tensor], requests: int, name: str):
    """Arrays indexed by request id cover all requests of the table."""
    if t is not None and t.shape[0] != requests:
        raise ValueError(f"{name} needs one entry for each of {requests} requests, has {t.shape[0]}")


def _token_rows(t: torch.Tensor, heads: int, dim: int, name: str, dev: int):
    """Requests, tokens and elements between tokens of a [B][T][heads][dim] tensor whose heads
    are contiguous."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        _on_current_device(t, name)
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    dims = t.shape
    if len(dims) != 4 or dims[2] != heads or dims[3] != dim:
        raise ValueError(f"{name} must be [B][T][{heads}][{dim}], got {list(dims)}")
    b, n = dims[0], dims[1]
    s = t.stride()
    step = s[1] if n > 1 else (s[0] if b > 1 else heads * dim)
    if s[3] != 1 or (heads > 1 and s[2] != dim) or (b > 1 and s[0] != n * step):
        raise ValueError(f"{name} needs contiguous heads and one stride between all tokens")
    return b, n, step


def sfi_qk_norm_rope(shape: AttnShape, rope: Optional[Rope], q: torch.Tensor, k: torch.Tensor,
                     v: Optional[torch.Tensor], q_out: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     positions: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                     seq_lens: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                     kv: Optional[PagedKV] = None, req_ids: Optional[torch.Tensor] = None,
                     batch: Optional[int] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """Head norm and rotation of the new tokens; q, k, v [B][T][heads][D] may be views of one
    fused projection. positions int32 [num_axes][B][T] (or [B][T] with one axis)."""
    hq, hkv, d = shape.num_q_heads, shape.num_kv_heads, shape.head_dim
    dev = torch._C._cuda_getDevice()
    B, T, qs = _token_rows(q, hq, d, "q", dev)
    kb, kt, ks = _token_rows(k, hkv, d, "k", dev)
    vb, vt, vs = (B, T, 0) if v is None else _token_rows(v, hkv, d, "v", dev)
    if kb != B or kt != T or vb != B or vt != T:
        raise ValueError("q, k and v need the same requests and tokens")
    _need_here(q_out, torch.bfloat16, "q_out", dev)
    if q_out.shape != q.shape or (k_out is not None and k_out.shape != k.shape):
        raise ValueError("q_out and k_out need the shapes of q and k")
    if (q_weight is not None and q_weight.numel() != d) or (k_weight is not None and k_weight.numel() != d):
        raise ValueError(f"q_weight and k_weight must have {d} values")
    if positions is not None and positions.numel() != (rope.num_axes if rope is not None else 1) * B * T:
        raise ValueError("positions must be [num_axes][B][T]")
    if (new_lens is not None and new_lens.numel() != B) or (seq_lens is not None and seq_lens.numel() != B):
        raise ValueError("new_lens and seq_lens need one entry per request")
    kv_c = None
    if kv is not None:
        if kv.page_table.dim() != 2 or kv.page_table.shape[0] != B or kv.seq_lens.numel() != B:
            raise ValueError("q, k and v need one entry for each request of the pages (page_table, seq_lens)")
        kv_c = ctypes.byref(kv.c())
        for name in ("k_pool", "v_pool", "page_table", "seq_lens"):
            if getattr(kv, name).get_device() != dev:
                _on_current_device(getattr(kv, name), name)
        dims = kv.k_pool.shape
        if len(dims) != 4 or dims[1] != hkv or dims[2] != shape.page_size or dims[3] != d or kv.v_pool.shape != dims:
            raise ValueError(f"the pools must be [num_pages][{hkv}][{shape.page_size}][{d}]")
    st = _abi.lib().sfi_qk_norm_rope(
        ctypes.byref(shape.c()), None if rope is None else ctypes.byref(rope.c(dev)), q.data_ptr(), qs,
        k.data_ptr(), ks, None if v is None else v.data_ptr(), vs, _ptr_here(q_weight, torch.bfloat16, "q_weight", dev),
        _ptr_here(k_weight, torch.bfloat16, "k_weight", dev), eps,
        _ptr_here(positions, torch.int32, "positions", dev), B * T, T,
        _ptr_here(new_lens, torch.int32, "new_lens", dev), _ptr_here(seq_lens, torch.int32, "seq_lens", dev),
        q_out.data_ptr(), _ptr_here(k_out, torch.bfloat16, "k_out", dev), kv_c,
        _ptr_here(req_ids, torch.int32, "req_ids", dev), _count(B, batch, req_ids),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_qk_norm_rope")


@dataclass
class PagedKV4(_Handle):
    """Paged 4-bit cache: pool uint8 [num_pages][Hkv][18 D] (alloc_kv4_pool), page_table int32
    [B][max_pages], seq_lens int32 [B]; k_scale and v_scale are powers of two."""
    pool: torch.Tensor
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    k_scale: float = 1.0
    v_scale: float = 1.0

    _tensors = ("pool", "page_table", "seq_lens")

    def _make(self, dev: int) -> _abi.sfi_paged_kv4:
        _need_here(self.pool, torch.uint8, "pool", dev)
        _need_here(self.page_table, torch.int32, "page_table", dev)
        _need_here(self.seq_lens, torch.int32, "seq_lens", dev)
        if self.pool.dim() != 3:
            raise ValueError(f"pool must be [num_pages][Hkv][18 D], got {list(self.pool.shape)}")
        if self.page_table.dim() != 2 or self.seq_lens.numel() != self.page_table.shape[0]:
            raise ValueError("seq_lens needs one entry per row of page_table")
        self.__dict__["_dims"] = tuple(self.pool.shape[1:])
        self.__dict__["_requests"] = self.page_table.shape[0]
        return _abi.sfi_paged_kv4(self.pool.data_ptr(), self.pool.shape[0], self.page_table.shape[1],
                                  self.page_table.data_ptr(), self.seq_lens.data_ptr(), self.k_scale, self.v_scale)


@dataclass
class CompactKV4(_Handle):
    """4-bit compact blocks: pool uint8 [total_pages][18 D]; page_offset int64 [B]; capacity
    (blocks per KV head) and count (selected rows) int32 [B]."""
    pool: torch.Tensor
    page_offset: torch.Tensor
    capacity: torch.Tensor
    count: torch.Tensor

    _tensors = ("pool", "page_offset", "capacity", "count")

    def _make(self, dev: int) -> _abi.sfi_compact_kv4:
        _need_here(self.pool, torch.uint8, "compact.pool", dev)
        _need_here(self.page_offset, torch.int64, "compact.page_offset", dev)
        _need_here(self.capacity, torch.int32, "compact.capacity", dev)
        _need_here(self.count, torch.int32, "compact.count", dev)
        self.__dict__["_requests"] = self.page_offset.numel()
        if self.capacity.numel() != self.page_offset.numel() or self.count.numel() != self.page_offset.numel():
            raise ValueError("compact.page_offset, capacity and count need one entry per request")
        if self.pool.dim() != 2:
            raise ValueError(f"compact.pool must be [total_pages][18 D], got {list(self.pool.shape)}")
        self.__dict__["_bytes"] = self.pool.shape[1]
        return _abi.sfi_compact_kv4(self.pool.data_ptr(), self.pool.shape[0], self.page_offset.data_ptr(),
                                    self.capacity.data_ptr(), self.count.data_ptr())


def _kv4(shape: AttnShape, kv: PagedKV4, dev: int):
    c = kv.c(dev)
    if kv._dims != (shape.num_kv_heads, 18 * shape.head_dim):
        raise ValueError(f"pool must be [num_pages][{shape.num_kv_heads}][{18 * shape.head_dim}], "
                         f"got {list(kv.pool.shape)}")
    return ctypes.byref(c)


def _compact4(shape: AttnShape, kv: PagedKV4, compact: CompactKV4, dev: int):
    c = compact.c(dev)
    if compact._bytes != 18 * shape.head_dim:
        raise ValueError(f"compact.pool must be [total_pages][{18 * shape.head_dim}]")
    if compact._requests != kv._requests:
        raise ValueError(f"compact needs one entry for each of {kv._requests} requests, has {compact._requests}")
    return ctypes.byref(c)


def alloc_kv4_pool(shape: AttnShape, num_pages: int, device="cuda") -> torch.Tensor:
    """A zero-filled pool of the 4-bit cache."""
    return torch.zeros((num_pages, shape.num_kv_heads, 18 * shape.head_dim), dtype=torch.uint8, device=device)


def alloc_kv4_compact(shape: AttnShape, rows, device="cuda") -> CompactKV4:
    """4-bit compact blocks for rows[r] = sink + k_r rows per KV head of request r."""
    cap = torch.tensor([(int(n) + 15) // 16 for n in rows], dtype=torch.int64)
    ends = torch.cumsum(cap * shape.num_kv_heads, 0)
    pool = torch.zeros((max(1, int(ends[-1]) if len(cap) else 1), 18 * shape.head_dim), dtype=torch.uint8, device=device)
    return CompactKV4(pool, (ends - cap * shape.num_kv_heads).to(device), cap.to(torch.int32).to(device),
                      torch.zeros(len(cap), dtype=torch.int32, device=device))


def _rows4(t: torch.Tensor, dtype, shape: AttnShape, heads: int, name: str, dev: int) -> int:
    """Tokens of a [B][T][heads][D] tensor."""
    _need_here(t, dtype, name, dev)
    dims = t.shape
    if len(dims) != 4 or dims[2] != heads or dims[3] != shape.head_dim:
        raise ValueError(f"{name} must be [B][T][{heads}][{shape.head_dim}], got {list(dims)}")
    return dims[1]


def sfi_kv4_append(shape: AttnShape, kv: PagedKV4, k_new: torch.Tensor, v_new: torch.Tensor,
                   new_lens: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                   batch: Optional[int] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """k_new, v_new [B][T][Hkv][D]; either may be a view of a fused projection (contiguous heads)."""
    dev = torch._C._cuda_getDevice()
    kb, T, ks = _token_rows(k_new, shape.num_kv_heads, shape.head_dim, "k_new", dev)
    vb, vt, vs = _token_rows(v_new, shape.num_kv_heads, shape.head_dim, "v_new", dev)
    kv_c = _kv4(shape, kv, dev)
    B = kv._requests
    if kb != B or vb != B or vt != T:
        raise ValueError(f"k_new and v_new need the same shape, with one entry for each of {B} requests")
    _indexed(new_lens, B, "new_lens")
    st = _abi.lib().sfi_kv4_append(
        ctypes.byref(shape.c()), kv_c, k_new.data_ptr(), ks, v_new.data_ptr(), vs, T,
        _ptr_here(new_lens, torch.int32, "new_lens", dev), _ptr_here(req_ids, torch.int32, "req_ids", dev),
        _count(B, batch, req_ids), _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_kv4_append")


def sfi_kv4_read(shape: AttnShape, kv: PagedKV4, k_out: torch.Tensor, v_out: torch.Tensor,
                 first: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                 batch: Optional[int] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    T = _rows4(k_out, torch.bfloat16, shape, shape.num_kv_heads, "k_out", dev)
    _need_here(v_out, torch.bfloat16, "v_out", dev)
    if v_out.shape != k_out.shape:
        raise ValueError("k_out and v_out need the same shape")
    kv_c = _kv4(shape, kv, dev)
    B = kv._requests
    _indexed(k_out, B, "k_out")
    _indexed(first, B, "first")
    st = _abi.lib().sfi_kv4_read(
        ctypes.byref(shape.c()), kv_c, k_out.data_ptr(), v_out.data_ptr(), T,
        _ptr_here(first, torch.int32, "first", dev), _ptr_here(req_ids, torch.int32, "req_ids", dev),
        _count(B, batch, req_ids), _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_kv4_read")


def sfi_kv4_compact_gather(shape: AttnShape, kv: PagedKV4, idx: torch.Tensor, count: torch.Tensor, sink: int,
                           compact: CompactKV4, req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                           dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    kv_c = _kv4(shape, kv, dev)
    B = kv._requests
    dims = idx.shape
    if len(dims) != 3 or dims[0] != B or dims[1] != shape.num_kv_heads:
        raise ValueError(f"idx must be [{B}][{shape.num_kv_heads}][k_cap], got {list(dims)}")
    _indexed(count, B, "count")
    st = _abi.lib().sfi_kv4_compact_gather(
        ctypes.byref(shape.c()), kv_c, _ptr_here(idx, torch.int32, "idx", dev),
        _ptr_here(count, torch.int32, "count", dev), dims[2], int(sink), _compact4(shape, kv, compact, dev),
        _ptr_here(req_ids, torch.int32, "req_ids", dev), _count(B, batch, req_ids),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_kv4_compact_gather")


def _kv4_query(shape: AttnShape, kv: PagedKV4, q: torch.Tensor, out: torch.Tensor, lse: Optional[torch.Tensor],
               dev: int) -> int:
    T = _rows4(q, torch.bfloat16, shape, shape.num_q_heads, "q", dev)
    _need_here(out, torch.float32, "out", dev)
    dims = q.shape
    if out.shape != dims or (lse is not None and lse.shape != dims[:3]):
        raise ValueError("out needs the shape of q, lse that without its last dimension")
    _indexed(q, kv._requests, "q")
    return T


def sfi_kv4_dense_attn(shape: AttnShape, kv: PagedKV4, sink: int, recent: int, q: torch.Tensor, out: torch.Tensor,
                       lse: Optional[torch.Tensor] = None, scores: Optional[torch.Tensor] = None,
                       req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                       workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                       stream=None):
    """q [B][T][Hq][D] (T query tokens per request), out fp32 of that shape, lse [B][T][Hq],
    scores [B][Hkv][score_stride]."""
    dev = torch._C._cuda_getDevice()
    kv_c = _kv4(shape, kv, dev)
    T = _kv4_query(shape, kv, q, out, lse, dev)
    B, stride = kv._requests, 0
    if scores is not None:
        dims = scores.shape
        if len(dims) != 3 or dims[0] != B or dims[1] != shape.num_kv_heads:
            raise ValueError(f"scores must be [{B}][{shape.num_kv_heads}][score_stride], got {list(dims)}")
        stride = dims[2]
    st = _abi.lib().sfi_kv4_dense_attn(
        ctypes.byref(shape.c()), kv_c, int(sink), int(recent), q.data_ptr(), T, out.data_ptr(),
        _ptr_here(lse, torch.float32, "lse", dev), _ptr_here(scores, torch.float32, "scores", dev), stride,
        _ptr_here(req_ids, torch.int32, "req_ids", dev), _count(B, batch, req_ids),
        _ptr_here(workspace, torch.uint8, "workspace", dev), 0 if workspace is None else workspace.numel(),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_kv4_dense_attn")


def sfi_kv4_fast_attn(shape: AttnShape, kv: PagedKV4, compact: CompactKV4, sink: int, recent: int, q: torch.Tensor,
                      out: torch.Tensor, lse: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                      batch: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                      dev_status: Optional[torch.Tensor] = None, stream=None):
    """q [B][T][Hq][D] (T query tokens per request), out fp32 of that shape, lse [B][T][Hq]."""
    dev = torch._C._cuda_getDevice()
    kv_c = _kv4(shape, kv, dev)
    T = _kv4_query(shape, kv, q, out, lse, dev)
    st = _abi.lib().sfi_kv4_fast_attn(
        ctypes.byref(shape.c()), kv_c, _compact4(shape, kv, compact, dev), int(sink), int(recent), q.data_ptr(), T,
        out.data_ptr(), _ptr_here(lse, torch.float32, "lse", dev), _ptr_here(req_ids, torch.int32, "req_ids", dev),
        _count(kv._requests, batch, req_ids), _ptr_here(workspace, torch.uint8, "workspace", dev),
        0 if workspace is None else workspace.numel(), _ptr_here(dev_status, torch.int32, "dev_status", dev),
        _stream_here(stream, dev))
    _check(st, "sfi_kv4_fast_attn")


def sfi_kv4_workspace_size(shape: AttnShape, batch: int, num_tokens: int = 1) -> int:
    return int(_abi.lib().sfi_kv4_workspace_size(ctypes.byref(shape.c()), int(batch), int(num_tokens)))


def alloc_kv4_workspace(shape: AttnShape, batch: int, num_tokens: int = 1, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the 4-bit attention calls, valid for every batch size 1..batch,
    and for other shapes whose size it holds."""
    return torch.zeros(max(256, sfi_kv4_workspace_size(shape, batch, num_tokens)), dtype=torch.uint8, device=device)


@dataclass
class PageMap(_Handle):
    """Who holds which page: page_table int32 [num_reqs][max_pages], seq_lens int32 [num_reqs],
    ref_count int32 [num_pages] (holders of each page)."""
    page_table: torch.Tensor
    seq_lens: torch.Tensor
    ref_count: torch.Tensor

    _tensors = ("page_table", "seq_lens", "ref_count")

    def _make(self, dev: int) -> _abi.sfi_page_map:
        _need_here(self.page_table, torch.int32, "page_table", dev)
        _need_here(self.seq_lens, torch.int32, "seq_lens", dev)
        _need_here(self.ref_count, torch.int32, "ref_count", dev)
        dims = self.page_table.shape
        if len(dims) != 2 or self.seq_lens.numel() != dims[0]:
            raise ValueError("page_table must be [num_reqs][max_pages], seq_lens [num_reqs]")
        return _abi.sfi_page_map(self.page_table.data_ptr(), self.seq_lens.data_ptr(), self.ref_count.data_ptr(),
                                 dims[0], dims[1], self.ref_count.numel(), 16)


class PagePools:
    """The pools of a cache whose pages share their ids: contiguous tensors [num_pages][...] of
    one page size (each layer's k_pool and v_pool, or the 4-bit pools). Keeps the tensors and
    a device array of their addresses; a call is refused when one of them lies elsewhere by then (the
    array is not written again in a call, which a graph may be capturing)."""

    def __init__(self, pools):
        if not pools:
            raise ValueError("at least one pool is needed")
        first = pools[0]
        for t in pools:
            _need(t, t.dtype, "pool")
            if t.get_device() != first.get_device() or t.shape[0] != first.shape[0] or t.nbytes != first.nbytes:
                raise ValueError("the pools need the same device, number of pages and page size")
            if t.data_ptr() % 16:
                raise ValueError("a pool must be 16-byte aligned")
        self.pools = list(pools)
        self._at = [t.data_ptr() for t in pools]
        self.addresses = torch.tensor(self._at, dtype=torch.int64).to(first.device)
        self._c = _abi.sfi_page_pools(self.addresses.data_ptr(), len(pools), first.nbytes // max(1, first.shape[0]),
                                      first.shape[0])

    def __getstate__(self):
        return {"pools": self.pools}

    def __setstate__(self, state):
        self.__init__(state["pools"])

    def c(self) -> _abi.sfi_page_pools:
        _on_current_device(self.addresses, "pools")
        if [t.data_ptr() for t in self.pools] != self._at:
            raise ValueError("a pool has other memory than when PagePools was made: make it anew")
        return self._c


def sfi_page_copy(pools: PagePools, src: torch.Tensor, dst: torch.Tensor, dev_status: Optional[torch.Tensor] = None,
                  stream=None):
    dev = torch._C._cuda_getDevice()
    if src.numel() != dst.numel():
        raise ValueError("src and dst need the same number of pages")
    st = _abi.lib().sfi_page_copy(
        ctypes.byref(pools.c()), _ptr_here(src, torch.int32, "src", dev), _ptr_here(dst, torch.int32, "dst", dev),
        src.numel(), _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_page_copy")


def sfi_page_fork(page_map: PageMap, src: torch.Tensor, dst: torch.Tensor, fork_lens: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    if src.numel() != dst.numel() or (fork_lens is not None and fork_lens.numel() != src.numel()):
        raise ValueError("src, dst and fork_lens need one entry per branch")
    st = _abi.lib().sfi_page_fork(
        ctypes.byref(page_map.c(dev)), _ptr_here(src, torch.int32, "src", dev), _ptr_here(dst, torch.int32, "dst", dev),
        _ptr_here(fork_lens, torch.int32, "fork_lens", dev), src.numel(),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_page_fork")


def sfi_page_reserve(page_map: PageMap, pools: Optional[PagePools], new_lens: torch.Tensor,
                     reqs: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    if reqs is not None and reqs.numel() != new_lens.numel():
        raise ValueError("reqs and new_lens need one entry per request")
    st = _abi.lib().sfi_page_reserve(
        ctypes.byref(page_map.c(dev)), None if pools is None else ctypes.byref(pools.c()),
        _ptr_here(new_lens, torch.int32, "new_lens", dev), _ptr_here(reqs, torch.int32, "reqs", dev),
        new_lens.numel(), _ptr_here(workspace, torch.uint8, "workspace", dev),
        0 if workspace is None else workspace.numel(), _ptr_here(dev_status, torch.int32, "dev_status", dev),
        _stream_here(stream, dev))
    _check(st, "sfi_page_reserve")


def sfi_page_free(page_map: PageMap, reqs: torch.Tensor, dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    st = _abi.lib().sfi_page_free(
        ctypes.byref(page_map.c(dev)), _ptr_here(reqs, torch.int32, "reqs", dev), reqs.numel(),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_page_free")


def sfi_page_trim(page_map: PageMap, new_lens: torch.Tensor, reqs: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    if reqs is not None and reqs.numel() != new_lens.numel():
        raise ValueError("reqs and new_lens need one entry per request")
    st = _abi.lib().sfi_page_trim(
        ctypes.byref(page_map.c(dev)), _ptr_here(new_lens, torch.int32, "new_lens", dev),
        _ptr_here(reqs, torch.int32, "reqs", dev), new_lens.numel(), _ptr_here(dev_status, torch.int32, "dev_status", dev),
        _stream_here(stream, dev))
    _check(st, "sfi_page_trim")


def sfi_page_compact(page_map: PageMap, pools: PagePools, table_out: torch.Tensor, ref_out: torch.Tensor,
                     live_out: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    dev = torch._C._cuda_getDevice()
    if (table_out.shape != page_map.page_table.shape or ref_out.numel() != page_map.ref_count.numel()
            or live_out.numel() < 1):
        raise ValueError("table_out and ref_out need the shapes of page_table and ref_count, live_out one entry")
    st = _abi.lib().sfi_page_compact(
        ctypes.byref(page_map.c(dev)), ctypes.byref(pools.c()), _ptr_here(table_out, torch.int32, "table_out", dev),
        _ptr_here(ref_out, torch.int32, "ref_out", dev), _ptr_here(live_out, torch.int32, "live_out", dev),
        _ptr_here(workspace, torch.uint8, "workspace", dev), 0 if workspace is None else workspace.numel(),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_page_compact")


def sfi_page_workspace_size(page_map: PageMap) -> int:
    return int(_abi.lib().sfi_page_workspace_size(ctypes.byref(page_map.c())))


def alloc_page_workspace(page_map: PageMap) -> torch.Tensor:
    """A workspace of sfi_page_reserve and sfi_page_compact for this map."""
    return torch.empty(sfi_page_workspace_size(page_map), dtype=torch.uint8, device=page_map.ref_count.device)


def _pages_here(shape: AttnShape, kv: PagedKV, dev: int):
    """The C view of bf16 pages on the current device whose pools have the shape's heads; the number of requests."""
    c = kv.c(dev)
    k, v, table = kv.k_pool, kv.v_pool, kv.page_table
    if k.get_device() != dev or v.get_device() != dev or table.get_device() != dev or kv.seq_lens.get_device() != dev:
        for name in kv._tensors:
            _on_current_device(getattr(kv, name), name)
    dims, table = k.shape, table.shape
    if dims != (dims[0], shape.num_kv_heads, shape.page_size, shape.head_dim) or v.shape != dims:
        raise ValueError(f"the pools must be [num_pages][{shape.num_kv_heads}][{shape.page_size}][{shape.head_dim}]")
    if len(table) != 2 or kv.seq_lens.numel() != table[0]:
        raise ValueError("seq_lens needs one entry per row of page_table")
    return ctypes.byref(c), table[0]


def sfi_window_attn(shape: AttnShape, kv: PagedKV, sink: int, recent: int, q: torch.Tensor, out: torch.Tensor,
                    lse: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                    req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None):
    """Attention of each request's newest tokens through a sliding window with sinks; q [B][T][Hq][D]
    may be a view of a fused projection (contiguous heads), out bf16 [B][T][Hq][D], lse [B][T][Hq]."""
    dev = torch._C._cuda_getDevice()
    B, T, step = _token_rows(q, shape.num_q_heads, shape.head_dim, "q", dev)
    kv_c, requests = _pages_here(shape, kv, dev)
    _indexed(q, requests, "q")
    _indexed(new_lens, requests, "new_lens")
    _need_here(out, torch.bfloat16, "out", dev)
    if out.shape != q.shape or (lse is not None and lse.shape != q.shape[:3]):
        raise ValueError("out needs the shape of q, lse that without its last dimension")
    st = _abi.lib().sfi_window_attn(
        ctypes.byref(shape.c()), kv_c, int(sink), int(recent), q.data_ptr(), step, B, T,
        _ptr_here(new_lens, torch.int32, "new_lens", dev), out.data_ptr(), _ptr_here(lse, torch.float32, "lse", dev),
        _ptr_here(req_ids, torch.int32, "req_ids", dev), _count(B, batch, req_ids),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_window_attn")


def _weights(shape: AttnShape, mass: torch.Tensor, requests: int, name: str, dev: int) -> int:
    """The row stride of a [B][Hkv][stride] tensor of weights."""
    _need_here(mass, torch.float32, name, dev)
    dims = mass.shape
    if len(dims) != 3 or dims[0] != requests or dims[1] != shape.num_kv_heads:
        raise ValueError(f"{name} must be [{requests}][{shape.num_kv_heads}][stride], got {list(dims)}")
    return dims[2]


def sfi_attn_mass(shape: AttnShape, kv: PagedKV, sink: int, recent: int, q: torch.Tensor, lse: torch.Tensor,
                  mass: torch.Tensor, decay: float = 1.0, new_lens: Optional[torch.Tensor] = None,
                  req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None):
    """The attention weights of the newest tokens, added up per position into mass [B][Hkv][stride] (its former
    values times decay); q and lse as for sfi_window_attn."""
    dev = torch._C._cuda_getDevice()
    B, T, step = _token_rows(q, shape.num_q_heads, shape.head_dim, "q", dev)
    kv_c, requests = _pages_here(shape, kv, dev)
    _indexed(q, requests, "q")
    _indexed(new_lens, requests, "new_lens")
    _need_here(lse, torch.float32, "lse", dev)
    if lse.shape != q.shape[:3]:
        raise ValueError("lse needs the shape of q without its last dimension")
    st = _abi.lib().sfi_attn_mass(
        ctypes.byref(shape.c()), kv_c, int(sink), int(recent), q.data_ptr(), step, B, T,
        _ptr_here(new_lens, torch.int32, "new_lens", dev), lse.data_ptr(), mass.data_ptr(),
        _weights(shape, mass, requests, "mass", dev), float(decay), _ptr_here(req_ids, torch.int32, "req_ids", dev),
        _count(B, batch, req_ids), _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_attn_mass")


def sfi_kv_evict(shape: AttnShape, kv: PagedKV, mass: torch.Tensor, sink: int, recent: int, k_per_req: torch.Tensor,
                 idx_out: torch.Tensor, count_out: torch.Tensor, new_lens: torch.Tensor,
                 mass_out: Optional[torch.Tensor] = None, req_ids: Optional[torch.Tensor] = None,
                 batch: Optional[int] = None, dev_status: Optional[torch.Tensor] = None, stream=None):
    """Cuts each request's pages to its sink, its recent window and the k_per_req heaviest positions between;
    mass, mass_out [B][Hkv][stride], idx_out int32 [B][Hkv][k_cap], count_out and new_lens int32 [B]."""
    dev = torch._C._cuda_getDevice()
    kv_c, requests = _pages_here(shape, kv, dev)
    stride = _weights(shape, mass, requests, "mass", dev)
    if mass_out is not None and _weights(shape, mass_out, requests, "mass_out", dev) != stride:
        raise ValueError("mass and mass_out need the same shape")
    dims = idx_out.shape
    if len(dims) != 3 or dims[0] != requests or dims[1] != shape.num_kv_heads:
        raise ValueError(f"idx_out must be [{requests}][{shape.num_kv_heads}][k_cap], got {list(dims)}")
    for t, name in ((k_per_req, "k_per_req"), (count_out, "count_out"), (new_lens, "new_lens")):
        _need_here(t, torch.int32, name, dev)
        _indexed(t, requests, name)
    st = _abi.lib().sfi_kv_evict(
        ctypes.byref(shape.c()), kv_c, mass.data_ptr(), stride, int(sink), int(recent), k_per_req.data_ptr(), dims[2],
        _ptr_here(idx_out, torch.int32, "idx_out", dev), count_out.data_ptr(),
        None if mass_out is None else mass_out.data_ptr(), new_lens.data_ptr(),
        _ptr_here(req_ids, torch.int32, "req_ids", dev), _count(requests, batch, req_ids),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_kv_evict")


def _probability_rows(t: torch.Tensor, name: str, dev: int):
    """Requests, rows, values of a row and elements between rows of an fp32 tensor [B][rows][V]."""
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        _on_current_device(t, name)
    if t.dtype is not torch.float32:
        raise ValueError(f"{name} must be {torch.float32}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [B][rows][V], got {list(t.shape)}")
    b, n, v = t.shape
    s = t.stride()
    step = s[1] if n > 1 else (s[0] if b > 1 else v)
    if (v > 1 and s[2] != 1) or step < v or (b > 1 and s[0] != n * step):
        raise ValueError(f"{name} needs contiguous rows and one stride between all rows")
    return b, n, v, step


def sfi_verify_tokens(target: torch.Tensor, draft: Optional[torch.Tensor], tokens: torch.Tensor, u: torch.Tensor,
                      out_tokens: torch.Tensor, accepted: torch.Tensor, draft_lens: Optional[torch.Tensor] = None,
                      seq_lens: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                      req_ids: Optional[torch.Tensor] = None, batch: Optional[int] = None,
                      dev_status: Optional[torch.Tensor] = None, stream=None):
    """Which drafts the target keeps, and the token behind them: target fp32 [B][T + 1][V], draft fp32 [B][T][V] (None:
    the drafts were chosen, not drawn), tokens int32 [B][T], u fp32 [B][T + 1], out_tokens int32 [B][T + 1]."""
    dev = torch._C._cuda_getDevice()
    B, rows, V, ts = _probability_rows(target, "target", dev)
    T, ds = rows - 1, 0
    if draft is not None:
        db, dt, dv, ds = _probability_rows(draft, "draft", dev)
        if db != B or dt != T or dv != V:
            raise ValueError(f"draft must be [{B}][{T}][{V}], got {list(draft.shape)}")
    for t, dtype, name, dims in ((tokens, torch.int32, "tokens", (B, T)), (u, torch.float32, "u", (B, T + 1)),
                                 (out_tokens, torch.int32, "out_tokens", (B, T + 1)),
                                 (accepted, torch.int32, "accepted", (B,))):
        _need_here(t, dtype, name, dev)
        if tuple(t.shape) != dims:
            raise ValueError(f"{name} must be {list(dims)}, got {list(t.shape)}")
    for t, name in ((draft_lens, "draft_lens"), (seq_lens, "seq_lens"), (new_lens, "new_lens")):
        _indexed(t, B, name)
    st = _abi.lib().sfi_verify_tokens(
        target.data_ptr(), ts, None if draft is None else draft.data_ptr(), ds, tokens.data_ptr(), u.data_ptr(), V, T,
        _ptr_here(draft_lens, torch.int32, "draft_lens", dev), _ptr_here(seq_lens, torch.int32, "seq_lens", dev),
        out_tokens.data_ptr(), accepted.data_ptr(), _ptr_here(new_lens, torch.int32, "new_lens", dev),
        _ptr_here(req_ids, torch.int32, "req_ids", dev), _count(B, batch, req_ids),
        _ptr_here(dev_status, torch.int32, "dev_status", dev), _stream_here(stream, dev))
    _check(st, "sfi_verify_tokens")


def sfi_workspace_size(shape: AttnShape, batch: int, max_tokens: int, num_splits: int = 0) -> int:
    return int(_abi.lib().sfi_workspace_size(ctypes.byref(shape.c()), int(batch), int(max_tokens), int(num_splits)))


def sfi_plan_splits(shape: AttnShape, batch: int, max_tokens: int, num_splits: int = 0) -> int:
    return int(_abi.lib().sfi_plan_splits(ctypes.byref(shape.c()), int(batch), int(max_tokens), int(num_splits)))


def sfi_attn_cluster_capacity(cluster_size: int) -> int:
    return int(_abi.lib().sfi_attn_cluster_capacity(int(cluster_size)))


def sfi_version() -> int:
    return int(_abi.lib().sfi_version())


def alloc_workspace(shape: AttnShape, batch: int, max_tokens: int, num_splits: int = 0, device="cuda",
                    any_subset: bool = True) -> torch.Tensor:
    """A zero-filled workspace (at least 256 bytes; torch allocations are 256-byte aligned).

    With any_subset, it is large enough for every batch size 1..batch (calls on a
    subset of the requests plan their splits for the subset's size).
    """
    sizes = range(1, batch + 1) if any_subset else [batch]
    n = max([256] + [sfi_workspace_size(shape, b, max_tokens, num_splits) for b in sizes])
    return torch.zeros(n, dtype=torch.uint8, device=device)
