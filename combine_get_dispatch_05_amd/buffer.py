"""PyTorch-facing façade over libep.so with the call shapes of the pages' Buffer.

"DeepEP Buffer Class API for Expert Parallel Communication" describes a
``Buffer`` with ``get_dispatch_layout``, ``dispatch`` (6 results),
``combine`` (3 results), ``low_latency_dispatch`` (5 results),
``low_latency_combine`` (3 results), the low-latency mask-buffer utilities
and ``destroy``; "Chapter 10, V2: buffers beyond EP" (10.2) adds
``lb_prefetch_weights`` and ``lb_reduce_grads``.  This class keeps those
names and result arities so callers can switch; the slots that carried a CUDA
event or receive hook hold ``None`` (work is ordered on torch's current
stream instead).  The R ranks are logical partitions of this GPU's memory.

Only argument marshalling happens here: every step runs in the HIP kernels
behind the C ABI.  Tensors must live on the current CUDA (HIP) device.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass, fields
from functools import lru_cache
from typing import Optional

import torch

from . import abi


def _need(t: torch.Tensor, dtype, name: str, ndim: int):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _shape(t: torch.Tensor, shape, name: str):
    # The C ABI takes bare pointers, so every extent the kernels will index
    # is checked here, before a launch could read or write past a tensor.
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _same_device(*ts):
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        raise ValueError(f"tensors on different devices: {sorted(map(str, devs))}")


def _row(t: torch.Tensor, dtype, shape, name: str):
    """_need and _shape in one look where all is well: the small calls' host time counts."""
    if not (t.dtype == dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
        _need(t, dtype, name, len(shape))
        _shape(t, shape, name)


def _here(*ts) -> int:
    """The index of the tensors' one device, which has to be the current one: kernels go
    to its current stream."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != dev:
            _same_device(*ts)
            raise ValueError(f"tensors are on {t.device}, the current device is cuda:{dev}")
    return dev


def _fp8_pair(pair, name: str, ndim: int, row_blocks: bool):
    """Checks (codes, scales): codes float8_e4m3fn or uint8 with a last dimension
    of whole 128-element blocks, and one fp32 scale per block of a row (or, with
    row_blocks, per 128 x 128 block of a weight).  Returns both."""
    if not isinstance(pair, (tuple, list)) or len(pair) != 2:
        raise TypeError(f"{name} must be a pair (codes, scales)")
    q, sc = pair
    if q.dtype != torch.float8_e4m3fn:
        _need(q, torch.uint8, f"{name} codes", ndim)
    elif not (q.dim() == ndim and q.is_cuda and q.is_contiguous()):
        _need(q, torch.float8_e4m3fn, f"{name} codes", ndim)
    *lead, rows, width = q.shape
    if width % 128:
        raise ValueError(f"{name}: rows must be whole 128-element blocks")
    _row(sc, torch.float32, (*lead, -(-rows // 128) if row_blocks else rows, width // 128), f"{name} scales")
    return q, sc


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, use_fp8: bool = False, bf16_out: bool = True):
    """Root-mean-square norm of bf16 rows x [T, H], with residual [T, H] added
    first.  Returns (out, fp8, residual_out, rstd): out [T, H] bf16 (None without
    bf16_out), with use_fp8 the pair (codes [T, H] float8_e4m3fn, scales [T, H/128])
    in the format of low_latency_dispatch(use_fp8=True), the bf16 sum x + residual
    (None without residual) and rstd [T] fp32, which the backward pass takes."""
    _need(x, torch.bfloat16, "x", 2)
    T, H = x.shape
    _row(weight, torch.bfloat16, (H,), "weight")
    if residual is not None:
        _row(residual, torch.bfloat16, (T, H), "residual")
    if not (use_fp8 or bf16_out):
        raise ValueError("nothing to return: neither bf16_out nor use_fp8")
    if use_fp8 and H % 128:
        raise ValueError("use_fp8 needs rows of whole 128-element blocks")
    dev = _here(x, weight, residual)
    out = torch.empty_like(x) if bf16_out else None
    fp8 = (torch.empty_like(x, dtype=torch.float8_e4m3fn),
           torch.empty((T, H // 128), dtype=torch.float32, device=x.device)) if use_fp8 else (None, None)
    res = torch.empty_like(x) if residual is not None else None
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    if T > 0:
        at = abi.address
        abi.check(abi.lib().ep_rms_norm(T, H, eps, x.data_ptr(), at(residual), weight.data_ptr(), at(res),
                                        at(out), at(fp8[0]), at(fp8[1]), rstd.data_ptr(),
                                        abi.raw_stream(dev)), "ep_rms_norm")
    return out, fp8 if use_fp8 else None, res, rstd


def rms_norm_backward(dout: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      dresidual: Optional[torch.Tensor] = None):
    """Gradients of rms_norm: h is its residual_out (x without a residual), dresidual
    the gradient that arrived at residual_out.  Returns (dx [T, H] bf16, the gradient
    of x and of residual alike, and dweight [H] fp32)."""
    _need(dout, torch.bfloat16, "dout", 2)
    T, H = dout.shape
    _row(h, torch.bfloat16, (T, H), "h")
    _row(weight, torch.bfloat16, (H,), "weight")
    _row(rstd, torch.float32, (T,), "rstd")
    if dresidual is not None:
        _row(dresidual, torch.bfloat16, (T, H), "dresidual")
    dev = _here(dout, h, weight, rstd, dresidual)
    dx = torch.empty_like(dout)
    dweight = torch.empty(H, dtype=torch.float32, device=dout.device)
    size = abi.lib().ep_rms_norm_backward_workspace(T, H)
    work = torch.empty(size, dtype=torch.uint8, device=dout.device)
    abi.check(abi.lib().ep_rms_norm_backward(T, H, dout.data_ptr(), h.data_ptr(), weight.data_ptr(),
                                             rstd.data_ptr(), abi.address(dresidual), dx.data_ptr(),
                                             dweight.data_ptr(), work.data_ptr(), size,
                                             abi.raw_stream(dev)), "ep_rms_norm_backward")
    return dx, dweight


def fp8_product(a, w) -> torch.Tensor:
    """a (codes [M, K], scales [M, K/128]) times the transpose of w (codes [N, K],
    scales [ceil(N/128), K/128]), both float8_e4m3fn with fp32 scales: bf16 [M, N].
    Blocks are summed in fp32; inside one, of each eight products of neighbouring k the
    smaller seven can each lose up to 2^-13 of the largest (the matrix instruction aligns
    them)."""
    aq, asc = _fp8_pair(a, "a", 2, False)
    wq, wsc = _fp8_pair(w, "w", 2, True)
    (M, K), N = aq.shape, wq.shape[0]
    _shape(wq, (N, K), "w codes")
    dev = _here(aq, asc, wq, wsc)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=aq.device)
    if M > 0:
        abi.check(abi.lib().ep_fp8_product(M, N, K, aq.data_ptr(), asc.data_ptr(), wq.data_ptr(),
                                           wsc.data_ptr(), out.data_ptr(), abi.raw_stream(dev)),
                  "ep_fp8_product")
    return out


def _int32(n: int, name: str):
    if not -(1 << 31) <= n < 1 << 31:  # (ctypes would wrap it)
        raise ValueError(f"{name} must fit 32 bits, got {n}")


# The small calls' host time counts: the library is asked once for each size.
@lru_cache(maxsize=4096)
def _workspace(name: str, dims, *rest) -> int:
    for n in (*dims, *rest):
        _int32(n, "a size")
    return getattr(abi.lib(), name)(ctypes.byref(abi.Dims(*dims)), *rest)


@lru_cache(maxsize=4096)
def _adapter_workspace(T: int, K: int, N: int, r: int, L: int, back: int) -> int:
    for n in (T, K, N, r, L):
        _int32(n, "a size")
    return abi.lib().ep_adapter_workspace(ctypes.byref(abi.AdapterDims(T, K, N, r, L)), back)


def _adapter_args(x, adapter_ids, down, up, scales):
    _need(x, torch.bfloat16, "x", 2)
    _need(down, torch.bfloat16, "down", 3)
    _need(up, torch.bfloat16, "up", 3)
    (T, K), (L, r, _), N = x.shape, down.shape, up.shape[1]
    _row(adapter_ids, torch.int64, (T,), "adapter_ids")
    _shape(down, (L, r, K), "down")
    _shape(up, (L, N, r), "up")
    _row(scales, torch.float32, (L,), "scales")
    return T, K, N, r, L


def adapter_product(x: torch.Tensor, adapter_ids: torch.Tensor, down: torch.Tensor, up: torch.Tensor,
                    scales: torch.Tensor, base: Optional[torch.Tensor] = None, save: bool = False):
    """Low-rank adapters of many requests beside a shared projection: out[t] = base[t] + scales[a]
    (x[t] down_a^T) up_a^T with a = adapter_ids[t] (int64 [T]; outside [0, L): no adapter).  x [T, K] and
    base [T, N] (the projection's output; None: zeros) bf16, down [L, r, K], up [L, N, r] bf16 with r up to
    128, scales [L] fp32.  Returns (out [T, N] bf16, hidden): hidden [2, T, r] bf16, the rows' r values as
    sums of two, is what adapter_product_backward takes, None without save."""
    d = T, K, N, r, L = _adapter_args(x, adapter_ids, down, up, scales)
    if base is not None:
        _row(base, torch.bfloat16, (T, N), "base")
    dev, at = _here(x, adapter_ids, down, up, scales, base), x.device
    out = torch.empty(T, N, dtype=torch.bfloat16, device=at)
    hidden = torch.empty(2, T, r, dtype=torch.bfloat16, device=at) if save else None
    size = _adapter_workspace(*d, 0)
    work = torch.empty(size, dtype=torch.uint8, device=at) if size else None
    abi.check(abi.lib().ep_adapter_product(
        ctypes.byref(abi.AdapterDims(*d)), x.data_ptr(), adapter_ids.data_ptr(), down.data_ptr(), up.data_ptr(),
        scales.data_ptr(), abi.address(base), out.data_ptr(), abi.address(hidden), abi.address(work), size,
        abi.raw_stream(dev)), "ep_adapter_product")
    return out, hidden


def adapter_product_backward(dy: torch.Tensor, x: torch.Tensor, adapter_ids: torch.Tensor, down: torch.Tensor,
                             up: torch.Tensor, scales: torch.Tensor, hidden: torch.Tensor,
                             dx_base: Optional[torch.Tensor] = None):
    """Gradients of adapter_product given dy [T, N] bf16 (base's gradient is dy itself).  dx_base [T, K] bf16 is
    the projection's own gradient of x, to which the adapters' is added.  Returns (dx [T, K], ddown, dup), bf16;
    an adapter without tokens has zeros."""
    d = T, K, N, r, L = _adapter_args(x, adapter_ids, down, up, scales)
    _row(dy, torch.bfloat16, (T, N), "dy")
    _row(hidden, torch.bfloat16, (2, T, r), "hidden")
    if dx_base is not None:
        _row(dx_base, torch.bfloat16, (T, K), "dx_base")
    dev = _here(dy, x, adapter_ids, down, up, scales, hidden, dx_base)
    dx, ddown, dup = torch.empty_like(x), torch.empty_like(down), torch.empty_like(up)
    size = _adapter_workspace(*d, 1)
    work = torch.empty(size, dtype=torch.uint8, device=x.device)
    abi.check(abi.lib().ep_adapter_product_backward(
        ctypes.byref(abi.AdapterDims(*d)), dy.data_ptr(), x.data_ptr(), adapter_ids.data_ptr(), down.data_ptr(),
        up.data_ptr(), scales.data_ptr(), hidden.data_ptr(), abi.address(dx_base), dx.data_ptr(), ddown.data_ptr(),
        dup.data_ptr(), work.data_ptr(), size, abi.raw_stream(dev)), "ep_adapter_product_backward")
    return dx, ddown, dup


@dataclass(frozen=True)
class Router:
    """How experts are chosen from logits and weighted (include/ep.h, ep_router): num_topk of them
    by softmax or sigmoid scores, from the topk_groups best of num_groups groups, the
    weights divided by the chosen ones' sum (normalize) and multiplied by scale."""

    num_topk: int
    score: str = "softmax"
    num_groups: int = 1
    topk_groups: int = 1
    normalize: bool = True
    scale: float = 1.0

    def __post_init__(self):
        if self.score not in ("softmax", "sigmoid"):
            raise ValueError(f"score must be softmax or sigmoid, got {self.score!r}")
        if (self.num_topk | self.num_groups | self.topk_groups) >> 31:
            for n in (self.num_topk, self.num_groups, self.topk_groups):
                _int32(n, "a router's count")
        rule = abi.RouterRule(self.score == "sigmoid", self.num_groups, self.topk_groups, bool(self.normalize), self.scale)
        object.__setattr__(self, "_raw", ctypes.byref(rule))  # (which keeps it alive)

    def __reduce__(self):  # (an address is neither copied nor pickled)
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


@dataclass
class Layout:
    """Device copies of a dispatch layout ("What the Handle Contains")."""

    num_tokens_per_rank: torch.Tensor  # int32 [R]
    num_tokens_per_expert: torch.Tensor  # int32 [E]
    is_token_in_rank: torch.Tensor  # bool [T, R]
    rank_prefix_matrix: torch.Tensor  # int32 [R]
    channel_prefix_matrix: torch.Tensor  # int32 [R, C]
    recv_channel_prefix_matrix: torch.Tensor  # int32 [R, C]
    send_head: torch.Tensor  # int32 [T, R]
    recv_src_idx: torch.Tensor  # int32 [N]


class Handle:
    """Opaque dispatch layout owned by the library (freed on ``free()`` or
    garbage collection, ordered after the work already enqueued)."""

    def __init__(self, raw: int, d: abi.Dims, device: torch.device):
        self._raw = raw
        self.dims = d
        self.device = device

    @property
    def raw(self) -> ctypes.c_void_p:
        if not self._raw:
            raise ValueError("handle already freed")
        return ctypes.c_void_p(self._raw)

    @property
    def num_recv(self) -> int:
        """N, the number of packed rows (reads it back once)."""
        n = ctypes.c_int64(0)
        abi.check(abi.lib().ep_handle_num_recv(self.raw, ctypes.byref(n)), "ep_handle_num_recv")
        return int(n.value)

    @property
    def nbytes(self) -> int:
        return int(abi.lib().ep_handle_nbytes(self.raw))

    def layout(self) -> Layout:
        d = self.dims
        T, R, E, C = d.num_tokens, d.num_ranks, d.num_experts, d.num_channels
        n = self.num_recv
        i32 = dict(dtype=torch.int32, device=self.device)
        lay = Layout(torch.empty(R, **i32), torch.empty(E, **i32),
                     torch.empty((T, R), dtype=torch.uint8, device=self.device),
                     torch.empty(R, **i32), torch.empty((R, C), **i32), torch.empty((R, C), **i32),
                     torch.empty((T, R), **i32), torch.empty(max(n, 1), **i32))
        out = abi.LayoutOut(lay.num_tokens_per_rank.data_ptr(), lay.num_tokens_per_expert.data_ptr(),
                            lay.is_token_in_rank.data_ptr(), lay.rank_prefix_matrix.data_ptr(),
                            lay.channel_prefix_matrix.data_ptr(),
                            lay.recv_channel_prefix_matrix.data_ptr(), lay.send_head.data_ptr(),
                            lay.recv_src_idx.data_ptr(), n)
        abi.check(abi.lib().ep_handle_copy_layout(self.raw, ctypes.byref(out), abi.current_stream()),
                  "ep_handle_copy_layout")
        lay.is_token_in_rank = lay.is_token_in_rank.view(torch.bool)
        lay.recv_src_idx = lay.recv_src_idx[:n]
        return lay

    def free(self) -> None:
        if self._raw:
            abi.lib().ep_handle_free(ctypes.c_void_p(self._raw))
            self._raw = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


@dataclass
class LowLatencyHandle:
    """What low_latency_combine needs to find each (token, slot)'s cell."""

    src_info: torch.Tensor  # int32 [E/R, R, slots]
    topk_slot: torch.Tensor  # int32 [T, K]
    num_slots: int
    num_experts: int
    hidden: int


@dataclass
class ExpertRows:
    """Dispatched rows grouped by expert (expert_rows): pairs (row, slot) sorted by
    (expert, row, slot).  The pair tensors have room for every slot of the batch."""

    expert_offsets: torch.Tensor  # int32 [E + 1]
    pair_row: torch.Tensor  # int32 [pairs], sign bit: the only pair of its row
    pair_slot: torch.Tensor  # int32 [pairs], row * K + slot
    row_pair: torch.Tensor  # int32 [rows, K], -1 for a slot without a pair

    def _check(self, num_experts: int) -> None:
        # the kernels take all four as they are, so each is looked at in every call
        i32 = torch.int32
        _row(self.expert_offsets, i32, (num_experts + 1,), "the rows' expert_offsets")
        _row(self.pair_row, i32, (self.pair_row.shape[0] if self.pair_row.dim() else 0,), "the rows' pair_row")
        _row(self.pair_slot, i32, self.pair_row.shape, "the rows' pair_slot")
        _need(self.row_pair, i32, "the rows' row_pair", 2)

    def _tensors(self):
        return self.expert_offsets, self.pair_row, self.pair_slot, self.row_pair

    def _raw(self) -> abi.ExpertGroups:
        return abi.ExpertGroups(self.row_pair.shape[0], self.pair_row.shape[0],
                                self.expert_offsets.data_ptr(), self.pair_row.data_ptr(),
                                self.pair_slot.data_ptr(), self.row_pair.data_ptr())


class Buffer:
    """Expert-parallel layout / dispatch / combine over R logical ranks of one GPU."""

    def __init__(self, num_ranks: int, num_experts: int, num_channels: int = 1):
        if num_experts % num_ranks:
            raise ValueError("num_experts must be a multiple of num_ranks")
        self.num_ranks = int(num_ranks)
        self.num_experts = int(num_experts)
        self.num_channels = int(num_channels)
        self.destroyed = False
        self._mask = None  # device int32 [R], created by the first mask update

    # ------------------------------------------------------- rank masking
    def _mask_ptr(self):
        return abi.ptr(self._mask) if self._mask is not None else None

    def low_latency_update_mask_buffer(self, rank_to_mask: int, mask: bool = False) -> None:
        """Mask (True) or unmask (False) one rank for the low-latency calls."""
        if self._mask is None:
            self._mask = torch.zeros(self.num_ranks, dtype=torch.int32, device="cuda")
        abi.check(abi.lib().ep_mask_update(abi.ptr(self._mask), self.num_ranks, int(rank_to_mask),
                                           1 if mask else 0, abi.current_stream()),
                  "ep_mask_update")

    def low_latency_query_mask_buffer(self, mask_status: torch.Tensor) -> None:
        """Write the mask (0 active, 1 masked) into a CPU int32 tensor [R]."""
        if (mask_status.dtype != torch.int32 or mask_status.numel() != self.num_ranks
                or mask_status.is_cuda or not mask_status.is_contiguous()):
            raise ValueError("mask_status must be a contiguous CPU int32 tensor with one entry "
                             "per rank")
        if self._mask is None:
            mask_status.zero_()
            return
        abi.check(abi.lib().ep_mask_query(abi.ptr(self._mask), self.num_ranks,
                                          ctypes.c_void_p(mask_status.data_ptr()),
                                          abi.current_stream()), "ep_mask_query")

    def low_latency_clean_mask_buffer(self) -> None:
        """Mark every rank active again."""
        if self._mask is not None:
            abi.check(abi.lib().ep_mask_clean(abi.ptr(self._mask), self.num_ranks,
                                              abi.current_stream()), "ep_mask_clean")

    @property
    def num_local_experts(self) -> int:
        return self.num_experts // self.num_ranks

    def _dims(self, T: int, H: int, K: int) -> abi.Dims:
        return abi.dims(T, H, K, self.num_experts, self.num_ranks, self.num_channels)

    # -------------------------------------------------------------- layout
    def get_dispatch_layout(self, topk_idx: torch.Tensor, keep_handle: bool = False):
        """Returns (num_tokens_per_rank [R], num_tokens_per_expert [E],
        is_token_in_rank [T, R] bool, handle or None).  A kept handle can be
        passed to one ``dispatch`` together with the same ``topk_idx``.
        Ranks masked in the mask buffer receive nothing (their slots act as
        masked slots)."""
        _need(topk_idx, torch.int64, "topk_idx", 2)
        T, K = topk_idx.shape
        d = self._dims(T, 8, K)
        dev = topk_idx.device
        ntpr = torch.empty(self.num_ranks, dtype=torch.int32, device=dev)
        ntpe = torch.empty(self.num_experts, dtype=torch.int32, device=dev)
        itr = torch.empty((T, self.num_ranks), dtype=torch.uint8, device=dev)
        out = abi.LayoutOut(ntpr.data_ptr(), ntpe.data_ptr(), itr.data_ptr(), None, None, None,
                            None, None, 0)
        raw = ctypes.c_void_p()
        rc = abi.lib().ep_get_dispatch_layout(ctypes.byref(d), abi.ptr(topk_idx),
                                              abi.ptr(self._mask), ctypes.byref(out),
                                              ctypes.byref(raw) if keep_handle else None,
                                              abi.current_stream())
        h = Handle(raw.value, d, dev) if keep_handle and raw.value else None
        abi.check(rc, "ep_get_dispatch_layout")
        return ntpr, ntpe, itr.view(torch.bool), h

    # ------------------------------------------------------------ dispatch
    def dispatch(self, x: torch.Tensor, topk_idx: Optional[torch.Tensor] = None,
                 topk_weights: Optional[torch.Tensor] = None, handle: Optional[Handle] = None):
        """Returns (recv_x [N, H], recv_topk_idx [N, K] or None,
        recv_topk_weights [N, K] or None, num_recv_tokens_per_expert [R, E/R],
        handle, None).  Without a handle the layout is computed and N is read
        back (one host sync); with a handle from an earlier dispatch only the
        rows are packed and topk arguments are refused.  A fresh dispatch
        leaves out the ranks masked in the mask buffer."""
        _need(x, torch.bfloat16, "x", 2)
        T, H = x.shape
        if handle is None and topk_idx is None:
            raise ValueError("dispatch without a handle needs topk_idx")
        if topk_idx is not None:
            _need(topk_idx, torch.int64, "topk_idx", 2)
            if topk_idx.shape[0] != T:
                raise ValueError("topk_idx and x disagree on the number of tokens")
        if topk_weights is not None:
            if topk_idx is None:
                raise ValueError("topk_weights needs topk_idx")
            _need(topk_weights, torch.float32, "topk_weights", 2)
            _shape(topk_weights, topk_idx.shape, "topk_weights")
        _same_device(x, topk_idx, topk_weights)
        K = topk_idx.shape[1] if topk_idx is not None else handle.dims.num_topk
        d = self._dims(T, H, K)
        dev = x.device
        if handle is not None and handle.device != dev:
            raise ValueError("handle was made on another device")
        raw = ctypes.c_void_p(handle.raw.value if handle is not None else None)
        if handle is not None and handle.dims.num_tokens != T:
            raise ValueError("handle was made for another number of tokens")
        cap = handle.num_recv if handle is not None else int(abi.lib().ep_max_recv_rows(ctypes.byref(d)))
        recv_x = torch.empty((cap, H), dtype=torch.bfloat16, device=dev)
        rti = torch.empty((cap, K), dtype=torch.int64, device=dev) if topk_idx is not None else None
        rtw = torch.empty((cap, K), dtype=torch.float32, device=dev) if topk_weights is not None else None
        n = ctypes.c_int64(-1)
        mask = abi.ptr(self._mask) if handle is None else None
        rc = abi.lib().ep_dispatch(ctypes.byref(d), abi.ptr(x), abi.ptr(topk_idx),
                                   abi.ptr(topk_weights), mask, ctypes.byref(raw),
                                   abi.ptr(recv_x),
                                   abi.ptr(rti), abi.ptr(rtw), cap, ctypes.byref(n),
                                   abi.current_stream())
        if handle is None and raw.value:
            # owned from here on, so an error below still frees it
            handle = Handle(raw.value, d, dev)
        abi.check(rc, "ep_dispatch")
        N = int(n.value)
        lay_counts = None
        if topk_idx is not None:
            lay_counts = self._expert_counts(handle)
        return (recv_x[:N], rti[:N] if rti is not None else None,
                rtw[:N] if rtw is not None else None, lay_counts, handle, None)

    def _expert_counts(self, handle: Handle) -> torch.Tensor:
        ntpe = torch.empty(self.num_experts, dtype=torch.int32, device=handle.device)
        out = abi.LayoutOut(None, ntpe.data_ptr(), None, None, None, None, None, None, 0)
        abi.check(abi.lib().ep_handle_copy_layout(handle.raw, ctypes.byref(out),
                                                  abi.current_stream()),
                  "ep_handle_copy_layout")
        return ntpe.view(self.num_ranks, self.num_local_experts)

    # ------------------------------------------------------------- combine
    def combine(self, x: torch.Tensor, handle: Handle, topk_weights: Optional[torch.Tensor] = None,
                bias=None):
        """Returns (combined_x [T, H] bf16, combined_topk_weights [T, K] or
        None, None): the ascending-rank fp32 sum of each token's rows, plus
        the optional bias terms (a [T, H] bf16 tensor or a tuple of up to
        two), added before the single rounding.  Ranks masked in the mask
        buffer now are left out of the sums."""
        _need(x, torch.bfloat16, "x", 2)
        d = handle.dims
        if topk_weights is not None:
            _need(topk_weights, torch.float32, "topk_weights", 2)
            _shape(topk_weights, (x.shape[0], d.num_topk), "topk_weights")
        if handle.device != x.device:
            raise ValueError("handle was made on another device")
        T, H = d.num_tokens, x.shape[1]
        biases = [] if bias is None else ([bias] if isinstance(bias, torch.Tensor) else list(bias))
        if len(biases) > 2:
            raise ValueError("at most two bias tensors")
        for b in biases:
            _need(b, torch.bfloat16, "bias", 2)
            if tuple(b.shape) != (T, H):
                raise ValueError("bias must be [num_tokens, hidden]")
        _same_device(x, topk_weights, *biases)
        b0 = biases[0] if len(biases) > 0 else None
        b1 = biases[1] if len(biases) > 1 else None
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        cw = None
        if topk_weights is not None:
            cw = torch.empty((T, d.num_topk), dtype=torch.float32, device=x.device)
        abi.check(abi.lib().ep_combine(handle.raw, H, abi.ptr(x), x.shape[0], abi.ptr(topk_weights),
                                       abi.ptr(b0), abi.ptr(b1), abi.ptr(self._mask),
                                       abi.ptr(out), abi.ptr(cw),
                                       abi.current_stream()),
                  "ep_combine")
        return out, cw, None

    # --------------------------------------------------------- low latency
    def low_latency_dispatch(self, x: torch.Tensor, topk_idx: torch.Tensor,
                             num_max_dispatch_tokens_per_rank: int,
                             num_experts: Optional[int] = None, use_fp8: bool = False):
        """Returns (packed_x, packed_count [E/R, R], handle, None, None).
        packed_x is [E/R, R, slots, H] bf16, or with use_fp8 the pair
        (codes [E/R, R, slots, H] float8_e4m3fn, scales [E/R, R, slots, H/128]
        fp32).  Unused packed cells are left as allocated.  Ranks masked with
        low_latency_update_mask_buffer receive nothing."""
        if num_experts is not None and num_experts != self.num_experts:
            raise ValueError("num_experts differs from the buffer's")
        _need(x, torch.bfloat16, "x", 2)
        _need(topk_idx, torch.int64, "topk_idx", 2)
        T, H = x.shape
        K = topk_idx.shape[1]
        if topk_idx.shape[0] != T:
            raise ValueError("topk_idx and x disagree on the number of tokens")
        _same_device(x, topk_idx)
        S = int(num_max_dispatch_tokens_per_rank)
        d = self._dims(T, H, K)
        dev = x.device
        epr, R = self.num_local_experts, self.num_ranks
        count = torch.empty((epr, R), dtype=torch.int32, device=dev)
        src = torch.empty((epr, R, S), dtype=torch.int32, device=dev)
        slot = torch.empty((T, K), dtype=torch.int32, device=dev)
        if use_fp8:
            q = torch.empty((epr, R, S, H), dtype=torch.uint8, device=dev)
            sc = torch.empty((epr, R, S, H // 128), dtype=torch.float32, device=dev)
            abi.check(abi.lib().ep_ll_dispatch_fp8(ctypes.byref(d), S, abi.ptr(x), abi.ptr(topk_idx),
                                                   self._mask_ptr(), abi.ptr(q), abi.ptr(sc),
                                                   abi.ptr(count), abi.ptr(src), abi.ptr(slot),
                                                   abi.current_stream()),
                      "ep_ll_dispatch_fp8")
            packed = (q.view(torch.float8_e4m3fn), sc)
        else:
            packed = torch.empty((epr, R, S, H), dtype=torch.bfloat16, device=dev)
            abi.check(abi.lib().ep_ll_dispatch(ctypes.byref(d), S, abi.ptr(x), abi.ptr(topk_idx),
                                               self._mask_ptr(), abi.ptr(packed), abi.ptr(count),
                                               abi.ptr(src), abi.ptr(slot), abi.current_stream()),
                      "ep_ll_dispatch")
        return packed, count, LowLatencyHandle(src, slot, S, self.num_experts, H), None, None

    def low_latency_combine(self, x, topk_idx: torch.Tensor, topk_weights: torch.Tensor,
                            handle: LowLatencyHandle):
        """x has packed_x's layout [E/R, R, slots, H] (bf16), or is the FP8 pair
        (codes [E/R, R, slots, H] float8_e4m3fn or uint8, scales [E/R, R,
        slots, H/128] fp32) that low_latency_dispatch(use_fp8=True) returns,
        decoded with its scales in the sum.  Returns (combined_x [T, H] bf16,
        None, None)."""
        _need(topk_idx, torch.int64, "topk_idx", 2)
        _need(topk_weights, torch.float32, "topk_weights", 2)
        T, K = topk_idx.shape
        _shape(topk_weights, (T, K), "topk_weights")
        _shape(handle.topk_slot, (T, K), "the handle's topk_slot")
        if handle.num_experts != self.num_experts:
            raise ValueError("handle was made for another number of experts")
        cells = (self.num_local_experts, self.num_ranks, handle.num_slots)
        if isinstance(x, (tuple, list)):
            q, sc = x
            if q.dtype == torch.float8_e4m3fn:
                q = q.view(torch.uint8)
            _need(q, torch.uint8, "codes", 4)
            _need(sc, torch.float32, "scales", 4)
            H = q.shape[3]
            _shape(q, cells + (H,), "codes")
            if tuple(sc.shape) != tuple(q.shape[:3]) + (H // 128,):
                raise ValueError("scales must be [E/R, R, slots, H/128]")
            _same_device(q, sc, topk_idx, topk_weights, handle.topk_slot)
            d = self._dims(T, H, K)
            out = torch.empty((T, H), dtype=torch.bfloat16, device=q.device)
            abi.check(abi.lib().ep_ll_combine_fp8(ctypes.byref(d), handle.num_slots, abi.ptr(q),
                                                  abi.ptr(sc), abi.ptr(topk_idx),
                                                  abi.ptr(topk_weights), abi.ptr(handle.topk_slot),
                                                  self._mask_ptr(), abi.ptr(out),
                                                  abi.current_stream()),
                      "ep_ll_combine_fp8")
            return out, None, None
        _need(x, torch.bfloat16, "x", 4)
        H = x.shape[3]
        _shape(x, cells + (H,), "x")
        _same_device(x, topk_idx, topk_weights, handle.topk_slot)
        d = self._dims(T, H, K)
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
        abi.check(abi.lib().ep_ll_combine(ctypes.byref(d), handle.num_slots, abi.ptr(x),
                                          abi.ptr(topk_idx), abi.ptr(topk_weights),
                                          abi.ptr(handle.topk_slot), self._mask_ptr(),
                                          abi.ptr(out), abi.current_stream()),
                  "ep_ll_combine")
        return out, None, None

    # ------------------------------------------------------------- experts
    def _expert_weights(self, w13: torch.Tensor, w2: torch.Tensor, H: int) -> int:
        """Checks bf16 expert weights w13 [E, 2 I, H], w2 [E, H, I]; returns I."""
        _need(w13, torch.bfloat16, "w13", 3)
        _need(w2, torch.bfloat16, "w2", 3)
        inter = w2.shape[2]
        _shape(w13, (self.num_experts, 2 * inter, H), "w13")
        _shape(w2, (self.num_experts, H, inter), "w2")
        return inter

    def low_latency_expert_ffn(self, x, packed_count: torch.Tensor, handle: LowLatencyHandle, w13, w2,
                               out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The experts' gated feed-forward on the cells of low_latency_dispatch:
        act = silu(x Wg^T) * (x Wu^T), out = act W2^T for every used cell, in
        packed_x's layout [E/R, R, slots, H] bf16, which low_latency_combine takes.
        x is packed_x (bf16; w13 [E, 2 I, H] with the gate's rows first, w2 [E, H, I],
        bf16) or the FP8 pair of low_latency_dispatch(use_fp8=True) (w13 and w2 pairs
        of codes and scales [E, 2 I/128, H/128], [E, H/128, I/128]; the activation is
        quantised the same way between the products; an activation near a rounding border
        of its code can get the neighbouring one in a batch of another size, whose gate and
        up products take another kernel).  Unused cells of out are left as they were.
        packed_count must be that of the handle's dispatch."""
        _need(packed_count, torch.int32, "packed_count", 2)
        epr, R, S, H = self.num_local_experts, self.num_ranks, handle.num_slots, handle.hidden
        _shape(packed_count, (epr, R), "packed_count")
        if handle.num_experts != self.num_experts:
            raise ValueError("handle was made for another number of experts")
        T, K = handle.topk_slot.shape
        d = self._dims(T, H, K)
        cells = (epr, R, S)
        fp8 = isinstance(x, (tuple, list))
        if fp8:
            q, sc = _fp8_pair(x, "x", 4, False)
            _shape(q, cells + (H,), "x codes")
            (q13, s13), (q2, s2) = _fp8_pair(w13, "w13", 3, True), _fp8_pair(w2, "w2", 3, True)
            inter = q2.shape[2]
            _shape(q13, (self.num_experts, 2 * inter, H), "w13 codes")
            _shape(q2, (self.num_experts, H, inter), "w2 codes")
            dev = _here(q, sc, packed_count, q13, s13, q2, s2, handle.topk_slot, out)
        else:
            _need(x, torch.bfloat16, "x", 4)
            _shape(x, cells + (H,), "x")
            q = x
            inter = self._expert_weights(w13, w2, H)
            dev = _here(x, packed_count, w13, w2, handle.topk_slot, out)
        if out is None:
            out = torch.empty(cells + (H,), dtype=torch.bfloat16, device=q.device)
        else:
            _need(out, torch.bfloat16, "out", 4)
            _shape(out, cells + (H,), "out")
        if T == 0:
            return out
        s = abi.raw_stream(dev)
        if fp8:
            aq = torch.empty(cells + (inter,), dtype=torch.uint8, device=q.device)
            asc = torch.empty(cells + (inter // 128,), dtype=torch.float32, device=q.device)
            abi.check(abi.lib().ep_ll_expert_ffn_fp8(
                ctypes.byref(d), S, inter, abi.address(q), abi.address(sc), abi.address(packed_count),
                abi.address(q13), abi.address(s13), abi.address(q2), abi.address(s2), abi.address(aq),
                abi.address(asc), abi.address(out), s), "ep_ll_expert_ffn_fp8")
        else:
            act = torch.empty(cells + (inter,), dtype=torch.bfloat16, device=q.device)
            abi.check(abi.lib().ep_ll_expert_ffn(
                ctypes.byref(d), S, inter, abi.address(x), abi.address(packed_count), abi.address(w13),
                abi.address(w2), abi.address(act), abi.address(out), s), "ep_ll_expert_ffn")
        return out

    def expert_rows(self, recv_topk_idx: torch.Tensor, layout,
                    num_tokens: Optional[int] = None) -> ExpertRows:
        """Groups dispatched rows by expert.  recv_topk_idx [rows, K] is dispatch's;
        layout is its handle, or the rank_prefix_matrix (int32 [R]) together with
        num_tokens, the tokens of the batch (without it there is room for every slot
        of every row).  Rows at or past rank_prefix_matrix[-1] hold no pairs, so
        worst-case buffers can be given whole."""
        _need(recv_topk_idx, torch.int64, "recv_topk_idx", 2)
        N, K = recv_topk_idx.shape
        dev = recv_topk_idx.device
        if isinstance(layout, Handle):
            if layout.device != dev:
                raise ValueError("handle was made on another device")
            if layout.dims.num_experts != self.num_experts or layout.dims.num_ranks != self.num_ranks:
                raise ValueError("handle was made for other experts or ranks")
            num_tokens = layout.dims.num_tokens
            prefix = torch.empty(self.num_ranks, dtype=torch.int32, device=dev)
        else:
            prefix = layout
            _need(prefix, torch.int32, "rank_prefix_matrix", 1)
            _shape(prefix, (self.num_ranks,), "rank_prefix_matrix")
            num_tokens = N if num_tokens is None else int(num_tokens)
        index = _here(recv_topk_idx, prefix)
        if isinstance(layout, Handle):
            out = abi.LayoutOut(None, None, None, prefix.data_ptr(), None, None, None, None, 0)
            abi.check(abi.lib().ep_handle_copy_layout(layout.raw, ctypes.byref(out),
                                                      abi.raw_stream(index)), "ep_handle_copy_layout")
        cap = min(num_tokens, N) * K
        i32 = dict(dtype=torch.int32, device=dev)
        rows = ExpertRows(torch.empty(self.num_experts + 1, **i32), torch.empty(cap, **i32),
                          torch.empty(cap, **i32), torch.empty((N, K), **i32))
        counts = torch.empty(self.num_experts, **i32)
        abi.check(abi.lib().ep_expert_rows(
            ctypes.byref(self._dims(num_tokens, 8, K)), abi.address(prefix), abi.address(recv_topk_idx), N, cap,
            abi.address(counts), abi.address(rows.expert_offsets), abi.address(rows.pair_row),
            abi.address(rows.pair_slot), abi.address(rows.row_pair), abi.raw_stream(index)), "ep_expert_rows")
        return rows

    def _expert_args(self, x, rows: ExpertRows, topk_weights, w13, w2):
        rows._check(self.num_experts)
        _need(x, torch.bfloat16, "x", 2)
        N, H = x.shape
        K = rows.row_pair.shape[1]
        _shape(rows.row_pair, (N, K), "the rows' row_pair")
        _row(topk_weights, torch.float32, (N, K), "topk_weights")
        return N, H, K, self._expert_weights(w13, w2, H)

    def expert_ffn(self, x: torch.Tensor, rows: ExpertRows, topk_weights: torch.Tensor,
                   w13: torch.Tensor, w2: torch.Tensor, save: bool = False):
        """The experts between dispatch and combine: for every row of x [rows, H]
        (bf16) y = sum over its slots of topk_weights * (silu(x Wg^T) * (x Wu^T)) W2^T,
        zero for a row without a slot.  w13 [E, 2 I, H] (the gate's rows first) and
        w2 [E, H, I] are bf16.  Returns (y [rows, H] bf16, saved): saved is what
        expert_ffn_backward takes, the fp32 g and u of every pair, None without save.
        Workspace of a call: 4 H + 2 I bytes for every pair that rows has room for, so
        give expert_rows the number of tokens where it takes a bare prefix."""
        N, H, K, inter = self._expert_args(x, rows, topk_weights, w13, w2)
        index = _here(x, *rows._tensors(), topk_weights, w13, w2)
        dev, cap = x.device, rows.pair_row.shape[0]
        y = torch.empty_like(x)
        act = torch.empty((cap, inter), dtype=torch.bfloat16, device=dev)
        terms = torch.empty((cap, H), dtype=torch.float32, device=dev)
        saved = torch.empty((cap, 2 * inter), dtype=torch.float32, device=dev) if save else None
        raw = rows._raw()
        abi.check(abi.lib().ep_expert_ffn(
            ctypes.byref(self._dims(0, H, K)), inter, ctypes.byref(raw), abi.address(x),
            abi.address(topk_weights), abi.address(w13), abi.address(w2), abi.address(act), abi.address(saved),
            abi.address(terms), abi.address(y), abi.raw_stream(index)), "ep_expert_ffn")
        return y, saved

    def expert_ffn_backward(self, dy: torch.Tensor, x: torch.Tensor, rows: ExpertRows,
                            topk_weights: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                            saved: torch.Tensor):
        """Gradients of expert_ffn given dy [rows, H] bf16.  Returns (dx [rows, H] bf16,
        dtopk_weights [rows, K] fp32, dw13, dw2 bf16): dispatch's cached handle makes dy
        from the combined rows' gradient, combine sums dx and dtopk_weights back."""
        N, H, K, inter = self._expert_args(x, rows, topk_weights, w13, w2)
        _need(dy, torch.bfloat16, "dy", 2)
        _shape(dy, (N, H), "dy")
        cap, dev = rows.pair_row.shape[0], x.device
        _need(saved, torch.float32, "saved", 2)
        _shape(saved, (cap, 2 * inter), "saved")
        index = _here(dy, x, *rows._tensors(), topk_weights, w13, w2, saved)
        bf = dict(dtype=torch.bfloat16, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        dgu, act = torch.empty((cap, 2 * inter), **bf), torch.empty((cap, inter), **bf)
        terms, parts = torch.empty((cap, H), **f32), torch.empty((cap, -(-inter // 256)), **f32)
        dx, dweights = torch.empty_like(x), torch.empty((N, K), **f32)
        dw13, dw2 = torch.empty_like(w13), torch.empty_like(w2)
        raw = rows._raw()
        abi.check(abi.lib().ep_expert_ffn_backward(
            ctypes.byref(self._dims(0, H, K)), inter, ctypes.byref(raw), abi.address(dy), abi.address(x),
            abi.address(topk_weights), abi.address(w13), abi.address(w2), abi.address(saved), abi.address(dgu),
            abi.address(act), abi.address(terms), abi.address(parts), abi.address(dx), abi.address(dweights),
            abi.address(dw13), abi.address(dw2), abi.raw_stream(index)), "ep_expert_ffn_backward")
        return dx, dweights, dw13, dw2

    # -------------------------------------------------------------- router
    def _logits(self, logits: torch.Tensor) -> int:
        """Checks logits [T, E], fp32 or bf16; returns 1 for bf16."""
        bf16 = logits.dtype == torch.bfloat16
        if logits.dim() != 2:
            _need(logits, logits.dtype, "logits", 2)
        _row(logits, torch.bfloat16 if bf16 else torch.float32, (logits.shape[0], self.num_experts), "logits")
        if logits.shape[0] >> 31:
            _int32(logits.shape[0], "the number of tokens")
        return int(bf16)

    def route(self, logits: torch.Tensor, router: Router, bias: Optional[torch.Tensor] = None,
              score_sums: bool = False):
        """Chooses each token's experts from logits [T, E] (fp32 or bf16).  Returns (topk_idx [T, K]
        int64, topk_weights [T, K] fp32, sums): what dispatch and combine take, -1 with weight 0 where
        too few experts are left.  bias [E] fp32 is added to the scores for the choice alone.
        With score_sums, sums [E] fp32 is each expert's summed share of the tokens' scores, for a
        balancing loss.  Experts on ranks masked in the mask buffer, and those whose logit is -inf, are
        not chosen."""
        bf16 = self._logits(logits)
        T, K, E = logits.shape[0], router.num_topk, self.num_experts
        if bias is not None:
            _row(bias, torch.float32, (E,), "bias")
        dev, at, f32 = _here(logits, bias, self._mask), logits.device, torch.float32
        d = (T, 8, K, E, self.num_ranks, 1)
        idx = torch.empty(T, max(K, 0), dtype=torch.int64, device=at)
        weights = torch.empty(T, max(K, 0), dtype=f32, device=at)
        sums, work, size = None, None, 0
        if score_sums:
            sums = torch.empty(E, dtype=f32, device=at)
            size = _workspace("ep_route_workspace", d)
            work = torch.empty(size, dtype=torch.uint8, device=at)
        ptr = abi.address
        abi.check(abi.lib().ep_route(ctypes.byref(abi.Dims(*d)), router._raw, logits.data_ptr(), bf16, ptr(bias),
                                     ptr(self._mask), idx.data_ptr(), weights.data_ptr(), ptr(sums), ptr(work), size,
                                     abi.raw_stream(dev)), "ep_route")
        return idx, weights, sums

    def route_backward(self, dtopk_weights: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, router: Router,
                       dscore_sums: Optional[torch.Tensor] = None) -> torch.Tensor:
        """The gradient of route's logits (their type and shape) given those of topk_weights [T, K]
        fp32, as combine sums them back, and of the score sums [E] fp32.  topk_idx is route's."""
        bf16 = self._logits(logits)
        T, K = logits.shape[0], router.num_topk
        _row(dtopk_weights, torch.float32, (T, K), "dtopk_weights")
        _row(topk_idx, torch.int64, (T, K), "topk_idx")
        if dscore_sums is not None:
            _row(dscore_sums, torch.float32, (self.num_experts,), "dscore_sums")
        dev = _here(dtopk_weights, logits, topk_idx, dscore_sums)
        out = torch.empty_like(logits)
        abi.check(abi.lib().ep_route_backward(
            ctypes.byref(abi.Dims(T, 8, K, self.num_experts, self.num_ranks, 1)), router._raw, dtopk_weights.data_ptr(),
            logits.data_ptr(), bf16, topk_idx.data_ptr(), abi.address(dscore_sums), out.data_ptr(), abi.raw_stream(dev)),
            "ep_route_backward")
        return out

    # --------------------------------------------------------- whole layer
    def low_latency_moe(self, x: torch.Tensor, w_router: torch.Tensor, router: Router, w13, w2,
                        bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None):
        """A whole mixture-of-experts layer for up to 64 tokens x [T, H] bf16 and 512 experts, without
        dispatch and combine: logits x w_router^T (w_router [E, H] bf16 or fp32; summed in 64 bits),
        route (bias [E] fp32 for the choice alone), the chosen experts' gated feed-forward and the
        weighted sum, with residual [T, H] bf16 added.  w13 [E, 2 I, H] (the gate's rows first) and
        w2 [E, H, I] are bf16, or pairs (codes, scales) as for low_latency_expert_ffn; beside those too, x and
        the activation stay bf16.  Returns (y [T, H] bf16, topk_idx [T, K] int64, topk_weights
        [T, K] fp32).  Ranks masked in the mask buffer have none of their experts chosen."""
        E, K = self.num_experts, router.num_topk
        _need(x, torch.bfloat16, "x", 2)
        T, H = x.shape
        f32 = w_router.dtype == torch.float32
        _row(w_router, torch.float32 if f32 else torch.bfloat16, (E, H), "w_router")
        if bias is not None:
            _row(bias, torch.float32, (E,), "bias")
        if residual is not None:
            _row(residual, torch.bfloat16, (T, H), "residual")
        if isinstance(w13, (tuple, list)) or isinstance(w2, (tuple, list)):
            (w13, s13), (w2, s2) = _fp8_pair(w13, "w13", 3, True), _fp8_pair(w2, "w2", 3, True)
            inter = w2.shape[2]
            _shape(w13, (E, 2 * inter, H), "w13 codes")
            _shape(w2, (E, H, inter), "w2 codes")
        else:
            s13 = s2 = None
            inter = self._expert_weights(w13, w2, H)
        dev = _here(x, w_router, bias, residual, w13, s13, w2, s2, self._mask)
        ptr, at, d = abi.address, x.device, (T, H, K, E, self.num_ranks, 1)
        y = torch.empty_like(x)
        idx = torch.empty(T, max(K, 0), dtype=torch.int64, device=at)
        weights = torch.empty(T, max(K, 0), dtype=torch.float32, device=at)
        size = _workspace("ep_ll_moe_workspace", d, inter)
        work = torch.empty(size, dtype=torch.uint8, device=at)
        abi.check(abi.lib().ep_ll_moe(
            ctypes.byref(abi.Dims(*d)), inter, router._raw, x.data_ptr(), w_router.data_ptr(), f32, ptr(bias),
            ptr(self._mask), w13.data_ptr(), ptr(s13), w2.data_ptr(), ptr(s2), ptr(residual), idx.data_ptr(),
            weights.data_ptr(), y.data_ptr(), work.data_ptr(), size, abi.raw_stream(dev)), "ep_ll_moe")
        return y, idx, weights

    # ------------------------------------------------------ load balancing
    @staticmethod
    def _lb_args(redundant: torch.Tensor, expert: torch.Tensor, mapping: torch.Tensor):
        """Rows per replica / expert; one replica row per mapping entry, and
        replica rows the size of expert rows."""
        for t, n in ((redundant, "redundant tensor"), (expert, "expert tensor")):
            _need(t, torch.bfloat16, n, t.dim())
            if t.dim() < 1:
                raise ValueError(f"{n} needs a leading [rows] dimension")
        _need(mapping, torch.int64, "redundancy_mapping", 1)
        _same_device(redundant, expert, mapping)
        if redundant.shape[0] != mapping.numel():
            raise ValueError("the redundant tensor needs one row per redundancy_mapping entry")
        if tuple(redundant.shape[1:]) != tuple(expert.shape[1:]):
            raise ValueError("replica rows and expert rows must have the same shape")
        return int(torch.Size(expert.shape[1:]).numel())

    def lb_prefetch_weights(self, redundant_expert_weights: torch.Tensor,
                            expert_weights: torch.Tensor, redundancy_mapping: torch.Tensor,
                            num_sms: int = 0, previous_event=None):
        """redundant_expert_weights[j] = expert_weights[redundancy_mapping[j]]
        (bf16, one row per expert / replica).  Returns None."""
        P = self._lb_args(redundant_expert_weights, expert_weights, redundancy_mapping)
        abi.check(abi.lib().ep_lb_prefetch_weights(
            abi.ptr(expert_weights), abi.ptr(redundant_expert_weights), abi.ptr(redundancy_mapping),
            redundancy_mapping.numel(), expert_weights.shape[0], P, abi.current_stream()),
            "ep_lb_prefetch_weights")
        return None

    def lb_reduce_grads(self, redundant_expert_grads: torch.Tensor, expert_grads: torch.Tensor,
                        redundancy_mapping: torch.Tensor, num_sms: int = 0, previous_event=None):
        """Folds each replica's gradient into its expert (in place, fp32
        accumulation, replicas in ascending order, one rounding).  Returns None."""
        P = self._lb_args(redundant_expert_grads, expert_grads, redundancy_mapping)
        abi.check(abi.lib().ep_lb_reduce_grads(
            abi.ptr(redundant_expert_grads), abi.ptr(expert_grads), abi.ptr(redundancy_mapping),
            redundancy_mapping.numel(), expert_grads.shape[0], P, abi.current_stream()),
            "ep_lb_reduce_grads")
        return None

    def destroy(self) -> None:
        """Return pooled device memory of the current device."""
        abi.check(abi.lib().ep_pool_trim(), "ep_pool_trim")
        self.destroyed = True
