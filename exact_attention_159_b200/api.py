"""Thin Python binding over the C ABI (include/fa.h), same names.

Argument marshalling only: torch tensors (device memory) are turned into
pointers and sizes and passed to libfa.so on the current CUDA stream.  Every
computation runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import check

_BF16 = torch.bfloat16
_E4M3 = torch.float8_e4m3fn


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream_on(device: int, stream):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _stream(stream):
    if stream is None:  # the current stream's handle, without a Stream object around it
        return _stream_on(torch._C._cuda_getDevice(), None)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _shape(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("expected a [B, H, N, d] tensor")
    return tuple(int(x) for x in q.shape)


def _need(t: torch.Tensor, name: str, dtype, shape):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} cuda={t.is_cuda}")
    _on_current_device(t, name)


def _on_current_device(t: torch.Tensor, name: str):
    # the library launches on the current device; a pointer into another GPU's memory must not reach it
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _need_workspace(ws: torch.Tensor, nbytes: int):
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA tensor")
    _on_current_device(ws, "workspace")
    if ws.numel() * ws.element_size() < nbytes:
        raise ValueError(f"workspace: {ws.numel() * ws.element_size()} bytes, {nbytes} needed")


def fa_fwd(q, k, v, scale: float | None = None, causal: bool = False, out=None, lse=None, stream=None):
    """O, LSE = attention(q, k, v); q/k/v bf16 [B, H, N, d] on the GPU."""
    B, H, N, d = _shape(q)
    for t, nm in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, nm, _BF16, (B, H, N, d))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", _BF16, (B, H, N, d))
    _need(lse, "lse", torch.float32, (B, H, N))
    check(_lib.lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, N, d, scale,
                            int(bool(causal)), _stream(stream)), "fa_fwd")
    return out, lse


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(_lib.lib().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, do, lse, scale: float | None = None, causal: bool = False,
           dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ, dK, dV of attention given the forward's O and LSE and the upstream dO."""
    B, H, N, d = _shape(q)
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _need(t, nm, _BF16, (B, H, N, d))
    _need(lse, "lse", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    ws_bytes = fa_bwd_workspace_size(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    _need_workspace(workspace, ws_bytes)
    for t, nm in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        _need(t, nm, _BF16, (B, H, N, d))
    check(_lib.lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                            _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                            B, H, N, d, scale, int(bool(causal)), _stream(stream)), "fa_bwd")
    return dq, dk, dv


def fa_bwd_noalloc(q, k, v, o, do, lse, scale: float | None = None, causal: bool = False,
                   dq=None, dk=None, dv=None, stream=None):
    """fa_bwd on the library's fixed scratch array (no workspace; see include/fa.h for the size limit)."""
    B, H, N, d = _shape(q)
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _need(t, nm, _BF16, (B, H, N, d))
    _need(lse, "lse", torch.float32, (B, H, N))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    check(_lib.lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                                    _ptr(dv), B, H, N, d, scale, int(bool(causal)), _stream(stream)),
          "fa_bwd_noalloc")
    return dq, dk, dv


def _shape_qk(q, k):
    B, Hq, Nq, d = _shape(q)
    Bk, Hkv, Nk, dk = _shape(k)
    if Bk != B or dk != d:
        raise ValueError("q and k must agree in batch and head dimension")
    return B, Hq, Hkv, Nq, Nk, d


def fa_fwd_qk(q, k, v, scale: float | None = None, causal: bool = False, out=None, lse=None, stream=None):
    """O, LSE of grouped-query attention with Nq queries over Nk keys: q bf16 [B, Hq, Nq, d],
    k/v bf16 [B, Hkv, Nk, d] (Hq a multiple of Hkv; causal aligns the last query with the last key)."""
    B, Hq, Hkv, Nq, Nk, d = _shape_qk(q, k)
    _need(q, "q", _BF16, (B, Hq, Nq, d))
    for t, nm in ((k, "k"), (v, "v")):
        _need(t, nm, _BF16, (B, Hkv, Nk, d))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", _BF16, (B, Hq, Nq, d))
    _need(lse, "lse", torch.float32, (B, Hq, Nq))
    check(_lib.lib().fa_fwd_qk(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Nq, Nk, d, scale,
                               int(bool(causal)), _stream(stream)), "fa_fwd_qk")
    return out, lse


def fa_bwd_qk_workspace_size(B: int, Hq: int, Nq: int, d: int) -> int:
    return int(_lib.lib().fa_bwd_qk_workspace_size(B, Hq, Nq, d))


def fa_bwd_qk(q, k, v, o, do, lse, scale: float | None = None, causal: bool = False,
              dq=None, dk=None, dv=None, workspace=None, stream=None):
    """dQ [B, Hq, Nq, d] and dK, dV [B, Hkv, Nk, d] (summed over each key/value head's query heads)."""
    B, Hq, Hkv, Nq, Nk, d = _shape_qk(q, k)
    for t, nm in ((q, "q"), (o, "o"), (do, "do")):
        _need(t, nm, _BF16, (B, Hq, Nq, d))
    for t, nm in ((k, "k"), (v, "v")):
        _need(t, nm, _BF16, (B, Hkv, Nk, d))
    _need(lse, "lse", torch.float32, (B, Hq, Nq))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    ws_bytes = fa_bwd_qk_workspace_size(B, Hq, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    _need_workspace(workspace, ws_bytes)
    _need(dq, "dq", _BF16, (B, Hq, Nq, d))
    for t, nm in ((dk, "dk"), (dv, "dv")):
        _need(t, nm, _BF16, (B, Hkv, Nk, d))
    check(_lib.lib().fa_bwd_qk(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(workspace), workspace.numel() * workspace.element_size(),
                               B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)), _stream(stream)), "fa_bwd_qk")
    return dq, dk, dv


def fa_fwd_accumulate(q, k, v, o_acc, lse_acc, scale: float | None = None, causal: bool = False,
                      first: bool = False, stream=None) -> None:
    """Fold attention of q over one key block (k, v) into fp32 accumulators o_acc [B, Hq, Nq, d],
    lse_acc [B, Hq, Nq] by their log-sum-exp (first: initialise them)."""
    B, Hq, Hkv, Nq, Nk, d = _shape_qk(q, k)
    _need(q, "q", _BF16, (B, Hq, Nq, d))
    for t, nm in ((k, "k"), (v, "v")):
        _need(t, nm, _BF16, (B, Hkv, Nk, d))
    _need(o_acc, "o_acc", torch.float32, (B, Hq, Nq, d))
    _need(lse_acc, "lse_acc", torch.float32, (B, Hq, Nq))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    check(_lib.lib().fa_fwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(o_acc), _ptr(lse_acc), B, Hq, Hkv, Nq, Nk,
                                       d, scale, int(bool(causal)), int(bool(first)), _stream(stream)),
          "fa_fwd_accumulate")


def fa_bwd_prepare(o, do, lse, workspace=None, stream=None):
    """D and LSE*log2(e) of a query block into a (new or given) workspace, dQ accumulator zeroed;
    o, do bf16 [B, Hq, Nq, d], lse fp32 [B, Hq, Nq].  Returns the workspace."""
    B, Hq, Nq, d = _shape(o)
    for t, nm in ((o, "o"), (do, "do")):
        _need(t, nm, _BF16, (B, Hq, Nq, d))
    _need(lse, "lse", torch.float32, (B, Hq, Nq))
    ws_bytes = fa_bwd_qk_workspace_size(B, Hq, Nq, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=o.device)
    _need_workspace(workspace, ws_bytes)
    check(_lib.lib().fa_bwd_prepare(_ptr(o), _ptr(do), _ptr(lse), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), B, Hq, Nq, d, _stream(stream)),
          "fa_bwd_prepare")
    return workspace


def fa_bwd_accumulate(q, k, v, do, workspace, dk_acc, dv_acc, scale: float | None = None, causal: bool = False,
                      first: bool = False, stream=None) -> None:
    """Gradients of one key block: dQ added into the workspace, dK (scaled) and dV stored (first) or
    added into the fp32 accumulators dk_acc, dv_acc [B, Hkv, Nk, d]."""
    B, Hq, Hkv, Nq, Nk, d = _shape_qk(q, k)
    for t, nm in ((q, "q"), (do, "do")):
        _need(t, nm, _BF16, (B, Hq, Nq, d))
    for t, nm in ((k, "k"), (v, "v")):
        _need(t, nm, _BF16, (B, Hkv, Nk, d))
    for t, nm in ((dk_acc, "dk_acc"), (dv_acc, "dv_acc")):
        _need(t, nm, torch.float32, (B, Hkv, Nk, d))
    _need_workspace(workspace, fa_bwd_qk_workspace_size(B, Hq, Nq, d))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    check(_lib.lib().fa_bwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(dk_acc), _ptr(dv_acc),
                                       B, Hq, Hkv, Nq, Nk, d, scale, int(bool(causal)), int(bool(first)),
                                       _stream(stream)), "fa_bwd_accumulate")


def fa_bwd_finish(workspace, B: int, Hq: int, Nq: int, d: int, scale: float | None = None, out=None, stream=None):
    """dQ (bf16 [B, Hq, Nq, d]) from the workspace's accumulator."""
    _need_workspace(workspace, fa_bwd_qk_workspace_size(B, Hq, Nq, d))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    out = torch.empty((B, Hq, Nq, d), dtype=_BF16, device=workspace.device) if out is None else out
    _need(out, "out", _BF16, (B, Hq, Nq, d))
    check(_lib.lib().fa_bwd_finish(_ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), B, Hq,
                                   Nq, d, scale, _stream(stream)), "fa_bwd_finish")
    return out


class _Handle:
    """Tensors as the library is told of them, once: the attributes are not assigned again and the tensors stay in
    their memory (what they hold is read by every call)."""

    def __setattr__(self, name, value):
        if self.__dict__.get(name, value) is not value:  # (`batch.seq_lens += 1` assigns the same tensor again)
            raise AttributeError(f"{name} of a {type(self).__name__} is fixed: make another one")
        super().__setattr__(name, value)

    def _describe(self, struct, tensors):
        self._c, self._ref = struct, ctypes.byref(struct)
        self._places = tuple((t.data_ptr, t.data_ptr()) for t in tensors if t is not None)


class PagedCache(_Handle):
    """A paged key/value cache: k_pages, v_pages [num_pages, Hkv, page_size, d], bf16, or float8_e4m3fn
    with k_scale, v_scale fp32 [num_pages, Hkv] (a held value stands for code * scale; two tensors where
    tokens are appended, one for both is enough to attend).  page_size 16, 32, 64 or 128; d 64 or 128.
    Holds the tensors and describes them to the library; the caller hands out the pages."""

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        if k_pages.dim() != 4:
            raise ValueError("expected [num_pages, Hkv, page_size, d] pages")
        pages, heads, size, d = (int(x) for x in k_pages.shape)
        if k_pages.dtype not in (_BF16, _E4M3):
            raise ValueError(f"k_pages: expected {_BF16} or {_E4M3}, got {k_pages.dtype}")
        if size not in (16, 32, 64, 128) or d not in (64, 128):
            raise ValueError(f"page_size {size}, d {d}: expected page_size 16, 32, 64 or 128 and d 64 or 128")
        fp8 = k_pages.dtype == _E4M3
        for t, nm in ((k_pages, "k_pages"), (v_pages, "v_pages")):
            _need(t, nm, k_pages.dtype, (pages, heads, size, d))
        if (k_scale is None) == fp8 or (v_scale is None) == fp8:
            raise ValueError("k_scale and v_scale belong to float8_e4m3fn pages, both of them")
        if fp8:
            for t, nm in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _need(t, nm, torch.float32, (pages, heads))
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.num_pages, self.heads, self.page_size, self.d = pages, heads, size, d
        self.device = k_pages.device
        self._index = k_pages.get_device()
        self._describe(_lib.CacheStruct(_ptr(k_pages), _ptr(v_pages), _ptr(k_scale), _ptr(v_scale),
                                        _lib.FA_CACHE_E4M3 if fp8 else _lib.FA_CACHE_BF16, pages, heads, size, d),
                       (k_pages, v_pages, k_scale, v_scale))


class PagedBatch(_Handle):
    """B sequences of a paged cache: block_table int32 [B, max_pages], cu_q int32 [B + 1] (the token rows
    of each), seq_lens int32 [B] (tokens in all, the new ones last), max_q (no sequence has more new
    tokens).  The tensors are read when the kernels run: refill them in place from step to step (max_q and the
    tensors themselves are fixed; a batch of another size is another PagedBatch)."""

    def __init__(self, block_table, cu_q, seq_lens, max_q: int):
        if block_table.dim() != 2:
            raise ValueError("block_table: expected [B, max_pages]")
        B, max_pages = (int(x) for x in block_table.shape)
        if not 0 <= int(max_q) < 1 << 31:
            raise ValueError("max_q must not be negative, and fit 32 bits")
        _need(block_table, "block_table", torch.int32, (B, max_pages))
        _need(cu_q, "cu_q", torch.int32, (B + 1,))
        _need(seq_lens, "seq_lens", torch.int32, (B,))
        self.block_table, self.cu_q, self.seq_lens = block_table, cu_q, seq_lens
        self.B, self.max_pages, self.max_q = B, max_pages, int(max_q)
        self.device = block_table.device
        self._index = block_table.get_device()
        self._describe(_lib.BatchStruct(block_table.data_ptr(), cu_q.data_ptr(), seq_lens.data_ptr(), B, max_pages,
                                        self.max_q), (block_table, cu_q, seq_lens))


def _need_rows(t: torch.Tensor, name: str, heads: int, d: int, rows: int, device: int) -> int:
    """Checks token-major rows [rows, heads, d] with each row contiguous; returns the elements between rows."""
    if t.dtype != _BF16 or t.shape != (rows, heads, d) or t.get_device() != device:
        raise ValueError(f"{name}: expected {_BF16} {(rows, heads, d)} on the current device cuda:{device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    row, head, col = t.stride()
    if (col != 1 or head != d) and rows > 0 and heads > 0 and (col != 1 or heads > 1):
        raise ValueError(f"{name}: expected each token's {heads} x {d} elements contiguous, got strides {t.stride()}")
    return row if rows > 1 else heads * d


def _rows_of(t: torch.Tensor, name: str):
    if t.dim() != 3:
        raise ValueError(f"{name}: expected a [T, heads, d] tensor")
    return t.shape


def _on_stream(stream):
    """The context in which to allocate for a call on `stream`."""
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream)
                             else torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream))))


def _empty(like, shape, dtype, stream):
    """An uninitialised tensor on like's device for a call on `stream` (None: the current one), whose memory that
    stream reuses."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on_stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _same_device(cache: PagedCache, batch: PagedBatch) -> int:
    """The current device, which the cache and the batch have to be on, in the memory that they were made with."""
    cur = torch._C._cuda_getDevice()
    if cache._index != cur or batch._index != cur:
        raise ValueError(f"cache on {cache.device}, batch on {batch.device}, but the current device is cuda:{cur}")
    for handle in (cache, batch):
        for at, was in handle._places:
            if at() != was:
                raise ValueError(f"a tensor of the {type(handle).__name__} has left its memory (resized, or given other "
                                 "storage): make another one")
    return cur


def fa_cache_append(k, v, cache: PagedCache, batch: PagedBatch, cos=None, sin=None, interleaved: bool = False,
                    q=None, q_out=None, stream=None):
    """Append the new tokens' k, v (bf16 [T, Hkv, d]; rows may be strided, as slices of a fused projection)
    to the cache.  cos, sin fp32 [positions, rot / 2] rotate the keys, and the queries q (bf16 [T, Hq, d])
    into q_out (new, given, or q itself), by the tokens' positions: pairs (i, i + rot/2), or (2i, 2i + 1)
    when interleaved.  Returns the rotated queries (None without q)."""
    T, heads, d = _rows_of(k, "k")[0], cache.heads, cache.d
    cur = _same_device(cache, batch)
    ldk = _need_rows(k, "k", heads, d, T, cur)
    ldv = _need_rows(v, "v", heads, d, T, cur)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin belong together")
    rot = n_pos = ldq = ldqo = Hq = 0
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos: expected [positions, rot / 2]")
        n_pos, half = cos.shape
        rot = 2 * half
        if rot == 0 or rot > d or rot % 16:
            raise ValueError(f"cos, sin turn {rot} of {d} columns: expected a multiple of 16, at most {d}")
        for t, nm in ((cos, "cos"), (sin, "sin")):
            if t.dtype != torch.float32 or t.shape != cos.shape or not t.is_contiguous() or t.get_device() != cur:
                _need(t, nm, torch.float32, (n_pos, half))
    if q is not None:
        if rot == 0:
            raise ValueError("q is given to be rotated: it needs cos and sin")
        Hq = _rows_of(q, "q")[1]
        ldq = _need_rows(q, "q", Hq, d, T, cur)
        if heads == 0 or Hq % heads:
            raise ValueError(f"q: {Hq} heads over {heads} key/value heads")
        if q_out is None:
            q_out = _empty(q, (T, Hq, d), _BF16, stream)
            ldqo = Hq * d
        else:
            ldqo = _need_rows(q_out, "q_out", Hq, d, T, cur)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    check(_lib.lib().fa_cache_append(cache._ref, batch._ref, T, k.data_ptr(), ldk, v.data_ptr(), ldv, _ptr(q), ldq,
                                     _ptr(q_out), ldqo, Hq, _ptr(cos), _ptr(sin), rot, 1 if interleaved else 0,
                                     n_pos, _stream_on(cur, stream)), "fa_cache_append")
    return q_out


def fa_fwd_paged_workspace_size(cache: PagedCache, batch: PagedBatch, T: int, Hq: int) -> int:
    return int(_lib.lib().fa_fwd_paged_workspace_size(cache._ref, batch._ref, T, Hq))


def fa_fwd_paged(q, cache: PagedCache, batch: PagedBatch, scale: float | None = None, causal: bool = True,
                 out=None, lse=None, workspace=None, stream=None):
    """O [T, Hq, d], LSE [T, Hq] of the new tokens' queries q (bf16 [T, Hq, d]; rows may be strided) over
    their sequences in the cache: single tokens, a few, prompt chunks, or a mixture.  causal: token i of
    n new ones sees its sequence's keys but the last n - 1 - i.  A row that sees no key gets O = 0,
    LSE = -inf; rows behind the batch's last are left as they were."""
    T, Hq, _ = _rows_of(q, "q")
    cur, d = _same_device(cache, batch), cache.d
    ldq = _need_rows(q, "q", Hq, d, T, cur)
    if cache.heads == 0 or Hq % cache.heads:
        raise ValueError(f"q: {Hq} heads over {cache.heads} key/value heads")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    lib = _lib.lib()
    ws_bytes = lib.fa_fwd_paged_workspace_size(cache._ref, batch._ref, T, Hq)
    if workspace is None:
        workspace = _empty(q, (max(ws_bytes, 16),), torch.uint8, stream)
        ws_bytes = max(ws_bytes, 16)
    else:
        _need_workspace(workspace, ws_bytes)
        ws_bytes = workspace.numel() * workspace.element_size()
    if out is None:
        out = _empty(q, (T, Hq, d), _BF16, stream)
    else:
        _need(out, "out", _BF16, (T, Hq, d))
    if lse is None:
        lse = _empty(q, (T, Hq), torch.float32, stream)
    else:
        _need(lse, "lse", torch.float32, (T, Hq))
    check(lib.fa_fwd_paged(q.data_ptr(), ldq, cache._ref, batch._ref, T, out.data_ptr(), lse.data_ptr(),
                           workspace.data_ptr(), ws_bytes, Hq, scale, 1 if causal else 0,
                           _stream_on(cur, stream)), "fa_fwd_paged")
    return out, lse


def fa_lse_merge(o_part, lse_part, o_acc, lse_acc, first: bool = False, stream=None) -> None:
    """Fold a partial (O bf16 [..., d], LSE fp32 [...]) over one key set into an fp32 accumulator."""
    d = int(o_part.shape[-1])
    rows = o_part.numel() // d
    _need(o_part, "o_part", _BF16, tuple(o_part.shape))
    _need(o_acc, "o_acc", torch.float32, tuple(o_part.shape))
    _need(lse_part, "lse_part", torch.float32, tuple(o_part.shape[:-1]))
    _need(lse_acc, "lse_acc", torch.float32, tuple(o_part.shape[:-1]))
    check(_lib.lib().fa_lse_merge(_ptr(o_part), _ptr(lse_part), _ptr(o_acc), _ptr(lse_acc), rows, d,
                                  int(bool(first)), _stream(stream)), "fa_lse_merge")


def fa_accumulate_bf16(acc, x, first: bool = False, stream=None) -> None:
    """acc (fp32) = (0 if first else acc) + x (bf16), elementwise."""
    _need(acc, "acc", torch.float32, tuple(x.shape))
    _need(x, "x", _BF16, tuple(x.shape))
    check(_lib.lib().fa_accumulate_bf16(_ptr(acc), _ptr(x), x.numel(), int(bool(first)), _stream(stream)),
          "fa_accumulate_bf16")


def fa_accumulate_f32(acc, x, stream=None) -> None:
    """acc (fp32) += x (fp32), elementwise."""
    _need(acc, "acc", torch.float32, tuple(x.shape))
    _need(x, "x", torch.float32, tuple(x.shape))
    check(_lib.lib().fa_accumulate_f32(_ptr(acc), _ptr(x), x.numel(), _stream(stream)), "fa_accumulate_f32")


def fa_convert_f32_bf16(x, out=None, stream=None):
    """bf16 copy of an fp32 tensor (round to nearest even)."""
    out = torch.empty(x.shape, dtype=_BF16, device=x.device) if out is None else out
    _need(x, "x", torch.float32, tuple(x.shape))
    _need(out, "out", _BF16, tuple(x.shape))
    check(_lib.lib().fa_convert_f32_bf16(_ptr(x), _ptr(out), x.numel(), _stream(stream)), "fa_convert_f32_bf16")
    return out


def fa_last_device_status(stream=None) -> tuple[int, int]:
    """(status, detail) after synchronising the stream; see include/fa.h."""
    detail = ctypes.c_int(0)
    rc = _lib.lib().fa_last_device_status(_stream(stream), ctypes.byref(detail))
    return int(rc), int(detail.value)


def fa_set_softmax_options(tau: float = 8.0, poly: int = -1) -> None:
    """Rescale threshold and cubic-exp2 share (pairs per 16; -1 = per-head-dim default)."""
    check(_lib.lib().fa_set_softmax_options(float(tau), int(poly)), "fa_set_softmax_options")


def fa_set_forward_variant(cluster_pair: int = 0) -> None:
    check(_lib.lib().fa_set_forward_variant(int(cluster_pair)), "fa_set_forward_variant")


def fa_set_backward_variant(cluster_pair: int = 0) -> None:
    check(_lib.lib().fa_set_backward_variant(int(cluster_pair)), "fa_set_backward_variant")


def fa_exp2_eval(x: torch.Tensor, mode: int = 0, stream=None) -> torch.Tensor:
    """2^x on the device: mode 0 = cubic software exp2, 1 = SFU ex2."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA float32 tensor")
    _on_current_device(x, "x")
    y = torch.empty_like(x)
    check(_lib.lib().fa_exp2_eval(_ptr(x), _ptr(y), x.numel(), int(mode), _stream(stream)), "fa_exp2_eval")
    return y


def fa_profile_next(which: int, start, stop) -> None:
    """Have the next fa_fwd (0) / fa_bwd (1) record torch.cuda.Events around its main kernel."""
    h = lambda e: None if e is None else ctypes.c_void_p(e.cuda_event)
    check(_lib.lib().fa_profile_next(int(which), h(start), h(stop)), "fa_profile_next")


def fa_sm_clock_probe(out: torch.Tensor | None = None, stream=None):
    """Effective SM clock, measured on the device by a ~20 us probe kernel queued on `stream`
    behind whatever work is already queued there.  With `out` (a CUDA int64 tensor of 2 elements)
    it only queues the probe, which writes [cycles, nanoseconds] there (no synchronisation, so
    the GPU keeps the clock of the surrounding work); without, it synchronises and returns MHz."""
    own = out is None
    if own:
        out = torch.zeros(2, dtype=torch.int64, device="cuda")
    elif out.dtype != torch.int64 or not out.is_cuda or out.numel() != 2 or not out.is_contiguous():
        raise ValueError("out must be a contiguous CUDA int64 tensor of 2 elements")
    else:
        _on_current_device(out, "out")
    check(_lib.lib().fa_sm_clock_probe(_ptr(out), _stream(stream)), "fa_sm_clock_probe")
    if not own:
        return None
    torch.cuda.synchronize()
    cycles, ns = out.tolist()
    return 1000.0 * cycles / ns if ns > 0 else 0.0


def fa_strerror(code: int) -> str:
    return _lib.lib().fa_strerror(int(code)).decode()


def fa_version() -> int:
    return int(_lib.lib().fa_version())
