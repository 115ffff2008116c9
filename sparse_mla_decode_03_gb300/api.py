"""Thin Python binding of libsmla.so: argument marshalling only.

Every function forwards device pointers of torch tensors and the current CUDA
stream to the C entry point of the same name (include/smla.h) and raises
``SmlaError`` on a non-zero status.  All computation happens in the library's
CUDA kernels; there is no Python or CPU fallback.

With ``stream=`` another stream than the current one, what a call allocates is that stream's
memory, and arguments may be dropped as soon as the call returns.  That the inputs are ready on
that stream, and that results are read after it, stays with the caller."""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import _lib

DEFAULT_SCALE = 1.0 / math.sqrt(512)
NOPE = 448
QK = 512
ROW_BYTES = 584
ROW4_BYTES = 368             # rows of 4-bit values, at most MAX_ROW4_STRIDE apart
MAX_ROW4_STRIDE = 512
MAX_KV_TOKENS = 1 << 30      # the largest bound that smla_chunk_attention takes


class SmlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib.load()
        super().__init__(f"{where}: {lib.smla_status_string(status).decode()} ({status})")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise SmlaError(status, where)


def _stream(stream: Optional[torch.cuda.Stream]) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


_SAME = contextlib.nullcontext()


def _side(stream: Optional[torch.cuda.Stream], device: torch.device) -> Optional[torch.cuda.Stream]:
    """`stream`, if it is another than the device's current one."""
    if stream is None or stream.cuda_stream == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    return stream


def _empty(side: Optional[torch.cuda.Stream], shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    """What a call that runs on `side` allocates is that stream's memory: it is not handed out, before
    or after the call, to work of the current stream that does not wait for it."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        return torch.empty(shape, dtype=dtype, device=device)


def _keep(side: torch.cuda.Stream, *tensors: Optional[torch.Tensor]) -> None:
    """A call on `side` uses these tensors, and the caller the results on the current stream: the
    memory of one that is dropped is not handed out again before both have come past this point."""
    for t in tensors:
        if t is not None:
            t.record_stream(side)
            t.record_stream(torch.cuda.current_stream(t.device))


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def make_params(batch: int, num_heads: int, topk: int, num_rows: int, kv_row_stride: int,
                softmax_scale: float = DEFAULT_SCALE) -> _lib.SmlaParams:
    return _lib.SmlaParams(batch, num_heads, topk, 0, num_rows, kv_row_stride, softmax_scale)


def _check_rows(name: str, rows: torch.Tensor) -> int:
    """Checks a cache of rows, of 8- or 4-bit values by the bytes between them, which it returns (a
    single row has no neighbour: its width tells).  Rows that do not hold what their distance says, or reach
    into the next ones, would be read past their ends or as the other kind."""
    shape, strides = rows.shape, rows.stride()
    if len(shape) != 2 or rows.dtype != torch.uint8 or strides[1] != 1:
        raise ValueError(f"{name} must be uint8 [num_rows, stride>=584] with unit column stride")
    num, width = shape
    stride = strides[0] if num > 1 else ROW_BYTES if width >= ROW_BYTES else ROW4_BYTES
    if width < ROW4_BYTES or (width < ROW_BYTES if stride > MAX_ROW4_STRIDE else num > 1 and width > stride):
        raise ValueError(f"{name} rows must hold 584 bytes, or 368 at most 512 bytes apart (4-bit values)")
    return stride


def _params_from(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                 softmax_scale: float) -> _lib.SmlaParams:
    if q.dim() != 3 or q.shape[2] != QK or q.dtype != torch.bfloat16:
        raise ValueError("q must be bf16 [B, H, 512]")
    stride = _check_rows("kv_cache", kv_cache)
    if indices.dim() != 2 or indices.dtype != torch.int32 or indices.shape[0] != q.shape[0]:
        raise ValueError("indices must be int32 [B, topk]")
    for name, t in (("q", q), ("indices", indices)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if not (q.is_cuda and kv_cache.is_cuda and indices.is_cuda):
        raise ValueError("q, kv_cache and indices must be CUDA tensors")
    B, H, _ = q.shape
    return make_params(B, H, indices.shape[1], kv_cache.shape[0], stride, softmax_scale)


def smla_default_num_splits(params: _lib.SmlaParams) -> int:
    lib = _lib.load()
    n = ctypes.c_int32(0)
    _check(lib.smla_default_num_splits(ctypes.byref(params), ctypes.byref(n)),
           "smla_default_num_splits")
    return n.value


def smla_decode_plan(params: _lib.SmlaParams, num_splits: int = 0) -> Tuple[int, bool]:
    """(resolved split count, True if sparse_mla_decode merges the splits on chip)."""
    lib = _lib.load()
    S, fused = ctypes.c_int32(0), ctypes.c_int32(0)
    _check(lib.smla_decode_plan(ctypes.byref(params), num_splits, ctypes.byref(S),
                                ctypes.byref(fused)), "smla_decode_plan")
    return S.value, bool(fused.value)


def smla_workspace_size(params: _lib.SmlaParams, num_splits: int = 0) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    _check(lib.smla_workspace_size(ctypes.byref(params), num_splits, ctypes.byref(n)),
           "smla_workspace_size")
    return n.value


def sparse_mla_decode(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                      softmax_scale: float = DEFAULT_SCALE, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, num_splits: int = 0,
                      workspace: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None
                      ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Whole decode step.  Returns (out bf16 [B, H, 448], lse fp32 [B, H]).  kv_cache: rows of 584
    bytes, or of 368 (4-bit values; num_splits 0)."""
    p = _params_from(q, kv_cache, indices, softmax_scale)
    B, H = p.batch, p.num_heads
    need = smla_workspace_size(p, num_splits)
    side = _side(stream, q.device)
    if out is None:
        out = _empty(side, (B, H, NOPE), torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(side, (B, H), torch.float32, q.device)
    if workspace is None:
        workspace = _empty(side, need, torch.uint8, q.device)
    lib = _lib.load()
    st = lib.sparse_mla_decode(_ptr(q), _ptr(kv_cache), _ptr(indices), _ptr(out), _ptr(lse),
                               ctypes.byref(p), num_splits, _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream))
    if side is not None:
        _keep(side, q, kv_cache, indices, out, lse, workspace)
    _check(st, "sparse_mla_decode")
    return out, lse


def sparse_mla_decode_split(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                            num_splits: int, softmax_scale: float = DEFAULT_SCALE,
                            o_part: Optional[torch.Tensor] = None,
                            lse_part: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Split kernel alone.  Returns (o_part fp32 [B, H, S, 448], lse_part fp32 [B, H, S])."""
    p = _params_from(q, kv_cache, indices, softmax_scale)
    B, H, S = p.batch, p.num_heads, num_splits
    side = _side(stream, q.device)
    if o_part is None:
        o_part = _empty(side, (B, H, S, NOPE), torch.float32, q.device)
    if lse_part is None:
        lse_part = _empty(side, (B, H, S), torch.float32, q.device)
    lib = _lib.load()
    st = lib.sparse_mla_decode_split(_ptr(q), _ptr(kv_cache), _ptr(indices), ctypes.byref(p), S,
                                     _ptr(o_part), _ptr(lse_part), _stream(stream))
    if side is not None:
        _keep(side, q, kv_cache, indices, o_part, lse_part)
    _check(st, "sparse_mla_decode_split")
    return o_part, lse_part


def sparse_mla_combine(o_part: torch.Tensor, lse_part: torch.Tensor,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Combine kernel alone.  Returns (out bf16 [B, H, 448], lse fp32 [B, H])."""
    if o_part.dim() != 4 or o_part.shape[3] != NOPE or o_part.dtype != torch.float32:
        raise ValueError("o_part must be fp32 [B, H, S, 448]")
    if lse_part.shape != o_part.shape[:3] or lse_part.dtype != torch.float32:
        raise ValueError("lse_part must be fp32 [B, H, S]")
    if not (o_part.is_contiguous() and lse_part.is_contiguous()):
        raise ValueError("partials must be contiguous")
    B, H, S, _ = o_part.shape
    side = _side(stream, o_part.device)
    if out is None:
        out = _empty(side, (B, H, NOPE), torch.bfloat16, o_part.device)
    if lse is None:
        lse = _empty(side, (B, H), torch.float32, o_part.device)
    lib = _lib.load()
    st = lib.sparse_mla_combine(_ptr(o_part), _ptr(lse_part), B, H, S, _ptr(out), _ptr(lse),
                                _stream(stream))
    if side is not None:
        _keep(side, o_part, lse_part, out, lse)
    _check(st, "sparse_mla_combine")
    return out, lse


def sparse_mla_decode_noalloc(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                              softmax_scale: float = DEFAULT_SCALE,
                              out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None, num_splits: int = 0,
                              stream: Optional[torch.cuda.Stream] = None
                              ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Whole decode step with the split partials in the library's built-in scratch
    (no workspace argument; the C function allocates nothing).  Pass `out` and `lse`
    to keep the call itself free of allocations."""
    p = _params_from(q, kv_cache, indices, softmax_scale)
    side = _side(stream, q.device)
    if out is None:
        out = _empty(side, (p.batch, p.num_heads, NOPE), torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(side, (p.batch, p.num_heads), torch.float32, q.device)
    st = _lib.load().sparse_mla_decode_noalloc(_ptr(q), _ptr(kv_cache), _ptr(indices), _ptr(out),
                                               _ptr(lse), ctypes.byref(p), num_splits,
                                               _stream(stream))
    if side is not None:
        _keep(side, q, kv_cache, indices, out, lse)
    _check(st, "sparse_mla_decode_noalloc")
    return out, lse


def smla_paged_workspace_size(params: _lib.SmlaParams, num_splits: int = 0) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    _check(lib.smla_paged_workspace_size(ctypes.byref(params), num_splits, ctypes.byref(n)),
           "smla_paged_workspace_size")
    return n.value


def sparse_mla_decode_paged(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                            page_size: int, indices: torch.Tensor,
                            softmax_scale: float = DEFAULT_SCALE,
                            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            num_splits: int = 0, workspace: Optional[torch.Tensor] = None,
                            stream: Optional[torch.cuda.Stream] = None
                            ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Decode step over a paged cache: `indices` are logical positions in each query's
    sequence, `block_table` int32 [B, max_pages] maps its pages into `kv_pages`."""
    p = _params_from(q, kv_pages, indices, softmax_scale)
    if (block_table.dim() != 2 or block_table.dtype != torch.int32
            or block_table.shape[0] != p.batch or not block_table.is_contiguous()
            or not block_table.is_cuda):
        raise ValueError("block_table must be a contiguous CUDA int32 [B, max_pages] tensor")
    need = smla_paged_workspace_size(p, num_splits)
    side = _side(stream, q.device)
    if out is None:
        out = _empty(side, (p.batch, p.num_heads, NOPE), torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(side, (p.batch, p.num_heads), torch.float32, q.device)
    if workspace is None:
        workspace = _empty(side, need, torch.uint8, q.device)
    st = _lib.load().sparse_mla_decode_paged(
        _ptr(q), _ptr(kv_pages), _ptr(block_table), block_table.shape[1], page_size,
        _ptr(indices), _ptr(out), _ptr(lse), ctypes.byref(p), num_splits, _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    if side is not None:
        _keep(side, q, kv_pages, block_table, indices, out, lse, workspace)
    _check(st, "sparse_mla_decode_paged")
    return out, lse


def sparse_mla_decode_simt(q: torch.Tensor, kv_cache: torch.Tensor, indices: torch.Tensor,
                           softmax_scale: float = DEFAULT_SCALE,
                           out: Optional[torch.Tensor] = None,
                           lse: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None
                           ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The per-head fp32 SIMT form of the decode step (a reference point for the
    tensor-core path).  Returns (out bf16 [B, H, 448], lse fp32 [B, H])."""
    p = _params_from(q, kv_cache, indices, softmax_scale)
    side = _side(stream, q.device)
    if out is None:
        out = _empty(side, (p.batch, p.num_heads, NOPE), torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(side, (p.batch, p.num_heads), torch.float32, q.device)
    st = _lib.load().sparse_mla_decode_simt(_ptr(q), _ptr(kv_cache), _ptr(indices), _ptr(out),
                                            _ptr(lse), ctypes.byref(p), _stream(stream))
    if side is not None:
        _keep(side, q, kv_cache, indices, out, lse)
    _check(st, "sparse_mla_decode_simt")
    return out, lse


# ---------------------------------------------------------------------------
# The paged cache
# ---------------------------------------------------------------------------
def _ints(name: str, t: torch.Tensor, dims: int, device: torch.device) -> None:
    if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dims} dimension(s) on {device}")


def _pool(kv_pages: torch.Tensor, page_size: int) -> int:
    """Checks a pool of pages; the bytes between its rows."""
    stride = _check_rows("kv_pages", kv_pages)
    if not kv_pages.is_cuda:
        raise ValueError("kv_pages must be a CUDA tensor")
    if page_size < 1 or kv_pages.shape[0] < page_size:
        raise ValueError("kv_pages must hold a page of page_size >= 1 rows")
    return stride


def _stream_on(stream: Optional[torch.cuda.Stream], device: torch.device) -> int:
    """The handle of `stream`, or of the device's current stream (its raw handle: a Stream
    object costs more than a small launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return stream.cuda_stream


def _adr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _on(device: torch.device):
    """The device as the current one for a call (no switch where it is already)."""
    return _SAME if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def make_cache_params(num_pages: int, page_size: int, num_seqs: int, max_pages: int,
                      kv_row_stride: int = ROW_BYTES) -> _lib.SmlaCacheParams:
    return _lib.SmlaCacheParams(num_pages, page_size, num_seqs, max_pages, kv_row_stride)


def smla_cache_workspace_size(params: _lib.SmlaCacheParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load().smla_cache_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "smla_cache_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _cache_bytes(num_pages: int, num_seqs: int) -> int:
    """What smla_cache_workspace_size says: a matter of these two sizes alone."""
    return smla_cache_workspace_size(make_cache_params(num_pages, 1, num_seqs, 1))


def _cache_workspace(p: _lib.SmlaCacheParams, workspace: Optional[torch.Tensor], device: torch.device,
                     side: Optional[torch.cuda.Stream]) -> torch.Tensor:
    if workspace is None:
        return _empty(side, _cache_bytes(p.num_pages, p.num_seqs), torch.uint8, device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace


def _bytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _token_rows(name: str, kv: torch.Tensor, device: torch.device) -> int:
    """Checks bf16 [T, 512]; elements between its rows."""
    if kv.dim() != 2 or kv.shape[1] != QK or kv.dtype != torch.bfloat16 or kv.stride(1) != 1 or kv.device != device:
        raise ValueError(f"{name} must be bf16 [T, 512] with unit column stride on {device}")
    return kv.stride(0) if kv.shape[0] > 1 else QK


def _rows_of_heads(name: str, t: torch.Tensor, tokens: int, width: int, device: torch.device) -> Tuple[int, ...]:
    """Checks bf16 [tokens, H, width]; its strides."""
    stride = t.stride()
    if (len(stride) != 3 or stride[2] != 1 or t.shape[2] != width or t.shape[0] != tokens or t.dtype != torch.bfloat16
            or t.device != device):
        raise ValueError(f"{name} must be bf16 [{tokens}, H, {width}] with unit column stride on {device}")
    return stride


def _token_places(kv_pages: torch.Tensor, page_size: int, block_table: torch.Tensor, cu_q: torch.Tensor,
                  kv_lens: torch.Tensor) -> _lib.SmlaCacheParams:
    row_stride = _pool(kv_pages, page_size)
    dev = kv_pages.device
    _ints("block_table", block_table, 2, dev)
    _ints("cu_q", cu_q, 1, dev)
    _ints("kv_lens", kv_lens, 1, dev)
    B = block_table.shape[0]
    if cu_q.shape[0] != B + 1 or kv_lens.shape[0] != B:
        raise ValueError("cu_q must be [B + 1] and kv_lens [B] for a block_table of B rows")
    return make_cache_params(kv_pages.shape[0] // page_size, page_size, B, block_table.shape[1],
                             row_stride)


def smla_cache_append(kv: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                      page_size: int, cu_q: torch.Tensor, kv_lens: torch.Tensor,
                      stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantises new tokens and writes their rows (8- or 4-bit, as kv_pages has them).  kv bf16 [T, 512];
    sequence b's are kv[cu_q[b]:cu_q[b + 1]], the last ones of its kv_lens[b] tokens."""
    p = _token_places(kv_pages, page_size, block_table, cu_q, kv_lens)
    dev = kv_pages.device
    stride = _token_rows("kv", kv, dev)
    side = _side(stream, dev)
    with _on(dev):
        st = _lib.load().smla_cache_append(_adr(kv), stride, kv.shape[0], _adr(kv_pages), _adr(block_table),
                                           _adr(cu_q), _adr(kv_lens), ctypes.byref(p),
                                           _stream_on(stream, dev))
    if side is not None:
        _keep(side, kv, kv_pages, block_table, cu_q, kv_lens)
    _check(st, "smla_cache_append")


def smla_cache_append_rotary(kv: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                             page_size: int, cu_q: torch.Tensor, kv_lens: torch.Tensor,
                             rotary: torch.Tensor, interleaved: bool = True,
                             q_rope: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                             stream: Optional[torch.cuda.Stream] = None) -> None:
    """smla_cache_append with the position rotation on the way: the rope columns of kv by the token's
    row of rotary fp32 [positions, 64] (cosines of the 32 pairs, then sines), pairs (2 i, 2 i + 1) if
    interleaved, else (i, i + 32).  With q_rope bf16 [T, H, 64] the queries' rope columns are rotated
    too, into q[:, :, 448:] of q bf16 [T, H, 512] (which may be q_rope itself)."""
    p = _token_places(kv_pages, page_size, block_table, cu_q, kv_lens)
    dev = kv_pages.device
    stride = _token_rows("kv", kv, dev)
    if (rotary.dim() != 2 or rotary.shape[1] != QK - NOPE or rotary.dtype != torch.float32 or rotary.device != dev
            or not rotary.is_contiguous()):
        raise ValueError(f"rotary must be contiguous fp32 [positions, 64] on {dev}")
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q come together")
    T, H, q0, q1, r0, r1 = kv.shape[0], 0, 0, 0, 0, 0
    if q is not None:
        q0, q1, _ = _rows_of_heads("q", q, T, QK, dev)
        r0, r1, _ = _rows_of_heads("q_rope", q_rope, T, QK - NOPE, dev)
        H = q.shape[1]
        if q_rope.shape[1] != H:
            raise ValueError("q_rope and q must have as many heads")
        if (T > 1 and q0 < QK) or (H > 1 and q1 < QK) or (
                T > 1 and H > 1 and q0 < (H - 1) * q1 + QK and q1 < (T - 1) * q0 + QK):
            raise ValueError("the rows of q must not overlap")
        if T <= 1:
            q0 = r0 = 0
        if H <= 1:
            q1 = r1 = 0
    r = _lib.SmlaRotaryParams(_adr(rotary), _adr(q_rope), _adr(q), rotary.shape[0], r0, r1, q0, q1, H,
                              0 if interleaved else 1, 0)
    side = _side(stream, dev)
    with _on(dev):
        st = _lib.load().smla_cache_append_rotary(_adr(kv), stride, T, _adr(kv_pages), _adr(block_table), _adr(cu_q),
                                                  _adr(kv_lens), ctypes.byref(p), ctypes.byref(r),
                                                  _stream_on(stream, dev))
    if side is not None:
        _keep(side, kv, kv_pages, block_table, cu_q, kv_lens, rotary, q_rope, q)
    _check(st, "smla_cache_append_rotary")


def smla_cache_read(kv_pages: torch.Tensor, block_table: torch.Tensor, page_size: int, cu_q: torch.Tensor,
                    kv_lens: torch.Tensor, total_tokens: int, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values of the rows that smla_cache_append writes for the same cu_q and kv_lens: bf16
    [total_tokens, 512].  Entries without a row are left as they were (in a new out: undefined)."""
    p = _token_places(kv_pages, page_size, block_table, cu_q, kv_lens)
    dev = kv_pages.device
    side = _side(stream, dev)
    if out is None:
        out = _empty(side, (total_tokens, QK), torch.bfloat16, dev)
    stride = _token_rows("out", out, dev)
    if out.shape[0] != total_tokens:
        raise ValueError(f"out must be bf16 [{total_tokens}, 512]")
    with _on(dev):
        st = _lib.load().smla_cache_read(_adr(kv_pages), _adr(block_table), _adr(cu_q), _adr(kv_lens), _adr(out), stride,
                                         total_tokens, ctypes.byref(p), _stream_on(stream, dev))
    if side is not None:
        _keep(side, kv_pages, block_table, cu_q, kv_lens, out)
    _check(st, "smla_cache_read")
    return out


def smla_cache_reserve(page_size: int, ref_count: torch.Tensor, block_table: torch.Tensor,
                       target_lens: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> None:
    """Maps free pages until every sequence r has room for target_lens[r] tokens."""
    dev = ref_count.device
    _ints("ref_count", ref_count, 1, dev)
    _ints("block_table", block_table, 2, dev)
    _ints("target_lens", target_lens, 1, dev)
    if not ref_count.is_cuda or target_lens.shape[0] != block_table.shape[0]:
        raise ValueError("target_lens must be [B] for a block_table of B rows, on a CUDA device")
    p = make_cache_params(ref_count.shape[0], page_size, block_table.shape[0], block_table.shape[1])
    side = _side(stream, dev)
    ws = _cache_workspace(p, workspace, dev, side)
    with _on(dev):
        st = _lib.load().smla_cache_reserve(_adr(ref_count), _adr(block_table), _adr(target_lens),
                                            ctypes.byref(p), _adr(ws), _bytes(ws), _stream_on(stream, dev))
    if side is not None:
        _keep(side, ref_count, block_table, target_lens, ws)
    _check(st, "smla_cache_reserve")


def _page_state(kv_pages: torch.Tensor, page_size: int, ref_count: torch.Tensor,
                block_table: torch.Tensor) -> _lib.SmlaCacheParams:
    row_stride = _pool(kv_pages, page_size)
    dev = kv_pages.device
    _ints("ref_count", ref_count, 1, dev)
    _ints("block_table", block_table, 2, dev)
    if ref_count.shape[0] * page_size > kv_pages.shape[0]:
        raise ValueError("ref_count has more pages than kv_pages")
    return make_cache_params(ref_count.shape[0], page_size, block_table.shape[0], block_table.shape[1],
                             row_stride)


def smla_cache_fork(kv_pages: torch.Tensor, page_size: int, ref_count: torch.Tensor,
                    block_table: torch.Tensor, kv_lens: torch.Tensor, parents: torch.Tensor,
                    children: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> None:
    """Makes row children[i] a copy of row parents[i]: full pages shared, a partly filled
    last page copied into a free one."""
    p = _page_state(kv_pages, page_size, ref_count, block_table)
    dev = kv_pages.device
    _ints("kv_lens", kv_lens, 1, dev)
    _ints("parents", parents, 1, dev)
    _ints("children", children, 1, dev)
    if kv_lens.shape[0] != block_table.shape[0] or parents.shape != children.shape:
        raise ValueError("kv_lens must be [B], and parents and children equally long")
    side = _side(stream, dev)
    ws = _cache_workspace(p, workspace, dev, side)
    with _on(dev):
        st = _lib.load().smla_cache_fork(_adr(kv_pages), _adr(ref_count), _adr(block_table), _adr(kv_lens),
                                         _adr(parents), _adr(children), parents.shape[0], ctypes.byref(p),
                                         _adr(ws), _bytes(ws), _stream_on(stream, dev))
    if side is not None:
        _keep(side, kv_pages, ref_count, block_table, kv_lens, parents, children, ws)
    _check(st, "smla_cache_fork")


def smla_cache_free(ref_count: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
                    rows: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Empties the listed rows of the table and gives their pages back."""
    dev = ref_count.device
    _ints("ref_count", ref_count, 1, dev)
    _ints("block_table", block_table, 2, dev)
    _ints("kv_lens", kv_lens, 1, dev)
    _ints("rows", rows, 1, dev)
    if not ref_count.is_cuda or kv_lens.shape[0] != block_table.shape[0]:
        raise ValueError("kv_lens must be [B] for a block_table of B rows, on a CUDA device")
    p = make_cache_params(ref_count.shape[0], 1, block_table.shape[0], block_table.shape[1])
    side = _side(stream, dev)
    with _on(dev):
        st = _lib.load().smla_cache_free(_adr(ref_count), _adr(block_table), _adr(kv_lens), _adr(rows),
                                         rows.shape[0], ctypes.byref(p), _stream_on(stream, dev))
    if side is not None:
        _keep(side, ref_count, block_table, kv_lens, rows)
    _check(st, "smla_cache_free")


def smla_cache_compact(kv_pages: torch.Tensor, page_size: int, ref_count: torch.Tensor,
                       block_table: torch.Tensor, ref_count_out: Optional[torch.Tensor] = None,
                       block_table_out: Optional[torch.Tensor] = None,
                       info: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Moves the pages in use to the front of the pool; counts and table follow, in place
    unless other outputs are given.  Returns info: int32 [pages in use, pages moved]."""
    p = _page_state(kv_pages, page_size, ref_count, block_table)
    dev = kv_pages.device
    ref_out = ref_count if ref_count_out is None else ref_count_out
    table_out = block_table if block_table_out is None else block_table_out
    _ints("ref_count_out", ref_out, 1, dev)
    _ints("block_table_out", table_out, 2, dev)
    if ref_out.shape != ref_count.shape or table_out.shape != block_table.shape:
        raise ValueError("the outputs must have the shapes of ref_count and block_table")
    side = _side(stream, dev)
    if info is None:
        info = _empty(side, 2, torch.int32, dev)
    _ints("info", info, 1, dev)
    if info.shape[0] != 2:
        raise ValueError("info must be int32 [2]")
    ws = _cache_workspace(p, workspace, dev, side)
    with _on(dev):
        st = _lib.load().smla_cache_compact(_adr(kv_pages), _adr(ref_count), _adr(block_table), _adr(ref_out),
                                            _adr(table_out), _adr(info), ctypes.byref(p), _adr(ws),
                                            _bytes(ws), _stream_on(stream, dev))
    if side is not None:
        _keep(side, kv_pages, ref_count, block_table, ref_out, table_out, info, ws)
    _check(st, "smla_cache_compact")
    return info


def smla_cache_reorder_workspace_size(params: _lib.SmlaCacheParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load().smla_cache_reorder_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "smla_cache_reorder_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _reorder_bytes(num_seqs: int, max_pages: int) -> int:
    """What smla_cache_reorder_workspace_size says: a matter of these two sizes alone."""
    return smla_cache_reorder_workspace_size(make_cache_params(1, 1, num_seqs, max_pages))


def smla_cache_reorder(kv_pages: torch.Tensor, page_size: int, ref_count: torch.Tensor,
                       block_table: torch.Tensor, kv_lens: torch.Tensor, parents: torch.Tensor,
                       workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> None:
    """Row r of the table goes on from what row parents[r] held, in place: its lowest child takes a
    row over, the others share full pages and copy a last one, and rows without a child are freed.
    parents[r] < 0 empties row r."""
    p = _page_state(kv_pages, page_size, ref_count, block_table)
    dev = kv_pages.device
    _ints("kv_lens", kv_lens, 1, dev)
    _ints("parents", parents, 1, dev)
    if kv_lens.shape[0] != block_table.shape[0] or parents.shape[0] != block_table.shape[0]:
        raise ValueError("kv_lens and parents must be [B] for a block_table of B rows")
    side = _side(stream, dev)
    if workspace is None:
        workspace = _empty(side, _reorder_bytes(p.num_seqs, p.max_pages), torch.uint8, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    with _on(dev):
        st = _lib.load().smla_cache_reorder(_adr(kv_pages), _adr(ref_count), _adr(block_table), _adr(kv_lens),
                                            _adr(parents), ctypes.byref(p), _adr(workspace), _bytes(workspace),
                                            _stream_on(stream, dev))
    if side is not None:
        _keep(side, kv_pages, ref_count, block_table, kv_lens, parents, workspace)
    _check(st, "smla_cache_reorder")


_LOGITS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def make_beam_params(groups: int, beams: int, vocab: int, num_out: int, row_stride: Optional[int] = None,
                     logits_type: int = 0, end_token: int = 0) -> _lib.SmlaBeamParams:
    return _lib.SmlaBeamParams(groups, beams, vocab, num_out, vocab if row_stride is None else row_stride,
                               logits_type, end_token, 0)


def smla_beam_workspace_size(params: _lib.SmlaBeamParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load().smla_beam_workspace_size(ctypes.byref(params), ctypes.byref(n)), "smla_beam_workspace_size")
    return n.value


@functools.lru_cache(maxsize=256)
def _beam_bytes(groups: int, beams: int, vocab: int, num_out: int, logits_type: int) -> int:
    """What smla_beam_workspace_size says: a matter of these sizes and the type alone."""
    return smla_beam_workspace_size(make_beam_params(groups, beams, vocab, num_out, logits_type=logits_type))


def smla_beam_select(logits: torch.Tensor, scores: torch.Tensor, num_out: Optional[int] = None,
                     finished: Optional[torch.Tensor] = None, end_token: int = 0,
                     parents: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None,
                     out_scores: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The num_out (default: as many as beams) best continuations of each group by score +
    log-softmax(logits): logits fp32, bf16 or fp16 [G * K, V] (rows at least V elements apart), scores fp32
    [G, K].  Beams with finished (uint8 or bool [G * K]) keep their score and take end_token.  out_scores may
    be scores.  Returns (parents int32 [G, num_out], rows of logits; tokens int32; scores fp32), best first."""
    dev = logits.device
    if logits.dim() != 2 or logits.dtype not in _LOGITS or logits.stride(1) != 1 or not logits.is_cuda:
        raise ValueError("logits must be fp32, bf16 or fp16 [G * K, V] with unit column stride on a CUDA device")
    if scores.dim() != 2 or scores.dtype != torch.float32 or not scores.is_contiguous() or scores.device != dev:
        raise ValueError(f"scores must be contiguous fp32 [G, K] on {dev}")
    G, K = scores.shape
    V = logits.shape[1]
    if logits.shape[0] != G * K:
        raise ValueError("logits must have a row for each of scores")
    if finished is not None and (finished.dtype not in (torch.uint8, torch.bool) or finished.shape != (G * K,)
                                 or not finished.is_contiguous() or finished.device != dev):
        raise ValueError(f"finished must be contiguous uint8 or bool [G * K] on {dev}")
    n = K if num_out is None else num_out
    stride = logits.stride(0) if logits.shape[0] > 1 else V
    p = make_beam_params(G, K, V, n, stride, _LOGITS[logits.dtype], end_token)
    side = _side(stream, dev)
    got = []
    for name, t, dtype in (("parents", parents, torch.int32), ("tokens", tokens, torch.int32),
                           ("out_scores", out_scores, torch.float32)):
        if t is None:
            t = _empty(side, (G, max(n, 0)), dtype, dev)
        elif t.shape != (G, n) or t.dtype != dtype or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be contiguous {dtype} [{G}, {n}] on {dev}")
        got.append(t)
    if workspace is None:
        workspace = _empty(side, _beam_bytes(G, K, V, n, _LOGITS[logits.dtype]), torch.uint8, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    with _on(dev):
        st = _lib.load().smla_beam_select(_adr(logits), _adr(scores), _adr(finished), _adr(got[0]), _adr(got[1]),
                                          _adr(got[2]), ctypes.byref(p), _adr(workspace), _bytes(workspace),
                                          _stream_on(stream, dev))
    if side is not None:
        _keep(side, logits, scores, finished, *got, workspace)
    _check(st, "smla_beam_select")
    return got[0], got[1], got[2]


def make_chunk_params(batch: int, num_heads: int, total_q: int, page_size: int, max_pages: int,
                      num_rows: int, kv_row_stride: int, max_kv_tokens: int,
                      softmax_scale: float = DEFAULT_SCALE, logit_cap: float = 0.0
                      ) -> _lib.SmlaChunkParams:
    return _lib.SmlaChunkParams(batch, num_heads, total_q, page_size, max_pages, 0, num_rows,
                                kv_row_stride, max_kv_tokens, softmax_scale, logit_cap)


def smla_chunk_workspace_size(params: _lib.SmlaChunkParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib.load().smla_chunk_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "smla_chunk_workspace_size")
    return n.value


@functools.lru_cache(maxsize=1024)
def _chunk_bytes(batch: int, num_heads: int, total_q: int, row_bytes: int, max_kv_tokens: int) -> int:
    """What smla_chunk_workspace_size says: a matter of these sizes and of the kind of rows alone."""
    return smla_chunk_workspace_size(make_chunk_params(batch, num_heads, total_q, 1, 1, 1, row_bytes, max_kv_tokens))


def smla_chunk_attention(q: torch.Tensor, kv_pages: torch.Tensor, block_table: torch.Tensor,
                         page_size: int, cu_q: torch.Tensor, kv_lens: torch.Tensor,
                         softmax_scale: float = DEFAULT_SCALE, logit_cap: float = 0.0,
                         slopes: Optional[torch.Tensor] = None,
                         vis_begin: Optional[torch.Tensor] = None,
                         vis_end: Optional[torch.Tensor] = None,
                         max_kv_tokens: Optional[int] = None, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None
                         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of the chunk's tokens q bf16 [T, H, 512] (sequence b's are
    q[cu_q[b]:cu_q[b + 1]], the last ones of its kv_lens[b] cached tokens) over the paged
    cache, causal unless vis_begin / vis_end say otherwise.  max_kv_tokens bounds the sum of
    kv_lens (default: what the table can hold, 2^30 at most); from 256 rows of q (tokens times
    heads) a sequence on it sizes the workspace, 1,025 bytes a token, so a caller with a wide
    table gives the bound that it knows.  Returns (out bf16 [T, H, 448], lse fp32 [T, H])."""
    row_stride = _pool(kv_pages, page_size)
    dev = kv_pages.device
    if q.dim() != 3 or q.shape[2] != QK or q.dtype != torch.bfloat16 or not q.is_contiguous() or q.device != dev:
        raise ValueError(f"q must be contiguous bf16 [T, H, 512] on {dev}")
    T, H, _ = q.shape
    _ints("block_table", block_table, 2, dev)
    _ints("cu_q", cu_q, 1, dev)
    _ints("kv_lens", kv_lens, 1, dev)
    B, max_pages = block_table.shape
    if cu_q.shape[0] != B + 1 or kv_lens.shape[0] != B:
        raise ValueError("cu_q must be [B + 1] and kv_lens [B] for a block_table of B rows")
    for name, t in (("vis_begin", vis_begin), ("vis_end", vis_end)):
        if t is not None:
            _ints(name, t, 1, dev)
            if t.shape[0] != T:
                raise ValueError(f"{name} must be int32 [T]")
    if slopes is not None and (slopes.dtype != torch.float32 or slopes.shape != (H,)
                               or not slopes.is_contiguous() or slopes.device != dev):
        raise ValueError(f"slopes must be contiguous fp32 [H] on {dev}")
    side = _side(stream, dev)
    if out is None:
        out = _empty(side, (T, H, NOPE), torch.bfloat16, dev)
    elif out.shape != (T, H, NOPE) or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"out must be contiguous bf16 [{T}, {H}, {NOPE}] on {dev}")
    if lse is None:
        lse = _empty(side, (T, H), torch.float32, dev)
    elif lse.shape != (T, H) or lse.dtype != torch.float32 or not lse.is_contiguous() or lse.device != dev:
        raise ValueError(f"lse must be contiguous fp32 [{T}, {H}] on {dev}")
    if max_kv_tokens is None:
        max_kv_tokens = min(B * max_pages * page_size, MAX_KV_TOKENS)
    p = make_chunk_params(B, H, T, page_size, max_pages, kv_pages.shape[0], row_stride,
                          max_kv_tokens, softmax_scale, logit_cap)
    if workspace is None:
        workspace = _empty(side, _chunk_bytes(B, H, T, p.kv_row_stride, max_kv_tokens), torch.uint8, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    with _on(dev):
        st = _lib.load().smla_chunk_attention(
            _adr(q), _adr(kv_pages), _adr(block_table), _adr(cu_q), _adr(kv_lens), _adr(vis_begin),
            _adr(vis_end), _adr(slopes), _adr(out), _adr(lse), ctypes.byref(p), _adr(workspace),
            _bytes(workspace), _stream_on(stream, dev))
    if side is not None:
        _keep(side, q, kv_pages, block_table, cu_q, kv_lens, slopes, vis_begin, vis_end, out, lse, workspace)
    _check(st, "smla_chunk_attention")
    return out, lse


def smla_device_status(clear: bool = False) -> int:
    """Device status word (0, SMLA_ERR_TIMEOUT or SMLA_ERR_INDEX_RANGE); synchronises."""
    lib = _lib.load()
    v = ctypes.c_int32(0)
    _check(lib.smla_device_status(ctypes.byref(v), 1 if clear else 0), "smla_device_status")
    return v.value


def smla_status_string(status: int) -> str:
    return _lib.load().smla_status_string(status).decode()
