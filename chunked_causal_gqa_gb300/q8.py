"""Operators around an 8-bit KV cache (include/pfa.h, "Operators around an
8-bit KV cache"): norm and rotation of queries and keys, quantising K and V as
they are written, reading them back, and attention over the codes.

One step of a layer, for a batch of sequences that each got T new tokens
(lengths: their lengths with them, on the device) or for one chunk (start_pos):

    q, k = qk_norm_rope(q, k, q_weight, k_weight, inv_freq, lengths=lengths)
    cache_write_q8(k, v, cache, lengths=lengths)
    out = decode_attention_q8(q, cache, lengths)

Every call is enqueued on `stream` (default: the current stream) without
synchronising, allocates its outputs and workspace on that stream, and can be
captured into a CUDA graph after one call outside a capture.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple

import torch

from . import _binding
from ._binding import PfaError

_DTYPES = {torch.float32: _binding.PFA_F32, torch.bfloat16: _binding.PFA_BF16}
_BLOCKS = (16, 32, 64, 128)
_F8 = torch.float8_e4m3fn


class Q8Cache(NamedTuple):
    """K and V as e4m3 codes with one fp32 scale for each head and block of rows.

    k, v: float8_e4m3fn [num_kv_heads, max_seq_len, head_dim], or with a leading
    batch dimension; k_scale, v_scale: float32 [.., num_kv_heads, max_seq_len / block].
    The block (16, 32, 64 or 128 rows) follows from the shapes.
    """
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def slot(self, b: int) -> "Q8Cache":
        """Sequence b's part of a batch's cache (views)."""
        return Q8Cache(self.k[b], self.v[b], self.k_scale[b], self.v_scale[b])


def q8_cache(num_kv_heads: int, max_seq_len: int, head_dim: int, *, batch: int | None = None,
             block: int = 64, device=None) -> Q8Cache:
    """An empty 8-bit cache: max_seq_len is a multiple of block (16, 32, 64 or 128)."""
    if block not in _BLOCKS or max_seq_len <= 0 or max_seq_len % block:
        raise ValueError("block must be 16, 32, 64 or 128 and divide max_seq_len")
    lead = (num_kv_heads,) if batch is None else (batch, num_kv_heads)
    dev = device if device is not None else "cuda"
    k, v = (torch.zeros((*lead, max_seq_len, head_dim), dtype=torch.uint8, device=dev)
            .view(torch.float8_e4m3fn) for _ in "kv")
    ks, vs = (torch.zeros((*lead, max_seq_len // block), dtype=torch.float32, device=dev)
              for _ in "kv")
    return Q8Cache(k, v, ks, vs)


@functools.lru_cache(maxsize=None)
def _default_scale(head_dim: int) -> float:
    return float(torch.tensor(1.0 / math.sqrt(head_dim), dtype=torch.float32))


# A decode step's kernels take a few microseconds, so what the host does for a call is kept
# short: tensors are looked at once, the raw stream is asked for directly, and that every
# pointer is memory of the current device is left to the library, which checks it.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(name: str, dev: torch.device, stream, *args) -> None:
    """Runs library function `name` on dev (made current) and the stream."""
    index = dev.index
    fn = getattr(_binding.load(), name)
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise PfaError(rc, name)


def _empty(shape, dtype, dev, stream, strides=None):
    """An output or workspace, allocated on the stream that uses it."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _empty(shape, dtype, dev, None, strides)
    if strides is not None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=dev)
    return torch.empty(shape, dtype=dtype, device=dev)


def _check_cache(cache: Q8Cache):
    """(num_kv_heads, max_seq_len, head_dim, block, batch or None)."""
    k, v, ks, vs = cache
    shape, scales = k.shape, ks.shape
    n = len(shape)
    if n not in (3, 4) or v.shape != shape:
        raise ValueError("cache.k and cache.v must be [(B,) Hkv, max_seq_len, D] of one shape")
    if k.dtype != _F8 or v.dtype != _F8:
        raise ValueError("cache.k and cache.v must be float8_e4m3fn")
    if ks.dtype != torch.float32 or vs.dtype != torch.float32:
        raise ValueError("cache.k_scale and cache.v_scale must be float32")
    cap = shape[-2]
    blocks = scales[-1] if len(scales) == n - 1 else 0
    if (blocks == 0 or scales[:-1] != shape[:-2] or vs.shape != scales or cap % blocks
            or cap // blocks not in _BLOCKS):
        raise ValueError("scales must be [(B,) Hkv, max_seq_len / block], block 16, 32, 64 or 128")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    return shape[-3], cap, shape[-1], cap // blocks, shape[0] if n == 4 else None


def _row(shape, stride, name: str, dense_heads: bool = True) -> int:
    """Elements from one token's row to the next of a [(B,) T, heads, D] tensor."""
    D = shape[-1]
    if stride[-1] != 1 or (dense_heads and stride[-2] != D and shape[-2] > 1):
        raise ValueError(f"{name}'s heads and elements must be dense (strides (row, D, 1))")
    if shape[-3] > 1:
        if len(shape) == 4 and shape[0] > 1 and stride[0] != shape[1] * stride[1]:
            raise ValueError(f"{name}'s sequences must follow one another (stride T * row)")
        return stride[-3]
    return stride[0] if len(shape) == 4 and shape[0] > 1 else shape[-2] * D


def _span(shape, lengths, start_pos):
    """(B, T, start_pos, lengths pointer) of a tensor [T, .., ..] or [B, T, .., ..]."""
    if (lengths is None) == (start_pos is None):
        raise ValueError("pass either lengths (a batch) or start_pos (one sequence)")
    if lengths is None:
        if len(shape) != 3:
            raise ValueError("with start_pos the tensors are [T, heads, D] of one sequence")
        return 1, shape[0], int(start_pos), None
    if len(shape) != 4:
        raise ValueError("with lengths the tensors are [B, T, heads, D]")
    if lengths.dtype != torch.int64 or lengths.shape != shape[:1] or not lengths.is_contiguous():
        raise ValueError("lengths must be a contiguous int64 tensor [B]")
    return shape[0], shape[1], 0, lengths.data_ptr()


def _cuda(t: torch.Tensor) -> torch.device:
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors on one device")
    return t.device


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None, *,
                 start_pos: int | None = None, lengths: torch.Tensor | None = None,
                 eps: float = 1e-6, weight_offset: float = 0.0, interleaved: bool = False,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 stream=None) -> tuple:
    """RMS norm of each query and key head and rotation of its position (pfa_qk_norm_rope).

    q: [T, H, D] with start_pos, or [B, T, H, D] with lengths (int64 [B] on the
    device; token t of sequence b is at lengths[b] - T + t, rows at negative
    positions become zeros); k: the same with Hkv heads; rows may be columns of a
    wider projection buffer.  q_weight, k_weight: [D] of the same dtype, None: no
    norm; the factor is weight + weight_offset.  inv_freq: float64 [rot_dim / 2],
    radians a position, None: no rotation.  q_out may be q; k_out may be k or, for
    one sequence, rows of a cache: cache[:, a:b].transpose(0, 1).  Returns (q_out, k_out).
    """
    shape, k_shape, dt = q.shape, k.shape, q.dtype
    if (len(shape) not in (3, 4) or k_shape[:-2] != shape[:-2] or len(k_shape) != len(shape)
            or k_shape[-1] != shape[-1]):
        raise ValueError("q must be [(B,) T, H, D] and k [(B,) T, Hkv, D]")
    if dt not in _DTYPES or k.dtype != dt:
        raise ValueError("q and k must both be float32 or both bfloat16")
    H, D, Hkv = shape[-2], shape[-1], k_shape[-2]
    B, T, start, lens = _span(shape, lengths, start_pos)
    w = [None, None]
    for i, t in enumerate((q_weight, k_weight)):
        if t is not None:
            if t.shape != shape[-1:] or t.dtype != dt or not t.is_contiguous():
                raise ValueError("weights must be contiguous [D] tensors of q's dtype")
            w[i] = t.data_ptr()
    rot, freq = 0, None
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 tensor [rot_dim / 2]")
        rot = 2 * inv_freq.shape[0]
        freq = inv_freq.data_ptr()
    q_row, k_row = _row(shape, q.stride(), "q"), _row(k_shape, k.stride(), "k")
    dev = _cuda(q)
    if q_out is None:
        q_out, q_out_row = _empty(shape, dt, dev, stream), H * D
    elif q_out.shape != shape or q_out.dtype != dt:
        raise ValueError("q_out must match q in shape and dtype")
    else:
        q_out_row = _row(shape, q_out.stride(), "q_out")
    if k_out is None:
        k_out, k_out_row, k_out_head = _empty(k_shape, dt, dev, stream), Hkv * D, D
    elif k_out.shape != k_shape or k_out.dtype != dt:
        raise ValueError("k_out must match k in shape and dtype")
    else:
        strides = k_out.stride()
        k_out_row = _row(k_shape, strides, "k_out", dense_heads=False)
        k_out_head = strides[-2] if Hkv > 1 else D
    _call("pfa_qk_norm_rope", dev, stream, q.data_ptr(), k.data_ptr(), q_out.data_ptr(),
          k_out.data_ptr(), B, T, start, lens, H, Hkv, D, w[0], w[1], eps, weight_offset, freq,
          rot, 1 if interleaved else 0, _DTYPES[dt], q_row, k_row, q_out_row, k_out_row,
          k_out_head)
    return q_out, k_out


def cache_write_q8(k: torch.Tensor, v: torch.Tensor, cache: Q8Cache, *,
                   start_pos: int | None = None, lengths: torch.Tensor | None = None,
                   stream=None) -> Q8Cache:
    """Quantise new tokens into the cache in place (pfa_cache_write_q8); returns the cache.

    k, v: [T, Hkv, D] with start_pos (cache without a batch dimension), or
    [B, T, Hkv, D] with lengths, int64 [B] on the device: the sequences' lengths
    with the new tokens, which sit at lengths[b] - T .. lengths[b] - 1 (negative
    positions are padding and are skipped).
    """
    Hkv, cap, D, block, batch = _check_cache(cache)
    shape, dt = k.shape, k.dtype
    if (len(shape) != (3 if batch is None else 4) or v.shape != shape or shape[-1] != D
            or shape[-2] != Hkv or (batch is not None and shape[0] != batch)):
        raise ValueError("k and v must be [(B,) T, Hkv, D] for the cache's heads and batch")
    if dt not in _DTYPES or v.dtype != dt:
        raise ValueError("k and v must both be float32 or both bfloat16")
    B, T, start, lens = _span(shape, lengths, start_pos)
    k_row, v_row = _row(shape, k.stride(), "k"), _row(shape, v.stride(), "v")
    _call("pfa_cache_write_q8", _cuda(k), stream, k.data_ptr(), v.data_ptr(), cache.k.data_ptr(),
          cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), B, T, start,
          lens, Hkv, D, cap, block, _DTYPES[dt], k_row, v_row)
    return cache


def cache_read_q8(cache: Q8Cache, start: int = 0, stop: int | None = None, *,
                  dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, stream=None) -> tuple:
    """Rows start .. stop - 1 as (k, v) [(B,) Hkv, stop - start, D] of dtype (pfa_cache_read_q8).

    k_out, v_out: contiguous tensors of that shape and dtype to write to.
    """
    Hkv, cap, D, block, batch = _check_cache(cache)
    stop = cap if stop is None else int(stop)
    start = int(start)
    if not 0 <= start <= stop <= cap:
        raise ValueError(f"rows {start}:{stop} are not in the cache's {cap}")
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    rows = stop - start
    shape = (Hkv, rows, D) if batch is None else (batch, Hkv, rows, D)
    for o in (k_out, v_out):
        if o is not None and (o.shape != shape or o.dtype != dtype or not o.is_contiguous()):
            raise ValueError("k_out and v_out must be contiguous [(B,) Hkv, rows, D] of dtype")
    dev = _cuda(cache.k)
    if k_out is None:
        k_out = _empty(shape, dtype, dev, stream)
    if v_out is None:
        v_out = _empty(shape, dtype, dev, stream)
    _call("pfa_cache_read_q8", dev, stream, cache.k.data_ptr(), cache.v.data_ptr(),
          cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
          Hkv if batch is None else Hkv * batch, start, rows, D, cap, block, _DTYPES[dtype],
          rows * D)
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def _need(fn: str, device: int, *shape) -> int:
    """Workspace bytes of a shape on a device."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        rc = getattr(_binding.load(), fn)(*shape, ctypes.byref(n))
    if rc != 0:
        raise PfaError(rc, fn)
    return n.value


def _workspace(workspace, dev, stream, fn: str, *shape):
    """(tensor or None, pointer, bytes) of the workspace argument of an attention call."""
    if workspace is None:
        return None, None, 0
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        need = _need(fn, dev.index, *shape)
        if need == 0:
            return None, None, 0
        workspace = _empty((need,), torch.uint8, dev, stream)
        return workspace, workspace.data_ptr(), need
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on the output's device")
    return workspace, workspace.data_ptr(), workspace.numel()


def decode_attention_q8(q: torch.Tensor, cache: Q8Cache, lengths: torch.Tensor,
                        out: torch.Tensor | None = None, *, window: int = 0,
                        scale: float | None = None, stream=None,
                        workspace="auto") -> torch.Tensor:
    """Attention of each sequence's T newest tokens over its 8-bit cache (pfa_decode_attention_q8).

    q: [B, T, H, D] (T = 1 for plain decoding; T * H / Hkv <= 1024), float32 or
    bfloat16, D 128 or 512; cache: of a batch of B; lengths: int64 [B] on the device, the
    sequences' lengths with these tokens, read when the kernel runs.  Rows at
    negative positions (padding, empty slots) are zeros.  window <= 0 means global
    causal; scale defaults to 1/sqrt(head_dim) rounded to float32.  workspace: "auto"
    allocates it, or a uint8 CUDA tensor of decode_workspace_bytes_q8 bytes that no
    call that can run at the same time uses.
    """
    Hkv, cap, D, block, batch = _check_cache(cache)
    shape, dt = q.shape, q.dtype
    if len(shape) != 4 or batch is None or shape[0] != batch or shape[-1] != D:
        raise ValueError("q must be [B, T, H, D] for the cache's batch and head_dim")
    if dt not in _DTYPES:
        raise ValueError("q must be float32 or bfloat16")
    H = shape[2]
    B, T, _, lens = _span(shape, lengths, None)
    q_row = _row(shape, q.stride(), "q")
    dev, code = _cuda(q), _DTYPES[dt]
    if out is None:
        out, out_row = _empty(shape, dt, dev, stream), H * D
    elif out.shape != shape or out.dtype != dt:
        raise ValueError("out must match q in shape and dtype")
    else:
        out_row = _row(shape, out.stride(), "out")
    held, ws, ws_bytes = _workspace(workspace, dev, stream, "pfa_decode_workspace_bytes_q8", B, T,
                                    H, Hkv, D, code)
    _call("pfa_decode_attention_q8", dev, stream, q.data_ptr(), cache.k.data_ptr(),
          cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), out.data_ptr(),
          B, T, lens, H, Hkv, D, int(window), _default_scale(D) if scale is None else scale, code,
          q_row, out_row, cap, block, ws, ws_bytes)
    return out


def decode_workspace_bytes_q8(B: int, T: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of decode_attention_q8 for a shape, on the current device."""
    return _need("pfa_decode_workspace_bytes_q8", torch.cuda.current_device(), B, T, num_heads,
                 num_kv_heads, head_dim, _DTYPES[dtype])


def prefill_attention_q8(q: torch.Tensor, cache: Q8Cache, out: torch.Tensor | None = None, *,
                         start_pos: int, window: int = 0, scale: float | None = None, stream=None,
                         workspace="auto") -> torch.Tensor:
    """Prefill attention of one sequence's chunk over its 8-bit cache (pfa_prefill_attention_q8).

    q: [T, H, D], float32 or bfloat16, heads and elements dense (strides (qkv_dim, D, 1));
    cache: without a batch dimension (Q8Cache.slot), its rows up to start_pos + T
    written; out: None or a tensor with q's shape and strides.  A chunk of more than a few
    rows reads the visible rows back into the workspace (2 * Hkv * rows * D elements of
    q's dtype) and runs the attention of prefill_attention_cache on them.  Other
    arguments: as for prefill_attention_cache; workspace: "auto" or a uint8 CUDA tensor
    of prefill_workspace_bytes_q8 bytes.
    """
    Hkv, cap, D, block, batch = _check_cache(cache)
    shape, strides, dt = q.shape, q.stride(), q.dtype
    if len(shape) != 3 or batch is not None or shape[-1] != D:
        raise ValueError("q must be [T, H, D] for one sequence's cache (Q8Cache.slot)")
    if dt not in _DTYPES:
        raise ValueError("q must be float32 or bfloat16")
    T, H, _ = shape
    row = _row(shape, strides, "q")
    dev, code, start, window = _cuda(q), _DTYPES[dt], int(start_pos), int(window)
    if out is None:
        out = _empty(shape, dt, dev, stream, strides)
    elif out.shape != shape or out.dtype != dt or (T > 1 and out.stride() != strides):
        raise ValueError("out must match q in shape, strides and dtype")
    held, ws, ws_bytes = _workspace(workspace, dev, stream, "pfa_prefill_workspace_bytes_q8", T,
                                    start, H, Hkv, D, window, code)
    _call("pfa_prefill_attention_q8", dev, stream, q.data_ptr(), cache.k.data_ptr(),
          cache.v.data_ptr(), cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), out.data_ptr(),
          T, start, H, Hkv, D, window, _default_scale(D) if scale is None else scale, code, row,
          cap, block, ws, ws_bytes)
    return out


def prefill_workspace_bytes_q8(T: int, start_pos: int, num_heads: int, num_kv_heads: int,
                               head_dim: int, window: int = 0,
                               dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of prefill_attention_q8 for a shape, on the current device."""
    return _need("pfa_prefill_workspace_bytes_q8", torch.cuda.current_device(), T, start_pos,
                 num_heads, num_kv_heads, head_dim, window, _DTYPES[dtype])
