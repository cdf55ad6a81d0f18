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
from contextlib import nullcontext
from typing import NamedTuple

import torch

from . import _binding
from ._binding import PfaError

_DTYPES = {torch.float32: _binding.PFA_F32, torch.bfloat16: _binding.PFA_BF16}
_BLOCKS = (16, 32, 64, 128)


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


def _on(dev: torch.device):
    return nullcontext() if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _alloc(stream):
    """Where outputs and workspaces are allocated: on the stream that uses them."""
    return nullcontext() if stream is None else torch.cuda.stream(stream)


def _handle(dev, stream) -> int:
    return (torch.cuda.current_stream(dev) if stream is None else stream).cuda_stream


def _check_cache(cache: Q8Cache):
    """(num_kv_heads, max_seq_len, head_dim, block, batch or None)."""
    k, v, ks, vs = cache
    if k.dim() not in (3, 4) or v.shape != k.shape:
        raise ValueError("cache.k and cache.v must be [(B,) Hkv, max_seq_len, D] of one shape")
    if k.dtype != torch.float8_e4m3fn or v.dtype != torch.float8_e4m3fn:
        raise ValueError("cache.k and cache.v must be float8_e4m3fn")
    if ks.dtype != torch.float32 or vs.dtype != torch.float32:
        raise ValueError("cache.k_scale and cache.v_scale must be float32")
    *lead, cap, D = k.shape
    blocks = ks.shape[-1] if ks.dim() == k.dim() - 1 else 0
    if (blocks == 0 or ks.shape[:-1] != k.shape[:-2] or vs.shape != ks.shape or cap % blocks
            or cap // blocks not in _BLOCKS):
        raise ValueError("scales must be [(B,) Hkv, max_seq_len / block], block 16, 32, 64 or 128")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous()
            and vs.is_contiguous()):
        raise ValueError("the cache's tensors must be contiguous")
    return lead[-1], cap, D, cap // blocks, lead[0] if len(lead) == 2 else None


def _row(t: torch.Tensor, name: str) -> int:
    """Elements from one token's row to the next of a [(B,) T, heads, D] tensor."""
    D = t.shape[-1]
    if t.stride(-1) != 1 or (t.shape[-2] > 1 and t.stride(-2) != D):
        raise ValueError(f"{name}'s heads and elements must be dense (strides (row, D, 1))")
    return _token_row(t, name, t.shape[-2] * D)


def _token_row(t: torch.Tensor, name: str, dense: int) -> int:
    T = t.shape[-3]
    if t.dim() == 3:
        return t.stride(0) if T > 1 else dense
    B = t.shape[0]
    if T > 1:
        if B > 1 and t.stride(0) != T * t.stride(1):
            raise ValueError(f"{name}'s sequences must follow one another (stride T * row)")
        return t.stride(1)
    return t.stride(0) if B > 1 else dense


def _device(first: torch.Tensor, *others) -> torch.device:
    dev = first.device
    if dev.type != "cuda" or any(t is not None and t.device != dev for t in others):
        raise ValueError("all tensors must be CUDA tensors on one device")
    return dev


def _span(x: torch.Tensor, lengths, start_pos):
    """(B, T, start_pos, lengths pointer) of x [T, .., ..] or [B, T, .., ..]."""
    if (lengths is None) == (start_pos is None):
        raise ValueError("pass either lengths (a batch) or start_pos (one sequence)")
    if lengths is None:
        if x.dim() != 3:
            raise ValueError("with start_pos the tensors are [T, heads, D] of one sequence")
        return 1, x.shape[0], int(start_pos), None
    if x.dim() != 4:
        raise ValueError("with lengths the tensors are [B, T, heads, D]")
    if lengths.dtype != torch.int64 or lengths.shape != x.shape[:1] or not lengths.is_contiguous():
        raise ValueError("lengths must be a contiguous int64 tensor [B]")
    return x.shape[0], x.shape[1], 0, lengths.data_ptr()


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
    if q.dim() not in (3, 4) or k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] \
            or k.shape[-1] != q.shape[-1]:
        raise ValueError("q must be [(B,) T, H, D] and k [(B,) T, Hkv, D]")
    if q.dtype not in _DTYPES or k.dtype != q.dtype:
        raise ValueError("q and k must both be float32 or both bfloat16")
    H, D, Hkv = q.shape[-2], q.shape[-1], k.shape[-2]
    B, T, start, lens = _span(q, lengths, start_pos)
    for w in (q_weight, k_weight):
        if w is not None and (w.shape != (D,) or w.dtype != q.dtype or not w.is_contiguous()):
            raise ValueError("weights must be contiguous [D] tensors of q's dtype")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 tensor [rot_dim / 2]")
        rot = 2 * inv_freq.numel()
    for name, o, like in (("q_out", q_out, q), ("k_out", k_out, k)):
        if o is not None and (o.shape != like.shape or o.dtype != like.dtype):
            raise ValueError(f"{name} must match in shape and dtype")
    q_row, k_row = _row(q, "q"), _row(k, "k")
    dev = _device(q, k, q_weight, k_weight, inv_freq, lengths, q_out, k_out)
    if q_out is None or k_out is None:
        with _alloc(stream):
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=dev)
    if k_out.stride(-1) != 1:
        raise ValueError("k_out's elements must be dense")
    k_head = k_out.stride(-2) if Hkv > 1 else D
    with _on(dev):
        rc = _binding.load().pfa_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), B, T, start, lens, H,
            Hkv, D, None if q_weight is None else q_weight.data_ptr(),
            None if k_weight is None else k_weight.data_ptr(), eps, weight_offset,
            inv_freq.data_ptr() if rot else None, rot, 1 if interleaved else 0, _DTYPES[q.dtype],
            q_row, k_row, _row(q_out, "q_out"), _token_row(k_out, "k_out", Hkv * D), k_head,
            _handle(dev, stream))
    if rc != 0:
        raise PfaError(rc, "pfa_qk_norm_rope")
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
    if k.dim() != cache.k.dim() or k.shape != v.shape or k.shape[-2:] != (Hkv, D) \
            or (batch is not None and k.shape[0] != batch):
        raise ValueError("k and v must be [(B,) T, Hkv, D] for the cache's heads and batch")
    if k.dtype not in _DTYPES or v.dtype != k.dtype:
        raise ValueError("k and v must both be float32 or both bfloat16")
    B, T, start, lens = _span(k, lengths, start_pos)
    k_row, v_row = _row(k, "k"), _row(v, "v")
    dev = _device(k, v, *cache, lengths)
    with _on(dev):
        rc = _binding.load().pfa_cache_write_q8(
            k.data_ptr(), v.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(),
            cache.k_scale.data_ptr(), cache.v_scale.data_ptr(), B, T, start, lens, Hkv, D, cap,
            block, _DTYPES[k.dtype], k_row, v_row, _handle(dev, stream))
    if rc != 0:
        raise PfaError(rc, "pfa_cache_write_q8")
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
    shape = (*cache.k.shape[:-2], stop - start, D)
    for o in (k_out, v_out):
        if o is not None and (o.shape != shape or o.dtype != dtype or not o.is_contiguous()):
            raise ValueError("k_out and v_out must be contiguous [(B,) Hkv, rows, D] of dtype")
    dev = _device(*cache, k_out, v_out)
    with _alloc(stream):
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=dev)
        if v_out is None:
            v_out = torch.empty(shape, dtype=dtype, device=dev)
    with _on(dev):
        rc = _binding.load().pfa_cache_read_q8(
            cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
            cache.v_scale.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
            Hkv * (1 if batch is None else batch), start, stop - start, D, cap, block,
            _DTYPES[dtype], (stop - start) * D, _handle(dev, stream))
    if rc != 0:
        raise PfaError(rc, "pfa_cache_read_q8")
    return k_out, v_out


def _workspace(workspace, need: int, dev, stream):
    """(tensor or None, pointer, bytes) of the workspace argument of an attention call."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        if need == 0:
            return None, None, 0
        with _alloc(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is None:
        return None, None, 0
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the output's device")
    return workspace, workspace.data_ptr(), workspace.numel()


def _need(fn, *args) -> int:
    n = ctypes.c_size_t(0)
    rc = getattr(_binding.load(), fn)(*args, ctypes.byref(n))
    if rc != 0:
        raise PfaError(rc, fn)
    return n.value


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
    if q.dim() != 4 or batch is None or q.shape[0] != batch or q.shape[-1] != D:
        raise ValueError("q must be [B, T, H, D] for the cache's batch and head_dim")
    if q.dtype not in _DTYPES:
        raise ValueError("q must be float32 or bfloat16")
    H = q.shape[2]
    B, T, _, lens = _span(q, lengths, None)
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype):
        raise ValueError("out must match q in shape and dtype")
    q_row = _row(q, "q")
    dev = _device(q, *cache, lengths, out)
    dt = _DTYPES[q.dtype]
    if out is None:
        with _alloc(stream):
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    with _on(dev):
        auto = isinstance(workspace, str)
        need = _need("pfa_decode_workspace_bytes_q8", B, T, H, Hkv, D, dt) if auto else 0
        held, ws, ws_bytes = _workspace(workspace, need, dev, stream)
        rc = _binding.load().pfa_decode_attention_q8(
            q.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
            cache.v_scale.data_ptr(), out.data_ptr(), B, T, lens, H, Hkv, D, int(window),
            _default_scale(D) if scale is None else scale, dt, q_row, _row(out, "out"), cap, block,
            ws, ws_bytes, _handle(dev, stream))
    if rc != 0:
        raise PfaError(rc, "pfa_decode_attention_q8")
    return out


def decode_workspace_bytes_q8(B: int, T: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of decode_attention_q8 for a shape, on the current device."""
    return _need("pfa_decode_workspace_bytes_q8", B, T, num_heads, num_kv_heads, head_dim,
                 _DTYPES[dtype])


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
    if q.dim() != 3 or batch is not None or q.shape[-1] != D:
        raise ValueError("q must be [T, H, D] for one sequence's cache (Q8Cache.slot)")
    if q.dtype not in _DTYPES:
        raise ValueError("q must be float32 or bfloat16")
    T, H, _ = q.shape
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype
                            or (T > 1 and out.stride() != q.stride())):
        raise ValueError("out must match q in shape, strides and dtype")
    row = _row(q, "q")
    dev = _device(q, *cache, out)
    dt = _DTYPES[q.dtype]
    if out is None:
        with _alloc(stream):
            out = torch.empty_strided(q.shape, q.stride(), dtype=q.dtype, device=dev)
    with _on(dev):
        auto = isinstance(workspace, str)
        need = _need("pfa_prefill_workspace_bytes_q8", T, int(start_pos), H, Hkv, D, int(window),
                     dt) if auto else 0
        held, ws, ws_bytes = _workspace(workspace, need, dev, stream)
        rc = _binding.load().pfa_prefill_attention_q8(
            q.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
            cache.v_scale.data_ptr(), out.data_ptr(), T, int(start_pos), H, Hkv, D, int(window),
            _default_scale(D) if scale is None else scale, dt, row, cap, block, ws, ws_bytes,
            _handle(dev, stream))
    if rc != 0:
        raise PfaError(rc, "pfa_prefill_attention_q8")
    return out


def prefill_workspace_bytes_q8(T: int, start_pos: int, num_heads: int, num_kv_heads: int,
                               head_dim: int, window: int = 0,
                               dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of prefill_attention_q8 for a shape, on the current device."""
    return _need("pfa_prefill_workspace_bytes_q8", T, start_pos, num_heads, num_kv_heads, head_dim,
                 window, _DTYPES[dtype])
