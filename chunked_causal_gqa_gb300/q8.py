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

The checks, the allocations and the library calls are made by _pfa_torch.so
(csrc/pfa_torch.cpp), built beside libpfa.so: in Python they cost several times
what the kernels of a decode step take.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
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


_lock = threading.Lock()
_module = None


def _ext():
    """_pfa_torch.so (raises if it is missing or another torch's: build it with build.build())."""
    global _module
    if _module is None:
        with _lock:
            if _module is None:
                from . import build
                _binding.load()
                if not os.path.exists(build.EXT):
                    raise ImportError(
                        f"_pfa_torch.so not found at {build.EXT}; build it with "
                        "`python -c 'import chunked_causal_gqa_gb300.build as b; b.build_extension()'`")
                if build.built_environment() != build.extension_environment():
                    raise ImportError(
                        f"{build.EXT} was built for '{build.built_environment()}', this is "
                        f"'{build.extension_environment()}'; build it again with "
                        "`python -c 'import chunked_causal_gqa_gb300.build as b; b.build_extension()'`")
                spec = importlib.util.spec_from_file_location("_pfa_torch", build.EXT)
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                _module = module
    return _module


def _run(fn: str, stream, first: torch.Tensor, *args):
    """Calls the extension with `stream` (None: as it is) as the current stream."""
    f = getattr(_module or _ext(), fn)
    if stream is None:
        return f(*args)
    if stream.device != first.device:
        raise ValueError("stream must be one of the tensors' device")
    with torch.cuda.stream(stream):
        return f(*args)


def _workspace(workspace):
    """The extension's form: None allocates, False is none."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        return None
    return False if workspace is None else workspace


def _bytes(fn: str, *shape) -> int:
    n = ctypes.c_size_t(0)
    rc = getattr(_binding.load(), fn)(*shape, ctypes.byref(n))
    if rc != 0:
        raise PfaError(rc, fn)
    return n.value


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
    return _run("qk_norm_rope", stream, q, q, k, q_weight, k_weight, inv_freq, start_pos, lengths,
                eps, weight_offset, interleaved, q_out, k_out)


def cache_write_q8(k: torch.Tensor, v: torch.Tensor, cache: Q8Cache, *,
                   start_pos: int | None = None, lengths: torch.Tensor | None = None,
                   stream=None) -> Q8Cache:
    """Quantise new tokens into the cache in place (pfa_cache_write_q8); returns the cache.

    k, v: [T, Hkv, D] with start_pos (cache without a batch dimension), or
    [B, T, Hkv, D] with lengths, int64 [B] on the device: the sequences' lengths
    with the new tokens, which sit at lengths[b] - T .. lengths[b] - 1 (negative
    positions are padding and are skipped).
    """
    _run("cache_write", stream, k, k, v, cache, start_pos, lengths)
    return cache


def cache_read_q8(cache: Q8Cache, start: int = 0, stop: int | None = None, *,
                  dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, stream=None) -> tuple:
    """Rows start .. stop - 1 as (k, v) [(B,) Hkv, stop - start, D] of dtype (pfa_cache_read_q8).

    k_out, v_out: contiguous tensors of that shape and dtype to write to.
    """
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    return _run("cache_read", stream, cache.k, cache, start, stop, dtype == torch.bfloat16, k_out,
                v_out)


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
    return _run("decode", stream, q, q, cache, lengths, out, window, scale, _workspace(workspace))


def decode_workspace_bytes_q8(B: int, T: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of decode_attention_q8 for a shape, on the current device."""
    return _bytes("pfa_decode_workspace_bytes_q8", B, T, num_heads, num_kv_heads, head_dim,
                  _DTYPES[dtype])


def prefill_attention_q8(q: torch.Tensor, cache: Q8Cache, out: torch.Tensor | None = None, *,
                         start_pos: int, window: int = 0, scale: float | None = None, stream=None,
                         workspace="auto") -> torch.Tensor:
    """Prefill attention of one sequence's chunk over its 8-bit cache (pfa_prefill_attention_q8).

    q: [T, H, D], float32 or bfloat16, heads and elements dense (strides (qkv_dim, D, 1));
    cache: without a batch dimension (Q8Cache.slot), its rows up to start_pos + T
    written; out: None or a tensor with q's shape and strides.  A long bfloat16 chunk
    reads the visible rows back into the workspace (2 * Hkv * rows * D elements) and runs
    the attention of prefill_attention_cache on them; others run on the codes.  Other
    arguments: as for prefill_attention_cache; workspace: "auto" or a uint8 CUDA tensor
    of prefill_workspace_bytes_q8 bytes.
    """
    return _run("prefill", stream, q, q, cache, out, start_pos, window, scale,
                _workspace(workspace))


def prefill_workspace_bytes_q8(T: int, start_pos: int, num_heads: int, num_kv_heads: int,
                               head_dim: int, window: int = 0,
                               dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of prefill_attention_q8 for a shape, on the current device."""
    return _bytes("pfa_prefill_workspace_bytes_q8", T, start_pos, num_heads, num_kv_heads, head_dim,
                  window, _DTYPES[dtype])
