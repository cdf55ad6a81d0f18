"""Operators around a 4-bit KV cache (include/pfa.h, "Operators around a 4-bit KV
cache"): quantising K and V as they are written, reading them back, attention
over the codes, and evicting rows by the attention they have had.

One step of a layer, for a batch of sequences that each got T new tokens
(lengths: their rows with them, on the device):

    q, k = qk_norm_rope(q, k, q_weight, k_weight, inv_freq, lengths=positions)
    cache_write_q4(k, v, cache, lengths=lengths)
    out = decode_attention_q4(q, cache, lengths, weights=weights)

and now and then, with `weights` a zero-initialised float32 [B, Hkv, max_seq_len]
that the steps have added to:

    lengths, rows = cache_evict_q4(cache, weights, lengths, keep, recent=recent)

Calls are enqueued, allocate, and are captured as those of the 8-bit cache.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from .q8 import _DTYPES, _bytes, _run, _workspace


class Q4Cache(NamedTuple):
    """K and V as e2m1 codes, two to a byte, with one e4m3 scale for each 16 channels of a row.

    k, v: uint8 [num_kv_heads, max_seq_len, head_dim / 2], or with a leading batch
    dimension; k_scale, v_scale: float8_e4m3fn [.., max_seq_len, head_dim / 16].  A value is
    code * scale * 2**exponent, with k_exponent for all of K and v_exponent for all of V.
    """
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_exponent: int = 0
    v_exponent: int = 0

    def slot(self, b: int) -> "Q4Cache":
        """Sequence b's part of a batch's cache (views)."""
        return Q4Cache(self.k[b], self.v[b], self.k_scale[b], self.v_scale[b], self.k_exponent,
                       self.v_exponent)


def q4_cache(num_kv_heads: int, max_seq_len: int, head_dim: int, *, batch: int | None = None,
             k_exponent: int = 0, v_exponent: int = 0, device=None) -> Q4Cache:
    """An empty 4-bit cache: head_dim is a multiple of 16.

    Scales are a full three bits fine where the largest of 16 channels is between 6 * 2**-6 (0.094) and
    6 * 448 (2688) times 2**exponent; an exponent moves that range to the size of a layer's values.
    """
    if num_kv_heads <= 0 or max_seq_len <= 0 or head_dim <= 0 or head_dim % 16:
        raise ValueError("head_dim must be a multiple of 16, the other sizes positive")
    if not (-64 <= k_exponent <= 64 and -64 <= v_exponent <= 64):
        raise ValueError("exponents must be -64 .. 64")
    lead = (num_kv_heads,) if batch is None else (batch, num_kv_heads)
    dev = device if device is not None else "cuda"
    k, v = (torch.zeros((*lead, max_seq_len, head_dim // 2), dtype=torch.uint8, device=dev)
            for _ in "kv")
    ks, vs = (torch.zeros((*lead, max_seq_len, head_dim // 16), dtype=torch.uint8, device=dev)
              .view(torch.float8_e4m3fn) for _ in "kv")
    return Q4Cache(k, v, ks, vs, k_exponent, v_exponent)


def cache_write_q4(k: torch.Tensor, v: torch.Tensor, cache: Q4Cache, *,
                   start_pos: int | None = None, lengths: torch.Tensor | None = None,
                   stream=None) -> Q4Cache:
    """Quantise new tokens into the cache in place (pfa_cache_write_q4); returns the cache.

    k, v: [T, Hkv, D] with start_pos (cache without a batch dimension), or
    [B, T, Hkv, D] with lengths, int64 [B] on the device: the sequences' lengths
    with the new tokens, which sit at lengths[b] - T .. lengths[b] - 1 (negative
    positions are padding and are skipped).
    """
    _run("cache_write_q4", stream, k, k, v, cache, start_pos, lengths)
    return cache


def cache_read_q4(cache: Q4Cache, start: int = 0, stop: int | None = None, *,
                  dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, stream=None) -> tuple:
    """Rows start .. stop - 1 as (k, v) [(B,) Hkv, stop - start, D] of dtype (pfa_cache_read_q4).

    k_out, v_out: contiguous tensors of that shape and dtype to write to.
    """
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    return _run("cache_read_q4", stream, cache.k, cache, start, stop, dtype == torch.bfloat16,
                k_out, v_out)


def decode_attention_q4(q: torch.Tensor, cache: Q4Cache, lengths: torch.Tensor,
                        out: torch.Tensor | None = None, *, weights: torch.Tensor | None = None,
                        window: int = 0, scale: float | None = None, stream=None,
                        workspace="auto") -> torch.Tensor:
    """Attention of each sequence's T newest tokens over its 4-bit cache (pfa_decode_attention_q4).

    q: [B, T, H, D] (T = 1 for plain decoding; T * H / Hkv <= 1024), float32 or
    bfloat16, D 128 or 512; cache: of a batch of B; lengths: int64 [B] on the device, the
    sequences' rows with these tokens, read when the kernel runs.  Query rows at
    negative positions (padding, empty slots) are zeros.  weights: float32 [B, Hkv,
    max_seq_len], contiguous: the softmax weights of each row, summed over the tokens and
    the query heads of the kv head, are added to it.  window <= 0 means global causal; scale
    defaults to 1/sqrt(head_dim) rounded to float32.  workspace: "auto" allocates it, or a
    uint8 CUDA tensor of decode_workspace_bytes_q4 bytes that no call that can run at the
    same time uses.
    """
    return _run("decode_q4", stream, q, q, cache, lengths, out, weights, window, scale,
                _workspace(workspace))


def decode_workspace_bytes_q4(B: int, T: int, num_heads: int, num_kv_heads: int, head_dim: int,
                              max_seq_len: int, *, weights: bool = False,
                              dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of decode_attention_q4 for a shape, on the current device: they also serve every
    call of fewer tokens or sequences, of a smaller cache or without weights."""
    return _bytes("pfa_decode_workspace_bytes_q4", B, T, num_heads, num_kv_heads, head_dim,
                  _DTYPES[dtype], max_seq_len, 1 if weights else 0)


def prefill_attention_q4(q: torch.Tensor, cache: Q4Cache, out: torch.Tensor | None = None, *,
                         start_pos: int, window: int = 0, scale: float | None = None, stream=None,
                         workspace="auto") -> torch.Tensor:
    """Prefill attention of one sequence's chunk over its 4-bit cache (pfa_prefill_attention_q4).

    q: [T, H, D], float32 or bfloat16, heads and elements dense (strides (qkv_dim, D, 1));
    cache: without a batch dimension (Q4Cache.slot), its rows up to start_pos + T
    written; out: None or a tensor with q's shape and strides.  By rows T * H / Hkv, kv heads and keys
    a bfloat16 chunk runs on the codes (softmax weights of 11 bits) or reads the visible rows back into the
    workspace (2 * Hkv * rows * D elements) and runs the attention of prefill_attention_cache on them (weights
    of 8 bits): with groups of 4 and D 128 from 32 tokens on at 63488 keys of 8 kv heads, 38 at 16384, 62 at 4096;
    from 145 on at 63488 keys of one kv head.  float32 runs on the codes.  Other arguments: as for
    prefill_attention_cache; workspace: "auto" or a uint8 CUDA tensor of prefill_workspace_bytes_q4 bytes.
    """
    return _run("prefill_q4", stream, q, q, cache, out, start_pos, window, scale,
                _workspace(workspace))


def prefill_workspace_bytes_q4(T: int, start_pos: int, num_heads: int, num_kv_heads: int,
                               head_dim: int, window: int = 0,
                               dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of prefill_attention_q4 for a shape, on the current device: they also serve every
    call of fewer tokens, an earlier start_pos, or both."""
    return _bytes("pfa_prefill_workspace_bytes_q4", T, start_pos, num_heads, num_kv_heads, head_dim,
                  window, _DTYPES[dtype])


def cache_evict_q4(cache: Q4Cache, weights: torch.Tensor, lengths: torch.Tensor, keep: int, *,
                   recent: int = 0, lengths_out: torch.Tensor | None = None,
                   rows_out: torch.Tensor | None = None, stream=None) -> tuple:
    """Cut each sequence of more than `keep` rows down to `keep`, in place (pfa_cache_evict_q4).

    Of each kv head the `recent` newest rows stay and the heaviest others by weights (float32
    [B, Hkv, max_seq_len]; equal ones: the lower row), in their order, in rows 0 .. keep - 1;
    weights move with them and are 0 behind.  cache: of a batch of B; lengths: int64 [B] on
    the device.  Returns (lengths_out, rows_out): the new lengths, int64 [B] (lengths_out may
    be lengths), and the row that each kept row was, int32 [B, Hkv, keep], -1 behind a shorter
    sequence's last.

    Heads keep different rows: what a row's number was to positions (qk_norm_rope) and to
    `window` it is no longer, so count positions apart.
    """
    return _run("cache_evict_q4", stream, weights, cache, weights, lengths, keep, recent,
                lengths_out, rows_out)
