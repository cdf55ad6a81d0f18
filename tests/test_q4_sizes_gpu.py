"""Workspaces of the 4-bit cache's attention: one sized for the largest call holds every smaller one."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q4_reference as R
from tests import q8_reference as R8
from tests.test_q4_gpu import BF16, F32, attention_case, check_attention, lengths, ok, randn, within

pytestmark = pytest.mark.gpu


DECODE = [  # sequences, largest T, H, Hkv, D, cap, dtype
    (12, 8, 32, 8, 128, 4096, BF16),      # 4 to 32 rows of many heads: stored scores up to 24
    (12, 3, 64, 8, 128, 4096, BF16),      # 8, 16 and 24 rows
    (2, 4, 32, 8, 128, 30000, BF16),      # few heads: stored scores up to 8 rows
    (3, 5, 8, 2, 512, 500, BF16),
    (5, 6, 8, 2, 128, 700, F32),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_one_workspace_for_every_smaller_decode(case):
    B, T, H, Hkv, D, cap, dt = case
    ns = [min(cap, n) for n in (300, 17, 0, 1, 299, 64, 128, 5, 40, 211, 63, 250)[:B]]
    need = pkg.decode_workspace_bytes_q4(B, T, H, Hkv, D, cap, weights=True, dtype=dt)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=G.dev())
    for b in {B, (B + 1) // 2, 1}:
        for t in range(T, 0, -1):
            lens = ns[:b]
            full = (lens, t, H, Hkv, D, 0, 300, dt)
            small, q, k, v = attention_case(full, 7 * t + b)
            cache = pkg.q4_cache(Hkv, cap, D, batch=b)
            for to, of in zip(cache[:4], small[:4]):
                to.view(torch.uint8)[:, :, :300] = of.view(torch.uint8)
            assert pkg.decode_workspace_bytes_q4(b, t, H, Hkv, D, cap, dtype=dt) <= need
            w0 = torch.rand(b, Hkv, cap, device=G.dev())
            w = w0.clone()
            out = pkg.decode_attention_q4(q, cache, lengths(lens), weights=w, workspace=ws)
            check_attention(out, w[:, :, :300].contiguous(), w0[:, :, :300].contiguous(), q, k, v, full)
            assert torch.equal(w[:, :, 300:], w0[:, :, 300:])
            assert torch.equal(out, pkg.decode_attention_q4(q, cache, lengths(lens), workspace=ws))
            assert torch.equal(out, pkg.decode_attention_q4(q, cache, lengths(lens), weights=w0.clone()))
    with pytest.raises(pkg.PfaError, match="SCRATCH"):
        least = pkg.decode_workspace_bytes_q4(1, 1, H, Hkv, D, 300, dtype=dt)
        pkg.decode_attention_q4(q[:, :1], cache, lengths(lens), workspace=ws[:least - 256])
    ok()


PREFILL = [  # largest T, largest start, H, Hkv, D, window, dtype
    (700, 300, 4, 1, 128, 0, BF16),       # longer chunks read back less than the decode kernel's slots take
    (700, 300, 4, 1, 128, 90, BF16),
    (300, 700, 8, 8, 128, 0, BF16),
    (400, 640, 8, 2, 512, 0, BF16),
    (100, 300, 8, 2, 128, 0, F32),
]


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_one_workspace_for_every_smaller_chunk(case):
    T, start, H, Hkv, D, window, dt = case
    cap = start + T
    need = pkg.prefill_workspace_bytes_q4(T, start, H, Hkv, D, window, dt)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=G.dev())
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, seed=6, device=G.dev()), 1, -2)
    k, v = R.values(cache.k, cache.k_scale, 1), R.values(cache.v, cache.v_scale, -2)
    q = randn((T, H, D), dt, 4, 0.5)
    for t in sorted({T, T // 2, T // 5, 33, 12, 3, 1}, reverse=True):
        for at in {start, start // 3, 0}:
            n = at + t
            out = pkg.prefill_attention_q4(q[:t], cache, start_pos=at, window=window, workspace=ws)
            want, tol, _, _ = R.attention(q[:t], k, v, n, window, R8.default_scale(D), dt)
            if dt == BF16:                     # chunks that are read back round the weights to bf16
                a, _, _, _ = R.attention(q[:t], k, v.abs(), n, window, R8.default_scale(D), dt)
                tol = tol + 2.0 ** -8 * a * (1 + 2.0 ** -8)
            within(out, want, tol, f"{t} tokens at {at}")
    with pytest.raises(pkg.PfaError, match="SCRATCH"):
        pkg.prefill_attention_q4(q, cache, start_pos=start, window=window, workspace=None)
    ok()
