"""Accumulated weights where all scores together would pass four gigabytes: some sequences at a time."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests.test_q4_gpu import BF16, F32, attention_case, check_attention, lengths, ok

pytestmark = pytest.mark.gpu


CASES = [  # sequences, T, H, Hkv, D, cap, window, dtype
    (9, 32, 32, 8, 128, 131072, 0, F32),      # eight sequences at a time
    (18, 32, 16, 4, 512, 131000, 200, BF16),  # sixteen
    (44, 6, 32, 8, 128, 131072, 0, BF16),     # 42
    (5, 25, 24, 6, 512, 65500, 0, F32),       # all
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_scores_take_four_gigabytes_at_most(case):
    B, T, H, Hkv, D, cap, window, dt = case
    need = pkg.decode_workspace_bytes_q4(B, T, H, Hkv, D, cap, weights=True, dtype=dt)
    assert need <= (1 << 32) + (64 << 20)
    lens = [(300, 17, 0, 299, 64, 1, 211)[b % 7] for b in range(B)]
    full = (lens, T, H, Hkv, D, window, 300, dt)
    small, q, k, v = attention_case(full, 3)
    cache = pkg.q4_cache(Hkv, cap, D, batch=B)
    for to, of in zip(cache[:4], small[:4]):
        to.view(torch.uint8)[:, :, :300] = of.view(torch.uint8)
    w0 = torch.rand(B, Hkv, cap, device=G.dev())
    w = w0.clone()
    wide = torch.zeros(B, T, H + 4, D, dtype=dt, device=G.dev())          # columns of wider buffers
    wide[:, :, 2:-2] = q
    to = torch.full((B, T, H + 2, D), 5.0, dtype=dt, device=G.dev())
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=G.dev())
    out = pkg.decode_attention_q4(wide[:, :, 2:-2], cache, lengths(lens), to[:, :, 1:-1], weights=w, window=window,
                                  workspace=ws)
    check_attention(out, w[:, :, :300].contiguous(), w0[:, :, :300].contiguous(), q, k, v, full)
    assert torch.equal(w[:, :, 300:], w0[:, :, 300:]) and (to[:, :, 0] == 5).all() and (to[:, :, -1] == 5).all()
    again = w0.clone()
    other = pkg.decode_attention_q4(q, cache, lengths(lens), weights=again, window=window)
    assert torch.equal(other, out) and torch.equal(again, w)
    ok()
    # lengths out of range, of the last sequence alone
    lens[-1] = cap + 1
    again = w0.clone()
    other = torch.full_like(q, 3.0)
    pkg.decode_attention_q4(q, cache, lengths(lens), other, weights=again, window=window)
    ok(-11)
    # (not the same bits: how the list of work is cut, and so the order of sums, goes by all lengths of a launch)
    check_attention(other[:-1], again[:-1, :, :300].contiguous(), w0[:-1, :, :300].contiguous(), q, k, v,
                    (lens[:-1], *full[1:]))
    assert (other[-1] == 3).all() and torch.equal(again[-1], w0[-1])
    # captured, replayed over other lengths
    lens[-1] = 250
    n = lengths(lens)
    again, other = w0.clone(), torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.decode_attention_q4(q, cache, n, other, weights=again, window=window, workspace=ws)
    n.copy_(lengths([(x * 5 + b) % 301 for b, x in enumerate(lens)]))
    graph.replay()
    torch.cuda.synchronize()
    w = w0.clone()
    out = pkg.decode_attention_q4(q, cache, n, weights=w, window=window)
    # (bits: some rows that are seen now are NaN)
    assert torch.equal(other.view(torch.uint8), out.view(torch.uint8))
    assert torch.equal(again.view(torch.uint8), w.view(torch.uint8))
    ok()
