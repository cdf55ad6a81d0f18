"""Lengths that no sequence can have, in the operators that read them on the device."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,T", [(128, 128, 1), (128, 64, 3), (512, 512, 2), (80, 0, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_leaves_sequences_of_negative_length_unwritten(dt, D, rot, T, in_place):
    H, Hkv, lens = 5, 1, [-1, 7, 0, -(1 << 40), T, -T, -(1 << 63)]
    B = len(lens)
    g = torch.Generator().manual_seed(D + T)
    q, k = (torch.randn((B, T, h, D), generator=g).to(dt).to(G.dev()) for h in (H, Hkv))
    w = torch.ones(D, dtype=dt, device=G.dev())
    freq = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64, device=G.dev()) / max(rot // 2, 1)) if rot else None
    n = torch.tensor(lens, device=G.dev())
    want = pkg.qk_norm_rope(q, k, w, w, freq, lengths=n.clamp(min=0))
    assert pkg.last_device_error() == 0
    outs = (q, k) if in_place else tuple(torch.full_like(t, 3.0) for t in (q, k))
    before = [t.clone() for t in outs]
    pkg.qk_norm_rope(q, k, w, w, freq, lengths=n, q_out=outs[0], k_out=outs[1])
    assert pkg.last_device_error() == -11
    for b, length in enumerate(lens):
        for out, old, right in zip(outs, before, want):
            assert torch.equal(out[b], old[b] if length < 0 else right[b]), (b, length)
    assert pkg.last_device_error() == 0
