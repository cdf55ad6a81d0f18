"""Chunks whose attention runs on the cache's codes (bf16, head_dim 128): small weights, bounds
without a term for other paths, more pairs of tiles than SMs."""
import math

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q8_reference as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
F8 = torch.float8_e4m3fn


def ok():
    assert pkg.last_device_error() == 0


@pytest.mark.parametrize("bits", [20, 24, 26, 27])
@pytest.mark.parametrize("n", [20000, 131072])
def test_a_flat_tail_under_a_few_large_weights(n, bits):
    """Keys whose V is zero take nearly all the weight; what is left is the whole output.

    A weight is rounded to 11 bits, a small one by up to 2^-32 of the row's largest (a half below
    2^-14 is a multiple of 2^-24, and the largest is 2^7 or more).  Every row's sum of weights is
    at least the number of large ones."""
    T, H, Hkv, D, block, apart = 17, 8, 2, 128, 64, 1024
    sp, large = n - T, -(-(n - T) // apart)                 # a large key in every range of keys
    cap = -(-n // block) * block
    g = torch.Generator().manual_seed(n + bits)
    k = torch.zeros((Hkv, cap, D))
    k[:, 0:sp:apart] = 1.0
    v = torch.randn((Hkv, cap, D), generator=g) * 0.25 + 1.0   # all of one sign nearly: no cancelling
    v[:, 0:sp:apart] = 0.0
    cache = pkg.Q8Cache(*(t.to(F8).to(G.dev()) for t in (k, v)),
                        *(torch.ones((Hkv, cap // block), device=G.dev()) for _ in "kv"))
    # head h: the other keys' weights are 2^-bits * 2^(-h / 2) of the large ones'
    q = torch.ones((T, H, D), dtype=BF16)
    q *= (1 + torch.arange(H) / (2 * bits)).to(BF16)[:, None]
    q = q.to(G.dev())
    scale = bits * math.log(2) / D
    out = pkg.prefill_attention_q8(q, cache, start_pos=sp, scale=scale)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want, tol = R.attention(q, cache, n, 0, scale, BF16)
    small = n * 2.0 ** -32 * cache.v.double().abs().max().item() / large
    assert small < want.abs().median().item() / 3           # what is asked for shows
    over = ((out.double() - want).abs() - tol - small).max().item()
    assert over <= 0, f"{over:.3e} over the tolerance, outputs of {want.abs().median().item():.3e}"
    ok()


def test_a_chunk_of_more_rows_than_the_kernel_counts_is_refused():
    heads = 1 << 24                                         # 2^30 rows and more: q alone has 256 GB
    with pytest.raises(pkg.PfaError) as e:
        pkg.prefill_workspace_bytes_q8(100, 20000, heads, heads, 128)
    assert e.value.name == "PFA_ERR_SHAPE"
    assert pkg.prefill_workspace_bytes_q8(100, 20000, 160, 160, 128) > 0
