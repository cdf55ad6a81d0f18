"""Chunks whose attention runs on the cache's codes (bf16, head_dim 128): small weights, bounds
without a term for other paths, more pairs of tiles than SMs."""
import math

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q8_reference as R
from tests.test_q8_gpu import PREFILL

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


def codes_floor(cache, n, lo):
    """What the kernel on the codes adds to R.attention()'s bound: each weight is off by up to
    2^-32 of the row's largest, and the sum of weights is at least that one."""
    v = R.values(cache.v, cache.v_scale)[:, lo:n].abs().nan_to_num(0.0).amax().item()
    return (n - lo) * 2.0 ** -32 * v


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_chunks_from_the_codes_within_their_own_bound(case):
    T, sp, H, Hkv, block, window, scale = case
    n, D = sp + T, 128
    cap = -(-n // block) * block + block
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, seed=T + 50, device=G.dev(), dead=[n]))
    g = torch.Generator().manual_seed(T)
    q = (torch.randn((T, H, D), generator=g) * 2).to(BF16).to(G.dev())
    out = pkg.prefill_attention_q8(q, cache, start_pos=sp, window=window, scale=scale)
    want, tol = R.attention(q, cache, n, window, R.default_scale(D) if scale is None else scale, BF16)
    lo = max(0, sp - window + 1) if window else 0
    over = ((out.double() - want).abs() - tol - codes_floor(cache, n, lo)).max().item()
    assert over <= 0, f"{over:.3e} over the tolerance"
    ok()


@pytest.mark.parametrize("T,sp,window,D,codes", [
    (1, 0, 0, 128, False), (1, 300, 0, 128, False), (5, 123, 40, 128, False), (12, 3000, 0, 128, False),
    (16, 0, 0, 128, True), (17, 200, 0, 128, True), (37, 101, 0, 128, True), (64, 33, 0, 128, True),
    (1, 300, 0, 512, False), (5, 123, 40, 512, False), (17, 200, 0, 512, False),
    (64, 33, 0, 512, False), (130, 500, 0, 512, False), (130, 500, 77, 512, False)])
def test_bf16_chunks_without_the_read_back_keep_their_weights(T, sp, window, D, codes):
    """8/2 heads: the decode kernel up to 48 rows (head_dim 512: 575), the codes up to 256; neither
    rounds a weight to bf16."""
    Hkv, H, block, n = 2, 8, 32, sp + T
    cap = -(-n // block) * block + block
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, seed=T, device=G.dev(), dead=[n]))
    g = torch.Generator().manual_seed(T)
    q = (torch.randn((T, H, D), generator=g) * 2).to(BF16).to(G.dev())
    out = pkg.prefill_attention_q8(q, cache, start_pos=sp, window=window)
    want, tol = R.attention(q, cache, n, window, R.default_scale(D), BF16)
    if codes:
        tol = tol + codes_floor(cache, n, max(0, sp - window + 1) if window else 0)
    over = ((out.double() - want).abs() - tol).max().item()
    assert over <= 0, f"{over:.3e} over the tolerance"
    ok()


@pytest.mark.parametrize("T,sp,H,Hkv,heads", [
    (60, 3000, 160, 160, (0, 1, 80, 151, 152, 153, 159)),    # 160 pairs: a wave and 8 that are cut
    (30, 2000, 640, 160, (0, 607, 608, 611, 639)),
    (768, 15700, 64, 64, (0, 22, 23, 24, 40, 63)),           # 192 pairs of three lengths
])
def test_more_pairs_of_tiles_than_sms(T, sp, H, Hkv, heads):
    D, block, n = 128, 64, sp + T
    cap = -(-n // block) * block
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, seed=T, device=G.dev(), dead=[n]))
    g = torch.Generator().manual_seed(T)
    q = (torch.randn((T, H, D), generator=g) * 2).to(BF16).to(G.dev())
    out = pkg.prefill_attention_q8(q, cache, start_pos=sp)
    group = H // Hkv
    for h in heads:
        kv = slice(h // group, h // group + 1)
        part = pkg.Q8Cache(*(t[kv] for t in cache))
        want, tol = R.attention(q[:, h:h + 1], part, n, 0, R.default_scale(D), BF16)
        over = ((out[:, h:h + 1].double() - want).abs() - tol - codes_floor(part, n, 0)).max().item()
        assert over <= 0, f"head {h}: {over:.3e} over the tolerance"
    assert torch.equal(out, pkg.prefill_attention_q8(q, cache, start_pos=sp))
    ok()
