"""Reading back more rows of a head than one launch counts (2^30 pieces of 16 output bytes)."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def test_more_rows_than_one_launch_counts():
    Hkv, D, block, start = 2, 512, 128, 37                  # fp32: 128 pieces a row
    most = (1 << 30) // 128
    cap, stop = most + 4096, most + 4000                    # two launches, the second of 3963 rows
    g = torch.Generator(device=G.dev()).manual_seed(1)
    codes = torch.randint(0, 0x7f, (Hkv, cap, D), generator=g, dtype=torch.uint8, device=G.dev())
    codes = codes.view(torch.float8_e4m3fn)
    e = torch.randint(-9, 9, (Hkv, cap // block), generator=g, device=G.dev())
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    # K and V share their codes (8.6 GB) and differ in their scales; the outputs take 34 GB each
    cache = pkg.Q8Cache(codes, codes, scale, scale * 4)
    k, v = pkg.cache_read_q8(cache, start, stop, dtype=torch.float32)
    assert pkg.last_device_error() == 0
    step = 1 << 20
    for a in list(range(start, stop, step)) + [start + most - 7, stop - 1]:
        b = min(a + step, stop)
        s = scale[:, torch.arange(a, b, device=G.dev()) // block][..., None]
        want = codes[:, a:b].float() * s
        assert torch.equal(k[:, a - start:b - start], want), a
        assert torch.equal(v[:, a - start:b - start], want.mul_(4)), a
    del k, v, codes, cache, want, s
    torch.cuda.empty_cache()
