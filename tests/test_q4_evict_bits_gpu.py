"""The bits of the weights that an eviction leaves, for heads whose rows fit the registers once and for longer ones."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q4_reference as R
from tests.test_q4_gpu import F32, check_evict, lengths, ok, randn, raw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,cap,keep,recent", [
    ([5000, 1, 4097], 5003, 1025, 128), ([60000, 60001], 65536, 20000, 0),
    ([70000, 99999, 3], 100001, 30000, 11), ([140000, 65537], 150001, 65537, 5)], ids=str)
def test_weights_that_stay_have_the_bits_of_their_keys(lens, cap, keep, recent):
    Hkv, D = 2, 16
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=len(lens), seed=1, device=G.dev()))
    w = randn((len(lens), Hkv, cap), F32, 2, 3.0)
    pick = torch.randint(0, 12, w.shape, generator=torch.Generator().manual_seed(4)).to(G.dev())
    w[pick == 0] = -0.0
    w[pick == 1] = 0.0
    w.view(torch.int32)[pick == 2] = 0x7fc01234                 # NaN of both signs, with a payload
    w.view(torch.int32)[pick == 3] = -0x3fff00                  # 0xffc00100
    w0, before = w.clone(), raw(cache)
    left, rows = pkg.cache_evict_q4(cache, w, lengths(lens), keep, recent=recent)
    check_evict(cache, before, w, w0.cpu().to(G.dev()), lens, keep, recent, left.tolist(), rows)
    got, was = w.view(torch.int32), w0.view(torch.int32)
    zero_or = torch.where(w0 == 0, torch.zeros_like(was), torch.where(w0.isnan(), torch.full_like(was, 0x7fffffff), was))
    for b, n in enumerate(lens):
        if n <= keep:
            assert torch.equal(got[b], was[b])
            continue
        assert torch.equal(got[b, :, :keep], zero_or[b].gather(1, rows[b].long()))
        assert not got[b, :, keep:n].any() and torch.equal(got[b, :, n:], was[b, :, n:])
    ok()
