"""Which path a chunk over the 4-bit cache takes, seen by the workspace that it is refused without."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q4_reference as R
from tests import q8_reference as R8
from tests.test_q4_gpu import BF16, PREFILL, ok, randn, within

pytestmark = pytest.mark.gpu


def reads_back(q, cache, start, window=0):
    """Whether the chunk's rows are read back (which takes room for them) or not (room for the decode kernel's sums)."""
    T, H, D = q.shape
    Hkv = cache.k.shape[0]
    seen = T + (min(start, window - 1) if window else start)
    back = 2 * -(-Hkv * seen * D * 2 // 256) * 256
    codes = pkg.decode_workspace_bytes_q4(1, min(T, 1024 * Hkv // H), H, Hkv, D, 64, dtype=q.dtype)
    assert back != codes
    ws = torch.empty(min(back, codes), dtype=torch.uint8, device=G.dev())
    try:
        pkg.prefill_attention_q4(q, cache, start_pos=start, window=window, workspace=ws)
        return back < codes
    except pkg.PfaError:
        return back > codes


# keys, kv heads, head_dim, rows a kv head (groups of 4): those around the rule's border, measured on both sides
CODES = [(16384, 8, 128, 128), (4096, 8, 128, 192), (32768, 8, 128, 112), (8192, 4, 128, 224), (8192, 4, 128, 256),
         (4096, 2, 128, 512), (8192, 2, 128, 448), (16384, 2, 128, 384), (8192, 1, 128, 896), (32768, 1, 128, 512),
         (1024, 2, 128, 1024), (63488, 8, 128, 96), (64, 8, 512, 128), (4096, 2, 512, 512), (16384, 4, 512, 256),
         (1024, 2, 512, 256)]
BACK = [(16384, 8, 128, 160), (63488, 8, 128, 128), (4096, 8, 128, 320), (16384, 2, 128, 512), (63488, 1, 128, 768),
        (1024, 2, 512, 640), (512, 4, 512, 288), (512, 4, 512, 320), (512, 2, 512, 576), (512, 8, 512, 160),
        (1024, 4, 512, 320), (16384, 2, 512, 768)]


@pytest.mark.parametrize("case,back", [(c, False) for c in CODES] + [(c, True) for c in BACK], ids=str)
def test_a_chunk_takes_the_path_that_measures_less(case, back):
    keys, Hkv, D, rows = case
    cache = pkg.q4_cache(Hkv, keys, D)
    q = torch.zeros(rows // 4, 4 * Hkv, D, dtype=BF16, device=G.dev())
    assert reads_back(q, cache, keys - rows // 4) == back
    # a window's keys are those that count
    long = pkg.q4_cache(Hkv, 70000, D)
    assert reads_back(q, long, 69000, keys - rows // 4) == back
    ok()


def test_a_size_for_a_late_chunk_serves_the_earlier_ones_of_another_path():
    """head_dim 512, 8 kv heads: on the codes at 60000 keys, read back at 2000."""
    T, H, Hkv, D, cap = 40, 32, 8, 512, 60040
    q = randn((T, H, D), BF16, 1)
    cache = pkg.q4_cache(Hkv, cap, D)
    need = pkg.prefill_workspace_bytes_q4(T, 60000, H, Hkv, D)
    assert not reads_back(q, cache, 60000)
    ws = torch.empty(need, dtype=torch.uint8, device=G.dev())
    paths = set()
    for start in (0, 60, 500, 2000, 3000, 9000, 20000, 60000):
        paths.add(reads_back(q, cache, start))
        pkg.prefill_attention_q4(q, cache, start_pos=start, workspace=ws)
    assert len(paths) == 2
    ok()


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_chunks_on_the_codes_round_their_weights_to_halves(case):
    """The codes' own bound (weights of 11 bits) for each chunk that does not read the cache back."""
    T, start, H, Hkv, D, window, dt = case
    n = start + T
    cache = pkg.Q4Cache(*R.make_cache(Hkv, n + 9, D, seed=6, device=G.dev()), 1, -2)
    q = randn((T, H, D), dt, 4, 0.5)
    assert reads_back(q, cache, start, window) == (case == (300, 77, 8, 2, 512, 128, BF16))
    out = pkg.prefill_attention_q4(q, cache, start_pos=start, window=window)
    k, v = R.values(cache.k, cache.k_scale, 1), R.values(cache.v, cache.v_scale, -2)
    want, tol, _, _ = R.attention(q, k, v, n, window, R8.default_scale(D), dt)
    if reads_back(q, cache, start, window):    # the 16-bit kernels round the weights to bf16
        a, _, _, _ = R.attention(q, k, v.abs(), n, window, R8.default_scale(D), dt)
        tol = tol + 2.0 ** -8 * a * (1 + 2.0 ** -8)
    within(out, want, tol)
    ok()
