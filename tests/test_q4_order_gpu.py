"""The 4-bit cache's operators behind a kernel that writes the lengths late, and kernels whose first
call is under capture."""
import os
import subprocess
import sys

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q4_reference as R
from tests.test_q8_order_gpu import late  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# B, T, H, Hkv, D, cap, dtype: weights beside the join and behind it, one tile of rows and several,
# a batch whose list takes more than a warp
SHAPES = [(3, 1, 8, 1, 128, 2048, BF16), (2, 1, 32, 8, 128, 40000, BF16), (3, 5, 8, 1, 128, 8192, BF16),
          (2, 25, 8, 1, 128, 8192, F32), (3, 3, 16, 2, 512, 4096, BF16), (40, 1, 8, 2, 128, 1000, F32)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("captured", [False, True])
def test_lengths_written_late_by_the_kernel_in_front(shape, captured, late):  # noqa: F811
    B, T, H, Hkv, D, cap, dt = shape
    keep = cap // 3
    full = [t.clone() for t in R.make_cache(Hkv, cap, D, batch=B, seed=1, device=G.dev())]
    cache = pkg.Q4Cache(*[t.clone() for t in full])
    g = torch.Generator().manual_seed(2)
    q, k, v = ((torch.randn((B, T, n, D), generator=g)).to(dt).to(G.dev()) for n in (H, Hkv, Hkv))
    w = torch.zeros(B, Hkv, cap, device=G.dev())
    lens, by = (torch.zeros(B, dtype=torch.int64, device=G.dev()) for _ in range(2))
    out = torch.empty_like(q)
    rows = torch.empty(B, Hkv, keep, dtype=torch.int32, device=G.dev())
    left = torch.empty_like(lens)

    def step():
        pkg.cache_write_q4(k, v, cache, lengths=lens)
        pkg.decode_attention_q4(q, cache, lens, out, weights=w)
        pkg.cache_evict_q4(cache, w, lens, keep, recent=2, lengths_out=left, rows_out=rows)

    def reset():
        for t, s in zip(cache, full):
            t.view(torch.uint8).copy_(s.view(torch.uint8))
        w.zero_()

    def run():
        late(lens, by)
        step()
    run()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    steps = torch.randint(T, cap + 1, (4, B), generator=g)
    steps[0], steps[1], steps[2] = cap, T, cap
    for want in steps:
        reset()
        by.copy_(want.to(G.dev()) - lens)
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert torch.equal(lens.cpu(), want) and pkg.last_device_error() == 0
        got = [t.clone() for t in (*[c.view(torch.uint8) for c in cache[:4]], w, out, rows, left)]
        reset()
        torch.cuda.synchronize()
        step()                                     # the same with lengths that have been there for long
        torch.cuda.synchronize()
        for a, b in zip(got, (*[c.view(torch.uint8) for c in cache[:4]], w, out, rows, left)):
            assert torch.equal(a, b)


FIRST_UNDER_CAPTURE = """
import torch, chunked_causal_gqa_gb300 as pkg
dev = torch.device('cuda', 0)
pkg.cache_read_q4(pkg.q4_cache(1, 8, 128), 0, 8)          # one call of the library on the device
cases = [(1, 1, 8, 2, 128, 300, torch.bfloat16), (2, 2, 32, 8, 128, 9000, torch.bfloat16), (1, 9, 8, 1, 512, 700, torch.float32),
         (1, 1, 8, 2, 512, 5000, torch.float32)]
state = []
for B, T, H, Hkv, D, cap, dt in cases:
    c = pkg.q4_cache(Hkv, cap, D, batch=B)
    for t in c[:2]:
        t.random_(0, 256)
    for t in c[2:4]:
        t.view(torch.uint8).random_(30, 50)
    q = torch.randn(B, T, H, D, device=dev).to(dt)
    k = torch.randn(B, T, Hkv, D, device=dev).to(dt)
    state.append((c, q, k, torch.full((B,), cap - 3, device=dev), torch.zeros(B, Hkv, cap, device=dev), torch.empty_like(q)))
torch.cuda.synchronize()

def run():
    for c, q, k, n, w, out in state:
        pkg.cache_write_q4(k, k, c, lengths=n)
        pkg.decode_attention_q4(q, c, n, out, weights=w)
        pkg.cache_evict_q4(c, w, n, c.k.shape[2] // 2)
        pkg.prefill_attention_q4(q[0], c.slot(0), start_pos=100)

before = [[t.clone() for t in (*c[:4], w)] for c, q, k, n, w, out in state]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
got = [[t.clone() for t in (*c[:4], w, out)] for c, q, k, n, w, out in state]
for (c, q, k, n, w, out), old in zip(state, before):
    for t, s in zip((*c[:4], w), old):
        t.view(torch.uint8).copy_(s.view(torch.uint8))
run()
torch.cuda.synchronize()
for (c, q, k, n, w, out), want in zip(state, got):
    for t, s in zip((*c[:4], w, out), want):
        assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
assert pkg.last_device_error() == 0
print('same')
"""


def test_kernels_whose_first_call_is_under_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_UNDER_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr
