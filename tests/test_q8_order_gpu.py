"""Lengths that a kernel (or a copy) right in front of the 8-bit cache's operators writes: each
launch, the one that joins the parts of a head among them, has to see the new ones."""
import ctypes
import os
import subprocess

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from chunked_causal_gqa_gb300 import build
from tests import gpu_util as G
from tests import q8_reference as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# B, T, H, Hkv, D, dtype: 1, 3, 7 and 13 tiles of rows (the last three leave block places of an
# SM free while the first kernel runs), and a batch whose list takes more than a warp
SHAPES = [(3, 1, 8, 1, 128, BF16), (3, 5, 8, 1, 128, BF16), (2, 13, 16, 2, 128, BF16),
          (2, 25, 8, 1, 128, BF16), (3, 3, 16, 2, 512, BF16), (3, 5, 8, 1, 128, F32),
          (40, 1, 8, 2, 128, BF16)]
CAP, BLOCK = 8192, 64


@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """The writer of tests/late_lengths.cu."""
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "late_lengths.cu")
    lib = str(tmp_path_factory.mktemp("late") / "late.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-cudart",
                    "static", src, "-o", lib], check=True)
    f = ctypes.CDLL(lib).late_lengths_launch
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]

    def write(lengths, by):
        assert f(lengths.data_ptr(), by.data_ptr(), lengths.numel(),
                 torch.cuda.current_stream().cuda_stream) == 0
    return write


def setup(shape, seed=0):
    B, T, H, Hkv, D, dt = shape
    cache = pkg.Q8Cache(*R.make_cache(Hkv, CAP, D, BLOCK, batch=B, seed=seed, device=G.dev()))
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, T, H, D), generator=g) * 2).to(dt).to(G.dev())
    # lengths that move between a few keys and the whole cache: other parts of other heads each time
    steps = torch.randint(0, CAP + 1, (5, B), generator=g)
    steps[0], steps[1], steps[2], steps[3] = CAP, T, CAP, 0
    return cache, q, steps


def check(out, q, cache, lens, shape):
    T, D, dt = shape[1], shape[4], shape[5]
    assert pkg.last_device_error() == 0
    few = range(q.shape[0]) if q.shape[0] <= 4 else (0, 3, 17, q.shape[0] - 1)
    for b in few:
        want, tol = R.attention(q[b], cache.slot(b), int(lens[b]), 0, R.default_scale(D), dt)
        over = ((out[b].double() - want).abs() - tol).max().item()
        assert over <= 0, f"sequence {b} of length {int(lens[b])}: {over:.3e} over the tolerance"
    # and bit for bit what the same lengths give when they have been there for long
    torch.cuda.synchronize()
    still = pkg.decode_attention_q8(q, cache, lens.to(G.dev()))
    torch.cuda.synchronize()
    assert torch.equal(out, still)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("captured", [False, True])
def test_lengths_written_late_by_the_kernel_in_front(shape, captured, late):
    cache, q, steps = setup(shape)
    lens = torch.zeros(shape[0], dtype=torch.int64, device=G.dev())
    by = torch.zeros_like(lens)
    out = torch.empty_like(q)
    ws = torch.empty(pkg.decode_workspace_bytes_q8(*shape[:5], dtype=shape[5]), dtype=torch.uint8,
                     device=G.dev())

    def run():
        late(lens, by)
        pkg.decode_attention_q8(q, cache, lens, out=out, workspace=ws)
    run()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
    for want in steps:
        by.copy_(want.to(G.dev()) - lens)
        torch.cuda.synchronize()
        graph.replay() if captured else run()
        torch.cuda.synchronize()
        assert torch.equal(lens.cpu(), want)
        check(out, q, cache, want, shape)


@pytest.mark.parametrize("shape", SHAPES[:5], ids=str)
@pytest.mark.parametrize("how", ["kernel", "copy", "fill", "other stream"])
def test_lengths_written_inside_a_graph(shape, how):
    cache, q, steps = setup(shape, 1)
    lens = torch.zeros(shape[0], dtype=torch.int64, device=G.dev())
    src = torch.zeros_like(lens)
    side = torch.cuda.Stream()

    def run():
        if how == "kernel":
            lens.add_(src)
        elif how == "copy":
            lens.copy_(src)
        elif how == "fill":
            lens.zero_()
            lens.add_(src)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                lens.copy_(src)
                lens.mul_(1)
            torch.cuda.current_stream().wait_stream(side)
        return pkg.decode_attention_q8(q, cache, lens)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    lens.zero_()
    for want in steps:
        want = want.to(G.dev())
        src.copy_(want - lens if how == "kernel" else want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(lens, want)
        check(out, q, cache, want.cpu(), shape)


def test_a_step_behind_lengths_written_late(late):
    """norm + rotation, write and attention behind the writer, captured and replayed."""
    B, T, H, Hkv, D, cap = 3, 5, 8, 1, 128, 512
    cache = pkg.q8_cache(Hkv, cap, D, batch=B, block=32)
    w = torch.ones(D, dtype=BF16, device=G.dev())
    freq = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=G.dev()) / (D // 2))
    lens = torch.zeros(B, dtype=torch.int64, device=G.dev())
    by = torch.full_like(lens, T)
    qkv = torch.zeros((B, T, H + 2 * Hkv, D), dtype=BF16, device=G.dev())

    def step(write):
        if write:
            late(lens, by)
        q, k = pkg.qk_norm_rope(qkv[:, :, :H], qkv[:, :, H:H + Hkv], w, w, freq, lengths=lens)
        pkg.cache_write_q8(k, qkv[:, :, H + Hkv:], cache, lengths=lens)
        return q, k, pkg.decode_attention_q8(q, cache, lens)
    step(True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(True)
    lens.zero_()
    for t in cache:
        t.view(torch.uint8).zero_()
    for i in range(20):
        g = torch.Generator().manual_seed(i)
        qkv.copy_(torch.randn(qkv.shape, generator=g).to(BF16))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [T * (i + 1)] * B
        for b in range(B):
            want, tol = R.attention(got[0][b], cache.slot(b), T * (i + 1), 0, R.default_scale(D), BF16)
            assert ((got[2][b].double() - want).abs() <= tol).all()
        # the same step once more, on the same lengths, changes nothing
        once = [t.clone() for t in (*got, *(c.view(torch.uint8) for c in cache))]
        again = (*step(False), *(c.view(torch.uint8) for c in cache))
        for a, b in zip(once, again):
            assert torch.equal(a, b)
    assert pkg.last_device_error() == 0
