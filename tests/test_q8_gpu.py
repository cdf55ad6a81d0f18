"""The operators around the 8-bit cache on the GPU, against the plain 64-bit
forms of q8_reference.py: sizes, masks, strides, streams and graphs."""
import random

import numpy as np
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q8_reference as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


def ok(code=0):
    assert pkg.last_device_error() == code


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(G.dev())


def within(got, want, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = ((got - want).abs() - tol).max().item()
    assert over <= 0, f"{what}: {over:.3e} over the tolerance"


# ------------------------------------------------------------------ norm + rotation

NORM = [  # B, T, H, Hkv, D, dtype, rot, interleaved, norm
    (1, 1, 32, 8, 128, BF16, 128, False, True),
    (5, 1, 32, 8, 128, BF16, 128, False, True),
    (3, 4, 7, 1, 128, F32, 64, False, True),
    (1, 129, 8, 2, 512, BF16, 512, True, True),
    (1, 33, 8, 2, 512, F32, 128, True, True),
    (2, 3, 5, 5, 80, BF16, 32, False, True),
    (2, 3, 5, 5, 80, F32, 80, True, False),
    (1, 17, 3, 1, 16, BF16, 16, False, True),
    (1, 9, 4, 2, 144, F32, 0, False, True),
    (4, 2, 6, 2, 336, BF16, 96, True, False),
    (1, 3, 64, 64, 496, F32, 496, False, True),
    (1, 700, 12, 4, 64, BF16, 64, False, True),
]


def norm_tol(y, size, dtype):
    # the angle is rounded to a float of up to one half turn (2^-24 pi), sine and cosine are
    # off by 2^-23 each; the norm's factor by 2^-20 (sum of up to 512 squares in a tree of 21
    # steps, mean, rsqrt, three products); the rotation's products and sum by 2^-22 of the terms
    return R.HALF[dtype] * y.abs() + (1 + R.HALF[dtype]) * size * (
        3.2 * 2.0 ** -24 + 2 * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -22)


@pytest.mark.parametrize("case", NORM, ids=str)
@pytest.mark.parametrize("place", ["new", "in_place", "columns"])
def test_norm_rope(case, place):
    B, T, H, Hkv, D, dt, rot, inter, norm = case
    rng = random.Random(str(case))
    buf = randn((B, T, H + 2 * Hkv, D), dt, 1, 3.0)
    q, k = (buf[:, :, :H], buf[:, :, H:H + Hkv])
    if place == "new":
        q, k = q.clone(), k.clone()
    qw, kw = (randn((D,), dt, s, 0.3) if norm else None for s in (2, 3))
    freq = torch.tensor([5e5 ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64,
                        device=G.dev()) if rot else None
    lens = [rng.choice((0, T - 1, T, 4097, 131072, 1 << 20, (1 << 31) - 5000)) for _ in range(B)]
    lens = [max(0, n) for n in lens]
    q0, k0, rest = q.clone(), k.clone(), buf[:, :, H + Hkv:].clone()
    kwargs = dict(eps=1e-5, weight_offset=1.0, interleaved=inter)
    if place != "new":
        kwargs.update(q_out=q, k_out=k)
    d = torch.tensor(lens, device=G.dev())
    qo, ko = pkg.qk_norm_rope(q, k, qw, kw, freq, lengths=d, **kwargs)
    for b in range(B):
        pos = torch.arange(lens[b] - T, lens[b])
        for got, x, w in ((qo, q0, qw), (ko, k0, kw)):
            y, size = R.norm_rope(x[b], w, 1.0, 1e-5, freq, pos, inter)
            pad = (pos < 0).to(G.dev())[:, None, None]
            y = torch.where(pad, 0.0, y)
            within(got[b], y, torch.where(pad, 0.0, norm_tol(y, size, dt)), f"sequence {b}")
    assert torch.equal(buf[:, :, H + Hkv:], rest)
    if place == "new":
        assert torch.equal(q, q0) and torch.equal(k, k0)
    ok()


@pytest.mark.parametrize("T", [1, 2, 77])
def test_norm_rope_writes_rows_of_a_cache(T):
    H, Hkv, D, sp, cap = 8, 4, 128, 31, 200
    q, k = randn((T, H, D), BF16, 1), randn((T, Hkv, D), BF16, 2)
    w = randn((D,), BF16, 3)
    freq = 1e4 ** (-torch.arange(64, dtype=torch.float64, device=G.dev()) / 64)
    cache = torch.full((Hkv, cap, D), 7.0, dtype=BF16, device=G.dev())
    view = cache[:, sp:sp + T].transpose(0, 1)
    qo, ko = pkg.qk_norm_rope(q, k, w, w, freq, start_pos=sp, k_out=view)
    assert ko.data_ptr() == view.data_ptr()
    q1, k1 = pkg.qk_norm_rope(q, k, w, w, freq, start_pos=sp)
    assert torch.equal(qo, q1) and torch.equal(cache[:, sp:sp + T].transpose(0, 1), k1)
    assert (cache[:, :sp] == 7).all() and (cache[:, sp + T:] == 7).all()
    y, size = R.norm_rope(k, w, 0.0, 1e-6, freq, torch.arange(sp, sp + T), False)
    within(k1, y, norm_tol(y, size, BF16))


# ------------------------------------------------------------------ write and read back

WRITE = [  # B, T, Hkv, D, block, cap, dtype
    (1, 1, 8, 128, 64, 128, BF16),
    (6, 1, 2, 128, 16, 64, F32),
    (4, 3, 3, 128, 32, 96, BF16),
    (5, 70, 2, 512, 64, 256, BF16),
    (2, 129, 1, 512, 128, 256, F32),
    (3, 5, 2, 16, 16, 48, F32),
    (2, 40, 5, 80, 32, 128, BF16),
    (1, 1000, 2, 128, 64, 1024, BF16),
    (2, 300, 3, 496, 128, 384, F32),
]


def write_case(case, seed):
    B, T, Hkv, D, block, cap, dt = case
    rng = random.Random(seed)
    lens = [rng.randint(T, cap) for _ in range(B)]
    lens[0] = cap
    if B > 1:
        lens[1] = 0
    if B > 2:
        lens[2] = max(1, T // 2)                       # padded in front
    if B > 3:
        lens[3] = T                                    # starts an empty cache
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, batch=B, seed=seed, device=G.dev()))
    kv = randn((B, T, 2 * Hkv, D), dt, seed, 1.0)
    # sizes around the cache's own, so that some scales grow and some stay
    kv *= torch.tensor([2.0 ** rng.randint(-8, 6) for _ in range(B * T)], device=G.dev(), dtype=dt).view(B, T, 1, 1)
    return lens, cache, kv[:, :, :Hkv], kv[:, :, Hkv:]


def check_write(cache, before, k, v, lens, block):
    for b, n in enumerate(lens):
        T = k.shape[1]
        for x, c, s, c0, s0 in ((k, cache.k, cache.k_scale, before[0], before[2]),
                                (v, cache.v, cache.v_scale, before[1], before[3])):
            want, ws = R.write(x[b].cpu(), c0[b].cpu(), s0[b].cpu(), n - T, block)
            got = c[b].cpu().double()
            assert torch.equal(torch.isnan(got), torch.isnan(want)), b
            assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0)), b
            assert torch.equal(s[b].cpu().double(), ws), b
            assert torch.equal(c[b, :, max(n, 0):].view(torch.uint8), c0[b, :, max(n, 0):].view(torch.uint8))


@pytest.mark.parametrize("case", WRITE, ids=str)
def test_write(case):
    lens, cache, k, v = write_case(case, 11)
    before = [t.clone() for t in cache]
    d = torch.tensor(lens, device=G.dev())
    assert pkg.cache_write_q8(k, v, cache, lengths=d) is cache
    check_write(cache, before, k, v, lens, case[4])
    once = [t.clone() for t in cache]
    pkg.cache_write_q8(k, v, cache, lengths=d)                     # the same tokens again
    for a, b in zip(once, cache):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_write_values_at_the_edges(dt):
    """Zeros, subnormals, the largest numbers, infinities, NaN, and a block that grows row by row."""
    Hkv, D, block, cap = 2, 16, 16, 32
    rows = [0.0, 2.0 ** -140 if dt == F32 else 2.0 ** -130, 2.0 ** -100, 1.0, 448.0, 448.0 * 2, 449.0 * 4,
            float("inf"), float("nan"), -float("inf"), 1e30, -3e38, 3.0, 0.0]
    cache = pkg.q8_cache(Hkv, cap, D, block=block)
    for i, r in enumerate(rows):
        x = torch.full((1, Hkv, D), r, dtype=dt, device=G.dev())
        x[0, 1] *= 0.37
        x[0, :, ::3] = 0.0
        before = [t.clone()[None] for t in cache]
        pkg.cache_write_q8(x, x, cache, start_pos=i)
        check_write(pkg.Q8Cache(*(t[None] for t in cache)), before, x[None], x[None], [i + 1], block)
    ok()


def test_write_does_not_take_up_a_scale_of_another_occupant():
    """A block written from its first row on starts over; rows behind the new ones stay."""
    cache = pkg.Q8Cache(*R.make_cache(2, 64, 128, 32, seed=1, device=G.dev()))
    cache.k_scale.fill_(2.0 ** 40)
    x = randn((3, 2, 128), BF16, 5)
    before = [t.clone()[None] for t in cache]
    pkg.cache_write_q8(x, x, cache, start_pos=32)
    check_write(pkg.Q8Cache(*(t[None] for t in cache)), before, x[None], x[None], [35], 32)
    assert (cache.k_scale[:, 1] < 1).all() and (cache.k_scale[:, 0] == 2.0 ** 40).all()


def test_write_refuses_lengths_beyond_the_cache_on_the_device():
    cache = pkg.Q8Cache(*R.make_cache(2, 64, 128, 32, batch=3, seed=1, device=G.dev()))
    before = [t.clone() for t in cache]
    x = randn((3, 2, 2, 128), BF16, 5)
    pkg.cache_write_q8(x, x, cache, lengths=torch.tensor([65, -1, 64], device=G.dev()))
    ok(-11)
    for a, b in zip(before, cache):
        assert torch.equal(a[:2].view(torch.uint8), b[:2].view(torch.uint8))
    check_write(cache.__class__(*(t[2:] for t in cache)), [t[2:] for t in before], x[2:], x[2:], [64], 32)
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("shape", [(8, 256, 128, 64), (2, 512, 512, 16), (3, 96, 80, 32), (1, 128, 16, 128)])
def test_read(shape, dt):
    Hkv, cap, D, block = shape
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, seed=3, device=G.dev()))
    for a, b in ((0, cap), (0, 1), (cap - 1, cap), (5, 5), (block - 1, min(cap, block + 2)), (3, cap - 5)):
        k, v = pkg.cache_read_q8(cache, a, b, dtype=dt)
        assert k.dtype == dt and k.shape == (Hkv, b - a, D)
        assert torch.equal(k.double(), R.values(cache.k, cache.k_scale)[:, a:b])
        assert torch.equal(v.double(), R.values(cache.v, cache.v_scale)[:, a:b])
    batch = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, batch=3, seed=4, device=G.dev()))
    k, v = pkg.cache_read_q8(batch, 1, cap, dtype=dt)
    assert torch.equal(k.double(), R.values(batch.k, batch.k_scale)[:, :, 1:])
    assert torch.equal(v.double(), R.values(batch.v, batch.v_scale)[:, :, 1:])
    ok()


# ------------------------------------------------------------------ attention of few tokens

DECODE = [  # B, T, H, Hkv, D, block, cap, window, dtype
    (1, 1, 32, 8, 128, 64, 1024, 0, BF16),
    (1, 1, 4, 1, 128, 16, 4096, 0, BF16),
    (6, 1, 8, 2, 128, 32, 640, 0, BF16),
    (6, 1, 8, 2, 128, 32, 640, 0, F32),
    (5, 3, 8, 2, 128, 16, 320, 100, BF16),
    (5, 3, 8, 2, 128, 16, 320, 100, F32),
    (4, 1, 5, 1, 128, 64, 512, 33, F32),
    (3, 7, 40, 8, 128, 128, 256, 0, BF16),
    (3, 7, 40, 8, 128, 128, 256, 0, F32),
    (2, 1, 128, 1, 128, 64, 512, 0, BF16),
    (2, 2, 128, 1, 128, 64, 512, 1, F32),
    (4, 1, 8, 2, 512, 64, 512, 0, BF16),
    (4, 3, 8, 2, 512, 32, 320, 90, F32),
    (4, 5, 8, 2, 512, 16, 320, 0, BF16),
    (40, 5, 12, 2, 512, 32, 1024, 0, F32),
    (80, 6, 6, 2, 128, 64, 2048, 700, F32),
    (3, 1, 16, 1, 512, 128, 384, 5, F32),
    (2, 20, 16, 2, 128, 64, 320, 0, BF16),
    (40, 1, 2, 2, 128, 16, 96, 0, BF16),
    (3, 1, 6, 2, 128, 64, 20032, 0, BF16),
]


def decode_lens(B, T, cap, seed):
    rng = random.Random(seed)
    lens = [rng.randint(1, cap) for _ in range(B)]
    lens[0] = cap
    for i, n in ((1, 0), (2, max(1, T - 1)), (3, 1), (4, T), (5, cap - 1)):
        if i < B:
            lens[i] = n
    return lens


@pytest.mark.parametrize("case", DECODE, ids=str)
def test_decode(case):
    B, T, H, Hkv, D, block, cap, window, dt = case
    lens = decode_lens(B, T, cap, 7)
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, batch=B, seed=5, device=G.dev(), dead=lens))
    q = randn((B, T, H, D), dt, 6, 2.0)
    d = torch.tensor(lens, device=G.dev())
    out = pkg.decode_attention_q8(q, cache, d, window=window)
    for b, n in enumerate(lens):
        want, tol = R.attention(q[b], cache.slot(b), n, window, R.default_scale(D), dt)
        within(out[b], want, tol, f"sequence {b} of length {n}")
    assert torch.equal(out, pkg.decode_attention_q8(q, cache, d, window=window))
    ok()


def test_decode_masked_rows_may_hold_nan():
    """NaN in front of the window and behind the last key reaches no result."""
    cache = R.make_cache(2, 256, 128, 16, batch=1, seed=5, device=G.dev(), dead=[200])
    k, v, ks, vs = (t.view(torch.uint8) if t.dtype == F8 else t for t in cache)
    k[:, :, :150], v[:, :, :150] = 0x7f, 0xff
    ks[:, :, :150 // 16], vs[:, :, :150 // 16] = float("nan"), float("inf")
    cache = pkg.Q8Cache(k.view(F8), v.view(F8), ks, vs)
    for dt in (BF16, F32):
        q = randn((1, 1, 8, 128), dt, 1)
        out = pkg.decode_attention_q8(q, cache, torch.tensor([200], device=G.dev()), window=50)
        live = pkg.Q8Cache(cache.k[0], cache.v[0], cache.k_scale[0].nan_to_num(0.0),
                           cache.v_scale[0].nan_to_num(0.0, 0.0))
        want, tol = R.attention(q[0], live, 200, 50, R.default_scale(128), dt)
        within(out[0], want, tol)
    # a visible NaN is not hidden
    out = pkg.decode_attention_q8(q, cache, torch.tensor([200], device=G.dev()), window=51)
    assert torch.isnan(out).all()
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D", [128, 512])
def test_decode_extremes(D, dt):
    """Large and tiny queries, scales far apart between blocks, blocks of zeros, a negative and a zero scale."""
    Hkv, H, cap, block = 2, 8, 256, 16
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, batch=1, seed=8, device=G.dev()))
    e = torch.tensor([(-20, 0, -3, -9)[i % 4] for i in range(cap // block)], device=G.dev())
    cache.v_scale.copy_(torch.ldexp(torch.ones_like(cache.v_scale), e.expand_as(cache.v_scale)))
    cache.k_scale[:, :, 2] = 0.0
    cache.v_scale[:, :, 5] = 0.0
    d = torch.tensor([cap - 3], device=G.dev())
    for std, scale in ((2.0 ** -20, 2.0 ** 16), (2.0 ** 20, 2.0 ** -26), (1.0, 0.0), (1.0, -0.05)):
        q = randn((1, 1, H, D), dt, 9, std)
        q[0, 0, 1] = 0.0
        q[0, 0, 2, 1:] = 0.0
        out = pkg.decode_attention_q8(q, cache, d, scale=scale)
        want, tol = R.attention(q[0], cache.slot(0), cap - 3, 0, scale, dt)
        within(out[0], want, tol, f"std {std} scale {scale}")
    ok()


@pytest.mark.parametrize("D,dt", [(128, BF16), (128, F32), (512, BF16)])
def test_the_widest_window_is_none(D, dt):
    cache = R.make_cache(2, 256, D, 64, batch=3, seed=5, device=G.dev(), dead=[200, 2, 0])
    cache = pkg.Q8Cache(*cache)
    q = randn((3, 4, 8, D), dt, 6)
    d = torch.tensor([200, 2, 0], device=G.dev())
    want = pkg.decode_attention_q8(q, cache, d)
    for w in (256, 257, 2 ** 31 - 1):
        assert torch.equal(want, pkg.decode_attention_q8(q, cache, d, window=w))
    with pytest.raises(ValueError):
        pkg.decode_attention_q8(q, cache, d, window=2 ** 31)
    for T in (3, 50, 190):                     # decode kernel, codes (bf16, 128), read back
        x = randn((T, 8, D), dt, T)
        want = pkg.prefill_attention_q8(x, cache.slot(0), start_pos=200 - T)
        for w in (200, 2 ** 31 - 1):
            assert torch.equal(want, pkg.prefill_attention_q8(x, cache.slot(0), start_pos=200 - T, window=w))
    ok()


def test_decode_reads_a_cache_of_more_than_four_gigabytes():
    B, Hkv, cap, D, block = 5, 8, 1 << 20, 128, 64
    cache = pkg.q8_cache(Hkv, cap, D, batch=B, block=block)
    lens = [3, 70, 1, 0, 130]
    x = randn((1, 130, Hkv, D), BF16, 3)
    for b in (1, 4):
        pkg.cache_write_q8(x[0, :lens[b]], x[0, :lens[b]], cache.slot(b), start_pos=0)
    last = cache.slot(4)
    pkg.cache_write_q8(x[0], x[0], last, start_pos=cap - 130)
    k, _ = pkg.cache_read_q8(last, cap - 130, cap)
    assert (k.transpose(0, 1).float() - x[0].float()).abs().max() <= x.abs().max().item() * 2.0 ** -4
    q = randn((B, 1, 16, D), BF16, 4)
    d = torch.tensor(lens, device=G.dev())
    out = pkg.decode_attention_q8(q, cache, d)
    for b, n in enumerate(lens):
        part = pkg.Q8Cache(*(t[b, :, :192] for t in (cache.k, cache.v)),
                           *(t[b, :, :3] for t in (cache.k_scale, cache.v_scale)))
        want, tol = R.attention(q[b], part, n, 0, R.default_scale(D), BF16)
        within(out[b], want, tol, f"sequence {b}")
    out = pkg.decode_attention_q8(q[4:], pkg.Q8Cache(*(t[4:] for t in cache)),
                                  torch.tensor([cap], device=G.dev()), window=120)
    part = pkg.Q8Cache(*(t[4, :, cap - 192:] for t in (cache.k, cache.v)),
                       *(t[4, :, -3:] for t in (cache.k_scale, cache.v_scale)))
    want, tol = R.attention(q[4], part, 192, 120, R.default_scale(D), BF16)
    within(out[0], want, tol, "at the end of the cache")
    ok()


def test_decode_strided_rows_and_given_output():
    B, T, H, Hkv, D = 3, 2, 8, 2, 128
    cache = pkg.Q8Cache(*R.make_cache(Hkv, 128, D, 64, batch=B, seed=5, device=G.dev()))
    buf = randn((B, T, H + 3, D), BF16, 6)
    q = buf[:, :, 1:H + 1]
    dst = torch.full((B, T, H + 1, D), 3.0, dtype=BF16, device=G.dev())
    d = torch.tensor([128, 100, 1], device=G.dev())
    out = pkg.decode_attention_q8(q, cache, d, out=dst[:, :, :H])
    assert out.data_ptr() == dst.data_ptr()
    assert torch.equal(out, pkg.decode_attention_q8(q.contiguous(), cache, d))
    assert (dst[:, :, H:] == 3).all()
    ok()


def test_decode_lengths_are_checked_on_the_device():
    cache = pkg.Q8Cache(*R.make_cache(2, 128, 128, 64, batch=3, seed=5, device=G.dev()))
    q = randn((3, 1, 8, 128), BF16, 6)
    out = torch.full_like(q, 3.0)
    pkg.decode_attention_q8(q, cache, torch.tensor([129, 128, -1], device=G.dev()), out=out)
    ok(-11)
    assert (out[0] == 3).all() and (out[2] == 3).all()
    want, tol = R.attention(q[1], cache.slot(1), 128, 0, R.default_scale(128), BF16)
    within(out[1], want, tol)
    ok()


def test_decode_workspace():
    B, T, H, Hkv, D = 2, 1, 8, 2, 128
    cache = pkg.Q8Cache(*R.make_cache(Hkv, 4096, D, 64, batch=B, seed=5, device=G.dev()))
    q = randn((B, T, H, D), BF16, 6)
    d = torch.tensor([4096, 77], device=G.dev())
    want = pkg.decode_attention_q8(q, cache, d)
    n = pkg.decode_workspace_bytes_q8(B, T, H, Hkv, D)
    ws = torch.full((max(n, 1) + 256,), 0xff, dtype=torch.uint8, device=G.dev())    # NaN all over
    assert torch.equal(want, pkg.decode_attention_q8(q, cache, d, workspace=ws[:n]))
    assert (ws[n:] == 0xff).all()
    if n:
        for bad in (None, ws[:n - 1]):
            with pytest.raises(pkg.PfaError) as e:
                pkg.decode_attention_q8(q, cache, d, workspace=bad)
            assert e.value.name == "PFA_ERR_SCRATCH"
    ok()


def test_decode_of_more_sequences_than_one_launch_lists():
    """17000 short sequences (two launches), against 64 bits all at once."""
    B, H, D, cap = 17000, 2, 128, 16
    cache = pkg.Q8Cache(*R.make_cache(1, cap, D, 16, batch=B, seed=2, device=G.dev()))
    q = randn((B, 1, H, D), BF16, 3, 2.0)
    n = torch.randint(0, cap + 1, (B,), generator=torch.Generator().manual_seed(4)).to(G.dev())
    out = pkg.decode_attention_q8(q, cache, n)
    k, v = R.values(cache.k, cache.k_scale)[:, 0], R.values(cache.v, cache.v_scale)[:, 0]
    s = (q[:, 0].double() @ k.transpose(1, 2)) * R.default_scale(D)
    hidden = torch.arange(cap, device=G.dev()) >= n[:, None, None]
    p = torch.softmax(s.masked_fill(hidden, float("-inf")), -1).nan_to_num(0.0)
    want, a = p @ v, p @ v.abs()
    # half a step, the weights' 2^-11 (see attention()), scores of up to a few hundred off by
    # 10 * 2^-22 of their terms
    size = (q[:, 0].double().abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * R.default_scale(D)
    within(out[:, 0], want, 2.0 ** -8 * want.abs() + a * (2.0 ** -11 + 2.0 ** -20 + 2 * size * 10 * 2.0 ** -22)
           + 2.0 ** -39 * 30 * 16 * cache.v_scale.max().item())
    ok()


@pytest.mark.parametrize("case", [
    (7, 12, 8, 2, 128, 64, 4096, 0, BF16),     # 3 tiles of 16 rows
    (6, 52, 4, 1, 128, 32, 1024, 200, BF16),   # 13
    (6, 9, 20, 2, 512, 16, 512, 0, BF16),      # 6
    (3, 128, 16, 2, 128, 64, 512, 0, BF16),    # 64
    (5, 35, 8, 4, 128, 128, 1024, 0, F32),     # 5, the last of 6 rows
], ids=str)
def test_decode_of_several_row_tiles(case):
    test_decode(case)


# ------------------------------------------------------------------ chunks

def test_prefill_of_more_row_tiles_than_one_launch_lists():
    T, H, D = 2100, 128, 512                              # 16800 tiles of 16 rows
    cache = pkg.Q8Cache(*R.make_cache(1, 2176, D, 64, seed=3, device=G.dev(), dead=[T]))
    q = randn((T, H, D), F32, 4, 1.0)
    out = pkg.prefill_attention_q8(q, cache, start_pos=0)
    heads = [0, 77, 127]
    want, tol = R.attention(q[:, heads], cache, T, 0, R.default_scale(D), F32)
    within(out[:, heads], want, tol)
    ok()


@pytest.mark.parametrize("T", [8, 60, 300])
def test_prefill_in_a_graph(T):
    H, Hkv, D, cap = 8, 2, 128, 1024                      # decode kernel, codes, read back
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, 64, seed=3, device=G.dev()))
    q = randn((T, H, D), BF16, 1)
    want = pkg.prefill_attention_q8(q, cache, start_pos=cap - T).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkg.prefill_attention_q8(q, cache, start_pos=cap - T)
    q2 = randn((T, H, D), BF16, 2)
    for x in (q2, q.clone()):
        q.copy_(x)
        graph.replay()
    ok()
    assert torch.equal(out, want)


def test_prefill_from_the_codes_reports_a_wait_that_runs_out():
    H, Hkv, D, cap, T = 8, 2, 128, 1024, 60
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, 64, seed=3, device=G.dev()))
    q = randn((T, H, D), BF16, 1)
    want = pkg.prefill_attention_q8(q, cache, start_pos=cap - T)
    ok()
    pkg.debug_configure(wait_limit_ms=50.0, force_timeout=True)
    try:
        pkg.prefill_attention_q8(q, cache, start_pos=cap - T)
        status = pkg.last_device_error()
    finally:
        pkg.debug_configure(0.0, False)
    assert status == -7, pkg.status_string(status)
    assert torch.equal(want, pkg.prefill_attention_q8(q, cache, start_pos=cap - T))
    ok()


PREFILL = [  # T, start_pos, H, Hkv, block, window, scale: chunks from the codes
    (14, 0, 8, 2, 16, 0, None), (40, 3000, 8, 2, 16, 0, None), (33, 2999, 12, 2, 32, 130, None),
    (50, 700, 5, 1, 128, 0, None), (2, 900, 128, 1, 64, 0, None), (64, 0, 6, 2, 64, 20, None),
    (50, 1000, 8, 2, 64, 0, -0.07), (50, 1000, 8, 2, 64, 0, 0.0), (17, 40000, 8, 2, 64, 0, None),
    # one pair of tiles sees one key tile, the other two: no part without keys
    (5, 124, 48, 1, 64, 0, None), (5, 252, 48, 1, 64, 100, None),
    (190, 20000, 32, 8, 64, 0, None), (2, 500, 100, 1, 16, 7, None),
]


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill_from_the_codes(case):
    T, sp, H, Hkv, block, window, scale = case
    n, D = sp + T, 128
    cap = -(-n // block) * block + block
    cache = R.make_cache(Hkv, cap, D, block, seed=T, device=G.dev(), dead=[n])
    k, v, ks, vs = (t.view(torch.uint8) if t.dtype == F8 else t for t in cache)
    lo = max(0, sp - window + 1) if window else 0
    k[:, :lo], v[:, :lo] = 0x7f, 0xff                     # NaN in front of every window
    cache = pkg.Q8Cache(k.view(F8), v.view(F8), ks, vs)
    q = randn((T, H, D), BF16, T + 1, 2.0)
    out = pkg.prefill_attention_q8(q, cache, start_pos=sp, window=window, scale=scale)
    live = pkg.Q8Cache(*(t.view(torch.uint8).clone().view(F8) for t in (k, v)), ks, vs)
    for t in (live.k, live.v):
        t.view(torch.uint8)[:, :lo] = 0
    want, tol = R.attention(q, live, n, window, R.default_scale(D) if scale is None else scale, BF16)
    # beside attention()'s terms: weights up to 2^8 where the exponent's base lags, so small ones
    # round to 2^-25 of a weight of 1, times the largest V
    vmax = R.values(live.v, vs)[:, lo:n].abs().nan_to_num(0.0).amax().item()
    within(out, want, tol + (n - lo) * 2.0 ** -25 * vmax, f"T {T}")
    assert torch.equal(out, pkg.prefill_attention_q8(q, cache, start_pos=sp, window=window, scale=scale))
    ok()

@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D", [128, 512])
@pytest.mark.parametrize("T,sp,window", [(1, 0, 0), (1, 300, 0), (5, 123, 40), (16, 0, 0), (17, 200, 0),
                                         (64, 33, 0), (130, 500, 0), (130, 500, 77), (300, 0, 256)])
def test_prefill(T, sp, window, D, dt):
    Hkv, H, block = 2, 8, 32
    n = sp + T
    cap = -(-n // block) * block + block
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, block, seed=T, device=G.dev(), dead=[n]))
    q = randn((T, H + 2, D), dt, T, 2.0)[:, :H]
    out = pkg.prefill_attention_q8(q, cache, start_pos=sp, window=window)
    assert out.stride() == q.stride() or T == 1
    want, tol = R.attention(q, cache, n, window, R.default_scale(D), dt)
    # where bf16 rows are read back, the weights are rounded as prefill_attention rounds them: 2^-8
    v = R.values(cache.v, cache.v_scale)[:, :n].abs().amax().item()
    within(out, want, tol + (v * 2.0 ** -8 if dt == BF16 else 0.0), f"T {T}")
    ok()


def test_fp32_over_many_keys_is_fp32():
    """A tensor core's sum truncates: over 30000 keys in one run the bias must not show.

    Plain fp32 sums of n terms of random sign are off by some 2^-24 sqrt(log2 n) of their
    root mean square; this asks for 2^-20 of the outputs' (a 2-norm), 16 roundings."""
    cap, Hkv, H, D = 30016, 1, 8, 128
    cache = pkg.Q8Cache(*R.make_cache(Hkv, cap, D, 64, batch=1, seed=3, device=G.dev()))
    q = randn((1, 100, H, D), F32, 4, 0.02)                # flat weights: every key counts
    d = torch.tensor([cap], device=G.dev())
    out = pkg.decode_attention_q8(q, cache, d)
    want, _ = R.attention(q[0], cache.slot(0), cap, 0, R.default_scale(D), F32)
    assert (out[0].double() - want).norm() <= 2.0 ** -20 * want.norm()
    assert torch.equal(out[0], pkg.prefill_attention_q8(q[0], cache.slot(0), start_pos=cap - 100))
    ok()


def test_prefill_on_read_back_rows_is_prefill_attention():
    T, sp, H, Hkv, D = 300, 701, 8, 2, 512
    cache = pkg.Q8Cache(*R.make_cache(Hkv, 1024, D, 64, seed=3, device=G.dev(), dead=[sp + T]))
    q = randn((T, H, D), BF16, 1)
    k, v = pkg.cache_read_q8(cache, 0, sp + T)
    for w in (0, 200):
        lo = max(0, sp - w + 1) if w else 0
        want = pkg.prefill_attention(q, k[:, lo:].contiguous(), v[:, lo:].contiguous(), window=w)
        assert torch.equal(want, pkg.prefill_attention_q8(q, cache, start_pos=sp, window=w))
    n = pkg.prefill_workspace_bytes_q8(T, sp, H, Hkv, D)
    ws = torch.full((n + 256,), 0xff, dtype=torch.uint8, device=G.dev())
    assert torch.equal(pkg.prefill_attention(q, k, v),
                       pkg.prefill_attention_q8(q, cache, start_pos=sp, workspace=ws[:n]))
    assert (ws[n:] == 0xff).all()
    for bad in (None, ws[:n - 1]):
        with pytest.raises(pkg.PfaError):
            pkg.prefill_attention_q8(q, cache, start_pos=sp, workspace=bad)
    ok()


# ------------------------------------------------------------------ together

def _layer(B, H, Hkv, D, cap, block, dt):
    """Weights and an empty cache of one layer, and a step on them."""
    w = [randn((D,), dt, s, 0.2) for s in (1, 2)]
    freq = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=G.dev()) / (D // 2))
    cache = pkg.q8_cache(Hkv, cap, D, batch=B, block=block)

    def step(qkv, lengths, window=0, stream=None):
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        q, k = pkg.qk_norm_rope(q, k, *w, freq, lengths=lengths, weight_offset=1.0, stream=stream)
        pkg.cache_write_q8(k, v, cache, lengths=lengths, stream=stream)
        return q, k, pkg.decode_attention_q8(q, cache, lengths, window=window, stream=stream)
    return cache, step, w, freq


@pytest.mark.parametrize("D,dt", [(128, BF16), (128, F32), (512, BF16)])
def test_steps_of_a_layer_in_a_graph(D, dt):
    """Decode steps of a batch, captured once and replayed, against 64 bits on the tokens themselves."""
    B, T, H, Hkv, cap, block = 4, 2, 8, 2, 192, 32
    cache, step, w, freq = _layer(B, H, Hkv, D, cap, block, dt)
    qkv = randn((B, T, H + 2 * Hkv, D), dt, 1)
    lens = torch.tensor([0, T, 60, 100], device=G.dev())
    # the sequences' first tokens, as chunks
    for b in (2, 3):
        x = randn((int(lens[b]), 2 * Hkv, D), dt, 10 + b)
        pkg.cache_write_q8(x[:, :Hkv], x[:, Hkv:], cache.slot(b), start_pos=0)
    start = [t.clone() for t in cache]
    step(qkv, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(qkv, lens)
    for t, s in zip(cache, start):
        t.copy_(s)
    for i in range(6):
        qkv.copy_(randn(qkv.shape, dt, 100 + i))
        lens.copy_(torch.tensor([0, T * (i + 1), 60 + T * (i + 1), 100 + T * (i + 1)]))
        before = [t.clone() for t in cache]
        graph.replay()
        ok()
        n = lens.tolist()
        check_write(cache, before, got[1], qkv[:, :, H + Hkv:], n, block)
        for b in range(B):
            pos = torch.arange(n[b] - T, n[b])
            y, size = R.norm_rope(qkv[b, :, :H], w[0], 1.0, 1e-6, freq, pos, False)
            if n[b]:
                within(got[0][b], y, norm_tol(y, size, dt))
            want, tol = R.attention(got[0][b], cache.slot(b), n[b], 0, R.default_scale(D), dt)
            within(got[2][b], want, tol, f"step {i} sequence {b}")


def test_a_prompt_in_chunks_then_tokens():
    """norm + rotation, write, chunk attention for a prompt, then single tokens: all against 64 bits."""
    H, Hkv, D, block, cap, dt = 8, 2, 128, 64, 512, BF16
    cache, step, w, freq = _layer(1, H, Hkv, D, cap, block, dt)
    slot = cache.slot(0)
    sp = 0
    for T in (100, 1, 37, 190, 3):
        qkv = randn((T, H + 2 * Hkv, D), dt, sp)
        q, k = pkg.qk_norm_rope(qkv[:, :H], qkv[:, H:H + Hkv], *w, freq, start_pos=sp, weight_offset=1.0)
        pkg.cache_write_q8(k, qkv[:, H + Hkv:], slot, start_pos=sp)
        sp += T
        out = pkg.prefill_attention_q8(q, slot, start_pos=sp - T)
        want, tol = R.attention(q, slot, sp, 0, R.default_scale(D), dt)
        v = R.values(slot.v, slot.v_scale)[:, :sp].abs().amax().item()
        within(out, want, tol + v * 2.0 ** -8, f"chunk to {sp}")
    for _ in range(4):
        sp += 1
        qkv = randn((1, 1, H + 2 * Hkv, D), dt, sp)
        q, k, out = step(qkv, torch.tensor([sp], device=G.dev()))
        want, tol = R.attention(q[0], slot, sp, 0, R.default_scale(D), dt)
        within(out[0], want, tol, f"token {sp - 1}")
        # the two forms of a single token's attention are one
        assert torch.equal(out[0], pkg.prefill_attention_q8(q[0], slot, start_pos=sp - 1))
    ok()


def test_other_streams_and_two_calls_at_once():
    B, H, Hkv, D, cap, block = 3, 8, 2, 128, 4096, 64
    layers = [_layer(B, H, Hkv, D, cap, block, BF16) for _ in range(2)]
    lens = torch.tensor([4096, 3000, 17], device=G.dev())
    for i, (cache, *_) in enumerate(layers):
        for t, s in zip(cache, R.make_cache(Hkv, cap, D, block, batch=B, seed=i, device=G.dev())):
            t.copy_(s)
    qkv = [randn((B, 1, H + 2 * Hkv, D), BF16, i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(layers[i][1](qkv[i], lens, stream=streams[i])[2])
    torch.cuda.synchronize()
    for i in range(2):
        want = layers[i][1](qkv[i], lens)[2]
        for g in got[i]:
            assert torch.equal(g, want)
        for b in range(B):
            q = layers[i][1](qkv[i], lens)[0]
            ref, tol = R.attention(q[b], layers[i][0].slot(b), int(lens[b]), 0, R.default_scale(D), BF16)
            within(want[b], ref, tol)
    ok()


def test_empty_calls():
    cache = pkg.q8_cache(2, 64, 128, batch=2)
    slot = cache.slot(0)
    none = torch.zeros(2, 0, 8, 128, dtype=BF16, device=G.dev())
    d = torch.zeros(2, dtype=torch.int64, device=G.dev())
    assert pkg.decode_attention_q8(none, cache, d).shape == none.shape
    q, k = pkg.qk_norm_rope(none, none[:, :, :2], lengths=d)
    pkg.cache_write_q8(k, k, cache, lengths=d)
    assert pkg.prefill_attention_q8(none[0], slot, start_pos=5).shape == (0, 8, 128)
    assert pkg.cache_read_q8(slot, 7, 7)[0].shape == (2, 0, 128)
    one = torch.ones(2, 1, 8, 128, dtype=BF16, device=G.dev())
    assert (pkg.decode_attention_q8(one, cache, d) == 0).all()      # empty slots
    ok()
