"""The operators around the 4-bit cache on the GPU, against the plain 64-bit
forms of q4_reference.py: sizes, masks, strides, streams and graphs."""
import random

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q4_reference as R
from tests import q8_reference as R8

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


def raw(cache):
    return [t.view(torch.uint8).clone() for t in cache[:4]]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a[:4], b[:4]))


def lengths(ns):
    return torch.tensor(ns, dtype=torch.int64, device=G.dev())


# ------------------------------------------------------------------ write and read back

WRITE = [  # B, T, Hkv, D, cap, dtype
    (1, 1, 8, 128, 128, BF16),
    (6, 1, 2, 128, 64, F32),
    (4, 3, 3, 128, 97, BF16),
    (5, 70, 2, 512, 251, BF16),
    (2, 129, 1, 512, 256, F32),
    (3, 5, 2, 16, 48, F32),
    (2, 40, 5, 80, 128, BF16),
    (1, 1000, 2, 128, 1024, BF16),
    (2, 300, 3, 496, 383, F32),
]


@pytest.mark.parametrize("case", WRITE, ids=str)
@pytest.mark.parametrize("exps", [(0, 0), (3, -5)], ids=str)
def test_write(case, exps):
    B, T, Hkv, D, cap, dt = case
    rng = random.Random(7)
    lens = [rng.randint(T, cap) for _ in range(B)]
    lens[0] = cap
    if B > 1:
        lens[1] = 0
    if B > 2:
        lens[2] = max(1, T // 2)                       # padded in front
    if B > 3:
        lens[3] = T                                    # starts an empty cache
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=B, seed=3, device=G.dev()), *exps)
    kv = randn((B, T, 2 * Hkv, D), dt, 5)              # columns of one buffer
    kv *= torch.tensor([2.0 ** rng.randint(-8, 6) for _ in range(B * T)], device=G.dev(), dtype=dt).view(B, T, 1, 1)
    k, v = kv[:, :, :Hkv], kv[:, :, Hkv:]
    want = raw(cache)
    assert pkg.cache_write_q4(k, v, cache, lengths=lengths(lens)) is cache
    for x, c, s, e in ((k, 0, 2, exps[0]), (v, 1, 3, exps[1])):
        codes, scale = R.quantise(x, e)
        for b, n in enumerate(lens):
            lo = max(0, n - T)
            want[c][b, :, lo:n] = codes[b, T - (n - lo):].transpose(0, 1)
            want[s][b, :, lo:n] = scale[b, T - (n - lo):].transpose(0, 1)
    assert same(cache, want)
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("e", [0, 7, -64, 64])
def test_write_one_sequence_at_the_edges(dt, e):
    """Zeros of both signs, subnormals, the largest numbers, infinities, NaN, and every border between two codes."""
    D, Hkv, cap = 64, 2, 80
    ties = [0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, -0.0]
    rows = [[t * s for t in ties] for s in (1.0, 1.125, 1.875, 2.0 ** -9, 3 * 2.0 ** -9, 448.0, 2.0 ** -6)]
    # the largest of a group on a border between two scales, and beside it
    rows += [[6 * s * (1 + i * d) for d in (0, 2.0 ** -7, -2.0 ** -8)] + [0.0] * 13
             for i in (0, 1) for s in (1.0625, 1.1875, 17 * 2.0 ** -10, 2.0 ** -10, 432.0, 464.0, 480.0)]
    rows += [[x] + [1.0] * 15 for x in (0.0, -0.0, 1e-40, 2.0 ** -126, 1e30, -3e38, float("inf"), -float("inf"),
                                        float("nan"), 2700.0)]
    rows += [[0.0] * 16, [-0.0] * 16, [1e-30] * 16, [-2.0 ** -11] * 16]
    x = torch.tensor(rows, dtype=torch.float64)
    fin = torch.isfinite(x) & (x.abs() < 1e29) & (x.abs() > 1e-29)
    x = torch.where(fin, x * 2.0 ** e, x).to(dt)
    x = torch.cat((x, x.flip(0), -x, x), 0)[:4 * (len(rows) // 4) * 4]
    x = x.reshape(-1, 1, D).expand(-1, Hkv, D).contiguous().to(G.dev())
    cache = pkg.q4_cache(Hkv, cap, D, k_exponent=e, v_exponent=e)
    T = x.shape[0]
    assert T + 3 <= cap
    pkg.cache_write_q4(x, x, cache, start_pos=3)
    codes, scale = R.quantise(x, e)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert torch.equal(s.view(torch.uint8)[:, 3:3 + T], scale.transpose(0, 1))
        assert torch.equal(c[:, 3:3 + T], codes.transpose(0, 1))
        assert not c[:, :3].any() and not c[:, 3 + T:].any()
    k, v = pkg.cache_read_q4(cache, 3, 3 + T, dtype=F32)
    if abs(e) < 64:                                    # beyond fp32's range otherwise
        want = R.values(codes, scale.view(F8), e).transpose(0, 1)
        assert torch.equal(k.double().nan_to_num(1.25), want.nan_to_num(1.25)) and torch.equal(k.isnan(), v.isnan())
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_write_beside_every_border(dt):
    """For every scale the floats on and beside each border between two codes, of both signs, and a wide mixture."""
    s = torch.arange(1, 127, dtype=torch.uint8).view(F8).double()
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64)
    near = [(s[:, None] * t).float()]
    up = down = near[0]
    for _ in range(4):
        up, down = torch.nextafter(up, torch.tensor(1e30)), torch.nextafter(down, torch.tensor(0.0))
        near += [up, down]
    v = torch.nn.functional.pad(torch.stack(near, -1).reshape(126, -1), (0, 12)).reshape(126, 5, 15)
    v = torch.cat((v, 6 * s.float()[:, None, None].expand(126, 5, 1)), -1).reshape(-1, 16)
    g = torch.Generator().manual_seed(1)
    mix = torch.randn(40000, 16, generator=g) * (3 * torch.randn(40000, 1, generator=g)).exp()
    x = torch.cat((v, -v, mix)).to(dt).to(G.dev())
    x = x[:x.shape[0] // 8 * 8].reshape(-1, 1, 128)
    cache = pkg.q4_cache(1, x.shape[0], 128)
    pkg.cache_write_q4(x, x, cache, start_pos=0)
    codes, scale = R.quantise(x, 0)
    assert torch.equal(cache.k_scale.view(torch.uint8)[0], scale[:, 0]) and torch.equal(cache.k[0], codes[:, 0])
    ok()


def test_write_refuses_lengths_beyond_the_cache_on_the_device():
    cache = pkg.Q4Cache(*R.make_cache(2, 64, 128, batch=3, seed=1, device=G.dev()))
    before = raw(cache)
    x = randn((3, 2, 2, 128), BF16, 1)
    pkg.cache_write_q4(x, x, cache, lengths=lengths([65, -1, 64]))
    after = raw(cache)
    assert all(torch.equal(a[:2], b[:2]) and not torch.equal(a[2], b[2]) for a, b in zip(after, before))
    ok(-11)
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("D", [16, 80, 128, 512])
def test_read(D, dt):
    cap, Hkv = 77, 3
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=2, seed=4, device=G.dev()), -3, 5)
    scale = torch.arange(cache.k_scale.numel(), dtype=torch.int64).remainder(127).to(torch.uint8)
    cache.k_scale.view(torch.uint8).copy_(scale.view(cache.k_scale.shape))      # every scale
    for a, z in ((0, cap), (5, 6), (13, 76), (77, 77)):
        k, v = pkg.cache_read_q4(cache, a, z, dtype=dt)
        assert k.shape == (2, Hkv, z - a, D) and k.dtype == dt
        assert torch.equal(k.double(), R.values(cache.k, cache.k_scale, -3)[:, :, a:z])
        assert torch.equal(v.double(), R.values(cache.v, cache.v_scale, 5)[:, :, a:z])
    one = cache.slot(1)
    ko, vo = (torch.empty(Hkv, 10, D, dtype=dt, device=G.dev()) for _ in "kv")
    k, v = pkg.cache_read_q4(one, 60, 70, dtype=dt, k_out=ko, v_out=vo)
    assert k is ko and v is vo and torch.equal(ko.double(), R.values(one.k, one.k_scale, -3)[:, 60:70])
    one.v_scale.view(torch.uint8)[0, 61, 0] = 0x7f
    v = pkg.cache_read_q4(one, 60, 70, dtype=dt)[1]
    assert v[0, 1, :16].isnan().all() and v.isnan().sum() == 16
    ok()


# ------------------------------------------------------------------ attention

DECODE = [  # lens, T, H, Hkv, D, window, cap, dtype
    ([1], 1, 1, 1, 128, 0, 1, BF16),
    ([37], 1, 4, 1, 128, 0, 64, F32),
    ([1, 31, 32, 33, 0, 64, 200], 1, 32, 8, 128, 0, 257, BF16),
    ([200, 3, 0, 65, 2], 4, 10, 2, 128, 0, 200, BF16),
    ([200, 3, 0, 65, 2], 4, 10, 2, 128, 0, 200, F32),
    ([300, 299, 5], 3, 8, 2, 128, 33, 333, BF16),
    ([300, 299, 5], 3, 8, 2, 128, 33, 333, F32),
    ([1000, 40, 0], 1, 8, 1, 512, 0, 1024, BF16),
    ([500, 40, 0, 7], 5, 8, 2, 512, 100, 512, F32),
    ([130, 131], 16, 8, 8, 128, 0, 160, BF16),
    ([90], 32, 32, 8, 128, 0, 128, BF16),
    ([90, 20], 40, 6, 2, 128, 7, 128, F32),
    ([700], 8, 128, 1, 128, 0, 700, BF16),
    ([5000], 1, 16, 2, 128, 1, 5001, BF16),
    ([4097, 1], 2, 7, 7, 512, 0, 4100, BF16),
    ([2500], 1, 5, 1, 128, 0, 2501, F32),
    ([33, 64, 96, 17] * 20, 1, 4, 2, 128, 0, 100, BF16),
    ([9000, 10], 3, 40, 8, 128, 4000, 9001, BF16),
]


def attention_case(case, seed, exps=(0, 0)):
    lens, T, H, Hkv, D, window, cap, dt = case
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=len(lens), seed=seed, device=G.dev(), dead=lens), *exps)
    q = randn((len(lens), T, H, D), dt, seed + 1, 2.0 ** -exps[0])
    k = R.values(cache.k, cache.k_scale, exps[0])
    v = R.values(cache.v, cache.v_scale, exps[1])
    return cache, q, k, v


def check_attention(out, weights, w0, q, k, v, case, scale=None):
    lens, T, H, Hkv, D, window, cap, dt = case
    scale = R8.default_scale(D) if scale is None else scale
    for b, n in enumerate(lens):
        want, tol, acc, acc_tol = R.attention(q[b], k[b], v[b], n, window, scale, dt)
        within(out[b], want, tol, f"sequence {b} of {n}")
        if weights is not None:
            total = w0[b].double() + acc
            within(weights[b], total, acc_tol + 2.0 ** -24 * total, f"weights of sequence {b} of {n}")
            seen = torch.zeros(cap, dtype=torch.bool, device=out.device)
            seen[max(0, max(0, n - T) - window + 1) if window > 0 else 0:n] = True
            assert torch.equal(weights[b][:, ~seen], w0[b][:, ~seen])


@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"B{len(c[0])}x{c[0][0]}-T{c[1]}-{c[2]}/{c[3]}x{c[4]}-w{c[5]}-{str(c[7])[6:]}")
@pytest.mark.parametrize("with_weights", [False, True])
def test_decode(case, with_weights):
    lens, T, H, Hkv, D, window, cap, dt = case
    cache, q, k, v = attention_case(case, 21)
    before = raw(cache)
    w = w0 = None
    if with_weights:
        w0 = randn((len(lens), Hkv, cap), F32, 3).abs()
        w = w0.clone()
    out = pkg.decode_attention_q4(q, cache, lengths(lens), weights=w, window=window)
    check_attention(out, w, w0, q, k, v, case)
    assert same(cache, before)
    again = None if w is None else w0.clone()
    assert torch.equal(pkg.decode_attention_q4(q, cache, lengths(lens), weights=again, window=window), out)
    if w is not None:
        assert torch.equal(w, again)
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("exps", [(4, -7), (-60, 60), (64, -64)], ids=str)
def test_decode_exponents(dt, exps):
    case = ([100, 7], 2, 8, 2, 128, 0, 128, dt)
    cache, q, k, v = attention_case(case, 5, exps)
    w = torch.zeros(2, 2, 128, device=G.dev())
    out = pkg.decode_attention_q4(q, cache, lengths(case[0]), weights=w)
    check_attention(out, w, torch.zeros_like(w), q, k, v, case)
    ok()


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 6.0])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_decode_scales_and_strides(scale, dt):
    """Columns of a wider buffer in and out; scores that put all weight on one key."""
    case = ([150, 0, 64], 3, 6, 2, 128, 0, 160, dt)
    cache, q, k, v = attention_case(case, 8)
    wide = torch.full((3, 3, 10, 128), 7.0, dtype=dt, device=G.dev())
    wide[:, :, 2:8] = q
    to = torch.full((3, 3, 9, 128), 5.0, dtype=dt, device=G.dev())
    out = pkg.decode_attention_q4(wide[:, :, 2:8], cache, lengths(case[0]), to[:, :, 1:7], scale=scale)
    assert out.data_ptr() == to[:, :, 1:7].data_ptr()
    check_attention(out, None, None, q, k, v, case, scale)
    assert (to[:, :, :1] == 5).all() and (to[:, :, 7:] == 5).all()
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_decode_one_heavy_key_and_a_tail(dt):
    """Keys that grow along the sequence (the running maximum rises late), then one far above the rest whose V is 0."""
    Hkv, D, cap, n = 1, 128, 512, 500
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=1, seed=2, device=G.dev()))
    cache.k.fill_(0x22)                                     # ones
    ramp = torch.arange(cap, device=G.dev()) // 8 + 8       # scales rise with the row
    cache.k_scale.view(torch.uint8)[0, 0] = ramp[:, None].to(torch.uint8)
    cache.k_scale.view(torch.uint8)[0, 0, 77] = 0x58        # 16 where the largest of the others is 2
    cache.v_scale.view(torch.uint8)[0, 0, 77] = 0
    q = torch.full((1, 1, 4, D), 0.5, dtype=dt, device=G.dev())
    q[0, 0, 1] *= 0.03
    q[0, 0, 2] = 0
    q[0, 0, 3] *= -1
    case = ([n], 1, 4, Hkv, D, 0, cap, dt)
    w = torch.zeros(1, 1, cap, device=G.dev())
    out = pkg.decode_attention_q4(q, cache, lengths([n]), weights=w, scale=0.25)
    check_attention(out, w, torch.zeros_like(w), q, R.values(cache.k, cache.k_scale), R.values(cache.v, cache.v_scale),
                    case, 0.25)
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_decode_rows_that_are_not_finite_leave_the_others_right(dt, what):
    case = ([700, 130], 2, 8, 2, 128, 0, 704, dt)
    cache, q, k, v = attention_case(case, 31)
    clean = pkg.decode_attention_q4(q, cache, lengths(case[0]))
    check_attention(clean, None, None, q, k, v, case)
    q[0, 1, 2, 5] = what
    q[1, 0, 7] = what
    out = pkg.decode_attention_q4(q, cache, lengths(case[0]))
    bad = torch.zeros(2, 2, 8, dtype=torch.bool, device=G.dev())
    bad[0, 1, 2] = bad[1, 0, 7] = True
    assert not torch.isfinite(out[bad]).any() and torch.equal(out[~bad], clean[~bad])
    ok()


def test_decode_keys_that_some_tokens_do_not_see():
    """NaN rows behind a sequence, and before every token's window, touch nothing; the cut runs through a unit."""
    for n, T, window in ((100, 1, 0), (100, 3, 40), (129, 5, 64), (64, 1, 1), (1000, 2, 300)):
        for dt in (BF16, F32):
            case = ([n], T, 8, 2, 128, window, 1100, dt)
            cache, q, k, v = attention_case(case, n + T)
            lo = max(0, n - T - window + 1) if window else 0
            for s in (cache.k_scale, cache.v_scale):
                s.view(torch.uint8)[:, :, :lo] = 0x7f
            w = torch.zeros(1, 2, 1100, device=G.dev())
            out = pkg.decode_attention_q4(q, cache, lengths([n]), weights=w, window=window)
            k[:, :, :lo] = v[:, :, :lo] = 0
            check_attention(out, w, torch.zeros_like(w), q, k, v, case)
    ok()


def test_decode_reports_lengths_and_leaves_the_others_right():
    case = ([50, 60, 70], 2, 8, 2, 128, 0, 64, BF16)
    cache, q, k, v = attention_case(case, 9)
    w = torch.zeros(3, 2, 64, device=G.dev())
    out = torch.full_like(q, 3.0)
    pkg.decode_attention_q4(q, cache, lengths([50, -1, 65]), out, weights=w)
    ok(-11)
    assert (out[1:] == 3).all() and not w[1:].any()
    check_attention(out[:1], w[:1], torch.zeros_like(w), q, k, v, ([50], *case[1:]))


def test_decode_in_a_cache_beyond_32_bits():
    """The last slot of a cache whose codes pass 2^32 bytes, and its last rows."""
    B, Hkv, cap, D = 5, 8, 1 << 21, 128
    cache = pkg.q4_cache(Hkv, cap, D, batch=B)
    n, T = cap, 2
    k, v = randn((B, 300, Hkv, D), BF16, 1), randn((B, 300, Hkv, D), BF16, 2)
    ns = lengths([300, 300, 300, 300, n])
    pkg.cache_write_q4(k, v, cache, lengths=ns)
    q = randn((B, T, 16, D), BF16, 3)
    w = torch.zeros(B, Hkv, cap, device=G.dev())
    out = pkg.decode_attention_q4(q, cache, ns, weights=w, window=290)
    kk, vv = (R.values(c[:, :, -300:], s[:, :, -300:]) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    want, tol, acc, acc_tol = R.attention(q[4], kk[4], vv[4], 300, 290, R8.default_scale(D), BF16)
    within(out[4], want, tol)
    within(w[4, :, -300:], acc, acc_tol)
    assert not w[4, :, :-300].any()
    left, rows = pkg.cache_evict_q4(cache, w, ns, 64, recent=3)
    assert left.tolist() == [64] * 5
    top = acc[:, :297].float()
    for h in range(Hkv):
        kept = rows[4, h].long() - (cap - 300)
        assert kept.min() >= 0 and kept[-3:].tolist() == [297, 298, 299]
        assert torch.equal(cache.k[4, h, :64], R.quantise(k[4, kept, h], 0)[0])
        # the 61 heaviest, but for weights closer to one another than their tolerance
        edge = top[h].sort(descending=True).values[60]
        assert (top[h][kept[:61]] >= edge * (1 - 1e-4)).all()
    ok()


PREFILL = [  # T, start, H, Hkv, D, window, dtype
    (1, 0, 8, 2, 128, 0, BF16),
    (5, 40, 8, 2, 128, 0, BF16),
    (12, 500, 32, 8, 128, 0, BF16),
    (13, 500, 32, 8, 128, 0, BF16),
    (200, 300, 8, 2, 128, 0, BF16),
    (200, 300, 8, 2, 128, 100, BF16),
    (130, 0, 4, 1, 512, 0, BF16),
    (300, 77, 8, 2, 512, 128, BF16),
    (100, 50, 8, 2, 128, 0, F32),
    (600, 50, 6, 2, 128, 64, F32),
    (70, 400, 8, 2, 512, 0, F32),
]


@pytest.mark.parametrize("case", PREFILL, ids=str)
def test_prefill(case):
    T, start, H, Hkv, D, window, dt = case
    n = start + T
    cache = pkg.Q4Cache(*R.make_cache(Hkv, n + 9, D, seed=6, device=G.dev()), 1, -2)
    q = randn((T, H, D), dt, 4, 0.5)
    out = pkg.prefill_attention_q4(q, cache, start_pos=start, window=window)
    k, v = R.values(cache.k, cache.k_scale, 1), R.values(cache.v, cache.v_scale, -2)
    want, tol, _, _ = R.attention(q, k, v, n, window, R8.default_scale(D), dt)
    if dt == BF16:                     # long chunks: the 16-bit kernels round the weights to bf16
        j = torch.arange(n, device=G.dev())
        pos = torch.arange(start, n, device=G.dev())[:, None]
        hidden = (j > pos) | (j <= pos - window if window else torch.zeros_like(j, dtype=torch.bool))
        for h in range(H):
            kv = h // (H // Hkv)
            p = torch.softmax((q[:, h].double() @ k[kv, :n].T * R8.default_scale(D)).masked_fill(hidden, float("-inf")), -1)
            tol[:, h] += 2.0 ** -8 * (p @ v[kv, :n].abs()) * (1 + 2.0 ** -8)
    within(out, want, tol)
    wide = torch.zeros(T, H + 3, D, dtype=dt, device=G.dev())
    wide[:, 1:H + 1] = q
    assert torch.equal(pkg.prefill_attention_q4(wide[:, 1:H + 1], cache, start_pos=start, window=window), out)
    ok()


# ------------------------------------------------------------------ eviction

EVICT = [  # lens, Hkv, D, cap, keep, recent
    ([10], 1, 128, 16, 4, 1),
    ([10], 1, 128, 16, 1, 0),
    ([10], 1, 128, 16, 1, 1),
    ([100, 0, 33, 34, 100, 1], 2, 128, 100, 33, 5),
    ([100, 64, 63, 99], 8, 512, 128, 64, 64),
    ([1000, 999, 3], 3, 16, 1001, 500, 0),
    ([777, 778], 2, 80, 800, 776, 20),
    ([5000, 1, 4097], 2, 128, 5003, 1025, 128),
    ([2000], 1, 496, 2000, 1999, 7),
    ([40000, 20000], 2, 128, 40001, 16385, 3),
    ([300] * 50, 4, 128, 300, 100, 10),
    ([70000, 99999, 3], 1, 16, 100001, 30000, 11),
    ([140000, 150001], 1, 32, 150001, 70001, 5),
]


def check_evict(cache, before, w, w0, lens, keep, recent, left, rows):
    for b, n in enumerate(lens):
        assert left[b] == min(n, keep)
        kept = R.evict(w0[b], n, keep, recent)
        for h, r in enumerate(kept):
            assert rows[b, h].tolist() == r + [-1] * (keep - len(r)), (b, h)
            if n <= keep:
                assert torch.equal(w[b, h].nan_to_num(7.0), w0[b, h].nan_to_num(7.0))
            else:
                at = torch.tensor(r, device=w.device)
                assert torch.equal(w[b, h, :keep].nan_to_num(7.0), w0[b, h, at].nan_to_num(7.0))
                assert not w[b, h, keep:n].any()
                assert torch.equal(w[b, h, n:].nan_to_num(7.0), w0[b, h, n:].nan_to_num(7.0))
                for t, t0 in zip(raw(cache), before):
                    assert torch.equal(t[b, h, :keep], t0[b, h, at])
            for t, t0 in zip(raw(cache), before):
                if n <= keep:
                    assert torch.equal(t[b, h], t0[b, h])
                else:
                    assert torch.equal(t[b, h, keep:], t0[b, h, keep:])


@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"B{len(c[0])}x{c[0][0]}-{c[1]}x{c[2]}-cap{c[3]}-keep{c[4]}-recent{c[5]}")
@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "odd"])
def test_evict(case, kind):
    lens, Hkv, D, cap, keep, recent = case
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=len(lens), seed=1, device=G.dev()))
    w = randn((len(lens), Hkv, cap), F32, 2, 3.0).exp()
    if kind == "ties":
        w = (w * 2).round().clamp(max=5)
    elif kind == "equal":
        w.fill_(0.5)
    elif kind == "odd":                        # both signs and zeros, subnormals, infinities, NaN
        w *= randn(w.shape, F32, 3).sign()
        pick = torch.randint(0, 30, w.shape, generator=torch.Generator().manual_seed(4)).to(G.dev())
        for i, x in enumerate((0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e-41, -1e-41, 3e38)):
            w[pick == i] = x
    w0, before = w.clone(), raw(cache)
    n = lengths(lens)
    left, rows = pkg.cache_evict_q4(cache, w, n, keep, recent=recent)
    assert left.dtype == torch.int64 and rows.dtype == torch.int32 and n.tolist() == lens
    check_evict(cache, before, w, w0.cpu().to(G.dev()), lens, keep, recent, left.tolist(), rows)
    ok()


def test_evict_in_place_lengths_given_rows_and_bad_lengths():
    cache = pkg.Q4Cache(*R.make_cache(2, 64, 128, batch=4, seed=1, device=G.dev()))
    w = randn((4, 2, 64), F32, 2).abs()
    w0, before = w.clone(), raw(cache)
    n = lengths([64, 65, -3, 20])
    rows = torch.zeros(4, 2, 30, dtype=torch.int32, device=G.dev())
    left, got = pkg.cache_evict_q4(cache, w, n, 30, recent=4, lengths_out=n, rows_out=rows)
    assert left is n and got is rows and n.tolist() == [30, 65, -3, 20]
    ok(-11)
    assert (rows[1:3] == -1).all() and torch.equal(w[1:3], w0[1:3])
    assert all(torch.equal(a[1:], b[1:]) for a, b in zip(raw(cache), before))
    check_evict(cache, before, w, w0, [64], 30, 4, [30], rows)


# ------------------------------------------------------------------ together

def serve(steps, cache, w, n, pos, inputs, freq, keep, out, side=None):
    """Decode steps of a layer: rotation, write, attention with weights; the cache is cut when told to."""
    for i in steps:
        q, k, v = inputs[i]
        qr, kr = pkg.qk_norm_rope(q, k, None, None, freq, lengths=pos, stream=side)
        pkg.cache_write_q4(kr, v, cache, lengths=n, stream=side)
        pkg.decode_attention_q4(qr, cache, n, out[i], weights=w, stream=side)
        if i % 8 == 7:
            pkg.cache_evict_q4(cache, w, n, keep, recent=4, lengths_out=n, stream=side)
        n += 1
        pos += 1


def test_a_served_batch_evicts_as_it_goes():
    """40 tokens of three sequences in a cache of 24 rows, against 64-bit forms of every step."""
    B, H, Hkv, D, cap, keep = 3, 8, 2, 128, 24, 12
    freq = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=G.dev()) / (D // 2))
    cache = pkg.q4_cache(Hkv, cap, D, batch=B, v_exponent=-1)
    w = torch.zeros(B, Hkv, cap, device=G.dev())
    n, pos = lengths([1, 1, 1]), lengths([1, 1, 1])
    held = [[[] for _ in range(Hkv)] for _ in range(B)]          # (codes and scales of k and v, weight)
    for step in range(40):
        q, k, v = (randn((B, 1, heads, D), BF16, 100 * step + i) for i, heads in enumerate((H, Hkv, Hkv)))
        qr, kr = pkg.qk_norm_rope(q, k, None, None, freq, lengths=pos)
        pkg.cache_write_q4(kr, v, cache, lengths=n)
        out = pkg.decode_attention_q4(qr, cache, n, weights=w)
        rows = n.tolist()
        for b in range(B):
            for h in range(Hkv):
                held[b][h].append([*R.quantise(kr[b, 0, h], 0), *R.quantise(v[b, 0, h], -1), 0.0])
                assert rows[b] == len(held[b][h])
                for t, i in ((cache.k, 0), (cache.k_scale, 1), (cache.v, 2), (cache.v_scale, 3)):
                    want = torch.stack([x[i] for x in held[b][h]])
                    assert torch.equal(t.view(torch.uint8)[b, h, :rows[b]], want)
            kk = R.values(cache.k[b], cache.k_scale[b])
            vv = R.values(cache.v[b], cache.v_scale[b], -1)
            want, tol, acc, acc_tol = R.attention(qr[b], kk, vv, rows[b], 0, R8.default_scale(D), BF16)
            within(out[b], want, tol)
            for h in range(Hkv):
                for j, x in enumerate(held[b][h]):
                    x[4] += acc[h, j].item()
            sums = torch.tensor([[x[4] for x in held[b][h]] for h in range(Hkv)], device=G.dev(), dtype=torch.float64)
            within(w[b, :, :rows[b]], sums, 1e-5 * sums + 1e-6)
            assert not w[b, :, rows[b]:].any()
        if step % 8 == 7:
            w0 = w.clone()
            n, kept = pkg.cache_evict_q4(cache, w, n, keep, recent=4)
            for b in range(B):
                want = R.evict(w0[b], rows[b], keep, 4)
                for h in range(Hkv):
                    assert kept[b, h].tolist() == (want[h] + [-1] * keep)[:keep]
                    held[b][h] = [held[b][h][j] for j in want[h]]
        n = n + 1
        pos = pos + 1
    ok()


def test_a_graph_replays_steps_and_eviction():
    B, H, Hkv, D, cap, keep = 2, 8, 2, 128, 24, 12
    freq = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=G.dev()) / (D // 2))
    inputs = [tuple(randn((B, 1, heads, D), BF16, 10 * i + j) for j, heads in enumerate((H, Hkv, Hkv))) for i in range(8)]

    def fresh():
        return (pkg.q4_cache(Hkv, cap, D, batch=B), torch.zeros(B, Hkv, cap, device=G.dev()), lengths([1, 3]),
                lengths([1, 3]), [torch.zeros_like(q) for q, _, _ in inputs])

    cache, w, n, pos, out = fresh()
    for _ in range(3):
        serve(range(8), cache, w, n, pos, inputs, freq, keep, out)
    c2, w2, n2, pos2, out2 = fresh()
    start = [t.clone() for t in (*c2[:4], w2, n2, pos2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve(range(8), c2, w2, n2, pos2, inputs, freq, keep, out2)
    for t, s in zip((*c2[:4], w2, n2, pos2), start):
        assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))       # nothing ran yet
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert same(cache, c2) and torch.equal(w, w2) and torch.equal(n, n2)
    assert all(torch.equal(a, b) for a, b in zip(out, out2))
    ok()


def test_on_another_stream():
    B, H, Hkv, D, cap, keep = 2, 8, 2, 128, 24, 12
    freq = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device=G.dev()) / (D // 2))
    inputs = [tuple(randn((B, 1, heads, D), BF16, 10 * i + j) for j, heads in enumerate((H, Hkv, Hkv))) for i in range(8)]
    got = []
    for side in (None, torch.cuda.Stream()):
        cache, w = pkg.q4_cache(Hkv, cap, D, batch=B), torch.zeros(B, Hkv, cap, device=G.dev())
        n, pos, out = lengths([1, 3]), lengths([1, 3]), [torch.zeros_like(q) for q, _, _ in inputs]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            serve(range(8), cache, w, n, pos, inputs, freq, keep, out, side)
        torch.cuda.synchronize()
        got.append((raw(cache), w, n, out))
    (c, w, n, out), (c2, w2, n2, out2) = got
    assert same(c, c2) and torch.equal(w, w2) and torch.equal(n, n2) and all(torch.equal(a, b) for a, b in zip(out, out2))
    ok()


def test_refuses_tensors_off_the_gpu_and_small_workspaces():
    case = ([50, 60], 2, 8, 2, 128, 0, 64, BF16)
    cache, q, k, v = attention_case(case, 9)
    n = lengths(case[0])
    w = torch.zeros(2, 2, 64, device=G.dev())
    need = pkg.decode_workspace_bytes_q4(2, 2, 8, 2, 128, 64, weights=True)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=G.dev())
    out = pkg.decode_attention_q4(q, cache, n, weights=w, workspace=ws)
    assert torch.equal(out, pkg.decode_attention_q4(q, cache, n))
    with pytest.raises(pkg.PfaError, match="SCRATCH"):
        pkg.decode_attention_q4(q, cache, n, weights=w, workspace=ws[:need - 256])
    with pytest.raises(pkg.PfaError, match="SCRATCH"):
        pkg.decode_attention_q4(q, cache, n, weights=w, workspace=None)
    with pytest.raises(pkg.PfaError, match="DEVICE"):
        pkg.decode_attention_q4(q, cache, n.cpu())
    with pytest.raises(pkg.PfaError, match="DEVICE"):
        pkg.decode_attention_q4(q, cache, n, weights=w.cpu())
    with pytest.raises(pkg.PfaError, match="DEVICE"):
        pkg.cache_evict_q4(cache, w, n.cpu(), 20)
    with pytest.raises(pkg.PfaError, match="ALIAS"):
        pkg.decode_attention_q4(q, cache, n, q)
    with pytest.raises(ValueError):
        pkg.decode_attention_q4(q, cache, n, weights=w[:, :, :32])
    ok()
