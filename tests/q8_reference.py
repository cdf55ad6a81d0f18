"""Plain 64-bit forms of the operators around the 8-bit cache, for the tests.

They run on whatever device the inputs are on and share no code with the
package.  Caches are tuples (k, v, k_scale, v_scale) of float8_e4m3fn codes
[Hkv, cap, D] and float32 scales [Hkv, cap / block] of ONE sequence.
"""
import math

import torch

# off by at most half a step, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def norm_rope(x, weight, offset, eps, inv_freq, pos, interleaved):
    """x [T, heads, D], pos [T] (python ints or int64) -> (y, size of the terms in y)."""
    x = x.double()
    T, _, D = x.shape
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + eps) * (weight.double() + offset)
    y, size = x.clone(), x.abs()
    if inv_freq is not None:
        n = inv_freq.numel()
        a = torch.as_tensor(pos, device=x.device).double()[:, None, None] * inv_freq
        i = torch.arange(n, device=x.device)
        i, j = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        u, w = x[..., i], x[..., j]
        y[..., i] = u * a.cos() - w * a.sin()
        y[..., j] = u * a.sin() + w * a.cos()
        size[..., i] = size[..., j] = u.abs() + w.abs()
    return y, size


def to_e4m3(x):
    """Nearest e4m3 value (64 bits), ties to even; not finite -> NaN.  |x| <= 448."""
    ok = torch.isfinite(x)
    z = torch.where(ok, x, torch.zeros_like(x))
    _, e = torch.frexp(z)
    step = torch.ldexp(torch.ones_like(z), (e - 1).clamp(min=-6) - 3)
    return torch.where(ok, (z / step).round() * step, torch.full_like(z, float("nan")))


def block_scale(a):
    """Smallest power of two s >= 2^-126 with a / s <= 448; 0 for a = 0."""
    if a == 0:
        return 0.0
    s = 2.0 ** -126
    while a / s > 448:
        s *= 2
    return s


def write(x, codes, scale, first, block):
    """New codes (64-bit values) and scales of one sequence: x [T, Hkv, D] at rows first ..  (CPU)."""
    T, Hkv, D = x.shape
    codes, scale, x = codes.double(), scale.double(), x.double()
    codes, scale = codes.clone(), scale.clone()
    low, end = max(first, 0), first + T
    for h in range(Hkv):
        for c in range(low // block, -(-end // block) if end > low else 0):
            lo, hi = max(low, c * block), min(end, (c + 1) * block)
            new = x[lo - first:hi - first, h]
            fin = new[torch.isfinite(new)]
            a = float(fin.abs().max()) if fin.numel() else 0.0
            had = float(scale[h, c]) if lo > c * block else 0.0
            s = max(had, block_scale(a))
            if lo > c * block:
                old = codes[h, c * block:lo] * had
                codes[h, c * block:lo] = to_e4m3(old / s) if s else to_e4m3(old)
            codes[h, lo:hi] = to_e4m3(new / s if s else new)
            scale[h, c] = s
    return codes, scale


def values(codes, scale):
    """What codes and scales stand for, 64 bits."""
    block = codes.shape[-2] // scale.shape[-1]
    return codes.double() * scale.double().repeat_interleave(block, -1)[..., None]


def attention(q, cache, n, window, scale, dtype):
    """q [T, H, D] at positions n - T .. n - 1.  Returns (out, tolerance), both [T, H, D], 64 bits.

    The tolerance of the kernels that read the codes:
      - half a step of the output's type;
      - the weights' rounding: half precision (2^-11 at bf16) or a high and a low
        half (2^-21 at fp32), each times sum p |v|;
      - the scores: q is exact (bf16) or off by 2^-21 (fp32, a high and a low half), and
        D / 16 products of 16 are added in fp32, at most 2^-22 of the terms' size each;
        an error d of a score is one of 2 d of every weight;
      - the sum over keys: 2^-22 for each 16 of them;
      - small weights: a half (the low half at fp32) below 2^-14 is a multiple of 2^-24, so off by up to 2^-25
        whatever its size.  It stands for e_j vs_j / vmax * 2^14 with e_j = 2^(s_j - m), vmax the
        largest V scale seen: undone, 2^-39 vmax / vs_j of weight, that is 2^-39 vmax |code_j| of
        the sum, which is divided by sum e_j >= 1 (the largest e_j is 1).  It shows only where all
        weights of size meet V values of zero.
    """
    T, H, D = q.shape
    blk = cache[0].shape[-2] // cache[2].shape[-1]
    k, v = values(cache[0], cache[2]), values(cache[1], cache[3])
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    first = max(0, n - T)
    if n <= first:
        return out, tol
    lo = max(0, first - window + 1) if window > 0 else 0
    j = torch.arange(lo, n, device=q.device)
    pos = torch.arange(first, n, device=q.device)[:, None]
    hidden = (j > pos) | (j <= pos - window if window > 0 else torch.zeros_like(j, dtype=torch.bool))
    f32 = dtype == torch.float32
    for h in range(H):
        kk, vv = k[h // (H // k.shape[0]), lo:n], v[h // (H // k.shape[0]), lo:n]
        x = q[T - (n - first):, h].double()
        s = (x @ kk.T * scale).masked_fill(hidden, float("-inf"))
        size = (x.abs() @ kk.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(-1, keepdim=True)
        p = torch.softmax(s, -1)
        o = p @ vv
        a = p @ vv.abs()
        codes = cache[1][h // (H // k.shape[0]), lo:n].double().abs()
        vs = cache[3][h // (H // k.shape[0]), lo // blk:(n - 1) // blk + 1].double().max()
        c = (2.0 ** -21 if f32 else 2.0 ** -11) + (n - lo + 16) / 16 * 2.0 ** -22 \
            + 2 * size * ((D / 16 + 2) * 2.0 ** -22 + (2.0 ** -21 if f32 else 0.0))
        out[T - (n - first):, h] = o
        tol[T - (n - first):, h] = HALF[dtype] * o.abs() + (1 + HALF[dtype]) * (c * a + 2.0 ** -39 * vs * codes.sum(0))
    return out, tol


def default_scale(D):
    return float(torch.tensor(1.0 / math.sqrt(D), dtype=torch.float32))


def make_cache(Hkv, cap, D, block, batch=None, seed=0, device="cpu", dead=None):
    """A filled cache whose blocks differ in size; rows >= dead[b] (all b) hold NaN codes."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    lead = (Hkv,) if batch is None else (batch, Hkv)
    out = []
    for _ in "kv":
        x = torch.randint(0, 256, (*lead, cap, D), generator=g, dtype=torch.uint8)
        x = torch.where((x & 0x7f) == 0x7f, x - 1, x)                     # no NaN among the live codes
        x = torch.where((x & 0x7f) >= 0x70, x - 0x20, x)                  # magnitudes up to 30
        e = torch.randint(-6, 0, (*lead, cap // block), generator=g)
        s = torch.ldexp(torch.ones(e.shape), e) / 4
        out.append((x, s))
    (k, ks), (v, vs) = out
    if dead is not None:
        for b, n in enumerate(dead):
            for t, s in ((k, ks), (v, vs)):
                part = t[b] if batch is not None else t
                part[..., n:, :] = 0x7f
                part = s[b] if batch is not None else s
                part[..., -(-n // block):] = float("nan")
    f8 = torch.float8_e4m3fn
    return tuple(t.to(device) for t in (k.view(f8), v.view(f8), ks, vs))
