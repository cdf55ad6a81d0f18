"""Plain 64-bit forms of the operators around the 4-bit cache, for the tests.

They run on whatever device the inputs are on and share no code with the package.
"""
import torch

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# off by at most half a step, relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
F8 = torch.float8_e4m3fn


def _e4m3():
    """Every finite e4m3 value >= 0, in order: the index is the code."""
    return [m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127]


def nearest(a, values):
    """Index of the value nearest to each a >= 0 (64 bits), the even index of two; the last beyond them."""
    v = torch.tensor(values, dtype=torch.float64, device=a.device)
    up = torch.searchsorted(v, a.contiguous()).clamp(max=len(values) - 1)
    down = (up - 1).clamp(min=0)
    u, d = (v[up] - a).abs(), (a - v[down]).abs()
    return torch.where((u < d) | ((u == d) & (up % 2 == 0)) | (a > values[-1]), up, down)


def quantise(x, exponent):
    """x [..., D] -> (packed codes [..., D / 2] uint8, scale codes [..., D / 16] uint8)."""
    y = x.double().unflatten(-1, (-1, 16)) * 2.0 ** -exponent
    ok = torch.isfinite(y).all(-1)
    y = torch.where(ok[..., None], y, 0.0)
    six = torch.full((), 6.0, dtype=torch.float64, device=x.device)
    s = nearest(y.abs().amax(-1) / six, _e4m3())
    f = torch.tensor(_e4m3(), dtype=torch.float64, device=x.device)[s][..., None]
    c = nearest(y.abs() / torch.where(f > 0, f, 1.0), E2M1) + 8 * torch.signbit(y).long()
    c = torch.where(f > 0, c, 0).flatten(-2)
    s = torch.where(ok, s, 0x7f)
    return (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8), s.to(torch.uint8)


def values(codes, scale, exponent=0):
    """What packed codes [..., D / 2] and scales [..., D / 16] stand for, 64 bits."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    return t[c] * scale.double().repeat_interleave(16, -1) * 2.0 ** exponent


def attention(q, k, v, n, window, scale, dtype, exponent=0):
    """q [T, H, D] at rows n - T .. n - 1 of k and v [Hkv, cap, D] (64 bits; v is values() times
    2**exponent).  Returns (out, tolerance, weights [Hkv, cap], tolerance).

    The tolerance:
      - half a step of the output's type;
      - the weights' rounding: half precision (2^-11 at bf16) or a high and a low
        half (2^-21 at fp32), each times sum p |v|;
      - the scores: q is exact (bf16) or off by 2^-21 (fp32, a high and a low half), and
        D / 16 products of 16 (twice as many at fp32) are added in fp32, at most 2^-22 of the
        terms' size each; an error d of a score is one of 2 d of every weight;
      - the sum over keys: 2^-22 for each 16 of them;
      - small weights: a half (the low half at fp32) below 2^-14 is a multiple of 2^-24, off by up to
        2^-25.  A weight is 2^(s - base) 2^11, and base at most the largest s: undone, 2^-36 of the largest
        weight, which is at most the sum; times |v| of each key.
    The accumulated weights leave out the roundings to halves: scores as above, and an addition in
    fp32 (2^-24 of the sum) for each row.
    """
    T, H, D = q.shape
    Hkv, cap = k.shape[:2]
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    acc = torch.zeros(Hkv, cap, dtype=torch.float64, device=q.device)
    acc_tol = torch.zeros_like(acc)
    first = max(0, n - T)
    if n <= first:
        return out, tol, acc, acc_tol
    lo = max(0, first - window + 1) if window > 0 else 0
    j = torch.arange(lo, n, device=q.device)
    pos = torch.arange(first, n, device=q.device)[:, None]
    hidden = (j > pos) | (j <= pos - window if window > 0 else torch.zeros_like(j, dtype=torch.bool))
    f32 = dtype == torch.float32
    for h in range(H):
        g = h // (H // Hkv)
        kk, vv = k[g, lo:n], v[g, lo:n]
        x = q[T - (n - first):, h].double()
        s = (x @ kk.T * scale).masked_fill(hidden, float("-inf"))
        size = (x.abs() @ kk.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(-1, keepdim=True)
        p = torch.softmax(s, -1)
        o = p @ vv
        a = p @ vv.abs()
        score = 2 * size * (((2 if f32 else 1) * D / 16 + 2) * 2.0 ** -22 + (2.0 ** -21 if f32 else 0.0))
        keys = (n - lo + 16) / 16 * 2.0 ** -22
        c = (2.0 ** -21 if f32 else 2.0 ** -11) + keys + score
        out[T - (n - first):, h] = o
        tol[T - (n - first):, h] = HALF[dtype] * o.abs() + (1 + HALF[dtype]) * (c * a + 2.0 ** -36 * vv.abs().sum(0))
        acc[g, lo:n] += p.sum(0)
        acc_tol[g, lo:n] += ((score + keys) * p).sum(0)
    rows = T * (H // Hkv)
    return out, tol, acc, acc_tol + (rows + 4) * 2.0 ** -24 * acc


def evict(weights, n, keep, recent):
    """The kept rows of one sequence of n rows: weights [Hkv, cap] -> list for each head, in order."""
    if n <= keep:
        return [list(range(n)) for _ in weights]
    kept = []
    for w in weights[:, :n - recent].tolist():
        heavy = sorted(range(n - recent), key=lambda j: (-(float("inf") if w[j] != w[j] else w[j]), w[j] == w[j], j))
        kept.append(sorted(heavy[:keep - recent]) + list(range(n - recent, n)))
    return kept


def make_cache(Hkv, cap, D, batch=None, seed=0, device="cpu", dead=None):
    """A filled cache (codes and scales) whose groups differ in size; rows >= dead[b] (all b) have NaN scales."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    lead = (Hkv,) if batch is None else (batch, Hkv)
    out = []
    for _ in "kv":
        c = torch.randint(0, 256, (*lead, cap, D // 2), generator=g, dtype=torch.uint8)
        s = torch.randint(16, 56, (*lead, cap, D // 16), generator=g, dtype=torch.uint8)   # 2^-6 .. 0.94
        out.append((c, s))
    (k, ks), (v, vs) = out
    if dead is not None:
        for b, n in enumerate(dead):
            for s in (ks, vs):
                (s[b] if batch is not None else s)[..., n:, :] = 0x7f
    return k.to(device), v.to(device), ks.view(F8).to(device), vs.view(F8).to(device)
