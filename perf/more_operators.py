"""Cases of the operators around a 4-bit KV cache: the cache's write and read-back, the attention over it (few
tokens of a batch, with or without the accumulated weight of each key, and chunks of one sequence), and the
eviction of rows by that weight.

The cache holds K and V as e2m1 codes, two to a byte, with one e4m3 scale for each 16 channels of a row; a value is
code * scale * 2**exponent, the exponent one number for all of K (of V).  `run` computes an operator in elementary
torch operations; with `own` set it calls the package.

Codes are returned as they lie in the cache, packed, and have to be equal: what a row is quantised to is exact.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 16


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the new token of 32 sequences goes into the cache at 32 different positions
        dict(name="write_step", op="write", B=32, T=1, Hkv=8, D=128, dtype="bf16", cap=8192, start=-1, ke=0, ve=0, mix=2),
        # a prefill chunk of a 64k prompt goes into the cache
        dict(name="write_chunk", op="write", B=1, T=2048, Hkv=8, D=128, dtype="bf16", cap=65536, start=61445, ke=0,
             ve=-3, mix=0),
        # the whole 64k cache of a layer read back
        dict(name="read_64k", op="read", Hkv=8, D=128, dtype="bf16", cap=65536, start=0, stop=63488, ke=0, ve=-3),
        # an odd range of rows of a wide-head layer, fp32
        dict(name="read_f32_odd", op="read", Hkv=2, D=512, dtype="f32", cap=8191, start=5003, stop=8191, ke=1, ve=0),
        # one sequence at a full 128k context: nothing but the cache's bytes counts
        dict(name="decode_one_128k", op="decode", B=1, T=1, H=32, Hkv=8, D=128, dtype="bf16", cap=131072, window=0,
             longest=131072, weights=False, ke=0, ve=-3, mix=3),
        # a served batch of uneven sequences, one slot empty, the keys' weights counted for a later eviction
        dict(name="decode_batch", op="decode", B=32, T=1, H=32, Hkv=8, D=128, dtype="bf16", cap=8192, window=0,
             longest=8192, weights=True, ke=0, ve=0, mix=4),
        # three drafted tokens of four short sequences, wide heads, sliding window, fp32
        dict(name="decode_f32_draft", op="decode", B=4, T=3, H=8, Hkv=2, D=512, dtype="f32", cap=2048, window=1024,
             longest=1358, weights=False, ke=0, ve=0, mix=5),
        # the last 32 tokens of a prompt weigh its keys before some of them are evicted
        dict(name="decode_observe", op="decode", B=1, T=32, H=32, Hkv=8, D=128, dtype="bf16", cap=16384, window=0,
             longest=16384, weights=True, ke=0, ve=0, mix=6),
        # a 64k prompt cut down to a quarter of its keys
        dict(name="evict_one_64k", op="evict", B=1, Hkv=8, D=128, cap=65536, longest=63488, keep=16384, recent=512, mix=7),
        # a served batch brought back to its budget
        dict(name="evict_batch", op="evict", B=32, Hkv=8, D=128, cap=8192, longest=8192, keep=2048, recent=256, mix=8),
        # the steady prefill chunk of a 64k prompt
        dict(name="prefill_64k", op="prefill", T=2048, H=32, Hkv=8, D=128, dtype="bf16", cap=65536, window=0, start=61440,
             ke=0, ve=-3),
        # the last, short chunk of a 64k prompt
        dict(name="prefill_64k_t12", op="prefill", T=12, H=32, Hkv=8, D=128, dtype="bf16", cap=65536, window=0, start=63360,
             ke=0, ve=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "decode", "decode", "evict", "evict", "prefill"))
    D = rng.choice((128, 128, 512))
    Hkv = rng.choice((1, 2, 4, 8)) if D == 128 else rng.choice((1, 2, 4))
    G = rng.choice((1, 2, 4, 5, 8))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    ex = dict(ke=rng.choice((0, 0, 2)), ve=rng.choice((0, -3, -7)))
    if op == "write":
        batch = rng.random() < 0.5
        T = rng.randint(1, 8) if batch else _log(rng, 1, 8192)
        start = -1 if batch else _log(rng, 1, 50000) - 1
        cap = rng.randint(64, 4096) if batch else start + T + rng.randint(0, 64)
        return dict(op=op, B=_log(rng, 1, 64) if batch else 1, T=T, Hkv=Hkv, D=D, dtype=dtype, cap=cap, start=start,
                    mix=rng.randrange(1000), **ex)
    if op == "read":
        cap = _log(rng, 16, 65536)
        start = rng.randrange(cap)
        return dict(op=op, Hkv=Hkv, D=D, dtype=dtype, cap=cap, start=start, stop=rng.randint(start + 1, cap), **ex)
    window = rng.choice((0, 0, 0, 1024, 333))
    if op == "decode":
        B = _log(rng, 1, 48)
        cap = _log(rng, 64, 131072 if B < 3 else 262144 // B)
        weights = rng.random() < 0.5
        T = rng.choice((1, 1, 1, 2, 4, 7))
        if weights and B < 5 and cap < 20000:
            T = rng.choice((1, 4, 16, 32))
        return dict(op=op, B=B, T=T, H=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, cap=cap, window=window,
                    longest=rng.randint(max(1, cap // 2), cap), weights=weights, mix=rng.randrange(1000), **ex)
    if op == "evict":
        B = _log(rng, 1, 48)
        cap = _log(rng, 64, 131072 if B < 3 else 262144 // B)
        keep = rng.randint(1, cap)
        return dict(op=op, B=B, Hkv=Hkv, D=D, cap=cap, longest=rng.randint(max(1, cap // 2), cap), keep=keep,
                    recent=rng.randint(0, min(keep, 512)), mix=rng.randrange(1000))
    H = Hkv * min(G, 4)
    T = _log(rng, 1, 2048)
    start = _log(rng, 1, 30000) - 1
    return dict(op=op, T=T, H=H, Hkv=Hkv, D=D, dtype=dtype, cap=start + T + rng.randint(0, 100), window=window, start=start,
                **ex)


def _lengths(case):
    """Lengths of the batch's sequences, new tokens included: uneven, the first the longest, one slot empty."""
    r = random.Random(case["mix"])
    B, T = case["B"], case.get("T", 0)
    most = case.get("longest", case["cap"])
    n = [r.randint(min(T, most), most) for _ in range(B)]
    n[0] = most
    if B > 4:
        n[3] = 0
    return n


# ------------------------------------------------------------------ inputs

def _randn(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std)


def _quantise(x, exponent):
    """x [..., D] fp32 -> (codes [..., D / 2] uint8, scales [..., D / 16] e4m3)."""
    y = (x.double() * 2.0 ** -exponent).unflatten(-1, (-1, GROUP))        # quotients lie next to borders
    six = y.new_full((), 6.0)                                  # a tensor: by a number torch multiplies with 1 / 6
    s = (y.abs().amax(-1) / six).clamp(max=448).float().to(F8)
    f = s.double()[..., None]
    a = torch.where(f > 0, y.abs() / f, 0.0)
    m = sum((a > t).to(torch.uint8) for t in (0.25, 1.25, 2.5, 5.0))        # ties go to the even code
    m = m + sum((a >= t).to(torch.uint8) for t in (0.75, 1.75, 3.5))
    c = torch.where(f > 0, m | (torch.signbit(y).to(torch.uint8) << 3), 0).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _values(codes, scale, exponent):
    """What the cache stands for, fp32 [..., D]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    pair = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    return (pair.unflatten(-1, (-1, GROUP)) * (scale.float() * 2.0 ** exponent)[..., None]).flatten(-2)


def _filled(shape, exponent, gen):
    """Codes and scales of a cache tensor of `shape`: normal values, channels and rows of unlike size, a head at a time."""
    *lead, cap, D = shape
    codes = torch.empty((*lead, cap, D // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((*lead, cap, D // GROUP), dtype=torch.uint8, device=DEV)
    for c, s in zip(codes.view(-1, cap, D // 2), scale.view(-1, cap, D // GROUP)):
        x = _randn((cap, D), gen, 2.0 ** exponent) * (1 + _randn((D,), gen, 0.3).abs()) * (_randn((cap, 1), gen, 0.3)).exp()
        a, b = _quantise(x, exponent)
        c.copy_(a)
        s.copy_(b.view(torch.uint8))
    return codes, scale.view(F8)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, D, dt = case["op"], case["D"], DTYPES[case.get("dtype", "bf16")]
    s = dict(case=case)
    batch = op in ("decode", "evict") or (op == "write" and case["start"] < 0)
    if batch:
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int64, device=DEV)
    ke, ve = case.get("ke", 0), case.get("ve", 0)
    shape = (case["Hkv"], case["cap"], D)
    if batch:
        shape = (case["B"], *shape)
    (k, ks), (v, vs) = (_filled(shape, e, gen) for e in (ke, ve))
    s["cache"] = [k, v, ks, vs]
    if op == "write":
        B, T, Hkv = case["B"], case["T"], case["Hkv"]
        kv = _randn((B, T, 2 * Hkv, D), gen)
        kv[:, :, :Hkv] *= 2.0 ** ke
        kv[:, :, Hkv:] *= 2.0 ** ve
        kv = kv.to(dt) if batch else kv[0].to(dt)
        s["k"], s["v"] = kv[..., :Hkv, :], kv[..., Hkv:, :]     # columns of one projection's output
    elif op in ("decode", "prefill"):
        qshape = (case["T"], case["H"], D)
        s["q"] = _randn((case["B"], *qshape) if batch else qshape, gen, 2.0 ** -ke).to(dt)
    if op == "evict" or case.get("weights"):
        # what some steps have left: few heavy keys, a long tail, nothing behind a sequence's last row
        w = (_randn((case["B"], case["Hkv"], case["cap"]), gen, 2.0) - 4).exp_()
        s["weights"] = torch.where(torch.arange(case["cap"], device=DEV) < s["lengths"][:, None, None], w, 0.0)
    return s


# ------------------------------------------------------------------ plain forms

def _write(x, codes, scale, first, exponent):
    """Writes x [B, T, Hkv, D] at rows first.. of codes [B, Hkv, cap, D / 2]; `first` [B].  In place."""
    B, T = x.shape[:2]
    c, s = _quantise(x.float(), exponent)
    rows = first[:, None] + torch.arange(T, device=DEV)
    b = torch.arange(B, device=DEV)[:, None].expand(B, T)
    ok = rows >= 0
    codes.transpose(1, 2)[b[ok], rows[ok]] = c[ok]
    scale.view(torch.uint8).transpose(1, 2)[b[ok], rows[ok]] = s.view(torch.uint8)[ok]


def _attention(q, k, v, pos, window):
    """q [B, T, H, D], k and v [B, Hkv, L, D] fp32, pos [B, T] -> fp32 [B, T, H, D] and the keys' weights [B, Hkv, L]."""
    B, T, H, D = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    j = torch.arange(L, device=DEV)
    see = (j <= pos[..., None]) & (pos[..., None] >= 0)
    if window > 0:
        see &= j > pos[..., None] - window
    any_row = see.any(1)[:, None, :, None]                      # rows no token sees hold anything
    k, v = torch.where(any_row, k, 0.0), torch.where(any_row, v, 0.0)
    x = q.float().reshape(B, T, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = (x @ k.transpose(-1, -2)).mul_(1 / math.sqrt(D)).reshape(B, Hkv, -1, T, L)
    s.masked_fill_(~see[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    n = s.sum(-1, keepdim=True)
    s /= torch.where(n > 0, n, torch.ones_like(n))
    o = (s.reshape(B, Hkv, -1, L) @ v).reshape(B, Hkv, -1, T, D)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, H, D), s.sum((2, 3))


def _evict(cache, weights, lengths, keep, recent):
    """Keeps the `recent` newest rows of each head and the heaviest others, in their order.  In place."""
    cap = weights.shape[-1]
    n = lengths[:, None, None]
    j = torch.arange(cap, device=DEV)
    first = torch.where(j >= n, float("-inf"), torch.where(j >= n - recent, float("inf"), weights))
    rows = first.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values     # ties: lowest index
    full = n > keep
    rows = torch.where(full, rows, j[:keep])
    for t in cache:
        b = t.view(torch.uint8)
        b[:, :, :keep] = b.gather(2, rows[..., None].expand(*rows.shape, b.shape[-1]))
    kept = weights.gather(2, rows)
    weights[:, :, :keep] = kept
    weights[:, :, keep:] = torch.where(full & (j[keep:] < n), 0.0, weights[:, :, keep:])
    return lengths.clamp(max=keep), torch.where(full | (j[:keep] < n), rows, -1).to(torch.int32)


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import chunked_causal_gqa_gb300 as pfa
        cache = pfa.Q4Cache(*s["cache"], case.get("ke", 0), case.get("ve", 0))
        if op == "write":
            where = dict(lengths=s["lengths"]) if "lengths" in s else dict(start_pos=case["start"])
            pfa.cache_write_q4(s["k"], s["v"], cache, **where)
            return s["cache"]
        if op == "read":
            return pfa.cache_read_q4(cache, case["start"], case["stop"], dtype=DTYPES[case["dtype"]])
        if op == "decode":
            o = pfa.decode_attention_q4(s["q"], cache, s["lengths"], weights=s.get("weights"), window=case["window"])
            return [o] + ([s["weights"]] if case["weights"] else [])
        if op == "evict":
            n, rows = pfa.cache_evict_q4(cache, s["weights"], s["lengths"], case["keep"], recent=case["recent"])
            return [n, rows, s["weights"]] + s["cache"]
        return pfa.prefill_attention_q4(s["q"], cache, start_pos=case["start"], window=case["window"])
    k, v, ks, vs = s["cache"]
    ke, ve = case.get("ke", 0), case.get("ve", 0)
    if op == "write":
        batch = "lengths" in s
        first = s["lengths"] - case["T"] if batch else torch.full((1,), case["start"], device=DEV)
        up = (lambda t: t) if batch else (lambda t: t[None])
        _write(up(s["k"]), up(k), up(ks), first, ke)
        _write(up(s["v"]), up(v), up(vs), first, ve)
        return s["cache"]
    if op == "read":
        dt, cut = DTYPES[case["dtype"]], slice(case["start"], case["stop"])
        return _values(k[:, cut], ks[:, cut], ke).to(dt), _values(v[:, cut], vs[:, cut], ve).to(dt)
    if op == "decode":
        T = case["T"]
        pos = s["lengths"][:, None] - T + torch.arange(T, device=DEV)
        o, w = _attention(s["q"], _values(k, ks, ke), _values(v, vs, ve), pos, case["window"])
        return [o.to(s["q"].dtype)] + ([s["weights"].add_(w)] if case["weights"] else [])
    if op == "evict":
        n, rows = _evict(s["cache"], s["weights"], s["lengths"], case["keep"], case["recent"])
        return [n, rows, s["weights"]] + s["cache"]
    T, W = case["T"], case["window"]
    lo = max(0, case["start"] - W + 1) if W else 0
    cut = slice(lo, case["start"] + T)
    pos = case["start"] - lo + torch.arange(T, device=DEV)[None]
    o, _ = _attention(s["q"][None], _values(k[:, cut], ks[:, cut], ke)[None], _values(v[:, cut], vs[:, cut], ve)[None], pos, W)
    return o[0].to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    es = 4 if case.get("dtype") == "f32" else 2
    row = D // 2 + D // GROUP                                   # bytes of a row of K or V of a head
    if op == "write":
        n = case["B"] * case["T"]
        if case["start"] < 0:
            n = sum(min(x, case["T"]) for x in _lengths(case))
        return {"bytes": n * Hkv * 2 * (D * es + row), "flops": 3 * n * Hkv * 2 * D}
    if op == "read":
        n = (case["stop"] - case["start"]) * Hkv * 2
        return {"bytes": n * (D * es + row), "flops": n * D}
    if op == "evict":
        cut = [n for n in _lengths(case) if n > case["keep"]]
        kept = len(cut) * case["keep"]
        # every weight of a sequence that is cut is read, and written as the kept one or as zero
        return {"bytes": Hkv * (8 * sum(cut) + kept * (2 * 2 * row)) + case["B"] * (Hkv * case["keep"] * 4 + 16),
                "flops": 3 * Hkv * sum(cut)}
    lens = _lengths(case) if op == "decode" else [case["start"] + case["T"]]
    T, W = case["T"], case["window"]
    rows = pairs = 0
    for n in lens:
        first = max(0, n - T)
        if W <= 0:
            rows += n
            pairs += (n * (n + 1) - first * (first + 1)) // 2
        else:
            rows += n - max(0, first - W + 1)
            pairs += sum(min(p + 1, W) for p in range(first, n))
    qo = 2 * len(lens) * T * case["H"] * D * es
    return {"bytes": qo + rows * Hkv * (2 * row + (8 if case.get("weights") else 0)), "flops": 4.0 * D * case["H"] * pairs}


# ------------------------------------------------------------------ 64 bits

def _nearest_e4m3(x):
    """Nearest e4m3 value, ties to even, of 64-bit x >= 0; 448 beyond it."""
    _, e = torch.frexp(x)
    steps = torch.tensor([2.0 ** (i - 3) for i in range(-6, 10)], dtype=torch.float64, device=DEV)
    step = steps[(e - 1).clamp(-6, 9).long() + 6]
    return ((x / step).round() * step).clamp(max=448.0)


def _nearest_code(a):
    """Code of the e2m1 magnitude nearest to 64-bit a >= 0, the even code of two."""
    to = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    up = torch.searchsorted(to, a.contiguous()).clamp(max=7)     # first value >= a
    down = (up - 1).clamp(min=0)
    far_up, far_down = to[up] - a, a - to[down]
    take_up = (far_up < far_down) | ((far_up == far_down) & (up % 2 == 0))
    return torch.where(take_up | (a > 6), up, down)


def _exact_write(x, codes, scale, firsts, exponent):
    codes, scale = codes.clone(), scale.double()
    for b, p in enumerate(firsts):
        a, z = max(p, 0), p + x.shape[1]
        if z <= a:
            continue
        y = x[b, a - p:].double().transpose(0, 1) / 2.0 ** exponent           # [Hkv, rows, D]
        g = y.reshape(*y.shape[:2], -1, GROUP)
        s = _nearest_e4m3(g.abs().amax(-1) / torch.full((), 6.0, dtype=torch.float64, device=DEV))
        c = _nearest_code(g.abs() / torch.where(s > 0, s, 1.0)[..., None])
        c = torch.where((s > 0)[..., None], c + 8 * torch.signbit(g).long(), 0).reshape(y.shape)
        codes[b, :, a:z] = (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)
        scale[b, :, a:z] = s
    return codes, scale


def _exact_attention(q, k, v, n, window):
    """q [T, H, D] at positions n - T .., k and v [Hkv, L, D] in 64 bits; a head at a time -> out, weights [Hkv, L]."""
    T, H, D = q.shape
    out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
    weights = torch.zeros(k.shape[:2], dtype=torch.float64, device=DEV)
    first = max(0, n - T)
    if n <= 0:
        return out, weights
    lo = max(0, first - window + 1) if window > 0 else 0
    j = torch.arange(lo, n, device=DEV)
    pos = torch.arange(first, n, device=DEV)[:, None]
    hidden = j > pos
    if window > 0:
        hidden |= j <= pos - window
    for h in range(H):
        g = h // (H // k.shape[0])
        s = q[T - (n - first):, h].double() @ k[g, lo:n].T / math.sqrt(D)
        p = torch.softmax(s.masked_fill_(hidden, float("-inf")), -1)
        out[T - (n - first):, h] = p @ v[g, lo:n]
        weights[g, lo:n] += p.sum(0)
    return out, weights


def _exact_evict(cache, weights, lengths, keep, recent):
    cache, weights = [t.view(torch.uint8).clone() for t in cache], weights.double()
    left = [min(n, keep) for n in lengths]
    rows = torch.full((*weights.shape[:2], keep), -1, dtype=torch.int32, device=DEV)
    for b, n in enumerate(lengths):
        rows[b, :, :left[b]] = torch.arange(left[b], device=DEV)
        if n <= keep:
            continue
        heavy = (-weights[b, :, :n - recent]).sort(dim=-1, stable=True).indices[:, :keep - recent].sort(-1).values
        for h, r in enumerate(heavy):
            r = torch.cat((r, torch.arange(n - recent, n, device=DEV)))
            rows[b, h] = r
            w = weights[b, h, r]
            weights[b, h, :n] = 0
            weights[b, h, :keep] = w
            for t in cache:
                t[b, h, :keep] = t[b, h, r]
    return [torch.tensor(left, device=DEV), rows, weights] + cache[:2] + [t.view(F8).double() for t in cache[2:]]


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case.get("T", 0)
    k, v, ks, vs = s["cache"]
    if op == "evict":
        return _exact_evict(s["cache"], s["weights"], _lengths(case), case["keep"], case["recent"])
    ke, ve = case["ke"], case["ve"]
    if op == "write":
        batch = "lengths" in s
        up = (lambda t: t) if batch else (lambda t: t[None])
        firsts = [n - T for n in _lengths(case)] if batch else [case["start"]]
        kc, kn = _exact_write(up(s["k"]), up(k), up(ks), firsts, ke)
        vc, vn = _exact_write(up(s["v"]), up(v), up(vs), firsts, ve)
        return [kc, vc, kn, vn] if batch else [kc[0], vc[0], kn[0], vn[0]]

    def full(codes, scale, exponent):
        mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
        c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
        return torch.where(c >= 8, -1.0, 1.0) * mag[c % 8] * scale.double().repeat_interleave(GROUP, -1) * 2.0 ** exponent

    if op == "read":
        cut = slice(case["start"], case["stop"])
        return full(k[:, cut], ks[:, cut], ke), full(v[:, cut], vs[:, cut], ve)
    if op == "decode":
        got = [_exact_attention(s["q"][b], full(k[b], ks[b], ke), full(v[b], vs[b], ve), n, case["window"])
               for b, n in enumerate(_lengths(case))]
        out = torch.stack([o for o, _ in got])
        return [out, s["weights"].double() + torch.stack([w for _, w in got])] if case["weights"] else [out]
    return _exact_attention(s["q"], full(k, ks, ke), full(v, vs, ve), case["start"] + T, case["window"])[0]
