"""Cases of the operators around an 8-bit KV cache: norm and rotation of queries and keys, the cache's write
and read-back, and the attention over it (single tokens of a batch, and chunks of one sequence).

The cache holds K and V as e4m3 values with one power-of-two fp32 scale for each head and block of `block`
tokens.  `run` computes an operator in elementary torch operations; with `own` set it calls the package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: eight sequences, one new token each
        dict(name="norm_rope_step", op="norm_rope", B=8, T=1, H=32, Hkv=8, D=128, dtype="bf16", rot=128,
             interleaved=False, norm=True, start=-1, mix=1),
        # a prefill chunk deep in a 64k prompt, columns of one projection buffer, K written into its cache rows
        dict(name="norm_rope_chunk", op="norm_rope", B=1, T=2048, H=32, Hkv=8, D=128, dtype="bf16", rot=128,
             interleaved=False, norm=True, start=61440, mix=0),
        # an odd prompt length, wide heads, a quarter of each head rotated in neighbouring pairs
        dict(name="norm_rope_f32_odd", op="norm_rope", B=1, T=1358, H=8, Hkv=2, D=512, dtype="f32", rot=128,
             interleaved=True, norm=True, start=0, mix=0),
        # the new token of 32 sequences goes into the 8-bit cache at 32 different positions
        dict(name="write_step", op="write", B=32, T=1, Hkv=8, D=128, dtype="bf16", block=64, cap=8192, start=-1, mix=2),
        # a prefill chunk goes into the cache from the middle of a block on
        dict(name="write_chunk", op="write", B=1, T=2048, Hkv=8, D=128, dtype="bf16", block=64, cap=65536,
             start=61445, mix=0),
        # the whole 64k cache of a layer read back
        dict(name="read_64k", op="read", Hkv=8, D=128, dtype="bf16", block=64, cap=65536, start=0, stop=63488),
        # an odd range of rows of a wide-head layer, small blocks, fp32
        dict(name="read_f32_odd", op="read", Hkv=2, D=512, dtype="f32", block=16, cap=8192, start=5003, stop=8191),
        # one sequence at a full 128k context: nothing but the cache's bytes counts
        dict(name="decode_one_128k", op="decode", B=1, T=1, H=32, Hkv=8, D=128, dtype="bf16", block=64,
             cap=131072, window=0, longest=131072, mix=3),
        # a served batch of uneven sequences, some slots empty
        dict(name="decode_batch", op="decode", B=32, T=1, H=32, Hkv=8, D=128, dtype="bf16", block=64, cap=8192,
             window=0, longest=8192, mix=4),
        # three drafted tokens of four short sequences, wide heads, sliding window, fp32
        dict(name="decode_f32_draft", op="decode", B=4, T=3, H=8, Hkv=2, D=512, dtype="f32", block=32, cap=2048,
             window=1024, longest=1358, mix=5),
        # the steady prefill chunk of a 64k prompt
        dict(name="prefill_64k", op="prefill", T=2048, H=32, Hkv=8, D=128, dtype="bf16", block=64, cap=65536,
             window=0, start=61440),
        # the last, short chunk of a 64k prompt
        dict(name="prefill_64k_t128", op="prefill", T=128, H=32, Hkv=8, D=128, dtype="bf16", block=64, cap=65536,
             window=0, start=63360),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "write", "read", "decode", "decode", "prefill"))
    D = rng.choice((128, 128, 512))
    Hkv = rng.choice((1, 2, 4, 8)) if D == 128 else rng.choice((1, 2, 4))
    G = rng.choice((1, 2, 4, 5, 8))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    block = rng.choice((16, 32, 64, 128))
    if op == "norm_rope":
        batch = rng.random() < 0.5
        T = rng.randint(1, 4) if batch else _log(rng, 1, 8192)
        return dict(op=op, B=_log(rng, 1, 64) if batch else 1, T=T, H=Hkv * G, Hkv=Hkv, D=D, dtype=dtype,
                    rot=rng.choice((D, D, D // 2, D // 4, 0)), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.8, start=-1 if batch else _log(rng, 1, 500000) - 1, mix=rng.randrange(1000))
    if op == "write":
        batch = rng.random() < 0.5
        T = rng.randint(1, 8) if batch else _log(rng, 1, 8192)
        start = -1 if batch else _log(rng, 1, 50000) - 1
        cap = block * rng.randint(8, 4096 // block) if batch else -(-(start + T) // block) * block + block
        return dict(op=op, B=_log(rng, 1, 64) if batch else 1, T=T, Hkv=Hkv, D=D, dtype=dtype, block=block, cap=cap,
                    start=start, mix=rng.randrange(1000))
    if op == "read":
        cap = block * _log(rng, 1, 65536 // block)
        start = rng.randrange(cap)
        return dict(op=op, Hkv=Hkv, D=D, dtype=dtype, block=block, cap=cap, start=start,
                    stop=rng.randint(start + 1, cap))
    window = rng.choice((0, 0, 0, 1024, 333))
    if op == "decode":
        B = _log(rng, 1, 48)
        cap = block * max(1, _log(rng, 64, 131072 if B < 3 else 262144 // B) // block)
        return dict(op=op, B=B, T=rng.choice((1, 1, 1, 2, 4, 7)), H=Hkv * G, Hkv=Hkv, D=D, dtype=dtype, block=block,
                    cap=cap, window=window, longest=rng.randint(max(1, cap // 2), cap), mix=rng.randrange(1000))
    H = Hkv * min(G, 4)
    T = _log(rng, 1, 2048)
    start = _log(rng, 1, 30000) - 1
    return dict(op=op, T=T, H=H, Hkv=Hkv, D=D, dtype=dtype, block=block, cap=-(-(start + T) // block) * block,
                window=window, start=start)


def _lengths(case):
    """Lengths of the batch's sequences after the new tokens: uneven, the first the longest, one slot empty."""
    r = random.Random(case["mix"])
    B, T = case["B"], case["T"]
    if case["op"] == "norm_rope":
        return [r.randint(T, 131072) for _ in range(B)]
    most = case.get("longest", case["cap"])
    n = [r.randint(min(T, most), most) for _ in range(B)]
    n[0] = most
    if B > 4:
        n[3] = 0
    return n


# ------------------------------------------------------------------ inputs

def _randn(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std)


def _pow2_scale(amax):
    """The smallest power of two s >= 2**-126 with amax / s <= 448 (0 where amax is 0), from the number's own bits."""
    m, e = torch.frexp(amax)                                    # 448 = 0.875 * 2**9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    s = ((e + 127) << 23).to(torch.int32).view(torch.float32)
    return torch.where(amax > 0, s, torch.zeros_like(amax))


def _filled(shape, block, gen):
    """A cache tensor of `shape` (..., cap, D) and its scales: normal values whose size changes from block to block."""
    *lead, cap, D = shape
    nb = cap // block
    size = torch.randint(-3, 2, (*lead, nb, 1, 1), generator=gen, device=DEV).float().exp2_()
    x = _randn((*lead, nb, block, D), gen).mul_(size)
    scale = _pow2_scale(x.abs().amax((-1, -2)))
    codes = x.div_(scale[..., None, None]).to(F8)
    return codes.reshape(shape), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, D, dt = case["op"], case["D"], DTYPES[case["dtype"]]
    s = dict(case=case)
    batch = case.get("B", 1) > 1 or case.get("start", -1) < 0 or op == "decode"
    if op in ("norm_rope", "write", "decode") and batch:
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int64, device=DEV)
    if op == "norm_rope":
        B, T, H, Hkv = case["B"], case["T"], case["H"], case["Hkv"]
        qkv = _randn((B, T, H + 2 * Hkv, D), gen).to(dt)       # one projection's output: q, k and v columns
        qkv = qkv if batch else qkv[0]
        s["q"], s["k"] = qkv[..., :H, :], qkv[..., H:H + Hkv, :]
        s["q_weight"] = (1 + _randn((D,), gen, 0.1)).to(dt) if case["norm"] else None
        s["k_weight"] = (1 + _randn((D,), gen, 0.1)).to(dt) if case["norm"] else None
        R = case["rot"]
        s["inv_freq"] = (1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)) if R else None
        if not batch:                                          # a chunk's keys land in rows of the layer's cache
            cache = torch.zeros((Hkv, T + 64, D), dtype=dt, device=DEV)
            s["k_out"] = cache[:, 64:64 + T].transpose(0, 1)
        return s
    if op == "write":
        B, T, Hkv = case["B"], case["T"], case["Hkv"]
        kv = _randn((B, T, 2 * Hkv, D), gen, 2.0).to(dt)
        s["k"], s["v"] = kv[:, :, :Hkv], kv[:, :, Hkv:]
        shape = (B, Hkv, case["cap"], D)
        if not batch:
            s["k"], s["v"], shape = s["k"][0], s["v"][0], shape[1:]
        s["cache"] = [t for _ in "kv" for t in _filled(shape, case["block"], gen)]
    elif op == "read":
        s["cache"] = [t for _ in "kv" for t in _filled((case["Hkv"], case["cap"], D), case["block"], gen)]
    else:
        shape = (case["Hkv"], case["cap"], D)
        qshape = (case["T"], case["H"], D)
        if op == "decode":
            shape, qshape = (case["B"], *shape), (case["B"], *qshape)
        s["q"] = _randn(qshape, gen).to(dt)
        s["cache"] = [t for _ in "kv" for t in _filled(shape, case["block"], gen)]
    s["cache"] = [s["cache"][0], s["cache"][2], s["cache"][1], s["cache"][3]]     # k, v, k_scale, v_scale
    return s


# ------------------------------------------------------------------ plain forms

def _positions(s, T):
    """Position of each row: [T], or [B, T] where the lengths are on the device."""
    t = torch.arange(T, device=DEV)
    if "lengths" in s:
        return s["lengths"][:, None] - T + t
    return s["case"]["start"] + t


def _norm_rope(x, weight, inv_freq, pos, interleaved):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    if inv_freq is not None:
        a = pos.double()[..., None, None] * inv_freq
        c, n = a.cos().float(), a.sin().float()
        R = 2 * inv_freq.numel()
        r, rest = y[..., :R], y[..., R:]
        if interleaved:
            p, q = r[..., 0::2], r[..., 1::2]
            r = torch.stack((p * c - q * n, p * n + q * c), -1).flatten(-2)
        else:
            p, q = r[..., :R // 2], r[..., R // 2:]
            r = torch.cat((p * c - q * n, p * n + q * c), -1)
        y = torch.cat((r, rest), -1)
    return torch.where((pos >= 0)[..., None, None], y, torch.zeros_like(y)).to(x.dtype)


def _write(x, codes, scale, first, T, block):
    """Writes x [B, T, Hkv, D] at rows first.. of codes [B, Hkv, cap, D]; `first` [B].  In place."""
    raw = codes.view(torch.uint8)
    last = first + T
    low = first.clamp(min=0) // block
    most = (T + block - 2) // block + 1                        # blocks that T rows can touch
    # a sequence that touches fewer has its last one more than once, with the same values
    blocks = torch.minimum(low[:, None] + torch.arange(most, device=DEV), (last - 1).clamp(min=0)[:, None] // block)
    rows = blocks[..., None] * block + torch.arange(block, device=DEV)            # [B, most, block]
    t = rows - first[:, None, None]
    new = (t >= 0) & (t < T)
    hit = new.any(2)[..., None]
    live = (t < 0) & hit
    b = torch.arange(len(first), device=DEV)[:, None]
    old, s_old = raw[b[..., None], :, rows], scale[b, :, blocks]                  # [B, most, block, Hkv, D], [B, most, Hkv]
    src = x[b[..., None], t.clamp(0, T - 1)].float()
    amax = torch.where(new[..., None, None], src, 0.0).abs().amax((2, 4))
    keep = torch.where(live.any(2)[..., None], s_old, 0.0)
    s_new = torch.maximum(keep, _pow2_scale(amax))
    inv = torch.where(s_new > 0, 1 / s_new, 0.0)
    was = (old.view(F8).float() * (keep * inv)[:, :, None, :, None]).to(F8).view(torch.uint8)
    now = (src * inv[:, :, None, :, None]).to(F8).view(torch.uint8)
    raw[b[..., None], :, rows] = torch.where(new[..., None, None], now, torch.where(live[..., None, None], was, old))
    scale[b, :, blocks] = torch.where(hit, s_new, s_old)


def _values(codes, scale, block):
    """What the cache stands for, fp32: [..., cap, D]."""
    return (codes.float().unflatten(-2, (-1, block)) * scale[..., None, None]).flatten(-3, -2)


def _attention(q, k, v, pos, window):
    """q [B, T, H, D], k and v [B, Hkv, L, D] fp32, pos [B, T] -> fp32 [B, T, H, D]."""
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
    o = s.reshape(B, Hkv, -1, L) @ v
    o = o.reshape(B, Hkv, -1, T, D) / torch.where(n > 0, n, torch.ones_like(n))
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, H, D)


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import chunked_causal_gqa_gb300 as pfa
        where = dict(lengths=s["lengths"]) if "lengths" in s else dict(start_pos=case.get("start"))
        if op == "norm_rope":
            return pfa.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["inv_freq"], eps=1e-6,
                                    interleaved=case["interleaved"], k_out=s.get("k_out"), **where)
        cache = pfa.Q8Cache(*s["cache"])
        if op == "write":
            pfa.cache_write_q8(s["k"], s["v"], cache, **where)
            return s["cache"]
        if op == "read":
            return pfa.cache_read_q8(cache, case["start"], case["stop"], dtype=DTYPES[case["dtype"]])
        if op == "decode":
            return pfa.decode_attention_q8(s["q"], cache, s["lengths"], window=case["window"])
        return pfa.prefill_attention_q8(s["q"], cache, start_pos=case["start"], window=case["window"])
    if op == "norm_rope":
        pos = _positions(s, case["T"])
        q = _norm_rope(s["q"], s["q_weight"], s["inv_freq"], pos, case["interleaved"])
        k = _norm_rope(s["k"], s["k_weight"], s["inv_freq"], pos, case["interleaved"])
        if "k_out" in s:
            k = s["k_out"].copy_(k)
        return q, k
    k, v, ks, vs = s["cache"]
    block = case["block"]
    if op == "write":
        batch = k.dim() == 4
        first = s["lengths"] - case["T"] if batch else torch.full((1,), case["start"], device=DEV)
        for_one = (lambda t: t) if batch else (lambda t: t[None])
        _write(for_one(s["k"]), for_one(k), for_one(ks), first, case["T"], block)
        _write(for_one(s["v"]), for_one(v), for_one(vs), first, case["T"], block)
        return s["cache"]
    if op == "read":
        dt, a, b = DTYPES[case["dtype"]], case["start"], case["stop"]
        lo, hi = a // block, -(-b // block)
        cut = slice(a - lo * block, b - lo * block)
        one = lambda c, n: _values(c[:, lo * block:hi * block], n[:, lo:hi], block)[:, cut].to(dt).contiguous()  # noqa: E731
        return one(k, ks), one(v, vs)
    if op == "decode":
        o = _attention(s["q"], _values(k, ks, block), _values(v, vs, block), _positions(s, case["T"]), case["window"])
        return o.to(s["q"].dtype)
    lo = max(0, case["start"] - case["window"] + 1) // block if case["window"] else 0
    k, v = _values(k[:, lo * block:], ks[:, lo:], block), _values(v[:, lo * block:], vs[:, lo:], block)
    pos = _positions(s, case["T"])[None] - lo * block
    return _attention(s["q"][None], k[None], v[None], pos, case["window"])[0].to(s["q"].dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, D = case["op"], case["D"]
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "norm_rope":
        n = case["B"] * case["T"] * (case["H"] + case["Hkv"]) * D
        return {"bytes": 2 * n * es + 2 * D * es + 4 * case["rot"], "flops": 8 * n}
    if op == "write":
        n = case["B"] * case["T"] * case["Hkv"] * D * 2
        if "start" in case and case["start"] < 0:
            n = sum(min(x, case["T"]) for x in _lengths(case)) * case["Hkv"] * D * 2
        return {"bytes": n * (es + 1) + n // (D * case["block"]) * 4, "flops": 3 * n}
    if op == "read":
        n = (case["stop"] - case["start"]) * case["Hkv"] * D * 2
        return {"bytes": n * (es + 1), "flops": n}
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
    kv = rows * case["Hkv"] * 2 * (D + 4.0 / case["block"])
    return {"bytes": qo + kv, "flops": 4.0 * D * case["H"] * pairs}


# ------------------------------------------------------------------ 64 bits

def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, of 64-bit x within +-448."""
    _, e = torch.frexp(x)
    step = torch.tensor([2.0 ** (i - 3) for i in range(-6, 9)], dtype=torch.float64, device=DEV)[(e - 1).clamp(-6, 8).long() + 6]
    return (x / step).round() * step


def _exact_write(x, codes, scale, firsts, T, block):
    codes, scale = codes.double(), scale.double()
    powers = torch.tensor([2.0 ** i for i in range(-126, 128)], dtype=torch.float64, device=DEV)
    cap = codes.shape[-2]
    for b, p in enumerate(firsts):
        a, z = max(p, 0), p + T
        if z <= a or z > cap:
            continue
        for c in range(a // block, (z - 1) // block + 1):
            lo, hi = max(a, c * block), min(z, (c + 1) * block)
            new = x[b, lo - p:hi - p].double().transpose(0, 1)                   # [Hkv, rows, D]
            ratio = new.abs().amax((1, 2)) / 448
            need = torch.where(ratio > 0, powers[torch.searchsorted(powers, ratio)], ratio)
            had = scale[b, :, c] if lo > c * block else torch.zeros_like(need)
            to = torch.maximum(had, need)
            div = torch.where(to > 0, to, torch.ones_like(to))[:, None, None]
            if lo > c * block:
                codes[b, :, c * block:lo] = _round_e4m3(codes[b, :, c * block:lo] * had[:, None, None] / div)
            codes[b, :, lo:hi] = _round_e4m3(new / div)
            scale[b, :, c] = to
    return codes, scale


def _exact_attention(q, k, v, n, window):
    """q [T, H, D] at positions n - T .., k and v [Hkv, L, D] in 64 bits; a head at a time."""
    T, H, D = q.shape
    out = torch.zeros(T, H, D, dtype=torch.float64, device=DEV)
    first = max(0, n - T)
    if n <= 0:
        return out
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
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, T, D = case["op"], case.get("T", 0), case["D"]
    if op == "norm_rope":
        n = s["lengths"][:, None] - T if "lengths" in s else case["start"]
        pos = (n + torch.arange(T, device=DEV)).double()
        R = case["rot"]
        got = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            if w is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            if R:
                i = torch.arange(0, R, 2, device=DEV) if case["interleaved"] else torch.arange(R // 2, device=DEV)
                j = i + 1 if case["interleaved"] else i + R // 2
                turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[..., None] * s["inv_freq"])
                z = torch.complex(x[..., i], x[..., j]) * turn[..., None, :]
                x = x.clone()
                x[..., i], x[..., j] = z.real, z.imag
            got.append(torch.where((pos >= 0)[..., None, None], x, 0.0))
        return tuple(got)
    k, v, ks, vs = s["cache"]
    block = case["block"]
    if op == "write":
        batch = k.dim() == 4
        up = (lambda t: t) if batch else (lambda t: t[None])
        firsts = [n - T for n in _lengths(case)] if batch else [case["start"]]
        kc, kn = _exact_write(up(s["k"]), up(k), up(ks), firsts, T, block)
        vc, vn = _exact_write(up(s["v"]), up(v), up(vs), firsts, T, block)
        return [kc, vc, kn, vn] if batch else [kc[0], vc[0], kn[0], vn[0]]
    full = lambda c, n: c.double() * n.double().repeat_interleave(block, -1)[..., None]  # noqa: E731
    if op == "read":
        return full(k, ks)[:, case["start"]:case["stop"]], full(v, vs)[:, case["start"]:case["stop"]]
    if op == "decode":
        return torch.stack([_exact_attention(s["q"][b], full(k[b], ks[b]), full(v[b], vs[b]), n, case["window"])
                            for b, n in enumerate(_lengths(case))])
    return _exact_attention(s["q"], full(k, ks), full(v, vs), case["start"] + T, case["window"])
