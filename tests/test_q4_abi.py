"""Refusals of the operators around the 4-bit cache, on any machine: argument
checks of the C entries (before any device is touched) and of the binding."""
import ctypes

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from chunked_causal_gqa_gb300 import _binding, build
from tests import q4_reference as R

NULL, SHAPE, DTYPE, ALIGN, DEVICE, VALUE, ALIAS, SCRATCH = -1, -2, -3, -4, -5, -8, -9, -10
F32, BF16 = _binding.PFA_F32, _binding.PFA_BF16
GB = 1 << 30
Q, K, V, O, W, LEN, LOUT, ROWS = (i * GB for i in range(1, 9))        # disjoint fake device pointers
K4, V4, KS, VS, WS = (i * GB for i in range(9, 14))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _binding.load()


@pytest.fixture
def last():
    """What a call with nothing wrong gives here: the device check's answer."""
    return DEVICE if not torch.cuda.is_available() else None


def write(lib, k=K, v=V, k4=K4, v4=V4, ks=KS, vs=VS, B=1, T=4, sp=0, ln=None, Hkv=2, D=128, cap=250,
          ke=0, ve=0, dt=BF16, kst=None, vst=None):
    n = Hkv * D
    return lib.pfa_cache_write_q4(k, v, k4, v4, ks, vs, B, T, sp, ln, Hkv, D, cap, ke, ve, dt,
                                  n if kst is None else kst, n if vst is None else vst, None)


def test_write_refusals(lib, last):
    assert write(lib, dt=-1) == DTYPE
    for bad in (dict(D=8), dict(D=24), dict(D=528), dict(Hkv=0), dict(cap=0), dict(cap=2 ** 31), dict(sp=247),
                dict(T=251), dict(B=2), dict(sp=-1), dict(kst=255), dict(vst=8), dict(B=-1, ln=LEN),
                dict(B=2 ** 30, ln=LEN, Hkv=65536)):
        assert write(lib, **bad) == SHAPE, bad
    for bad in (dict(ke=65), dict(ve=-65)):
        assert write(lib, **bad) == VALUE, bad
    for bad in (dict(k=None), dict(v=None), dict(k4=None), dict(vs=None)):
        assert write(lib, **bad) == NULL, bad
    for bad in (dict(k=K + 8), dict(v4=V4 + 8), dict(ks=KS + 4), dict(kst=260), dict(ln=LEN + 2),
                dict(vs=VS + 8, D=512), dict(vs=VS + 1, D=96)):
        assert write(lib, **bad) == ALIGN, bad
    for bad in (dict(k4=V4), dict(k4=K), dict(v=VS), dict(ks=K4 + 8), dict(ks=VS), dict(ln=V4), dict(vs=V4)):
        assert write(lib, **bad) == ALIAS, bad
    assert write(lib, T=0, k=None, v=None, k4=None, v4=None, ks=None, vs=None) == 0
    if last is not None:
        assert write(lib) == last
        assert write(lib, B=3, ln=LEN, ke=64, ve=-64) == last
        assert write(lib, D=80, k4=K4 + 8, ks=KS + 1, vs=VS + 3) == last   # five scales a row


def read(lib, k4=K4, v4=V4, ks=KS, vs=VS, ko=K, vo=V, heads=2, start=3, rows=70, D=128, cap=250, ke=0,
         ve=0, dt=BF16, st=None):
    return lib.pfa_cache_read_q4(k4, v4, ks, vs, ko, vo, heads, start, rows, D, cap, ke, ve, dt,
                                 rows * D if st is None else st, None)


def test_read_refusals(lib, last):
    assert read(lib, dt=2) == DTYPE
    for bad in (dict(heads=-1), dict(start=-1), dict(rows=-1), dict(start=250, rows=7), dict(D=24),
                dict(st=70 * 128 - 8), dict(cap=0), dict(heads=2 ** 45), dict(start=2 ** 62, rows=2 ** 62)):
        assert read(lib, **bad) == SHAPE, bad
    assert read(lib, ke=-70) == VALUE
    for bad in (dict(ko=None), dict(vo=None), dict(v4=None), dict(ks=None)):
        assert read(lib, **bad) == NULL, bad
    for bad in (dict(ko=K + 8), dict(k4=K4 + 4), dict(st=70 * 128 + 4), dict(ks=KS + 2)):
        assert read(lib, **bad) == ALIGN, bad
    for bad in (dict(ko=V), dict(vo=K4 + 256), dict(ko=VS)):
        assert read(lib, **bad) == ALIAS, bad
    assert read(lib, rows=0) == 0 and read(lib, heads=0) == 0
    if last is not None:
        assert read(lib) == last


def decode(lib, q=Q, k4=K4, v4=V4, ks=KS, vs=VS, o=O, wt=W, B=2, T=1, ln=LEN, H=8, Hkv=2, D=128, w=0,
           scale=0.1, dt=BF16, qs=None, os=None, cap=250, ke=0, ve=0, ws=WS, n=GB):
    return lib.pfa_decode_attention_q4(q, k4, v4, ks, vs, o, wt, B, T, ln, H, Hkv, D, w, scale, dt,
                                       H * D if qs is None else qs, H * D if os is None else os,
                                       cap, ke, ve, ws, n, None)


def test_decode_refusals(lib, last):
    n = ctypes.c_size_t(5)
    assert decode(lib, dt=9) == DTYPE
    for bad in (dict(H=6, Hkv=4), dict(H=0), dict(D=64), dict(D=256), dict(H=258, Hkv=2), dict(B=-1),
                dict(T=-1), dict(T=257), dict(cap=0), dict(qs=1000), dict(os=1000)):
        assert decode(lib, **bad) == SHAPE, bad
    for bad in (dict(scale=float("nan")), dict(ke=65), dict(ve=-65), dict(scale=1e30, ke=64)):
        assert decode(lib, **bad) == VALUE, bad
    for bad in (dict(q=None), dict(o=None), dict(ln=None), dict(k4=None), dict(vs=None)):
        assert decode(lib, **bad) == NULL, bad
    for bad in (dict(q=Q + 8), dict(o=O + 2), dict(ln=LEN + 4), dict(ws=WS + 16), dict(qs=1028),
                dict(wt=W + 2), dict(ks=KS + 4)):
        assert decode(lib, **bad) == ALIGN, bad
    for bad in (dict(o=Q), dict(o=K4), dict(o=VS), dict(ln=O), dict(wt=Q), dict(wt=O), dict(wt=VS),
                dict(wt=LEN)):
        assert decode(lib, **bad) == ALIAS, bad
    assert decode(lib, B=0) == 0 and decode(lib, T=0) == 0
    size = lib.pfa_decode_workspace_bytes_q4
    assert size(2, 1, 8, 2, 128, BF16, 250, 1, None) == NULL
    assert size(2, 1, 8, 3, 128, BF16, 250, 1, ctypes.byref(n)) == SHAPE
    assert size(2, 1, 8, 2, 128, BF16, 0, 1, ctypes.byref(n)) == SHAPE
    assert size(2, 300, 8, 2, 128, BF16, 250, 1, ctypes.byref(n)) == SHAPE
    assert size(0, 1, 8, 2, 128, BF16, 250, 1, ctypes.byref(n)) == 0
    assert n.value == 0
    if last is not None:
        assert decode(lib) == last and decode(lib, wt=None) == last
        assert size(2, 1, 8, 2, 128, BF16, 250, 1, ctypes.byref(n)) == last


def prefill(lib, q=Q, k4=K4, v4=V4, ks=KS, vs=VS, o=O, T=100, sp=7, H=8, Hkv=2, D=128, w=0,
            scale=0.1, dt=BF16, row=None, cap=250, ke=0, ve=0, ws=WS, n=GB):
    return lib.pfa_prefill_attention_q4(q, k4, v4, ks, vs, o, T, sp, H, Hkv, D, w, scale, dt,
                                        H * D if row is None else row, cap, ke, ve, ws, n, None)


def test_prefill_refusals(lib, last):
    n = ctypes.c_size_t(5)
    assert prefill(lib, dt=9) == DTYPE
    for bad in (dict(H=6, Hkv=4), dict(D=64), dict(T=-1), dict(sp=-1), dict(sp=157), dict(cap=100),
                dict(row=1000), dict(H=258, Hkv=2)):
        assert prefill(lib, **bad) == SHAPE, bad
    for bad in (dict(scale=float("inf")), dict(ke=99), dict(scale=-1e25, ke=64)):
        assert prefill(lib, **bad) == VALUE, bad
    for bad in (dict(q=None), dict(o=None), dict(ks=None)):
        assert prefill(lib, **bad) == NULL, bad
    for bad in (dict(q=Q + 8), dict(ws=WS + 128), dict(row=1028), dict(v4=V4 + 8)):
        assert prefill(lib, **bad) == ALIGN, bad
    for bad in (dict(o=Q + 256), dict(o=V4)):
        assert prefill(lib, **bad) == ALIAS, bad
    assert prefill(lib, T=0, q=None, o=None) == 0
    size = lib.pfa_prefill_workspace_bytes_q4
    assert size(100, 7, 8, 2, 128, 0, BF16, None) == NULL
    assert size(100, -7, 8, 2, 128, 0, BF16, ctypes.byref(n)) == SHAPE
    assert size(0, 7, 8, 2, 128, 0, BF16, ctypes.byref(n)) == 0
    assert n.value == 0
    if last is not None:
        assert prefill(lib) == last


def evict(lib, k4=K4, v4=V4, ks=KS, vs=VS, wt=W, B=2, ln=LEN, Hkv=2, D=128, cap=250, keep=50, recent=7,
          lo=LOUT, ro=ROWS):
    return lib.pfa_cache_evict_q4(k4, v4, ks, vs, wt, B, ln, Hkv, D, cap, keep, recent, lo, ro, None)


def test_evict_refusals(lib, last):
    for bad in (dict(B=-1), dict(Hkv=0), dict(D=24), dict(cap=0), dict(keep=0), dict(keep=251), dict(recent=-1),
                dict(recent=51), dict(B=2 ** 30, Hkv=65536)):
        assert evict(lib, **bad) == SHAPE, bad
    for bad in (dict(k4=None), dict(wt=None), dict(ln=None), dict(lo=None), dict(ro=None), dict(vs=None)):
        assert evict(lib, **bad) == NULL, bad
    for bad in (dict(k4=K4 + 8), dict(wt=W + 2), dict(ln=LEN + 4), dict(lo=LOUT + 4), dict(ro=ROWS + 2),
                dict(ks=KS + 4)):
        assert evict(lib, **bad) == ALIGN, bad
    for bad in (dict(wt=K4), dict(ro=W), dict(lo=W), dict(ln=ROWS), dict(lo=LEN + 8), dict(ro=KS), dict(lo=ROWS),
                dict(k4=V4), dict(ks=VS), dict(lo=VS)):
        assert evict(lib, **bad) == ALIAS, bad
    assert evict(lib, B=0) == 0
    if last is not None:
        assert evict(lib) == last
        assert evict(lib, lo=LEN) == last                              # lengths in place
        assert evict(lib, keep=250, recent=250) == last


def test_binding_checks_tensors():
    cache = pkg.Q4Cache(*R.make_cache(2, 100, 128))
    batch = pkg.Q4Cache(*R.make_cache(2, 100, 128, batch=3))
    q, k = torch.zeros(3, 1, 8, 128), torch.zeros(3, 1, 2, 128)
    n = torch.ones(3, dtype=torch.int64)
    w = torch.zeros(3, 2, 100)
    bad = [
        lambda: pkg.cache_write_q4(k, k, batch),                            # neither position
        lambda: pkg.cache_write_q4(k, k, cache, lengths=n),                 # a slot's cache
        lambda: pkg.cache_write_q4(k[:2], k[:2], batch, lengths=n[:2]),
        lambda: pkg.cache_write_q4(k, k[..., :64], batch, lengths=n),
        lambda: pkg.cache_write_q4(k.half(), k.half(), batch, lengths=n),
        lambda: pkg.cache_write_q4(k, k, batch[:4], lengths=n),             # no exponents
        lambda: pkg.cache_write_q4(k, k, batch, lengths=n),                 # CPU tensors
        lambda: pkg.cache_read_q4(cache, 5, 3),
        lambda: pkg.cache_read_q4(cache, 0, 101),
        lambda: pkg.cache_read_q4(cache, dtype=torch.float16),
        lambda: pkg.cache_read_q4(cache._replace(k_scale=cache.k_scale[:, :1])),
        lambda: pkg.cache_read_q4(cache._replace(k_scale=cache.k_scale.view(torch.uint8))),
        lambda: pkg.cache_read_q4(cache._replace(k=cache.k.view(torch.int8))),
        lambda: pkg.cache_read_q4(cache._replace(k=cache.k.transpose(0, 1))),
        lambda: pkg.decode_attention_q4(q, cache, n),
        lambda: pkg.decode_attention_q4(q[..., :64], batch, n),
        lambda: pkg.decode_attention_q4(q, batch, n.float()),
        lambda: pkg.decode_attention_q4(q, batch, n, out=q.bfloat16()),
        lambda: pkg.decode_attention_q4(q, batch, n, weights=w[:, :, :50]),
        lambda: pkg.decode_attention_q4(q, batch, n, weights=w.double()),
        lambda: pkg.decode_attention_q4(q, batch, n),                       # CPU tensors
        lambda: pkg.prefill_attention_q4(q[:, 0], batch, start_pos=0),
        lambda: pkg.prefill_attention_q4(q[:, 0], cache, start_pos=0),      # CPU tensors
        lambda: pkg.cache_evict_q4(cache, w[0], n[:1], 5),
        lambda: pkg.cache_evict_q4(batch, w, n, 0),
        lambda: pkg.cache_evict_q4(batch, w, n, 101),
        lambda: pkg.cache_evict_q4(batch, w, n, 5, recent=6),
        lambda: pkg.cache_evict_q4(batch, w, n, 5, lengths_out=n.int()),
        lambda: pkg.cache_evict_q4(batch, w, n, 5, rows_out=torch.zeros(3, 2, 4, dtype=torch.int32)),
        lambda: pkg.cache_evict_q4(batch, w, n, 5),                         # CPU tensors
        lambda: pkg.q4_cache(2, 100, 100, device="cpu"),
        lambda: pkg.q4_cache(2, 100, 128, k_exponent=65, device="cpu"),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    c = pkg.q4_cache(2, 100, 64, batch=3, v_exponent=-2, device="cpu")
    assert c.k.shape == (3, 2, 100, 32) and c.k_scale.shape == (3, 2, 100, 4)
    assert c.slot(1).k.data_ptr() == c.k[1].data_ptr() and c.slot(1).v_exponent == -2


def test_reference_forms_agree_with_hand_worked_values():
    x = torch.zeros(1, 16)
    x[0, :10] = torch.tensor([6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1])
    c, s = R.quantise(x, 0)
    assert s.tolist() == [[0x38]]                                            # 1.0
    assert c[0, :5].tolist() == [0xf7, 0x20, 0x42, 0x64, 0xf6]
    assert R.values(c, s.view(R.F8))[0, :10].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4, -6]
    # 6.375 / 6 = 1.0625 lies between 1 and 1.125, and 1 is the even one
    assert R.quantise(torch.full((1, 16), 6.375), 0)[1].item() == 0x38
    assert R.quantise(torch.full((1, 16), 6.376), 0)[1].item() == 0x39
    assert R.quantise(torch.full((1, 16), 6.376 * 2 ** 5), 5)[1].item() == 0x39
    x[0, 3] = float("inf")
    c, s = R.quantise(x, 0)
    assert s.item() == 0x7f and not c.any()
    table = torch.tensor(R._e4m3(), dtype=torch.float64)
    assert torch.equal(torch.arange(127, dtype=torch.uint8).view(R.F8).double(), table)
    assert R.evict(torch.tensor([[1.0, 3.0, 3.0, 0.5, 9.0, 0.0]]), 6, 4, 1) == [[1, 2, 4, 5]]
    assert R.evict(torch.tensor([[3.0, 3.0, 3.0, 0.5]]), 4, 2, 0) == [[0, 1]]
    k = torch.tensor([0.0, 1.0, 2.0]).log().clamp(min=-1e9).double()         # weights 0 : 1 : 2
    kv = torch.zeros(1, 3, 16, dtype=torch.float64)
    kv[0, :, 0] = k
    v = torch.arange(48, dtype=torch.float64).view(1, 3, 16)
    q = torch.zeros(1, 1, 16)
    q[0, 0, 0] = 1
    out, _, acc, _ = R.attention(q, kv, v, 3, 0, 1.0, torch.float32)
    assert torch.allclose(out[0, 0], (v[0, 1] + 2 * v[0, 2]) / 3)
    assert torch.allclose(acc[0], torch.tensor([0.0, 1 / 3, 2 / 3], dtype=torch.float64))
