"""Refusals of the operators around the 8-bit cache, on any machine: argument
checks of the C entries (before any device is touched) and of the binding."""
import ctypes

import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from chunked_causal_gqa_gb300 import _binding, build
from tests import q8_reference as R

NULL, SHAPE, DTYPE, ALIGN, DEVICE, VALUE, ALIAS, SCRATCH = -1, -2, -3, -4, -5, -8, -9, -10
F32, BF16 = _binding.PFA_F32, _binding.PFA_BF16
GB = 1 << 30
Q, K, QO, KO, W, FR, LEN = (i * GB for i in range(1, 8))        # disjoint fake device pointers
K8, V8, KS, VS, WS = (i * GB for i in range(8, 13))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _binding.load()


@pytest.fixture
def last():
    """What a call with nothing wrong gives here: the device check's answer."""
    return DEVICE if not torch.cuda.is_available() else None


def norm(lib, q=Q, k=K, qo=QO, ko=KO, B=1, T=4, sp=0, ln=None, H=8, Hkv=2, D=128, qw=W, kw=W,
         eps=1e-6, off=0.0, fr=FR, rot=128, inter=0, dt=BF16, qs=None, ks=None, qos=None, kos=None,
         koh=None):
    qs, qos = (H * D if x is None else x for x in (qs, qos))
    ks, kos = (Hkv * D if x is None else x for x in (ks, kos))
    return lib.pfa_qk_norm_rope(q, k, qo, ko, B, T, sp, ln, H, Hkv, D, qw, kw, eps, off, fr, rot,
                                inter, dt, qs, ks, qos, kos, D if koh is None else koh, None)


def test_norm_rope_refusals(lib, last):
    assert norm(lib, dt=5) == DTYPE
    for bad in (dict(D=136, rot=16), dict(D=528), dict(D=0), dict(rot=8), dict(rot=144),
                dict(rot=-16), dict(H=0), dict(Hkv=-1), dict(T=-1), dict(sp=-1), dict(B=2),
                dict(sp=2 ** 31), dict(qs=8 * 128 - 8), dict(ks=128), dict(qos=0), dict(koh=64),
                dict(kos=130 * 8, koh=1024, T=9)):                 # tokens and heads interleave
        assert norm(lib, **bad) == SHAPE, bad
    for bad in (dict(eps=float("nan")), dict(eps=-1.0), dict(off=float("inf"))):
        assert norm(lib, **bad) == VALUE, bad
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(fr=None)):
        assert norm(lib, **bad) == NULL, bad
    for bad in (dict(q=Q + 8), dict(ko=KO + 2), dict(qw=W + 4), dict(fr=FR + 4), dict(ln=LEN + 4),
                dict(qs=8 * 128 + 4), dict(koh=132, kos=2 * 132 + 4)):
        assert norm(lib, **bad) == ALIGN, bad
    for bad in (dict(qo=Q + 16), dict(qo=K), dict(ko=Q), dict(ko=QO), dict(ko=K + 256),
                dict(qo=Q, qos=9 * 128), dict(qw=QO), dict(fr=KO), dict(ln=QO, sp=0)):
        assert norm(lib, **bad) == ALIAS, bad
    assert norm(lib, T=0, q=None, k=None, qo=None, ko=None) == 0
    assert norm(lib, B=0, ln=LEN) == 0
    if last is not None:
        assert norm(lib) == last
        assert norm(lib, qw=None, kw=None, fr=None, rot=0) == last
        assert norm(lib, qo=Q, ko=K) == last                       # in place
        row = 12 * 128                                             # columns of one buffer, in place
        assert norm(lib, k=Q + 8 * 256, qo=Q, ko=Q + 8 * 256, qs=row, ks=row, qos=row, kos=row) == last
        assert norm(lib, k=Q + 8 * 256 - 16, qo=Q, ko=KO, qs=row, ks=row, qos=row) == ALIAS
        assert norm(lib, kos=128, koh=512 * 128) == last           # rows of a cache


def write(lib, k=K, v=Q, k8=K8, v8=V8, ks=KS, vs=VS, B=1, T=4, sp=0, ln=None, Hkv=2, D=128, cap=256,
          block=64, dt=BF16, kst=None, vst=None):
    n = Hkv * D
    return lib.pfa_cache_write_q8(k, v, k8, v8, ks, vs, B, T, sp, ln, Hkv, D, cap, block, dt,
                                  n if kst is None else kst, n if vst is None else vst, None)


def test_write_refusals(lib, last):
    assert write(lib, dt=-1) == DTYPE
    for bad in (dict(D=8), dict(D=520), dict(Hkv=0), dict(block=48), dict(block=256), dict(cap=250),
                dict(cap=0), dict(sp=253), dict(T=257), dict(B=2), dict(sp=-1), dict(kst=255),
                dict(vst=8), dict(B=-1, ln=LEN), dict(B=2 ** 30, ln=LEN, Hkv=65536)):
        assert write(lib, **bad) == SHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(k8=None), dict(vs=None)):
        assert write(lib, **bad) == NULL, bad
    for bad in (dict(k=K + 8), dict(v8=V8 + 8), dict(ks=KS + 2), dict(kst=260), dict(ln=LEN + 2)):
        assert write(lib, **bad) == ALIGN, bad
    for bad in (dict(k8=V8), dict(k8=K), dict(v=VS), dict(ks=K8 + 4), dict(ks=VS), dict(ln=V8)):
        assert write(lib, **bad) == ALIAS, bad
    assert write(lib, T=0, k=None, v=None, k8=None, v8=None, ks=None, vs=None) == 0
    if last is not None:
        assert write(lib) == last
        assert write(lib, B=3, ln=LEN, sp=0) == last


def read(lib, k8=K8, v8=V8, ks=KS, vs=VS, ko=KO, vo=QO, heads=2, start=3, rows=70, D=128, cap=256,
         block=64, dt=BF16, st=None):
    return lib.pfa_cache_read_q8(k8, v8, ks, vs, ko, vo, heads, start, rows, D, cap, block, dt,
                                 rows * D if st is None else st, None)


def test_read_refusals(lib, last):
    assert read(lib, dt=2) == DTYPE
    for bad in (dict(heads=-1), dict(start=-1), dict(rows=-1), dict(start=250, rows=7), dict(D=24),
                dict(st=70 * 128 - 8), dict(block=1), dict(cap=100), dict(heads=2 ** 45),
                dict(start=2 ** 62, rows=2 ** 62)):
        assert read(lib, **bad) == SHAPE, bad
    for bad in (dict(ko=None), dict(vo=None), dict(v8=None), dict(ks=None)):
        assert read(lib, **bad) == NULL, bad
    for bad in (dict(ko=KO + 8), dict(k8=K8 + 4), dict(st=70 * 128 + 4)):
        assert read(lib, **bad) == ALIGN, bad
    for bad in (dict(ko=QO), dict(vo=K8 + 256), dict(ko=VS)):
        assert read(lib, **bad) == ALIAS, bad
    assert read(lib, rows=0) == 0 and read(lib, heads=0) == 0
    if last is not None:
        assert read(lib) == last


def decode(lib, q=Q, k8=K8, v8=V8, ks=KS, vs=VS, o=QO, B=2, T=1, ln=LEN, H=8, Hkv=2, D=128, w=0,
           scale=0.1, dt=BF16, qs=None, os=None, cap=256, block=64, ws=WS, n=GB):
    return lib.pfa_decode_attention_q8(q, k8, v8, ks, vs, o, B, T, ln, H, Hkv, D, w, scale, dt,
                                       H * D if qs is None else qs, H * D if os is None else os,
                                       cap, block, ws, n, None)


def test_decode_refusals(lib, last):
    n = ctypes.c_size_t(5)
    assert decode(lib, dt=9) == DTYPE
    for bad in (dict(H=6, Hkv=4), dict(H=0), dict(D=64), dict(D=256), dict(H=258, Hkv=2), dict(B=-1),
                dict(T=-1), dict(T=257), dict(block=8), dict(cap=255), dict(qs=1000), dict(os=1000)):
        assert decode(lib, **bad) == SHAPE, bad
    assert decode(lib, scale=float("nan")) == VALUE
    for bad in (dict(q=None), dict(o=None), dict(ln=None), dict(k8=None), dict(vs=None)):
        assert decode(lib, **bad) == NULL, bad
    for bad in (dict(q=Q + 8), dict(o=QO + 2), dict(ln=LEN + 4), dict(ws=WS + 16), dict(qs=1028)):
        assert decode(lib, **bad) == ALIGN, bad
    for bad in (dict(o=Q), dict(o=K8), dict(o=VS), dict(ln=QO)):
        assert decode(lib, **bad) == ALIAS, bad
    assert decode(lib, B=0) == 0 and decode(lib, T=0) == 0
    assert lib.pfa_decode_workspace_bytes_q8(2, 1, 8, 2, 128, BF16, None) == NULL
    assert lib.pfa_decode_workspace_bytes_q8(2, 1, 8, 3, 128, BF16, ctypes.byref(n)) == SHAPE
    assert lib.pfa_decode_workspace_bytes_q8(0, 1, 8, 2, 128, BF16, ctypes.byref(n)) == 0
    assert n.value == 0
    if last is not None:
        assert decode(lib) == last
        assert lib.pfa_decode_workspace_bytes_q8(2, 1, 8, 2, 128, BF16, ctypes.byref(n)) == last


def prefill(lib, q=Q, k8=K8, v8=V8, ks=KS, vs=VS, o=QO, T=100, sp=7, H=8, Hkv=2, D=128, w=0,
            scale=0.1, dt=BF16, row=None, cap=256, block=64, ws=WS, n=GB):
    return lib.pfa_prefill_attention_q8(q, k8, v8, ks, vs, o, T, sp, H, Hkv, D, w, scale, dt,
                                        H * D if row is None else row, cap, block, ws, n, None)


def test_prefill_refusals(lib, last):
    n = ctypes.c_size_t(5)
    assert prefill(lib, dt=9) == DTYPE
    for bad in (dict(H=6, Hkv=4), dict(D=64), dict(T=-1), dict(sp=-1), dict(sp=157), dict(cap=100),
                dict(row=1000), dict(block=512), dict(H=258, Hkv=2)):
        assert prefill(lib, **bad) == SHAPE, bad
    assert prefill(lib, scale=float("inf")) == VALUE
    for bad in (dict(q=None), dict(o=None), dict(ks=None)):
        assert prefill(lib, **bad) == NULL, bad
    for bad in (dict(q=Q + 8), dict(ws=WS + 128), dict(row=1028), dict(v8=V8 + 8)):
        assert prefill(lib, **bad) == ALIGN, bad
    for bad in (dict(o=Q + 256), dict(o=V8)):
        assert prefill(lib, **bad) == ALIAS, bad
    assert prefill(lib, T=0, q=None, o=None) == 0
    assert lib.pfa_prefill_workspace_bytes_q8(100, 7, 8, 2, 128, 0, BF16, None) == NULL
    assert lib.pfa_prefill_workspace_bytes_q8(100, -7, 8, 2, 128, 0, BF16, ctypes.byref(n)) == SHAPE
    assert lib.pfa_prefill_workspace_bytes_q8(0, 7, 8, 2, 128, 0, BF16, ctypes.byref(n)) == 0
    assert n.value == 0
    if last is not None:
        assert prefill(lib) == last


def test_binding_checks_tensors():
    cache = pkg.Q8Cache(*R.make_cache(2, 128, 128, 64))
    batch = pkg.Q8Cache(*R.make_cache(2, 128, 128, 64, batch=3))
    q, k = torch.zeros(3, 1, 8, 128), torch.zeros(3, 1, 2, 128)
    n = torch.ones(3, dtype=torch.int64)
    bad = [
        lambda: pkg.qk_norm_rope(q, k),                                     # neither position
        lambda: pkg.qk_norm_rope(q, k, start_pos=0),                        # a batch wants lengths
        lambda: pkg.qk_norm_rope(q, k, lengths=n.int()),
        lambda: pkg.qk_norm_rope(q, k, lengths=n[:2]),
        lambda: pkg.qk_norm_rope(q, k[:, :, :, :64], lengths=n),
        lambda: pkg.qk_norm_rope(q, k.bfloat16(), lengths=n),
        lambda: pkg.qk_norm_rope(q, k, torch.ones(64), lengths=n),
        lambda: pkg.qk_norm_rope(q, k, None, None, torch.ones(8), lengths=n),   # fp32 inv_freq
        lambda: pkg.qk_norm_rope(q.transpose(1, 2), k.transpose(1, 2), lengths=n),
        lambda: pkg.qk_norm_rope(q, k, lengths=n, q_out=q[:2]),
        lambda: pkg.cache_write_q8(k, k, cache, lengths=n),                 # a slot's cache
        lambda: pkg.cache_write_q8(k[:2], k[:2], batch, lengths=n[:2]),
        lambda: pkg.cache_write_q8(k, k[..., :64], batch, lengths=n),
        lambda: pkg.cache_write_q8(k.half(), k.half(), batch, lengths=n),
        lambda: pkg.cache_read_q8(cache, 5, 3),
        lambda: pkg.cache_read_q8(cache, 0, 129),
        lambda: pkg.cache_read_q8(cache, dtype=torch.float16),
        lambda: pkg.cache_read_q8(cache._replace(k_scale=cache.k_scale[:, :1])),
        lambda: pkg.cache_read_q8(cache._replace(k=cache.k.view(torch.uint8))),
        lambda: pkg.cache_read_q8(cache._replace(k=cache.k.transpose(0, 1))),
        lambda: pkg.decode_attention_q8(q, cache, n),
        lambda: pkg.decode_attention_q8(q[..., :64], batch, n),
        lambda: pkg.decode_attention_q8(q, batch, n.float()),
        lambda: pkg.decode_attention_q8(q, batch, n, out=q.bfloat16()),
        lambda: pkg.decode_attention_q8(q, batch, n),                       # CPU tensors
        lambda: pkg.prefill_attention_q8(q[:, 0], batch, start_pos=0),
        lambda: pkg.prefill_attention_q8(q[:, 0], cache, start_pos=0),      # CPU tensors
        lambda: pkg.q8_cache(2, 100, 128, block=64, device="cpu"),
        lambda: pkg.q8_cache(2, 128, 128, block=8, device="cpu"),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    c = pkg.q8_cache(2, 128, 64, batch=3, block=32, device="cpu")
    assert c.k.shape == (3, 2, 128, 64) and c.k_scale.shape == (3, 2, 4)
    assert c.slot(1).k.data_ptr() == c.k[1].data_ptr()


def test_reference_forms_agree_with_hand_worked_values():
    # 449 needs a scale of 2: 449 / 2 = 224.5 lies between 224 and 240
    assert R.block_scale(448.0) == 1.0 and R.block_scale(449.0) == 2.0 and R.block_scale(0.0) == 0.0
    assert R.to_e4m3(torch.tensor([224.5, 232.0, 248.0, 2.0 ** -10, 3 * 2.0 ** -10])).tolist() == \
        [224.0, 224.0, 256.0, 0.0, 2.0 ** -8]
    codes = torch.zeros(1, 16, 16, dtype=torch.uint8).view(torch.float8_e4m3fn)
    x = torch.full((1, 1, 16), 448.0)
    c, s = R.write(x, codes, torch.zeros(1, 1), 0, 16)
    assert s.item() == 1.0 and c[0, 0, 0] == 448.0
    c, s = R.write(4 * x, c.float().to(torch.float8_e4m3fn), s.float(), 1, 16)
    assert s.item() == 4.0 and c[0, 0, 0] == 112.0 and c[0, 1, 0] == 448.0
