"""The 4-bit cache's attention on paths that sizes alone reach: chunks that read the cache back, batches of
more sequences than one list of work holds, calls side by side, graphs that share a workspace."""
import pytest
import torch

import chunked_causal_gqa_gb300 as pkg
from tests import gpu_util as G
from tests import q4_reference as R
from tests import q8_reference as R8
from tests.test_q4_gpu import BF16, F32, attention_case, check_attention, lengths, ok, randn, within

pytestmark = pytest.mark.gpu


READ_BACK = [  # T, start, H, Hkv, D, window
    (1100, 117, 8, 2, 128, 0),
    (1100, 117, 8, 2, 128, 200),
    (2000, 0, 4, 1, 128, 0),
    (700, 1333, 16, 8, 128, 0),
    (700, 1333, 16, 8, 128, 64),
    (400, 640, 8, 2, 512, 0),
]


@pytest.mark.parametrize("case", READ_BACK, ids=str)
def test_a_chunk_that_reads_the_cache_back(case):
    T, start, H, Hkv, D, window = case
    n = start + T
    seen = T + (min(start, window - 1) if window else start)       # rows that the chunk sees
    assert pkg.prefill_workspace_bytes_q4(T, start, H, Hkv, D, window) >= 2 * Hkv * seen * D * 2
    cache = pkg.Q4Cache(*R.make_cache(Hkv, n + 9, D, seed=16, device=G.dev(), batch=1, dead=[n])).slot(0)
    cache = cache._replace(k_exponent=1, v_exponent=-2)
    q = randn((T, H, D), BF16, 14, 0.5)
    out = pkg.prefill_attention_q4(q, cache, start_pos=start, window=window)
    k, v = R.values(cache.k, cache.k_scale, 1), R.values(cache.v, cache.v_scale, -2)
    want, tol, _, _ = R.attention(q, k, v, n, window, R8.default_scale(D), BF16)
    # the 16-bit kernels round the weights to bf16
    j, pos = torch.arange(n, device=G.dev()), torch.arange(start, n, device=G.dev())[:, None]
    hidden = (j > pos) | (j <= pos - window if window else torch.zeros_like(j, dtype=torch.bool))
    for h in range(H):
        kv = h // (H // Hkv)
        p = torch.softmax((q[:, h].double() @ k[kv, :n].T * R8.default_scale(D)).masked_fill(hidden, float("-inf")), -1)
        tol[:, h] += 2.0 ** -8 * (p @ v[kv, :n].abs()) * (1 + 2.0 ** -8)
    within(out, want, tol)
    ok()


@pytest.mark.parametrize("T", [1, 3])
def test_more_sequences_than_one_list_of_work_holds(T):
    B, H, Hkv, D, cap = 16500, 2, 1, 128, 6
    cache = pkg.Q4Cache(*R.make_cache(Hkv, cap, D, batch=B, seed=21, device=G.dev()))
    q = randn((B, T, H, D), BF16, 22)
    ns = [(7 * b + b // 100) % (cap + 1) for b in range(B)]
    w0 = torch.rand(B, Hkv, cap, device=G.dev())
    w = w0.clone()
    out = pkg.decode_attention_q4(q, cache, lengths(ns), weights=w)
    some = [0, 1, 2, 3, 4, 5, 6, 4095, 5460, 5461, 8191, 8192, 16383, 16384, 16385, 16386, 16387, B - 2, B - 1]
    at = torch.tensor(some, device=G.dev())
    k, v = (R.values(c[at], s[at]) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    check_attention(out[at], w[at], w0[at], q[at], k, v, ([ns[b] for b in some], T, H, Hkv, D, 0, cap, BF16))
    # the others: what each gives in a batch of its own
    for b0 in range(0, B, 1500):
        z = slice(b0, b0 + 1500)
        w1 = w0[z].clone()
        one = pkg.decode_attention_q4(q[z], pkg.Q4Cache(cache.k[z], cache.v[z], cache.k_scale[z], cache.v_scale[z]),
                                      lengths(ns[z]), weights=w1)
        assert torch.equal(one, out[z])
        # sums and scores are equal; the order of the tokens' and heads' weights may be another
        within(w1, w[z].double(), 2.0 ** -20 * w[z].double())
    ok()


def test_calls_at_the_same_time():
    """Four streams, each with weights and workspaces of its own, over one cache."""
    case = ([3000, 17, 2999, 0], 2, 8, 2, 128, 0, 3001, BF16)
    cache, _, _, _ = attention_case(case, 31)
    n = lengths(case[0])
    qs = [randn((4, 2, 8, 128), BF16, 40 + i) for i in range(4)]
    want = []
    for q in qs:
        w = torch.zeros(4, 2, 3001, device=G.dev())
        want.append((pkg.decode_attention_q4(q, cache, n, weights=w), w))
    ws = [torch.zeros(4, 2, 3001, device=G.dev()) for _ in qs]
    outs = [torch.empty_like(q) for q in qs]
    need = pkg.decode_workspace_bytes_q4(4, 2, 8, 2, 128, 3001, weights=True)
    scratch = [torch.empty(need, dtype=torch.uint8, device=G.dev()) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for w in ws:
            w.zero_()
        torch.cuda.synchronize()
        for q, w, out, s, z in zip(qs, ws, outs, streams, scratch):
            pkg.decode_attention_q4(q, cache, n, out, weights=w, stream=s, workspace=z)
        torch.cuda.synchronize()
        for (o, w), out, w1 in zip(want, outs, ws):
            assert torch.equal(o, out) and torch.equal(w, w1)
    ok()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_graphs_that_share_a_workspace(dt):
    """Two calls of different shapes, captured over one workspace that held NaN, replayed in turn."""
    a, b = ([2000, 5], 1, 8, 2, 128, 0, 2001, dt), ([300], 9, 8, 2, 128, 50, 300, dt)
    calls, need = [], 0
    for i, case in enumerate((a, b)):
        cache, q, _, _ = attention_case(case, 50 + i)
        n, w = lengths(case[0]), torch.zeros(len(case[0]), 2, case[6], device=G.dev())
        need = max(need, pkg.decode_workspace_bytes_q4(len(case[0]), case[1], 8, 2, 128, case[6], weights=True, dtype=dt))
        out = pkg.decode_attention_q4(q, cache, n, weights=w, window=case[5])
        calls.append((q, cache, n, case[5], out, w.clone(), torch.zeros_like(out), w.zero_()))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=G.dev())
    graphs = []
    for q, cache, n, window, _, _, out, w in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkg.decode_attention_q4(q, cache, n, out, weights=w, window=window, workspace=ws)
        graphs.append(graph)
    for _ in range(3):
        for graph, (*_, want, acc, out, w) in zip(graphs, calls):
            w.zero_()
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(w, acc)
    ok()


MANY = [  # T, H, Hkv, D, window, dtype: 40 sequences, enough units for the larger tiles
    (2, 30, 6, 128, 0, BF16),      # 10 rows
    (4, 32, 8, 128, 0, BF16),      # 16
    (4, 32, 8, 128, 70, BF16),
    (17, 6, 6, 128, 0, BF16),      # 17
    (5, 32, 8, 128, 0, BF16),      # 20
    (3, 64, 8, 128, 33, BF16),     # 24
    (5, 25, 5, 128, 0, BF16),      # 25
    (12, 32, 8, 128, 0, BF16),     # 48
    (11, 30, 6, 128, 100, BF16),   # 55
    (4, 32, 8, 128, 0, F32),
    (5, 32, 8, 128, 65, F32),
    (3, 30, 6, 512, 0, BF16),
    (2, 60, 6, 512, 60, F32),
]


@pytest.mark.parametrize("case", MANY, ids=str)
@pytest.mark.parametrize("with_weights", [False, True])
def test_many_rows_and_sequences(case, with_weights):
    T, H, Hkv, D, window, dt = case
    lens, cap = [1000, 999, 1, 0, 64, 333, 17, 2, 512, 961] * 4, 1000
    full = (lens, T, H, Hkv, D, window, cap, dt)
    cache, q, k, v = attention_case(full, 61, (2, -3))
    w0 = torch.rand(len(lens), Hkv, cap, device=G.dev()) if with_weights else None
    w = w0.clone() if with_weights else None
    out = pkg.decode_attention_q4(q, cache, lengths(lens), weights=w, window=window)
    check_attention(out, w, w0, q, k, v, full)
    again = pkg.decode_attention_q4(q, cache, lengths(lens), weights=None if w0 is None else w0.clone(), window=window)
    assert torch.equal(out, again)
    ok()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_many_rows_one_of_them_not_finite(what):
    """A row of a tile that is not finite leaves the tile's others right, and keys that are not finite leave
    those right that do not see them."""
    lens, cap, T, H, Hkv, D = [1000, 700] * 20, 1000, 6, 32, 8, 128
    full = (lens, T, H, Hkv, D, 0, cap, BF16)
    cache, q, k, v = attention_case(full, 71)
    n = lengths(lens)
    good = pkg.decode_attention_q4(q, cache, n)
    bad = q.clone()
    bad[3, 2, 5, 7] = what
    out = pkg.decode_attention_q4(bad, cache, n)
    assert out[3, 2, 5].isnan().all()
    rest = torch.ones(q.shape[:3], dtype=torch.bool, device=G.dev())
    rest[3, 2, 5] = False
    assert torch.equal(out[rest], good[rest])
    cache.k_scale.view(torch.uint8)[4, 1, 999, 0] = 0x7f       # the last token's own key
    out = pkg.decode_attention_q4(q, cache, n)
    assert out[4, 5, 4:8].isnan().all()
    rest = torch.ones(q.shape[:3], dtype=torch.bool, device=G.dev())
    rest[4, 5, 4:8] = False
    assert not out[rest].isnan().any() and torch.equal(out[rest], good[rest])
    ok()


AGAIN = [  # lens, T, H, Hkv, window: few heads, or many rows
    ([3001], 3, 8, 2, 0),              # 12 rows
    ([3001, 64], 9, 8, 8, 70),         # 9
    ([3001, 1, 0, 7], 16, 4, 4, 0),    # 16
    ([3001, 129], 16, 16, 2, 0),       # 128
    ([3001, 129], 43, 6, 2, 0),        # 129
    ([300, 5, 260], 100, 20, 2, 33),   # 1000
    ([2000] * 12, 26, 8, 8, 0),        # 26 rows of many heads
    ([32, 33], 32, 8, 2, 0),           # chunks that are all or nearly all of a sequence
]


@pytest.mark.parametrize("case", AGAIN, ids=lambda c: f"B{len(c[0])}x{c[0][0]}-T{c[1]}-{c[2]}/{c[3]}-w{c[4]}")
def test_weights_without_stored_scores(case):
    lens, T, H, Hkv, window = case
    cap, rows = max(lens) + 2, T * H // Hkv
    extra = (pkg.decode_workspace_bytes_q4(len(lens), T, H, Hkv, 128, cap, weights=True) -
             pkg.decode_workspace_bytes_q4(len(lens), T, H, Hkv, 128, cap))
    assert extra < len(lens) * Hkv * rows * 8 + 512               # the rows' sums, no scores
    full = (lens, T, H, Hkv, 128, window, cap, BF16)
    cache, q, k, v = attention_case(full, 81, (3, -1))
    w0 = torch.rand(len(lens), Hkv, cap, device=G.dev())
    w = w0.clone()
    out = pkg.decode_attention_q4(q, cache, lengths(lens), weights=w, window=window)
    check_attention(out, w, w0, q, k, v, full)
    assert torch.equal(out, pkg.decode_attention_q4(q, cache, lengths(lens), window=window))
    again = w0.clone()
    pkg.decode_attention_q4(q, cache, lengths(lens), weights=again, window=window)
    assert torch.equal(w, again)
    ok()


def test_weights_without_stored_scores_report_lengths():
    case = ([700, 701, 700], 10, 8, 2, 128, 0, 700, BF16)
    cache, q, k, v = attention_case(([700, 700, 700], *case[1:]), 91)
    w = torch.zeros(3, 2, 700, device=G.dev())
    out = torch.full_like(q, 3.0)
    pkg.decode_attention_q4(q, cache, lengths(case[0]), out, weights=w)
    ok(-11)
    for b in (0, 2):
        want, tol, acc, acc_tol = R.attention(q[b], k[b], v[b], 700, 0, R8.default_scale(128), BF16)
        within(out[b], want, tol)
        within(w[b], acc, acc_tol + 2.0 ** -24 * acc)
    assert (out[1] == 3).all() and not w[1].any()
