"""GPU parity of the serving operators against the fp64 oracle: attention with a sliding
window and sinks, KV cache append, decode against the caches and behind a shared prefix,
sampling.

Attention tolerance, element by element. With A = sum_j p_j |v_j| of the element: each
weight is rounded to bf16 (half a step, 2^-8 of its value), which moves the sum by at
most 2^-8 A; the exponentials are within 7.5e-5 of their values in the numerator and the
sum (together below 2^-12 A), the fp32 scores and sums add less than 2^-12 A at these
sizes; the result is rounded to bf16 once, 2^-8 of itself. So
|y - ref| <= (2^-8 + 2^-11) A + 2^-8 (1 + 2^-6) |ref| + 2^-126.
Copies and drawn tokens are exact."""

import math

import numpy as np
import pytest
import torch

import oracle as O
import workloads as WL

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import tensor_sharded_linear_columnparallel_b200 as T
    return T


@pytest.fixture(autouse=True)
def _clean(T):
    yield
    torch.cuda.synchronize()
    assert T.tps_device_error() == T.TPS_OK


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def close(y, ref, mag, what=""):
    y = f64(y)
    assert y.shape == ref.shape, (what, y.shape, ref.shape)
    tol = (2.0 ** -8 + 2.0 ** -11) * mag + 2.0 ** -8 * (1 + 2.0 ** -6) * np.abs(ref) + 2.0 ** -126
    err = np.abs(y - ref)
    assert np.isfinite(y).all(), what
    assert (err <= tol).all(), f"{what}: {(err / tol).max():.3f} of the tolerance at {np.unravel_index((err / tol).argmax(), err.shape)}"


def geom(hq, hkv, tp):
    kvs = hkv // tp if hkv % tp == 0 else 1
    return tp * kvs, tp * (hq // tp + 2 * kvs) * D


# ============================================================ window attention
WINDOWS = [  # nseq, S, hq, hkv, tp, window, nsink, std
    (1, 1, 2, 1, 1, 1, 0, 1.0),
    (1, 128, 2, 1, 1, 1, 0, 1.0),        # every query sees itself alone
    (1, 300, 4, 2, 2, 17, 0, 1.0),
    (1, 700, 2, 1, 1, 128, 4, 1.0),      # window = block
    (1, 700, 2, 1, 1, 129, 4, 1.0),
    (1, 700, 2, 1, 1, 127, 4, 3.0),
    (2, 641, 4, 4, 4, 200, 130, 1.0),    # sinks over a block border, odd number of query blocks
    (3, 520, 4, 1, 2, 64, 1, 1.0),       # KV head replicated
    (1, 900, 7, 1, 1, 256, 128, 1.0),
    (2, 384, 2, 2, 1, 10 ** 9, 10 ** 9, 1.0),   # plain causal
    (1, 1500, 2, 1, 1, 300, 4, 1.0),
    (1, 1025, 2, 1, 1, 2, 1000, 1.0),    # nearly everything is a sink
    (1, 2048, 2, 2, 2, 512, 0, 6.0),     # peaked softmax
]


@pytest.mark.parametrize("nseq,S,hq,hkv,tp,window,nsink,std", WINDOWS)
def test_window_attention(T, nseq, S, hq, hkv, tp, window, nsink, std):
    qkv = WL.gen_normal((nseq * S, geom(hq, hkv, tp)[1]), std, 901)
    A = T.sharded_window_attention(qkv.cuda(), nseq, S, T.Heads(hq, hkv, D), tp, window, nsink)
    close(A, *O.window_attention_sharded(qkv, hq, hkv, D, tp, nseq, S, window, nsink))
    assert torch.equal(A, T.sharded_window_attention(qkv.cuda(), nseq, S, T.Heads(hq, hkv, D), tp, window, nsink))


def test_window_attention_many_items_per_cta(T):
    """More work items than SMs, with and without a second query tile."""
    nseq, S, hq, hkv, tp, W, ns = 13, 333, 32, 8, 8, 100, 5
    qkv = WL.gen_normal((nseq * S, geom(hq, hkv, tp)[1]), 1.0, 902)
    A = T.sharded_window_attention(qkv.cuda(), nseq, S, T.Heads(hq, hkv, D), tp, W, ns)
    close(A, *O.window_attention_sharded(qkv, hq, hkv, D, tp, nseq, S, W, ns))


def test_window_attention_wide_window_equals_causal_attention(T):
    qkv = WL.gen_normal((2 * 450, geom(8, 2, 2)[1]), 1.0, 903).cuda()
    A = T.sharded_window_attention(qkv, 2, 450, T.Heads(8, 2, D), 2, 450)
    assert torch.equal(A, T.sharded_gqa_attention(qkv, 2, 450, T.Heads(8, 2, D), 2, True))


def test_window_attention_sequences_do_not_touch(T):
    """NaN tokens of the next sequence, in the same 128-key block, change nothing; rows
    behind the last sequence keep their bits."""
    S = 70
    qkv = WL.gen_normal((2 * S, geom(2, 1, 1)[1]), 1.0, 904)
    ref = O.window_attention_sharded(qkv[:S], 2, 1, D, 1, 1, S, 30, 2)
    bad = qkv.clone()
    bad[S:] = float("nan")
    out = torch.full((2 * S + 3, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    T.sharded_window_attention(bad.cuda(), 2, S, T.Heads(2, 1, D), 1, 30, 2, out=out[:2 * S])
    close(out[:S], *ref)
    assert (out[2 * S:] == 7.0).all()


# ============================================================ caches
def caches(nseq, nkv, cap, seed, fill=None):
    if fill is not None:
        return [torch.full((nseq, nkv, cap, D), fill, dtype=torch.bfloat16) for _ in range(2)]
    return [WL.gen_normal((nseq, nkv, cap, D), 1.0, seed + i) for i in range(2)]


APPENDS = [  # nseq, S, hq, hkv, tp, cap, nsink, pos, count
    (1, 1, 2, 1, 1, 1, 0, [5], [1]),
    (3, 7, 4, 2, 2, 16, 0, [0, 3, 9], [7, 0, 7]),
    (3, 50, 4, 1, 2, 13, 4, [0, 2, 100], [50, 9, 77]),    # the ring wraps within the call; count above S
    (4, 5, 8, 8, 4, 9, 8, [-1, 0, 7, 8], [5, 5, 5, -3]),   # unused row, one ring slot
    (2, 300, 4, 4, 1, 130, 2, None, None),
    (2, 3, 2, 1, 1, 70, 1, [2 ** 31 - 4, 2 ** 30], [3, 2]),
]


@pytest.mark.parametrize("nseq,S,hq,hkv,tp,cap,nsink,pos,count", APPENDS)
def test_kv_append_bit_exact(T, nseq, S, hq, hkv, tp, cap, nsink, pos, count):
    nkv, cols = geom(hq, hkv, tp)
    qkv = WL.gen_normal((nseq * S, cols), 1.0, 911)
    k, v = caches(nseq, nkv, cap, 912)
    kg, vg = k.cuda(), v.cuda()
    vec = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
    T.sharded_kv_append(qkv.cuda(), nseq, S, T.Heads(hq, hkv, D), tp, kg, vg, pos=vec(pos), count=vec(count), nsink=nsink)
    kr, vr = f64(k).copy(), f64(v).copy()
    O.kv_append(qkv, hq, hkv, D, tp, nseq, S, pos or [0] * nseq, count or [S] * nseq, nsink, kr, vr)
    assert np.array_equal(f64(kg), kr) and np.array_equal(f64(vg), vr)


DECODES = [  # hq, hkv, tp, cap, nsink, window, positions
    (2, 1, 1, 1, 0, 1, [0, 3, -1]),
    (4, 2, 2, 64, 0, 64, [0, 1, 62, 63, 64, 1000]),
    (4, 1, 2, 300, 4, 200, [0, 3, 4, 5, 127, 128, 203, 204, 299, 300, 301, 555, -7]),   # KV head replicated
    (32, 8, 8, 516, 4, 512, [10, 515, 516, 5000]),
    (7, 1, 1, 260, 130, 130, [129, 130, 131, 259, 260, 700]),                             # sinks over a block border
    (12, 4, 4, 1000, 1, 37, [0, 36, 37, 38, 998, 999, 1000, 40000]),
    (16, 1, 1, 200, 0, 190, [199, 200, 389]),
    (40, 2, 1, 150, 2, 148, [1, 149, 150]),                                               # 20 query heads per KV head
    (8, 8, 1, 640, 0, 128, [639, 640, 100]),                                              # one query head per KV head
]


@pytest.mark.parametrize("hq,hkv,tp,cap,nsink,window,pos", DECODES)
@pytest.mark.parametrize("std", [1.0, 4.0])
def test_window_decode(T, hq, hkv, tp, cap, nsink, window, pos, std):
    """Against the oracle, with NaN in every slot that no position was written to."""
    nseq = len(pos)
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    qkv = WL.gen_normal((nseq, cols), std, 921)
    k, v = caches(nseq, nkv, cap, 922)
    for b, t in enumerate(pos):
        written = {O.cache_slot(j, nsink, cap) for j in range(max(0, t - 2 * cap), t)} | set(range(min(nsink, max(t, 0))))
        for s in set(range(cap)) - written:
            k[b, :, s] = float("nan")
            v[b, :, s] = float("nan")
    kg, vg, pg = k.cuda(), v.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda")
    ws = T.decode_workspace(nseq, h, tp)
    out = T.sharded_window_decode(qkv.cuda(), h, tp, pg, window, kg, vg, ws, nsink=nsink)
    kr, vr = f64(k).copy(), f64(v).copy()
    ref, mag = O.cached_decode(qkv, hq, hkv, D, tp, pos, window, nsink, kr, vr)
    close(out, ref, mag)
    assert np.array_equal(f64(kg), kr, equal_nan=True) and np.array_equal(f64(vg), vr, equal_nan=True)
    again = T.sharded_window_decode(qkv.cuda(), h, tp, pg, window, kg, vg, ws, nsink=nsink)
    assert torch.equal(out, again)
    assert T.tps_sync_status(ws) == T.TPS_OK


@pytest.mark.parametrize("nseq,cap", [(40, 700), (1, 9000), (3, 4000), (150, 130)])
def test_window_decode_split_over_ctas(T, nseq, cap):
    """Work that is cut at any place: ragged positions, one long sequence, more rows than SMs."""
    hq, hkv, tp = 8, 2, 2
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    g = torch.Generator().manual_seed(nseq)
    pos = torch.randint(-1, 2 * cap, (nseq,), generator=g, dtype=torch.int32)
    if nseq == 1:
        pos[0] = 3 * cap
    qkv = WL.gen_normal((nseq, cols), 1.0, 931)
    k, v = caches(nseq, nkv, cap, 932)
    kg, vg = k.cuda(), v.cuda()
    ws = T.decode_workspace(nseq, h, tp)
    out = T.sharded_window_decode(qkv.cuda(), h, tp, pos.cuda(), cap - 4, kg, vg, ws, nsink=4)
    kr, vr = f64(k), f64(v)
    close(out, *O.cached_decode(qkv, hq, hkv, D, tp, pos.tolist(), cap - 4, 4, kr, vr))


PREFIXES = [  # hq, hkv, tp, prefix, cap, positions
    (2, 1, 1, 1, 4, [0]),
    (4, 2, 2, 0, 40, [0, 39, 40, -1, 7]),
    (4, 2, 2, 130, 40, [0, 39, 40, -1, 7]),       # pos = cap: unused
    (32, 8, 8, 1000, 300, [0, 5, 299, 128, 127, 200, -1, 64]),
    (7, 1, 1, 257, 64, list(range(0, 40, 2))),     # 7 x 20 rows: two query tiles
    (8, 1, 1, 640, 16, [i % 17 - 1 for i in range(70)]),
    (4, 1, 2, 5000, 20, [3, 19]),                  # KV head replicated, a prefix split over many CTAs
    (16, 16, 4, 384, 10, [1, 2, 3]),
    (40, 2, 1, 200, 8, [0, 7, 3]),                 # 20 query heads per KV head
]


@pytest.mark.parametrize("hq,hkv,tp,prefix,cap,pos", PREFIXES)
@pytest.mark.parametrize("std", [1.0, 4.0])
def test_prefix_decode(T, hq, hkv, tp, prefix, cap, pos, std):
    nseq = len(pos)
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    qkv = WL.gen_normal((nseq, cols), std, 941)
    k, v = caches(nseq, nkv, cap, 942)
    for b, t in enumerate(pos):
        k[b, :, max(0, t):] = float("nan")
        v[b, :, max(0, t):] = float("nan")
    pk, pv = WL.gen_normal((nkv, prefix, D), 1.0, 944), WL.gen_normal((nkv, prefix, D), 1.0, 945)
    kg, vg, pg = k.cuda(), v.cuda(), torch.tensor(pos, dtype=torch.int32, device="cuda")
    ws = T.decode_workspace(nseq, h, tp, prefix)
    args = (pk.cuda(), pv.cuda()) if prefix else (None, None)
    out = T.sharded_prefix_decode(qkv.cuda(), h, tp, *args, pg, kg, vg, ws)
    kr, vr = f64(k).copy(), f64(v).copy()
    live = [t if 0 <= t < cap else -1 for t in pos]
    ref, mag = O.cached_decode(qkv, hq, hkv, D, tp, live, cap, 0, kr, vr, f64(pk), f64(pv))
    close(out, ref, mag)
    assert np.array_equal(f64(kg), kr, equal_nan=True) and np.array_equal(f64(vg), vr, equal_nan=True)
    assert torch.equal(out, T.sharded_prefix_decode(qkv.cuda(), h, tp, *args, pg, kg, vg, ws))
    assert T.tps_sync_status(ws) == T.TPS_OK


def test_decode_large_scores_and_far_apart_maxima(T):
    """Scores whose maximum moves by hundreds from block to block, up and down."""
    hq, hkv, tp, cap, P = 4, 1, 1, 512, 700
    h = T.Heads(hq, hkv, D)
    qkv = WL.gen_normal((2, 6 * D), 1.0, 951)
    k, v = caches(2, 1, cap, 952)
    pk, pv = WL.gen_normal((1, P, D), 1.0, 953), WL.gen_normal((1, P, D), 1.0, 954)
    ramp = torch.linspace(0.0, 12.0, cap)[:, None]
    k[0] = (k[0].float() * ramp).to(torch.bfloat16)
    k[1] = (k[1].float() * ramp.flip(0)).to(torch.bfloat16)
    pk[0, 300:310] *= 16
    pos = [510, 400]
    for prefix in (False, True):
        kg, vg = k.cuda(), v.cuda()
        pg = torch.tensor(pos, dtype=torch.int32, device="cuda")
        ws = T.decode_workspace(2, h, tp, P if prefix else 0)
        args = (pk.cuda(), pv.cuda()) if prefix else (None, None)
        out = T.sharded_prefix_decode(qkv.cuda(), h, tp, *args, pg, kg, vg, ws)
        ref, mag = O.cached_decode(qkv, hq, hkv, D, tp, pos, cap, 0, f64(k).copy(), f64(v).copy(),
                                   *((f64(pk), f64(pv)) if prefix else (None, None)))
        # scores of this size carry an fp32 error of their own: |s| <= 1200, so a weight moves by up
        # to 1200 * 128 * 2^-24 = 2^-6.7 of itself in the worst order of the 128 products
        close(out, ref, mag * (1 + 2.0 ** -6.7 / 2.0 ** -8))


def test_decode_graph_replay_with_new_positions_on_another_stream(T):
    """A captured step replays with the positions and tokens of its replay; the workspace
    serves every replay."""
    hq, hkv, tp, cap, ns, W, P = 8, 2, 2, 100, 4, 90, 300
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    n = 3
    k, v = caches(n, nkv, cap, 961)
    pk, pv = WL.gen_normal((nkv, P, D), 1.0, 963), WL.gen_normal((nkv, P, D), 1.0, 964)
    kg, vg, k2, v2, pkg, pvg = k.cuda(), v.cuda(), k.cuda(), v.cuda(), pk.cuda(), pv.cuda()
    qkv = torch.zeros(n, cols, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws1, ws2 = T.decode_workspace(n, h, tp), T.decode_workspace(n, h, tp, P)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for _ in range(2):
            T.sharded_window_decode(qkv, h, tp, pos, W, kg, vg, ws1, nsink=ns)
            T.sharded_prefix_decode(qkv, h, tp, pkg, pvg, pos, k2, v2, ws2)
        st.synchronize()
        kg.copy_(k), vg.copy_(v), k2.copy_(k), v2.copy_(v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            a = T.sharded_window_decode(qkv, h, tp, pos, W, kg, vg, ws1, nsink=ns)
            b = T.sharded_prefix_decode(qkv, h, tp, pkg, pvg, pos, k2, v2, ws2)
    torch.cuda.synchronize()
    refs = [f64(x).copy() for x in (k, v, k, v)]
    for i, p in enumerate([[0, 40, 99], [98, -1, 41], [250, 97, 0]]):
        x = WL.gen_normal((n, cols), 1.0, 970 + i)
        qkv.copy_(x), pos.copy_(torch.tensor(p, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        close(a, *O.cached_decode(x, hq, hkv, D, tp, p, W, ns, *refs[:2]))
        live = [t if t < cap else -1 for t in p]
        close(b, *O.cached_decode(x, hq, hkv, D, tp, live, cap, 0, *refs[2:], f64(pk), f64(pv)))


# ============================================================ sampling
def sample_ref(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    l = f64(logits)
    get = lambda x, i, d: d if x is None else float(x[i])
    r = [O.sample_row(l[i], float(u[i]), get(temperature, i, 1.0), int(get(top_k, i, 0)), get(top_p, i, 1.0),
                      get(min_p, i, 0.0)) for i in range(l.shape[0])]
    return np.array([x[0] for x in r]), np.array([x[1] for x in r])


def check_sample(T, logits, u, **kw):
    dev = lambda x: None if x is None else x.cuda()
    idx, logp = T.logits_sample(logits.cuda(), u.cuda(), **{n: dev(x) for n, x in kw.items()})
    ri, rl = sample_ref(logits, u, **kw)
    assert np.array_equal(idx.cpu().numpy(), ri), [(a, b) for a, b in zip(idx.tolist(), ri.tolist()) if a != b][:5]
    fin = np.isfinite(rl)
    got = f64(logp)
    # a share of 2^-44 units: the weight is off by half a unit; the logarithm is rounded to fp32
    assert np.allclose(got[fin], rl[fin], rtol=2.0 ** -23, atol=1e-6), np.abs(got[fin] - rl[fin]).max()
    assert np.array_equal(got[~fin], rl[~fin])


def rows(m, V, spread, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, V, generator=g) * spread).to(dtype), torch.rand(m, generator=g), g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [8, 96, 1000, 4104, 33008])
@pytest.mark.parametrize("filters", ["none", "k", "p", "q", "kp", "kpq", "mixed"])
def test_logits_sample(T, V, dtype, filters):
    m = 9
    logits, u, g = rows(m, V, 2.0, V + len(filters), dtype)
    kw = dict(temperature=0.4 + 1.6 * torch.rand(m, generator=g))
    if "k" in filters or filters == "mixed":
        kw["top_k"] = torch.randint(1, min(V, 200) + 1, (m,), generator=g, dtype=torch.int32)
    if "p" in filters or filters == "mixed":
        kw["top_p"] = 0.2 + 0.79 * torch.rand(m, generator=g)
    if "q" in filters or filters == "mixed":
        kw["min_p"] = 0.2 * torch.rand(m, generator=g)
    if filters == "mixed":
        for n, off in (("top_k", 0), ("top_p", 1.0), ("min_p", 0.0)):
            kw[n][torch.rand(m, generator=g) < 0.4] = off
        kw["temperature"][:2] = torch.tensor([0.0, -1.0])
        kw["top_k"][3] = V + 5
    check_sample(T, logits, u, **kw)


def test_logits_sample_defaults_and_extremes(T):
    logits, _, g = rows(8, 504, 3.0, 5)
    u = torch.tensor([0.0, 1.0, 0.99999994, -3.0, 7.0, float("nan"), 0.5, 1e-30])
    ref_u = torch.tensor([0.0, 1.0, 0.99999994, 0.0, 1.0, 0.0, 0.5, 1e-30])
    idx, _ = T.logits_sample(logits.cuda(), u.cuda())
    assert np.array_equal(idx.cpu().numpy(), sample_ref(logits, ref_u)[0])
    hot = torch.tensor([1e-6, 1e-30, 1e30, 0.01, 100.0, float("inf"), float("nan"), 1.0])
    check_sample(T, logits, torch.rand(8, generator=g), temperature=hot)


def test_logits_sample_ties(T):
    """Equal logits everywhere, and groups of them across the cut of every filter."""
    m, V = 12, 2048
    g = torch.Generator().manual_seed(6)
    u = torch.rand(m, generator=g)
    flat = torch.zeros(m, V)
    steps = torch.randint(0, 5, (m, V), generator=g).float()
    signed = torch.where(torch.rand(m, V, generator=g) < 0.5, torch.tensor(0.0), torch.tensor(-0.0))
    for l in (flat, steps, signed):
        check_sample(T, l, u)
        check_sample(T, l, u, top_k=torch.arange(1, m + 1, dtype=torch.int32) * 37)
        check_sample(T, l, u, top_p=torch.linspace(0.0, 0.98, m))
        check_sample(T, l, u, top_k=torch.full((m,), 700, dtype=torch.int32), top_p=torch.linspace(0.03, 0.97, m),
                     min_p=torch.linspace(0.0, 1.0, m))


def test_logits_sample_masked_logits(T):
    m, V = 10, 1024
    logits, u, g = rows(m, V, 2.0, 7)
    logits[torch.rand(m, V, generator=g) < 0.9] = -math.inf
    logits[1] = -math.inf
    logits[2] = float("nan")
    logits[3] = -math.inf
    logits[3, 1000] = -5.0
    logits[4, 17] = math.inf
    logits[5, [3, 900]] = math.inf
    logits[6] = torch.finfo(torch.float32).min
    logits[7, ::2] = float("nan")
    for kw in ({}, dict(top_k=torch.full((m,), 300, dtype=torch.int32)), dict(top_p=torch.full((m,), 0.9)),
               dict(min_p=torch.full((m,), 0.05)),
               dict(top_k=torch.full((m,), 5, dtype=torch.int32), top_p=torch.full((m,), 0.7),
                    temperature=torch.full((m,), 0.5))):
        check_sample(T, logits, u, **kw)


def test_logits_sample_outliers_and_large_vocabulary(T):
    """One logit far above (or below) the rest, and a vocabulary near the limit: numpy does
    the sorting here, the definition is the same."""
    m, V = 4, 262144
    logits, u, g = rows(m, V, 1.0, 8)
    logits[1, 77777] = 60.0
    logits[2, 5] = -3e38
    logits[3] *= 0.001
    for k, p in ((0, 1.0), (50, 1.0), (0, 0.9), (100000, 0.95), (3000, 0.5)):
        idx, _ = T.logits_sample(logits.cuda(), u.cuda(), top_k=torch.full((m,), k, dtype=torch.int32, device="cuda"),
                                 top_p=torch.full((m,), p, device="cuda"))
        for i in range(m):
            l = f64(logits[i])
            w = np.exp(l - l.max())
            order = np.lexsort((np.arange(V), -l))[:k or V]
            pp = float(np.float32(p))
            if pp < 1:
                c = np.cumsum(w[order])
                order = order[np.concatenate([[0.0], c[:-1]]) < pp * c[-1]]
            kept = np.sort(order)
            c = np.cumsum(w[kept])
            assert idx[i].item() == kept[np.searchsorted(c, float(u[i]) * c[-1], side="right")], (i, k, p)


def test_logits_sample_frequencies(T):
    """u on a grid draws every token with its share, within one grid step."""
    V, n = 16, 4096
    l = torch.linspace(-2, 2, V)
    u = (torch.arange(n) + 0.5) / n
    idx, logp = T.logits_sample(l.repeat(n, 1).cuda().contiguous(), u.cuda())
    share = np.bincount(idx.cpu().numpy(), minlength=V) / n
    p = torch.softmax(l.double(), 0).numpy()
    assert np.abs(share - p).max() <= 1.0 / n
    assert np.allclose(np.exp(f64(logp)), p[idx.cpu().numpy()], rtol=1e-5)


def test_logits_sample_many_rows(T):
    logits, u, g = rows(1500, 256, 2.0, 9)
    check_sample(T, logits, u, top_k=torch.randint(0, 40, (1500,), generator=g, dtype=torch.int32),
                 top_p=0.3 + 0.8 * torch.rand(1500, generator=g))


@pytest.mark.parametrize("m,V,dtype", [(2, 70000, torch.bfloat16), (20, 70000, torch.float32),
                                       (40, 70000, torch.bfloat16), (150, 40000, torch.float32),
                                       (150, 40000, torch.bfloat16), (30, 2056, torch.float32)])
def test_logits_sample_rows_over_clusters(T, m, V, dtype):
    """Rows in 1 to 8 CTAs of either size; logits so close together that the cut's bin holds a
    few tokens, hundreds, or more than the list; top_k past what is drawn from a list at once."""
    n = min(m, 6)                              # distinct rows, taken in turn
    for i, spread in enumerate((0.05, 0.4, 4.0)):
        logits, u, g = rows(n, V, spread, 40 + i, dtype)
        p = torch.rand(n, generator=g)
        p[0] = 0.0
        k = torch.randint(0, 1000, (n,), generator=g, dtype=torch.int32)
        q = 0.9 * torch.rand(n, generator=g)
        q[::2] = 0.0
        t = 0.2 + torch.rand(n, generator=g)
        turn = torch.arange(m) % n
        for kw in (dict(top_p=p), dict(top_k=k), dict(top_k=k, top_p=p, min_p=q), dict(top_p=p, min_p=q)):
            kw["temperature"] = t
            ri, rl = sample_ref(logits, u, **kw)
            idx, logp = T.logits_sample(logits[turn].cuda(), u[turn].cuda(), **{x: y[turn].cuda() for x, y in kw.items()})
            assert np.array_equal(idx.cpu().numpy(), ri[turn])
            assert np.allclose(f64(logp), rl[turn], rtol=2.0 ** -23, atol=1e-6)


@pytest.mark.parametrize("m,H,V,tp", [(1, 64, 512, 2), (33, 256, 4096, 8), (70, 128, 1000, 1)])
def test_vocab_parallel_sample_integer_logits(T, m, H, V, tp):
    """Integer products are exact in fp32, so the drawn token is the oracle's."""
    X, W = WL.gen_int((m, H), -2, 2, 981), WL.gen_int((H, V), -1, 1, 982)
    g = torch.Generator().manual_seed(3)
    u, t = torch.rand(m, generator=g), 2.0 + 6 * torch.rand(m, generator=g)
    p, k = 0.5 + 0.5 * torch.rand(m, generator=g), torch.randint(0, 60, (m,), generator=g, dtype=torch.int32)
    pw = T.tp_shard_weights(T.KIND_COLUMN, W.cuda(), tp)
    idx, logp = T.vocab_parallel_sample(X.cuda(), H, V, tp, pw, u.cuda(), temperature=t.cuda(), top_k=k.cuda(),
                                        top_p=p.cuda())
    ri, rl = sample_ref(torch.from_numpy(O.to_f64(X) @ O.to_f64(W)), u, t, k, p)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.allclose(f64(logp), rl, rtol=2.0 ** -23, atol=1e-6)
    greedy, _ = T.vocab_parallel_sample(X.cuda(), H, V, tp, pw, u.cuda(), temperature=torch.zeros(m, device="cuda"))
    assert torch.equal(greedy, T.vocab_parallel_argmax(X.cuda(), H, V, tp, pw)[0])


# ============================================================ together
def test_prefill_then_decode_with_sampled_tokens(T):
    """A small model's serving loop: windowed prefill, append, then steps of QKV, decode,
    o_proj, lm_head and sampling, captured into a graph; every step against the oracle on
    the values that the step read."""
    hq, hkv, tp, Hd, V, S, W, ns, steps = 8, 2, 2, 256, 512, 150, 64, 4, 5
    n, cap = 2, ns + W
    h = T.Heads(hq, hkv, D)
    nkv, cols = geom(hq, hkv, tp)
    Wqkv = WL.gen_normal((Hd, (hq + 2 * hkv) * D), Hd ** -0.5, 991).cuda()
    Wo = WL.gen_normal((hq * D, Hd), (hq * D) ** -0.5, 992).cuda()
    Wl = WL.gen_normal((Hd, V), 2 * Hd ** -0.5, 993).cuda()
    emb = WL.gen_normal((V, Hd), 1.0, 994).cuda()
    pq = T.tp_shard_weights(T.KIND_QKV, Wqkv, tp, heads=h)
    po = T.tp_shard_weights(T.KIND_ROW, Wo, tp)
    pl = T.tp_shard_weights(T.KIND_COLUMN, Wl, tp)
    tok = torch.randint(0, V, (n, S), generator=torch.Generator().manual_seed(1)).cuda()
    qkv = T.column_parallel_forward(emb[tok.view(-1)], pq, T.KIND_QKV, (hq + 2 * hkv) * D, tp, heads=h)
    A = T.sharded_window_attention(qkv, n, S, h, tp, W, ns)
    close(A, *O.window_attention_sharded(qkv.cpu(), hq, hkv, D, tp, n, S, W, ns))
    k = torch.full((n, nkv, cap, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    T.sharded_kv_append(qkv, n, S, h, tp, k, v, nsink=ns)
    ws = T.decode_workspace(n, h, tp)
    lws = T.workspace(T.FN_SAMPLE, n, V, Hd, tp)
    pos = torch.full((n,), S, dtype=torch.int32, device="cuda")
    u = torch.zeros(n, device="cuda")
    par = dict(temperature=torch.full((n,), 0.8, device="cuda"), top_k=torch.full((n,), 40, dtype=torch.int32, device="cuda"),
               top_p=torch.full((n,), 0.9, device="cuda"), min_p=torch.full((n,), 0.02, device="cuda"))
    cur = tok[:, -1].to(torch.int32).clone()

    def step():
        x = T.column_parallel_forward(emb[cur.long()], pq, T.KIND_QKV, (hq + 2 * hkv) * D, tp, heads=h)
        a = T.sharded_window_decode(x, h, tp, pos, W, k, v, ws, nsink=ns)
        y = T.row_parallel_forward(a, po, Hd, tp)
        idx, _ = T.vocab_parallel_sample(y, Hd, V, tp, pl, u, lws, **par)
        cur.copy_(idx)
        pos.add_(1)
        return x, a, y, idx

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in (k, v, pos, cur)]
    with torch.cuda.stream(st):
        step()
        st.synchronize()
        for t, s in zip((k, v, pos, cur), keep):
            t.copy_(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            x, a, y, idx = step()
    torch.cuda.synchronize()
    kr, vr = f64(k).copy(), f64(v).copy()
    for i in range(steps):
        u.copy_(torch.rand(n, generator=torch.Generator().manual_seed(i)))
        g.replay()
        torch.cuda.synchronize()
        close(a, *O.cached_decode(x.cpu(), hq, hkv, D, tp, [S + i] * n, W, ns, kr, vr), what=f"step {i}")
        # the token from the logits that the step left in its workspace
        logits = lws[256:256 + n * V * 4].view(torch.float32).view(n, V).cpu()
        ref = O.to_f64(y.cpu()) @ O.to_f64(Wl.cpu())
        assert np.abs(f64(logits) - ref).max() <= 1e-4 * (1 + np.abs(ref).max())
        cpu = {a_: b_.cpu() for a_, b_ in par.items()}
        assert np.array_equal(idx.cpu().numpy(), sample_ref(logits, u.cpu(), **cpu)[0])
    assert pos.tolist() == [S + steps] * n


def test_refused_calls(T):
    h = T.Heads(4, 2, D)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    cols = geom(4, 2, 2)[1]
    k, v, pos, ws = z(2, 2, 8, D), z(2, 2, 8, D), z(2, dtype=torch.int32), T.decode_workspace(2, h, 2)
    with pytest.raises(ValueError):
        T.sharded_window_attention(z(4, cols), 1, 5, h, 2, 4)
    with pytest.raises(ValueError):
        T.sharded_kv_append(z(4, cols), 2, 2, h, 2, k, z(2, 2, 9, D))
    with pytest.raises(ValueError):
        T.sharded_kv_append(z(4, cols), 2, 2, h, 2, k, v, pos=z(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        T.sharded_window_decode(z(2, cols), h, 2, z(2, dtype=torch.int64), 4, k, v, ws)
    with pytest.raises(ValueError):
        T.sharded_window_decode(z(2, cols), h, 2, pos, 4, k[:, :, ::2], v[:, :, ::2], ws)
    with pytest.raises(ValueError):
        T.sharded_prefix_decode(z(2, cols), h, 2, z(2, 5, D), z(2, 6, D), pos, k, v, ws)
    with pytest.raises(T.TpsError) as e:
        T.sharded_window_decode(z(2, cols), h, 2, pos, 9, k, v, ws)
    assert e.value.status == T.TPS_ERR_ARG
    with pytest.raises(T.TpsError) as e:
        T.sharded_window_decode(z(2, cols), h, 2, pos, 4, k, v, ws[:64])
    assert e.value.status == T.TPS_ERR_WORKSPACE
    with pytest.raises(T.TpsError) as e:
        T.logits_sample(z(2, 12), z(2, dtype=torch.float32))
    assert e.value.status == T.TPS_ERR_ALIGN
    with pytest.raises(ValueError):
        T.logits_sample(z(2, 16), z(3, dtype=torch.float32))
    with pytest.raises(ValueError):
        T.logits_sample(z(2, 16, dtype=torch.float16), z(2, dtype=torch.float32))
    assert T.logits_sample(z(0, 16), z(0, dtype=torch.float32))[0].numel() == 0
    assert T.sharded_window_attention(z(0, cols), 0, 5, h, 2, 4).numel() == 0


def test_explicit_stream(T):
    """Every call on a stream given as an argument, behind work of that stream."""
    st = torch.cuda.Stream()
    h = T.Heads(4, 2, D)
    nkv, cols = geom(4, 2, 2)
    S, cap = 140, 150
    qkv = WL.gen_normal((S, cols), 1.0, 995)
    src, x = qkv.pin_memory(), torch.zeros(S, cols, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(1, nkv, cap, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, pos = T.decode_workspace(1, h, 2), torch.tensor([S - 1], dtype=torch.int32, device="cuda")
    logits, u, g = rows(3, 504, 2.0, 996)
    lg, ug = logits.cuda(), u.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        x.copy_(src, non_blocking=True)
    A = T.sharded_window_attention(x, 1, S, h, 2, 60, 3, stream=st)
    T.sharded_kv_append(x[:S - 1], 1, S - 1, h, 2, k, v, nsink=3, stream=st)
    out = T.sharded_window_decode(x[S - 1:], h, 2, pos, 60, k, v, ws, nsink=3, stream=st)
    idx, _ = T.logits_sample(lg, ug, stream=st)
    st.synchronize()
    ref, mag = O.window_attention_sharded(qkv, 4, 2, D, 2, 1, S, 60, 3)
    close(A, ref, mag)
    close(out, ref[-1:], mag[-1:])
    assert np.array_equal(idx.cpu().numpy(), sample_ref(logits, u)[0])


# ============================================================ the ends of the ranges
@pytest.mark.parametrize("prefix", [0, 200])
def test_decode_more_sequences_than_threads(T, prefix):
    """900 sequences, a third of them unused: the kernel's scan over the positions takes
    several steps."""
    hq, hkv, tp, cap, n = 4, 1, 1, 40, 900
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    g = torch.Generator().manual_seed(7)
    pos = torch.randint(-20, cap, (n,), generator=g, dtype=torch.int32)
    qkv = WL.gen_normal((n, cols), 1.0, 1001)
    k, v = caches(n, nkv, cap, 1002)
    pk, pv = WL.gen_normal((nkv, prefix, D), 1.0, 1004), WL.gen_normal((nkv, prefix, D), 1.0, 1005)
    kg, vg = k.cuda(), v.cuda()
    ws = T.decode_workspace(n, h, tp, prefix)
    args = (pk.cuda(), pv.cuda()) if prefix else (None, None)
    out = T.sharded_prefix_decode(qkv.cuda(), h, tp, *args, pos.cuda(), kg, vg, ws)
    kr, vr = f64(k).copy(), f64(v).copy()
    close(out, *O.cached_decode(qkv, hq, hkv, D, tp, pos.tolist(), cap, 0, kr, vr, f64(pk), f64(pv)))
    assert np.array_equal(f64(kg), kr) and np.array_equal(f64(vg), vr)


def test_decode_workspace_shared_by_calls_of_other_sizes(T):
    """One workspace, made for the largest of them, serves calls of any sizes in turn."""
    hq, hkv, tp, P = 16, 4, 2, 300
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    sizes = [(1, 5000, 0), (900, 260, 0), (3, 2000, P), (900, 150, P), (2, 9000, 0), (50, 900, 0)]
    shared = torch.zeros(max(T.tps_decode_workspace_bytes(n, h, tp, P) for n, _, _ in sizes), dtype=torch.uint8, device="cuda")
    pk, pv = WL.gen_normal((nkv, P, D), 1.0, 1101).cuda(), WL.gen_normal((nkv, P, D), 1.0, 1102).cuda()
    for n, cap, prefix in sizes:
        qkv = WL.gen_normal((n, cols), 1.0, 1103).cuda()
        k, v = (x.cuda() for x in caches(n, nkv, cap, 1104))
        pos = torch.full((n,), cap - 1, dtype=torch.int32, device="cuda")
        args = (pk, pv) if prefix else (None, None)
        got = T.sharded_prefix_decode(qkv, h, tp, *args, pos, k, v, shared)
        want = T.sharded_prefix_decode(qkv, h, tp, *args, pos, k, v, T.decode_workspace(n, h, tp, prefix))
        assert torch.equal(got, want), (n, cap, prefix)



def test_two_graphs_share_a_workspace(T):
    """A windowed and a prefix step, each captured once with the same workspace, replayed in
    turn with new positions."""
    hq, hkv, tp, P, cap = 16, 4, 2, 500, 400
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    pk, pv = WL.gen_normal((nkv, P, D), 1.0, 1111), WL.gen_normal((nkv, P, D), 1.0, 1112)
    pkg, pvg = pk.cuda(), pv.cuda()
    ws = T.decode_workspace(9, h, tp, P)
    sets = []
    for i, n in enumerate((9, 2)):
        qkv = WL.gen_normal((n, cols), 1.0, 1113 + i)
        k, v = caches(n, nkv, cap, 1115 + 2 * i)
        pos = torch.zeros(n, dtype=torch.int32, device="cuda")
        x, kg, vg, out = qkv.cuda(), k.cuda(), v.cuda(), torch.empty(n, hq * D, dtype=torch.bfloat16, device="cuda")

        def step(i=i, x=x, pos=pos, kg=kg, vg=vg, out=out):
            if i:
                T.sharded_window_decode(x, h, tp, pos, 300, kg, vg, ws, 5, out)
            else:
                T.sharded_prefix_decode(x, h, tp, pkg, pvg, pos, kg, vg, ws, out)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        kg.copy_(k)
        vg.copy_(v)
        sets.append((g, qkv, pos, out, f64(k).copy(), f64(v).copy()))
    for r in range(3):
        for i, (g, qkv, pos, out, kr, vr) in enumerate(sets):
            p = [(37 * r + 131 * b) % cap for b in range(qkv.shape[0])]
            pos.copy_(torch.tensor(p, dtype=torch.int32))
            g.replay()
        torch.cuda.synchronize()
        for i, (g, qkv, pos, out, kr, vr) in enumerate(sets):
            more = () if i else (f64(pk), f64(pv))
            close(out, *O.cached_decode(qkv, hq, hkv, D, tp, pos.tolist(), 300 if i else cap, 5 if i else 0, kr, vr, *more))



@pytest.mark.parametrize("hq", [96, 128, 160])
def test_decode_many_query_heads_per_kv_head(T, hq):
    h, n, cap, P = T.Heads(hq, 1, D), 3, 70, 150
    cols = (hq + 2) * D
    qkv, (k, v) = WL.gen_normal((n, cols), 1.0, 1011), caches(n, 1, cap, 1012)
    pk, pv = WL.gen_normal((1, P, D), 1.0, 1014), WL.gen_normal((1, P, D), 1.0, 1015)
    pos = torch.tensor([0, 69, 33], dtype=torch.int32)
    ws = T.decode_workspace(n, h, 1, P)
    out = T.sharded_window_decode(qkv.cuda(), h, 1, pos.cuda(), cap, k.cuda(), v.cuda(), ws)
    close(out, *O.cached_decode(qkv, hq, 1, D, 1, pos.tolist(), cap, 0, f64(k).copy(), f64(v).copy()))
    call = lambda: T.sharded_prefix_decode(qkv.cuda(), h, 1, pk.cuda(), pv.cuda(), pos.cuda(), k.cuda(), v.cuda(), ws)
    if hq > 128:
        with pytest.raises(T.TpsError) as e:
            call()
        assert e.value.status == T.TPS_ERR_UNIMPLEMENTED
    else:
        close(call(), *O.cached_decode(qkv, hq, 1, D, 1, pos.tolist(), cap, 0, f64(k).copy(), f64(v).copy(), f64(pk), f64(pv)))


def test_cache_offsets_beyond_32_bits(T):
    """Caches of 5 GB each: the last sequence's slots lie behind 2^32 bytes and 2^31 elements."""
    hq, hkv, tp, n, cap, ns, W = 4, 2, 1, 5, 2_000_000, 3, 300
    h = T.Heads(hq, hkv, D)
    nkv, cols = geom(hq, hkv, tp)
    kg = torch.zeros(n, nkv, cap, D, dtype=torch.bfloat16, device="cuda")
    vg = torch.zeros(n, nkv, cap, D, dtype=torch.bfloat16, device="cuda")
    S = 400
    qkv = WL.gen_normal((n * S, cols), 1.0, 1021)
    first = [0, cap - 200, 10 * cap + 7, 1_999_000, cap - 1]
    pos = torch.tensor(first, dtype=torch.int32, device="cuda")
    T.sharded_kv_append(qkv.cuda(), n, S, h, tp, kg, vg, pos=pos, nsink=ns)
    new = WL.gen_normal((n, cols), 1.0, 1022)
    ws = T.decode_workspace(n, h, tp)
    out = T.sharded_window_decode(new.cuda(), h, tp, pos + S, W, kg, vg, ws, nsink=ns)
    x = O.to_f64(qkv).reshape(n, S, cols)
    y = O.to_f64(new)
    for b in range(n):
        vis = [t - first[b] for t in range(first[b] + S - W + 1, first[b] + S)]     # the window's older tokens
        sinks = [t - first[b] if first[b] <= t else None for t in range(ns)]        # None: never written, zeros
        for hd in range(hq):
            kc, vc = (hq + hd // 2) * D, (hq + hkv + hd // 2) * D
            pick = lambda c: np.stack([np.zeros(D) if i is None else x[b, i, c:c + D] for i in sinks + vis] + [y[b, c:c + D]])
            ref, mag = O.attend(y[b, hd * D:(hd + 1) * D], pick(kc), pick(vc))
            close(out[b, hd * D:(hd + 1) * D], ref, mag, f"sequence {b}")


def test_decode_steps_without_a_pause(T):
    """Many steps in a row, with and without a prefix, on one workspace: every one gives the
    first one's bits."""
    hq, hkv, tp, n, cap, P = 32, 8, 8, 24, 300, 4000
    h = T.Heads(hq, hkv, D)
    nkv, cols = geom(hq, hkv, tp)
    g = torch.Generator().manual_seed(3)
    qkv, (k, v) = WL.gen_normal((n, cols), 1.0, 1031).cuda(), [t.cuda() for t in caches(n, nkv, cap, 1032)]
    pk, pv = WL.gen_normal((nkv, P, D), 1.0, 1034).cuda(), WL.gen_normal((nkv, P, D), 1.0, 1035).cuda()
    pos = torch.randint(-1, cap, (n,), generator=g, dtype=torch.int32).cuda()
    ws = T.decode_workspace(n, h, tp, P)
    both = lambda: (T.sharded_prefix_decode(qkv, h, tp, pk, pv, pos, k, v, ws),
                    T.sharded_window_decode(qkv, h, tp, pos, cap - 2, k, v, ws, nsink=2))
    first = both()
    later = [both() for _ in range(60)]
    torch.cuda.synchronize()
    for a, b in later:
        assert torch.equal(a, first[0]) and torch.equal(b, first[1])
    assert T.tps_sync_status(ws) == T.TPS_OK


def test_two_streams_at_once(T):
    """Decode steps and draws on two streams, each with its own workspace."""
    hq, hkv, tp, n, cap = 32, 8, 8, 16, 900
    h = T.Heads(hq, hkv, D)
    nkv, cols = geom(hq, hkv, tp)
    sets = []
    for i in range(2):
        qkv, (k, v) = WL.gen_normal((n, cols), 1.0, 1041 + i).cuda(), [t.cuda() for t in caches(n, nkv, cap, 1043 + 2 * i)]
        pos = torch.randint(0, cap, (n,), generator=torch.Generator().manual_seed(i), dtype=torch.int32).cuda()
        logits, u, _ = rows(8, 33008, 2.0, 1050 + i)
        sets.append((qkv, k, v, pos, T.decode_workspace(n, h, tp), logits.cuda(), u.cuda(), torch.cuda.Stream()))
    run = lambda s, st: (T.sharded_window_decode(s[0], h, tp, s[3], cap, s[1], s[2], s[4], stream=st),
                         T.logits_sample(s[5], s[6], top_p=torch.full((8,), 0.9, device="cuda"), stream=st)[0])
    want = [run(s, None) for s in sets]
    torch.cuda.synchronize()
    got = [[run(s, s[7]) for s in sets] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for (a, i), (b, j) in zip(pair, want):
            assert torch.equal(a, b) and torch.equal(i, j)


@pytest.mark.parametrize("nsink", [0, 3])
def test_window_decode_at_the_last_positions(T, nsink):
    """Positions up to 2^31 - 1, the largest that an int32 holds."""
    hq, hkv, tp, cap = 4, 2, 1, 203
    h, W = T.Heads(hq, hkv, D), cap - nsink - 1
    nkv, cols = geom(hq, hkv, tp)
    pos = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 1 - cap]
    n = len(pos)
    qkv = WL.gen_normal((n, cols), 1.0, 1201)
    k, v = caches(n, nkv, cap, 1202)
    kg, vg = k.cuda(), v.cuda()
    out = T.sharded_window_decode(qkv.cuda(), h, tp, torch.tensor(pos, dtype=torch.int32, device="cuda"), W, kg, vg,
                                  T.decode_workspace(n, h, tp), nsink=nsink)
    kr, vr = f64(k).copy(), f64(v).copy()
    O.kv_append(qkv, hq, hkv, D, tp, n, 1, pos, [1] * n, nsink, kr, vr)
    assert np.array_equal(f64(kg), kr) and np.array_equal(f64(vg), vr)
    q = f64(qkv)
    for b, t in enumerate(pos):
        slots = [O.cache_slot(j, nsink, cap) for j in [*range(nsink), *range(t - W + 1, t + 1)]]
        for hd in range(hq):
            g = hd // (hq // hkv)
            ref, mag = O.attend(q[b, hd * D:(hd + 1) * D], kr[b, g, slots], vr[b, g, slots])
            close(out[b, hd * D:(hd + 1) * D], ref, mag, f"position {t}")


# ============================================================ masks over clusters
def sample_by_numpy(logits, u, temperature, top_k, top_p, min_p):
    """sample_row with numpy's sorts and sums, for long rows."""
    l = f64(logits)
    l[np.isnan(l)] = -np.inf
    mx = l.max()
    if mx == -np.inf:
        return -1, -np.inf
    w = np.where(l == mx, 1.0, 0.0) if mx == np.inf else np.exp((l - mx) / temperature)
    order = np.lexsort((np.arange(len(l)), -l))[:top_k or len(l)]
    if top_p < 1:
        c = np.cumsum(w[order])
        order = order[np.concatenate([[0.0], c[:-1]]) < top_p * c[-1]]
    kept = np.sort(order)
    kept = kept[(w[kept] >= min_p) & (w[kept] > 0)]
    c = np.cumsum(w[kept])
    i = min(np.searchsorted(c, u * c[-1], side="right"), len(kept) - 1)
    return kept[i], math.log(w[kept[i]] / c[-1])


MASKS = {  # part of a row of V logits that is hidden, by token
    "tail": lambda i, V: i >= V - V * 5 // 32,
    "head": lambda i, V: i < V // 3,
    "all but the last few": lambda i, V: i < V - 11,
    "all but one": lambda i, V: i != V // 2 + 5,
    "middle and scattered": lambda i, V: ((i > V // 8) & (i < V // 2)) | (i % 3 == 0),
    "all": lambda i, V: i >= 0,
}


@pytest.mark.parametrize("m,V,dtype", [(6, 40000, torch.float32), (6, 128256, torch.bfloat16),
                                       (64, 128256, torch.bfloat16), (200, 70000, torch.float32)])
@pytest.mark.parametrize("hide", ["-inf", "nan", "lowest", "-1e4"])
def test_logits_sample_masks_over_clusters(T, m, V, dtype, hide):
    """Whole parts of the CTAs of a cluster hidden: by -inf, NaN, the type's lowest value, or -1e4.
    top_k is larger than what some masks leave."""
    value = {"-inf": -math.inf, "nan": math.nan, "lowest": torch.finfo(dtype).min, "-1e4": -1e4}[hide]
    logits, u, g = rows(len(MASKS), V, 1.5, 61, dtype)
    for r, mask in enumerate(MASKS.values()):
        logits[r, mask(torch.arange(V), V)] = value
    if math.isfinite(value):
        logits[-1, 0] = 0.0                    # a row of equal lowest values has weights; here all but one have none
    turn = torch.arange(m) % len(MASKS)
    none = dict(temperature=0.7, top_k=0, top_p=1.0, min_p=0.0)
    for kw in ({}, dict(top_k=50), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=3000, top_p=0.8), dict(top_k=9, min_p=0.2)):
        par = {**none, **kw}
        ref = [sample_by_numpy(logits[i], float(u[i]), *(float(np.float32(par[x])) if x != "top_k" else par[x] for x in none))
               for i in range(len(MASKS))]
        idx, logp = T.logits_sample(logits[turn].cuda(), u[turn].cuda(), **{
            x: torch.full((m,), y, dtype=torch.int32 if x == "top_k" else torch.float32, device="cuda") for x, y in par.items()})
        ri, rl = np.array([x[0] for x in ref])[turn], np.array([x[1] for x in ref])[turn]
        assert np.array_equal(idx.cpu().numpy(), ri), (kw, idx.tolist()[:6], ri.tolist()[:6])
        fin = np.isfinite(rl)
        assert np.allclose(f64(logp)[fin], rl[fin], rtol=2.0 ** -23, atol=1e-6)
        assert np.array_equal(f64(logp)[~fin], rl[~fin])


@pytest.mark.parametrize("m,V", [(6, 40000), (64, 128256)])
def test_logits_sample_infinities_over_clusters(T, m, V):
    """+inf in one CTA only, or in two, beside finite logits, -inf and NaN; top_k of one token, and
    of more than the others."""
    logits, u, g = rows(6, V, 1.5, 62)
    logits[0, V - 3] = math.inf
    logits[1, [5, V - 5]] = math.inf
    logits[2, :V // 2] = -math.inf
    logits[2, 1::2] = math.nan
    logits[3, V // 3] = math.inf
    logits[3, V // 2:] = -math.inf
    logits[4, 100:] = math.nan
    logits[4, :90] = -math.inf
    turn = torch.arange(m) % 6
    for k, p, q in ((0, 1.0, 0.0), (1, 1.0, 0.0), (V // 2 + 7, 1.0, 0.0), (0, 0.6, 0.0), (0, 1.0, 0.3), (40, 0.9, 0.01)):
        ref = [sample_by_numpy(logits[i], float(u[i]), 1.0, k, float(np.float32(p)), float(np.float32(q))) for i in range(6)]
        full = lambda x, t=torch.float32: torch.full((m,), x, dtype=t, device="cuda")
        idx, logp = T.logits_sample(logits[turn].cuda(), u[turn].cuda(), top_k=full(k, torch.int32), top_p=full(p), min_p=full(q))
        assert np.array_equal(idx.cpu().numpy(), np.array([x[0] for x in ref])[turn]), (k, p, q)
        assert np.allclose(f64(logp), np.array([x[1] for x in ref])[turn], rtol=2.0 ** -23, atol=1e-6)


@pytest.mark.parametrize("hide", [-math.inf, torch.finfo(torch.float32).min, -1e4])
@pytest.mark.parametrize("top_k,top_p", [(0, 0.9), (50, 1.0)])
def test_logits_sample_masked_rows_are_as_fast(T, hide, top_k, top_p):
    """A masked tail, or a mask that leaves 30 tokens, costs no more than three times the whole row:
    the cut is found from the bins and the list. Bit by bit it takes 64 passes over the row."""
    m, V = 8, 128256
    full = lambda x, t=torch.float32: torch.full((m,), x, dtype=t, device="cuda")
    kw = dict(top_k=full(top_k, torch.int32), top_p=full(top_p))
    logits, u, _ = rows(m, V, 0.5, 63)
    tail, few = logits.clone(), logits.clone()
    tail[:, V - 20000:] = hide
    few[:, 30:] = hide
    u = u.cuda()

    def time_us(l):
        l = l.cuda()
        best = math.inf
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(400_000)         # the calls are issued meanwhile
            a.record()
            for _ in range(10):
                T.logits_sample(l, u, **kw)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best
    whole = time_us(logits)
    times = [time_us(tail), time_us(few)]
    print(f"\nwhole {whole:.1f} us, masked tail {times[0]:.1f} us, 30 tokens {times[1]:.1f} us")
    assert max(times) <= 3 * whole, (whole, times)


def test_decode_workspace_serves_smaller_batches(T):
    """A workspace made for the largest batch serves it when rows leave, and other prefixes: the
    same bits as a workspace of the call's own. One made for a shorter prefix gives fewer parts."""
    hq, hkv, tp, P, cap = 32, 8, 8, 16384, 20
    nkv, cols = geom(hq, hkv, tp)
    h = T.Heads(hq, hkv, D)
    pk, pv = WL.gen_normal((nkv, P, D), 1.0, 1211), WL.gen_normal((nkv, P, D), 1.0, 1212)
    qkv, (k, v) = WL.gen_normal((65, cols), 1.0, 1213), caches(65, nkv, cap, 1214)
    shared, least = T.decode_workspace(65, h, tp, P), T.decode_workspace(65, h, tp, 1)
    for n, prefix in ((65, P), (64, P), (33, P), (32, P), (1, P), (64, 2304), (8, 2304), (65, 0), (1, 1)):
        x, kg, vg = qkv[:n].cuda(), k[:n].cuda().contiguous(), v[:n].cuda().contiguous()
        pos = torch.arange(n, dtype=torch.int32, device="cuda") % cap
        args = (pk[:, :prefix].cuda().contiguous(), pv[:, :prefix].cuda().contiguous()) if prefix else (None, None)
        call = lambda ws: T.sharded_prefix_decode(x, h, tp, *args, pos, kg, vg, ws)
        got = call(shared)
        assert torch.equal(got, call(T.decode_workspace(n, h, tp, prefix))), (n, prefix)
        if n == 33:
            ref, mag = O.cached_decode(qkv[:n], hq, hkv, D, tp, pos.tolist(), cap, 0, f64(k[:n]).copy(), f64(v[:n]).copy(),
                                       f64(pk), f64(pv))
            close(got, ref, mag)
            close(call(least), ref, mag)
    with pytest.raises(T.TpsError) as e:
        call(T.decode_workspace(1, h, tp))
    assert e.value.status == T.TPS_ERR_WORKSPACE


def test_prefix_decode_refuses_half_a_prefix(T):
    h = T.Heads(4, 2, D)
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    call = lambda pk, pv: T.sharded_prefix_decode(z(2, geom(4, 2, 2)[1]), h, 2, pk, pv, z(2, dtype=torch.int32), z(2, 2, 8, D),
                                                  z(2, 2, 8, D), T.decode_workspace(2, h, 2, 5))
    with pytest.raises(TypeError):
        call(None, z(2, 5, D))
    with pytest.raises(TypeError):
        call(z(2, 5, D), None)
    for pk in (z(5, D), z(1, 5, D), z(2, 5, 64), z(2, 10, D)[:, ::2]):
        with pytest.raises(ValueError):
            call(pk, z(2, 5, D))
