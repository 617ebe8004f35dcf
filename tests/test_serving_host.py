"""CPU checks of the serving operators: the oracle against closed forms and brute force,
and the host-side argument checks of the entry points (no call here launches a kernel)."""

import ctypes
import math

import numpy as np
import pytest

import oracle as O
import workloads as WL

GOOD = 1 << 20   # a 16-byte aligned address that the host never dereferences


@pytest.fixture(scope="module")
def T():
    import tensor_sharded_linear_columnparallel_b200 as T
    return T


# ---------------------------------------------------------------- oracle
def test_visible_positions_by_hand():
    assert O.visible_positions(0, 1, 0) == [0]
    assert O.visible_positions(5, 2, 0) == [4, 5]
    assert O.visible_positions(5, 2, 1) == [0, 4, 5]
    assert O.visible_positions(5, 100, 3) == [0, 1, 2, 3, 4, 5]
    assert O.visible_positions(3, 2, 9) == [0, 1, 2, 3]


@pytest.mark.parametrize("hq,hkv,tp", [(4, 2, 1), (4, 2, 2), (4, 2, 4), (4, 1, 2)])
def test_window_attention_limits(hq, hkv, tp):
    """A window of the whole sequence is causal attention; a window of one token without
    sinks returns that token's V; equal scores give the mean of the visible V rows."""
    d, S = 8, 7
    kvs = max(1, hkv // tp)
    qkv = O.to_f64(WL.gen_normal((2 * S, tp * (hq // tp + 2 * kvs) * d), 1.0, 7))
    ref = O.gqa_attention_sharded(qkv, hq, hkv, d, tp, 2, S, True)
    for w, ns in ((S, 0), (100, 3), (1, S)):
        assert np.allclose(O.window_attention_sharded(qkv, hq, hkv, d, tp, 2, S, w, ns)[0], ref, atol=1e-12)
    one, _ = O.window_attention_sharded(qkv, hq, hkv, d, tp, 2, S, 1, 0)
    x = qkv.reshape(2 * S, tp, hq // tp + 2 * kvs, d)
    G = hq // tp // kvs
    v = np.repeat(x[:, :, hq // tp + kvs:], G, axis=2).reshape(2 * S, hq * d)
    assert np.allclose(one, v, atol=1e-12)
    flat = qkv.copy().reshape(2 * S, tp, hq // tp + 2 * kvs, d)
    flat[:, :, :hq // tp] = 0.0
    got, _ = O.window_attention_sharded(flat.reshape(2 * S, -1), hq, hkv, d, tp, 2, S, 2, 1)
    vb = v.reshape(2, S, hq * d)
    assert np.allclose(got.reshape(2, S, -1)[1, 5], (vb[1, 0] + vb[1, 4] + vb[1, 5]) / 3, atol=1e-12)


def test_cache_slots_are_a_ring_behind_the_sinks():
    assert [O.cache_slot(t, 2, 5) for t in range(9)] == [0, 1, 2, 3, 4, 2, 3, 4, 2]
    assert [O.cache_slot(t, 0, 3) for t in range(5)] == [0, 1, 2, 0, 1]


@pytest.mark.parametrize("window,nsink,cap", [(4, 0, 4), (3, 2, 9), (5, 1, 6), (16, 0, 16)])
def test_decode_steps_equal_prefill(window, nsink, cap):
    """Tokens decoded one by one through the ring give the rows of the windowed prefill."""
    hq, hkv, d, tp, S = 4, 2, 8, 2, 13
    qkv = O.to_f64(WL.gen_normal((S, tp * (2 + 2) * d), 1.0, 11))
    ref, _ = O.window_attention_sharded(qkv, hq, hkv, d, tp, 1, S, window, nsink)
    k, v = np.full((1, 2, cap, d), np.nan), np.full((1, 2, cap, d), np.nan)
    for t in range(S):
        got, _ = O.cached_decode(qkv[t:t + 1], hq, hkv, d, tp, [t], window, nsink, k, v)
        assert np.allclose(got[0], ref[t], atol=1e-12), t


def test_prefix_is_the_same_as_a_longer_sequence():
    hq, hkv, d, tp = 2, 1, 8, 1
    qkv = O.to_f64(WL.gen_normal((6, 4 * d), 1.0, 12))
    ref = O.gqa_attention_sharded(qkv, hq, hkv, d, tp, 1, 6, True)
    pk, pv = qkv[None, :4, 2 * d:3 * d], qkv[None, :4, 3 * d:]
    k, v = np.zeros((1, 1, 3, d)), np.zeros((1, 1, 3, d))
    for t in range(2):
        got, _ = O.cached_decode(qkv[4 + t:5 + t], hq, hkv, d, tp, [t], 3, 0, k, v, pk, pv)
        assert np.allclose(got[0], ref[4 + t], atol=1e-12)


def test_sample_row_by_hand():
    l = np.log([1.0, 4.0, 2.0, 1.0])
    for u, want in ((0.0, 0), (0.124, 0), (0.126, 1), (0.62, 1), (0.63, 2), (0.88, 3), (0.9999, 3)):
        assert O.sample_row(l, u)[0] == want
    assert O.sample_row(l, 0.5)[1] == pytest.approx(math.log(0.5))
    assert [O.sample_row(l, u, top_k=2)[0] for u in (0.0, 0.6, 0.7)] == [1, 1, 2]
    assert [O.sample_row(l, u, top_k=3)[0] for u in (0.0, 0.2, 0.99)] == [0, 1, 2]    # the tie keeps index 0
    assert [O.sample_row(l, u, top_p=0.5)[0] for u in (0.0, 0.99)] == [1, 1]           # 4/8 reaches 0.5 by itself
    assert [O.sample_row(l, u, top_p=0.51)[0] for u in (0.0, 0.99)] == [1, 2]
    assert [O.sample_row(l, u, min_p=0.3)[0] for u in (0.0, 0.99)] == [1, 2]
    assert [O.sample_row(l, u, top_k=2, top_p=0.6)[0] for u in (0.0, 0.99)] == [1, 1]  # 4/6 of the two left
    assert O.sample_row(l, 0.7, temperature=0.0) == (1, 0.0)
    assert O.sample_row([2.0, 2.0], 0.9, temperature=-1.0)[0] == 0
    assert O.sample_row([-np.inf, np.nan, 1.0], 0.0)[0] == 2
    assert O.sample_row([-np.inf, np.nan], 0.0) == (-1, -np.inf)
    assert O.sample_row([np.inf, 3.0, np.inf], 0.6)[0] == 2
    assert O.sample_row(l, 1.0)[0] == 3


@pytest.mark.parametrize("mistake", ["drop_sink", "include_old", "ring_without_sinks"])
def test_planted_window_mistakes_show(mistake):
    hq, hkv, d, tp, S, W, ns, cap = 2, 1, 8, 1, 9, 3, 1, 5
    qkv = O.to_f64(WL.gen_normal((S, 4 * d), 1.0, 13))
    ref, _ = O.window_attention_sharded(qkv, hq, hkv, d, tp, 1, S, W, ns)
    if mistake == "ring_without_sinks":
        k, v = np.zeros((1, 1, cap, d)), np.zeros((1, 1, cap, d))
        for t in range(S):
            O.kv_append(qkv[t:t + 1], hq, hkv, d, tp, 1, 1, [t], [1], 0, k, v)
        got, _ = O.cached_decode(qkv[S - 1:], hq, hkv, d, tp, [S - 1], W, ns, k, v)
        assert not np.allclose(got[0], ref[-1], atol=1e-3)
    else:
        w, s = (W, 0) if mistake == "drop_sink" else (W + 1, ns)
        got, _ = O.window_attention_sharded(qkv, hq, hkv, d, tp, 1, S, w, s)
        assert not np.allclose(got, ref, atol=1e-3)


# ---------------------------------------------------------------- host-side checks
def heads(T, hq=32, hkv=8, d=128):
    return ctypes.byref(T.tps_heads(hq, hkv, d))


def test_window_attention_checks(T):
    f, h = T.lib.sharded_window_attention, heads(T)
    call = lambda qkv=GOOD, n=1, S=16, hd=h, tp=8, w=4, ns=1, out=GOOD: f(qkv, n, S, hd, tp, w, ns, out, None)
    assert call(hd=None) == T.TPS_ERR_ARG
    assert call(w=0) == T.TPS_ERR_ARG
    assert call(ns=-1) == T.TPS_ERR_ARG
    assert call(n=-1) == T.TPS_ERR_ARG
    assert call(n=1 << 20, S=1 << 20) == T.TPS_ERR_ARG
    assert call(tp=3) == T.TPS_ERR_DIVISIBILITY
    assert call(hd=heads(T, d=64)) == T.TPS_ERR_UNIMPLEMENTED
    assert call(qkv=None) == T.TPS_ERR_ARG
    assert call(out=GOOD + 8) == T.TPS_ERR_ALIGN
    assert call(S=0, qkv=None, out=None) == T.TPS_OK


def test_kv_append_checks(T):
    f, h = T.lib.sharded_kv_append, heads(T)
    def call(qkv=GOOD, n=2, S=4, hd=h, tp=8, pos=GOOD, cnt=GOOD, ns=1, k=GOOD, v=GOOD, cap=8):
        return f(qkv, n, S, hd, tp, pos, cnt, ns, k, v, cap, None)
    assert call(hd=None) == T.TPS_ERR_ARG
    assert call(ns=8) == T.TPS_ERR_ARG          # no slot behind the sinks
    assert call(ns=-1) == T.TPS_ERR_ARG
    assert call(cap=0) == T.TPS_ERR_ARG
    assert call(cap=1 << 31) == T.TPS_ERR_ARG
    assert call(S=-1) == T.TPS_ERR_ARG
    assert call(tp=5) == T.TPS_ERR_DIVISIBILITY
    assert call(hd=heads(T, d=96)) == T.TPS_ERR_UNIMPLEMENTED
    assert call(v=None) == T.TPS_ERR_ARG
    assert call(k=GOOD + 4) == T.TPS_ERR_ALIGN
    assert call(pos=GOOD + 2) == T.TPS_ERR_ALIGN
    assert call(n=0, qkv=None, k=None, v=None) == T.TPS_OK


def test_decode_checks(T):
    h = heads(T)
    need = T.lib.tps_decode_workspace_bytes(2, h, 8, 0)
    assert need >= 256
    def win(qkv=GOOD, n=2, hd=h, tp=8, pos=GOOD, w=4, ns=1, k=GOOD, v=GOOD, cap=8, out=GOOD, ws=GOOD, nb=need):
        return T.lib.sharded_window_decode(qkv, n, hd, tp, pos, w, ns, k, v, cap, out, ws, nb, None)
    assert win(hd=None) == T.TPS_ERR_ARG
    assert win(w=0) == T.TPS_ERR_ARG
    assert win(w=8) == T.TPS_ERR_ARG            # longer than the ring behind the sink
    assert win(ns=8) == T.TPS_ERR_ARG
    assert win(n=-1) == T.TPS_ERR_ARG
    assert win(pos=None) == T.TPS_ERR_ARG
    assert win(ws=None) == T.TPS_ERR_ARG
    assert win(nb=need - 1) == T.TPS_ERR_WORKSPACE
    assert win(tp=7) == T.TPS_ERR_DIVISIBILITY
    assert win(hd=heads(T, d=256)) == T.TPS_ERR_UNIMPLEMENTED
    assert win(out=GOOD + 2) == T.TPS_ERR_ALIGN
    assert win(n=0, qkv=None, pos=None, k=None, v=None, out=None, ws=None, nb=0) == T.TPS_OK
    need_p = T.lib.tps_decode_workspace_bytes(2, h, 8, 1000)
    assert need_p >= need
    def pre(qkv=GOOD, n=2, hd=h, tp=8, pk=GOOD, pv=GOOD, P=1000, pos=GOOD, k=GOOD, v=GOOD, cap=8, out=GOOD, ws=GOOD,
            nb=need_p):
        return T.lib.sharded_prefix_decode(qkv, n, hd, tp, pk, pv, P, pos, k, v, cap, out, ws, nb, None)
    assert pre(P=-1) == T.TPS_ERR_ARG
    assert pre(pk=None) == T.TPS_ERR_ARG
    assert pre(pv=GOOD + 8) == T.TPS_ERR_ALIGN
    assert pre(cap=0) == T.TPS_ERR_ARG
    assert pre(nb=16) == T.TPS_ERR_WORKSPACE
    assert pre(n=0) == T.TPS_OK
    assert T.lib.tps_decode_workspace_bytes(2, heads(T, d=64), 8, 0) == 0
    assert T.lib.tps_decode_workspace_bytes(-1, h, 8, 0) == 0
    assert T.lib.tps_decode_workspace_bytes(2, h, 3, 0) == 0
    assert T.lib.tps_decode_workspace_bytes(2, None, 8, 0) == 0


def test_sampling_checks(T):
    def smp(l=GOOD, dt=T.DTYPE_F32, m=2, V=64, u=GOOD, t=None, k=None, p=None, q=None, idx=GOOD, lp=None):
        return T.lib.logits_sample(l, dt, m, V, u, t, k, p, q, idx, lp, None)
    assert smp(dt=3) == T.TPS_ERR_DTYPE
    assert smp(V=60) == T.TPS_ERR_ALIGN
    assert smp(V=0) == T.TPS_ERR_ARG
    assert smp(m=-1) == T.TPS_ERR_ARG
    assert smp(V=393224) == T.TPS_ERR_UNIMPLEMENTED
    assert smp(u=None) == T.TPS_ERR_ARG
    assert smp(idx=None) == T.TPS_ERR_ARG
    assert smp(l=GOOD + 4) == T.TPS_ERR_ALIGN
    assert smp(k=GOOD + 1) == T.TPS_ERR_ALIGN
    assert smp(m=0, l=None, u=None, idx=None) == T.TPS_OK
    need = T.tps_workspace_bytes(T.FN_SAMPLE, 2, 64, 32, 2)
    assert need >= 256 + 2 * 64 * 4
    def vps(X=GOOD, m=2, H=32, w=GOOD, V=64, tp=2, u=GOOD, idx=GOOD, ws=GOOD, nb=need):
        return T.lib.vocab_parallel_sample(X, m, H, w, V, tp, u, None, None, None, None, idx, None, ws, nb, None)
    assert vps(tp=3) == T.TPS_ERR_DIVISIBILITY
    assert vps(V=72) == T.TPS_ERR_ALIGN          # 36 columns per shard
    assert vps(ws=None) == T.TPS_ERR_ARG
    assert vps(nb=256) == T.TPS_ERR_WORKSPACE
    assert vps(m=-1) == T.TPS_ERR_ARG
    assert vps(m=0, X=None, ws=None, nb=0) == T.TPS_OK


@pytest.mark.parametrize("hq,hkv,tp", [(32, 8, 8), (32, 8, 4), (64, 8, 8), (28, 4, 2), (16, 1, 4), (32, 32, 4), (4, 1, 1)])
def test_decode_workspace_grows_with_its_sizes(T, hq, hkv, tp):
    """A workspace for a batch behind a prefix is large enough for fewer sequences and shorter prefixes."""
    h = heads(T, hq, hkv)
    lens = (0, 1, 128, 1000, 2304, 5000, 16384, 100000)
    need = np.array([[T.lib.tps_decode_workspace_bytes(n, h, tp, P) for P in lens] for n in range(0, 260)], dtype=np.int64)
    assert (need > 0).all()
    assert (np.diff(need, axis=0) >= 0).all(), np.argwhere(np.diff(need, axis=0) < 0)[:5]
    assert (np.diff(need, axis=1) >= 0).all(), np.argwhere(np.diff(need, axis=1) < 0)[:5]


def test_workspaces_on_a_device_given_by_number(T, monkeypatch):
    """Device 0 is the first GPU, not the current one."""
    import contextlib
    seen = []
    monkeypatch.setattr(T.torch, "zeros", lambda *a, device, **k: seen.append(T.torch.device(device)))
    monkeypatch.setattr(T.torch.cuda, "device", lambda d: contextlib.nullcontext())
    for given, want in ((0, "cuda:0"), (1, "cuda:1"), ("cuda:1", "cuda:1"), (None, "cuda")):
        T.workspace(T.FN_SAMPLE, 1, 64, 64, 1, device=given)
        T.decode_workspace(1, T.Heads(4, 2, 128), 1, device=given)
        assert [str(d) for d in seen] == [want] * 2
        seen.clear()
