"""Serving operators of the sharded Transformer block: what each costs and computes.

Five operators, each in a plain form (elementary torch operations) and as a call of
the framework:

* ``window_attention``  prefill attention on local heads with a sliding window and a
  few first tokens that stay visible
* ``kv_append``         K and V of a QKV output into the shards' KV caches (rings
  behind the first tokens)
* ``window_decode``     one new token per sequence against such a cache
* ``prefix_decode``     one new token per sequence of a batch that shares a prefix
* ``sample``            temperature, top-k, top-p and min-p sampling, from logits or
  over the vocabulary-parallel lm_head

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from a seed,
``run`` is one pass, ``work`` the bytes and operations that the pass cannot do
without, ``exact`` the same outputs in 64 bits.
"""

import math

import torch

own = False

D = 128   # head dimension of the attention on local heads


# ---------------------------------------------------------------- cases
def listed():
    return [
        # prefill of a medium prompt with a short window, the block's 32/8-head geometry
        dict(name="window_attention_s2048", op="window_attention", nseq=1, S=2048, hq=32, hkv=8, tp=8, window=512,
             nsink=4),
        # a small batch of ragged-size prompts, window and sinks off the 128 grid, KV heads replicated
        dict(name="window_attention_odd", op="window_attention", nseq=3, S=1337, hq=32, hkv=4, tp=8, window=301,
             nsink=37),
        # long-context prefill with the 64/8-head geometry: the largest attention
        dict(name="window_attention_s16384", op="window_attention", nseq=1, S=16384, hq=64, hkv=8, tp=8, window=4096,
             nsink=4),
        # a prompt's K and V into the ring behind the sinks; more tokens than the ring holds
        dict(name="kv_append_prompt", op="kv_append", nseq=4, S=2048, hq=32, hkv=8, tp=8, cap=1028, nsink=4),
        # one token of a small decode batch, the call a serving loop makes every step
        dict(name="kv_append_token", op="kv_append", nseq=16, S=1, hq=32, hkv=8, tp=8, cap=2052, nsink=4),
        # a single user's step: latency
        dict(name="window_decode_b1", op="window_decode", nseq=1, hq=32, hkv=8, tp=8, cap=2052, nsink=4, window=2048,
             maxpos=6000, idle=0),
        # a full decode batch in steady state, caches far larger than L2
        dict(name="window_decode_b32", op="window_decode", nseq=32, hq=32, hkv=8, tp=8, cap=4100, nsink=4,
             window=4096, maxpos=20000, idle=0),
        # a few users behind a system prompt, one slot of the batch unused
        dict(name="prefix_decode_b8", op="prefix_decode", nseq=8, hq=32, hkv=8, tp=8, prefix=1000, cap=256, idle=1),
        # a large batch behind a long document
        dict(name="prefix_decode_b64", op="prefix_decode", nseq=64, hq=32, hkv=8, tp=8, prefix=16384, cap=512, idle=0),
        # one row of a Llama-3-sized vocabulary: latency
        dict(name="sample_m1", op="sample", m=1, V=128256, H=0, tp=1, f32=True, spread=2.5, filters=7),
        # a decode batch of bf16 logits, every row with its own parameters, some without filters
        dict(name="sample_m64", op="sample", m=64, V=128256, H=0, tp=1, f32=False, spread=1.5, filters=-1),
        # the whole step: lm_head and sampling
        dict(name="sample_lm_head_m32", op="sample", m=32, V=128256, H=4096, tp=8, f32=True, spread=1.0, filters=7),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window_attention", "kv_append", "window_decode", "prefix_decode", "sample"])
    hq, hkv, tp = rng.choice([(32, 8, 8), (32, 8, 4), (64, 8, 8), (32, 4, 8), (32, 32, 4), (28, 4, 2), (16, 1, 4)])
    case = dict(op=op)
    if op == "window_attention":
        S = _logint(rng, 1, 8192)
        nseq = max(1, min(_logint(rng, 1, 16), 16384 // S))
        case.update(nseq=nseq, S=S, hq=hq, hkv=hkv, tp=tp, window=_logint(rng, 1, max(2, S)),
                    nsink=rng.choice([0, 1, 4, 16, 77, 130]))
    elif op == "kv_append":
        S = _logint(rng, 1, 4096)
        nseq = max(1, min(_logint(rng, 1, 64), 16384 // S))
        nsink = rng.choice([0, 1, 4, 64])
        case.update(nseq=nseq, S=S, hq=hq, hkv=hkv, tp=tp, cap=nsink + _logint(rng, 1, 4096), nsink=nsink)
    elif op == "window_decode":
        nsink = rng.choice([0, 1, 4, 64, 200])
        window = _logint(rng, 1, 8192)
        nkv = max(tp, hkv)
        nseq = max(1, min(_logint(rng, 1, 128), (32 * 4100 * 8) // ((window + nsink) * nkv)))
        case.update(nseq=nseq, hq=hq, hkv=hkv, tp=tp, cap=nsink + window + rng.choice([0, 0, 5, 100]), nsink=nsink,
                    window=window, maxpos=_logint(rng, 1, 30000), idle=rng.choice([0, 0, 1]))
    elif op == "prefix_decode":
        nkv = max(tp, hkv)
        prefix = rng.choice([0, _logint(rng, 1, 16384), _logint(rng, 128, 16384)])
        cap = _logint(rng, 1, 1024)
        nseq = max(1, min(_logint(rng, 1, 128), (64 * 512 * 8) // (cap * nkv)))
        case.update(nseq=nseq, hq=hq, hkv=hkv, tp=tp, prefix=prefix, cap=cap, idle=rng.choice([0, 0, 1]))
    else:
        V = 8 * _logint(rng, 1, 16032)
        m = max(1, min(_logint(rng, 1, 128), (64 * 128256) // V))
        case.update(m=m, V=V, H=rng.choice([0, 0, 256, 1024]), tp=1, f32=rng.random() < 0.5,
                    spread=rng.choice([0.5, 1.5, 2.5, 6.0]), filters=rng.choice([0, 1, 2, 4, 3, 7, -1, -1]))
        if case["H"]:
            case["f32"] = True
            case["spread"] = 1.0
    return case


# ---------------------------------------------------------------- inputs
def _geom(case):
    hq, hkv, tp = case["hq"], case["hkv"], case["tp"]
    qs = hq // tp
    kvs = hkv // tp if hkv % tp == 0 else 1
    return qs, kvs, tp * kvs, tp * (qs + 2 * kvs) * D


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _positions(g, n, hi, idle):
    """Positions 0..hi of the new tokens, int32; `idle` slots of the batch carry -1."""
    pos = torch.randint(0, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    if idle and n > 1:
        pos[torch.randint(0, n, (1,), generator=g, device="cuda")] = -1
    return pos


def _sample_inputs(case, g):
    m, V, H = case["m"], case["V"], case["H"]
    st = {}
    if H:
        # multiples of 1/8 and of a power of two: every logit is exact in 32 bits, so the
        # token does not depend on the order in which a product is summed
        st["X"] = ((_randn(g, m, H, dtype=torch.float32) * 8).round() / 8).clamp(-4, 4).to(torch.bfloat16)
        s = 2.0 ** round(math.log2(2.0 / math.sqrt(H)))
        W = torch.empty(H, V, device="cuda", dtype=torch.bfloat16)
        for a in range(0, H, 256):
            w = torch.randn(min(256, H - a), V, generator=g, device="cuda")
            W[a:a + 256] = (w * 4).round().div_(4).clamp_(-4, 4).mul_(s).to(torch.bfloat16)
        st["W"] = W
    else:
        st["logits"] = _randn(g, m, V, dtype=torch.float32).mul_(case["spread"])
        if not case["f32"]:
            st["logits"] = st["logits"].to(torch.bfloat16)
    f = case["filters"]
    on = [torch.ones(m, device="cuda", dtype=torch.bool) if f < 0 or f >> b & 1 else None for b in range(3)]
    if f < 0:   # every row switches each filter on or off for itself
        on = [torch.rand(m, generator=g, device="cuda") < 0.5 for _ in range(3)]
    rnd = lambda: torch.rand(m, generator=g, device="cuda")
    st["temperature"] = 0.3 + 1.2 * rnd()
    k = (1 + 199 * rnd()).to(torch.int32)
    p = 0.5 + 0.49 * rnd()
    q = 0.01 + 0.1 * rnd()
    st["top_k"] = None if on[0] is None else torch.where(on[0], k, torch.zeros_like(k))
    st["top_p"] = None if on[1] is None else torch.where(on[1], p, torch.ones_like(p))
    st["min_p"] = None if on[2] is None else torch.where(on[2], q, torch.zeros_like(q))
    st["u"] = rnd()
    return st


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "sample":
        return _sample_inputs(case, g)
    qs, kvs, nkv, cols = _geom(case)
    n = case["nseq"]
    st = {"qkv": _randn(g, n * case.get("S", 1), cols)}
    if op == "window_attention":
        return st
    st["k"] = _randn(g, n, nkv, case["cap"], D)
    st["v"] = _randn(g, n, nkv, case["cap"], D)
    if op == "kv_append":
        st["pos"] = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
        st["count"] = torch.randint(max(1, case["S"] // 2), case["S"] + 1, (n,), generator=g, device="cuda",
                                    dtype=torch.int32)
    elif op == "window_decode":
        st["pos"] = _positions(g, n, case["maxpos"], case["idle"])
    else:
        st["pos"] = _positions(g, n, case["cap"] - 1, case["idle"])
        st["pk"] = _randn(g, nkv, case["prefix"], D)
        st["pv"] = _randn(g, nkv, case["prefix"], D)
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = dict(case)
    if own:
        import tensor_sharded_linear_columnparallel_b200 as T
        if case["op"] == "sample":
            if case["H"]:
                st["packed"] = T.tp_shard_weights(T.KIND_COLUMN, st.pop("W"), case["tp"])
                st["ws"] = T.workspace(T.FN_SAMPLE, case["m"], case["V"], case["H"], case["tp"])
        else:
            st["heads"] = T.Heads(case["hq"], case["hkv"], D)
            if case["op"] in ("window_decode", "prefix_decode"):
                st["ws"] = T.decode_workspace(case["nseq"], st["heads"], case["tp"], case.get("prefix", 0))
    return st


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if own:
        return _own(case["op"], case, state)
    return _PLAIN[case["op"]](case, state)


def _own(op, case, st):
    import tensor_sharded_linear_columnparallel_b200 as T
    if op == "window_attention":
        return T.sharded_window_attention(st["qkv"], case["nseq"], case["S"], st["heads"], case["tp"], case["window"],
                                          case["nsink"])
    if op == "kv_append":
        T.sharded_kv_append(st["qkv"], case["nseq"], case["S"], st["heads"], case["tp"], st["k"], st["v"],
                            pos=st["pos"], count=st["count"], nsink=case["nsink"])
        return st["k"], st["v"]
    if op == "window_decode":
        out = T.sharded_window_decode(st["qkv"], st["heads"], case["tp"], st["pos"], case["window"], st["k"], st["v"],
                                      st["ws"], nsink=case["nsink"])
        return out, st["k"], st["v"]
    if op == "prefix_decode":
        out = T.sharded_prefix_decode(st["qkv"], st["heads"], case["tp"], st["pk"], st["pv"], st["pos"], st["k"],
                                      st["v"], st["ws"])
        return out, st["k"], st["v"]
    kw = dict(temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
    if case["H"]:
        return T.vocab_parallel_sample(st["X"], case["H"], case["V"], case["tp"], st["packed"], st["u"], st["ws"],
                                       **kw)
    return T.logits_sample(st["logits"], st["u"], **kw)


def _split(case, qkv, nseq, S):
    """q [nseq, S, nkv, G, D], k and v [nseq, S, nkv, D] of a shard-major QKV output."""
    qs, kvs, nkv, _ = _geom(case)
    x = qkv.view(nseq, S, case["tp"], qs + 2 * kvs, D)
    q = x[:, :, :, :qs].reshape(nseq, S, nkv, qs // kvs, D)
    k = x[:, :, :, qs:qs + kvs].reshape(nseq, S, nkv, D)
    v = x[:, :, :, qs + kvs:].reshape(nseq, S, nkv, D)
    return q, k, v


def _softmax(s):
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(s - m)
    return e / e.sum(-1, keepdim=True).clamp_min(1e-38)


def _plain_window_attention(case, st):
    nseq, S, W, ns = case["nseq"], case["S"], case["window"], case["nsink"]
    q, k, v = _split(case, st["qkv"], nseq, S)
    out = torch.empty(nseq, S, case["hq"] * D, device="cuda", dtype=torch.bfloat16)
    scale = 1.0 / math.sqrt(D)
    for b in range(nseq):
        kf, vf = k[b].float().transpose(0, 1), v[b].float().transpose(0, 1)   # [nkv, S, D]
        for a in range(0, S, 512):
            e = min(S, a + 512)
            lo = max(0, a - W + 1)
            keys = torch.cat([torch.arange(0, min(ns, lo), device="cuda"), torch.arange(lo, e, device="cuda")])
            t = torch.arange(a, e, device="cuda")[:, None]
            see = (keys <= t) & ((t - keys < W) | (keys < ns))                  # [T, J]
            qf = q[b, a:e].float().permute(1, 2, 0, 3)                          # [nkv, G, T, D]
            nkv, G, n, _ = qf.shape
            s = torch.matmul(qf.reshape(nkv, G * n, D), kf[:, keys].transpose(1, 2)) * scale
            s = s.view(nkv, G, n, -1).masked_fill(~see, -math.inf)
            o = torch.matmul(_softmax(s).view(nkv, G * n, -1), vf[:, keys])
            out[b, a:e] = o.view(nkv * G, n, D).transpose(0, 1).reshape(n, -1)
    return out.view(nseq * S, -1)


def _slot(t, nsink, cap):
    """Cache slot of position t: the first nsink positions keep theirs, the rest share a ring."""
    return torch.where(t < nsink, t, nsink + (t - nsink) % max(1, cap - nsink))


def _plain_kv_append(case, st):
    nseq, S, cap, ns = case["nseq"], case["S"], case["cap"], case["nsink"]
    _, k, v = _split(case, st["qkv"], nseq, S)
    pos, last = st["pos"].long()[:, None], (st["pos"] + st["count"]).long()[:, None]   # first, one past the newest
    R = max(1, cap - ns)
    b = torch.arange(nseq, device="cuda")[:, None]
    if S <= R:                                              # every token has a slot of its own
        t = pos + torch.arange(S, device="cuda")[None, :]
        s = _slot(t, ns, cap)
        for name, new in (("k", k), ("v", v)):
            st[name][b, :, s] = torch.where((t < last)[:, :, None, None], new, st[name][b, :, s])
        return st["k"], st["v"]
    j = torch.arange(cap, device="cuda")[None, :]
    ring = last - 1 - (last - 1 - j) % R                    # the newest position that ring slot j can hold
    p = torch.where(j < ns, j, ring)
    take = (p >= pos) & (p < last) & ((j < ns) | (p >= ns))
    src = (p - pos).clamp(0, S - 1)
    for name, new in (("k", k), ("v", v)):
        st[name].copy_(torch.where(take[:, None, :, None], new[b, src].transpose(1, 2), st[name]))
    return st["k"], st["v"]


def _decode(case, st, live, s, see, pk=None, pv=None):
    """Append the new tokens of the live rows at slots s, then attend: see [n, cap] says which
    slots each row sees, pk and pv are a prefix that every row sees first."""
    q, k, v = _split(case, st["qkv"], case["nseq"], 1)
    b = torch.arange(case["nseq"], device="cuda")
    for name, new in (("k", k), ("v", v)):
        st[name][b, :, s] = torch.where(live[:, None, None], new[:, 0], st[name][b, :, s])
    out = torch.zeros(case["nseq"], case["hq"] * D, device="cuda", dtype=torch.bfloat16)
    scale = 1.0 / math.sqrt(D)
    nkv, G = q.shape[2], q.shape[3]
    step = 8
    pkf = None if pk is None else pk.float()
    pvf = None if pv is None else pv.float()
    for a in range(0, case["nseq"], step):
        e = min(case["nseq"], a + step)
        n = e - a
        qf = q[a:e, 0].float()                                                    # [n, nkv, G, D]
        sc = torch.matmul(qf, st["k"][a:e].float().transpose(2, 3)) * scale       # [n, nkv, G, cap]
        sc = sc.masked_fill(~(see[a:e] & live[a:e, None])[:, None, None, :], -math.inf)
        vs = st["v"][a:e].float().masked_fill(~see[a:e][:, None, :, None], 0.0)
        if pk is not None and pk.shape[1]:
            qp = qf.permute(1, 0, 2, 3).reshape(nkv, n * G, D)
            sp = torch.matmul(qp, pkf.transpose(1, 2)) * scale
            sc = torch.cat([sp.view(nkv, n, G, -1).transpose(0, 1), sc], -1)
        p = _softmax(sc)
        P = sc.shape[-1] - see.shape[-1]
        o = torch.matmul(p[..., P:], vs)
        if P:
            pp = p[..., :P].permute(1, 0, 2, 3).reshape(nkv, n * G, P)
            o = o + torch.matmul(pp, pvf).view(nkv, n, G, D).transpose(0, 1)
        out[a:e] = torch.where(live[a:e, None], o.reshape(n, -1), torch.zeros((), device="cuda")).to(torch.bfloat16)
    return out, st["k"], st["v"]


def _plain_window_decode(case, st):
    cap, ns, W = case["cap"], case["nsink"], case["window"]
    pos = st["pos"].long()
    live = pos >= 0
    t = pos.clamp_min(0)
    R = cap - ns
    j = torch.arange(cap, device="cuda")[None, :]
    age = (t[:, None] - ns - (j - ns)) % R                 # tokens between the newest and the one in ring slot j
    ring = (j >= ns) & (age < W) & (t[:, None] - age >= ns)
    see = ((j < ns) & (j <= t[:, None])) | ring
    return _decode(case, st, live, _slot(t, ns, cap), see)


def _plain_prefix_decode(case, st):
    pos = st["pos"].long()
    live = (pos >= 0) & (pos < case["cap"])
    t = pos.clamp_min(0)
    see = torch.arange(case["cap"], device="cuda")[None, :] <= t[:, None]
    return _decode(case, st, live, t, see, st["pk"], st["pv"])


def _plain_sample(case, st):
    if case["H"]:
        logits = torch.matmul(st["X"].float(), st["W"].float())
    else:
        logits = st["logits"].float()
    m, V = logits.shape
    l = logits.double()   # 64 bits: the draw falls next to the borders of a cumulative sum
    w = torch.exp((l - l.amax(1, keepdim=True)) / st["temperature"].double()[:, None])
    if st["top_k"] is not None or st["top_p"] is not None:
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices
        ws = w.gather(1, order)
        rank = torch.arange(V, device="cuda")[None, :]
        keep = torch.ones_like(ws, dtype=torch.bool)
        if st["top_k"] is not None:
            k = st["top_k"][:, None]
            keep &= (k <= 0) | (rank < k)
        if st["top_p"] is not None:
            p = st["top_p"].double()[:, None]
            ks = ws * keep
            cum = ks.cumsum(1)
            keep &= (p >= 1) | (cum - ks < p * cum[:, -1:]) | (rank == 0)
        w = torch.zeros_like(w).scatter(1, order, torch.where(keep, ws, torch.zeros_like(ws)))
    if st["min_p"] is not None:
        w = torch.where(w >= st["min_p"].double()[:, None], w, torch.zeros_like(w))
    cdf = w.cumsum(1)
    hit = cdf > st["u"].double()[:, None] * cdf[:, -1:]
    idx = hit.to(torch.int8).argmax(1)
    logp = torch.log(w.gather(1, idx[:, None])[:, 0] / cdf[:, -1])
    return idx.to(torch.int32), logp.float()


_PLAIN = {"window_attention": _plain_window_attention, "kv_append": _plain_kv_append,
          "window_decode": _plain_window_decode, "prefix_decode": _plain_prefix_decode, "sample": _plain_sample}


# ---------------------------------------------------------------- work
def _visible(t, W, ns):
    """Keys that the query at position t sees."""
    return min(t + 1, W) + min(ns, max(0, t + 1 - W))


def _expected_positions(case, hi):
    """A spread of positions standing for the seed's (the count does not depend on the seed)."""
    n = case["nseq"]
    live = n - (1 if case["idle"] and n > 1 else 0)
    return [int((i + 0.5) * (hi + 1) / live) for i in range(live)]


def work(case):
    op = case["op"]
    if op == "sample":
        m, V, H = case["m"], case["V"], case["H"]
        b = 28 * m
        if H:
            return {"bytes": b + 2 * H * V + 2 * m * H, "flops": 2 * m * H * V + 2 * m * V}
        return {"bytes": b + m * V * (4 if case["f32"] else 2), "flops": 2 * m * V}
    qs, kvs, nkv, cols = _geom(case)
    n, hq = case["nseq"], case["hq"]
    if op == "window_attention":
        S = case["S"]
        pairs = sum(_visible(t, case["window"], case["nsink"]) for t in range(S)) * n
        return {"bytes": 2 * n * S * (cols + hq * D), "flops": 4 * D * hq * pairs}
    if op == "kv_append":
        S = case["S"]
        rows = n * min((S + max(1, S // 2)) / 2, case["cap"])
        return {"bytes": int(rows * nkv * D * 2 * 2 * 2), "flops": 0}
    row = 2 * nkv * D * 2                                   # K and V of one token, every shard
    if op == "window_decode":
        seen = sum(_visible(t, case["window"], case["nsink"]) for t in _expected_positions(case, case["maxpos"]))
        return {"bytes": seen * row + n * (2 * cols + row + 2 * hq * D), "flops": 4 * D * hq * seen}
    seen = sum(t + 1 for t in _expected_positions(case, case["cap"] - 1))
    P = case["prefix"]
    return {"bytes": (seen + P) * row + n * (2 * cols + row + 2 * hq * D), "flops": 4 * D * hq * (seen + P * n)}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = _inputs(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(case, st)
    if op == "kv_append":
        return _exact_kv_append(case, st)
    n, hq, hkv, tp = case["nseq"], case["hq"], case["hkv"], case["tp"]
    qs, kvs, nkv, cols = _geom(case)
    S = case.get("S", 1)
    rows = st["qkv"].view(n, S, cols)
    out = torch.zeros(n, S, hq * D, device="cuda", dtype=torch.float64)
    pos = st["pos"].tolist() if "pos" in st else None
    for h in range(hq):
        r, lq = divmod(h, qs)
        lk = lq // (qs // kvs)
        base = r * (qs + 2 * kvs) * D
        qc, kc, vc = base + lq * D, base + (qs + lk) * D, base + (qs + kvs + lk) * D
        for b in range(n):
            Q = rows[b, :, qc:qc + D].double()
            K, V = rows[b, :, kc:kc + D].double(), rows[b, :, vc:vc + D].double()
            if op == "window_attention":
                for a in range(0, S, 2048):
                    e = min(S, a + 2048)
                    ti = torch.arange(a, e, device="cuda").view(-1, 1)
                    tj = torch.arange(0, e, device="cuda").view(1, -1)
                    s = (Q[a:e] @ K[:e].T) / math.sqrt(D)
                    hidden = (tj > ti) | ((ti - tj >= case["window"]) & (tj >= case["nsink"]))
                    s[hidden] = -math.inf
                    out[b, a:e, h * D:(h + 1) * D] = torch.softmax(s, -1) @ V[:e]
                continue
            t = pos[b]
            if t < 0:
                continue
            g = r * kvs + lk
            if op == "window_decode":
                R = case["cap"] - case["nsink"]
                old = [p for p in range(max(0, t - case["window"] + 1), t)]
                old = sorted(set(old) | set(range(min(case["nsink"], t))))
                slots = [p if p < case["nsink"] else case["nsink"] + (p - case["nsink"]) % R for p in old]
                sl = torch.tensor(slots, device="cuda", dtype=torch.long)
                Ks = torch.cat([st["k"][b, g, sl].double(), K])
                Vs = torch.cat([st["v"][b, g, sl].double(), V])
            else:
                Ks = torch.cat([st["pk"][g].double(), st["k"][b, g, :t].double(), K])
                Vs = torch.cat([st["pv"][g].double(), st["v"][b, g, :t].double(), V])
            s = (Ks @ Q[0]) / math.sqrt(D)
            out[b, 0, h * D:(h + 1) * D] = torch.softmax(s, 0) @ Vs
    out = out.view(n * S, -1)
    return out if op == "window_attention" else (out, None, None)


def _exact_kv_append(case, st):
    """Token after token in order, a newer one replacing the older one of its slot."""
    qs, kvs, nkv, _ = _geom(case)
    x = st["qkv"].view(case["nseq"], case["S"], case["tp"], qs + 2 * kvs, D)
    R = case["cap"] - case["nsink"]
    for b, (t0, c) in enumerate(zip(st["pos"].tolist(), st["count"].tolist())):
        src = {}
        for i in range(c):
            t = t0 + i
            src[t if t < case["nsink"] else case["nsink"] + (t - case["nsink"]) % R] = i
        slots, rows = torch.tensor(list(src.items()), device="cuda").T
        for j in range(kvs):
            for name, o in (("k", qs + j), ("v", qs + kvs + j)):
                st[name][b, j::kvs, slots] = x[b, rows, :, o].transpose(0, 1)
    return st["k"].double(), st["v"].double()


def _exact_sample(case, st):
    import numpy as np
    m, V = case["m"], case["V"]
    if case["H"]:
        X, W = st["X"].double(), st["W"]
        logits = torch.cat([X @ W[:, a:a + 16384].double() for a in range(0, V, 16384)], 1).cpu().numpy()
    else:
        logits = st["logits"].double().cpu().numpy()
    get = lambda name, i, none: none if st[name] is None else st[name][i].item()
    idx, logp = np.zeros(m, np.int32), np.zeros(m, np.float64)
    for i in range(m):
        l = logits[i]
        k, p, q = get("top_k", i, 0), get("top_p", i, 1.0), get("min_p", i, 0.0)
        w = np.exp((l - l.max()) / st["temperature"][i].item())
        order = np.lexsort((np.arange(V), -l))
        if k > 0:
            order = order[:k]
        if p < 1.0:
            before = np.concatenate([[0.0], np.cumsum(w[order])])
            n = int(np.searchsorted(before[:-1], p * before[-1], side="left"))   # tokens whose mass before is below p
            order = order[:max(1, n)]
        kept = np.sort(order)
        kept = kept[w[kept] >= q]
        c = np.cumsum(w[kept])
        j = min(int(np.searchsorted(c, st["u"][i].item() * c[-1], side="right")), len(kept) - 1)
        idx[i], logp[i] = kept[j], math.log(w[kept[j]] / c[-1])
    return torch.from_numpy(idx), torch.from_numpy(logp)
