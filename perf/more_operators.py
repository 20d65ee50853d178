"""Cases that measure what each request of a shared step has of its own: low-rank adapters beside the 4-bit products,
probabilities at its temperature, and the verification of its drafted tokens.

``listed()`` and ``draw()`` give cases, ``prepare`` makes what a serving loop has in hand, ``run`` is one pass: with ``own``
through the library's entry points, without it in plain torch operations.  ``exact`` restates each operator in fp64.

* lora: ``out[m] = base[m] + scale[a] * up[a] (down[a] x[m])`` with ``a = adapter[m]``; -1 leaves ``base[m]``.
* softmax: ``p[t] = softmax(logits[t] / temperature[t])``, fp32; temperature 0 is 1 at the largest logit.
* verify: sequence b has drafted tokens ``d_i``, target rows ``p_0 .. p_n`` and draft rows ``q_0 .. q_{n-1}``.  A token is
  accepted while ``u_i q_i(d_i) < p_i(d_i)``; the next one is the first j with ``sum_{k <= j} w_k > v sum w``, where
  ``w = max(p - q, 0)`` of the rejected row, or ``p_n``.  Without draft rows q is 1 at the drafted token.
"""
import math

import torch

own = False

F = {"f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token of one request, the attention projection: latency
        _lora("lora_m1", rows=1, run=1, pool=8, K=4096, N=4096, R=16),
        # a decode batch: every row another request, 48 adapters of uneven rank, some rows without one
        _lora("lora_decode_m64", rows=64, run=1, pool=48, K=4096, N=4096, R=64, uneven=True, without=0.1),
        # drafted tokens of an odd number of requests, fp32 activations, small layer
        _lora("lora_verify_m132_f32", dtype="f32", rows=132, run=4, pool=16, K=896, N=1152, R=8),
        # three prompts, each with its adapter
        _lora("lora_prompt_m2048", rows=2048, run=683, pool=8, K=4096, N=4096, R=32),
        # a chunk of a prompt and the decode tokens of 63 other requests in one call, the qkv projection
        _lora("lora_mixed_m1563", rows=1563, run=1500, tail=63, pool=64, K=4096, N=6144, R=64, uneven=True),
        # long prompts, the up projection
        _lora("lora_prompt_m8192", rows=8192, run=2500, pool=8, K=4096, N=14336, R=64),
        # probabilities of one decode step of one request: latency
        _softmax("softmax_t1", rows=1, V=128256),
        # an odd vocabulary, fp32 logits, each row its temperature, some of them 0
        _softmax("softmax_t85_f32", dtype="f32", rows=85, V=32003, temperatures=True),
        # all rows of a verify batch, 64 requests with 4 drafted tokens each
        _softmax("softmax_t320", rows=320, V=128256, temperatures=True),
        # one request: latency
        _verify("verify_b1", batch=1, drafts=4, V=128256),
        # a verify batch
        _verify("verify_b64", batch=64, drafts=4, V=128256),
        # drafts without probabilities (looked up in the prompt), ragged, odd vocabulary
        _verify("verify_b200_lookup", batch=200, drafts=8, V=32003, ragged=True, rows_of_draft=False),
    ]


def _lora(name, **kw):
    c = {"name": name, "op": "lora", "dtype": "f16", "tail": 0, "uneven": False, "without": 0.0}
    c.update(kw)
    return c


def _softmax(name, **kw):
    c = {"name": name, "op": "softmax", "dtype": "f16", "temperatures": False}
    c.update(kw)
    return c


def _verify(name, **kw):
    c = {"name": name, "op": "verify", "ragged": False, "rows_of_draft": True}
    c.update(kw)
    return c


def draw(rng):
    def logu(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    kind = rng.choice(["decode", "verify", "prompt", "mixed", "softmax", "softmax", "drafts", "drafts"])
    if kind == "softmax":
        V = logu(1000, 160000)
        c = _softmax("", dtype=rng.choice(["f16", "f16", "f32"]), V=V, rows=logu(1, min(512, 40000000 // V)),
                     temperatures=rng.random() < 0.6)
    elif kind == "drafts":
        V = logu(1000, 160000)
        n = rng.randint(1, 12)
        c = _verify("", V=V, batch=logu(1, max(1, min(256, 40000000 // (V * (n + 1))))), drafts=n, ragged=rng.random() < 0.5,
                    rows_of_draft=rng.random() < 0.75)
    else:
        dtype = rng.choice(["f16", "f16", "f16", "f32"])
        K = 16 * logu(16, 896)
        N = logu(64, 14336) if rng.random() < 0.25 else 64 * logu(1, 224)
        R = rng.choice([8, 16, 16, 32, 64, 128])
        pool = logu(1, max(1, min(128, 400000000 // (R * (K + N)))))
        c = _lora("", dtype=dtype, K=K, N=N, R=R, pool=pool, uneven=rng.random() < 0.4, without=rng.choice([0.0, 0.0, 0.2]))
        if kind == "decode":
            c.update(rows=logu(1, 256), run=1)
        elif kind == "verify":
            n = rng.randint(2, 16)
            c.update(rows=n * logu(1, 32), run=n)
        else:
            top = min(8192, 200000000 // (K + 2 * N))
            rows = logu(257, max(258, top // (2 if dtype == "f32" else 1)))
            tail = min(rows // 2, logu(1, 128)) if kind == "mixed" else 0
            c.update(rows=rows, run=max(1, (rows - tail) // rng.randint(1, 4)), tail=tail)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------
# What a serving loop has in hand
# ---------------------------------------------------------------------------------------


def _rng(device, seed, salt):
    g = torch.Generator(device=device)
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFFFFFFFFFF)
    return g


def _plan(c):
    """Host numbers of a case, the same for every seed so that its work is: who has which adapter and rank, how many tokens
    were drafted and where the first is rejected."""
    g = torch.Generator()
    g.manual_seed(29)
    if c["op"] == "lora":
        body = c["rows"] - c["tail"]
        runs = -(-body // c["run"]) + c["tail"]
        adapter = torch.randint(0, c["pool"], (runs,), generator=g)
        adapter[torch.rand(runs, generator=g) < c["without"]] = -1
        length = torch.ones(runs, dtype=torch.int64)
        n = runs - c["tail"]
        length[:n] = c["run"]
        length[n - 1] = body - (n - 1) * c["run"]
        adapter = torch.repeat_interleave(adapter, length)
        ranks = torch.full((c["pool"],), c["R"])
        if c["uneven"]:
            ranks = 8 * torch.randint(1, c["R"] // 8 + 1, (c["pool"],), generator=g)
        return adapter, ranks
    B = c["batch"]
    n = torch.full((B,), c["drafts"])
    if c["ragged"]:
        n = torch.randint(0, c["drafts"] + 1, (B,), generator=g)
        n[0] = c["drafts"]
    stop = n - (torch.rand(B, generator=g) * (n + 1)).long().clamp(max=n)  # tokens accepted
    return n, stop


def _lora_inputs(c, seed, dev):
    adapter, ranks = _plan(c)
    M, K, N, R, P = c["rows"], c["K"], c["N"], c["R"], c["pool"]
    g = _rng(dev, seed, 1)
    dt = F[c["dtype"]]
    x = torch.randn(M, K, generator=g, device=dev).to(dt)
    base = torch.randn(M, N, generator=g, device=dev).to(dt)
    down = (torch.randn(P, R, K, generator=g, device=dev) * K ** -0.5).half()
    up = (torch.randn(P, N, R, generator=g, device=dev) * 0.5 * R ** -0.5).half()
    scales = 0.5 + torch.rand(P, generator=g, device=dev)
    return x, base, down, up, scales, adapter.int().to(dev), ranks.int().to(dev)


def _logits(c, seed, dev):
    g = _rng(dev, seed, 2)
    x = (torch.randn(c["rows"], c["V"], generator=g, device=dev) * 2.5).to(F[c["dtype"]])
    t = None
    if c["temperatures"]:
        t = torch.tensor([0.7, 1.0, 0.0, 1.3], device=dev)[torch.randint(0, 4, (c["rows"],), generator=g, device=dev)]
    return x, t


def _pick(w, r):
    """Indices drawn from the rows of weights w by r in (0, 1)."""
    cum = w.double().cumsum(-1)
    return torch.searchsorted(cum, (r.double() * cum[:, -1])[:, None]).clamp(max=w.shape[1] - 1)[:, 0]


def _draft_inputs(c, seed, dev):
    """Probabilities of a target and of a draft that resembles it, and drafted tokens of which the plan's numbers are accepted:
    those from min(p, q), the first rejected one from max(q - p, 0), as in sampling that ends there."""
    n, stop = _plan(c)
    B, V, D = c["batch"], c["V"], int(n.sum())
    g = _rng(dev, seed, 3)
    start = torch.zeros(B + 1, dtype=torch.int64)
    start[1:] = n.cumsum(0)
    seq = torch.repeat_interleave(torch.arange(B), n)
    i = torch.arange(D) - start[seq]
    p = torch.empty(D + B, V, device=dev)
    q = torch.empty(D, V, device=dev)
    tokens = torch.zeros(D, dtype=torch.int64, device=dev)
    u = torch.rand(D, generator=g, device=dev) * 0.98 + 0.01
    accept = (i < stop[seq]).to(dev)
    step = max(1, (1 << 27) // V)
    row_of = torch.arange(D) + seq  # target rows of the drafted tokens
    for a in range(0, D + B, step):
        b = min(D + B, a + step)
        logits = torch.randn(b - a, V, generator=g, device=dev) * 2.5
        p[a:b] = torch.softmax(logits, -1)
        mine = ((row_of >= a) & (row_of < b)).nonzero()[:, 0]
        if len(mine) == 0:
            continue
        lo, hi = int(mine[0]), int(mine[-1]) + 1
        at = (row_of[lo:hi] - a).to(dev)
        if c["rows_of_draft"]:
            q[lo:hi] = torch.softmax(logits[at] + 0.6 * torch.randn(hi - lo, V, generator=g, device=dev), -1)
            pp, qq = p[a:b][at], q[lo:hi]
            w = torch.where(accept[lo:hi, None], torch.minimum(pp, qq), (qq - pp).clamp(min=0))
        else:
            w = p[a:b][at]
        tokens[lo:hi] = _pick(w, torch.rand(hi - lo, generator=g, device=dev))
        pt = p[a:b][at].gather(1, tokens[lo:hi, None])[:, 0]
        qt = q[lo:hi].gather(1, tokens[lo:hi, None])[:, 0] if c["rows_of_draft"] else torch.ones_like(pt)
        ratio = (pt / qt).clamp(max=1)
        u[lo:hi] = torch.where(accept[lo:hi], u[lo:hi] * ratio, ratio + u[lo:hi] * (1 - ratio))
    v = torch.rand(B, generator=g, device=dev)
    return p, q if c["rows_of_draft"] else None, tokens.int(), start.int().to(dev), u, v


def prepare(case, seed):
    dev = torch.device("cuda")
    c = dict(case)
    st = {"case": c}
    if c["op"] == "lora":
        keys = ("x", "base", "down", "up", "scales", "adapter", "ranks")
        st.update(zip(keys, _lora_inputs(c, seed, dev)))
    elif c["op"] == "softmax":
        st.update(zip(("logits", "temperature"), _logits(c, seed, dev)))
    else:
        st.update(zip(("target", "draft", "tokens", "start", "u", "v"), _draft_inputs(c, seed, dev)))
    return st


# ---------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------


def _plain_lora(st):
    c = st["case"]
    x, R, P = st["x"].float(), c["R"], c["pool"]
    adapter = st["adapter"].long()
    has = adapter >= 0
    a = adapter.clamp(min=0)
    keep = torch.arange(R, device=x.device) < st["ranks"][:, None]  # [P, R]
    factor = torch.where(has, st["scales"][a], torch.zeros_like(st["scales"][a]))
    if c["rows"] <= 2 * P:  # each row's adapter, gathered
        s = torch.matmul(st["down"][a].float(), x[:, :, None])[:, :, 0]
        s = s * keep[a] * factor[:, None]
        d = torch.matmul(st["up"][a].float(), s[:, :, None])[:, :, 0]
    else:  # every adapter for every row, masked
        s = torch.matmul(x, st["down"].float().view(P * R, -1).t()).view(-1, P, R)
        mine = torch.arange(P, device=x.device) == a[:, None]
        s = s * (mine[:, :, None] & keep) * factor[:, None, None]
        d = torch.matmul(s.view(-1, P * R), st["up"].float().permute(0, 2, 1).reshape(P * R, -1))
    return (st["base"].float() + d).to(st["x"].dtype)


def _plain_softmax(st):
    x, t = st["logits"].float(), st["temperature"]
    top = x.amax(-1, keepdim=True)
    if t is None:
        e = (x - top).exp()
        return e / e.sum(-1, keepdim=True)
    cold = t == 0
    e = ((x - top) / torch.where(cold, torch.ones_like(t), t)[:, None]).exp()
    p = e / e.sum(-1, keepdim=True)
    j = torch.arange(x.shape[1], device=x.device)
    first = torch.where(x == top, j, x.shape[1]).amin(-1, keepdim=True)
    return torch.where(cold[:, None], (j == first).float(), p)


def _plain_verify(st):
    c = st["case"]
    p, q, d, start, B, D = st["target"], st["draft"], st["tokens"].long(), st["start"].long(), c["batch"], st["tokens"].shape[0]
    dev = p.device
    at = torch.arange(D, device=dev)
    seq = torch.searchsorted(start, at, right=True) - 1
    pt = p[at + seq, d].double()
    qt = q[at, d].double() if q is not None else torch.ones_like(pt)
    bad = ~(st["u"].double() * qt < pt)
    n = start[1:] - start[:-1]
    accepted = n.clone()
    accepted.scatter_reduce_(0, seq, torch.where(bad, at - start[seq], c["drafts"] + 1), "amin")
    row = start[:-1] + torch.arange(B, device=dev) + accepted
    w = p[row].double()
    rejected = accepted < n
    if D > 0:
        r = (start[:-1] + accepted).clamp(max=D - 1)
        if q is not None:
            other = q[r].double()
        else:
            other = torch.zeros_like(w)
            other[torch.arange(B, device=dev), d[r]] = 1.0
        w = torch.where(rejected[:, None], (w - other).clamp(min=0), w)
    cum = w.cumsum(-1)
    nxt = (cum <= st["v"].double()[:, None] * cum[:, -1:]).sum(-1)
    out = torch.full((D + B,), -1, dtype=torch.int32, device=dev)
    first = start[:-1] + torch.arange(B, device=dev)
    out[at + seq] = torch.where(at - start[seq] < accepted[seq], d, -1).int()
    out[first + accepted] = nxt.int()
    return {"tokens": out, "accepted": accepted.int()}


# ---------------------------------------------------------------------------------------
# The interface
# ---------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"lora": _plain_lora, "softmax": _plain_softmax, "verify": _plain_verify}[op](state)
    import gemm_mnb_gemv_gb300 as mnb
    if op == "lora":
        pool = state.get("pool")
        if pool is None:  # the handle that a serving loop keeps
            pool = state["pool"] = mnb.MnbLoraPool(state["down"], state["up"], ranks=state["ranks"], scales=state["scales"])
        return mnb.mnb_lora(state["x"], pool, state["adapter"], base=state["base"])
    if op == "softmax":
        return mnb.mnb_softmax(state["logits"], temperature=state["temperature"])
    tokens, accepted = mnb.mnb_verify(state["target"], state["draft"], state["tokens"], state["start"], state["u"], state["v"])
    return {"tokens": tokens, "accepted": accepted}


def work(case):
    c = dict(case)
    if c["op"] == "lora":
        adapter, ranks = _plan(c)
        e = 2 if c["dtype"] == "f16" else 4
        M, K, N = c["rows"], c["K"], c["N"]
        live = adapter[adapter >= 0]
        n = e * (int(len(live)) * K + 2 * M * N) + 2 * int(ranks[live.unique()].sum()) * (K + N) + 4 * M
        return {"bytes": float(n), "flops": float(2 * int(ranks[live].sum()) * (K + N) + M * N)}
    if c["op"] == "softmax":
        e = 2 if c["dtype"] == "f16" else 4
        return {"bytes": float(c["rows"] * c["V"] * (e + 4)), "flops": float(c["rows"] * c["V"] * 4)}
    n, stop = _plan(c)
    rejected = int((stop < n).sum()) if c["rows_of_draft"] else 0
    V, B, D = c["V"], c["batch"], int(n.sum())
    return {"bytes": float(4 * V * (B + rejected) + 24 * D + 20 * B), "flops": float(V * (B + 2 * rejected))}


def exact(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    f64 = torch.float64
    if c["op"] == "lora":
        x, base, down, up, scales, _, _ = _lora_inputs(c, seed, dev)
        adapter, ranks = _plan(c)
        out = base.to(f64)
        for a in adapter[adapter >= 0].unique().tolist():
            rows = (adapter == a).nonzero()[:, 0].to(dev)
            r = int(ranks[a])
            delta = x[rows].to(f64) @ down[a, :r].to(f64).T @ up[a, :, :r].to(f64).T
            out[rows] += float(scales[a]) * delta
        return out
    if c["op"] == "softmax":
        x, t = _logits(c, seed, dev)
        out = torch.empty(x.shape, dtype=f64, device=dev)
        for i in range(c["rows"]):
            z = x[i].to(f64)
            temp = 1.0 if t is None else float(t[i])
            if temp == 0.0:
                best = int((z == z.max()).nonzero()[0, 0])
                out[i] = 0
                out[i, best] = 1
            else:
                out[i] = torch.exp(z / temp - torch.logsumexp(z / temp, 0))
        return out
    p, q, tokens, start, u, v = _draft_inputs(c, seed, dev)
    s, d = start.tolist(), tokens.tolist()
    out, count = [], []
    for b in range(c["batch"]):
        got = []
        residual = None
        for k in range(s[b], s[b + 1]):
            prow = p[k + b]
            qt = 1.0 if q is None else float(q[k, d[k]])
            if float(u[k]) * qt < float(prow[d[k]]):
                got.append(d[k])
                continue
            residual = prow.to(f64)
            if q is None:
                residual[d[k]] = 0
            else:
                residual = torch.relu(residual - q[k].to(f64))
            break
        if residual is None:
            residual = p[s[b + 1] + b].to(f64)
        cum = torch.cumsum(residual, 0)
        past = cum > float(v[b]) * cum[-1]
        count.append(len(got))
        got.append(int(past.nonzero()[0, 0]))
        out += got + [-1] * (s[b + 1] - s[b] + 1 - len(got))
    i32 = torch.int32
    return {"tokens": torch.tensor(out, dtype=i32, device=dev), "accepted": torch.tensor(count, dtype=i32, device=dev)}
