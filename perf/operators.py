"""Cases that measure the paged 4-bit key/value cache: append, read back and attention.

``listed()`` and ``draw()`` give cases, ``prepare`` makes what a serving loop has in hand,
``run`` is one pass: with ``own`` through the library's entry points, without it in plain
torch operations in fp32.  ``exact`` restates each operator in fp64 on the unpacked numbers.

A cache is ``pages`` uint8 ``[num_pages, kv_heads, record]``; a record holds ``page_size / 16``
blocks of 16 tokens.  With D = head_dim and ng = D / group, a block is

* K codes, 16 x D/2 bytes: token r's row holds 32-bit words in the order (t, w), t in 0..3, w in
  0..D/32-1; nibble n of word (t, w) is element 32 w + 8 t + n (for D = 256 the word sits at
  w ^ 4 in odd rows);
* V codes, 16 x D/2 bytes in the order (g, r', w), g in 0..7, w in 0..D/64-1; nibble 4 h + n
  (h in 0..1, n in 0..3) of word (g, r', w) is element 64 w + 32 h + 4 g + n of token
  r' ^ x(g), x(g) = 8 (g / 2 % 2) for D = 64, 8 (g % 2) for 128 and g % 2 for 256;
* K parameters, then V parameters: fp16 pairs (scale, offset) in the order (group, token).

An element's value is offset + code * scale.
"""
import math

import torch

own = False

F = {"f16": torch.float16, "f32": torch.float32}


def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "f16", "q_heads": 32, "kv_heads": 8, "head_dim": 128, "group": 128,
         "page_size": 16}
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of one sequence: latency
        _case("append_t1", "append", tokens=1, rot=128, interleaved=False, max_pos=32768),
        # one decode step of an odd batch, fp32 activations, small heads, part of a head rotated, pairs interleaved
        _case("append_t33_f32_d64", "append", dtype="f32", q_heads=14, kv_heads=2, head_dim=64, group=32, page_size=32,
              tokens=33, rot=32, interleaved=True, max_pos=8192),
        # a prefill chunk
        _case("append_t2048", "append", tokens=2048, rot=128, interleaved=False, max_pos=32768, group=64, page_size=64),
        # the prompts of a large batch at once
        _case("append_t16381", "append", tokens=16381, rot=128, interleaved=False, max_pos=32768),
        # one conversation, one token, a short odd context: latency
        _case("decode_b1_kv1000", "attention", batch=1, q_len=1, kv_min=1000, kv_max=1000, window=0),
        # one token over a very long context: the cache's bytes, split over the whole GPU
        _case("decode_b1_kv131071", "attention", batch=1, q_len=1, kv_min=131071, kv_max=131071, window=0, group=64,
              page_size=64),
        # a serving batch of ragged contexts
        _case("decode_b64_kv8192", "attention", batch=64, q_len=1, kv_min=1, kv_max=8192, window=0),
        # fp32 activations, 7 query heads a key head, heads of 64, a sliding window
        _case("decode_b16_f32_d64_window", "attention", dtype="f32", q_heads=14, kv_heads=2, head_dim=64, group=32,
              page_size=32, batch=16, q_len=1, kv_min=100, kv_max=16384, window=4096),
        # speculative verify: a few drafted tokens a sequence
        _case("verify_b16_q4_kv4096", "attention", batch=16, q_len=4, kv_min=512, kv_max=4096, window=0, group=64),
        # verify of a long draft over a long context, 16 query heads a key head
        _case("verify_b4_q16_kv32768", "attention", q_heads=32, kv_heads=2, batch=4, q_len=16, kv_min=8192, kv_max=32768,
              window=0, page_size=64),
        # a prompt from its first token, ragged
        _case("prefill_b2_t2048", "attention", batch=2, q_len=2048, kv_min=1500, kv_max=2048, window=0),
        # a chunk of a long prompt over its prefix
        _case("chunk_t2048_kv32768", "attention", batch=1, q_len=2048, kv_min=32768, kv_max=32768, window=0, page_size=64),
    ]


def draw(rng):
    def logu(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))

    kv = rng.choice([1, 2, 4, 8])
    D = rng.choice([64, 128, 128, 256])
    c = {"dtype": rng.choice(["f16", "f16", "f16", "f32"]), "q_heads": kv * rng.choice([1, 2, 4, 5, 7, 8]), "kv_heads": kv,
         "head_dim": D, "group": rng.choice([g for g in (32, 64, 128) if g <= D]), "page_size": rng.choice([16, 32, 64, 128])}
    if rng.random() < 0.35:
        rot = rng.choice([D, D, D // 2])
        c.update(op="append", tokens=logu(1, 8192), rot=rot, interleaved=rng.random() < 0.3, max_pos=32768)
        return c
    kind = rng.choice(["decode", "decode", "verify", "prefill"])
    if kind == "decode":
        b = logu(1, 64)
        top = logu(64, min(131071, 400000 // b))
        q = 1
    elif kind == "verify":
        b, q = logu(1, 16), rng.randint(2, 16)
        top = logu(256, 32768 // max(1, b // 4))
    else:
        b, q = rng.choice([1, 1, 2, 3]), logu(17, 2048)
        top = q + logu(1, 8192)
        c["q_heads"] = min(c["q_heads"], 32 // kv * kv)
    lo = max(1, top // rng.choice([1, 2, 8]))
    window = rng.choice([0, 0, 0, logu(16, 4096)])
    c.update(op="attention", batch=b, q_len=q, kv_min=lo, kv_max=top, window=window)
    return c


def _rng(device, seed, salt):
    g = torch.Generator(device=device)
    g.manual_seed((seed * 1000003 + salt) & 0x7FFFFFFFFFFFFFFF)
    return g


# ---------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------


def _quantise(x, group):
    """codes (uint8, shape of x), scale and offset (fp16, ``[..., D / group]``) of fp32 x."""
    v = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    lo, hi = v.amin(-1), v.amax(-1)
    offset = lo.clamp(-65504.0, 65504.0).half()
    scale = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).clamp(max=65504.0).half()
    s = scale.float()
    inv = torch.where(s == 0, torch.zeros_like(s), torch.ones_like(s) / s)
    code = torch.round((v - offset.float()[..., None]) * inv[..., None]).clamp(0, 15).to(torch.uint8)
    return code.reshape(x.shape), scale, offset


def _swizzle(D, device):
    """``[8, 16]``: the place in a V block of token r for dim chunk g."""
    g, r = torch.arange(8, device=device)[:, None], torch.arange(16, device=device)[None, :]
    return r ^ {64: (g // 2 % 2) * 8, 128: (g % 2) * 8, 256: g % 2}[D]


def _k_bytes(codes):
    """K rows of bytes ``[N, D/2]`` of codes ``[N, D]`` (token r % 16 == n % 16 of its block given by order)."""
    N, D = codes.shape
    b = codes.view(N, D // 2, 2)
    b = b[..., 0] | (b[..., 1] << 4)
    return b.view(N, D // 32, 4, 4).permute(0, 2, 1, 3).reshape(N, 4, D // 32, 4)


def _pack_k(codes):
    """codes ``[X, 16, D]`` -> bytes ``[X, 8 D]``."""
    X, _, D = codes.shape
    b = _k_bytes(codes.reshape(X * 16, D)).view(X, 16, 4, D // 32, 4)
    if D == 256:
        b = torch.stack([b[:, 0::2], b[:, 1::2].roll(4, dims=3)], dim=2).reshape(X, 16, 4, D // 32, 4)
    return b.reshape(X, 8 * D)


def _pack_v(codes):
    """codes ``[X, 16, D]`` -> bytes ``[X, 8 D]``."""
    X, _, D = codes.shape
    b = codes.view(X, 16, D // 2, 2)
    b = (b[..., 0] | (b[..., 1] << 4)).view(X, 16, D // 64, 2, 8, 2).permute(0, 4, 1, 2, 3, 5).reshape(X, 8, 16, D // 16)
    place = _swizzle(D, codes.device)  # its own inverse
    return b[:, torch.arange(8, device=codes.device)[:, None], place].reshape(X, 8 * D)


def _pack(k, v, kp, vp):
    """Block bytes ``[X, block]`` of codes ``[X, 16, D]`` and parameters fp16 ``[X, 16, ng, 2]``."""
    X = k.shape[0]
    kp, vp = (p.permute(0, 2, 1, 3).contiguous().view(torch.uint8).reshape(X, -1) for p in (kp, vp))
    return torch.cat([_pack_k(k), _pack_v(v), kp, vp], dim=1)


def _unpack(blocks, D, group):
    """fp32 values K, V ``[X, 16, D]`` of block bytes ``[X, block]``."""
    X, ng = blocks.shape[0], D // group
    kb, vb = blocks[:, : 8 * D], blocks[:, 8 * D: 16 * D]
    par = blocks[:, 16 * D:].contiguous().view(torch.float16).view(X, 2, ng, 16, 2).permute(1, 0, 3, 2, 4).float()

    def nibbles(b):
        return torch.stack([b & 15, b >> 4], dim=-1)

    kb = kb.reshape(X, 16, 4, D // 32, 4)
    if D == 256:
        kb = torch.stack([kb[:, 0::2], kb[:, 1::2].roll(4, dims=3)], dim=2).reshape(X, 16, 4, D // 32, 4)
    k = nibbles(kb.permute(0, 1, 3, 2, 4)).reshape(X, 16, D)
    place = _swizzle(D, blocks.device)
    vb = vb.reshape(X, 8, 16, D // 16)[:, torch.arange(8, device=blocks.device)[:, None], place]
    v = nibbles(vb.view(X, 8, 16, D // 64, 2, 2).permute(0, 2, 3, 4, 1, 5)).reshape(X, 16, D)
    out = []
    for c, p in ((k, par[0]), (v, par[1])):
        c = c.view(X, 16, ng, group).float() * p[..., :1] + p[..., 1:]
        out.append(c.reshape(X, 16, D))
    return out


def _rotate(x, cos, sin, rot, interleaved):
    """fp32 rotation of the first ``rot`` dims of x ``[T, H, D]``; cos, sin ``[T, rot / 2]``."""
    c, s = cos[:, None, :], sin[:, None, :]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    p, q = a * c - b * s, b * c + a * s
    r = torch.stack([p, q], dim=-1).reshape(r.shape) if interleaved else torch.cat([p, q], dim=-1)
    return torch.cat([r, x[..., rot:]], dim=-1)


def _plain_append(st):
    c = st["case"]
    D, group, ps, Hk = c["head_dim"], c["group"], c["page_size"], c["kv_heads"]
    pos = st["positions"].long()
    cos, sin = st["cos"][pos], st["sin"][pos]
    q = _rotate(st["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(st["q"].dtype)
    kc, ks, ko = _quantise(_rotate(st["k"].float(), cos, sin, c["rot"], c["interleaved"]), group)
    vc, vs, vo = _quantise(st["v"].float(), group)
    T, ng, bb = kc.shape[0], D // group, 16 * D + 128 * (D // group)
    pages = st["pages"].view(st["pages"].shape[0], Hk, ps // 16, bb)
    slot = st["slots"]
    page, blk, r = slot // ps, slot % ps // 16, slot % 16
    # the bytes of one token inside its block
    one = torch.zeros(T * Hk, 16, D, dtype=torch.uint8, device=kc.device)
    ar = torch.arange(T, device=kc.device)
    rows = r[:, None].expand(T, Hk).reshape(-1)
    one[torch.arange(T * Hk, device=kc.device), rows] = kc.view(T * Hk, D)
    kb = _pack_k(one).view(T * Hk, 16, D // 2)[torch.arange(T * Hk, device=kc.device), rows].view(T, Hk, D // 2)
    place = _swizzle(D, kc.device)[:, r].t()  # [T, 8]
    b = vc.view(T, Hk, D // 2, 2)
    vb = (b[..., 0] | (b[..., 1] << 4)).view(T, Hk, D // 64, 2, 8, 2).permute(0, 1, 4, 2, 3, 5).reshape(T, Hk, 8, D // 16)
    h = torch.arange(Hk, device=kc.device)[None, :]
    view_k = pages[..., : 8 * D].view(*pages.shape[:3], 16, D // 2)
    view_k[page[:, None], h, blk[:, None], r[:, None]] = kb
    view_v = pages[..., 8 * D: 16 * D].view(*pages.shape[:3], 8, 16, D // 16)
    g = torch.arange(8, device=kc.device)[None, None, :]
    view_v[page[:, None, None], h[..., None], blk[:, None, None], g, place[:, None, :]] = vb
    par = torch.stack([torch.stack([ks, ko], -1), torch.stack([vs, vo], -1)], dim=2)  # [T, Hk, 2, ng, 2] fp16
    view_p = pages[..., 16 * D:].view(*pages.shape[:3], 2, ng, 16, 4)
    view_p[page[:, None], h, blk[:, None], :, :, r[:, None]] = par.view(torch.uint8).reshape(T, Hk, 2, ng, 4)
    # read back
    kf, vf = _unpack(pages[page[:, None], h, blk[:, None]].reshape(T * Hk, bb), D, group)
    sel = torch.arange(T * Hk, device=kc.device)
    kf, vf = (x[sel, rows].view(T, Hk, D).to(st["q"].dtype) for x in (kf, vf))
    return {"q": q, "k": kf, "v": vf}


def _plain_attention(st):
    c = st["case"]
    D, group, ps, Hk, B = c["head_dim"], c["group"], c["page_size"], c["kv_heads"], c["batch"]
    G = c["q_heads"] // Hk
    table, kv_len, q_start = st["page_table"].long(), st["kv_len"].long(), st["q_start"].long()
    S = table.shape[1] * ps
    bb = 16 * D + 128 * (D // group)
    blocks = st["pages"][table].view(B, -1, Hk, ps // 16, bb).permute(0, 2, 1, 3, 4).reshape(-1, bb)
    k, v = (x.view(B, Hk, S, D) for x in _unpack(blocks, D, group))
    q_len = q_start[1:] - q_start[:-1]
    mq = c["q_len"]
    i = torch.arange(mq, device=table.device)
    idx = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[idx].view(B, mq, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, mq * G, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"]).view(B, Hk, mq, G, S)
    j = torch.arange(S, device=table.device)
    pos = (kv_len - q_len)[:, None] + i
    keep = (j[None, None] <= pos[..., None]) & (j[None, None] < kv_len[:, None, None])
    if c["window"]:
        keep &= j[None, None] > pos[..., None] - c["window"]
    s.masked_fill_(~keep[:, None, :, None, :], float("-inf"))
    top = s.amax(-1, keepdim=True)
    s.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hk, mq * G, S), v).view(B, Hk, mq, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.permute(0, 2, 1, 3, 4).reshape(B, mq, Hk * G, D)
    return o[i[None, :] < q_len[:, None]].to(st["q"].dtype)


# ---------------------------------------------------------------------------------------
# The interface
# ---------------------------------------------------------------------------------------


def _geometry(c, seed):
    """Host numbers of a case: sequence lengths (the same for every seed, so that its work is), slots, pages."""
    g, lengths = torch.Generator(), torch.Generator()
    g.manual_seed(seed * 7919 + 17)
    lengths.manual_seed(17)
    ps = c["page_size"]
    if c["op"] == "append":
        T = c["tokens"]
        pages = -(-T // ps) + 3
        slots = torch.randperm(pages * ps, generator=g)[:T] if T < 64 else None
        if slots is None:  # whole prompts: runs of consecutive slots, pages in any order
            order = torch.randperm(pages, generator=g)
            slots = (order[:, None] * ps + torch.arange(ps)).reshape(-1)[5: 5 + T]
        positions = torch.randint(0, c["max_pos"], (T,), generator=g)
        return {"pages": pages, "slots": slots, "positions": positions}
    B, q = c["batch"], c["q_len"]
    kv = torch.randint(c["kv_min"], c["kv_max"] + 1, (B,), generator=lengths)
    kv[-1] = c["kv_max"]
    ql = torch.full((B,), q)
    if q > 1:  # ragged: every second sequence brings fewer tokens
        ql[1::2] = torch.randint(1, q + 1, (B // 2,), generator=lengths)
    ql = torch.minimum(ql, kv)
    npages = -(-kv.max().item() // ps)
    need = -(-kv // ps)
    total = int(need.sum()) + 2
    order = torch.randperm(total, generator=g)
    table = torch.zeros(B, npages, dtype=torch.int64)
    at = 0
    for b in range(B):
        table[b, : need[b]] = order[at: at + need[b]]
        at += int(need[b])
    start = torch.zeros(B + 1, dtype=torch.int64)
    start[1:] = ql.cumsum(0)
    return {"pages": total, "kv": kv, "ql": ql, "table": table, "start": start}


def _qkv(c, seed, device):
    """Rows of the fused qkv product: q, k, v as strided views of one ``[T, (Hq + 2 Hk) D]``."""
    T, Hq, Hk, D = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
    x = torch.randn(T, (Hq + 2 * Hk) * D, generator=_rng(device, seed, 1), device=device).to(F[c["dtype"]])
    a, b = Hq * D, (Hq + Hk) * D
    return x[:, :a].view(T, Hq, D), x[:, a:b].view(T, Hk, D), x[:, b:].view(T, Hk, D)


def _tables(c, device):
    half = c["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    ang = torch.arange(c["max_pos"], dtype=torch.float64)[:, None] * inv
    return ang.cos().float().to(device), ang.sin().float().to(device)


def _cache_numbers(c, seed, pages, device):
    """Codes and parameters of every token of a filled cache, in plain order: two of
    (codes ``[tokens, Hk, D]``, scale, offset ``[tokens, Hk, ng]``).  Keys have channels of uneven size."""
    N, Hk, D = pages * c["page_size"], c["kv_heads"], c["head_dim"]
    g = _rng(device, seed, 2)
    channel = torch.exp(0.4 * torch.randn(Hk, D, generator=g, device=device))
    out = []
    for mult in (channel, None):
        codes = torch.empty(N, Hk, D, dtype=torch.uint8, device=device)
        scale = torch.empty(N, Hk, D // c["group"], dtype=torch.float16, device=device)
        offset = torch.empty_like(scale)
        step = max(16, (1 << 28) // (Hk * D))
        for a in range(0, N, step):
            x = torch.randn(min(step, N - a), Hk, D, generator=g, device=device)
            x = x if mult is None else x * mult
            codes[a: a + step], scale[a: a + step], offset[a: a + step] = _quantise(x, c["group"])
        out.append((codes, scale, offset))
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    c = dict(case)
    D, Hk, ps, ng = c["head_dim"], c["kv_heads"], c["page_size"], c["head_dim"] // c["group"]
    geo = _geometry(c, seed)
    st = {"case": c, "scale": 1.0 / math.sqrt(D)}
    bb = 16 * D + 128 * ng
    if c["op"] == "append":
        q, k, v = _qkv(c, seed, dev)
        cos, sin = _tables(c, dev)
        st.update(q=q, k=k, v=v, cos=cos, sin=sin, slots=geo["slots"].to(dev), positions=geo["positions"].int().to(dev),
                  pages=torch.zeros(geo["pages"], Hk, ps // 16 * bb, dtype=torch.uint8, device=dev))
        return st
    pages = torch.empty(geo["pages"], Hk, ps // 16 * bb, dtype=torch.uint8, device=dev)
    (kc, ks, ko), (vc, vs, vo) = _cache_numbers(c, seed, geo["pages"], dev)

    def blocks(x, a, b):  # [tokens, Hk, ...] -> [pages * Hk * blocks, 16, ...]
        x = x[a * ps: b * ps]
        return x.view(b - a, ps // 16, 16, Hk, x.shape[-1]).permute(0, 3, 1, 2, 4).reshape(-1, 16, x.shape[-1])

    step = max(1, (1 << 27) // (ps * Hk * D))
    for a in range(0, geo["pages"], step):
        b = min(geo["pages"], a + step)
        kp = torch.stack([blocks(ks, a, b), blocks(ko, a, b)], dim=-1)
        vp = torch.stack([blocks(vs, a, b), blocks(vo, a, b)], dim=-1)
        pages[a:b] = _pack(blocks(kc, a, b), blocks(vc, a, b), kp, vp).view(b - a, Hk, -1)
    T = int(geo["start"][-1])
    q = torch.randn(T, c["q_heads"], D, generator=_rng(dev, seed, 3), device=dev).to(F[c["dtype"]])
    st.update(q=q, pages=pages, page_table=geo["table"].int().to(dev), kv_len=geo["kv"].int().to(dev),
              q_start=geo["start"].int().to(dev))
    return st


def run(state):
    c = state["case"]
    if not own:
        return _plain_append(state) if c["op"] == "append" else _plain_attention(state)
    import gemm_mnb_gemv_gb300 as mnb
    cache = state.get("cache")
    if cache is None:  # the handle that a serving loop keeps
        cache = state["cache"] = mnb.MnbKv4Cache(state["pages"], c["page_size"], c["head_dim"], c["group"])
    if c["op"] == "append":
        q = mnb.mnb_kv4_append(cache, state["k"], state["v"], state["slots"], q=state["q"], positions=state["positions"],
                               cos=state["cos"], sin=state["sin"], interleaved=c["interleaved"])
        k, v = mnb.mnb_kv4_read(cache, state["slots"], dtype=state["q"].dtype)
        return {"q": q, "k": k, "v": v}
    return mnb.mnb_kv4_attention(state["q"], cache, state["q_start"], state["kv_len"], state["page_table"],
                                 scale=state["scale"], causal=True, window=c["window"])


def _pairs(c, geo):
    """(query, key) pairs that the masks leave, and the keys that some query of each sequence sees."""
    pairs, keys = 0, 0
    w = c["window"] or (1 << 40)
    for n, q in zip(geo["kv"].tolist(), geo["ql"].tolist()):
        pos = torch.arange(n - q, n, dtype=torch.int64)
        pairs += int(torch.minimum(pos + 1, torch.tensor(w)).sum())
        keys += min(n, q - 1 + w)
    return pairs, keys


def work(case):
    c = dict(case)
    e = 2 if c["dtype"] == "f16" else 4
    Hq, Hk, D = c["q_heads"], c["kv_heads"], c["head_dim"]
    token = Hk * (D + 8 * (D // c["group"]))  # bytes of one token's codes and parameters, K and V
    if c["op"] == "append":
        T = c["tokens"]
        n = e * T * (Hq + 2 * Hk) * D + e * T * Hq * D + T * token + T * (12 + 4 * c["rot"])  # append
        n += T * token + 2 * e * T * Hk * D + 8 * T                                             # read back
        return {"bytes": float(n), "flops": float(T * (3 * (Hq + Hk) * c["rot"] + 14 * Hk * D))}
    geo = _geometry(c, 1)
    pairs, keys = _pairs(c, geo)
    T = int(geo["ql"].sum())
    return {"bytes": float(keys * token + 2 * e * T * Hq * D + 4 * int((-(-geo["kv"] // c["page_size"])).sum())),
            "flops": float(4 * D * Hq * pairs)}


def exact(case, seed):
    c = dict(case)
    D, group, ps, Hk, Hq = c["head_dim"], c["group"], c["page_size"], c["kv_heads"], c["q_heads"]
    dev = torch.device("cuda")
    geo = _geometry(c, seed)
    f64 = torch.float64
    if c["op"] == "append":
        q, k, v = (x.to(f64) for x in _qkv(c, seed, dev))
        cos, sin = (t.to(f64)[geo["positions"].to(dev)][:, None, :, None] for t in _tables(c, dev))
        rot = c["rot"]

        def turn(x):  # each pair as a complex number, times cos + i sin
            y, n = x.clone(), x.shape[0]
            r = x[..., :rot].reshape(n, -1, rot // 2, 2) if c["interleaved"] else x[..., :rot].reshape(n, -1, 2, rot // 2).transpose(2, 3)
            m = torch.cat([cos, -sin, sin, cos], dim=-1).view(n, 1, rot // 2, 2, 2)
            r = (m @ r[..., None])[..., 0]
            y[..., :rot] = r.reshape(n, -1, rot) if c["interleaved"] else r.transpose(2, 3).reshape(n, -1, rot)
            return y

        def held(x):  # what 4 bits with this group's fp16 scale and offset stand for
            x = x.reshape(x.shape[0], Hk, D // group, group)
            lo, _ = x.min(-1, keepdim=True)
            hi, _ = x.max(-1, keepdim=True)
            off, step = lo.half().to(f64), ((hi - lo) / 15).half().to(f64)
            code = torch.where(step > 0, ((x - off) / step).round(), torch.zeros_like(x)).clamp(0, 15)
            return (off + code * step).reshape(x.shape[0], Hk, D)

        return {"q": turn(q), "k": held(turn(k)), "v": held(v)}
    T = int(geo["start"][-1])
    q = torch.randn(T, Hq, D, generator=_rng(dev, seed, 3), device=dev).to(F[c["dtype"]]).to(f64)
    numbers = _cache_numbers(c, seed, geo["pages"], dev)
    out = torch.zeros(T, Hq, D, dtype=f64, device=dev)
    G = Hq // Hk
    for b in range(c["batch"]):
        n, a, e = int(geo["kv"][b]), int(geo["start"][b]), int(geo["start"][b + 1])
        j = torch.arange(n)
        slot = (geo["table"][b][j // ps] * ps + j % ps).to(dev)
        key = j.to(dev)
        pos = torch.arange(n - (e - a), n, device=dev)
        hidden = key[None] > pos[:, None]
        if c["window"]:
            hidden |= key[None] <= pos[:, None] - c["window"]
        for h in range(Hk):
            K, V = (s[slot, h].to(f64).repeat_interleave(group, -1) * x[slot, h].to(f64)
                    + o[slot, h].to(f64).repeat_interleave(group, -1) for x, s, o in numbers)
            for g in range(G):
                s = (q[a:e, h * G + g] @ K.T) / math.sqrt(D)
                out[a:e, h * G + g] = torch.softmax(s.masked_fill(hidden, float("-inf")), -1) @ V
    return out
