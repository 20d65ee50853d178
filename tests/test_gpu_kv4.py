"""Paged 4-bit key/value cache on the GPU: append and read bit for bit, attention against fp64.

Tolerances of the attention, from the roundings that its arithmetic may make (u = 2^-11 for fp16 activations,
2^-20 for fp32, where operands are split into two fp16 parts and exponentials are approximate):
* a key or a probability rounded once to u relative, a value too, and the result: 4 u (|out| + sum_j p_j |v_j|);
* a score off by ds <= u * scale * sum_d |q_d k_d| moves every probability by a factor e^(2 ds).
As a norm, independent roundings add up as squares: at most 2 u of the result (fp16), 4 u (fp32). Results below
2^-14 are fp16 subnormals: their last rounding is up to 2^-25 whatever their size.
"""
from __future__ import annotations

from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

from oracle import kv4_oracle_np as orc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import gemm_mnb_gemv_gb300 as mnb
    return mnb, torch, torch.device("cuda:0")


NP = {"f16": np.float16, "f32": np.float32}


def _tables(rng, rows, rot):
    ang = rng.uniform(-3.2, 3.2, (rows, rot // 2))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


@pytest.mark.parametrize("D,group,ps,Hq,Hk,T,dtype,rot,interleaved", [
    (64, 32, 16, 3, 1, 1, "f16", 64, False),
    (64, 64, 32, 14, 2, 5, "f32", 32, True),
    (128, 32, 48, 8, 8, 33, "f16", 128, False),
    (128, 64, 16, 32, 8, 70, "f16", 16, True),
    (128, 128, 64, 5, 1, 129, "f32", 96, False),
    (128, 128, 16, 0, 2, 3, "f16", 0, False),
    (256, 32, 16, 7, 1, 2, "f16", 256, True),
    (256, 64, 32, 2, 2, 65, "f32", 256, False),
    (256, 128, 128, 16, 2, 7, "f16", 128, False),
])
def test_append_and_read_are_bit_exact(env, D, group, ps, Hq, Hk, T, dtype, rot, interleaved):
    mnb, torch, dev = env
    rng = np.random.default_rng(D + T)
    x = (rng.standard_normal((T, (Hq + 2 * Hk) * D)) * rng.choice([0.01, 1, 50], (T, 1))).astype(NP[dtype])
    k0, v0 = x[:, Hq * D:(Hq + Hk) * D].reshape(T, Hk, D), x[:, (Hq + Hk) * D:].reshape(T, Hk, D)
    k0[0, 0, :group], v0[0, 0, :group] = 0.25, 0.0      # constant groups: scale 0
    if T > 2:
        v0[2, 0, group - 1], k0[1, -1, 3] = np.inf, np.nan
    pages = -(-T // ps) + 2
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    if T > 4:
        slots[3] = -1
    pos = rng.integers(0, 40, T).astype(np.int32)
    cos, sin = _tables(rng, 40, rot) if rot else (None, None)
    xd = torch.from_numpy(x).to(dev)
    q, k, v = (t.view(T, -1, D) for t in (xd[:, :Hq * D], xd[:, Hq * D:(Hq + Hk) * D], xd[:, (Hq + Hk) * D:]))
    start = rng.integers(0, 256, (pages, Hk, ps // 16 * orc.block_bytes(D, group))).astype(np.uint8)
    cache = mnb.MnbKv4Cache(torch.from_numpy(start).to(dev), ps, D, group)
    up = lambda a: None if a is None else torch.from_numpy(a).to(dev)  # noqa: E731
    got_q = mnb.mnb_kv4_append(cache, k, v, up(slots), q=q if Hq else None, positions=up(pos), cos=up(cos), sin=up(sin),
                               interleaved=interleaved)
    f = np.float32
    want = orc.append(start, k0.astype(f), v0.astype(f), pos, cos, sin, interleaved, slots, ps, group)
    got = cache.pages.cpu().numpy().reshape(-1)
    # parameters that are NaN may differ in their bits; everything else is compared as bytes
    diff = got != want
    if diff.any():
        a, b = got.view("<f2"), want.view("<f2")
        both = np.repeat(np.isnan(a) & np.isnan(b), 2)
        assert not (diff & ~both).any()
        blk = orc.block_bytes(D, group)
        assert (np.nonzero(diff)[0] % blk >= 16 * D).all()
    if Hq:
        with np.errstate(over="ignore"):
            want_q = orc.rotate(x[:, :Hq * D].reshape(T, Hq, D), pos, cos, sin, interleaved).astype(NP[dtype])
        np.testing.assert_array_equal(got_q.cpu().numpy(), want_q)
    rk, rv = mnb.mnb_kv4_read(cache, up(slots), dtype=k.dtype)
    with np.errstate(over="ignore", invalid="ignore"):
        wk, wv = (a.astype(NP[dtype]) for a in orc.read(want, slots, ps, Hk, D, group))
    np.testing.assert_array_equal(rk.cpu().numpy(), wk)
    np.testing.assert_array_equal(rv.cpu().numpy(), wv)
    if T > 2:
        assert np.isnan(rv[2, 0, :group].float().cpu().numpy()).all() and np.isnan(wk[1, -1]).any()
    mnb.mnb_check_device_status()


def test_append_in_place_extremes_and_bad_indices(env):
    mnb, torch, dev = env
    D, T, Hk = 128, 6, 1
    rng = np.random.default_rng(9)
    q = torch.from_numpy(rng.standard_normal((T, 2, D)).astype(np.float16)).to(dev)
    k = torch.from_numpy((rng.standard_normal((T, Hk, D)) * 1e30).astype(np.float32)).to(dev)
    cos, sin = (torch.from_numpy(t).to(dev) for t in _tables(rng, 8, D))
    cache = mnb.mnb_kv4_cache_alloc(2, 16, Hk, D, 64, dev)
    # fp32 values beyond the fp16 range saturate
    mnb.mnb_kv4_append(cache, k, k, torch.arange(T, device=dev))
    rk, _ = mnb.mnb_kv4_read(cache, torch.arange(T, device=dev), dtype=torch.float32)
    assert torch.isfinite(rk).all() and float(rk.abs().max()) <= 65504 * 16
    # q_out = q, a position and a slot out of range
    kv = torch.ones((T, Hk, D), dtype=torch.float16, device=dev)
    pos = torch.tensor([0, 1, 8, 3, -1, 7], dtype=torch.int32, device=dev)
    slots = torch.tensor([16, 17, 18, 32, 20, 21], device=dev)
    want = orc.rotate(q.cpu().numpy(), np.clip(pos.cpu().numpy(), 0, 7), cos.cpu().numpy(), sin.cpu().numpy(), False)
    want[[2, 4]] = 0
    before = cache.pages.clone()
    got = mnb.mnb_kv4_append(cache, kv, kv, slots, q=q, positions=pos, cos=cos, sin=sin, q_out=q)
    assert got is q
    np.testing.assert_array_equal(q.cpu().numpy(), want.astype(np.float16))
    with pytest.raises(mnb.MnbError) as e:
        mnb.mnb_check_device_status()
    assert e.value.status == mnb.MNB_ERR_INVALID_ARG
    _, rv = mnb.mnb_kv4_read(cache, torch.tensor([16, 17, 18, 20, 21, -1], device=dev))
    np.testing.assert_array_equal(rv[:, 0, 0].cpu().numpy(), [1, 1, 0, 0, 1, 0])
    assert torch.equal(before[0], cache.pages[0])
    _, rv = mnb.mnb_kv4_read(cache, torch.tensor([32, 1 << 40], device=dev))
    assert not rv.any()
    with pytest.raises(mnb.MnbError):
        mnb.mnb_check_device_status()
    mnb.mnb_check_device_status()


def _cache(env, rng, D, group, ps, Hk, pages, kscale=1.0, vscale=1.0):
    """A cache of random codes and parameters (bytes of quantised normal numbers, packed by the oracle's maps)."""
    mnb, torch, dev = env
    ng, bb = D // group, orc.block_bytes(D, group)
    n = pages * Hk * (ps // 16)
    blocks = np.zeros((n, bb), np.uint8)
    for is_v, (place, mult) in enumerate(((orc.k_place, kscale), (orc.v_place, vscale))):
        x = (rng.standard_normal((n, 16, D)) * mult).astype(np.float32)
        code, scale, offset = orc.quantise(x, group)
        m = np.array([[place(D, r, d) for d in range(D)] for r in range(16)]).reshape(-1, 2)
        c = code.reshape(n, -1).astype(np.uint8)
        for bit in (0, 4):
            at = m[:, 1] == bit
            blocks[:, m[at, 0]] |= c[:, at] << bit
        par = np.stack([scale, offset], -1).transpose(0, 2, 1, 3)  # [n, ng, 16, 2]
        at = 16 * D + is_v * ng * 64
        blocks[:, at: at + ng * 64] = np.ascontiguousarray(par).view(np.uint8).reshape(n, -1)
    host = blocks.reshape(pages, Hk, -1)
    return host, mnb.MnbKv4Cache(torch.from_numpy(host).to(dev), ps, D, group)


def _check(out, lse, want, dtype, what=""):
    ref, ref_lse, mag, reach = want
    got = out.double().cpu().numpy()
    u = 2.0 ** -11 if dtype == "f16" else 2.0 ** -20
    ds = u * reach[..., None]
    tol = 4 * u * (np.abs(ref) + mag) + np.expm1(2 * ds) * mag + 1e-30
    if dtype == "f16":
        tol = tol + 2.0 ** -24  # subnormal results
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.3g} of the tolerance"
    norm = np.linalg.norm(ref)
    if norm and (reach.max() < 40):
        bound = 2 * u * norm + 2.0 ** -25 * np.sqrt(ref.size) if dtype == "f16" else 4 * u * norm
        assert np.linalg.norm(got - ref) <= bound, (what, np.linalg.norm(got - ref) / norm)
    if lse is not None:
        l = lse.double().cpu().numpy()
        none = np.isinf(ref_lse)
        np.testing.assert_array_equal(none, np.isinf(l))
        assert (l[none] < 0).all()
        tol = u * reach[~none] + 2.0 ** -19 * (1 + np.abs(ref_lse[~none]))
        assert (np.abs(l - ref_lse)[~none] <= tol).all(), what


def _run(env, rng, D, group, ps, Hk, G, lens, dtype, causal=True, window=0, scale=None, poison=False, kscale=1.0,
         vscale=1.0, q=None):
    """lens: (query tokens, keys) of each sequence."""
    mnb, torch, dev = env
    need = [-(-n // ps) for _, n in lens]
    pages = sum(need) + 3
    host, cache = _cache(env, rng, D, group, ps, Hk, pages, kscale, vscale)
    order = rng.permutation(pages)
    width = max(max(need), 1) + 1
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
    if poison:  # whatever lies beyond the keys: NaN parameters, page indices that are not looked at
        used = np.zeros((pages, ps), bool)
        for b, (_, n) in enumerate(lens):
            j = np.arange(n)
            used[table[b, j // ps], j % ps] = True
            table[b, need[b]:] = 2 ** 31 - 1
        bb, ng = orc.block_bytes(D, group), D // group
        par = host.reshape(pages, Hk, ps // 16, bb)[..., 16 * D:].reshape(pages, Hk, ps // 16, 2 * ng, 16, 4).copy()
        mask = ~used.reshape(pages, 1, ps // 16, 1, 16)
        par[np.broadcast_to(mask, par.shape[:-1])] = 0xff
        host.reshape(pages, Hk, ps // 16, bb)[..., 16 * D:] = par.reshape(pages, Hk, ps // 16, -1)
        cache = mnb.MnbKv4Cache(torch.from_numpy(host).to(dev), ps, D, group)
    start = np.concatenate([[0], np.cumsum([a for a, _ in lens])]).astype(np.int32)
    kv = np.array([n for _, n in lens], np.int32)
    T = int(start[-1])
    if q is None:
        q = rng.standard_normal((T, Hk * G, D)).astype(NP[dtype])
    scale = scale or 1 / np.sqrt(D)
    scale = float(np.float32(scale))
    qd = torch.from_numpy(q).to(dev)
    up = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    lse = torch.full((T, Hk * G), 7.0, device=dev)
    out = mnb.mnb_kv4_attention(qd, cache, up(start), up(kv), up(table), scale, causal=causal, window=window, lse=lse)
    want = orc.attention(q, host, start, kv, table, ps, Hk, group, scale, causal, window)
    _check(out, lse, want, dtype, mnb.mnb_last_variant())
    again = mnb.mnb_kv4_attention(qd, cache, up(start), up(kv), up(table), scale, causal=causal, window=window)
    assert torch.equal(out, again)
    mnb.mnb_check_device_status()
    return mnb.mnb_last_variant()


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 64), (1, 0), (1, 130), (1, 1031)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D,group,ps,Hk,G", [
    (64, 32, 16, 2, 7), (64, 64, 64, 1, 1), (128, 32, 32, 1, 8), (128, 64, 16, 2, 4), (128, 128, 48, 3, 5),
    (256, 32, 16, 1, 2), (256, 128, 64, 2, 8), (128, 128, 16, 1, 16), (64, 32, 128, 1, 20), (256, 64, 32, 1, 12)])
def test_decode(env, D, group, ps, Hk, G, dtype):
    _run(env, np.random.default_rng(D + G), D, group, ps, Hk, G, DECODE, dtype, poison=True)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D,group,ps,Hk,G,window,causal", [
    (128, 128, 16, 2, 4, 0, True), (128, 64, 64, 1, 8, 33, True), (64, 32, 16, 1, 3, 0, False), (256, 64, 32, 1, 4, 0, True),
    (128, 32, 16, 1, 1, 1, True), (64, 64, 32, 2, 16, 100, True), (128, 128, 16, 1, 5, 20, False)])
def test_a_few_tokens_a_sequence(env, D, group, ps, Hk, G, window, causal, dtype):
    """Verify: ragged, a sequence without tokens, more tokens than keys (rows that see nothing)."""
    lens = [(4, 100), (1, 333), (0, 50), (16, 16), (5, 3), (7, 0), (2, 129), (3, 700)]
    _run(env, np.random.default_rng(G), D, group, ps, Hk, G, lens, dtype, causal=causal, window=window, poison=True)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D,group,ps,Hk,G,window,causal,lens", [
    (128, 128, 16, 1, 4, 0, True, [(130, 130), (1, 77), (257, 300)]),
    (64, 32, 64, 2, 2, 0, True, [(65, 400), (0, 0), (200, 200)]),
    (128, 64, 16, 1, 3, 50, True, [(150, 150), (100, 391), (40, 30)]),
    (128, 32, 32, 1, 2, 0, False, [(90, 140), (129, 128)]),
    (256, 128, 16, 1, 2, 0, True, [(70, 140), (33, 33)]),
    (64, 64, 16, 1, 1, 7, True, [(300, 301)]),
])
def test_chunks(env, D, group, ps, Hk, G, window, causal, lens, dtype):
    _run(env, np.random.default_rng(D), D, group, ps, Hk, G, lens, dtype, causal=causal, window=window, poison=True)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 500)], [(3, 300), (2, 90)], [(140, 260)]])
def test_value_sizes(env, lens, dtype):
    """Tiny and huge keys and values, a row of zeros, scores far apart (one key takes all), scale 0 of q."""
    rng = np.random.default_rng(3)
    T = sum(a for a, _ in lens)
    for kscale, vscale, qscale in [(1, 1e-4, 1), (1, 3000, 1), (8, 1, 8), (1e-3, 1, 100), (1, 1, 0)]:
        q = (rng.standard_normal((T, 4, 128)) * qscale).astype(NP[dtype])
        _run(env, rng, 128, 64, 16, 1, 4, lens, dtype, kscale=kscale, vscale=vscale, q=q)
    if dtype == "f32":  # activations that fp16 does not hold
        q = (rng.standard_normal((T, 4, 128)) * 1e6).astype(np.float32)
        _run(env, rng, 128, 64, 16, 1, 4, lens, dtype, q=q, scale=1e-7)
        q = (rng.standard_normal((T, 4, 128)) * 1e-8).astype(np.float32)
        _run(env, rng, 128, 64, 16, 1, 4, lens, dtype, q=q, scale=1e7)


@pytest.mark.parametrize("lens", [[(1, 200), (1, 40)], [(3, 100), (2, 90)], [(140, 260), (9, 20)]])
def test_non_finite_rows_stay_alone(env, lens):
    """A query row with NaN or inf, and a NaN value seen by some tokens: the other rows are as without them."""
    mnb, torch, dev = env
    rng = np.random.default_rng(4)
    D, ps, Hk, G = 128, 16, 1, 3
    T = sum(a for a, _ in lens)
    pages = sum(-(-n // ps) for _, n in lens)
    host, cache = _cache(env, rng, D, 64, ps, Hk, pages)
    width = max(-(-n // ps) for _, n in lens)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, (_, n) in enumerate(lens):
        w = -(-n // ps)
        table[b, :w] = np.arange(at, at + w)
        at += w
    start = torch.tensor(np.concatenate([[0], np.cumsum([a for a, _ in lens])]), dtype=torch.int32, device=dev)
    kv = torch.tensor([n for _, n in lens], dtype=torch.int32, device=dev)
    q = torch.from_numpy(rng.standard_normal((T, G, D)).astype(np.float16)).to(dev)
    args = (cache, start, kv, torch.from_numpy(table).to(dev), 0.1)
    clean = mnb.mnb_kv4_attention(q, *args)
    bad = q.clone()
    bad[0, 1, 5] = float("nan")
    bad[T - 1, 0, 7] = float("inf")
    got = mnb.mnb_kv4_attention(bad, *args)
    hit = torch.zeros((T, G), dtype=torch.bool, device=dev)
    hit[0, 1] = hit[T - 1, 0] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert torch.isnan(got[0, 1]).all()
    # a NaN group of the last key of sequence 0: only its last token sees it
    n = lens[0][1]
    bb = orc.block_bytes(D, 64)
    blk = host.reshape(-1, bb)[(n - 1) // 16]
    at = orc.param_place(D, 64, (n - 1) % 16, 1, True)
    blk[at: at + 4] = 0xff
    cache2 = mnb.MnbKv4Cache(torch.from_numpy(host).to(dev), ps, D, 64)
    got = mnb.mnb_kv4_attention(q, cache2, *args[1:])
    last = lens[0][0] - 1
    assert torch.isnan(got[last, :, 64:]).all() and torch.equal(got[last, :, :64], clean[last, :, :64])
    rest = [t for t in range(T) if t != last]
    assert torch.equal(got[rest], clean[rest])
    mnb.mnb_check_device_status()


def test_bad_pages_and_lengths(env):
    """A page index outside the cache leaves its keys out, a length beyond the table is cut; the status word says so."""
    mnb, torch, dev = env
    rng = np.random.default_rng(5)
    D, ps, Hk, G = 128, 16, 2, 4
    host, cache = _cache(env, rng, D, 128, ps, Hk, 12)
    for q_len in (1, 3, 140):
        table = np.array([[3, -1, 5, 12, 7, 2 ** 31 - 1, 0, 1, 2, 4], [6, 8, 9, 10, 11, 0, 1, 2, 3, 4]], np.int32)
        kv = np.array([160, 1000], np.int32)
        start = np.array([0, q_len, 2 * q_len], np.int32)
        q = rng.standard_normal((2 * q_len, Hk * G, D)).astype(np.float16)
        up = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        out = mnb.mnb_kv4_attention(up(q), cache, up(start), up(kv), up(table), 0.09)
        want = orc.attention(q, host, start, np.array([160, 160]), table, ps, Hk, 128, 0.09, True, 0)
        _check(out, None, want, "f16")
        with pytest.raises(mnb.MnbError) as e:
            mnb.mnb_check_device_status()
        assert e.value.status == mnb.MNB_ERR_INVALID_ARG
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1])
def test_a_window_beyond_every_key(env, window, dtype):
    """It leaves nothing out, for tokens at negative positions (more tokens than keys) either."""
    lens = [(5, 3), (1, 40), (60, 20)]
    for causal in (False, True):
        _run(env, np.random.default_rng(17), 64, 64, 16, 1, 2, lens, dtype, causal=causal, window=window)


def test_query_ranges_are_clamped(env):
    """q_start that runs past T or backwards reads and writes nothing outside q and out."""
    mnb, torch, dev = env
    rng = np.random.default_rng(6)
    host, cache = _cache(env, rng, 64, 64, 16, 1, 8)
    q = torch.from_numpy(rng.standard_normal((5, 2, 64)).astype(np.float16)).to(dev)
    kv = torch.full((3,), 40, dtype=torch.int32, device=dev)
    table = torch.arange(9, dtype=torch.int32, device=dev).view(3, 3) % 8
    guard = torch.full((25, 2, 64), 3.0, dtype=torch.float16, device=dev)
    out = guard[10:15]
    for start in ([0, 3, 2, 5], [-4, 2, 9, 100], [0, 0, 0, 2 ** 31 - 1], [7, -1, 6, 3]):
        mnb.mnb_kv4_attention(q, cache, torch.tensor(start, dtype=torch.int32, device=dev), kv, table, 0.1, out=out)
    torch.cuda.synchronize()
    assert (guard[:10] == 3).all() and (guard[15:] == 3).all()
    try:
        mnb.mnb_check_device_status()
    except mnb.MnbError:
        pass


def test_strided_q_other_stream_and_graph(env):
    """q as a view of a fused product, a stream of its own, and a captured call that follows new lengths and keys."""
    mnb, torch, dev = env
    rng = np.random.default_rng(7)
    D, ps, Hk, G, B = 128, 16, 2, 4, 3
    host, cache = _cache(env, rng, D, 64, ps, Hk, 40)
    x = torch.from_numpy(rng.standard_normal((B, (Hk * G + 2 * Hk) * D)).astype(np.float16)).to(dev)
    q = x[:, : Hk * G * D].view(B, Hk * G, D)
    table = torch.arange(36, dtype=torch.int32, device=dev).view(B, 12)
    start = torch.arange(B + 1, dtype=torch.int32, device=dev)
    kv = torch.tensor([5, 100, 192], dtype=torch.int32, device=dev)
    plain = mnb.mnb_kv4_attention(q.contiguous(), cache, start, kv, table, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mnb.mnb_kv4_attention(q, cache, start, kv, table, 0.1, stream=side)
    side.synchronize()
    assert torch.equal(got, plain)
    out = torch.empty_like(plain)
    ws = torch.empty(max(16, mnb.mnb_kv4_attention_workspace_bytes(B, B, Hk * G, Hk, D)), dtype=torch.uint8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.mnb_kv4_attention(q, cache, start, kv, table, 0.1, workspace=ws, out=out)
    for lens in ([5, 100, 192], [191, 0, 17], [64, 65, 1]):
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        want = orc.attention(q.cpu().numpy(), host, [0, 1, 2, 3], lens, table.cpu().numpy(), ps, Hk, 64,
                             float(np.float32(0.1)), True, 0)
        _check(out, None, want, "f16", str(lens))
    mnb.mnb_check_device_status()


def test_kept_workspaces(env):
    """Calls without a workspace: the default stream's is kept and grows, others allocate theirs; shapes in turn, three
    streams at once and a captured call beside eager ones give what calls with a workspace of their own give."""
    mnb, torch, dev = env
    rng = np.random.default_rng(18)
    D, ps, Hk, G = 128, 16, 1, 4
    _, cache = _cache(env, rng, D, 128, ps, Hk, 130)
    table = torch.arange(120, dtype=torch.int32, device=dev).view(2, 60)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    calls = []
    for n in (1, 3, 8, 90):
        q = torch.from_numpy(rng.standard_normal((2 * n, Hk * G, D)).astype(np.float16)).to(dev)
        args = (q, cache, i32(0, n, 2 * n), i32(900, 333), table, 0.09)
        ws = torch.empty(mnb.mnb_kv4_attention_workspace_bytes(2 * n, 2, Hk * G, Hk, D), dtype=torch.uint8, device=dev)
        calls.append((args, mnb.mnb_kv4_attention(*args, workspace=ws), ws.numel()))
    mnb._default_workspace.clear()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = mnb.mnb_kv4_attention(*calls[1][0])
    streams = [torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for turn in range(10):
        outs = []
        with torch.cuda.stream(streams[1]):
            graph.replay()
        for s in streams:
            with torch.cuda.stream(s):
                for k in range(4):
                    outs.append((k, mnb.mnb_kv4_attention(*calls[(k + turn) % 4][0]), turn))
        torch.cuda.synchronize()
        for k, o, t in outs:
            assert torch.equal(o, calls[(k + t) % 4][1])
        assert torch.equal(captured, calls[1][1])
    assert mnb._default_workspace[0].numel() >= calls[3][2]

    def thread(k):
        for _ in range(300):
            out = mnb.mnb_kv4_attention(*calls[k][0])
        return torch.equal(out, calls[k][1])

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(thread, range(4)))


def test_offsets_beyond_32_bits(env):
    """A cache of more than 4 GiB: append, read and attention in its last pages."""
    mnb, torch, dev = env
    rng = np.random.default_rng(8)
    D, ps, Hk, G, n = 128, 64, 8, 4, 150
    pages = (5 << 30) // (Hk * 4 * orc.block_bytes(D, 128))
    cache = mnb.MnbKv4Cache(torch.empty((pages, Hk, 4 * orc.block_bytes(D, 128)), dtype=torch.uint8, device=dev), ps, D,
                            128)
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device=dev)
    j = torch.arange(n, device=dev)
    slots = table[0].long()[j // ps] * ps + j % ps
    k = torch.from_numpy(rng.standard_normal((n, Hk, D)).astype(np.float16)).to(dev)
    v = torch.from_numpy(rng.standard_normal((n, Hk, D)).astype(np.float16)).to(dev)
    mnb.mnb_kv4_append(cache, k, v, slots)
    rk, rv = mnb.mnb_kv4_read(cache, slots, dtype=torch.float32)
    for r, x in ((rk, k), (rv, v)):
        c, s, o = orc.quantise(x.float().cpu().numpy(), 128)
        np.testing.assert_array_equal(r.cpu().numpy(), o.astype(np.float32) + c.astype(np.float32) * s.astype(np.float32))
    K, V = rk.double(), rv.double()
    for q_len in (1, 5, 130):
        q = torch.from_numpy(rng.standard_normal((q_len, Hk * G, D)).astype(np.float16)).to(dev)
        out = mnb.mnb_kv4_attention(q, cache, torch.tensor([0, q_len], dtype=torch.int32, device=dev),
                                    torch.tensor([n], dtype=torch.int32, device=dev), table, 0.09)
        s = torch.einsum("ihgd,jhd->hgij", q.double().view(q_len, Hk, G, D), K) * 0.09
        s = s.masked_fill(j[None] > n - q_len + torch.arange(q_len, device=dev)[:, None], float("-inf"))
        want = torch.einsum("hgij,jhd->ihgd", s.softmax(-1), V).reshape(q_len, Hk * G, D)
        assert float((out.double() - want).norm() / want.norm()) <= 2.0 ** -10
    mnb.mnb_check_device_status()


def test_a_long_context_against_fp64(env):
    """Many splits of one sequence: 20000 keys, ragged beside short ones."""
    _run(env, np.random.default_rng(11), 64, 64, 64, 1, 2, [(1, 20000), (1, 3), (1, 700)], "f16")
    _run(env, np.random.default_rng(12), 64, 64, 64, 1, 1, [(1, 9000)], "f32", window=5000)


def test_append_then_attend_as_a_decode_loop(env):
    """Tokens appended one step at a time are seen by the attention of that step."""
    mnb, torch, dev = env
    rng = np.random.default_rng(13)
    D, ps, Hk, G, B = 128, 16, 2, 2, 2
    cache = mnb.mnb_kv4_cache_alloc(8, ps, Hk, D, 64, dev)
    table = torch.tensor([[3, 1, 6], [0, 7, 2]], dtype=torch.int32, device=dev)
    cos, sin = _tables(rng, 64, D)
    cd, sd = torch.from_numpy(cos).to(dev), torch.from_numpy(sin).to(dev)
    start = torch.arange(B + 1, dtype=torch.int32, device=dev)
    host = np.zeros(tuple(cache.pages.shape), np.uint8)
    for step in range(20):
        pos = torch.tensor([step, step + 17], dtype=torch.int32, device=dev)
        slots = torch.stack([table[b, int(pos[b]) // ps].long() * ps + int(pos[b]) % ps for b in range(B)])
        x = rng.standard_normal((B, (G + 2) * Hk, D)).astype(np.float16)
        xd = torch.from_numpy(x).to(dev)
        q = mnb.mnb_kv4_append(cache, xd[:, G * Hk:(G + 1) * Hk], xd[:, (G + 1) * Hk:], slots, q=xd[:, : G * Hk],
                               positions=pos, cos=cd, sin=sd)
        out = mnb.mnb_kv4_attention(q, cache, start, pos + 1, table, 0.1)
        p = pos.cpu().numpy()
        host = orc.append(host, x[:, G * Hk:(G + 1) * Hk].astype(np.float32), x[:, (G + 1) * Hk:].astype(np.float32), p,
                          cos, sin, False, slots.cpu().numpy(), ps, 64).reshape(host.shape)
        np.testing.assert_array_equal(cache.pages.cpu().numpy(), host)
        want = orc.attention(q.cpu().numpy(), host, [0, 1, 2], p + 1, table.cpu().numpy(), ps, Hk, 64,
                             float(np.float32(0.1)), True, 0)
        _check(out, None, want, "f16", f"step {step}")
    mnb.mnb_check_device_status()


def test_binding_refusals(env):
    mnb, torch, dev = env
    cache = mnb.mnb_kv4_cache_alloc(2, 16, 2, 128, 64, dev)
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device=dev)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    slots = torch.arange(3, device=dev)
    with pytest.raises(ValueError):
        mnb.mnb_kv4_append(cache, h(3, 2, 64), h(3, 2, 128), slots)
    with pytest.raises(ValueError):
        mnb.mnb_kv4_append(cache, h(3, 128, 2).transpose(1, 2), h(3, 2, 128), slots)
    with pytest.raises(TypeError):
        mnb.mnb_kv4_append(cache, h(3, 2, 128), h(3, 2, 128).float(), slots)
    with pytest.raises(TypeError):
        mnb.mnb_kv4_append(cache, h(3, 2, 128).bfloat16(), h(3, 2, 128).bfloat16(), slots)
    with pytest.raises(TypeError):
        mnb.mnb_kv4_append(cache, h(3, 2, 128), h(3, 2, 128), slots.int())
    with pytest.raises(ValueError):
        mnb.mnb_kv4_append(cache, h(3, 2, 128), h(3, 2, 128), slots[:2])
    with pytest.raises(ValueError):
        mnb.mnb_kv4_attention(h(3, 4, 128), cache, i32(3), i32(3), i32(3, 2), 0.1)
    with pytest.raises(ValueError):
        mnb.mnb_kv4_attention(h(3, 4, 64), cache, i32(4), i32(3), i32(3, 2), 0.1)
    with pytest.raises(ValueError):
        mnb.MnbKv4Cache(cache.pages[:, :, :64].contiguous(), 16, 128, 64)
    with pytest.raises(mnb.MnbError):
        mnb.MnbKv4Cache(cache.pages, 16, 96, 64)
    with pytest.raises(mnb.MnbError):
        mnb.mnb_kv4_cache_alloc(2, 10, 2, 128, 64, dev)


def test_more_sequences_than_threads_look_at(env):
    """More than 128 sequences: the work list is scanned in turns."""
    rng = np.random.default_rng(14)
    lens = [(int(rng.integers(0, 3)), int(rng.integers(0, 60))) for _ in range(300)] + [(1, 400)]
    _run(env, rng, 64, 64, 16, 1, 2, lens, "f16")
    lens = [(int(rng.integers(0, 60)), int(rng.integers(1, 90))) for _ in range(140)]
    assert _run(env, rng, 64, 32, 16, 1, 2, lens, "f16") == "kv4_tile_tcgen05"


@pytest.mark.parametrize("G,tokens,variant", [(4, 1, "kv4_stream_f16_rows8"), (4, 3, "kv4_stream_f16_rows16"),
                                              (4, 12, "kv4_stream_f16_rows16"), (4, 13, "kv4_tile_tcgen05")])
def test_variant_by_rows(env, G, tokens, variant):
    assert _run(env, np.random.default_rng(15), 128, 128, 16, 1, G, [(tokens, 70), (tokens, 200)], "f16") == variant


def test_programmatic_launch_and_workspace_reuse(env):
    """Append, attention and append again back to back, one workspace, each launched before the last has ended."""
    mnb, torch, dev = env
    rng = np.random.default_rng(16)
    D, ps, Hk, G, B = 128, 16, 2, 4, 4
    cos, sin = (torch.from_numpy(t).to(dev) for t in _tables(rng, 64, D))
    start = torch.arange(B + 1, dtype=torch.int32, device=dev)
    table = torch.arange(B * 4, dtype=torch.int32, device=dev).view(B, 4)
    x = [torch.from_numpy(rng.standard_normal((B, (G + 2) * Hk, D)).astype(np.float16)).to(dev) for _ in range(30)]
    results = []
    for pdl in (False, True):
        cache = mnb.mnb_kv4_cache_alloc(B * 4, ps, Hk, D, 64, dev)
        ws = torch.empty(mnb.mnb_kv4_attention_workspace_bytes(B, B, G * Hk, Hk, D), dtype=torch.uint8, device=dev)
        pos = [torch.full((B,), i, dtype=torch.int32, device=dev) for i in range(30)]
        slots = [table[:, i // ps].long() * ps + i % ps for i in range(30)]
        kv = [p + 1 for p in pos]
        outs = [torch.empty((B, G * Hk, D), dtype=torch.float16, device=dev) for _ in range(30)]
        torch.cuda.synchronize()
        mnb.mnb_set_programmatic_launch(pdl)
        try:
            for i in range(30):
                q = mnb.mnb_kv4_append(cache, x[i][:, G * Hk:(G + 1) * Hk], x[i][:, (G + 1) * Hk:], slots[i],
                                       q=x[i][:, : G * Hk], positions=pos[i], cos=cos, sin=sin)
                mnb.mnb_kv4_attention(q, cache, start, kv[i], table, 0.1, workspace=ws, out=outs[i])
        finally:
            mnb.mnb_set_programmatic_launch(False)
        torch.cuda.synchronize()
        results.append(outs + [cache.pages])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    mnb.mnb_check_device_status()


def test_layer_example(env):
    """The example's layer: 4-bit products, append, attention, from prompts to captured decode steps. Its check is
    against fp32 torch rounded to fp16, so the fp16 norm bound holds."""
    from examples import decode_layer
    _, _, error = decode_layer.run(batch=3, prompt=90, steps=5, q_heads=8, kv_heads=2, head_dim=128, hidden=512, page_size=16)
    assert error <= 2.0 ** -10
