"""Adapters, probabilities and verification of drafted tokens on the GPU, against fp64 and whole-number arithmetic.

Tolerances, with a = sum_r |up s| and b = sum_r |up| sum_k |down x| of the oracle:
* lora, fp16: the result's rounding 2^-11 |out| (2^-25 where it is subnormal), s rounded once: 2^-11 a, and fp32 sums of K
  products and then R, each step of which may cut off one last place: (K / 8 + R + 64) 2^-23 b.
* lora, fp32: the result's rounding 2^-24 |out|, x and s as two fp16 parts: 2^-22 b each, the sums as above with steps of 4: (K / 4 + R + 64)
  2^-23 b.
* softmax: z = (x - max) / T has three roundings, 3 |z| 2^-24 of p; the exponential 2 last places, 2^-22; the sum of V terms by
  threads that add at most V / 512 + 64 of them in turn, the same again for the factors that follow: (V / 512 + 80) 2^-24;
  results below 2^-126 may be anything from 0 to that.
* verify: equal.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import requests_oracle_np as orc

pytestmark = pytest.mark.gpu

NP = {"f16": np.float16, "f32": np.float32}


@pytest.fixture(scope="module")
def env():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import gemm_mnb_gemv_gb300 as mnb
    return mnb, torch, torch.device("cuda:0")


def _lora_inputs(rng, M, K, N, R, count, dtype, ranks="all", without=0.2):
    x = rng.standard_normal((M, K)).astype(NP[dtype])
    base = rng.standard_normal((M, N)).astype(NP[dtype])
    down = (rng.standard_normal((count, R, K)) / np.sqrt(K)).astype(np.float16)
    up = (rng.standard_normal((count, N, R)) / np.sqrt(R)).astype(np.float16)
    scales = rng.uniform(-2, 2, count).astype(np.float32)
    adapter = rng.integers(0, count, M).astype(np.int32)
    adapter[rng.random(M) < without] = -1
    r = None
    if ranks == "uneven":
        r = rng.integers(0, R + 1, count).astype(np.int32)
        for i in range(count):  # what lies beyond an adapter's rank has no part in anything
            down[i, r[i]:] = np.nan
            up[i, :, r[i]:] = np.inf
    return x, base, down, up, r, scales, adapter


def _lora_bound(K, R, dtype, out, a, b):
    if dtype == "f16":
        return 2.0 ** -11 * np.abs(out) + 2.0 ** -25 + 2.0 ** -11 * a + (K / 8 + R + 64) * 2.0 ** -23 * b
    return 2.0 ** -24 * np.abs(out) + 2.0 ** -21 * b + (K / 4 + R + 64) * 2.0 ** -23 * b + 1e-37


def _check_lora(got, x, base, down, up, ranks, scales, adapter, dtype):
    got = got.cpu().numpy().astype(np.float64)
    want, a, b = orc.lora(x, down, up, ranks, scales, adapter, base)
    err, tol = np.abs(got - want), _lora_bound(x.shape[1], down.shape[1], dtype, want, a, b)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())
    none = (adapter < 0) | (adapter >= len(down))
    if base is not None:
        np.testing.assert_array_equal(got[none], base[none].astype(np.float64))


def _up(torch, dev, *arrays):
    return [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M,K,N,R,count,ranks", [
    (1, 16, 1, 8, 1, "all"),
    (1, 256, 64, 8, 3, "uneven"),
    (2, 48, 7, 16, 2, "all"),
    (3, 4096, 130, 16, 5, "all"),
    (15, 272, 33, 24, 4, "uneven"),
    (16, 512, 96, 32, 16, "all"),
    (17, 1024, 257, 32, 40, "uneven"),
    (40, 896, 1152, 64, 6, "all"),
    (64, 2048, 200, 64, 64, "uneven"),
    (65, 80, 4097, 128, 3, "uneven"),
    (130, 640, 64, 128, 130, "all"),
    (333, 144, 72, 72, 2, "uneven"),
    (1024, 64, 40, 8, 7, "all"),
    (1025, 112, 31, 8, 7, "uneven"),
    (1100, 256, 264, 16, 2, "all"),
    (1281, 208, 40, 32, 100, "uneven"),
    (1500, 96, 136, 64, 3, "all"),
    (2100, 128, 96, 128, 5, "uneven"),
])
def test_lora(env, M, K, N, R, count, ranks, dtype):
    mnb, torch, dev = env
    rng = np.random.default_rng(M * 31 + K)
    x, base, down, up, r, scales, adapter = _lora_inputs(rng, M, K, N, R, count, dtype, ranks)
    xd, bd, dd, ud, rd, sd, ad = _up(torch, dev, x, base, down, up, r, scales, adapter)
    got = mnb.mnb_lora(xd, mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd), ad, base=bd)
    _check_lora(got, x, base, down, up, r, scales, adapter, dtype)
    again = bd.clone()
    assert mnb.mnb_lora(xd, mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd), ad, base=again, out=again) is again
    assert torch.equal(again, got)  # in place, and the same bits on every run
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M,K,N,R,run", [
    (1030, 2048, 1000, 16, 515),     # clusters of 8
    (2048, 16, 32, 32, 683),         # most CTAs have no part of K and N
    (3000, 1104, 521, 64, 2999),
    (5000, 528, 648, 40, 1500),
    (9000, 384, 320, 128, 4000),
    (20000, 144, 200, 64, 7000),     # one CTA takes several tiles
    (20000, 64, 72, 8, 20000),
    (1700, 8192, 136, 128, 1600),    # a prompt and 100 rows of their own
])
def test_lora_prompts(env, M, K, N, R, run, dtype):
    """Runs of rows with one adapter, as prompts have them, and rows that change with every one at the end."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M + R)
    x, base, down, up, r, scales, adapter = _lora_inputs(rng, M, K, N, R, 6, dtype, "uneven" if R == 40 else "all", without=0)
    tail = min(M % run, 100)
    adapter[:M - tail] = (np.arange(M - tail) // run) % 6
    if M == 5000:
        adapter[1500:3000] = -1
    xd, bd, dd, ud, rd, sd, ad = _up(torch, dev, x, base, down, up, r, scales, adapter)
    pool = mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd)
    got = mnb.mnb_lora(xd, pool, ad, base=bd)
    _check_lora(got, x, base, down, up, r, scales, adapter, dtype)
    again = bd.clone()
    mnb.mnb_lora(xd, pool, ad, base=again, out=again)
    assert torch.equal(again, got)
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M", [3, 300, 1600])
def test_lora_views_of_fused_products(env, M, dtype):
    """x, base and out as column ranges of wider matrices; what lies beside out stays as it was."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M)
    K, N, wide = 160, 72, 72 + 32 + 11 * 8
    x, base, down, up, r, scales, adapter = _lora_inputs(rng, M, K, N, 16, 4, dtype)
    xw = torch.randn(M, K + 24, device=dev).to(torch.from_numpy(x).dtype)
    bw, ow = torch.randn(M, wide, device=dev).to(xw.dtype), torch.full((M, wide), 7.0, device=dev).to(xw.dtype)
    xw[:, 8:8 + K], bw[:, 32:32 + N] = _up(torch, dev, x, base)
    dd, ud, sd, ad = _up(torch, dev, down, up, scales, adapter)
    got = mnb.mnb_lora(xw[:, 8:8 + K], mnb.MnbLoraPool(dd, ud, scales=sd), ad, base=bw[:, 32:32 + N], out=ow[:, 16:16 + N])
    _check_lora(got, x, base, down, up, None, scales, adapter, dtype)
    assert (ow[:, :16] == 7).all() and (ow[:, 16 + N:] == 7).all()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("N", [1, 31, 65, 518, 1027])
@pytest.mark.parametrize("M", [40, 700, 1600, 2500])
def test_lora_odd_strides(env, M, N, dtype):
    """Rows of base and out that begin anywhere, in place and apart; what lies beside out stays as it was."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M + N)
    x, base, down, up, r, scales, adapter = _lora_inputs(rng, M, 96, N, 24, 3, dtype, "uneven", without=0.1)
    adapter[M // 8: M // 2] = 1
    xd, bd, dd, ud, rd, sd, ad = _up(torch, dev, x, base, down, up, r, scales, adapter)
    pool = mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd)
    for more in (9, 14):
        wide = torch.full((M, N + 8 + more), 7.0, device=dev).to(bd.dtype)
        wide[:, 8:8 + N] = bd
        apart = torch.full((M, N + more), 5.0, device=dev).to(bd.dtype)
        got = mnb.mnb_lora(xd, pool, ad, base=wide[:, 8:8 + N], out=apart[:, :N])
        _check_lora(got, x, base, down, up, r, scales, adapter, dtype)
        assert (apart[:, N:] == 5).all()
        mnb.mnb_lora(xd, pool, ad, base=wide[:, 8:8 + N], out=wide[:, 8:8 + N])
        assert torch.equal(wide[:, 8:8 + N], got) and (wide[:, :8] == 7).all() and (wide[:, 8 + N:] == 7).all()
        none = mnb.mnb_lora(xd, pool, ad, out=apart[:, :N])
        _check_lora(none, x, None, down, up, r, scales, adapter, dtype)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_lora_without_base_scales_and_with_bad_indices(env, dtype):
    mnb, torch, dev = env
    rng = np.random.default_rng(5)
    x, _, down, up, _, _, adapter = _lora_inputs(rng, 50, 64, 30, 8, 3, dtype)
    dd, ud = _up(torch, dev, down, up)
    adapter[::7] = 3
    adapter[1::7] = -5
    adapter[2] = 2 ** 31 - 1
    adapter[3] = -2 ** 31
    xd, ad = _up(torch, dev, x, adapter)
    mnb.mnb_check_device_status()
    got = mnb.mnb_lora(xd, mnb.MnbLoraPool(dd, ud), ad)
    _check_lora(got, x, None, down, up, None, None, adapter, dtype)
    assert not got.cpu().numpy()[(adapter < 0) | (adapter > 2)].any()
    with pytest.raises(mnb.MnbError, match="INVALID_ARG"):
        mnb.mnb_check_device_status()
    mnb.mnb_check_device_status()


def test_lora_rows_of_any_size(env):
    """Rows from 1e-7 to the largest that the products bear keep their precision; a row with inf or NaN stays alone."""
    mnb, torch, dev = env
    rng = np.random.default_rng(6)
    for dtype, sizes in (("f16", [1e-7, 1e-3, 1.0, 1e4]), ("f32", [1e-30, 1e-3, 1.0, 1e30])):
        x, base, down, up, _, scales, adapter = _lora_inputs(rng, 20, 96, 50, 16, 2, dtype, without=0)
        x = (x.astype(np.float64) * np.resize(sizes, 20)[:, None]).astype(NP[dtype])
        base *= 0
        if dtype == "f16":  # s beyond fp16: 96 products of up to 4e4 * 30
            down[0] *= np.float16(300)
            scales *= np.float32(1e-4)
        args = _up(torch, dev, x, base, down, up, scales, adapter)
        call = lambda xd: mnb.mnb_lora(xd, mnb.MnbLoraPool(args[2], args[3], scales=args[4]), args[5], base=args[1])  # noqa: E731
        got = call(args[0])
        _check_lora(got, x, base, down, up, None, scales, adapter, dtype)
        bad = args[0].clone()
        bad[4, 3], bad[9, 60] = float("inf"), float("nan")
        odd = call(bad)
        keep = torch.ones(20, dtype=torch.bool, device=dev)
        keep[[4, 9]] = False
        assert torch.equal(odd[keep], got[keep])
        assert not torch.isfinite(odd[9]).any() and not torch.isfinite(odd[4]).any()


def test_lora_captured_graph_follows_its_inputs(env):
    mnb, torch, dev = env
    rng = np.random.default_rng(7)
    x, base, down, up, r, scales, adapter = _lora_inputs(rng, 40, 256, 100, 32, 9, "f16", "uneven")
    xd, bd, dd, ud, rd, sd, ad = _up(torch, dev, x, base, down, up, r, scales, adapter)
    pool, out = mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd), torch.empty_like(bd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mnb.mnb_lora(xd, pool, ad, base=bd, out=out)
    for i in range(3):
        adapter = rng.integers(-1, 9, 40).astype(np.int32)
        ad.copy_(torch.from_numpy(adapter))
        graph.replay()
        _check_lora(out, x, base, down, up, r, scales, adapter, "f16")


def test_lora_pool_beyond_32_bits(env):
    """The last adapter of a pool of more than 2^32 elements."""
    mnb, torch, dev = env
    K, N, R = 16384, 64, 128
    count = 2 ** 32 // (K * R) + 1
    down = torch.zeros(count, R, K, dtype=torch.float16, device=dev)
    up = torch.zeros(count, N, R, dtype=torch.float16, device=dev)
    rng = np.random.default_rng(8)
    x, base, d, u, _, _, _ = _lora_inputs(rng, 2, K, N, R, 1, "f16")
    down[-1:], up[-1:], xd, bd = _up(torch, dev, d, u, x, base)
    ad = torch.full((2,), count - 1, dtype=torch.int32, device=dev)
    got = mnb.mnb_lora(xd, mnb.MnbLoraPool(down, up), ad, base=bd)
    _check_lora(got, x, base, d, u, None, None, np.zeros(2, np.int32), "f16")


# ---------------------------------------------------------------------------------------


def _check_softmax(got, x, temperature):
    got, V = got.cpu().numpy().astype(np.float64), x.shape[1]
    want = orc.softmax(x, temperature)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    for r in range(len(x)):
        t = 1.0 if temperature is None else float(temperature[r])
        if np.isnan(want[r]).any():
            continue
        if t == 0 or x[r].max() == -np.inf:
            np.testing.assert_array_equal(got[r], want[r])
            continue
        with np.errstate(invalid="ignore"):
            z = np.abs((x[r].astype(np.float64) - x[r].max()) / t)
        z = np.where(want[r] == 0, 0, z)
        tol = want[r] * (3 * z + 4 + V / 512 + 80) * 2.0 ** -24 + 2.0 ** -126
        assert (np.abs(got[r] - want[r]) <= tol).all(), (r, float((np.abs(got[r] - want[r]) / tol).max()))


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("rows,V", [(1, 1), (2, 7), (3, 512), (1, 4099), (5, 32003), (1, 128256), (40, 5001), (700, 130), (161, 2048),
                                    (1, 300001), (330, 9000), (33, 17001), (6, 200003),
                                    (9, 131058), (20, 131059), (40, 70003), (65, 32001), (129, 16385)])
def test_softmax(env, rows, V, dtype):
    mnb, torch, dev = env
    rng = np.random.default_rng(rows + V)
    x = (rng.standard_normal((rows, V)) * 4).astype(NP[dtype])
    x[rng.random((rows, V)) < 0.05] = -np.inf
    t = rng.choice([0.0, 0.3, 1.0, 2.5, 1e-42, 1e30], rows).astype(np.float32)
    t[0] = 1.0
    xd, td = _up(torch, dev, x, t)
    _check_softmax(mnb.mnb_softmax(xd), x, None)
    finite = np.where(t < 1e-30, 0, t)  # next to 0: 1 shared by the largest
    got = mnb.mnb_softmax(xd, temperature=td)
    sure = (t == 0) | (t > 1e-30)
    if sure.any():
        _check_softmax(got[torch.from_numpy(sure).to(dev)], x[sure], finite[sure])
    for r in np.nonzero(~sure)[0]:
        top = x[r] == x[r].max()
        if x[r].max() > -np.inf:
            np.testing.assert_allclose(got[r].cpu().numpy(), top / top.sum(), rtol=1e-6)


@pytest.mark.parametrize("rows,V", [(3, 1), (5, 999), (40, 16377), (7, 40001), (35, 40001), (130, 17001)])
def test_softmax_in_place(env, rows, V):
    mnb, torch, dev = env
    rng = np.random.default_rng(V)
    x = rng.standard_normal((rows, V)).astype(np.float32)
    t = rng.choice([0.0, 0.5, 1.0], rows).astype(np.float32)
    xd, td = _up(torch, dev, x, t)
    want = mnb.mnb_softmax(xd, temperature=td)
    assert mnb.mnb_softmax(xd, temperature=td, out=xd) is xd
    assert torch.equal(xd, want)
    _check_softmax(xd, x, t)


def test_softmax_odd_rows_and_views(env):
    mnb, torch, dev = env
    V = 1003
    x = np.random.default_rng(9).standard_normal((10, V)).astype(np.float32)
    x[0] = -np.inf
    x[1, 5] = np.nan
    x[2, 6] = np.inf
    x[3, [9, 700]] = 50.0
    x[4] = 3e38
    x[5, 1:] = -3e38
    x[8, 100] = np.inf
    t = np.float32([1, 1, 1, 0, 1, 1, -1, np.nan, 0, 0])
    wide = torch.zeros(10, V + 6, device=dev)
    wide[:, 3:3 + V] = torch.from_numpy(x).to(dev)
    view = wide[:, 4:4 + V - 1]  # 16 bytes into the row
    got = mnb.mnb_softmax(view, temperature=torch.from_numpy(t).to(dev))
    _check_softmax(got, x[:, 1:], t)
    assert not got[0].any()
    assert int(got[3].argmax()) == 8 and float(got[3].sum()) == 1


# ---------------------------------------------------------------------------------------


def _draft_case(rng, B, V, top, lookup):
    n = rng.integers(0, top + 1, B)
    n[-1] = top
    start = np.concatenate([[0], n.cumsum()]).astype(np.int32)
    D = int(start[-1])
    soft = lambda z: (np.exp(z) / np.exp(z).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
    z = rng.standard_normal((D + B, V)) * 2
    target = soft(z)
    seq = np.repeat(np.arange(B), n)
    draft = None if lookup else soft(z[np.arange(D) + seq] + 0.5 * rng.standard_normal((D, V)))
    src = target[np.arange(D) + seq] if lookup else draft
    cum = src.astype(np.float64).cumsum(-1)
    tokens = np.minimum((cum < (rng.random(D) * cum[:, -1] if D else np.zeros(0))[:, None]).sum(-1), V - 1).astype(np.int32)
    if lookup and D:
        tokens[::2] = target[(np.arange(D) + seq)[::2]].argmax(-1)
    return target, draft, tokens, start, rng.random(D).astype(np.float32), rng.random(B).astype(np.float32)


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("B,V,top", [(1, 1, 0), (1, 2, 1), (1, 1000, 4), (3, 33, 2), (2, 128256, 3), (20, 5003, 8), (300, 257, 5), (9, 1028, 40),
                                     (700, 1026, 1), (3, 270001, 2), (70, 9001, 3), (40, 20001, 2), (520, 700, 1)])
def test_verify(env, B, V, top, lookup):
    mnb, torch, dev = env
    case = _draft_case(np.random.default_rng(B + V), B, V, top, lookup)
    tokens, accepted = mnb.mnb_verify(*_up(torch, dev, *case))
    want, want_n = orc.verify(*case)
    np.testing.assert_array_equal(accepted.cpu().numpy(), want_n)
    np.testing.assert_array_equal(tokens.cpu().numpy(), want)


@pytest.mark.parametrize("apart,every", [(1, 1), (1, 3), (30, 16)])
def test_verify_borders(env, apart, every):
    """Probabilities whose sums are exact, at random numbers on and next to every border."""
    mnb, torch, dev = env
    V = 300
    rng = np.random.default_rng(3)
    k = rng.integers(0, 9, V)
    k[[0, 1, 17, V - 1]] = 0
    k[100] += 1024 - k.sum()
    p = np.zeros(V * apart, np.float32)
    p[::apart] = k / 1024
    edges = np.unique(np.concatenate([[0], k.cumsum()]))[:-1]
    u = (edges / 1024).astype(np.float32)
    v = np.concatenate([u, np.nextafter(u, np.float32(1)), np.nextafter(u, np.float32(-1)), np.float32([1, 2, -1, np.nan, 1e-45, 1e-20])])[::every]
    B = len(v)
    zero = np.zeros(0, np.float32)
    case = (np.tile(p, (B, 1)), None, zero.astype(np.int32), np.zeros(B + 1, np.int32), zero, v.astype(np.float32))
    tokens, accepted = mnb.mnb_verify(*_up(torch, dev, *case))
    np.testing.assert_array_equal(tokens.cpu().numpy(), orc.verify(*case)[0])
    assert not accepted.any()
    assert (p[tokens.cpu().numpy()] > 0).all()  # nothing impossible is drawn


@pytest.mark.parametrize("V,times", [(400, 1), (400, 40), (9001, 1)])
def test_verify_odd_values(env, V, times):
    mnb, torch, dev = env
    rng = np.random.default_rng(4)
    target, draft, tokens, start, u, v = _draft_case(rng, 16, V, 2, False)
    start = np.arange(0, 33, 2).astype(np.int32)
    z = rng.dirichlet(np.ones(V), 48).astype(np.float32)
    target, draft = z, z[:32].copy()
    tokens = rng.integers(0, V, 32).astype(np.int32)
    u = np.full(32, 0.5, np.float32)
    draft[:8] = target[[0, 1, 3, 4, 6, 7, 9, 10]]   # p - q is 0 everywhere
    u[:8] = 1.0                                     # and rejected: drawn from p
    target[12:15] = 0                               # all 0
    target[15] = np.nan
    draft[11] = np.nan
    tokens[14], tokens[17] = V, -1                  # no such tokens
    target[24, 7], target[24, 9] = np.inf, -3.0
    draft[20, tokens[20]] = 0                       # drawn though the draft gave it 0
    many = lambda x: np.concatenate([x] * times)  # noqa: E731
    start = np.arange(0, 32 * times + 1, 2).astype(np.int32)
    case = (many(target), many(draft), many(tokens), start, many(u), many(v))
    mnb.mnb_check_device_status()
    got, accepted = mnb.mnb_verify(*_up(torch, dev, *case))
    want, want_n = orc.verify(*case)
    np.testing.assert_array_equal(accepted.cpu().numpy(), want_n)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert (want == -1).any()
    with pytest.raises(mnb.MnbError, match="INVALID_ARG"):
        mnb.mnb_check_device_status()


@pytest.mark.parametrize("B", [5, 600])
def test_verify_padded_batch(env, B):
    """Room for more drafted tokens than the sequences have: what lies behind them is neither used nor written."""
    mnb, torch, dev = env
    target, draft, tokens, start, u, v = _draft_case(np.random.default_rng(15), B, 300, 3, False)
    D, more = len(tokens), 11
    case = (np.concatenate([target, np.full((more, 300), np.nan, np.float32)]), np.concatenate([draft, np.full((more, 300), np.nan, np.float32)]),
            np.concatenate([tokens, np.full(more, 1 << 30, np.int32)]), start, np.concatenate([u, np.full(more, np.nan, np.float32)]), v)
    out = torch.full((D + more + B,), -7, dtype=torch.int32, device=dev)
    mnb.mnb_verify(*_up(torch, dev, *case), tokens=out)
    want = orc.verify(target, draft, tokens, start, u, v)[0]
    np.testing.assert_array_equal(out.cpu().numpy(), np.concatenate([want, np.full(more, -7)]))
    mnb.mnb_check_device_status()


def test_verify_views(env):
    """Rows that lie apart, at any multiple of four bytes."""
    mnb, torch, dev = env
    case = _draft_case(np.random.default_rng(11), 6, 1009, 3, False)
    target, draft, tokens, start, u, v = _up(torch, dev, *case)
    tw, dw = torch.rand(len(target), 1009 + 14, device=dev), torch.rand(len(draft), 1009 + 9, device=dev)
    tw[:, 4:1013], dw[:, 8:1017] = target, draft
    got, accepted = mnb.mnb_verify(tw[:, 4:1013], dw[:, 8:1017], tokens, start, u, v)
    want, want_n = orc.verify(*case)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    np.testing.assert_array_equal(accepted.cpu().numpy(), want_n)


# ---------------------------------------------------------------------------------------


def _step_inputs(mnb, torch, dev, B=5, n=3, K=256, V=515, pools=4):
    """A verify step: hidden states, a 4-bit output product with adapters, temperatures, drafts."""
    import mnb_synth as syn
    from tests.helpers import upload_weight
    rng = np.random.default_rng(12)
    M = B * (n + 1)
    w = syn.make_weight(syn.custom("verify_step", M, K, V, 32, scale_lo=0.02, scale_hi=0.05))
    parts = upload_weight(w, dev)
    x, _, down, up, r, scales, adapter = _lora_inputs(rng, M, K, V, 16, pools, "f16", "uneven")
    adapter = np.repeat(rng.integers(-1, pools, B), n + 1).astype(np.int32)
    t = np.repeat(rng.choice([0.0, 0.8, 1.2], B), n + 1).astype(np.float32)
    draft = rng.dirichlet(np.ones(V), B * n).astype(np.float32)
    tokens = rng.integers(0, V, B * n).astype(np.int32)
    start = np.arange(0, B * n + 1, n).astype(np.int32)
    u, v = rng.random(B * n).astype(np.float32) ** 4, rng.random(B).astype(np.float32)
    xd, dd, ud, rd, sd, ad, td, qd, kd, std, u1, v1 = _up(torch, dev, x, down, up, r, scales, adapter, t, draft, tokens, start, u, v)
    pool = mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd)

    repacked = mnb.mnb_repack(parts[0], K, V, 32)

    def step():
        y = mnb.mnb_gemm(xd, *parts, K, V, 32, repacked=repacked)
        mnb.mnb_lora(xd, pool, ad, base=y, out=y)
        p = mnb.mnb_softmax(y, temperature=td)
        return (y, p, *mnb.mnb_verify(p, qd, kd, std, u1, v1))

    from oracle import mnb_oracle as mo
    Y, S = mo.matmul(x, w.packed, w.scales, w.zero_points, K, V, 32)
    return step, (x, down, up, r, scales, adapter, Y, S, t, draft, tokens, start, u, v)


def _check_step(outputs, inputs):
    y, p, tokens, accepted = (o.cpu().numpy() for o in outputs)
    x, down, up, r, scales, adapter, Y, S, t, draft, drafted, start, u, v = inputs
    want, a, b = orc.lora(x, down, up, r, scales, adapter, Y)
    tol = 2e-3 * S + 1e-5 + _lora_bound(x.shape[1], down.shape[1], "f16", want, a, b)
    assert (np.abs(y - want) <= tol).all()
    import torch
    _check_softmax(torch.from_numpy(p), y, t)
    got = orc.verify(p, draft, drafted, start, u, v)
    np.testing.assert_array_equal(tokens, got[0])
    np.testing.assert_array_equal(accepted, got[1])


@pytest.mark.parametrize("programmatic", [False, True])
def test_verify_step(env, programmatic):
    """Product, adapters, probabilities, verification: eager, on another stream, captured and replayed."""
    mnb, torch, dev = env
    step, inputs = _step_inputs(mnb, torch, dev)
    torch.cuda.synchronize()
    mnb.mnb_set_programmatic_launch(programmatic)
    try:
        first = step()
        _check_step(first, inputs)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph):
            captured = step()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, captured):
            assert torch.equal(a, b) and torch.equal(a, c)
    finally:
        mnb.mnb_set_programmatic_launch(False)
    mnb.mnb_check_device_status()


def test_bindings_refuse(env):
    mnb, torch, dev = env
    h = dict(dtype=torch.float16, device=dev)
    pool = mnb.MnbLoraPool(torch.zeros(2, 8, 32, **h), torch.zeros(2, 12, 8, **h))
    x, idx = torch.zeros(3, 32, **h), torch.zeros(3, dtype=torch.int32, device=dev)
    cases = [
        (TypeError, "adapter must be torch.int32", lambda: mnb.mnb_lora(x, pool, idx.long())),
        (ValueError, "adapter must be", lambda: mnb.mnb_lora(x, pool, idx[:2].clone())),
        (ValueError, "x must be", lambda: mnb.mnb_lora(x[:, :16], pool, idx)),
        (TypeError, "x must be", lambda: mnb.mnb_lora(None, pool, idx)),
        (TypeError, "x must be float16 or float32", lambda: mnb.mnb_lora(x.bfloat16(), pool, idx)),
        (TypeError, "base must be torch.float16", lambda: mnb.mnb_lora(x, pool, idx, base=torch.zeros(3, 12, device=dev))),
        (ValueError, "base must be", lambda: mnb.mnb_lora(x, pool, idx, base=torch.zeros(3, 11, **h))),
        (ValueError, "one after the other", lambda: mnb.mnb_lora(x, pool, idx, base=torch.zeros(12, 3, **h).t())),
        (mnb.MnbError, "base_stride", lambda: mnb.mnb_lora(x, pool, idx, base=torch.zeros(1, 12, **h).expand(3, 12))),
        (mnb.MnbError, "max_rank", lambda: mnb.MnbLoraPool(torch.zeros(2, 4, 32, **h), torch.zeros(2, 12, 4, **h))),
        (ValueError, "up must be", lambda: mnb.MnbLoraPool(torch.zeros(2, 8, 32, **h), torch.zeros(1, 12, 8, **h))),
        (mnb.MnbError, "K=4294967312", lambda: mnb.MnbLoraPool(torch.zeros(2, 8, 1, **h).expand(2, 8, 2 ** 32 + 16), pool.up)),
        (mnb.MnbError, "N=4294967297", lambda: mnb.MnbLoraPool(pool.down, torch.zeros(2, 1, 8, **h).expand(2, 2 ** 32 + 1, 8))),
        (ValueError, "contiguous", lambda: mnb.MnbLoraPool(torch.zeros(2, 8, 64, **h)[:, :, :32], torch.zeros(2, 12, 8, **h))),
        (TypeError, "scales must be torch.float32", lambda: mnb.MnbLoraPool(pool.down, pool.up, scales=torch.zeros(2, **h))),
        (ValueError, "logits must be", lambda: mnb.mnb_softmax(x[0])),
        (TypeError, "logits must be float16 or float32", lambda: mnb.mnb_softmax(x.double())),
        (ValueError, "temperature must be", lambda: mnb.mnb_softmax(x, temperature=torch.zeros(2, device=dev))),
        (TypeError, "out must be", lambda: mnb.mnb_softmax(x, out=x)),
    ]
    p, q = torch.zeros(5, 9, device=dev), torch.zeros(3, 9, device=dev)
    start, u, v = torch.zeros(3, dtype=torch.int32, device=dev), torch.zeros(3, device=dev), torch.zeros(2, device=dev)
    cases += [
        (ValueError, "target must be", lambda: mnb.mnb_verify(p[:4], q, idx, start, u, v)),
        (ValueError, "draft must be", lambda: mnb.mnb_verify(p, q[:2], idx, start, u, v)),
        (TypeError, "target must be torch.float32", lambda: mnb.mnb_verify(p.half(), q, idx, start, u, v)),
        (ValueError, "draft_start must be", lambda: mnb.mnb_verify(p, q, idx, start[:2].clone(), u, v)),
        (TypeError, "u_accept must be torch.float32", lambda: mnb.mnb_verify(p, q, idx, start, idx, v)),
        (ValueError, "target, draft_tokens and u_next", lambda: mnb.mnb_verify(p, q, None, start, u, v)),
    ]
    for kind, word, call in cases:
        with pytest.raises(kind, match=word):
            call()


def test_threads_share_a_workspace(env):
    """Calls of every kind that has a workspace, of four host threads on one stream with one workspace: the launches of each
    stay together."""
    from concurrent.futures import ThreadPoolExecutor
    mnb, torch, dev = env
    rng = np.random.default_rng(14)
    D, pages, length = 64, 20, 1200
    cache = mnb.MnbKv4Cache(torch.zeros(mnb.mnb_kv4_cache_bytes(pages, 64, 2, D, 32), dtype=torch.uint8, device=dev).view(pages, 2, -1),
                            64, D, 32)
    k, q = (torch.randn(n, 2, D, device=dev).half() for n in (length, 2))
    mnb.mnb_kv4_append(cache, k, k, torch.arange(length, device=dev))
    start, lens, table = _up(torch, dev, np.int32([0, 2]), np.int32([length]), np.arange(pages, dtype=np.int32)[None])
    x, base, down, up, _, scales, adapter = _up(torch, dev, *_lora_inputs(rng, 1500, 64, 96, 16, 5, "f16"))
    pool = mnb.MnbLoraPool(down, up, scales=scales)
    logits = torch.randn(130, 40000, device=dev)
    drafts = _up(torch, dev, *_draft_case(rng, 600, 2000, 1, True))
    forms = [lambda w: mnb.mnb_kv4_attention(q, cache, start, lens, table, 0.1, workspace=w),
             lambda w: mnb.mnb_lora(x, pool, adapter, base=base, workspace=w),
             lambda w: mnb.mnb_softmax(logits, workspace=w),
             lambda w: mnb.mnb_verify(*drafts, workspace=w)[0]]
    wants = [f(None) for f in forms]
    torch.cuda.synchronize()
    shared = torch.empty(1 << 24, dtype=torch.uint8, device=dev)
    for workspace in (None, shared):
        with ThreadPoolExecutor(4) as threads:
            outs = list(threads.map(lambda f: [f(workspace) for _ in range(100)], forms))
        for got, want in zip(outs, wants):
            assert all(torch.equal(o, want) for o in got)
    mnb.mnb_check_device_status()


def test_graphs_replayed_at_once(env):
    """Two captured runs of calls with workspaces, replayed on two streams at the same time, inputs changed in between."""
    mnb, torch, dev = env
    rng = np.random.default_rng(16)
    graphs = []
    for M, rows in ((1500, 130), (700, 300)):
        x, base, down, up, _, scales, adapter = _up(torch, dev, *_lora_inputs(rng, M, 64, 96, 16, 5, "f16"))
        pool = mnb.MnbLoraPool(down, up, scales=scales)
        logits = torch.randn(rows, 40000, device=dev)
        drafts = _up(torch, dev, *_draft_case(rng, 600, 2000, 1, True))

        def run(x=x, base=base, pool=pool, adapter=adapter, logits=logits, drafts=drafts):
            return mnb.mnb_lora(x, pool, adapter, base=base), mnb.mnb_softmax(logits), *mnb.mnb_verify(*drafts)

        run()
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs = run()
        graphs.append((side, graph, outs, run, adapter, logits))
    for turn in range(3):
        for _, _, _, _, adapter, logits in graphs:
            adapter.copy_(torch.roll(adapter, 37)), logits.mul_(1.5)
        torch.cuda.synchronize()
        for _ in range(10):
            for side, graph, *_ in graphs:
                with torch.cuda.stream(side):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, outs, run, _, _ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, run())), turn
    mnb.mnb_check_device_status()


def test_no_rows(env):
    mnb, torch, dev = env
    h = dict(dtype=torch.float16, device=dev)
    pool = mnb.MnbLoraPool(torch.zeros(2, 8, 32, **h), torch.zeros(2, 12, 8, **h))
    i32 = dict(dtype=torch.int32, device=dev)
    assert mnb.mnb_lora(torch.zeros(0, 32, **h), pool, torch.zeros(0, **i32)).shape == (0, 12)
    assert mnb.mnb_softmax(torch.zeros(0, 5, **h)).shape == (0, 5)
    none = torch.zeros(0, device=dev)
    tokens, accepted = mnb.mnb_verify(torch.zeros(0, 5, device=dev), None, torch.zeros(0, **i32), torch.zeros(1, **i32), none, none)
    assert tokens.shape == (0,) and accepted.shape == (0,)


def test_workspaces_of_other_streams_are_held(env):
    """On a stream of their own, calls allocate their workspaces: no output of the call may get the same bytes."""
    mnb, torch, dev = env
    case = _draft_case(np.random.default_rng(13), 600, 2000, 1, True)
    want, want_n = orc.verify(*case)
    args = _up(torch, dev, *case)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(4):
            room = torch.empty(mnb.mnb_verify_workspace_bytes(600, 2000), dtype=torch.uint8, device=dev)
            del room  # what the next allocation of these bytes gets
            tokens, accepted = mnb.mnb_verify(*args)
    side.synchronize()
    np.testing.assert_array_equal(tokens.cpu().numpy(), want)
    np.testing.assert_array_equal(accepted.cpu().numpy(), want_n)


def test_example_runs(env):
    from examples import verify_step
    accepted, _, _ = verify_step.run(batch=5, drafts=3, steps=3, vocab=1003 * 32, hidden=256, adapters=3, rank=8)
    assert 0 <= accepted <= 3
