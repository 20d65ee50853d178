"""Adapters, probabilities and verification on the GPU where one path ends and the next begins, against fp64 and whole numbers.

Tolerances beyond those of the entry points' other tests:
* lora, fp16, rows of x with one element that is not 0: down x is exact in fp32 (22 bits), so what is left is the result's rounding
  2^-11 |out| (2^-25 where it is subnormal), s as two fp16 parts, 2^-22 a with a = sum_r |up s|, and fp32 sums of 2 R products, each
  step of which may cut off one last place: (2 R + 16) 2^-23 a.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import requests_oracle_np as orc
from tests.test_gpu_requests import _check_lora, _lora_inputs, _up, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R", [8, 16, 24, 32, 64, 72, 128])
@pytest.mark.parametrize("M,run", [(20, 1), (300, 60), (1500, 1), (2500, 700), (2500, 2500), (9000, 3000)])
def test_lora_fp16_keeps_the_first_products_precision(env, M, run, R):  # noqa: F811
    """Bases that the adapters' results cancel: what is left shows the bits of down x beyond fp16."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M + R)
    K, N = 208, 264
    x, _, down, up, _, scales, adapter = _lora_inputs(rng, M, K, N, R, 5, "f16", without=0)
    adapter[:] = np.arange(M) // run % 5
    at = rng.integers(0, K, M)
    one = x[np.arange(M), at]
    x[:] = 0
    x[np.arange(M), at] = one
    base = (-orc.lora(x, down, up, None, scales, adapter, None)[0]).astype(np.float16)
    want, a, _ = orc.lora(x, down, up, None, scales, adapter, base)
    xd, bd, dd, ud, sd, ad = _up(torch, dev, x, base, down, up, scales, adapter)
    got = mnb.mnb_lora(xd, mnb.MnbLoraPool(dd, ud, scales=sd), ad, base=bd).cpu().numpy().astype(np.float64)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -22 * a + (2 * R + 16) * 2.0 ** -23 * a
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("M,K,N,R", [(9000, 160, 2600, 128), (6000, 64, 4100, 64), (4000, 16, 32, 128), (20000, 96, 200, 16), (3000, 4096, 32, 72)])
def test_lora_prompts_between_rows_without_adapter(env, M, K, N, R, in_place):  # noqa: F811
    """Prompts without an adapter or with one of rank 0 between others: their tiles run through the tensor cores' kernel without
    products, and where base and out are apart without anything else that its warps wait for together."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M + K + R)
    x, base, down, up, _, scales, _ = _lora_inputs(rng, M, K, N, R, 4, "f16")
    ranks = np.int32([R, 0, R - 3, 1])
    adapter = np.repeat(np.int32([-1, -1, 0, 1, -1, 2, 1, 1, -1, 3, -1]), -(-M // 11))[:M].copy()
    adapter[rng.integers(0, M, 40)] = 2
    xd, bd, dd, ud, rd, sd, ad = _up(torch, dev, x, base, down, up, ranks, scales, adapter)
    pool = mnb.MnbLoraPool(dd, ud, ranks=rd, scales=sd)
    first = None
    for _ in range(20):
        out = bd.clone() if in_place else torch.full_like(bd, float("nan"))
        mnb.mnb_lora(xd, pool, ad, base=out if in_place else bd, out=out)
        first = out if first is None else first
        assert torch.equal(out, first)
    _check_lora(first, x, base, down, up, ranks, scales, adapter, "f16")
    assert mnb.mnb_last_variant() == "lora_tile_tcgen05"
    mnb.mnb_check_device_status()


# What stands for u_accept below 0, at 1 and above, or is not a number, and the probabilities of a token that is accepted, or not, with it:
# u is held to 0 .. 1 - 2^-24.
HELD = [(1.0, 0.25, 0.25, True), (2.0, 0.25, 0.25, True), (np.inf, 1.0, 1.0, True), (1.0, 0.25, 0.5, False), (-1.0, 2.0 ** -30, 1.0, True),
        (np.nan, 2.0 ** -30, 1.0, True), (0.0, 0.0, 0.5, False), (1.0, 1 - 2.0 ** -24, 1.0, False), (-np.inf, 0.0, 0.5, False)]


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("times", [1, 80])
def test_verify_holds_u_accept_below_one(env, times, lookup):  # noqa: F811
    mnb, torch, dev = env
    held = [h for h in HELD if not lookup or h[2] == 1.0] * times
    B, V = len(held), 40
    target, draft = np.zeros((2 * B, V), np.float32), np.zeros((B, V), np.float32)
    for b, (_, p, q, _) in enumerate(held):
        target[2 * b, [7, 9]] = p, 1 - p
        target[2 * b + 1, 11] = 1
        draft[b, [7, 9]] = q, 1 - q
    case = (target, None if lookup else draft, np.full(B, 7, np.int32), np.arange(B + 1, dtype=np.int32),
            np.float32([h[0] for h in held]), np.zeros(B, np.float32))
    tokens, accepted = (t.cpu().numpy() for t in mnb.mnb_verify(*_up(torch, dev, *case)))
    np.testing.assert_array_equal(accepted, [h[3] for h in held])
    want, want_n = orc.verify(*case)
    np.testing.assert_array_equal(accepted, want_n)
    np.testing.assert_array_equal(tokens, want)


@pytest.mark.parametrize("B,V", [(1, 700), (3, 128256), (30, 9001), (70, 33003), (600, 1500), (2, 270001)])
def test_verify_draws_from_the_target_where_nothing_is_left(env, B, V):  # noqa: F811
    """A rejected token whose row of the draft is nowhere below the target's: as one with a probability of 0 whose two rows are the same.
    Rows of zeros among them, from which nothing can be drawn, and rejections with something left."""
    mnb, torch, dev = env
    rng = np.random.default_rng(B + V)
    p = rng.random((2 * B, V), dtype=np.float32)
    p[rng.random((2 * B, V)) < 0.5] = 0
    p[:, 5] = 0
    p[:, 6] += 0.1
    p = (p / p.sum(-1, keepdims=True)).astype(np.float32)
    draft = p[::2].copy()
    kinds = np.arange(B) % 5
    for b in range(B):
        if kinds[b] == 1:
            draft[b] *= 1.0 + rng.random(V, dtype=np.float32)     # above the target wherever that is not 0
        elif kinds[b] == 2:
            p[2 * b] = 0
        elif kinds[b] == 3:
            draft[b] = np.roll(draft[b], 1)
        elif kinds[b] == 4:
            draft[b, V - 1], p[2 * b, V - 1] = 0, 2.0 ** -50      # a last element is left
    case = (p, draft, np.full(B, 5, np.int32), np.arange(B + 1, dtype=np.int32), np.full(B, 0.5, np.float32), rng.random(B, dtype=np.float32))
    tokens, accepted = (t.cpu().numpy() for t in mnb.mnb_verify(*_up(torch, dev, *case)))
    want, want_n = orc.verify(*case)
    np.testing.assert_array_equal(tokens, want)
    np.testing.assert_array_equal(accepted, want_n)
    assert not accepted.any() and (tokens[::2][kinds == 2] == -1).all() and (tokens[::2][kinds == 4] == V - 1).all()
    assert (p[2 * np.arange(B)[kinds < 2], tokens[::2][kinds < 2]] > 0).all()


def test_bindings_refuse_what_is_no_tensor(env):  # noqa: F811
    mnb, torch, dev = env
    h, i32 = dict(dtype=torch.float16, device=dev), dict(dtype=torch.int32, device=dev)
    down, up = torch.zeros(2, 8, 32, **h), torch.zeros(2, 12, 8, **h)
    pool, x, idx = mnb.MnbLoraPool(down, up), torch.zeros(3, 32, **h), torch.zeros(3, **i32)
    p, q = torch.zeros(5, 9, device=dev), torch.zeros(3, 9, device=dev)
    start, u, v = torch.zeros(3, **i32), torch.zeros(3, device=dev), torch.zeros(2, device=dev)
    for wrong in ([0, 0, 0], (1.0,), 7, np.zeros(3, np.float32)):
        cases = {
            "pool": lambda: mnb.mnb_lora(x, wrong, idx),
            "x": lambda: mnb.mnb_lora(wrong, pool, idx),
            "adapter": lambda: mnb.mnb_lora(x, pool, wrong),
            "base": lambda: mnb.mnb_lora(x, pool, idx, base=wrong),
            "out": lambda: mnb.mnb_lora(x, pool, idx, out=wrong),
            "ranks": lambda: mnb.MnbLoraPool(down, up, ranks=wrong),
            "scales": lambda: mnb.MnbLoraPool(down, up, scales=wrong),
            "workspace": lambda: mnb.mnb_lora(x, pool, idx, workspace=wrong),
            "logits": lambda: mnb.mnb_softmax(wrong),
            "temperature": lambda: mnb.mnb_softmax(x, temperature=wrong),
            "draft": lambda: mnb.mnb_verify(p, wrong, idx, start, u, v),
            "draft_start": lambda: mnb.mnb_verify(p, q, idx, wrong, u, v),
            "u_accept": lambda: mnb.mnb_verify(p, q, idx, start, wrong, v),
            "tokens": lambda: mnb.mnb_verify(p, q, idx, start, u, v, tokens=wrong),
            "accepted": lambda: mnb.mnb_verify(p, q, idx, start, u, v, accepted=wrong),
        }
        for name, call in cases.items():
            with pytest.raises(TypeError, match=f"^{name} must be a"):
                call()


def test_threads_on_streams_of_their_own(env):  # noqa: F811
    """Calls of one launch and of several, of six host threads that each have a stream: they may overlap as they like."""
    from concurrent.futures import ThreadPoolExecutor

    from tests.test_gpu_requests import _draft_case
    mnb, torch, dev = env
    rng = np.random.default_rng(17)
    kinds = [_up(torch, dev, *_draft_case(rng, B, V, 3, lookup)) for B, V, lookup in ((2, 5003, False), (7, 2000, True), (600, 900, True))]
    logits = [torch.randn(rows, V, device=dev) for rows, V in ((3, 1000), (2, 40000), (130, 20000))]
    forms = [lambda c=c: mnb.mnb_verify(*c) for c in kinds] + [lambda x=x: (mnb.mnb_softmax(x),) for x in logits]
    wants = [f() for f in forms]
    torch.cuda.synchronize()

    def work(f):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            outs = [f() for _ in range(100)]
        side.synchronize()
        return outs

    with ThreadPoolExecutor(len(forms)) as threads:
        results = list(threads.map(work, forms))
    for outs, want in zip(results, wants):
        assert all(torch.equal(a, b) for out in outs for a, b in zip(out, want))
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("rows,V", [(6, 9), (12, 1003), (6, 16377), (6, 70001), (60, 40001)])
def test_softmax_of_the_largest_temperatures(env, rows, V):  # noqa: F811
    """Logits as large as fp32 holds, at temperatures that bring them to an ordinary range, or beyond it to the same for all. (1 / T is
    subnormal from 2^126 on: up to 3 more last places of z, which the tolerance's 80 cover, as z is 6 at most.)"""
    mnb, torch, dev = env
    rng = np.random.default_rng(V)
    x = (rng.uniform(-1, 1, (rows, V)) * 3.4e38).astype(np.float32)
    x[1, :V // 2] = -3.4e38
    x[2] = np.sort(x[2])
    t = np.resize(np.float32([np.inf, 3.4e38, 1.5e38, 1.2e38, np.inf, 5e37]), rows)
    xd, td = _up(torch, dev, x, t)
    from tests.test_gpu_requests import _check_softmax
    got = mnb.mnb_softmax(xd, temperature=td)
    _check_softmax(got, x, t)
    np.testing.assert_allclose(got[0].cpu().numpy() * V, 1, rtol=(V / 512 + 100) * 2.0 ** -24)


def _runs(M, count):
    """Adapters of long runs of rows, and of single rows at the end."""
    adapter = (np.arange(M) * 3 // M % count).astype(np.int32)
    tail = min(M // 4, 40)
    adapter[M - tail:] = np.arange(tail) % count
    return adapter


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M", [20, 300, 1600, 2500])
def test_lora_bad_indices_wherever_they_are(env, M, dtype):  # noqa: F811
    """At the first row of a tile, whose adapter the clusters look at themselves, within runs and among single rows."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M)
    x, base, down, up, _, scales, _ = _lora_inputs(rng, M, 64, 136, 16, 4, dtype)
    adapter = _runs(M, 4)
    for first in (0, 128, 5 * 128, 64 * 3, M - 3, 7, M // 2 + 1):
        if first < M:
            adapter[first] = rng.choice(np.int32([4, 2 ** 31 - 1, 1 << 20]))
    if M > 1000:
        adapter[1024:1152] = 5  # a whole tile
    adapter[[3, M // 2]] = -2 ** 31, -7
    xd, bd, dd, ud, sd, ad = _up(torch, dev, x, base, down, up, scales, adapter)
    pool = mnb.MnbLoraPool(dd, ud, scales=sd)
    mnb.mnb_check_device_status()
    got = mnb.mnb_lora(xd, pool, ad, base=bd)
    with pytest.raises(mnb.MnbError, match="INVALID_ARG.*an adapter of mnb_lora"):
        mnb.mnb_check_device_status()
    _check_lora(got, x, base, down, up, None, scales, adapter, dtype)
    again = bd.clone()
    mnb.mnb_lora(xd, pool, ad, base=again, out=again)
    assert torch.equal(again, got)
    with pytest.raises(mnb.MnbError, match="INVALID_ARG"):
        mnb.mnb_check_device_status()
    none = mnb.mnb_lora(xd, pool, ad)
    _check_lora(none, x, None, down, up, None, scales, adapter, dtype)
    assert not none.cpu().numpy()[(adapter < 0) | (adapter > 3)].any()
    good = np.where(adapter > 3, -1, adapter)
    with pytest.raises(mnb.MnbError, match="INVALID_ARG"):
        mnb.mnb_check_device_status()
    assert torch.equal(mnb.mnb_lora(xd, pool, torch.from_numpy(good).to(dev), base=bd), got)
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("R", [16, 40, 128])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("M", [20, 300, 1600, 2500])
def test_lora_rows_of_any_size_beside_each_other(env, M, dtype, R):  # noqa: F811
    """Rows from the smallest to the largest keep their precision, and one with inf or NaN stays alone: in runs and among single rows."""
    mnb, torch, dev = env
    rng = np.random.default_rng(M + R)
    sizes = {"f16": [1e-7, 1e-3, 1.0, 1e4], "f32": [1e-30, 1e-3, 1.0, 1e30]}[dtype]
    x, base, down, up, _, scales, _ = _lora_inputs(rng, M, 96, 72, R, 3, dtype, without=0)
    adapter = _runs(M, 3)
    x = (x.astype(np.float64) * np.resize(sizes, M)[:, None]).astype(x.dtype)
    base *= 0
    if dtype == "f16":  # s beyond fp16
        down[0] *= np.float16(300)
        scales *= np.float32(1e-4)
    xd, bd, dd, ud, sd, ad = _up(torch, dev, x, base, down, up, scales, adapter)
    pool = mnb.MnbLoraPool(dd, ud, scales=sd)
    got = mnb.mnb_lora(xd, pool, ad, base=bd)
    _check_lora(got, x, base, down, up, None, scales, adapter, dtype)
    rows = [4, 9, M // 2, M // 2 + 1, M - 9, M - 2]
    bad = xd.clone()
    for i, r in enumerate(rows):
        bad[r, (3, 60, 95)[i % 3]] = (float("inf"), float("nan"), -float("inf"))[i // 2]
    odd = mnb.mnb_lora(bad, pool, ad, base=bd)
    keep = torch.ones(M, dtype=torch.bool, device=dev)
    keep[rows] = False
    assert torch.equal(odd[keep], got[keep])
    assert not torch.isfinite(odd[rows]).any()
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("R", [24, 64, 104, 128])
@pytest.mark.parametrize("tiles", [10, 19, 20, 23, 28, 33, 42, 56, 70, 140])
def test_lora_prompts_of_every_length(env, tiles, R):  # noqa: F811
    """As many tiles as make the tensor cores' kernel take clusters of 8, 7, 6, 5, 4, 3, 2 and 1 CTAs, whose shares of the exchange differ;
    the last tile is not full."""
    mnb, torch, dev = env
    M, K, N = tiles * 128 - 37, 272, 328
    rng = np.random.default_rng(tiles + R)
    x, base, down, up, _, scales, adapter = _lora_inputs(rng, M, K, N, R, 3, "f16", without=0)
    adapter[:] = np.arange(M) * 3 // M
    xd, bd, dd, ud, sd, ad = _up(torch, dev, x, base, down, up, scales, adapter)
    got = mnb.mnb_lora(xd, mnb.MnbLoraPool(dd, ud, scales=sd), ad, base=bd)
    assert mnb.mnb_last_variant() == "lora_tile_tcgen05"
    # s as two parts: what _check_lora allows for one is out of the way
    want, a, b = orc.lora(x, down, up, None, scales, adapter, base)
    tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2.0 ** -22 * a + (K / 8 + 2 * R + 64) * 2.0 ** -23 * b
    err = np.abs(got.cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())
    mnb.mnb_check_device_status()
