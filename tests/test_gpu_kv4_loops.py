"""Attention over the paged 4-bit cache where a CTA takes many key tiles and several pieces of work.

The kernels cut all key tiles of a call into one range for each CTA, so short calls give a CTA one tile. Here the
shares are worked out first and each test asserts that its shape reaches the loops: later tiles of a piece,
reuse of every ring, the change from one piece to the next. Results are compared with fp64 on the GPU, from the values
that the cache holds (which the append and read tests compare bit for bit), within the tolerances of
``test_gpu_kv4``, and with a second run bit for bit.
"""
from __future__ import annotations

from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

from tests.test_gpu_kv4 import _check, env  # noqa: F401

pytestmark = pytest.mark.gpu

STREAM_CTAS = 4  # an SM, at most


def _shares(lens, Hk, G, rows, keys, cost, ctas, causal=True, window=0):
    """Key tiles of each piece of each CTA: [[tiles, ..], ..]; `rows` and `keys` of a tile, `cost` of a piece in tiles."""
    pieces = []
    for q_len, n in lens:
        for rt in range(-(-q_len * G // rows)):
            first, last = rt * rows // G, min(q_len - 1, (rt * rows + rows - 1) // G)
            hi = min(n, n - q_len + last + 1) if causal else n
            lo = max(0, n - q_len + first - window + 1) if window else 0
            t0 = lo // keys
            pieces += [max(t0 + 1, -(-max(hi, 0) // keys)) - t0] * Hk
    total = sum(p + cost for p in pieces)
    ctas = min(ctas, total)
    out, at, used = [], 0, 0  # piece, units of it that are taken
    for i in range(ctas):
        left = total // ctas + (1 if i < total % ctas else 0)
        own = []
        while left:
            take = min(left, pieces[at] + cost - used)
            tiles = max(0, used + take - cost) - max(0, used - cost)
            if tiles:
                own.append(tiles)
            left -= take
            used += take
            if used == pieces[at] + cost:
                at, used = at + 1, 0
        out.append(own)
    return out


def _reaches(shares, tiles, pieces, part=0.3):
    """Most CTAs have `tiles` key tiles in all, and this part of them at least `pieces` pieces."""
    assert np.median([sum(s) for s in shares]) >= tiles, np.median([sum(s) for s in shares])
    assert np.mean([len(s) >= pieces for s in shares]) >= part, np.mean([len(s) >= pieces for s in shares])
    assert max(max(s, default=0) for s in shares) >= 3


class Filled:
    """A cache with `lens` sequences of random keys and values, pages in random order, times ksize(j) and vsize(j)."""

    def __init__(self, env, seed, D, group, ps, Hk, lens, ksize=None, vsize=None):
        mnb, torch, dev = env
        self.env, self.D, self.Hk, self.lens = env, D, Hk, lens
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        need = [-(-n // ps) for _, n in lens]
        self.cache = mnb.mnb_kv4_cache_alloc(sum(need) + 2, ps, Hk, D, group, dev)
        order = torch.randperm(sum(need) + 2, generator=gen, device=dev)
        table = torch.zeros((len(lens), max(need)), dtype=torch.int64, device=dev)
        self.slots, self.kv, at = [], [], 0
        for b, (_, n) in enumerate(lens):
            table[b, : need[b]] = order[at: at + need[b]]
            at += need[b]
            j = torch.arange(n, device=dev)
            self.slots.append(table[b, j // ps] * ps + j % ps)
            kv = [torch.randn((n, Hk, D), generator=gen, device=dev) for _ in range(2)]
            for x, size in zip(kv, (ksize, vsize)):
                if size is not None:
                    x *= size(j.float())[:, None, None]
            if n:
                mnb.mnb_kv4_append(self.cache, kv[0], kv[1], self.slots[b])
            self.kv.append(kv)
        self.table = table.int()
        self.kv_len = torch.tensor([n for _, n in lens], dtype=torch.int32, device=dev)
        self.start = torch.tensor(np.cumsum([0] + [a for a, _ in lens]), dtype=torch.int32, device=dev)
        self.gen = gen

    def queries(self, G, dtype, size=1.0):
        _, torch, dev = self.env
        T = sum(a for a, _ in self.lens)
        q = torch.randn((T, self.Hk * G, self.D), generator=self.gen, device=dev) * size
        return q.to(torch.float16 if dtype == "f16" else torch.float32)

    def store(self, b):
        """Appends sequence b again, after changes of kv[b]."""
        self.env[0].mnb_kv4_append(self.cache, *self.kv[b], self.slots[b])

    def attend(self, q, scale, causal=True, window=0, lse=None):
        return self.env[0].mnb_kv4_attention(q, self.cache, self.start, self.kv_len, self.table, scale, causal=causal,
                                             window=window, lse=lse)

    def want(self, q, scale, causal=True, window=0, held=None):
        """As the oracle's `attention`: out, lse, sum_j p_j |v_j|, largest scale * sum_d |q_d k_jd|, fp64.  With held =
        (half step, smallest half step of p relative to the row's largest, whether groups share it, largest |code| in a
        product) also the bound of what holding p_j * V scale in fewer bits does to each element."""
        mnb, torch, dev = self.env
        T, Hq, D = q.shape
        G = Hq // self.Hk
        f64 = torch.float64
        out, mag = torch.zeros((T, Hq, D), dtype=f64, device=dev), torch.zeros((T, Hq, D), dtype=f64, device=dev)
        lse = torch.full((T, Hq), float("-inf"), dtype=f64, device=dev)
        reach = torch.zeros((T, Hq), dtype=f64, device=dev)
        bound = torch.zeros((T, Hq, D), dtype=f64, device=dev)
        for b, (q_len, n) in enumerate(self.lens):
            if not q_len or not n:
                continue
            a = int(self.start[b])
            K, V = (x.double() for x in mnb.mnb_kv4_read(self.cache, self.slots[b], dtype=torch.float32))
            j, pos = torch.arange(n, device=dev), n - q_len + torch.arange(q_len, device=dev)
            hide = torch.zeros((q_len, n), dtype=torch.bool, device=dev)
            if causal:
                hide |= j[None] > pos[:, None]
            if window:
                hide |= j[None] <= pos[:, None] - window
            for h in range(Hq):
                x, k, v = q[a: a + q_len, h].double(), K[:, h // G], V[:, h // G]
                s = (x @ k.T * scale).masked_fill(hide, float("-inf"))
                l = s.logsumexp(-1)
                p = torch.exp(s - torch.where(torch.isinf(l), torch.zeros_like(l), l)[:, None])
                out[a: a + q_len, h], mag[a: a + q_len, h] = p @ v, p @ v.abs()
                lse[a: a + q_len, h] = l
                reach[a: a + q_len, h] = (x.abs() @ k.abs().T * abs(scale)).masked_fill(hide, 0.0).amax(-1)
                if held:
                    half, least, shared, code = held
                    g = self.cache.group_size
                    step = (v.view(n, -1, g).amax(-1) - v.view(n, -1, g).amin(-1)) / 15  # V scales, up to their rounding
                    for i in range(D // g):
                        product = p * step[:, i]
                        floor = p.amax(-1, keepdim=True) * least * (step.max() if shared else step[:, i])
                        lost = torch.maximum(half * product, torch.minimum(product, floor))
                        bound[a: a + q_len, h, i * g: (i + 1) * g] = code * lost.sum(-1, keepdim=True)
        return tuple(t.cpu().numpy() for t in (out, lse, mag, reach) + ((bound,) if held else ()))

    def check(self, q, dtype, scale, causal=True, window=0):
        mnb, torch, dev = self.env
        lse = torch.full(q.shape[:2], 7.0, device=dev)
        scale = float(np.float32(scale))
        out = self.attend(q, scale, causal, window, lse)
        variant = mnb.mnb_last_variant()
        for _ in range(3):
            assert torch.equal(out, self.attend(q, scale, causal, window)), variant
        mnb.mnb_check_device_status()
        _check(out, lse, self.want(q, scale, causal, window), dtype, variant)
        return out, variant


def _sms(env):
    return env[1].cuda.get_device_properties(0).multi_processor_count


PROMPTS = [(700, 3000), (900, 3000)]
DRAFTS = [(16 - i % 5, 500 + 137 * i) for i in range(24)]


@pytest.mark.parametrize("D,group,ps,Hk,G,lens,causal,window", [
    (128, 128, 16, 8, 4, PROMPTS, True, 0),
    (128, 32, 64, 8, 4, PROMPTS, True, 700),
    (128, 64, 16, 4, 7, [(511, 511), (700, 1900), (40, 2500), (900, 901)], True, 0),
    (128, 128, 32, 8, 4, [(300, 1500), (420, 900), (256, 2000)], False, 0),
    (64, 64, 16, 8, 4, PROMPTS, True, 0),
    (64, 32, 128, 6, 5, [(650, 2222), (800, 3100)], True, 0),
    (128, 64, 16, 8, 4, DRAFTS, True, 0),
])
def test_prompts_of_several_pieces(env, D, group, ps, Hk, G, lens, causal, window):  # noqa: F811
    """tcgen05 kernel: a row tile's four warps leave a piece and enter the next one each in its own time."""
    shares = _shares(lens, Hk, G, 256, 128, 3, min(160, _sms(env)), causal, window)
    _reaches(shares, 8, 2)
    f = Filled(env, D + G, D, group, ps, Hk, lens)
    _, variant = f.check(f.queries(G, "f16"), "f16", D ** -0.5, causal, window)
    assert variant == "kv4_tile_tcgen05"


def _check_parts(out, want, dtype, rows, parts, what):
    """The norm bound of `test_gpu_kv4` for these rows' elements of each part of the head by itself (their scores must
    be ordinary), and its bound for each element."""
    ref, _, mag, reach = (x[rows] for x in want)
    got = out.double().cpu().numpy()[rows]
    assert reach.max() < 40
    _check(out[rows], None, (ref, None, mag, reach), dtype, what)
    u = 2.0 ** -11 if dtype == "f16" else 2.0 ** -20
    for part in np.split(np.arange(ref.shape[-1]), parts):
        a, b = got[..., part], ref[..., part]
        bound = 2 * u * np.linalg.norm(b) + 2.0 ** -25 * np.sqrt(b.size) if dtype == "f16" else 4 * u * np.linalg.norm(b)
        assert np.linalg.norm(a - b) <= bound, (what, part[0], np.linalg.norm(a - b) / np.linalg.norm(b))


# (query tokens, keys), window, the odd token: the tcgen05 kernel, then the streaming one
UNEVEN = [((300, 300), 0, 220), ((200, 450), 100, 340), ((3, 300), 0, 298), ((1, 300), 100, 190)]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("factor", [100, 1000, 10000])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("lens,window,odd", UNEVEN)
def test_a_token_of_another_size(env, D, group, lens, window, odd, factor, dtype):  # noqa: F811
    """One token's key or value is larger than all others of its tile: rows that don't see it are as exact as without it."""
    q_len, n = lens
    pos = n - q_len + np.arange(q_len)
    hidden = (pos < odd) | ((window > 0) & (pos - window >= odd))
    for which in (0, 1):
        f = Filled(env, D + group, D, group, 16, 2, [lens], None, lambda j: 0.05 + 0 * j)
        f.kv[0][which][odd] *= factor
        f.store(0)
        q, scale = f.queries(4, dtype), float(np.float32(D ** -0.5))
        out = f.attend(q, scale, True, window)
        assert env[0].mnb_last_variant() == ("kv4_tile_tcgen05" if q_len > 100 and dtype == "f16" else env[0].mnb_last_variant())
        want = f.want(q, scale, True, window)
        _check_parts(out, want, dtype, hidden, 1, (which, factor))
        if which == 1:  # with a key of ordinary size the rows that do see it are ordinary too
            _check(out, None, want, dtype, "all rows")
    env[0].mnb_check_device_status()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("factor", [100, 1000, 10000])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 64)])
@pytest.mark.parametrize("lens,window,odd", UNEVEN)
def test_groups_of_another_size(env, D, group, lens, window, odd, factor, dtype):  # noqa: F811
    """The first group of every key and value is larger than the others, and q has zeros there: scores are ordinary, and
    the other groups' results are as exact as without it."""
    f = Filled(env, D + group, D, group, 16, 2, [lens], None, lambda j: 0.05 + 0 * j)
    for x in f.kv[0]:
        x[..., :group] *= factor
    f.store(0)
    q, scale = f.queries(4, dtype), float(np.float32(D ** -0.5))
    q[..., :group] = 0
    out = f.attend(q, scale, True, window)
    _check_parts(out, f.want(q, scale, True, window), dtype, np.ones(lens[0], bool), D // group, factor)
    env[0].mnb_check_device_status()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D,group,lens,window", [(64, 64, (1, 300), 100), (128, 128, (1, 300), 100), (128, 64, (3, 300), 100),
                                                 (256, 128, (1, 300), 100), (128, 64, (90, 300), 100)])
def test_a_value_that_no_row_sees(env, D, group, lens, window, dtype):  # noqa: F811
    """It lies in a key tile that is read, below the window, and is larger than the others by almost all of fp16's range."""
    f = Filled(env, D, D, group, 16, 2, [lens], None, lambda j: 0.001 + 0 * j)
    q, scale = f.queries(4, dtype), float(np.float32(D ** -0.5))
    clean = f.attend(q, scale, True, window)
    first = lens[1] - lens[0] - window + 1
    f.kv[0][1][first - 3] = 40000.0 * f.kv[0][1][first - 3].sign()
    f.store(0)
    out = f.attend(q, scale, True, window)
    _check(out, None, f.want(q, scale, True, window), dtype, env[0].mnb_last_variant())
    if env[0].mnb_last_variant() != "kv4_tile_tcgen05":
        assert env[1].equal(out, clean)
    env[0].mnb_check_device_status()


RAGGED = [8192, 1, 7000, 0, 3333, 17, 5000, 8191, 128, 129, 6100, 2049, 4096, 7777, 900, 8000, 6500, 30, 5555, 7123, 4444,
          8188, 2500, 6001, 7400, 3000, 8100]


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("tokens", [1, 4])
@pytest.mark.parametrize("D,group,ps,Hk,G,window", [
    (64, 32, 16, 8, 4, 0), (64, 64, 64, 7, 3, 5000), (128, 32, 32, 8, 4, 0), (128, 64, 128, 8, 4, 6000), (128, 128, 16, 8, 4, 0),
    (256, 32, 16, 8, 4, 0), (256, 64, 48, 7, 2, 0), (256, 128, 16, 8, 4, 4500)])
def test_decode_and_verify_of_many_tiles(env, D, group, ps, Hk, G, window, tokens, dtype):  # noqa: F811
    """Streaming kernel: several steps of every warp, rings in use again, one piece after the other, ragged."""
    lens = [(min(n, 1 + i % tokens), n) if n else (1, 0) for i, n in enumerate(RAGGED)]
    average = -(-sum(a for a, _ in lens) // len(lens)) * G
    rows = 8 if average <= 8 else 16
    keys = 64 if D == 256 and rows == 16 else 128
    _reaches(_shares(lens, Hk, G, rows, keys, 3, STREAM_CTAS * _sms(env), True, window), 7, 2, 0.15)
    f = Filled(env, D + G + tokens, D, group, ps, Hk, lens)
    _, variant = f.check(f.queries(G, dtype), dtype, D ** -0.5, True, window)
    assert variant == f"kv4_stream_{dtype}_rows{rows}"


# keys that grow make every row's reference rise over sums that it has; values of 0.003 to 3000 in waves of a few tiles
LONG = {"decode": [(1, 8000), (1, 8192), (1, 5000)] * 6, "verify": [(4, 8000), (3, 8192), (4, 6000)] * 6,
        "prompts": [(700, 3000), (900, 2900)]}


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("form", LONG)
def test_sizes_that_change_along_a_sequence(env, form, D, group, dtype):  # noqa: F811
    lens, Hk, G = LONG[form], 8, 4
    tiles = form == "prompts" and dtype == "f16" and D <= 128
    rows, keys, ctas = (256, 128, _sms(env)) if tiles else (8 if form == "decode" else 16, 128, STREAM_CTAS * _sms(env))
    _reaches(_shares(lens, Hk, G, rows, keys, 3, ctas), 5, 2, 0.15)
    f = Filled(env, D, D, group, 16, Hk, lens, lambda j: 0.05 + 3.5 * (j / 8192) ** 0.5,
               lambda j: 3 * 10 ** (3 * env[1].sin(j / 150)))
    _, variant = f.check(f.queries(G, dtype), dtype, D ** -0.5)
    assert (variant == "kv4_tile_tcgen05") == tiles


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("form", LONG)
def test_one_key_takes_all_among_values_of_many_sizes(env, form, D, group, dtype):  # noqa: F811
    """Scores so far apart that a row is one or two keys, whose elements may be near zero while the parts that make them up
    are not.  The bound of an element is `_check`'s and what the held probabilities add to it:

    * streaming, fp16: p * V scale is rounded to fp16, to 2^-12 of it or, among the subnormals, to 2^-25 where the row's largest
      p times the largest scale is 2^8 at least; it multiplies |c - 8| <= 8;
    * streaming, fp32: two fp16 make it 2^-23, and the scale is that of its own 16 keys (within 2 here);
    * tcgen05: p itself, where values beyond 2^11 (16 V scales; up to 2^15 here) take up to 2^5 from it; it multiplies up to 16 scales.
    """
    lens, Hk, G = LONG[form], 8, 4
    tiles = form == "prompts" and dtype == "f16" and D <= 128
    f = Filled(env, D, D, group, 16, Hk, lens, lambda j: 0.05 + 15 * (j / 8192) ** 0.5,
               lambda j: 3 * 10 ** (3 * env[1].sin(j / 150)))
    q, scale = f.queries(G, dtype), float(np.float32(D ** -0.5))
    held = (2.0 ** -12, 2.0 ** -28, True, 16) if tiles else (2.0 ** -12, 2.0 ** -33, True, 8) if dtype == "f16" else (
        2.0 ** -23, 2.0 ** -32, False, 8)
    out = f.attend(q, scale).double().cpu().numpy()
    ref, _, mag, reach, bound = f.want(q, scale, held=held)
    u = 2.0 ** -11 if dtype == "f16" else 2.0 ** -20
    tol = 4 * u * (np.abs(ref) + mag) + np.expm1(2 * u * reach[..., None]) * (mag + bound) + bound
    if dtype == "f16":
        tol = tol + 2.0 ** -24
    assert reach.max() > 60 and np.isfinite(out).all()
    assert (np.abs(out - ref) <= tol).all(), np.max(np.abs(out - ref) / tol)
    env[0].mnb_check_device_status()


@pytest.mark.parametrize("form,dtype", [(form, dtype) for form in LONG for dtype in ("f16", "f32")])
def test_a_nan_deep_in_a_long_sequence(env, form, dtype):  # noqa: F811
    """A value of sequence 1 that is not finite: rows that see it get NaN in its group, all others what they had; a row of q
    with NaN harms itself alone."""
    _, torch, dev = env
    lens, Hk, G, D, group = LONG[form], 8, 4, 128, 32
    f = Filled(env, 5, D, group, 16, Hk, lens)
    q, scale = f.queries(G, dtype), float(np.float32(D ** -0.5))
    clean = f.attend(q, scale)
    at = lens[1][1] - (400 if form == "prompts" else 2 if form == "verify" else 3000)
    f.kv[1][1][at, 3, 40] = float("inf")
    f.store(1)
    q2 = q.clone()
    q2[0, 5, 7] = float("nan")
    got = f.attend(q2, scale)
    a, (q_len, n) = int(f.start[1]), lens[1]
    sees = torch.arange(n - q_len, n, device=dev) >= at
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[a: a + q_len, 3 * G: 4 * G, 32:64] = sees[:, None, None]
    assert 0 < int(sees.sum()) and (form == "decode" or int(sees.sum()) < q_len)
    hit[0, 5] = True
    assert torch.isnan(got[hit]).all()
    assert torch.equal(got[~hit], clean[~hit])
    env[0].mnb_check_device_status()


@pytest.mark.parametrize("dtype,D", [("f16", 128), ("f16", 256), ("f32", 128)])
@pytest.mark.parametrize("chunk", [40, 512, 1500])
def test_a_chunk_beside_decode_tokens(env, chunk, dtype, D):  # noqa: F811
    """A serving batch: one kernel takes all of it, by the average of rows."""
    lens = [(1, 300 + 61 * i) for i in range(31)] + [(chunk, 3000)] + [(1, 4000 - 77 * i) for i in range(32)]
    f = Filled(env, D + chunk, D, 128, 16, 4, lens)
    _, variant = f.check(f.queries(4, dtype), dtype, D ** -0.5)
    assert (variant == "kv4_tile_tcgen05") == (chunk == 1500 and dtype == "f16" and D == 128)


@pytest.mark.parametrize("kept", [True, False])
def test_threads_share_a_workspace(env, kept):  # noqa: F811
    """Calls of four host threads on one stream with one workspace: each is two launches, which stay together."""
    mnb, torch, dev = env
    need, forms = 0, []
    for i, lens in enumerate(([(1, 3000), (1, 700)], [(4, 2500)], [(90, 1500)], [(1, 4000)])):
        f = Filled(env, i, 128, 64, 16, 2, lens)
        q = f.queries(4, "f16")
        forms.append((f, q, f.attend(q, 0.09)))
        need = max(need, mnb.mnb_kv4_attention_workspace_bytes(q.shape[0], len(lens), 8, 2, 128))
    torch.cuda.synchronize()
    shared = None if kept else torch.empty(need, dtype=torch.uint8, device=dev)

    def calls(i):
        f, q, want = forms[i]
        outs = [mnb.mnb_kv4_attention(q, f.cache, f.start, f.kv_len, f.table, 0.09, workspace=shared) for _ in range(200)]
        return all(torch.equal(o, want) for o in outs)

    with ThreadPoolExecutor(4) as pool:
        assert all(pool.map(calls, range(4)))
    mnb.mnb_check_device_status()


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("form", LONG)
def test_strided_q_and_programmatic_launch_of_several_pieces(env, form, D, dtype):  # noqa: F811
    """q as a view of a fused product whose other columns are NaN, calls launched before the last has ended: as with q by
    itself, one call after the other."""
    mnb, torch, dev = env
    f = Filled(env, D, D, 64, 16, 4, LONG[form])
    q = f.queries(5, dtype)
    T = q.shape[0]
    plain = f.attend(q, 0.07)
    torch.cuda.synchronize()
    fused = torch.full((T, 28 * D), float("nan"), dtype=q.dtype, device=dev)
    view = fused[:, 4 * D: 24 * D].view(T, 20, D)
    mnb.mnb_set_programmatic_launch(True)
    try:
        view.copy_(q)
        outs = [f.attend(view, 0.07) for _ in range(6)]
    finally:
        mnb.mnb_set_programmatic_launch(False)
    torch.cuda.synchronize()
    assert torch.isfinite(plain).all() and all(torch.equal(o, plain) for o in outs)
    mnb.mnb_check_device_status()
