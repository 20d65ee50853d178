"""Append and read of many tokens: above 304 a block takes a token's heads in passes (several in flight), then its next
token, and the read takes four tokens a lane.  Bit for bit against the oracle."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import kv4_oracle_np as orc
from tests.test_gpu_kv4 import NP, _tables, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,group,ps,Hq,Hk,T,dtype,rot,interleaved,in_place", [
    (128, 128, 16, 8, 2, 305, "f16", 128, False, False),
    (128, 32, 64, 48, 9, 643, "f16", 128, False, True),       # 3 + 2 + 2 passes, four in flight
    (128, 64, 16, 20, 9, 1301, "f32", 64, True, False),       # 2 + 2 + 2 passes, two in flight
    (64, 64, 32, 14, 2, 1301, "f16", 32, True, True),
    (64, 32, 16, 33, 1, 1300, "f32", 64, False, True),
    (256, 128, 128, 16, 2, 1303, "f16", 256, False, False),
    (256, 32, 16, 17, 5, 642, "f32", 96, False, True),
    (256, 64, 48, 9, 5, 306, "f16", 256, True, True),
    (128, 128, 16, 0, 3, 1302, "f16", 0, False, False),
])
def test_many_tokens_are_bit_exact(env, D, group, ps, Hq, Hk, T, dtype, rot, interleaved, in_place):  # noqa: F811
    """With padding (slots of -1) and, where tokens have positions, positions and slots out of range anywhere in a block's run."""
    mnb, torch, dev = env
    rng = np.random.default_rng(D + T)
    x = (rng.standard_normal((T, (Hq + 2 * Hk), D)) * rng.choice([0.01, 1, 50], (T, 1, 1))).astype(NP[dtype])
    q0, k0, v0 = x[:, :Hq], x[:, Hq: Hq + Hk], x[:, Hq + Hk:]
    k0[T - 1, 0, :group], v0[T // 2, 0, :group] = 0.25, 0.0  # constant groups
    v0[T - 2, -1, 5] = np.inf
    pages = -(-T // ps) + 2
    slots = rng.permutation(pages * ps)[:T].astype(np.int64)
    slots[[3, T // 3, T - 5]] = -1
    pos = rng.integers(0, 300, T).astype(np.int32)
    bad = np.zeros(T, bool)
    beyond = np.zeros(T, bool)
    beyond[[7, T - 3]] = True
    if rot:
        bad[[0, 11, T // 2 + 1, T - 4]] = True
    cos, sin = _tables(rng, 300, rot) if rot else (None, None)
    given_pos, given_slots = pos.copy(), slots.copy()
    given_pos[bad] = rng.choice([-1, 300, 2 ** 31 - 1, -2 ** 31], bad.sum())
    given_slots[beyond] = rng.choice([pages * ps, 2 ** 40], beyond.sum())
    stored = np.where(bad | beyond, -1, slots)
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    start = rng.integers(0, 256, (pages, Hk, ps // 16 * orc.block_bytes(D, group))).astype(np.uint8)
    cache = mnb.MnbKv4Cache(up(start), ps, D, group)
    fused = up(x)
    q = (up(q0) if in_place else fused[:, :Hq]) if Hq else None
    got_q = mnb.mnb_kv4_append(cache, fused[:, Hq: Hq + Hk], fused[:, Hq + Hk:], up(given_slots), q=q, positions=up(given_pos),
                               cos=up(cos), sin=up(sin), interleaved=interleaved, q_out=q if in_place else None)
    with pytest.raises(mnb.MnbError):  # the index bit, for slots beyond the cache
        mnb.mnb_check_device_status()
    f = np.float32
    want = orc.append(start, k0.astype(f), v0.astype(f), pos, cos, sin, interleaved, stored, ps, group)
    got = cache.pages.cpu().numpy().reshape(-1)
    diff = got != want
    if diff.any():  # parameters that are NaN may differ in their bits
        a, b = got.view("<f2"), want.view("<f2")
        assert not (diff & ~np.repeat(np.isnan(a) & np.isnan(b), 2)).any()
        assert (np.nonzero(diff)[0] % orc.block_bytes(D, group) >= 16 * D).all()
    if Hq:
        assert got_q is q or not in_place
        with np.errstate(over="ignore"):
            want_q = orc.rotate(q0, pos, cos, sin, interleaved).astype(NP[dtype])
        want_q[bad] = 0
        np.testing.assert_array_equal(got_q.cpu().numpy(), want_q)
    for read_dtype in ("f16", "f32"):
        at = rng.permutation(T)
        rk, rv = mnb.mnb_kv4_read(cache, up(stored[at]), dtype=torch.float16 if read_dtype == "f16" else torch.float32)
        with np.errstate(over="ignore", invalid="ignore"):
            wk, wv = (a.astype(NP[read_dtype]) for a in orc.read(want, stored[at], ps, Hk, D, group))
        np.testing.assert_array_equal(rk.cpu().numpy(), wk)
        np.testing.assert_array_equal(rv.cpu().numpy(), wv)
    mnb.mnb_check_device_status()
    mnb.mnb_kv4_read(cache, up(given_slots))
    with pytest.raises(mnb.MnbError):
        mnb.mnb_check_device_status()
