"""Numpy restatement of the paged 4-bit key/value cache and its attention (test infrastructure).

Written from the format's definition, element by element, apart from the library: where the
definition is fp32 with one rounding per operation (rotation, quantisation) the numpy
operations are the same IEEE ones, so results are compared bit for bit; attention is fp64.
"""
from __future__ import annotations

import numpy as np


def block_bytes(D: int, group: int) -> int:
    return 16 * D + 128 * (D // group)


def k_place(D: int, r: int, d: int) -> tuple[int, int]:
    """(byte in the block, bit) of K element d of row r."""
    w, t, n = d // 32, d % 32 // 8, d % 8
    if D == 256 and r % 2:
        w ^= 4
    return r * (D // 2) + (t * (D // 32) + w) * 4 + n // 2, n % 2 * 4


def v_place(D: int, r: int, d: int) -> tuple[int, int]:
    """(byte in the block, bit) of V element d of row r."""
    w, h, g, n = d // 64, d % 64 // 32, d % 32 // 4, d % 4
    x = {64: g // 2 % 2 * 8, 128: g % 2 * 8, 256: g % 2}[D]
    word = (g * 16 + (r ^ x)) * (D // 64) + w
    nib = 4 * h + n
    return 8 * D + word * 4 + nib // 2, nib % 2 * 4


def param_place(D: int, group: int, r: int, gi: int, is_v: bool) -> int:
    """Byte in the block of the (scale, offset) pair of group gi of row r."""
    return 16 * D + ((D // group if is_v else 0) * 16 + gi * 16 + r) * 4


def _maps(D):
    k = np.array([[k_place(D, r, d) for d in range(D)] for r in range(16)])
    v = np.array([[v_place(D, r, d) for d in range(D)] for r in range(16)])
    return k, v


def _address(slot, head, page_size, kv_heads, D, group):
    """(offset of the block, row) of a slot in the bytes of the whole cache."""
    bb = block_bytes(D, group)
    page, at = slot // page_size, slot % page_size
    return ((page * kv_heads + head) * (page_size // 16) + at // 16) * bb, at % 16


def rotate(x, positions, cos, sin, interleaved):
    """fp32 ``[T, H, D]``: each product and sum rounded once."""
    x = x.astype(np.float32).copy()
    if cos is None:
        return x
    half = cos.shape[1]
    c, s = cos[positions][:, None, :], sin[positions][:, None, :]
    a_at = np.arange(half) * 2 if interleaved else np.arange(half)
    b_at = a_at + 1 if interleaved else a_at + half
    a, b = x[..., a_at].copy(), x[..., b_at].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., a_at] = a * c - b * s
        x[..., b_at] = b * c + a * s
    return x


def quantise(x, group):
    """codes uint8 (shape of x), scale and offset fp16 ``[..., D / group]`` of fp32 x."""
    f = np.float32
    v = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    with np.errstate(all="ignore"):
        lo, hi = v.min(-1), v.max(-1)
        offset = np.clip(lo, f(-65504), f(65504)).astype(np.float16)
        scale = np.minimum((hi - lo) * (f(1) / f(15)), f(65504)).astype(np.float16)
        bad = ~np.isfinite(v).all(-1)
        offset[bad] = scale[bad] = np.nan
        s = scale.astype(f)
        inv = np.where(s == 0, f(0), f(1) / s)
        code = np.rint((v - offset.astype(f)[..., None]) * inv[..., None])
        code = np.where(bad[..., None], 0, np.clip(np.nan_to_num(code), 0, 15)).astype(np.uint8)
    return code.reshape(x.shape), scale, offset


def append(pages, k, v, positions, cos, sin, interleaved, slots, page_size, group):
    """Writes rotated, quantised K and V of fp32 ``[T, H, D]`` into ``pages`` (uint8, flat copy is returned)."""
    T, H, D = k.shape
    out = pages.reshape(-1).copy()
    km, vm = _maps(D)
    kc, ks, ko = quantise(rotate(k, positions, cos, sin, interleaved), group)
    vc, vs, vo = quantise(v.astype(np.float32), group)
    for t in range(T):
        if slots[t] < 0:
            continue
        for h in range(H):
            base, r = _address(int(slots[t]), h, page_size, H, D, group)
            for m, c in ((km[r], kc[t, h]), (vm[r], vc[t, h])):
                for (byte, bit), code in zip(m, c):
                    out[base + byte] = (int(out[base + byte]) & ~(15 << bit)) | (int(code) << bit)
            for is_v, (s, o) in enumerate(((ks, ko), (vs, vo))):
                for gi in range(D // group):
                    at = base + param_place(D, group, r, gi, bool(is_v))
                    out[at: at + 4] = np.array([s[t, h, gi], o[t, h, gi]], dtype="<f2").view(np.uint8)
    return out


def read(pages, slots, page_size, kv_heads, D, group, dtype=np.float32):
    """Values K, V ``[T, kv_heads, D]`` of slots (zeros for negative ones): offset + code * scale, in ``dtype``
    arithmetic (fp32: one rounding, as code * scale is exact)."""
    flat = pages.reshape(-1)
    km, vm = _maps(D)
    bb = block_bytes(D, group)
    slots = np.asarray(slots, dtype=np.int64)
    out = []
    for is_v, m in enumerate((km, vm)):
        y = np.zeros((len(slots), kv_heads, D), dtype=dtype)
        for h in range(kv_heads):
            s = np.maximum(slots, 0)
            base = ((s // page_size * kv_heads + h) * (page_size // 16) + s % page_size // 16) * bb
            r = s % 16
            code = flat[base[:, None] + m[r, :, 0]] >> m[r, :, 1] & 15
            gi = np.arange(D // group)
            at = base[:, None] + 16 * D + ((is_v * (D // group) + gi) * 16 + r[:, None]) * 4
            par = np.stack([flat[at + i] for i in range(4)], -1).view("<f2").astype(dtype)
            sc, of = (np.repeat(par[..., i], group, axis=-1) for i in (0, 1))
            y[:, h] = np.where(slots[:, None] < 0, 0, of + code.astype(dtype) * sc)
        out.append(y)
    return out


def attention(q, pages, q_start, kv_len, page_table, page_size, kv_heads, group, scale, causal, window):
    """fp64 out ``[T, Hq, D]`` and lse ``[T, Hq]``, with what scales rounding errors: sum_j p_j |v_j| ``[T, Hq, D]``
    and the largest scale * sum_d |q_d k_jd| over the keys a token sees, ``[T, Hq]``."""
    T, Hq, D = q.shape
    q = q.astype(np.float64)
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, reach = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    num_pages = pages.shape[0]
    G = Hq // kv_heads
    for b in range(len(kv_len)):
        a, e, n = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        if e <= a or n <= 0:
            continue
        j = np.arange(n)
        page = page_table[b][j // page_size].astype(np.int64)
        there = (page >= 0) & (page < num_pages)
        slot = np.where(there, page, 0) * page_size + j % page_size
        K, V = read(pages, slot, page_size, kv_heads, D, group, np.float64)
        for i in range(e - a):
            pos = n - (e - a) + i
            see = there.copy()
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            if not see.any():
                continue
            for h in range(Hq):
                k, v = K[see, h // G], V[see, h // G]
                s = scale * (k @ q[a + i, h])
                m = s.max()
                p = np.exp(s - m)
                out[a + i, h] = p @ v / p.sum()
                mag[a + i, h] = p @ np.abs(v) / p.sum()
                lse[a + i, h] = m + np.log(p.sum())
                reach[a + i, h] = abs(scale) * (np.abs(k) @ np.abs(q[a + i, h])).max()
    return out, lse, mag, reach
