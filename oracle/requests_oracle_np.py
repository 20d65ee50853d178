"""Oracle of what each request of a shared step has of its own: low-rank adapters, probabilities, verification of drafted
tokens.  fp64 numpy, and whole numbers where the operator is exact; no code of the library."""
from __future__ import annotations

import numpy as np


def lora(x, down, up, ranks, scales, adapter, base):
    """``(out, a, b)`` in fp64: the result, sum_r |up s| and sum_r |up| sum_k |down x| (each times |scale|), which error bounds
    are made of.  ``base`` may be None."""
    x, M, N = np.asarray(x, np.float64), len(adapter), up.shape[1]
    out = np.zeros((M, N)) if base is None else np.asarray(base, np.float64).copy()
    a, b = np.zeros((M, N)), np.zeros((M, N))
    for i in np.unique(adapter):
        if i < 0 or i >= len(down):
            continue
        r = down.shape[1] if ranks is None else int(np.clip(ranks[i], 0, down.shape[1]))
        c = 1.0 if scales is None else float(scales[i])
        d, u = down[i, :r].astype(np.float64), up[i, :, :r].astype(np.float64)
        rows = np.nonzero(adapter == i)[0]
        s = x[rows] @ d.T
        out[rows] += c * (s @ u.T)
        a[rows] = abs(c) * (np.abs(s) @ np.abs(u).T)
        b[rows] = abs(c) * ((np.abs(x[rows]) @ np.abs(d).T) @ np.abs(u).T)
    return out, a, b


def softmax(x, temperature):
    """fp64 probabilities; rows without a logit above -inf are 0."""
    x = np.asarray(x, np.float64)
    out = np.zeros(x.shape)
    for r, row in enumerate(x):
        t = 1.0 if temperature is None else float(temperature[r])
        top = row.max()
        if np.isnan(row).any() or np.isnan(t) or t < 0:
            out[r] = np.nan
        elif top == -np.inf:
            pass
        elif t == 0:
            out[r, int(np.argmax(row))] = 1
        elif top == np.inf:
            out[r] = np.nan
        else:
            e = np.exp((row - top) / t)
            out[r] = e / e.sum()
    return out


def _held(p):
    """Probabilities held to 0..1, as whole numbers of 2^-60."""
    p = np.nan_to_num(np.asarray(p, np.float64), nan=0.0, posinf=1.0, neginf=0.0).clip(0, 1)
    return [int(v) for v in np.rint(np.ldexp(p, 60))]


def verify(target, draft, draft_tokens, draft_start, u_accept, u_next):
    """``(tokens, accepted)`` by whole-number arithmetic."""
    B, V = len(draft_start) - 1, target.shape[1]
    tokens, accepted = np.full(len(target), -1, np.int32), np.zeros(B, np.int32)
    unit = lambda v: float(np.clip(np.nan_to_num(np.float64(v), nan=0.0), 0, 1))  # noqa: E731
    number = lambda v: min(unit(v), 1 - 2.0 ** -24)  # noqa: E731  a random number: below 1
    for b in range(B):
        s0, s1 = int(draft_start[b]), int(draft_start[b + 1])
        w = None
        for k in range(s0, s1):
            d = int(draft_tokens[k])
            p = target[k + b]
            if 0 <= d < V and number(u_accept[k]) * (1.0 if draft is None else unit(draft[k, d])) < unit(p[d]):
                tokens[k + b] = d
                accepted[b] += 1
                continue
            w = _held(p)
            if draft is None:
                rest = [0 if j == d else v for j, v in enumerate(w)]
            else:
                rest = [max(v - o, 0) for v, o in zip(w, _held(draft[k]))]
            if sum(rest):
                w = rest
            break
        if w is None:
            w = _held(target[s1 + b])
        total = sum(w)
        at = s0 + b + accepted[b]
        if total == 0:
            continue
        num, den = number(u_next[b]).as_integer_ratio()
        run = 0
        for j, v in enumerate(w):
            run += v
            if run * den > num * total:
                tokens[at] = j
                break
    return tokens, accepted
