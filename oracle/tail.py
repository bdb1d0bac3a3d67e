"""Float64 references of the tail of a step (test infrastructure only): low-rank
adapters beside a projection, the residual RMS norm, and log probabilities over
the head's logits, each with the error scale that its checks need.

The definitions are the ones that include/q4nx.h states for q4nx_lora_add,
q4nx_add_rmsnorm and q4nx_token_logprobs; every value is formed row by row.
"""
from __future__ import annotations

import math

import numpy as np


def lora_ref(x, A, B, scale, ids, base, ranks=None):
    """y[m] = base[m] + scale[e] B_e (A_e x[m]) and its error scale, both float64.

    x [M, K], A [E, R, K], B [E, N, R], base [M, N] as floats; an id outside
    [0, E) adds nothing.  The second result is sum |scale b| sum |a x|.
    """
    y = np.asarray(base, dtype=np.float64).copy()
    mag = np.zeros_like(y)
    E, R, _ = A.shape
    for m, e in enumerate(ids):
        if not 0 <= e < E:
            continue
        r = R if ranks is None else min(max(int(ranks[e]), 0), R)
        a, b = A[e, :r].astype(np.float64), B[e, :, :r].astype(np.float64)
        s, v = float(scale[e]), x[m].astype(np.float64)
        y[m] += s * (b @ (a @ v))
        mag[m] = abs(s) * (np.abs(b) @ (np.abs(a) @ np.abs(v)))
    return y, mag


def add_rmsnorm_ref(y, r, w, eps):
    """(s, x) of s = y + r (y may be None) and x = s w / sqrt(mean s^2 + eps), float64."""
    s = np.asarray(r, dtype=np.float64) + (0.0 if y is None else np.asarray(y, dtype=np.float64))
    return s, s * np.asarray(w, dtype=np.float64) / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)


def token_logprobs_ref(y, tokens, k):
    """Of one row of logits: (logp of tokens, entropy, top ids, top logps, spread).

    NaN and -inf have probability 0; several +inf share it all.  The sums are
    math.fsum's.  spread = sum p |y - max|, the scale of an exponent's error.
    """
    y = np.asarray(y, dtype=np.float32).astype(np.float64)
    n = len(y)
    alive = [i for i in range(n) if y[i] > -math.inf]        # False for NaN
    nan = math.nan
    if not alive:
        return [nan] * len(tokens), nan, [-1] * k, [nan] * k, 0.0
    m = max(y[i] for i in alive)
    d = {i: 0.0 if y[i] == m else y[i] - m for i in alive}
    first = next(i for i in alive if d[i] == 0.0)
    e = {i: math.exp(d[i]) for i in alive}
    rest = math.fsum(v for i, v in e.items() if i != first)
    lz = math.log1p(rest)
    H = lz - math.fsum(e[i] * d[i] for i in alive if e[i] > 0) / (1 + rest)
    spread = math.fsum(-e[i] * d[i] for i in alive if e[i] > 0) / (1 + rest)
    lp = [nan if not 0 <= t < n else d[t] - lz if t in d else -math.inf for t in tokens]
    top = sorted(alive, key=lambda i: (-y[i], i))[:k]
    pad = k - len(top)
    return lp, H, top + [-1] * pad, [d[i] - lz for i in top] + [nan] * pad, spread
