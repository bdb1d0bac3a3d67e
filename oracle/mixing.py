"""Float64 references of the token mixing of a layer (test infrastructure only):
rotation and the paged cache, attention behind a shared prefix, and linear
attention with decay, each with the magnitudes that its checks need.

The definitions are the ones that include/q4nx.h states for q4nx_kv_append,
q4nx_attention and q4nx_linear_attn; every row is formed by itself.
"""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# the cache's layout: logical [pages, heads, tokens, dim] and back
# ---------------------------------------------------------------------------
def pack_k(x):
    P, H, T, D = x.shape
    return np.ascontiguousarray(x.reshape(P, H, T // 16, 16, D // 8, 8).transpose(0, 1, 2, 4, 3, 5))


def unpack_k(x):
    P, H, a, b, _, _ = x.shape
    return np.ascontiguousarray(x.transpose(0, 1, 2, 4, 3, 5)).reshape(P, H, 16 * a, 8 * b)


def pack_v(x):
    P, H, T, D = x.shape
    return np.ascontiguousarray(x.reshape(P, H, T // 8, 8, D).transpose(0, 1, 2, 4, 3))


def unpack_v(x):
    P, H, a, D, _ = x.shape
    return np.ascontiguousarray(x.transpose(0, 1, 2, 4, 3)).reshape(P, H, 8 * a, D)


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------
def rope_ref(x, pos, inv_freq, dim, interleaved):
    """x [M, heads, D] turned by pos[m] * inv_freq[i] over its first dim dimensions, and the
    magnitude |a| + |b| of each result; float64."""
    x = np.asarray(x, dtype=np.float64)
    y, mag = x.copy(), np.abs(x)
    if dim:
        t = np.asarray(pos, dtype=np.int64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None, :]
        c, s = np.cos(t)[:, None, :], np.sin(t)[:, None, :]
        ia = np.arange(dim // 2) * 2 if interleaved else np.arange(dim // 2)
        ib = ia + 1 if interleaved else ia + dim // 2
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attention_ref(q, k, v, scale):
    """One row and head over the keys that it sees: (out, lse, sum p |v|, the exponents' error scale).

    q [D], k and v [n, D]; a score of -inf counts as unseen.  The error scale is
    max_j |scale| sum_i |q_i k_ji| + max |s_j| over the keys seen.
    """
    D = q.shape[0]
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    if k.shape[0] == 0:
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    with np.errstate(invalid="ignore"):
        s = scale * (k @ q)
    seen = ~(s == -np.inf)
    if not seen.any():
        return np.zeros(D), -np.inf, np.zeros(D), 0.0
    s, k, v = s[seen], k[seen], v[seen]
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    p /= l
    off = abs(scale) * (np.abs(k) @ np.abs(q)).max() + np.abs(s).max()
    return p @ v, m + np.log(l), p @ np.abs(v), off


def attention_batch_ref(q, q_start, kv_len, own, prefix, scale, group):
    """Rows of every sequence: q [M, Hq, D]; own(s, h) and prefix(h) give (k, v) of a sequence's tokens and of the
    prefix.  Returns out, lse, sum p |v| and the exponents' error scale, NaN in rows of no sequence."""
    M, H, D = q.shape
    out, mag = np.full((M, H, D), np.nan), np.full((M, H, D), np.nan)
    lse, off = np.full((M, H), np.nan), np.full((M, H), np.nan)
    for s in range(len(kv_len)):
        n, L = q_start[s + 1] - q_start[s], kv_len[s]
        for kh in range(H // group):
            ko, vo = own(s, kh)
            kp, vp = prefix(kh)
            for i in range(n):
                see = min(max(L - n + i + 1, 0), L)
                k, v = np.concatenate([kp, ko[:see]]), np.concatenate([vp, vo[:see]])
                m = q_start[s] + i
                for h in range(kh * group, (kh + 1) * group):
                    out[m, h], lse[m, h], mag[m, h], off[m, h] = attention_ref(q[m, h], k, v, scale)
    return out, lse, mag, off


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def linear_attn_ref(q, k, v, decay, scale, S):
    """The recurrence of one sequence and head: (out [T, dv], state, and both with every term's magnitude).

    q, k [T, dk], v [T, dv], decay [T], S [dk, dv]."""
    q, k, v, decay, S = (np.asarray(x, dtype=np.float64) for x in (q, k, v, decay, S))
    A = np.abs(S)
    out, mag = np.zeros(v.shape), np.zeros(v.shape)
    for t in range(q.shape[0]):
        f = np.exp(decay[t])
        S = (0.0 if f == 0 else f * S) + np.outer(k[t], v[t])
        A = (0.0 if f == 0 else f * A) + np.outer(np.abs(k[t]), np.abs(v[t]))
        out[t], mag[t] = scale * (q[t] @ S), abs(scale) * (np.abs(q[t]) @ A)
    return out, S, mag, A
