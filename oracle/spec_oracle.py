"""CPU oracle of a speculative decoding step over the quantized cache, in fp64.

Written from the definitions in include/kvq.h (kvq_qk_norm_rope,
kvq_decode_attention_tree, kvq_verify_tree, kvq_append_accepted); the cache and
the score formula are those of kvq_oracle.
"""
from __future__ import annotations

import math
from typing import List, Optional, Sequence, Tuple

import numpy as np

from . import kvq_oracle as O


def rotate_exact(x: np.ndarray, positions: np.ndarray, base: float) -> np.ndarray:
    """Rotate-half RoPE of rows [n, 128] at int positions, the angles reduced in extended precision."""
    i = np.arange(64, dtype=np.longdouble)
    theta = np.power(np.longdouble(base), -i / 64)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    a = np.fmod(positions.astype(np.longdouble)[:, None] * theta, two_pi).astype(np.float64)
    x = x.astype(np.float64)
    lo, hi = x[:, :64], x[:, 64:]
    return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)


def head_norm(x: np.ndarray, w: Optional[np.ndarray], eps: float) -> np.ndarray:
    """w x / sqrt(mean(x^2) + eps) along the last axis (w None: x)."""
    x = x.astype(np.float64)
    if w is None:
        return x
    return w.astype(np.float64) * x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))


def ancestors(parents: Sequence[int]) -> np.ndarray:
    """[n, n] truth values: whether node m (column) is node n (row) or above it."""
    n = len(parents)
    out = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            out[i] = out[p]
        out[i, i] = True
    return out


def decode_attention_tree(q: np.ndarray, caches: List[List["O.HeadCache"]], k_draft: np.ndarray, v_draft: np.ndarray,
                          parents: np.ndarray, scale: Optional[float] = None) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """q [B, N, Hq, d], k_draft / v_draft [B, H, N, d] (float32).  Returns out, lse and ``slack``.

    slack [B, N, Hq, d] bounds what f16 tensor-core operands may cost: with u = 2^-11 (half an f16
    step, relative) on Keys, Values and probabilities and 2^-25 where a probability is below 2^-14,
      |ds| <= scale sum_c |q_c k_c| u,   |do| <= sum_t p_t |v_t| (exp(2 max|ds|) (1 + u)^2 - 1) + n_small 2^-25 max|v|
    (a probability is taken relative to a maximum that is at most 2^8 stale: the largest one is at least 1).
    """
    B, N, Hq, d = q.shape
    H = len(caches[0])
    g = Hq // H
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    u = 2.0 ** -11
    out, slack, lse = np.zeros((B, N, Hq, d)), np.zeros((B, N, Hq, d)), np.zeros((B, N, Hq))
    for b in range(B):
        seen = ancestors(parents[b])
        for h in range(H):
            k, v = O.attention_keys(caches[b][h])
            for n in range(N):
                kk = np.concatenate([k, k_draft[b, h][seen[n]].astype(np.float64)])
                vv = np.concatenate([v, v_draft[b, h][seen[n]].astype(np.float64)])
                qq = q[b, n, h * g:(h + 1) * g].astype(np.float64)
                s = qq @ kk.T * sc
                ds = (np.abs(qq) @ np.abs(kk).T * abs(sc) * u).max(-1)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                el = p.sum(-1, keepdims=True)
                small = (p < 2.0 ** -14).sum(-1)
                out[b, n, h * g:(h + 1) * g] = p @ vv / el
                lse[b, n, h * g:(h + 1) * g] = m[:, 0] + np.log(el[:, 0])
                grow = np.exp(2 * ds) * (1 + u) ** 2 - 1 + 2.0 ** -18  # (fp32 sums, exp2 and the division)
                slack[b, n, h * g:(h + 1) * g] = (p @ np.abs(vv) / el) * grow[:, None] + \
                    (small * 2.0 ** -25 / el[:, 0])[:, None] * np.abs(vv).max()
    return out, lse, slack


def verify_tree(target: np.ndarray, draft: Optional[np.ndarray], tokens: np.ndarray, parents: np.ndarray,
                uniforms: np.ndarray):
    """One sequence: target [N, V], draft [N, V] or None.  Returns (path list, next token or -1)."""
    N, V = target.shape
    at, path = 0, [0]
    w, total = target[0].astype(np.float64), 1.0
    for c in range(1, N):
        if parents[c] != at or not 0 <= tokens[c] < V:
            continue
        x = tokens[c]
        if draft is None:
            q = np.zeros(V)
            q[x] = 1.0
        else:
            q = draft[at].astype(np.float64)
        if float(uniforms[c]) * (total * q[x]) < w[x]:
            at = c
            path.append(c)
            w, total = target[c].astype(np.float64), 1.0
        else:
            w = np.maximum(w - total * q, 0.0)
            total = w.sum()
    if not (w.sum() > 0 and np.isfinite(w.sum())):
        w = target[at].astype(np.float64)
    if not (w.sum() > 0 and np.isfinite(w.sum())):
        return path, -1
    cum = np.cumsum(w)
    past = np.nonzero(cum > float(uniforms[0]) * cum[-1])[0]
    return path, int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])
