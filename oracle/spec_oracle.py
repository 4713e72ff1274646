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


def f16_operand_errors(hc: "O.HeadCache") -> Tuple[np.ndarray, np.ndarray]:
    """Bounds [T, d] on what f16 tensor-core operands change of the cache's Keys and Values (see below)."""
    spec, u, step = hc.spec, 2.0 ** -11, 2.0 ** -25
    out = []
    for sink, codes, s, z, scale, resid in ((hc.sink_k, hc.k_codes, hc.k_s, hc.k_z, hc.k_scale, hc.resid_k),
                                            (hc.sink_v, hc.v_codes, hc.v_s, hc.v_z, hc.v_scale, hc.resid_v)):
        if spec.is_fp8:      # the codes are exact; bf16 Values are rounded in units of the scale
            unit = float(scale) * (256.0 if spec.fmt == "fp8_e5m2" else 1.0)
            mid, rest = np.zeros(codes.shape), [np.abs(x.astype(np.float64)) * (u + 2.0 ** -22) + step * unit for x in (sink, resid)]
        else:
            rest = [np.abs(x.astype(np.float64)) * u + step for x in (sink, resid)]
            if spec.is_bf16 or not len(codes):
                mid = np.zeros((0, spec.d))
            else:
                rep = len(codes) // len(s)
                s, z = (np.repeat(np.repeat(x.astype(np.float64), rep, 0), spec.d // x.shape[1], 1) for x in (s, z))
                half = 2.0 ** (spec.bits - 1)
                m, c = codes - half, s * (half - z)
                mid = u * (1 + u) * (np.abs(s * m) + np.abs(c) + np.abs(s * m + c)) + step * (np.abs(m) + 2)
        out.append(np.concatenate([rest[0], mid, rest[1]]))
    return out[0], out[1]


def decode_attention_tree(q: np.ndarray, caches: List[List["O.HeadCache"]], k_draft: np.ndarray, v_draft: np.ndarray,
                          parents: np.ndarray, scale: Optional[float] = None) -> Tuple[np.ndarray, ...]:
    """q [B, N, Hq, d], k_draft / v_draft [B, H, N, d] (float32).  Returns out, lse, ``slack`` and ``lslack``.

    slack [B, N, Hq, d] bounds what f16 tensor-core operands may cost, with u = 2^-11 (half an f16 step, relative):
    a Key or Value x is off by dx <= u |x| + 2^-25, in an integer layer, where it is s m + c with an exact centred
    code m and s and c = s (2^(b-1) - z) rounded to f16 first, by dx <= u (|s m| + |c| + |x|) (1 + u) + 2^-25 (|m| + 2)
    (2^-25: half a step below 2^-14); a probability by u, or 2^-25 where it is below 2^-14 (it is taken relative to a
    maximum that is at most 2^8 stale: the largest one is at least 1).  With ds = scale sum_c |q_c| dk_c
      |dlse| <= max ds,  |do| <= sum_t p_t (|v_t| (exp(2 max ds) (1 + u) - 1) + dv_t exp(2 max ds) (1 + u)) + n_small 2^-25 max|v|
    """
    B, N, Hq, d = q.shape
    H = len(caches[0])
    g = Hq // H
    sc = 1.0 / math.sqrt(d) if scale is None else scale
    u = 2.0 ** -11
    out, slack, lse, lslack = (np.zeros((B, N, Hq) + x) for x in ((d,), (d,), (), ()))
    for b in range(B):
        seen = ancestors(parents[b])
        for h in range(H):
            k, v = O.attention_keys(caches[b][h])
            dk, dv = f16_operand_errors(caches[b][h])
            for n in range(N):
                kk = np.concatenate([k, k_draft[b, h][seen[n]].astype(np.float64)])
                vv = np.concatenate([v, v_draft[b, h][seen[n]].astype(np.float64)])
                qq = q[b, n, h * g:(h + 1) * g].astype(np.float64)
                s = qq @ kk.T * sc
                dkk = np.concatenate([dk, np.abs(kk[len(k):]) * u + 2.0 ** -25])
                dvv = np.concatenate([dv, np.abs(vv[len(v):]) * u + 2.0 ** -25])
                ds = (np.abs(qq) @ dkk.T * abs(sc)).max(-1)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                el = p.sum(-1, keepdims=True)
                small = (p < 2.0 ** -14).sum(-1)
                out[b, n, h * g:(h + 1) * g] = p @ vv / el
                lse[b, n, h * g:(h + 1) * g] = m[:, 0] + np.log(el[:, 0])
                grow = np.exp(2 * ds) * (1 + u) - 1 + 2.0 ** -18  # (fp32 sums, exp2 and the division)
                lslack[b, n, h * g:(h + 1) * g] = ds + 2.0 ** -18 * (1 + np.abs(lse[b, n, h * g:(h + 1) * g]))
                slack[b, n, h * g:(h + 1) * g] = (p @ np.abs(vv) / el) * grow[:, None] + \
                    (p @ dvv / el) * (1 + grow[:, None]) + (small * 2.0 ** -25 / el[:, 0])[:, None] * np.abs(vv).max()
    return out, lse, slack, lslack


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
