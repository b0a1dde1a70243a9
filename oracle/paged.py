"""CPU oracle for the paged cache operators: qk_norm_rope, kv_append, paged_attention.

TEST INFRASTRUCTURE ONLY: the same rules as ``oracle.compressor`` apply (only
the tests and the smoke check may import it; it shares no code with the CUDA
library). Everything is float64; inputs are the exact values of the 16-bit
tensors. Beside each result stands the sum of magnitudes that its rounding
errors scale with, so that tests can derive their tolerances.

* norm: y = x / sqrt(mean(x^2) + eps) * w over a head's channels.
* rotation of the last R channels, pair (a, b), table columns j and R/2 + j:
  a' = a cos_j - b sin_j, b' = b cos_{R/2+j} + a sin_{R/2+j}; "interleaved" pairs
  are channels (2j, 2j+1) of the rotated part, "halves" (j, R/2 + j).
* position p of sequence b is row p % page of block table[b][p // page].
* the token at position p sees n(p) = 0 if p + 1 < key_block else
  (p + 1 - key_block) // key_stride + 1 keys, of those the last ``window``;
  out = sum softmax(scale q.k) v, lse = log sum exp(scale q.k); none: 0, -inf.
"""

from __future__ import annotations

import dataclasses

import numpy as np


def norm_rope(x, weight, sin, cos, pairs: str, eps: float):
    """x [T, H, D]; weight [D] or None; sin / cos [T, R] or None. Returns (y, mag):
    |y| <= mag, with mag the sum of the magnitudes of the terms of each y."""
    y = np.asarray(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    mag = np.abs(y)
    if cos is None:
        return y, mag
    R, D = cos.shape[1], y.shape[-1]
    out, om = y.copy(), mag.copy()
    for j in range(R // 2):
        ia, ib = (D - R + 2 * j, D - R + 2 * j + 1) if pairs == "interleaved" else (D - R + j, D - R // 2 + j)
        ca, sa = cos[:, None, j].astype(np.float64), sin[:, None, j].astype(np.float64)
        cb, sb = cos[:, None, R // 2 + j].astype(np.float64), sin[:, None, R // 2 + j].astype(np.float64)
        a, b = y[:, :, ia], y[:, :, ib]
        out[:, :, ia] = a * ca - b * sa
        out[:, :, ib] = b * cb + a * sb
        om[:, :, ia] = np.abs(a * ca) + np.abs(b * sa)
        om[:, :, ib] = np.abs(b * cb) + np.abs(a * sb)
    return out, om


def cache_rows(table, cu_seqlens, start_pos, page):
    """(token, cache row) of every token of a sequence."""
    res = []
    for b in range(len(cu_seqlens) - 1):
        for i in range(int(cu_seqlens[b]), int(cu_seqlens[b + 1])):
            p = int(start_pos[b]) + i - int(cu_seqlens[b])
            res.append((i, int(table[b][p // page]) * page + p % page))
    return res


def visible(p: int, key_block: int = 1, key_stride: int = 1, window: int = 0):
    """Keys [lo, hi) that the token at position p sees."""
    hi = 0 if p + 1 < key_block else (p + 1 - key_block) // key_stride + 1
    return (max(0, hi - window) if window else 0), hi


@dataclasses.dataclass
class AttnResult:
    out: np.ndarray       # [T, Hq, D]
    lse: np.ndarray       # [T, Hq]
    weight_mag: np.ndarray  # [T, Hq, D] sum_j softmax_j |v_j|
    v_mag: np.ndarray     # [T, Hq, D] sum over the seen keys of |v_j|
    score_mag: np.ndarray  # [T, Hq] max over the seen keys of scale * sum_d |q_d k_d|
    n: np.ndarray         # [T] keys seen
    rows: np.ndarray      # bool [T]: the token belongs to a sequence


def paged_attention(q, k_cache, v_cache, table, cu_seqlens, start_pos, scale, *, key_block=1, key_stride=1,
                    window=0) -> AttnResult:
    """q [T, Hq, D]; caches [blocks, page, Hk, D], all exact values."""
    T, Hq, D = q.shape
    page, Hk = k_cache.shape[1], k_cache.shape[2]
    G = Hq // Hk
    q = q.astype(np.float64)
    out = np.zeros((T, Hq, D))
    wm, vm = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    sm = np.zeros((T, Hq))
    n = np.zeros(T, dtype=np.int64)
    rows = np.zeros(T, dtype=bool)
    for b in range(len(cu_seqlens) - 1):
        t0, t1 = int(cu_seqlens[b]), int(cu_seqlens[b + 1])
        if t1 <= t0:
            continue
        rows[t0:t1] = True
        span = [visible(int(start_pos[b]) + i, key_block, key_stride, window) for i in range(t1 - t0)]
        first, last = min(s[0] for s in span), max(s[1] for s in span)
        if last <= first:
            continue
        at = [int(table[b][j // page]) * page + j % page for j in range(first, last)]
        kk = k_cache.reshape(-1, Hk, D)[at].astype(np.float64)
        vv = v_cache.reshape(-1, Hk, D)[at].astype(np.float64)
        for i, (lo, hi) in enumerate(span):
            n[t0 + i] = hi - lo
            if hi <= lo:
                continue
            a, z = kk[lo - first:hi - first], vv[lo - first:hi - first]
            for h in range(Hq):
                x = a[:, h // G] @ q[t0 + i, h] * scale
                m = x.max()
                e = np.exp(x - m)
                s = e.sum()
                v = z[:, h // G]
                out[t0 + i, h] = e @ v / s
                wm[t0 + i, h] = e @ np.abs(v) / s
                vm[t0 + i, h] = np.abs(v).sum(0)
                lse[t0 + i, h] = m + np.log(s)
                sm[t0 + i, h] = scale * (np.abs(a[:, h // G]) @ np.abs(q[t0 + i, h])).max()
    return AttnResult(out=out, lse=lse, weight_mag=wm, v_mag=vm, score_mag=sm, n=n, rows=rows)
