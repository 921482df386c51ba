"""Float64 reference of a sampling step: norms of query and key heads with the
rotation of their pairs and the gradients, and attention over a paged cache
whose requests share prefixes.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``: imported by ``tests/``
and never by the library.  The root-mean-square norm is the usual one, taken
over each head.
"""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np

from . import serving


def norm(x: np.ndarray, eps: float):
    """(x r, r) of heads x [..., d], r = (mean(x^2) + eps)^(-1/2)."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def qk_norm_rope(x, w, positions, axis: Sequence[int], inv_freq: Sequence[float], neighbours: bool, eps: float):
    """x [T, H, d], w [d] -> Rot(w n), float64."""
    return serving.rope_axes(norm(x, eps)[0] * np.asarray(w, np.float64), positions, axis, inv_freq, neighbours)


def qk_norm_rope_bwd(dy, x, w, positions, axis, inv_freq, neighbours: bool, eps: float):
    """(dx, dw) of qk_norm_rope, from the derivative of each head: with f(x) = x r,
    df = r (I - n n^T / d) (a symmetric matrix), n = f."""
    w = np.asarray(w, np.float64)
    g = serving.rope_axes(dy, positions, axis, inv_freq, neighbours, inverse=True)
    n, r = norm(x, eps)
    u = g * w
    dx = np.empty_like(u)
    d = u.shape[-1]
    for t in range(u.shape[0]):
        for h in range(u.shape[1]):
            dx[t, h] = r[t, h] * (np.eye(d) - np.outer(n[t, h], n[t, h]) / d) @ u[t, h]
    return dx, (g * n).sum((0, 1))


def decode_shared(q, k_of, v_of, table, lens, starts, shared, page_size: int, window_left: int, scale: float,
                  Hkv: Optional[int] = None):
    """q [B, Nq, Hq, d] over a cache whose requests starts[g] .. starts[g + 1] - 1
    share their first shared[g] tokens: those are read through the table's row
    of the group's longest request, all others through the request's own.
    k_of, v_of: (page, slot) -> [Hkv, d].  Returns (o, lse [B, Hq, Nq], a): a = sum_j P_j |v_j|."""
    q = np.asarray(q, np.float64)
    B, Nq, Hq, d = q.shape
    o, a = np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, Hq, Nq), -np.inf)
    for g in range(len(shared)):
        members = range(int(starts[g]), int(starts[g + 1]))
        if not len(members):
            continue
        longest = max(members, key=lambda b: (int(lens[b]), -b))
        for b in members:
            n = int(lens[b])
            if n == 0:
                continue
            at = [(int(table[longest if j < shared[g] else b, j // page_size]), j % page_size) for j in range(n)]
            k = np.array([k_of(p, t) for p, t in at], np.float64)  # [n, Hkv, d]
            v = np.array([v_of(p, t) for p, t in at], np.float64)
            heads = Hq // k.shape[1]
            for i in range(Nq):
                pos = n - Nq + i
                lo = max(0, pos - window_left) if window_left >= 0 else 0
                if pos < 0:
                    continue
                for h in range(Hq):
                    s = scale * (k[lo:pos + 1, h // heads] @ q[b, i, h])
                    m = s.max()
                    p = np.exp(s - m)
                    lse[b, h, i] = m + np.log(p.sum())
                    p /= p.sum()
                    o[b, i, h] = p @ v[lo:pos + 1, h // heads]
                    a[b, i, h] = p @ np.abs(v[lo:pos + 1, h // heads])
    return o, lse, a
