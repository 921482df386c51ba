"""Float64 / exact-integer reference of one serving step: planning pages from
request lengths, rotary positions with several axes, the 8-bit paged cache's
write side, and attention over that cache.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``: imported by ``tests/``
and never by the library.

Sources (zerotofrontier.app "efficient-attention/flash-2-3"): "Paged KV
caches, a preview of serving" (block tables, pages taken from a free list when
the last one fills), "FP8, and the outlier problem" (e4m3 with one scale per
block).  The rotary embedding is the usual one: pair p of a head turns by
position * frequency; with several axes each pair takes the position of its
own axis.
"""
from __future__ import annotations

from typing import List, Optional, Sequence

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode

NEG_INF = -np.inf


class PlanError(RuntimeError):
    """The step cannot be planned; ``code`` is the device error the library records."""

    def __init__(self, code: int):
        self.code = code
        super().__init__(hex(code))


def page_plan(ctx: Sequence[int], new: Sequence[int], free: Sequence[int], free_count: int, table: np.ndarray,
              page_size: int, max_tokens: int):
    """One request after the other, one token after the other.  Returns
    (seq_lens, cu_new, page, slot, position, free_count, table); raises PlanError."""
    table = table.copy()
    max_blocks = table.shape[1]
    if any(c < 0 or n < 0 or c + n > max_blocks * page_size for c, n in zip(ctx, new)) or sum(new) > max_tokens or \
            not 0 <= free_count <= len(free):
        raise PlanError(0x2001)
    stack = list(free[:free_count])
    page: List[int] = []
    slot: List[int] = []
    position: List[int] = []
    cu = [0]
    for b, (c, n) in enumerate(zip(ctx, new)):
        for t in range(c, c + n):
            if t % page_size == 0:
                if not stack:
                    raise PlanError(0x2002)
                table[b, t // page_size] = stack.pop()
            page.append(int(table[b, t // page_size]))
            slot.append(t % page_size)
            position.append(t)
        cu.append(cu[-1] + n)
    pad = max_tokens - len(page)
    return ([c + n for c, n in zip(ctx, new)], cu, page + [-1] * pad, slot + [-1] * pad, position + [0] * pad,
            len(stack), table)


def rope_axes(x: np.ndarray, positions: np.ndarray, axis: Sequence[int], inv_freq: Sequence[float],
              neighbours: bool, inverse: bool = False) -> np.ndarray:
    """x [T, H, d], positions [n_axes, T] -> rotated, float64.  Pair by pair."""
    x = np.asarray(x, np.float64)
    out = x.copy()
    half = x.shape[-1] // 2
    for p in range(half):
        if axis[p] < 0:
            continue
        a = np.asarray(positions[axis[p]], np.float64) * inv_freq[p]
        if inverse:
            a = -a
        i, j = (2 * p, 2 * p + 1) if neighbours else (p, p + half)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., i] * s + x[..., j] * c
    return out


def pow2_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s; 0 for 0."""
    if amax == 0:
        return 0.0
    e = -126
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def kv8_append(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, page: Sequence[int], slot: Sequence[int],
               copy_src: Optional[Sequence[int]] = None) -> None:
    """x [n, H, d] (bf16 values); codes [pages, H, P, d] uint8 and scales
    [pages, H] updated in place.  Copies read the cache as it was."""
    n = len(page)
    runs = []
    i = 0
    while i < n:
        if page[i] == -1:
            i += 1
            continue
        j = i + 1
        while j < n and page[j] == page[i] and slot[j] == slot[j - 1] + 1:
            j += 1
        runs.append((i, j))
        i = j
    was_codes, was_scales = codes.copy(), scales.copy()
    for i, j in runs:
        pg, first = page[i], slot[i]
        src = copy_src[i] if copy_src is not None and copy_src[i] >= 0 else pg
        for h in range(x.shape[1]):
            v = np.asarray(x[i:j, h], np.float64)
            fine = v[np.isfinite(v)]
            own = pow2_scale(float(np.max(np.abs(fine))) if fine.size else 0.0)
            old = float(was_scales[src, h]) if first > 0 else 0.0
            s = max(own, old)
            for t in range(first):
                c = e4m3_decode(was_codes[src, h, t])
                codes[pg, h, t] = _encode(c * (old / s) if old > 0 else c * 0.0)
            codes[pg, h, first:first + j - i] = _encode(v / s if s > 0 else np.where(np.isfinite(v), 0.0, v))
            scales[pg, h] = s


def _encode(v) -> np.ndarray:
    """e4m3 codes; a NaN or an infinity is the NaN code."""
    v = np.asarray(v, np.float64)
    fine = np.isfinite(v)
    return np.where(fine, e4m3_encode(np.where(fine, v, 0.0)), 0x7F).astype(np.uint8)


def kv8_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """[pages, H, P, d] float64."""
    return e4m3_decode(codes) * np.asarray(scales, np.float64)[:, :, None, None]


def decode_kv8(q: np.ndarray, codes_k, codes_v, scales_k, scales_v, table, lens, window_left: int, scale: float):
    """q [B, Nq, Hq, d] -> (o, lse [B, Hq, Nq], a, f): float64; a = sum_j P_j |v_j|, the
    size that relative errors of P are measured against, and
    f = max_j (P_j vs_j) sum_j |v8_j|, that of errors of P vs relative to its largest."""
    q = np.asarray(q, np.float64)
    B, Nq, Hq, d = q.shape
    Hkv, P = codes_k.shape[1], codes_k.shape[2]
    g = Hq // Hkv
    o, a, f = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    lse = np.full((B, Hq, Nq), NEG_INF)
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            at = [(int(table[b, j // P]), j % P) for j in range(n)]
            k = np.array([e4m3_decode(codes_k[p, h, t]) * float(scales_k[p, h]) for p, t in at]).reshape(n, d)
            v = np.array([e4m3_decode(codes_v[p, h, t]) * float(scales_v[p, h]) for p, t in at]).reshape(n, d)
            vs = np.array([float(scales_v[p, h]) for p, t in at])
            v8 = np.array([np.abs(e4m3_decode(codes_v[p, h, t])) for p, t in at]).reshape(n, d)
            for i in range(Nq):
                pos = n - Nq + i
                lo = max(0, pos - window_left) if window_left >= 0 else 0
                if pos < 0:
                    continue
                for hq in range(h * g, (h + 1) * g):
                    s = scale * (k[lo:pos + 1] @ q[b, i, hq])
                    m = s.max()
                    w = np.exp(s - m)
                    lse[b, hq, i] = m + np.log(w.sum())
                    w /= w.sum()
                    o[b, i, hq] = w @ v[lo:pos + 1]
                    a[b, i, hq] = w @ np.abs(v[lo:pos + 1])
                    f[b, i, hq] = (w * vs[lo:pos + 1]).max() * v8[lo:pos + 1].sum(0)
    return o, lse, a, f
