"""Float64 definitions of the calls over a paged cache (page assignment, norm + rotation + write, attention).

Plain numpy, request by request and row by row; imports nothing from the library.
"""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0


def page_assign(P, lens, n_new, free_pages, head, tables, max_tokens, pos_offset=None):
    """Outputs of one step: dict of slots, positions, seq_ids, lens, indptr, head, tables (None: it cannot be carried out)."""
    tables = np.array(tables, np.int64)
    cap = tables.shape[1] * P
    if any(n < 0 or m < 0 or n + m > cap for n, m in zip(lens, n_new)):
        return None
    need = [-(-(n + m) // P) - -(-n // P) for n, m in zip(lens, n_new)]
    if sum(n_new) > max_tokens or head < 0 or head + sum(need) > len(free_pages):
        return None
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.zeros(max_tokens, np.int64)
    seq_ids = np.full(max_tokens, -1, np.int64)
    indptr = [0]
    for b, (n, m) in enumerate(zip(lens, n_new)):
        have = -(-n // P)
        for j in range(need[b]):
            tables[b, have + j] = free_pages[head]
            head += 1
        for i in range(m):
            t, row = indptr[-1] + i, n + i
            slots[t] = tables[b, row // P] * P + row % P
            positions[t] = row + (0 if pos_offset is None else pos_offset[b])
            seq_ids[t] = b
        indptr.append(indptr[-1] + m)
    return {"slots": slots, "positions": positions, "seq_ids": seq_ids, "lens": np.array(lens) + np.array(n_new),
            "indptr": np.array(indptr), "head": head, "tables": tables}


def rope_freqs(rot, kind, base, factor=1.0, low=1.0, high=4.0, original=8192):
    """(inv_freq [rot / 2], factor on cos and sin)."""
    out, scale = [], 1.0
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        if kind == "plain":
            out.append(theta)
        elif kind == "linear":
            out.append(theta / factor)
        elif kind == "banded":
            wave = 2 * math.pi / theta
            if wave < original / high:
                out.append(theta)
            elif wave > original / low:
                out.append(theta / factor)
            else:
                s = (original / wave - low) / (high - low)
                out.append((1 - s) * theta / factor + s * theta)
        else:
            def index(turns):
                return rot * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))
            lo, hi = max(0, math.floor(index(high))), min(rot - 1, math.ceil(index(low)))
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(r * theta / factor + (1 - r) * theta)
            scale = 0.1 * math.log(factor) + 1.0
    return np.array(out), scale


def norm_rope(x, positions, inv_freq, factor, layout, weight=None, bias=0.0, eps=0.0):
    """x [tokens, heads, d] -> (y, size): the normed and turned rows, and |a| + |b| of each element's pair (for bounds)."""
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + bias)
    size = np.abs(y)
    r = 0 if inv_freq is None else len(inv_freq)
    for p in range(r):
        ia, ib = (p, r + p) if layout == "half" else (2 * p, 2 * p + 1)
        angle = positions.astype(np.float64) * inv_freq[p]
        c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = (np.abs(a) + np.abs(b)) * abs(factor)
    return y, size


def paged_attend(q, k, v, scale, softcap=0.0, window=0, slopes=None):
    """One request and KV head: q [G, d], k, v [n, d] (its rows in order) -> (o [G, d], lse [G], mass [G, d], zmax).

    mass = sum_t p_t |v_t| and zmax = the largest sum_c |q_c k_c| scale of a seen row: what error bounds scale with.
    """
    n, d = k.shape
    G = q.shape[0]
    first = max(0, n - window) if window else 0
    if n == 0:
        return np.zeros((G, d)), np.full(G, -np.inf), np.zeros((G, d)), 0.0
    k, v = k[first:], v[first:]
    z = scale * (q @ k.T)
    zmax = float((scale * (np.abs(q) @ np.abs(k).T)).max())
    if softcap:
        z = softcap * np.tanh(z / softcap)
    if slopes is not None:
        z = z + np.asarray(slopes)[:, None] * (np.arange(first, n) - (n - 1))
    m = z.max(-1, keepdims=True)
    p = np.exp(z - m)
    total = p.sum(-1, keepdims=True)
    return p @ v / total, (m + np.log(total))[:, 0], p @ np.abs(v) / total, zmax
