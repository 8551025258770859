"""fp64 oracle of the rotary positions and the paged KV cache -- TEST
INFRASTRUCTURE ONLY (as the rest of this package: never imported by the
product library, never importing it).  Plain numpy, one row at a time."""
from __future__ import annotations

import numpy as np


def slots(axes, theta, shared):
    """(axis, frequency) of every slot."""
    rot = sum(axes)
    out = []
    for a, n in enumerate(axes):
        for i in range(n // 2):
            out.append((a, theta ** (-2.0 * len(out) / rot) if shared else theta ** (-2.0 * i / n)))
    return out


def table(axes, n_pos, theta=10000.0, shared=False):
    """[entries][2] fp64 (cos, sin): axis 0's positions x slots, then axis 1's, then axis 2's."""
    sl = slots(axes, theta, shared)
    rows = []
    for a in range(3):
        f = np.array([w for b, w in sl if b == a], dtype=np.float64)
        ang = np.arange(n_pos[a], dtype=np.float64)[:, None] * f
        rows.append(np.stack([np.cos(ang), np.sin(ang)], -1).reshape(-1, 2))
    return np.concatenate(rows)


def grid_coords(ids, grid_h, grid_w):
    ids = np.asarray(ids, dtype=np.int64)
    return np.stack([ids // (grid_w * grid_h), ids // grid_w % grid_h, ids % grid_w], -1)


def rope(x, coords, axes, theta=10000.0, halves=False, shared=False):
    """x fp64 [n][heads][d], coords int [n][3] -> rotated fp64."""
    y = np.array(x, dtype=np.float64)
    sl = slots(axes, theta, shared)
    n = len(sl)
    for r in range(y.shape[0]):
        for s, (a, f) in enumerate(sl):
            c, w = np.cos(coords[r][a] * f), np.sin(coords[r][a] * f)
            i, j = (s, s + n) if halves else (2 * s, 2 * s + 1)
            p, q = x[r, :, i].astype(np.float64), x[r, :, j].astype(np.float64)
            y[r, :, i] = p * c - q * w
            y[r, :, j] = p * w + q * c
    return y


def rope_partner(x, axes, halves):
    """|x0| + |x1| of every column's pair (0 for columns that are kept): the scale of the fp32 rounding errors."""
    n = sum(axes) // 2
    e = np.zeros_like(np.asarray(x, dtype=np.float64))
    for s in range(n):
        i, j = (s, s + n) if halves else (2 * s, 2 * s + 1)
        e[..., i] = e[..., j] = np.abs(x[..., i]) + np.abs(x[..., j])
    return e


def gather(pages, table_row, length):
    """pages [n_pages][page_size][h][d] -> the sequence's positions [length][h][d]."""
    p = pages.shape[1]
    return np.array([pages[table_row[j // p], j % p] for j in range(length)], dtype=pages.dtype).reshape(
        length, *pages.shape[2:])


def attention(q, k, v, limits, scale):
    """q fp64 [n][heads][d] over k, v fp64 [len][kv_heads][d]; row r sees the first min(len, limits[r]) keys.
    Returns (out, bound): bound[r][h][c] = sum_j p_j |v_j,c| * (1 + the largest scale * sum |q| |k|), from which
    tests scale their tolerance."""
    n, heads, d = q.shape
    length, kv_heads, _ = k.shape
    g = heads // kv_heads
    out, pv, top = np.zeros_like(q), np.zeros_like(q), np.zeros((n, heads, 1))
    for r in range(n):
        m = min(length, int(limits[r]))
        if m <= 0:
            continue
        for h in range(heads):
            s = scale * (k[:m, h // g] @ q[r, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[r, h] = p @ v[:m, h // g]
            pv[r, h] = p @ np.abs(v[:m, h // g])
            top[r, h] = scale * (np.abs(k[:m, h // g]) @ np.abs(q[r, h])).max()
    return out, pv, top
