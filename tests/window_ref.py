"""64-bit references of the windowed latent-cache operators, slot by slot in numpy (tests only)."""
from __future__ import annotations

import numpy as np

H, NOPE, ROPE, V, LORA, PAGE, ROW = 96, 128, 64, 128, 512, 64, 576
QDIM = NOPE + ROPE


def rows_of(pos0, row_start, R):
    """(slot, position) of every packed row; (-1, -1) for rows outside every slot or before position 0."""
    at = [(-1, -1)] * R
    for b, p0 in enumerate(pos0):
        lo, hi = (b, b + 1) if row_start is None else (int(row_start[b]), int(row_start[b + 1]))
        for r in range(max(lo, 0), min(hi, R)):
            p = int(p0) + r - lo
            at[r] = (b, p) if p >= 0 else (-1, -1)
    return at


def norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def pairs(interleaved):
    i = np.arange(ROPE // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + ROPE // 2)


def rotate(x, pos, inv_freq, interleaved):
    """The rotated entries and, per entry, the magnitude |a| + |b| of its pair (the scale of its error)."""
    if inv_freq is None:
        return x, np.abs(x)
    a, b = pairs(interleaved)
    angle = float(pos) * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle), np.sin(angle)
    y, mag = np.empty_like(x), np.empty_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    mag[..., a] = mag[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, mag


def query_row(q, pos, weight, eps, inv_freq, interleaved):
    """[96, 192] -> (values, error scale)."""
    x = norm(q, weight, eps)
    mag = np.abs(x)
    x = x.copy()
    x[..., NOPE:], mag[..., NOPE:] = rotate(x[..., NOPE:], pos, inv_freq, interleaved)
    return x, mag


def key_row(c, k, pos, cw, kw, eps, inv_freq, interleaved):
    """[512], [64] -> ([576] values, error scale)."""
    c = norm(c, cw, eps)
    k, mag = rotate(norm(k, kw, eps), pos, inv_freq, interleaved)
    return np.concatenate([c, k]), np.concatenate([np.abs(c), mag])


def visible(n, window, sink):
    """Positions that the last of n tokens attends to."""
    t = np.arange(max(n, 0))
    return t[(t < sink) | (t >= n - window)]


def latent_rows(slab, layer, table_row, t):
    """[len(t), 576] f64 rows of positions t; a -1 entry (or one outside the slab) reads as zeros."""
    page = table_row[t // PAGE]
    ok = (page >= 0) & (page < slab.shape[0])
    return np.where(ok[:, None], np.asarray(slab[np.where(ok, page, 0), layer, t % PAGE], np.float64), 0.0)


def attend(q_abs, slab, layer, table_row, n, window, sink, w_kv_b, scale):
    """One token row: q_abs [96, 576] -> (out [96, 128], o_lat [96, 512], p [96, T], rows [T, 576]), all f64;
    zeros for n == 0."""
    if n <= 0:
        return np.zeros((H, V)), np.zeros((H, LORA)), np.zeros((H, 0)), np.zeros((0, ROW))
    rows = latent_rows(slab, layer, table_row, visible(n, window, sink))
    s = np.asarray(q_abs, np.float64) @ rows.T * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o = p @ rows[:, :LORA]
    w_uv = np.asarray(w_kv_b, np.float64).reshape(H, NOPE + V, LORA)[:, NOPE:]
    return np.einsum("hvk,hk->hv", w_uv, o), o, p, rows


def out_tolerance(out, o, p, rows, w_kv_b, s_abs):
    """Bound of |kernel - reference| for one token row, element by element.

    The kernel's roundings: every p to bf16 (relative 2^-8), o_lat to f16 after a power of two that brings its
    row's largest entry to 1 or more (2^-11 / 2 of the entry, or half a subnormal step, 2^-25, which is at most
    2^-25 of the row's largest), the O of each split likewise when there are several (so sum_t p_t |row_t| and the
    largest of it stand for |o|, and both count twice), the output to bf16 (2^-8), f32 sums besides: each score within 640 * 2^-24 of sum |q||row| * scale
    (s_abs, per head and token: its exponential moves by as much), the hardware exponential 2^-21, the sums over
    tokens and latent entries 2^-15 in all.  A p that is off by a factor (1 + d_t) moves o by
    sum_t p_t d_t (row_t - o): at most max|d| * sum_t p_t |row_t - o|, here taken through |W_UV|."""
    w = np.abs(np.asarray(w_kv_b, np.float64).reshape(H, NOPE + V, LORA)[:, NOPE:])
    if p.shape[1] == 0:
        return np.zeros_like(out)
    d = 2.0 ** -8 + 2.0 ** -19 + 640 * 2.0 ** -24 * s_abs                      # [96, T]
    spread = np.einsum("ht,tk->hk", p * d, np.abs(rows[:, :LORA])) + np.einsum("ht,hk->hk", p * d, np.abs(o))
    mass = np.einsum("ht,tk->hk", p, np.abs(rows[:, :LORA]))
    half = 2 * (2.0 ** -12 * mass + 2.0 ** -25 * mass.max(-1, keepdims=True))
    return (np.einsum("hvk,hk->hv", w, spread + half + 2.0 ** -15 * mass) + 2.0 ** -8 * np.abs(out)) * 1.01 + 1e-30
