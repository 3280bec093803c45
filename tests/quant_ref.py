"""64-bit references of the 8-bit latent cache (tests only): its rows in numpy, and bounds of what its kernels may be off by."""
from __future__ import annotations

import numpy as np

from tests.window_ref import H, LORA, NOPE, PAGE, ROPE, ROW, V

QROW, QPAGE = 640, 41088
# every e4m3 code's value
_E, _M = (np.arange(256) >> 3) & 15, np.arange(256) & 7
E4M3 = np.where(_E > 0, (8 + _M) * 2.0 ** (_E - 10.0), _M * 2.0 ** -9)
E4M3[(_E == 15) & (_M == 7)] = np.nan
E4M3 = np.where(np.arange(256) >= 128, -E4M3, E4M3)


def to_codes(x):
    """The nearest e4m3 code, ties to the even one (|x| <= 448); NaN where x is none."""
    a = np.abs(np.nan_to_num(np.asarray(x, np.float64)))
    up = np.searchsorted(E4M3[:127], a)                      # the first code at or above
    hi = np.minimum(up, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - E4M3[lo], E4M3[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(E4M3[hi] == a, hi, code)
    code = np.where(np.isnan(x), 127, code)
    return (code | (np.signbit(x) << 7)).astype(np.uint8)


def bf16_bits(x):
    """f64 -> the nearest bf16's bits, ties to even (no NaN; the rounding to f32 on the way is exact for what is tested)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def bits_value(b):
    return (np.asarray(b, np.uint32) << 16).view(np.float32).astype(np.float64)


def exponent(c, k):
    """The n of rows with latents c [..., 512] and rope keys k [..., 64]."""
    m = np.where(np.isfinite(c), np.abs(c), 0).max(-1)
    r = np.where(np.isfinite(k), np.abs(k), 0).max(-1)
    f, e = np.frexp(m)
    n = np.where(m > 0, e - 9 + (f > 0.875), 0)
    return np.clip(np.maximum(n, np.frexp(r)[1] - 120), -96, 120)


def quantise(rows):
    """[..., 576] f64 -> codes u8 [..., 512], scale bits u16 [...], rope bits u16 [..., 64]."""
    c, k = rows[..., :LORA], rows[..., LORA:]
    n = exponent(c, k)
    down = 2.0 ** -n[..., None]
    with np.errstate(invalid="ignore"):
        return to_codes(np.where(np.isfinite(c), c * down, np.nan)), ((n + 127) << 7).astype(np.uint16), bf16_bits(k * down)


def pack(codes, scale, rope):
    """[..., 64, 512], [..., 64], [..., 64, 64] -> page blocks u8 [..., 41088]."""
    rows = np.concatenate([codes, np.ascontiguousarray(rope).view(np.uint8)], -1)
    return np.concatenate([rows.reshape(*rows.shape[:-2], PAGE * QROW), np.ascontiguousarray(scale).view(np.uint8)], -1)


def unpack(blocks):
    rows = blocks[..., :PAGE * QROW].reshape(*blocks.shape[:-1], PAGE, QROW)
    scale = np.ascontiguousarray(blocks[..., PAGE * QROW:]).view(np.uint16)
    return rows[..., :LORA], scale, np.ascontiguousarray(rows[..., LORA:]).view(np.uint16)


def values(blocks):
    """Page blocks [..., 41088] -> what they stand for, f64 [..., 64, 576]."""
    codes, scale, rope = unpack(blocks)
    return np.concatenate([E4M3[codes], bits_value(rope)], -1) * bits_value(scale)[..., None]


def row_values(blocks, layer, table_row, t):
    """[len(t), 576] f64 rows of positions t of a slab [n_pages, L, 41088], and their scales; -1 entries: zeros (scale 1)."""
    page = table_row[t // PAGE]
    ok = (page >= 0) & (page < blocks.shape[0])
    at, line = np.where(ok, page, 0), t % PAGE
    codes, scale, rope = unpack(blocks[at, layer])
    i = np.arange(len(t))
    s = np.where(ok, bits_value(scale[i, line]), 1.0)
    rows = np.concatenate([E4M3[codes[i, line]], bits_value(rope[i, line])], -1) * s[:, None]
    return np.where(ok[:, None], rows, 0.0), s


def attend(q_abs, rows, w_kv_b, scale):
    """One token row over the rows it sees: (out [96, 128], o_lat [96, 512], p [96, T])."""
    if len(rows) == 0:
        return np.zeros((H, V)), np.zeros((H, LORA)), np.zeros((H, 0))
    s = np.asarray(q_abs, np.float64) @ rows.T * scale
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    o = p @ rows[:, :LORA]
    w_uv = np.asarray(w_kv_b, np.float64).reshape(H, NOPE + V, LORA)[:, NOPE:]
    return np.einsum("hvk,hk->hv", w_uv, o), o, p


def out_tolerance(q_abs, out, o, p, rows, scales, w_kv_b, scale):
    """Bound of |kernel - reference| for one token row, element by element.

    What the kernel rounds:
      * p times its row's power of two (so that it can multiply codes) to a sum of two e4m3 numbers, the second in units of
        1/32: the first is within 2^-4 of it, the rest within 2^-4 of that, 2^-8 in all, by way of an f16 (2^-12); or, where
        the second is below its smallest step, within half a step, 2^-10 / 32 = 2^-15, and half the f16's, 2^-17, when the
        largest of them comes to 2 at least (the reference is one of them, and they are taken to 2 at the reference):
        1.25 * 2^-16 of it;
      * q to a sum of two e4m3 numbers likewise: exact for entries above 2^-14 of the largest of all heads, as a bf16 has 8
        bits, else within 2^-15, and half the step of the f16 it goes through (2^-24 at 2^-8 of it: 2^-17), where the largest
        comes to 2^7 at least: 1.25 * 2^-22 of it;
      * o_lat, and the O of each split, to f16 after a power of two (2^-12 of the entry or 2^-25 of the row's largest);
      * the output to bf16 (2^-8);
      * f32 sums besides: each score within 640 * 2^-24 of sum |q||row| * scale, the hardware exponential 2^-21, the sums
        over tokens and latent entries 2^-15 in all.
    Scores that are off by e_t, |e_t| <= ds_t, multiply each weight by exp(e_t):
        o' - o = sum_t p_t (exp(e_t) - 1) (row_t - o) / sum_t p_t exp(e_t),
    and with weights that are off by r_t of themselves besides, exp(e_t) (1 + r_t) for exp(e_t): so with d_t = p_t (exp(ds_t)
    (1 + r_t) - 1) it is at most sum_t d_t |row_t - o| / sum_t p_t exp(-ds_t) (1 - r_t), here taken through |W_UV|.  (For small
    ds_t that is p_t (ds_t + r_t) over 1.)"""
    w = np.abs(np.asarray(w_kv_b, np.float64).reshape(H, NOPE + V, LORA)[:, NOPE:])
    if p.shape[1] == 0:
        return np.zeros_like(out)
    q = np.abs(np.asarray(q_abs, np.float64))
    ds = scale * (640 * 2.0 ** -24 * q @ np.abs(rows).T + 1.25 * 2.0 ** -22 * q[:, :LORA].max() * np.abs(rows[:, :LORA]).sum(-1))
    size, r, ds = p * scales, 2.0 ** -8 + 2.0 ** -12 + 2.0 ** -19, np.minimum(ds, 300)
    d = p * (np.expm1(ds) * (1 + r) + r) + np.exp(ds) * 1.25 * 2.0 ** -16 * size.max(-1, keepdims=True) / scales
    c = np.abs(rows[:, :LORA])
    spread = (d @ c + d.sum(-1)[:, None] * np.abs(o)) / ((p * np.exp(-ds)).sum(-1)[:, None] * (1 - r))
    mass = p @ c
    half = 2 * (2.0 ** -12 * mass + 2.0 ** -25 * mass.max(-1, keepdims=True))
    return (np.einsum("hvk,hk->hv", w, spread + half + 2.0 ** -15 * mass) + 2.0 ** -8 * np.abs(out)) * 1.01 + 1e-30
