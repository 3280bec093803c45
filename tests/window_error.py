"""How far an output of the windowed attention is from the 64-bit definition as a whole (tests only), beside the bound of
every element in window_ref: that one adds all roundings with one sign, so where a window is long, and the outputs small,
it lets a window that is a page short pass, or one without its first tokens.

The roundings that show are two, each to bf16: p, and the output.  A relative error of such a rounding is spread evenly
over at most +-2^-8 (at a mantissa of 1; less above), 2^-8 / sqrt(3) = 0.00226 in the mean square.  The output's error is
that share of the output.  p's error moves the output by sum_t p_t d_t W row_t: with rows of independent entries these add
up like the output sum_t p_t W row_t itself does, so it is that share of the output again.  o_lat and a split's O in f16
add 2^-11 / sqrt(3) = 0.00028 each, f32 sums and exponentials less than 2^-15.  Together at most
sqrt(2 * 0.00226^2 + 2 * 0.00028^2) = 0.0032 of a row of 96 heads (random signs leave nothing of a mean over 12,288
entries); ROW_BOUND allows a tenth more.  A head alone has 128 entries and may have a few tokens that matter, so nothing
averages out: 2^-8 from each of the two, 0.0078, and 15 % for rows that are not quite orthogonal in 128 dimensions."""
from __future__ import annotations

import numpy as np

ROW_BOUND, HEAD_BOUND = 0.0035, 0.009


def relative(got, out):
    """(of the row, per head): the distance of got [96, 128] from out, relative to out."""
    e, n = np.linalg.norm(got - out, axis=-1), np.linalg.norm(out, axis=-1)
    return float(np.linalg.norm(e) / np.linalg.norm(n)), e / n


def accepts(got, out) -> bool:
    row, heads = relative(got, out)
    return bool(row <= ROW_BOUND and np.all(heads <= HEAD_BOUND))
