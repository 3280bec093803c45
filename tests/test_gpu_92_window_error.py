"""Windowed decode and chunks over long windows, each row as a whole against the 64-bit definition (window_error.py):
a token too many or too few, a lost split or a scale that is off shows there where it is within the bound of every
element."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests import window_error, window_ref as ref
from tests.test_gpu_87_window import SCALE, Case, f64, rows_to, seen_sets

pytestmark = pytest.mark.gpu


def check(c, got, slot, n, window, sink, rows):
    got, q, w, slab = f64(got), f64(c.q), f64(c.w), f64(c.slab[:, c.layer:c.layer + 1])
    for r in rows:
        out = ref.attend(q[r], slab, 0, c.table[slot[r]], n[r], window, sink, w, SCALE)[0]
        row, heads = window_error.relative(got[r], out)
        assert row <= window_error.ROW_BOUND and np.all(heads <= window_error.HEAD_BOUND), (r, n[r], row, heads.max())


@pytest.mark.parametrize("lens,window,sink,splits", [
    ([2000, 1100, 1024, 1000, 65, 1], 1024, 64, (0, 128, 256)), ([9000, 5000, 4096, 130], 4500, 100, (0, 128, 1024)),
    ([700, 301, 300, 299], 300, 1, (0, 128)), ([130, 64, 65, 200], 64, 4, (0, 128)), ([5000, 900], 10 ** 6, 0, (0, 128))])
def test_decode(gpu_lib, lens, window, sink, splits):
    c = Case(100 + window % 97, lens, len(lens))
    c.poison(seen_sets(lens, window, sink))
    for split in (*splits, k3mla.window_split_tokens(len(lens), c.max_ctx, window, sink)):
        check(c, c.decode(window, sink, split), range(len(lens)), lens, window, sink, range(len(lens)))
    assert c.err.item() == 0


def test_decode_of_a_batch(gpu_lib):
    lens = [4096 - 7 * b for b in range(64)]
    c = Case(101, lens, 64)
    check(c, c.decode(1024, 64), range(64), lens, 1024, 64, range(0, 64, 5))
    assert c.err.item() == 0


@pytest.mark.parametrize("lens,new,window,sink", [([2000, 1030, 300], [64, 30, 300], 1024, 64), ([700], [700], 300, 1),
                                                  ([4700, 4501], [9, 5], 4500, 100), ([200, 130], [70, 130], 64, 4)])
def test_chunk(gpu_lib, lens, new, window, sink):
    R = sum(new)
    c = Case(102 + window % 97, lens, R)
    pos0, start = [n - m for n, m in zip(lens, new)], np.concatenate([[0], np.cumsum(new)])
    slot, n = rows_to(start, pos0, R)
    check(c, c.chunk(pos0, start, window, sink), slot, n, window, sink, [*range(0, R, max(1, R // 12)), R - 1])
    assert c.err.item() == 0
