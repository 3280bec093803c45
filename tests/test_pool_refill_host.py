"""k3mla_pool_refill: the holes of a trimmed slot get pages again, so that kept rows can move there (no GPU needed)."""
from __future__ import annotations

import numpy as np
import pytest

from paged_latent_attention_k3mla_gb300 import k3mla


def test_refill_maps_the_holes_that_the_kept_rows_move_to():
    pool = k3mla.Pool(n_slots=2, max_ctx=1024, n_pages=16)
    assert pool.ensure(0, 600) == 0 and pool.trim(0, 600, 200, 65) == 4      # holes at pages 2 .. 5
    before, used = pool.table()[0].copy(), pool.stats()[1]
    assert pool.refill(0, 128) == 0 and np.array_equal(pool.table()[0], before)
    assert pool.refill(0, 265) == 3                                           # 65 + 200 rows: pages 0 .. 4
    t = pool.table()[0]
    assert np.all(t[2:5] >= 0) and t[5] == -1 and pool.stats()[1] == used + 3
    assert np.array_equal(t[[0, 1, 6, 7, 8, 9]], before[[0, 1, 6, 7, 8, 9]])
    assert len(set(t[t >= 0].tolist())) == (t >= 0).sum() and all(pool.refs(int(p)) == 1 for p in t[t >= 0])
    assert pool.cow(0, 130) is None                                           # a position there can be written again
    assert pool.refill(0, 265) == 0
    assert pool.truncate(0, 265) == 0 and pool.stats()[1] == 5
    assert pool.ensure(0, 266) == 0 and pool.ensure(0, 400) == 0 and pool.stats()[1] == 7
    assert pool.release(0) == 0 and pool.stats() == (16, 0) and all(pool.refs(p) == 0 for p in range(16))
    pool.close()


def test_refill_is_all_or_nothing_and_stays_inside_the_slot():
    pool = k3mla.Pool(n_slots=2, max_ctx=1024, n_pages=12)
    assert pool.ensure(0, 600) == 0 and pool.trim(0, 600, 64, 0) == 8 and pool.ensure(1, 64 * 7) == 0   # 3 free
    before = pool.table().copy()
    assert pool.refill(0, 600) == -2 and pool.refill(0, 256) == -2
    assert np.array_equal(pool.table(), before) and pool.stats() == (12, 9)
    assert pool.refill(0, 192) == 3 and pool.stats() == (12, 12)
    assert pool.refill(1, 1024) == 0                                          # nothing past what the slot maps
    assert np.array_equal(pool.table()[1], before[1])
    assert pool.refill(2, 1) == -3 and pool.refill(-1, 1) == -3 and pool.refill(0, 1025) == -4 and pool.refill(0, -1) == -1
    assert k3mla.load().k3mla_pool_refill(None, 0, 1) == -1
    with pytest.raises(k3mla.K3mlaError, match="32 bits"):
        pool.refill(0, 2 ** 32)
    pool.close()
