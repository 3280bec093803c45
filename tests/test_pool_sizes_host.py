"""Pools whose sizes are near 2^31 (no GPU needed)."""
from __future__ import annotations

import pytest

from paged_latent_attention_k3mla_gb300 import k3mla


@pytest.mark.parametrize("slots,max_ctx", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 64)])
def test_a_pool_too_large_for_memory_is_refused(slots, max_ctx):
    # its table alone would be 2^58 bytes, more than any address space
    with pytest.raises(k3mla.K3mlaError):
        k3mla.Pool(n_slots=slots, max_ctx=max_ctx, n_pages=1)


def test_contexts_as_long_as_an_int_holds():
    pool = k3mla.Pool(n_slots=1, max_ctx=2 ** 31 - 1, n_pages=3)
    assert pool.max_pages == 2 ** 25
    assert pool.ensure(0, 2 ** 31 - 1) == -2 and pool.ensure(0, 129) == 0 and pool.stats() == (3, 3)
    assert pool.trim(0, 2 ** 31 - 1, 1, 0) == 3 and pool.stats() == (3, 0)
    pool.close()
