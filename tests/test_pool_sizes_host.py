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


def test_pool_arguments_past_32_bits_are_refused():
    pool, far = k3mla.Pool(n_slots=2, max_ctx=128), 2 ** 32
    for call in (lambda: k3mla.Pool(far + 1, 128), lambda: k3mla.Pool(1, far + 128), lambda: k3mla.Pool(1, 128, far + 1),
                 lambda: pool.ensure(far, 64), lambda: pool.ensure(0, far + 64), lambda: pool.release(far),
                 lambda: pool.share_prefix(far + 1, 0, 0), lambda: pool.share_prefix(1, far, 0),
                 lambda: pool.share_prefix(1, 0, far), lambda: pool.cow(far, 0), lambda: pool.cow(0, far),
                 lambda: pool.refs(far), lambda: k3mla.expanded_cache_bytes(far + 1)):
        with pytest.raises(k3mla.K3mlaError, match="32 bits"):
            call()
    assert pool.stats() == (4, 0)
    pool.close()
