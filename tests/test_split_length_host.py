"""Split lengths and contexts near 2^31: the split counts that size the workspaces and the grids (no GPU needed)."""
from __future__ import annotations

import pytest

from paged_latent_attention_k3mla_gb300 import k3mla

NEAR = 2 ** 31 - 128                     # the longest split that is a multiple of 128


def up(x):
    return -(-x // 256) * 256


@pytest.mark.parametrize("max_ctx", [1, 4096, 2 ** 31 - 129, 2 ** 31 - 128])
def test_a_split_as_long_as_an_int_holds_is_one_split(max_ctx):
    want = up(2 * 96 * 512 * 2) + 2 * 1 * 96 * 16          # o_lat, one record a slot and head
    assert k3mla.decode_workspace_bytes(2, max_ctx, NEAR) == want
    assert k3mla.slot_split_tokens(max_ctx, NEAR) == NEAR


@pytest.mark.parametrize("max_ctx", [2 ** 31 - 4096, 2 ** 31 - 4000, 2 ** 31 - 1])
def test_contexts_as_long_as_an_int_holds_are_cut_by_the_default_rule(max_ctx):
    ns = -(-max_ctx // 4096)
    per = -(-max_ctx // ns)
    assert k3mla.slot_split_tokens(max_ctx) == -(-per // 128) * 128 == 4096
    assert k3mla.decode_workspace_bytes(1, max_ctx) == up(96 * 512 * 2) + up(ns * 96 * 512 * 4) + ns * 96 * 16
    # the windowed call counts its list of pages, which is held below 2^31 - 256 tokens
    ns = -(-min(-(-max_ctx // 64) * 64, 2 ** 31 - 256) // 4096)
    rec = ns * 96
    want = up(96 * 512 * 2) + up(96 * 4) + up(rec * 512 * 2) + up(rec * 4) + up(rec * 8)
    assert k3mla.window_decode_workspace_bytes(1, max_ctx, max_ctx) == want
