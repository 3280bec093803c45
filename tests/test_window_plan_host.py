"""k3mla_window_split_tokens: how long the splits of few slots may become for the expansion's sake (no GPU needed)."""
from __future__ import annotations

import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla

H, PAGE, TILE = 96, 64, 128
# the library's count where there is no device: 148
SMS = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148


def pages(B, max_ctx, window, sink, sms):
    """Pages of a split when sms SMs share the slots' lists, a pair a split."""
    most = min(-(-max_ctx // PAGE), -(-min(sink, max_ctx) // PAGE) + (min(window, max_ctx) + PAGE - 2) // PAGE + 1)
    tiles = -(-most * PAGE // TILE)
    return -(-tiles // max(1, sms // 2 // B)) * (TILE // PAGE)


@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 8, 39, 75, 76, 500])
@pytest.mark.parametrize("window", [1, 300, 1000, 2000, 4096, 8192, 16384, 32768, 131072, 2 ** 31 - 1])
def test_splits_are_at_most_six_pages_longer_than_on_the_whole_machine(B, window):
    for max_ctx in (window, 32768, 10 ** 6):
        for sink in (0, 4, 1000):
            full = pages(B, max_ctx, window, sink, SMS)
            got = k3mla.window_split_tokens(B, max_ctx, window, sink)
            assert got % TILE == 0 and got >= TILE
            if B in (2, 3, 4):
                left = pages(B, max_ctx, window, sink, SMS - H)
                assert got // PAGE == (left if left - full <= 6 else full)
            else:
                assert got // PAGE == min(full, (2 ** 31 - 1) // TILE * TILE // PAGE)
