"""Arguments of the windowed operators that the library or the binding used to take for something else (no GPU needed)."""
from __future__ import annotations

import pytest

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_window_host import chunk, decode


@pytest.mark.parametrize("call", [decode, chunk])
@pytest.mark.parametrize("scale", [0x7F32, 0x7F7F])
def test_a_scale_whose_product_with_log2e_is_infinite_is_refused(call, scale):
    lib = k3mla.load()
    assert call(lib, scale=scale) == -1
    assert b"scale" in lib.k3mla_last_error()
