"""Arguments of the windowed operators that the library or the binding used to take for something else (no GPU needed)."""
from __future__ import annotations

import types

import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_window_host import chunk, decode


@pytest.mark.parametrize("call", [decode, chunk])
@pytest.mark.parametrize("scale", [0x7F32, 0x7F7F])
def test_a_scale_whose_product_with_log2e_is_infinite_is_refused(call, scale):
    lib = k3mla.load()
    assert call(lib, scale=scale) == -1
    assert b"scale" in lib.k3mla_last_error()


class OnDevice(torch.Tensor):
    """A CPU tensor that says it lies on device 0: enough for the checks of the binding, which come before any use."""
    is_cuda = True

    def get_device(self):
        return 0


def fake(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def calls():
    i32 = torch.int32
    slab, table, w = fake(2, 2, 64, 576), fake(1, 2, dtype=i32), fake(24576, 512)
    pos, start, ws, err = fake(1, dtype=i32), fake(2, dtype=i32), fake(1 << 20, dtype=torch.uint8), fake(1, dtype=i32)
    q, qa, kv, out = fake(1, 96, 192), fake(1, 96, 576), fake(1, 576), fake(1, 96, 128)
    stream = types.SimpleNamespace(cuda_stream=0)
    return {
        "norm_rope_append": lambda layer, scale: k3mla.norm_rope_append(q, q, slab, layer, table, pos, None, kv[:, :512],
                                                                        kv[:, 512:], stream=stream),
        "window_decode": lambda layer, scale: k3mla.window_decode(qa, slab, layer, table, pos, w, scale, out, ws, 128, 10,
                                                                  stream=stream),
        "window_chunk_decode": lambda layer, scale: k3mla.window_chunk_decode(qa, slab, layer, table, pos, start, w, scale,
                                                                              out, ws, 128, 10, stream=stream),
        "paged_decode": lambda layer, scale: k3mla.paged_decode(qa, slab, layer, table, pos, w, scale, out, ws, 128,
                                                                stream=stream),
        "append_latent": lambda layer, scale: k3mla.append_latent(slab, layer, table, pos, kv[:, :512], kv[:, 512:],
                                                                  stream=stream),
        "diag_window_timeout": lambda layer, scale: k3mla.diag_window_timeout(qa, slab, layer, table, pos, w, scale, out, ws,
                                                                              128, 10, 0, 0, 1, 2000, err, stream=stream),
    }


@pytest.mark.parametrize("name", sorted(calls()))
@pytest.mark.parametrize("layer", [2 ** 32, 2 ** 32 + 1, -2 ** 32])
def test_a_layer_past_32_bits_is_refused(monkeypatch, name, layer):
    monkeypatch.setattr(k3mla, "_current_device", lambda: 0)
    with pytest.raises(k3mla.K3mlaError, match="layer = .* does not fit 32 bits"):
        calls()[name](layer, 0x3D94)


@pytest.mark.parametrize("name", ["window_decode", "window_chunk_decode", "paged_decode", "diag_window_timeout"])
@pytest.mark.parametrize("scale", [0x13D94, -1, 2 ** 32 + 0x3D94])
def test_a_scale_of_more_than_16_bits_is_refused(monkeypatch, name, scale):
    monkeypatch.setattr(k3mla, "_current_device", lambda: 0)
    with pytest.raises(k3mla.K3mlaError, match="bit pattern"):
        calls()[name](0, scale)


def test_a_context_past_32_bits_is_refused():
    far = 2 ** 32 + 4096
    for call in (lambda: k3mla.decode_workspace_bytes(1, far), lambda: k3mla.decode_layer_workspace_bytes(1, far),
                 lambda: k3mla.decode_exact_workspace_bytes(1, far), lambda: k3mla.chunk_decode_workspace_bytes(1, 1, far),
                 lambda: k3mla.slot_split_tokens(far), lambda: k3mla.batch_planned_split_tokens([5], far)):
        with pytest.raises(k3mla.K3mlaError, match="32 bits"):
            call()


def test_a_shape_may_be_any_sequence():
    t = fake(2, 3)
    for shape in ((2, 3), [2, 3], torch.Size([2, 3]), None):
        assert k3mla._dev(t, torch.bfloat16, shape, "t") == t.data_ptr()
        assert k3mla._at(0, t, torch.bfloat16, shape, "t") == t.data_ptr()
        with pytest.raises(k3mla.K3mlaError, match="runs on cuda:1"):
            k3mla._at(1, t, torch.bfloat16, shape, "t")
    for shape in ((3, 2), [3, 2], [2], ()):
        with pytest.raises(k3mla.K3mlaError, match="has shape"):
            k3mla._dev(t, torch.bfloat16, shape, "t")
        with pytest.raises(k3mla.K3mlaError, match="has shape"):
            k3mla._at(0, t, torch.bfloat16, shape, "t")


def test_a_unit_of_more_pages_than_the_waits_allow_is_refused():
    # 2^19 pages of a list in one unit: about half a second of the one that a wait lasts
    lib, n, cols = k3mla.load(), 2 ** 26, 2 ** 20
    for change in (dict(split=2 ** 26), dict(split=2 ** 31 - 128), dict(split=2 ** 25 + 128, window=2 ** 25, sink=64)):
        assert decode(lib, **{**dict(max_ctx=n, cols=cols, window=n, sink=0), **change}) == -1
        assert b"pages in one unit" in lib.k3mla_last_error()
    for change in (dict(window=n), dict(window=2 ** 31 - 1, sink=2 ** 31 - 1), dict(window=2 ** 25, sink=0)):
        assert chunk(lib, **{**dict(max_ctx=n, cols=cols), **change}) == -1
        assert b"pages in one unit" in lib.k3mla_last_error()
