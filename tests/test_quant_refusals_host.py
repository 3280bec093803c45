"""What the calls on the 8-bit cache refuse before anything is launched (no GPU needed)."""
from __future__ import annotations

import types

import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_window_refusals_host import fake

INVALID, WORKSPACE = -1, -6
P = 1 << 20      # an address that is never used


def decode(lib, **kw):
    a = dict(q=P, slab=P, n_pages=4, layers=2, layer=1, table=P, cols=4, ctx=P, w=P, scale=0x3D94, out=P, ws=P, ws_bytes=1 << 40,
             B=2, max_ctx=256, window=256, sink=0, split=0)
    a.update(kw)
    return lib.k3mla_quant_decode(a["q"], a["slab"], a["n_pages"], a["layers"], a["layer"], a["table"], a["cols"], a["ctx"],
                                  a["w"], a["scale"], a["out"], a["ws"], a["ws_bytes"], a["B"], a["max_ctx"], a["window"],
                                  a["sink"], a["split"], None, None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(n_pages=0), dict(layers=0), dict(layer=2), dict(layer=-1), dict(cols=0), dict(max_ctx=0), dict(window=0),
    dict(sink=-1), dict(split=-128), dict(split=100), dict(scale=0), dict(scale=0x8000), dict(scale=0x7F80), dict(scale=0x7F32),
    dict(q=None), dict(slab=None), dict(table=None), dict(ctx=None), dict(w=None), dict(out=None), dict(ws=None), dict(q=P + 8),
    dict(slab=P + 64), dict(w=P + 8), dict(out=P + 8), dict(ws=P + 128), dict(n_pages=1 << 30, layers=2, layer=0),
    dict(B=65536), dict(B=60000, max_ctx=1 << 20, cols=1 << 14, window=1 << 30, split=128, ws_bytes=1 << 60),
    dict(max_ctx=(1 << 25) + 64, cols=(1 << 19) + 1, window=1 << 30, split=1 << 26)])
def test_decode_refuses(kw):
    lib = k3mla.load()
    assert decode(lib, **kw) == INVALID
    assert lib.k3mla_last_error().startswith(b"k3mla_quant_decode: ")


def test_decode_wants_its_workspace_and_does_nothing_for_no_slots():
    lib = k3mla.load()
    need = k3mla.quant_decode_workspace_bytes(2, 256, 256)
    assert need > 0 and decode(lib, ws_bytes=need - 1) == WORKSPACE
    assert decode(lib, B=0, q=None, slab=None) == 0
    assert k3mla.quant_decode_workspace_bytes(0, 256, 256) == 0
    assert k3mla.quant_decode_workspace_bytes(1, 256, 0) == 0
    assert k3mla.quant_decode_workspace_bytes(1, 256, 1, 0, 100) == 0
    assert k3mla.quant_decode_workspace_bytes(3, 5000, 5000, 0, 128) > k3mla.quant_decode_workspace_bytes(3, 5000, 5000)
    assert k3mla.quant_split_tokens(1, 32768, 1 << 30) % 128 == 0


@pytest.mark.parametrize("sizes", [(1, 1, 1, 0), (5, 500, 500, 0), (40, 30000, 1 << 30, 0), (90, 30000, 4096, 64),
                                   (65535, 1 << 30, 1 << 30, 5), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_planned_splits_are_splits(sizes):
    split = k3mla.quant_split_tokens(*sizes)
    assert split > 0 and split % 128 == 0 and (sizes[0] <= 4 or split <= 1 << 25)


@pytest.mark.parametrize("call", ["k3mla_quant_write_pages", "k3mla_quant_read_pages", "k3mla_quant_copy_pages"])
def test_page_calls_refuse(call):
    f = getattr(k3mla.load(), call)
    for args in ((P, 0, P, 1, 1, P, P, 1), (P, 1, P, 0, 1, P, P, 1), (P, 1, P, 1, 0, P, P, 1), (P, 1, P, 1, 1, P, P, -1),
                 (P, 1, P, 1, 1, P, P, 65536), (None, 1, P, 1, 1, P, P, 1), (P, 1, None, 1, 1, P, P, 1), (P, 1, P, 1, 1, None, P, 1),
                 (P, 1, P, 1, 1, P, None, 1), (P + 8, 1, P, 1, 1, P, P, 1), (P, 1, P + 4, 1, 1, P, P, 1)):
        assert f(*args, None, None) == INVALID, args
        assert k3mla.load().k3mla_last_error().startswith(call.encode())
    assert f(None, 1, None, 1, 1, None, None, 0, None, None) == 0


def test_append_refuses_like_the_bf16_call():
    lib = k3mla.load()

    def call(slab=P, stride=512, R=2, layer=0, q_out=P):
        return lib.k3mla_quant_norm_rope_append(P, q_out, None, slab, 4, 1, layer, P, 4, P, None, None, P, stride, None, P, 64, None,
                                                1e-6, None, 0, 2, R, None, None)
    for kw in (dict(slab=None), dict(slab=P + 8), dict(stride=500), dict(stride=516), dict(R=3), dict(layer=1), dict(q_out=P + 32)):
        assert call(**kw) == INVALID, kw
        assert lib.k3mla_last_error().startswith(b"k3mla_quant_norm_rope_append: ")


def test_binding_refuses_wrong_tensors(monkeypatch):
    monkeypatch.setattr(k3mla, "_current_device", lambda: 0)
    i32, u8 = torch.int32, torch.uint8
    stream = types.SimpleNamespace(cuda_stream=0)
    q, slab, table, ctx = fake(1, 96, 576), fake(2, 1, 41088, dtype=u8), fake(1, 2, dtype=i32), fake(1, dtype=i32)
    w, out, ws, ids = fake(24576, 512), fake(1, 96, 128), fake(1 << 20, dtype=u8), fake(1, dtype=i32)

    def decode(slab=slab, q=q, layer=0, **kw):
        k3mla.quant_decode(q, slab, layer, table, ctx, w, 0x3D94, out, ws, 128, stream=stream, **kw)
    for kw in (dict(slab=fake(2, 1, 64, 576)), dict(slab=fake(2, 1, 41080, dtype=u8)), dict(slab=fake(2, 1, 41088, dtype=torch.int8)),
               dict(q=fake(1, 96, 512)), dict(layer=2 ** 32), dict(window=2 ** 31), dict(split_tokens=2 ** 32)):
        with pytest.raises(k3mla.K3mlaError):
            decode(**kw)
    for f, dst, src in ((k3mla.quant_write_pages, fake(2, 1, 64, 576), slab), (k3mla.quant_read_pages, slab, slab),
                        (k3mla.quant_write_pages, slab, fake(2, 2, 64, 576)), (k3mla.quant_copy_pages, slab, fake(2, 1, 64, 576)),
                        (k3mla.quant_write_pages, slab, fake(2, 1, 64, 576).transpose(0, 1))):
        with pytest.raises(k3mla.K3mlaError):
            f(dst, src, ids, ids, stream=stream)
    with pytest.raises(k3mla.K3mlaError):
        k3mla.quant_norm_rope_append(fake(1, 96, 192), fake(1, 96, 192), fake(2, 1, 64, 576), 0, table, ctx, None, fake(1, 512),
                                     fake(1, 64), stream=stream)
