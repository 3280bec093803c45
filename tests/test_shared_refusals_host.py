"""What the decode for shared prefixes refuses before anything is launched (no GPU needed), and its planning."""
from __future__ import annotations

import types

import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_window_refusals_host import fake

INVALID, WORKSPACE = -1, -6
P = 1 << 20      # an address that is never used


def decode(lib, **kw):
    a = dict(q=P, slab=P, n_pages=4, layers=2, layer=1, table=P, cols=4, ctx=P, start=P, shared=P, G=2, w=P, scale=0x3D94, out=P, ws=P,
             ws_bytes=1 << 60, B=3, max_shared=128, max_own=128, shared_split=0, own_split=0)
    a.update(kw)
    return lib.k3mla_shared_decode(a["q"], a["slab"], a["n_pages"], a["layers"], a["layer"], a["table"], a["cols"], a["ctx"], a["start"],
                                   a["shared"], a["G"], a["w"], a["scale"], a["out"], a["ws"], a["ws_bytes"], a["B"],
                                   a["max_shared"], a["max_own"], a["shared_split"], a["own_split"], None, None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(G=-1), dict(n_pages=0), dict(layers=0), dict(layer=2), dict(layer=-1), dict(cols=0), dict(max_shared=-1),
    dict(max_own=0), dict(shared_split=-2), dict(own_split=-1), dict(shared_split=-128),
    dict(shared_split=64), dict(own_split=-128), dict(own_split=100), dict(scale=0),
    dict(scale=0x8000), dict(scale=0x7F80), dict(scale=0x7F32), dict(q=None), dict(slab=None), dict(table=None), dict(ctx=None),
    dict(start=None), dict(shared=None), dict(w=None), dict(out=None), dict(ws=None), dict(q=P + 8), dict(slab=P + 8), dict(w=P + 8),
    dict(out=P + 8), dict(ws=P + 128), dict(B=65536), dict(G=(1 << 20) + 1), dict(n_pages=1 << 25, layers=1, layer=0),
    dict(B=60000, max_own=1 << 20, own_split=128), dict(max_shared=(1 << 25) + 64, shared_split=1 << 26),
    dict(max_own=(1 << 25) + 64, own_split=1 << 26), dict(max_shared=1 << 25, max_own=64, shared_split=-1, own_split=1 << 26),
    dict(B=60000, max_shared=1 << 20, shared_split=-1, own_split=128)])
def test_refused(kw):
    lib = k3mla.load()
    assert decode(lib, **kw) == INVALID
    assert lib.k3mla_last_error().startswith(b"k3mla_shared_decode: ")


def test_workspace_and_no_slots():
    lib = k3mla.load()
    need = k3mla.shared_decode_workspace_bytes(3, 128, 128)
    assert need > 0 and decode(lib, ws_bytes=need - 1) == WORKSPACE
    assert decode(lib, B=0, q=None) == 0
    for bad in ((0, 1, 1), (1, -1, 1), (1, 1, 0), (1, 1, 1, 100), (1, 1, 1, 0, -128)):
        assert k3mla.shared_decode_workspace_bytes(*bad) == 0
    assert k3mla.shared_decode_workspace_bytes(2, 4096, 64, 128) > k3mla.shared_decode_workspace_bytes(2, 4096, 64)
    assert k3mla.shared_decode_workspace_bytes(2, 2 ** 31 - 1, 2 ** 31 - 1) > 0
    assert k3mla.shared_decode_workspace_bytes(2, 2 ** 31 - 1, 2 ** 31 - 1, -1) > 0


@pytest.mark.parametrize("sizes", [(1, 0, 0, 1), (1, 1, 64, 1), (8, 1, 4096, 64), (64, 64, 100, 5000), (64, 1, 16384, 600),
                                   (65535, 1, 2 ** 31 - 1, 2 ** 31 - 1), (0, 0, 0, 0)])
def test_planned_splits_are_splits(sizes):
    shared, own = k3mla.shared_split_tokens(*sizes)
    assert (shared == k3mla.SHARED_NONE or shared > 0 and shared % 128 == 0) and own > 0 and own % 128 == 0
    assert k3mla.load().k3mla_shared_split_tokens(*sizes, None) == shared


def test_binding_refuses_wrong_tensors(monkeypatch):
    monkeypatch.setattr(k3mla, "_current_device", lambda: 0)
    i32 = torch.int32
    good = dict(q_abs=fake(2, 96, 576), slab=fake(2, 1, 64, 576), layer=0, block_table=fake(2, 2, dtype=i32), ctx_len=fake(2, dtype=i32),
                group_start=fake(2, dtype=i32), shared_len=fake(1, dtype=i32), w_kv_b=fake(24576, 512), scale_bf16=0x3D94,
                out=fake(2, 96, 128), workspace=fake(1 << 20, dtype=torch.uint8), max_shared=64, max_own=64,
                stream=types.SimpleNamespace(cuda_stream=0))
    for kw in (dict(group_start=fake(1, dtype=i32)), dict(group_start=fake(2, dtype=torch.int64)), dict(ctx_len=fake(3, dtype=i32)),
               dict(slab=fake(2, 1, 41088, dtype=torch.uint8)), dict(out=fake(2, 96, 64)), dict(layer=2 ** 32), dict(max_own=2 ** 31),
               dict(own_split=2 ** 32), dict(q_abs=fake(96, 2, 576).transpose(0, 1)), dict(scale_bf16=1 << 16)):
        with pytest.raises(k3mla.K3mlaError):
            k3mla.shared_decode(**{**good, **kw})
