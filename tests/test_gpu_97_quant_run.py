"""The operators of the 8-bit cache one after the other: a step captured and replayed, and pages behind 4 GB."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
H, V, LORA, PAGE, ROW = 96, 128, 512, 64, 576
SCALE_BITS = 0x3D94


def step(k3, st, stream=None):
    """Rows appended at the slots' last positions, queries absorbed, the slots attended to."""
    k3.quant_norm_rope_append(st["q"], st["q_out"], st["slab"], st["layer"], st["table"], st["pos"], None, st["kv"][:, :LORA],
                              st["kv"][:, LORA:], inv_freq=st["inv"], stream=stream)
    k3.absorb_q(st["q_out"], st["w"], st["q_abs"], stream=stream)
    k3.quant_decode(st["q_abs"], st["slab"], st["layer"], st["table"], st["ctx"], st["w"], SCALE_BITS, st["out"], st["ws"],
                    st["max_ctx"], split_tokens=128, stream=stream)


def state(k3, ctx, pages, table, layers, layer, seed):
    """A bf16 cache of rows for the pages that the table names, quantised into a slab of `pages` pages, and a step's inputs."""
    B, gen = len(ctx), torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    named = [int(p) for p in table.flatten() if p >= 0]
    rows = rand(len(named), layers, PAGE, ROW).bfloat16()
    slab = torch.empty(pages, layers, k3.QUANT_PAGE_BYTES, dtype=torch.uint8, device="cuda")
    src = torch.arange(len(named), dtype=torch.int32, device="cuda")
    dst = torch.tensor(named, dtype=torch.int32, device="cuda")
    k3.quant_write_pages(slab, rows, src, dst)
    ctx_len = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    return dict(q=rand(B, H, 192).bfloat16(), q_out=torch.empty(B, H, 192, dtype=torch.bfloat16, device="cuda"), slab=slab, layer=layer,
                table=torch.from_numpy(table).cuda(), pos=ctx_len - 1, ctx=ctx_len, kv=rand(B, ROW).bfloat16(),
                inv=(10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda(),
                w=(rand(H * 256, LORA) * LORA ** -0.5).bfloat16(), q_abs=torch.empty(B, H, ROW, dtype=torch.bfloat16, device="cuda"),
                out=torch.empty(B, H, V, dtype=torch.bfloat16, device="cuda"), max_ctx=max(ctx),
                ws=torch.empty(k3.quant_decode_workspace_bytes(B, max(ctx), max(ctx), 0, 128), dtype=torch.uint8, device="cuda"),
                ids=(src, dst))


TABLE = np.array([[3, 0, 7, 5], [1, -1, -1, -1], [4, 6, 2, -1]], np.int32)
CTX = [250, 1, 130]


def test_a_step_captured_and_replayed_on_another_stream(gpu_lib):
    k3 = gpu_lib
    st = state(k3, CTX, 8, TABLE, 2, 1, 1)
    clean = st["slab"].clone()
    step(k3, st)
    torch.cuda.synchronize()
    want, slab = st["out"].clone(), st["slab"].clone()
    assert torch.equal(slab[:, 0], clean[:, 0]) and not torch.equal(slab[:, 1], clean[:, 1])
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(k3, st)
    for _ in range(3):
        st["slab"].copy_(clean)
        st["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(st["out"], want) and torch.equal(st["slab"], slab)
    with torch.cuda.stream(s):                                # and eager, on that stream
        st["slab"].copy_(clean)
        step(k3, st)
    s.synchronize()
    assert torch.equal(st["out"], want) and torch.equal(st["slab"], slab)


def test_pages_behind_four_gigabytes(gpu_lib):
    """The same pages at the end of a slab of 4.5 GB: every operator gives the bits of the small one."""
    k3 = gpu_lib
    small, many = state(k3, CTX, 8, TABLE, 1, 0, 2), 110000
    far = np.array([104529, 109999, 54000, 104530, 104531, 60000, 109998, 104532], np.int32)   # (2^32 bytes are 104,530.7 pages)
    big = state(k3, CTX, many, np.where(TABLE < 0, -1, far[TABLE]).astype(np.int32), 1, 0, 2)
    for st in (small, big):
        step(k3, st)
    torch.cuda.synchronize()
    assert not small["out"].isnan().any() and torch.equal(small["out"], big["out"])
    where = torch.from_numpy(far).long().cuda()
    assert torch.equal(big["slab"][where], small["slab"])
    back = [torch.zeros(8, 1, PAGE, ROW, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for st, rows in zip((small, big), back):
        k3.quant_read_pages(rows, st["slab"], st["ids"][1], st["ids"][0])
    k3.quant_copy_pages(big["slab"], big["slab"], torch.tensor([109999], dtype=torch.int32, device="cuda"),
                        torch.tensor([104533], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(back[0], back[1]) and back[0].abs().sum() > 0
    assert torch.equal(big["slab"][104533], big["slab"][109999])
