"""Decode for slots that share their first pages while the group's first slots have ended: their table rows are cleared, and the
pages are those of the first slot that still attends."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_96_shared import H, ROW, SCALE_BITS, V, Case

pytestmark = pytest.mark.gpu
SPLITS = [(0, 0), (128, 128), (256, 0), (-1, 128)]


def end(c, slots, entry=-1):
    for b in slots:
        c.ctx[b] = 0
        c.table[b] = entry


@pytest.mark.parametrize("shared_split,own_split", SPLITS)
@pytest.mark.parametrize("size,ended", [(8, [0]), (8, [0, 1, 2]), (9, [0, 1, 2, 3]), (9, [0, 1, 2, 3, 5, 8]), (8, [3, 7]),
                                        (70, list(range(66))), (70, list(range(32)))])
def test_first_slots_have_ended(gpu_lib, size, ended, shared_split, own_split):
    c = Case([([300 + 64 + i % 50 for i in range(size)], 330), ([200, 190, 150], 128)], alone=[40], seed=size + len(ended))
    end(c, ended)
    end(c, [size])
    c.check(c.run(gpu_lib, shared_split, own_split))
    assert c.err.item() == 0


@pytest.mark.parametrize("shared_split,own_split", SPLITS)
def test_a_whole_group_has_ended(gpu_lib, shared_split, own_split):
    c = Case([([300] * 5, 256), ([400, 390], 320)], seed=3)
    end(c, range(5))
    c.check(c.run(gpu_lib, shared_split, own_split))
    assert c.err.item() == 0


@pytest.mark.parametrize("shared_split,own_split", SPLITS)
def test_what_an_ended_slot_s_table_holds_does_not_matter(gpu_lib, shared_split, own_split):
    """(a slot that holds fewer tokens than it is to share is flagged, and takes no part either)"""
    c = Case([([400, 390, 380, 370, 360], 320)], seed=4)
    end(c, [0], -2 ** 31)
    c.check(c.run(gpu_lib, shared_split, own_split))
    assert c.err.item() == 0
    c.ctx[0] = 100
    c.check(c.run(gpu_lib, shared_split, own_split), ctx=[0, 390, 380, 370, 360])
    assert c.err.item() == gpu_lib.DEV_CTX


def test_the_pool_s_first_slot_is_released(gpu_lib):
    """As a server runs it: four samples of one prompt, the one that held it first ends."""
    k3 = gpu_lib
    pool = k3.Pool(n_slots=4, max_ctx=1024, n_pages=40, shuffle_seed=6)
    prompt = 320
    assert pool.ensure(0, prompt) == 0
    for s in range(1, 4):
        assert pool.share_prefix(s, 0, prompt) == 0
    for s in range(4):
        assert pool.ensure(s, prompt + 1 + s) == 0
    pool.release(0)
    gen = torch.Generator(device="cuda").manual_seed(14)
    c = Case([([0, prompt + 2, prompt + 3, prompt + 4], prompt)], seed=14)
    c.table, c.layer, c.max_shared, c.max_own = pool.table()[:4].copy(), 0, prompt, 64
    assert (c.table[0] == -1).all() and (c.table[1, :5] >= 0).all()
    c.slab = torch.randn(40, 1, 64, ROW, generator=gen, device="cuda").bfloat16()
    for splits in SPLITS + [k3.shared_split_tokens(4, 1, prompt, 64)]:
        got = c.run(k3, *splits)
        c.check(got)
        assert got[1:].any() and not got[0].any()
    pool.close()


def test_a_captured_call_goes_on_when_the_first_slot_ends(gpu_lib):
    k3 = gpu_lib
    c = Case([([400, 390, 350, 360, 330], 320)], seed=15)
    slab, layer, table, ctx, start, shared, w, bits = c.args()
    ws = torch.full((k3.shared_decode_workspace_bytes(5, 320, 128, 128, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(5, H, V, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: k3.shared_decode(c.q, slab, layer, table, ctx, start, shared, w, bits, out, ws, 320, 128, 128, 128)  # noqa: E731
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    for gone in ([], [0], [0, 1], [0, 1, 2, 3]):
        lens = [0 if b in gone else n for b, n in enumerate([400, 390, 350, 360, 330])]
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        for b in gone:
            table[b] = -1
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, ctx=lens)
