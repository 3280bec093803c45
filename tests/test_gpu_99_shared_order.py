"""Decode for slots that share their first pages, all of whose inputs the kernels directly ahead of it have just written: queries,
tables, lengths, groups and cache rows, call after call without a pause."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_96_shared import H, V, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared_split,own_split", [(256, 128), (-1, 256)])
def test_inputs_written_by_the_kernels_ahead(gpu_lib, shared_split, own_split):
    k3 = gpu_lib
    cases = [Case([([700 - 9 * i - 40 * v for i in range(6)], 512), ([300 + v, 270, 260], 256)], alone=[90 + v], seed=20 + v)
             for v in range(3)]
    cols, pages = max(c.table.shape[1] for c in cases), max(c.slab.shape[0] for c in cases)
    own, want, inputs = max(c.max_own for c in cases), [], []
    for c in cases:
        want.append(c.run(k3, shared_split, own_split, max_own=own))
        slab, layer, table, ctx, start, shared, w, bits = c.args()
        inputs.append((c.q, torch.cat([slab, slab.new_zeros(pages - slab.shape[0], *slab.shape[1:])]),
                       torch.nn.functional.pad(table, (0, cols - table.shape[1]), value=-1), ctx, start, shared, w))
    q, slab, table, ctx, start, shared, w = (torch.empty_like(x) for x in inputs[0])
    ws = torch.empty(k3.shared_decode_workspace_bytes(10, 512, own, shared_split, own_split), dtype=torch.uint8, device="cuda")
    outs = [torch.full((10, H, V), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(60)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        w.copy_(inputs[i % 3][6])                              # (may be read early: it is not to be the last one)
        order = [(slab, 1), (start, 4), (shared, 5), (ctx, 3), (table, 2), (q, 0)]
        for dst, j in order[i % 6:] + order[:i % 6]:           # each of the others is the last one now and then
            dst.copy_(inputs[i % 3][j])
        k3.shared_decode(q, slab, 1, table, ctx, start, shared, w, 0x3D94, out, ws, 512, own, shared_split, own_split)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 3]), i
