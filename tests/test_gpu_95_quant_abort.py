"""The abort path of the bounded waits of the decode over the 8-bit cache, without any GPU fault: the diagnostic entry runs it
with one chunk of every unit never loaded and a short wait limit.  The call has to return with K3MLA_DEV_TIMEOUT in the error
word, and the plain call right behind it gives the bits that it gave before."""
from __future__ import annotations

import time

import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_gpu_94_quant_decode import MOST, SCALE_BITS, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx,split,tile", [([130], 0, 0), ([130], 0, 1), ([300, 130, 0, 64] * 30, 0, 1), ([1000, 700, 130], 256, 1),
                                            ([1500] * 20, 0, 7)])
def test_waits_run_out(gpu_lib, ctx, split, tile):
    c = Case(ctx, seed=len(ctx) + tile)
    want = c.run(k3mla, split=split)
    B, most = len(ctx), max(ctx)
    slab, table = torch.from_numpy(c.blocks).cuda(), torch.from_numpy(c.table).cuda()
    lens = torch.tensor(ctx, dtype=torch.int32).cuda()
    out = torch.empty(B, 96, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(k3mla.quant_decode_workspace_bytes(B, most, MOST, 0, split), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(2):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        k3mla.diag_quant_timeout(c.q, slab, c.layer, table, lens, c.w, SCALE_BITS, out, ws, most, MOST, 0, split,
                                 withhold_tile=tile, wait_us=2000, dev_err=err)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        assert err.item() == k3mla.DEV_TIMEOUT and took < 0.5, (err.item(), took)
        err.zero_()
        k3mla.quant_decode(c.q, slab, c.layer, table, lens, c.w, SCALE_BITS, out, ws, most, MOST, 0, split, dev_err=err)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and err.item() == 0


def test_diagnostic_arguments_are_checked(gpu_lib):
    c = Case([130], seed=1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(1, 96, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for tile, us in ((-1, 2000), (2 ** 30, 2000), (1, 50), (1, 200000)):
        with pytest.raises(k3mla.K3mlaError, match="withhold_tile"):
            k3mla.diag_quant_timeout(c.q, torch.from_numpy(c.blocks).cuda(), 1, torch.from_numpy(c.table).cuda(),
                                     torch.tensor([130], dtype=torch.int32).cuda(), c.w, SCALE_BITS, out, ws, 192, 100, 0, 0, tile,
                                     us, err)
    assert err.item() == 0
