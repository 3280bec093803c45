"""The abort path of the windowed kernel's bounded waits, without any GPU fault: the diagnostic entries run the windowed
calls with one page of every unit never loaded and a short wait limit.  The call has to return with K3MLA_DEV_TIMEOUT in
the error word, and the context, the workspace and the cache stay usable: the plain call right behind it gives the bits
that it gave before."""
from __future__ import annotations

import time

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_gpu_87_window import SCALE_BITS, Case

pytestmark = pytest.mark.gpu

H, V = 96, 128


def aborted(call, err):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    torch.cuda.synchronize()
    took = time.perf_counter() - t0
    assert err.item() == k3mla.DEV_TIMEOUT, f"device error word {err.item()}"
    assert took < 0.5, f"the aborted call took {took:.3f} s"
    err.zero_()


# a lone unit; a unit a cluster; several units a cluster, of which those of one page go through; splits to be merged
@pytest.mark.parametrize("lens,split,page", [([130], 0, 1), ([300, 130, 0, 64] * 15, 0, 1), ([300, 60, 0, 900] * 60, 0, 3),
                                             ([1000, 700, 130], 256, 2), ([1000] * 20, 256, 1)])
def test_decode_waits_run_out(gpu_lib, lens, split, page):
    c = Case(90, lens, len(lens))
    want = c.decode(1000, 3, split)
    table, ctx = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    out = torch.empty(len(lens), H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(k3mla.window_decode_workspace_bytes(len(lens), c.max_ctx, 1000, 3, split), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        aborted(lambda: k3mla.diag_window_timeout(c.q, c.slab, 1, table, ctx, c.w, SCALE_BITS, out, ws, c.max_ctx, 1000, 3,
                                                  split, withhold_page=page, wait_us=2000, dev_err=c.err), c.err)
        assert torch.equal(c.decode(1000, 3, split, ws=ws), want) and c.err.item() == 0


@pytest.mark.parametrize("lens,new,page", [([130], [1], 1), ([300, 900], [40, 7], 2), ([700] * 8, [60] * 8, 1)])
def test_chunk_waits_run_out(gpu_lib, lens, new, page):
    R = sum(new)
    c = Case(91, lens, R)
    pos0, start = [n - m for n, m in zip(lens, new)], np.concatenate([[0], np.cumsum(new)])
    want = c.chunk(pos0, start, 500, 3)
    table = torch.from_numpy(c.table).cuda()
    args = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (pos0, start.tolist())]
    out = torch.empty(R, H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(k3mla.window_chunk_decode_workspace_bytes(len(lens), R, c.max_ctx), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        aborted(lambda: k3mla.diag_window_chunk_timeout(c.q, c.slab, 1, table, *args, c.w, SCALE_BITS, out, ws, c.max_ctx, 500,
                                                        3, withhold_page=page, wait_us=2000, dev_err=c.err), c.err)
        assert torch.equal(c.chunk(pos0, start, 500, 3), want) and c.err.item() == 0


def test_diagnostic_arguments_are_checked(gpu_lib):
    c = Case(92, [130], 1)
    table, ctx = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    out = torch.empty(1, H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for page, us in ((0, 2000), (1, 50), (1, 200000), (2 ** 30, 2000)):
        with pytest.raises(k3mla.K3mlaError, match="withhold_page"):
            k3mla.diag_window_timeout(c.q, c.slab, 1, table, ctx, c.w, SCALE_BITS, out, ws, 192, 100, 0, 0, page, us, c.err)
        with pytest.raises(k3mla.K3mlaError, match="withhold_page"):
            k3mla.diag_window_chunk_timeout(c.q, c.slab, 1, table, ctx, start, c.w, SCALE_BITS, out, ws, 192, 100, 0, page, us,
                                            c.err)
    torch.cuda.synchronize()
    assert c.err.item() == 0
