"""The windowed operators where their arguments or values are far out: split lengths near 2^31."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests.test_gpu_87_window import SCALE_BITS, Case

pytestmark = pytest.mark.gpu

PAGE, H, V, ROW = 64, 96, 128, 576


def test_a_split_as_long_as_an_int_holds_is_one_split(gpu_lib):
    c = Case(80, [700, 64, 0, 300], 4)
    near = 2 ** 31 - 128
    whole = c.decode(500, 10, 1024)
    assert torch.equal(c.decode(500, 10, near), whole)
    c.check(whole, [0, 1, 2, 3], [700, 64, 0, 300], 500, 10)
    table, lens = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    out = torch.full((2, 4, H, V), float("nan"), dtype=torch.bfloat16, device="cuda")
    for i, split in enumerate((1024, near)):
        ws = torch.full((k3mla.decode_workspace_bytes(4, c.max_ctx, split),), 0xFF, dtype=torch.uint8, device="cuda")
        k3mla.paged_decode(c.q, c.slab, 1, table, lens, c.w, SCALE_BITS, out[i], ws, c.max_ctx, split, dev_err=c.err)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and not torch.isnan(out.float()).any() and c.err.item() == 0
