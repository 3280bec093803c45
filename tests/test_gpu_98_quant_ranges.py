"""Decode over the 8-bit latent cache where rows, queries and scores are very large, very small or far apart, each row as a whole
against the 64-bit definition (window_error.py; the roundings are those of test_gpu_98_quant_error.py).  The scores that decide
are of order one, or one token is ahead by a margin that is exact in 32 bits: a result that does not depend on the queries, or
has its heads in another order, is far outside the bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import quant_ref as qr
from tests import window_error
from tests.test_gpu_94_quant_decode import SCALE
from tests.test_gpu_98_quant_error import H, LORA, PAGE, ROW, Peaked, wr

pytestmark = pytest.mark.gpu


class Ranges(Peaked):
    """Slots of the given rows [n, 576] (f32, on the GPU); queries [B, 96, 576]."""

    def __init__(self, k3, slots, q, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ctx, self.layer = [len(rows) for rows in slots], 0
        need = [-(-n // PAGE) for n in self.ctx]
        ids = np.random.default_rng(seed).permutation(sum(need) + 1)
        self.table = np.full((len(slots), max(need)), -1, np.int32)
        pages = torch.zeros(len(ids), 1, PAGE, ROW, device="cuda")
        at = 0
        for b, rows in enumerate(slots):
            mine = ids[at:at + need[b]]
            self.table[b, :need[b]] = mine
            at += need[b]
            pages[torch.from_numpy(mine).cuda(), 0] = torch.nn.functional.pad(rows, (0, 0, 0, need[b] * PAGE - len(rows))).view(-1, PAGE, ROW)
        self.q = q.bfloat16()
        self.w = (torch.randn(H * 256, LORA, generator=gen, device="cuda") * LORA ** -0.5).bfloat16()
        self.blocks_of(k3, pages)

    def check_rows(self, got, **kw):
        super().check_rows(got, **kw)
        assert got.isfinite().all()
        with pytest.raises(AssertionError):
            super().check_rows(got.flip(1), **kw)


def rand(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=gen, device="cuda")


def rope_scores(rows, s):
    """Rope entries that make the scores s of queries with entry 1 there and 0 elsewhere."""
    rows[:, LORA:] = 0
    rows[:, LORA] = s / SCALE
    return rows


def rope_query(B):
    q = torch.zeros(B, H, ROW, device="cuda")
    q[:, :, LORA] = 1
    return q


def test_scores_of_minus_infinity(gpu_lib):
    """Rope keys of -inf: their tokens' weights are 0, where they fill the first tile of a split, too."""
    k3 = gpu_lib
    r = rand(6)
    slots = []
    for n, gone in ((600, slice(0, 128)), (600, slice(0, 300)), (300, slice(128, 256)), (600, slice(256, 512)), (100, slice(0, 99))):
        rows = rope_scores(r(n, ROW), 2 * r(n))
        rows[gone, LORA] = -float("inf")
        slots.append(rows)
    c = Ranges(k3, slots, rope_query(5))
    for split in (0, 128, 256):
        with np.errstate(invalid="ignore"):
            q, w = np.zeros((H, 1)) + 1, c.w.double().cpu().numpy()
            got = c.run(k3, split=split)
            for b, n in enumerate(c.ctx):
                rows, _ = qr.row_values(c.blocks, 0, c.table[b], wr.visible(n, 1 << 30, 0))
                rows = np.concatenate([rows[:, :LORA], np.where(np.isinf(rows[:, LORA:LORA + 1]), -1e30, rows[:, LORA:LORA + 1])], -1)
                out = qr.attend(np.concatenate([np.zeros((H, LORA)), q], -1), rows, w, SCALE)[0]
                row, heads = window_error.relative(got[b].double().cpu().numpy(), out)
                assert row <= window_error.ROW_BOUND and np.all(heads <= window_error.HEAD_BOUND), (b, split, row)
