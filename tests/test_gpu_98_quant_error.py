"""Decode over the 8-bit latent cache, each row as a whole against the 64-bit definition (window_error.py), where some tokens
take most of a row's mass and what they add is small: the first tokens of a trained model, or a few anywhere.  What such a
row answers comes from thousands of small weights, which the bound of every element, a sum of all their roundings, does
not see.

The roundings that show are window_error's two: a weight, here a sum of two e4m3 numbers, is within 2^-4 of 2^-4 = 2^-8 of
itself as a bf16 is, and the output is a bf16.  A pair's floor, 1.25 * 2^-22 of the largest product of weight and row scale
among 32 tokens, is below 2^-8 of every weight here that adds to the mean square; queries are exact down to 2^-14 of their
largest.  So its bounds hold unchanged."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import quant_ref as qr
from tests import window_error, window_ref as wr
from tests.test_gpu_94_quant_decode import MOST, SCALE, Case

pytestmark = pytest.mark.gpu
LORA, ROPE, PAGE, ROW, H = 512, 64, 64, 576, 96


class Peaked(Case):
    """Slots whose listed tokens {position: share} take their shares of every row's mass (about: heads differ), with latents
    2^-6 of the others' size but for one, which W_UV does not look at: the row's scale is an ordinary one, what it adds to
    the output is not.  The others have a common mean.  Rope entry 0 makes the shares."""

    def __init__(self, k3, slots, seed=0, mean=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        self.ctx, self.layer = [n for n, _ in slots], 0
        B, need = len(slots), [-(-n // PAGE) for n, _ in slots]
        pages = sum(need) + 1
        ids = np.random.default_rng(seed).permutation(pages)
        self.table = np.full((B, max(need)), -1, np.int32)
        rows = rand(pages, 1, PAGE, ROW)
        rows[..., :LORA] += mean * rand(LORA)
        rows[..., LORA] = 0
        self.q = (rand(B, H, ROW) * 0.5).bfloat16()
        self.q[:, :, LORA] = 1.0
        self.w = (rand(H * 256, LORA) * LORA ** -0.5).bfloat16()
        self.w[:, 0] = 0
        at = 0
        for b, (n, shares) in enumerate(slots):
            mine = ids[at:at + need[b]]
            self.table[b, :need[b]] = mine
            at += need[b]
            plain = rows[torch.from_numpy(mine).cuda(), 0].reshape(-1, ROW)[:n].bfloat16().double()
            mass = torch.exp(self.q[b].double() @ plain.T * SCALE).sum(-1).log().mean().item()   # of the others, in logits
            for t, share in shares.items():
                row = rows[int(mine[t // PAGE]), 0, t % PAGE]
                row[:LORA] *= 2.0 ** -6
                row[0] = 4.0
                row[LORA + 1:] = 0
                row[LORA] = (mass + np.log(share / (1 - sum(shares.values())))) / SCALE
        self.blocks_of(k3, rows)

    def blocks_of(self, k3, rows):
        slab = torch.empty(rows.shape[0], 1, qr.QPAGE, dtype=torch.uint8, device="cuda")
        ids = torch.arange(rows.shape[0], dtype=torch.int32, device="cuda")
        k3.quant_write_pages(slab, rows.bfloat16(), ids, ids)
        self.blocks = slab.cpu().numpy()

    def check_rows(self, got, window=MOST, sink=0, row_bound=window_error.ROW_BOUND, head_bound=window_error.HEAD_BOUND):
        q, w = self.q.double().cpu().numpy(), self.w.double().cpu().numpy()
        for b, n in enumerate(self.ctx):
            rows, _ = qr.row_values(self.blocks, self.layer, self.table[b], wr.visible(n, window, sink))
            row, heads = window_error.relative(got[b].double().cpu().numpy(), qr.attend(q[b], rows, w, SCALE)[0])
            assert row <= row_bound and np.all(heads <= head_bound), (b, n, row, float(heads.max()))


@pytest.mark.parametrize("n", [4096, 16384])
def test_first_tokens_that_take_most_of_the_mass(gpu_lib, n):
    c = Peaked(gpu_lib, [(n, {0: s}) for s in (0.5, 0.8, 0.9, 0.99)] + [(n - 100, {0: 0.3, 1: 0.3, 2: 0.3})], seed=n)
    for split in (n, 0, 512):
        c.check_rows(c.run(gpu_lib, split=split))
    c.check(c.run(gpu_lib, split=n))
    c.check_rows(c.run(gpu_lib, n // 2, 4, split=n), n // 2, 4)


def test_tokens_anywhere_that_take_most_of_the_mass(gpu_lib):
    """(and one that rises far above those before it, the last of its tile, the first and the last of the context)"""
    n = 8000
    slots = [{3000: 0.9}, {100: 0.3, 2900: 0.3, 6000: 0.3}, {127: 0.99}, {n - 1: 0.97}, {0: 0.05, 5000: 0.9, n - 1: 0.04},
             {31: 0.45, 32: 0.45}]
    c = Peaked(gpu_lib, [(n, s) for s in slots], seed=5)
    for split in (8064, 0, 1024):
        c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("n", [33, 64, 100, 129, 300])
def test_short_contexts(gpu_lib, n):
    c = Peaked(gpu_lib, [(n, {0: s}) for s in (0.5, 0.9, 0.99, 0.999)] + [(n, {n - 1: 0.99}), (n, {n // 2: 0.95})], seed=n)
    for split in (0, 128):
        c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("mean", [0.0, 1.0])
def test_ordinary_rows(gpu_lib, mean):
    c = Peaked(gpu_lib, [(n, {}) for n in (1, 2, 31, 64, 65, 130, 700, 1500, 5000)], seed=7, mean=mean)
    for split in (0, 128):
        c.check_rows(c.run(gpu_lib, split=split))
    c.check_rows(c.run(gpu_lib, 100, 3), 100, 3)


def test_scores_of_many_sizes(gpu_lib):
    """Heads from flat to a spread of 12 between one token's score and another's, so that a tile's largest weight differs from
    the next one's by powers of ten."""
    c = Peaked(gpu_lib, [(n, {}) for n in (200, 1000, 6000)], seed=8, mean=0.5)
    c.q = (c.q.float() * torch.logspace(-1, 1, H, base=10, device="cuda")[:, None]).bfloat16()
    for split in (0, 128, 6016):
        c.check_rows(c.run(gpu_lib, split=split))
