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


@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("low,high", [(-60, 60), (-80, 30), (-20, 110), (-85, -70), (100, 118), (-20, 125)])
def test_rows_far_apart_with_equal_scores(gpu_lib, low, high, split):
    """Small rows before large ones and behind them: what a small row adds is lost beside the large ones, but its weight is not."""
    r = rand(1)
    slots = []
    for n, first in ((512, 256), (512, 300), (200, 100)):
        rows = r(n, ROW)
        rows[:first, :LORA] *= 2.0 ** low
        rows[first:, :LORA] *= 2.0 ** high
        slots += [rope_scores(rows, 0 * rows[:, 0]), rope_scores(rows.flip(0), 0 * rows[:, 0])]
    c = Ranges(gpu_lib, slots, rope_query(6))
    c.q = (c.q * torch.linspace(0.5, 1.5, H, device="cuda")[:, None]).bfloat16()
    c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("spread", [10, 50])
def test_rows_far_apart_whose_weights_make_up_for_it(gpu_lib, spread, split):
    """(rows of 2^-spread to 2^spread, scores the other way round: all of them count in the output, the small ones in the sum)"""
    r = rand(2)
    slots = []
    for n in (700, 130, 40):
        rows, e = r(n, ROW), torch.rand(n, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda") * 2 * spread - spread
        rows[:, :LORA] *= torch.exp2(e)[:, None]
        slots.append(rope_scores(rows, -e * float(np.log(2.0)) + r(n)))
    c = Ranges(gpu_lib, slots, rope_query(3))
    c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("split", [0, 128])
@pytest.mark.parametrize("exponent", [80, 100, 118, 125, -70])
def test_rows_of_one_size(gpu_lib, exponent, split):
    r = rand(3)
    rows = r(2, 400, ROW) * 2.0 ** exponent
    q = rope_query(2)
    c = Ranges(gpu_lib, [rope_scores(rows[0], 3 * r(400)), rope_scores(rows[1, :70], 3 * r(70))], q)
    c.q = (c.q * torch.linspace(-1.5, 1.5, H, device="cuda")[:, None]).bfloat16()
    c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("split", [0, 128])
def test_rows_near_the_largest_bf16(gpu_lib, split):
    """Latents about 1.5 * 2^126, whose sums, not yet divided by the sum of exp, pass what f32 has.  (W_UV 2^-4 of its usual size:
    4.5 standard deviations of the outputs would be above the largest bf16.)"""
    r = rand(7)
    rows = (1 + 0.1 * r(2, 700, ROW)) * 1.5 * 2.0 ** 126
    c = Ranges(gpu_lib, [rope_scores(rows[0], 2 * r(700)), rope_scores(rows[1, :300], 2 * r(300))], rope_query(2))
    c.w *= 2.0 ** -4
    c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("exponent", [-100, -40, 0, 30, 60])
def test_queries_of_very_different_sizes_with_scores_of_order_one(gpu_lib, exponent):
    r = rand(4)
    q = r(2, H, ROW) * 0.5 * torch.exp2(3 * torch.linspace(-1, 1, H, device="cuda"))[:, None] * 2.0 ** exponent
    c = Ranges(gpu_lib, [r(260, ROW) * 2.0 ** -exponent, r(70, ROW) * 2.0 ** -exponent], q)
    for split in (0, 128):
        c.check_rows(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("exponent", [18, 22, 30, 45, 100])
def test_scores_beyond_what_an_exponential_stands(gpu_lib, exponent):
    """All scores 37 * 2^(exponent - 9), exact, but for one that is 2^-7 of it larger, or two: those are the answer."""
    r = rand(5)
    slots = []
    for n, best in ((300, [7]), (300, [299]), (700, [130, 400]), (64, [0, 63]), (1, [0])):
        rows = r(n, ROW)
        rows[:, LORA:] = 0
        rows[:, LORA] = 1
        rows[best, LORA] = 1 + 2.0 ** -7
        slots.append(rows)
    q = rope_query(5)
    q[:, :, LORA] = 2.0 ** exponent
    c = Ranges(gpu_lib, slots, q)
    for split in (0, 128):
        got = c.run(gpu_lib, split=split)
        c.check_rows(got)
        low = c.run(gpu_lib, 100, 1, split=split)
        c.check_rows(low, window=100, sink=1)


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
