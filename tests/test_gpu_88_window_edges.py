"""The windowed operators where their arguments or values are far out: split lengths near 2^31, many idle slots, single
infinities, waits that run out."""
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


def test_chunk_of_a_few_among_many_idle_slots(gpu_lib):
    # the planner passes every slot once: without that, 60,000 slots of which four have new rows take seconds, and
    # the waits for the units behind them run out
    B = 60_000
    new = np.zeros(B, np.int64)
    new[[0, 31, 32_000, B - 1]] = (5, 1, 130, 9)
    lens = np.where(new > 0, new + 70, 0)
    R = int(new.sum())
    c = Case(81, lens.tolist(), R)
    start = np.concatenate([[0], np.cumsum(new)])
    got = c.chunk(lens - new, start, 40, 3)
    assert c.err.item() == 0
    slot = np.repeat(np.arange(B), new)
    n = [int(lens[b] - new[b] + r - start[b] + 1) for r, b in enumerate(slot)]
    c.check(got, slot.tolist(), n, 40, 3, rows=range(0, R, 6))
    # none at all: every row is outside every slot
    got = c.chunk(lens - new, np.zeros(B + 1), 40, 3)
    assert torch.all(got == 0) and c.err.item() == 0


def test_chunk_of_more_slots_than_are_planned_is_refused(gpu_lib):
    c = Case(82, [70], 1)
    with pytest.raises(k3mla.K3mlaError, match="slots"):
        c.table = np.zeros((2 ** 20 + 1, 1), np.int32)
        c.chunk(np.zeros(2 ** 20 + 1), np.zeros(2 ** 20 + 2), 40, 3)


def relative(a, b):
    """Per row and head: the distance of a from b, relative to b."""
    a, b = a.double(), b.double()
    return (a - b).norm(dim=-1) / b.norm(dim=-1)


@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("token", [200, 201, 202, 203])
@pytest.mark.parametrize("dim", [3, 520])
def test_one_infinite_entry_is_the_same_for_a_chunk_and_its_rows_decodes(gpu_lib, dim, token, value):
    # Rows 0 .. 23 at positions 196 .. 219, window 6: the six rows from the token's own on see it, and by the token's
    # place in its group of four some rows of the same group do not.  Its score is +inf or -inf by the query's sign
    # (heads in turn).  In a latent entry (3) the infinity makes all that see it NaN, p = 0 included; in the rope part
    # (520) it only reaches the score: +inf is NaN, -inf leaves the token out.
    c = Case(83, [220], 24)
    c.q[:, 0::2, dim], c.q[:, 1::2, dim] = 1.0, -1.0
    clean = c.chunk([196], [0, 24], 6, 0)
    c.slab[int(c.table[0, token // PAGE]), 1, token % PAGE, dim] = value
    got = c.chunk([196], [0, 24], 6, 0)
    one = torch.cat([c.decode(6, 0, ctx=[197 + r], q=c.q[r:r + 1]) for r in range(24)])
    sees = torch.tensor([token in range(191 + r, 197 + r) for r in range(24)], device="cuda")
    assert sees.sum() == 6
    up = (c.q[..., dim].float() * value > 0) | (dim < 512)
    want = (sees[:, None] & up)[..., None].expand(24, H, V)
    assert torch.equal(torch.isnan(got), want) and torch.equal(torch.isnan(one), want)
    assert torch.equal(got[~sees], clean[~sees])
    if dim >= 512:
        # each is within 0.01 of the definition per head (2^-8 from the output and from p each, near-orthogonal rows)
        assert relative(got, one)[sees[:, None] & ~up].max() <= 0.02
    assert c.err.item() == 0
