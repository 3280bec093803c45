"""The 8-bit latent cache is written and read back as its definition says: whole pages bit for bit, appended rows within half a
step of the 64-bit values."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import quant_ref as qr
from tests import window_ref as wr

pytestmark = pytest.mark.gpu
LORA, ROPE, PAGE, ROW, H = 512, 64, 64, 576, 96


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).cuda().bfloat16()


def rows_of_all_kinds(seed, n):
    """bf16 rows [n, 576] as f64: ordinary ones, wide ranges, ties, extremes, zeros, NaN and infinities."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, ROW)) * 2.0 ** g.uniform(-3, 3, (n, 1))
    for i in range(n):
        kind = i % 12
        if kind == 1:
            x[i] *= 2.0 ** g.uniform(-30, 30, ROW)
        elif kind == 2:      # exact ties and the borders of the scale
            x[i, :LORA] = g.choice([17, 18.5, 224, 225, 447, 448, 449, -9.5, 1 / 512, 3 / 1024, 1 / 1024], LORA)
        elif kind == 3:
            x[i] = 0
        elif kind == 4:
            x[i, :LORA] = 0
        elif kind == 5:
            x[i] *= 2.0 ** -130
        elif kind == 6:
            x[i] = np.clip(x[i] * 2.0 ** 125, -3.3e38, 3.3e38)
        elif kind == 7:
            x[i, :LORA] *= 2.0 ** -100
        elif kind == 8:
            x[i, g.integers(0, LORA, 3)] = [np.nan, np.inf, -np.inf]
        elif kind == 9:
            x[i, LORA:] *= 2.0 ** 60
            x[i, :LORA] *= 2.0 ** -60
        elif kind == 10:
            x[i, LORA + 5] = np.inf
        elif kind == 11:
            x[i, :LORA] = np.nan
    with np.errstate(over="ignore"):
        return bf16(x).double().cpu().numpy()


def same_blocks(got, want):
    gc, gs, gr = qr.unpack(got)
    wc, ws, wrp = qr.unpack(want)
    nan = (wc & 127) == 127
    assert np.array_equal((gc & 127) == 127, nan) and np.array_equal(gc[~nan], wc[~nan])
    assert np.array_equal(gs, ws)
    assert np.array_equal(gr, wrp)


@pytest.mark.parametrize("layers,pages", [(1, 1), (3, 5), (24, 2)])
def test_written_pages_are_the_definition_bit_for_bit(gpu_lib, layers, pages):
    k3 = gpu_lib
    rows = rows_of_all_kinds(layers, (pages + 2) * layers * PAGE).reshape(pages + 2, layers, PAGE, ROW)
    slab = bf16(rows)
    before = torch.randint(0, 255, (pages + 3, layers, qr.QPAGE), dtype=torch.uint8, device="cuda")
    to = before.clone()
    g = torch.Generator().manual_seed(layers)
    src, dst = (torch.randperm(n, generator=g)[:pages].int() for n in (pages + 2, pages + 3))
    k3.quant_write_pages(to, slab, src.cuda(), dst.cuda())
    got, want = to.cpu().numpy(), before.cpu().numpy()
    with np.errstate(over="ignore"):
        want[dst.numpy()] = qr.pack(*qr.quantise(rows[src.numpy()]))
    keep = np.ones(pages + 3, bool)
    keep[dst.numpy()] = False
    assert np.array_equal(got[keep], want[keep])
    same_blocks(got[dst.numpy()], want[dst.numpy()])


def test_pages_read_back_are_what_the_codes_stand_for(gpu_lib):
    k3 = gpu_lib
    rows = rows_of_all_kinds(7, 4 * 2 * PAGE).reshape(4, 2, PAGE, ROW)
    with np.errstate(over="ignore", invalid="ignore"):
        blocks = qr.pack(*qr.quantise(rows))
        want = qr.values(blocks)
        # a latent above 248 * 2^120 is nearest to the code 256, and 256 * 2^120 = 2^128 lies past bf16's largest value,
        # (2 - 2^-7) 2^127, by more than half a step: it is an infinity there
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * np.inf, want)
    slab = torch.full((5, 2, PAGE, ROW), 7.0, dtype=torch.bfloat16, device="cuda")
    src, dst = torch.tensor([3, 0, 2], dtype=torch.int32).cuda(), torch.tensor([1, 4, 0], dtype=torch.int32).cuda()
    k3.quant_read_pages(slab, torch.from_numpy(blocks).cuda(), src, dst)
    got = slab.double().cpu().numpy()
    assert (got[[2, 3]] == 7).all()
    # (values below bf16's normal range round there once more: half of its smallest step)
    for s, d in ((3, 1), (0, 4), (2, 0)):
        w, g = want[s], got[d]
        finite = np.isfinite(w)
        assert np.array_equal(np.isnan(w), np.isnan(g)) and np.array_equal(w[~finite & ~np.isnan(w)], g[~finite & ~np.isnan(w)])
        assert (np.abs(w - g)[finite] <= np.where(np.abs(w) < 2.0 ** -126, 2.0 ** -134, 0)[finite]).all()


def test_a_page_written_read_and_written_again_keeps_its_values(gpu_lib):
    k3 = gpu_lib
    g = torch.Generator(device="cuda").manual_seed(3)
    slab = torch.randn(3, 2, PAGE, ROW, generator=g, device="cuda").bfloat16()
    ids = torch.arange(3, dtype=torch.int32, device="cuda")
    q = torch.zeros(3, 2, qr.QPAGE, dtype=torch.uint8, device="cuda")
    k3.quant_write_pages(q, slab, ids, ids)
    once, twice = torch.empty_like(slab), torch.empty_like(slab)
    k3.quant_read_pages(once, q, ids, ids)
    k3.quant_write_pages(q, once, ids, ids)
    k3.quant_read_pages(twice, q, ids, ids)
    assert torch.equal(once, twice)
    x = slab.double().cpu().numpy()
    n = qr.exponent(x[..., :LORA], x[..., LORA:])
    err = np.abs(x - once.double().cpu().numpy())
    assert np.array_equal(once[..., LORA:].cpu().view(torch.int16).numpy(), slab[..., LORA:].cpu().view(torch.int16).numpy())
    assert (err[..., :LORA] <= np.maximum(2.0 ** -4 * np.abs(x[..., :LORA]), 2.0 ** (n - 10.0)[..., None])).all()


def test_bad_ids_are_flagged_and_skipped_and_copies_are_copies(gpu_lib):
    k3 = gpu_lib
    slab = torch.randn(3, 2, PAGE, ROW, device="cuda").bfloat16()
    q = torch.zeros(4, 2, qr.QPAGE, dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for src, dst in ((-1, 0), (3, 0), (0, 4), (0, -1)):
        err = torch.zeros(1, **i32)
        k3.quant_write_pages(q, slab, torch.tensor([src], **i32), torch.tensor([dst], **i32), dev_err=err)
        assert err.item() == k3.DEV_BAD_PAGE and not q.any()
    err = torch.zeros(1, **i32)
    k3.quant_read_pages(slab.clone(), q, torch.tensor([3], **i32), torch.tensor([2], **i32), dev_err=err)
    assert err.item() == 0
    k3.quant_read_pages(slab, q, torch.tensor([4], **i32), torch.tensor([0], **i32), dev_err=err)
    assert err.item() == k3.DEV_BAD_PAGE and slab[0].any()
    k3.quant_write_pages(q, slab, torch.arange(3, **i32), torch.arange(3, **i32))
    want = q.clone()
    want[3], want[0] = q[1], q[2]
    k3.quant_copy_pages(q, q, torch.tensor([1, 2], **i32), torch.tensor([3, 0], **i32))
    assert torch.equal(q, want)
    k3.quant_copy_pages(q, q, torch.zeros(0, **i32), torch.zeros(0, **i32))


@pytest.mark.parametrize("norms,rotate,interleaved,at", [(True, True, False, False), (True, True, True, True),
                                                         (False, False, False, False), (False, True, False, False)])
@pytest.mark.parametrize("rows", ["one each", "ragged"])
def test_appended_rows_are_within_half_a_step(gpu_lib, norms, rotate, interleaved, at, rows):
    k3 = gpu_lib
    g = np.random.default_rng(5 + interleaved)
    B = 5
    new = [1] * B if rows == "one each" else [3, 0, 70, 1, 9]
    pos0 = np.array([0, 63, 60, -1, 130])
    start = np.concatenate([[0], np.cumsum(new)])
    R = int(start[-1]) + (0 if rows == "one each" else 2)          # two rows behind the last slot
    L, layer, pages = 2, 1, 14
    table = np.full((B, 3), -1, np.int32)
    ids = g.permutation(pages)
    for b in range(B):
        table[b, :] = ids[3 * b:3 * b + 3] if b < 4 else [-1, -1, 13 if 13 not in ids[:12] else -1]
    q = bf16(g.standard_normal((R, H, 192)))
    kv = bf16(g.standard_normal((R, 600)) * 2.0 ** g.uniform(-2, 2, (R, 1)))   # rows 600 apart
    w = [bf16(np.exp(0.3 * g.standard_normal(n))) if norms else None for n in (192, LORA, ROPE)]
    inv = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda() if rotate else None
    rope0 = np.array([5, 70000, 3, 9, 1], np.int32) if at else None
    before = torch.randint(0, 255, (pages, L, qr.QPAGE), dtype=torch.uint8, device="cuda")
    slab, q_out = before.clone(), torch.full_like(q, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda x: None if x is None else torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    k3.quant_norm_rope_append(q, q_out, slab, layer, dev(table), dev(pos0), None if rows == "one each" else dev(start),
                              kv[:, 8:8 + LORA], kv[:, 528:528 + ROPE], q_weight=w[0], c_weight=w[1], k_weight=w[2], eps=1e-6,
                              inv_freq=inv, interleaved=interleaved, dev_err=err, rope_pos0=dev(rope0))
    # the queries are those of the bf16 call, bit for bit
    other = torch.zeros(pages, L, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    q_ref = torch.full_like(q, 7.0)
    k3.norm_rope_append(q, q_ref, other, layer, dev(table), dev(pos0), None if rows == "one each" else dev(start),
                        kv[:, 8:8 + LORA], kv[:, 528:528 + ROPE], q_weight=w[0], c_weight=w[1], k_weight=w[2], eps=1e-6,
                        inv_freq=inv, interleaved=interleaved, rope_pos0=dev(rope0))
    assert torch.equal(q_out, q_ref)
    got, want = slab.cpu().numpy(), before.cpu().numpy()
    wts = [None if x is None else x.double().cpu().numpy() for x in w]
    x = kv.double().cpu().numpy()
    touched = np.zeros((pages, PAGE), bool)
    missed = False
    for r, (b, pos) in enumerate(wr.rows_of(pos0, None if rows == "one each" else start, R)):
        if b < 0:
            continue
        page = table[b, pos // PAGE] if pos // PAGE < 3 else -1
        if page < 0:
            missed = True
            continue
        turn = pos if rope0 is None else int(rope0[b]) + pos - int(pos0[b])
        row, mag = wr.key_row(x[r, 8:8 + LORA], x[r, 528:528 + ROPE], turn, wts[1], wts[2], 1e-6,
                              None if inv is None else inv.double().cpu().numpy(), interleaved)
        touched[page, pos % PAGE] = True
        codes, scale, rope = (v[page, layer, pos % PAGE] for v in qr.unpack(got))
        s = qr.bits_value(scale)
        # f32 on the way: a norm's sum and root and two products 2^-18, an angle of up to 2^17 turns rounded once
        m = np.abs(row[:LORA]).max()
        assert m <= 448 * s * (1 + 2.0 ** -17) and m > 224 * s * (1 - 2.0 ** -17)
        c = qr.E4M3[codes] * s
        assert (np.abs(c - row[:LORA]) <= np.maximum(2.0 ** -4 * np.abs(row[:LORA]), 2.0 ** -10 * s) * (1 + 2.0 ** -10)
                + 2.0 ** -17 * np.abs(row[:LORA])).all()
        k = qr.bits_value(rope) * s
        assert (np.abs(k - row[LORA:]) <= 2.0 ** -8 * np.abs(row[LORA:]) + 2.0 ** -17 * mag[LORA:]).all()
    assert err.item() == (k3.DEV_UNMAPPED if missed else 0)
    rows_g = got[..., :PAGE * qr.QROW].reshape(pages, L, PAGE, qr.QROW)
    rows_w = want[..., :PAGE * qr.QROW].reshape(pages, L, PAGE, qr.QROW)
    assert np.array_equal(rows_g[:, 0], rows_w[:, 0]) and np.array_equal(rows_g[:, 1][~touched], rows_w[:, 1][~touched])
    sg, sw = (v[..., PAGE * qr.QROW:].copy().view(np.uint16) for v in (got, want))
    assert np.array_equal(sg[:, 0], sw[:, 0]) and np.array_equal(sg[:, 1][~touched], sw[:, 1][~touched])
