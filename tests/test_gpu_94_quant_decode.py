"""Decode over the 8-bit latent cache against its 64-bit definition, at the lengths, masks and values where it can go wrong."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import quant_ref as qr
from tests import window_ref as wr

pytestmark = pytest.mark.gpu
LORA, ROPE, PAGE, ROW, H, V = 512, 64, 64, 576, 96, 128
SCALE_BITS, SCALE = 0x3D94, 0.072265625
MOST = 1 << 30


class Case:
    """A batch: slots of the given contexts over scattered pages; every page of the slab is full of ordinary rows, and what
    no slot owns is garbage."""

    def __init__(self, ctx, seed=0, cols=None, layers=2, layer=1, spread=0.5, q_spread=0.0):
        g = np.random.default_rng(seed)
        self.ctx, self.layer = list(ctx), layer
        B = len(self.ctx)
        need = [-(-max(0, n) // PAGE) for n in self.ctx]
        cols = cols or max([1] + need)
        pages = sum(need) + 3
        ids = g.permutation(pages)
        self.table = np.full((B, cols), -1, np.int32)
        at = 0
        for b in range(B):
            k = min(need[b], cols)
            self.table[b, :k] = ids[at:at + k]
            at += k
        rows = g.standard_normal((pages, layers, PAGE, ROW), dtype=np.float32).astype(np.float64)
        rows[..., :LORA] *= 2.0 ** (spread * g.standard_normal((pages, layers, PAGE, 1)))
        self.blocks = qr.pack(*qr.quantise(wr_bf16(rows)))
        q = g.standard_normal((B, H, ROW)) * 0.5
        q[..., LORA:] *= 2
        q *= 2.0 ** (q_spread * g.standard_normal((B, H, 1)))
        self.q = torch.from_numpy(q.astype(np.float32)).cuda().bfloat16()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w = (torch.randn(H * 256, LORA, generator=gen, device="cuda") * LORA ** -0.5).bfloat16()

    def stale(self):
        """What lies behind the last token of every slot becomes NaN codes, rope entries and scales."""
        for b, n in enumerate(self.ctx):
            if n > 0 and n % PAGE:
                page = self.table[b, n // PAGE]
                if page >= 0:
                    block = self.blocks[page, self.layer]
                    block[:PAGE * qr.QROW].reshape(PAGE, qr.QROW)[n % PAGE:] = 0xFF
                    block[PAGE * qr.QROW:].view(np.uint16)[n % PAGE:] = 0xFFFF
        return self

    def run(self, k3, window=MOST, sink=0, split=0, max_ctx=None, err=None, slots=None, out=None):
        slots = list(range(len(self.ctx))) if slots is None else slots
        B = len(slots)
        max_ctx = max_ctx or max([1] + self.ctx)
        ws = torch.full((max(256, k3.quant_decode_workspace_bytes(B, max_ctx, window, sink, split)),), 0xFF, dtype=torch.uint8,
                        device="cuda")
        out = torch.full((B, H, V), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
        k3.quant_decode(self.q[slots].contiguous(), torch.from_numpy(self.blocks).cuda(), self.layer,
                        torch.from_numpy(self.table[slots]).cuda(),
                        torch.tensor([self.ctx[b] for b in slots], dtype=torch.int32).cuda(), self.w, SCALE_BITS, out, ws,
                        max_ctx, window, sink, split, dev_err=err)
        torch.cuda.synchronize()
        return out

    def check(self, got, window=MOST, sink=0, cap=None, slots=None):
        q, w = self.q.double().cpu().numpy(), self.w.double().cpu().numpy()
        for i, b in enumerate(slots if slots is not None else range(len(self.ctx))):
            n = min(max(0, self.ctx[b]), cap or 1 << 40)
            rows, scales = qr.row_values(self.blocks, self.layer, self.table[b], wr.visible(n, window, sink))
            out, o, p = qr.attend(q[b], rows, w, SCALE)
            err = np.abs(got[i].double().cpu().numpy() - out)
            tol = qr.out_tolerance(q[b], out, o, p, rows, scales, w, SCALE)
            assert (err <= tol).all(), (b, n, float((err / tol).max()))


def wr_bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


EDGES = [1, 0, 63, 64, 65, 127, 128, 129, 191, 192, 193, 300, 2, 640]


@pytest.mark.parametrize("split", [0, 128, 256])
def test_lengths_around_pages_and_tiles(gpu_lib, split):
    c = Case(EDGES, seed=1).stale()
    c.check(c.run(gpu_lib, split=split))


@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (64, 0), (65, 4), (100, 64), (128, 130), (5, 1000), (300, 1)])
@pytest.mark.parametrize("split", [0, 128])
def test_windows_and_first_tokens(gpu_lib, window, sink, split):
    c = Case(EDGES, seed=2).stale()
    c.check(c.run(gpu_lib, window, sink, split), window, sink)


def test_many_splits_and_a_long_slot(gpu_lib):
    c = Case([5000, 17, 4097], seed=3).stale()
    for split in (0, 128, 1024):
        c.check(c.run(gpu_lib, split=split))


def test_twenty_slots_of_several_splits(gpu_lib):
    """(the merge of its own)"""
    g = np.random.default_rng(4)
    c = Case([int(x) for x in g.integers(1, 700, 20)], seed=4).stale()
    c.check(c.run(gpu_lib, split=128))


def test_unmapped_pages_are_zero_rows_and_bad_ids_too(gpu_lib):
    k3 = gpu_lib
    c = Case([400, 64, 200], seed=5)
    c.table[0, 2] = -1
    c.table[1, 0] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = c.run(k3, err=err)
    assert err.item() == 0
    c.check(want)
    assert not want[1].any()
    for bad in (-2, c.blocks.shape[0], 2 ** 31 - 1, -2 ** 31):
        c.table[0, 2] = bad
        err.zero_()
        assert torch.equal(c.run(k3, err=err), want)
        assert err.item() == k3.DEV_BAD_PAGE


def test_lengths_past_the_bound_are_clamped_and_flagged(gpu_lib):
    k3 = gpu_lib
    c = Case([300, 500, -4], seed=6)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.check(c.run(k3, max_ctx=200, err=err), cap=200)
    assert err.item() == k3.DEV_CTX
    short = Case([1000, 90], seed=7, cols=3)
    err.zero_()
    short.check(short.run(k3, max_ctx=1000, err=err), cap=192)
    assert err.item() == k3.DEV_CTX


@pytest.mark.parametrize("window,sink", [(MOST, 0), (70, 3)])
def test_rows_of_very_different_sizes(gpu_lib, window, sink):
    """Scales between 2^-30 and 2^20, and heads whose queries differ by as much as logits allow."""
    c = Case([700, 130, 65], seed=8, spread=5.0, q_spread=2.0)
    c.check(c.run(gpu_lib, window, sink), window, sink)
    c.check(c.run(gpu_lib, window, sink, 128), window, sink)


def test_scores_that_grow_with_the_position(gpu_lib):
    """The reference has to move in nearly every tile, up and by large steps."""
    c = Case([1500, 900], seed=9)
    for b, n in enumerate(c.ctx):
        for t in range(n):
            block = c.blocks[c.table[b, t // PAGE], c.layer]
            row = block[:PAGE * qr.QROW].reshape(PAGE, qr.QROW)[t % PAGE]
            rope = row[LORA:].view(np.uint16)
            s = qr.bits_value(block[PAGE * qr.QROW:].view(np.uint16)[t % PAGE])
            x = np.zeros(ROPE)
            x[0] = 0.25 * t * (1 if b == 0 else -1)
            rope[:] = qr.bf16_bits(x / s)
    c.q[:, :, LORA] = 1.0
    c.q[:, ::3, LORA] = -1.0     # heads whose best token is the first one
    c.check(c.run(gpu_lib))
    c.check(c.run(gpu_lib, split=128))


def test_a_seen_nan_makes_its_slot_nan_and_an_unseen_one_nothing(gpu_lib):
    k3 = gpu_lib
    c = Case([300, 300], seed=10)
    want = c.run(k3, 100, 2)
    block = c.blocks[c.table[0, 1], c.layer]            # tokens 64..127 of slot 0: neither sinks nor in the window
    rows = block[:PAGE * qr.QROW].reshape(PAGE, qr.QROW)
    rows[5, 3] = 0x7F
    rows[7, LORA:LORA + 2].view(np.uint16)[:] = 0x7F80
    page = c.blocks[c.table[0, 3], c.layer][:PAGE * qr.QROW].reshape(PAGE, qr.QROW)   # tokens 192..255: 200 is the first seen
    page[0, :] = 0x7F
    assert torch.equal(c.run(k3, 100, 2), want)
    page[9, 500] = 0xFF
    got = c.run(k3, 100, 2)
    assert got[0].isnan().all() and torch.equal(got[1], want[1])


def test_non_finite_queries_stay_in_their_head(gpu_lib):
    k3 = gpu_lib
    c = Case([200, 700], seed=11)
    want = c.run(k3, split=128)
    c.q[0, 5, 7] = float("nan")
    c.q[1, 60, 100] = float("inf")
    c.q[1, 90, LORA + 3] = float("nan")
    got = c.run(k3, split=128)
    assert got[0, 5].isnan().all() and got[1, 60].isnan().all() and got[1, 90].isnan().all()
    rest = torch.ones(2, H, dtype=torch.bool, device="cuda")
    rest[0, 5] = rest[1, 60] = rest[1, 90] = False
    assert torch.equal(got[rest], want[rest])


def test_zero_queries_average_the_rows(gpu_lib):
    c = Case([200], seed=12)
    c.q.zero_()
    c.check(c.run(gpu_lib))


def test_a_slot_does_not_depend_on_its_batch(gpu_lib):
    k3 = gpu_lib
    c = Case([4500, 64, 0, 777, 129], seed=13).stale()
    whole = c.run(k3, max_ctx=4500)
    again = c.run(k3, max_ctx=4500)
    assert torch.equal(whole, again)
    for b in range(5):
        assert torch.equal(c.run(k3, max_ctx=4500, slots=[b])[0], whole[b]), b
    order = [3, 0, 4, 2, 1]
    assert torch.equal(c.run(k3, max_ctx=4500, slots=order), whole[order])


def test_every_way_to_add_splits_up_gives_the_same_bits(gpu_lib):
    """One slot in one split apart, the sums of a slot's splits are taken by the expansion (few slots) or by a kernel before it,
    a warp or four a row, up to four records at once or in turn."""
    k3 = gpu_lib
    g = np.random.default_rng(14)
    ctx = [int(x) for x in g.integers(1, 1500, 20)]
    ctx[:3] = [512, 385, 1500]
    c = Case(ctx, seed=14).stale()
    whole = c.run(k3, split=128, max_ctx=1500)
    c.check(whole)
    for slots in (list(range(16)), [2, 0, 19, 7, 11], [4, 2, 1], [2]):
        assert torch.equal(c.run(k3, split=128, max_ctx=1500, slots=slots), whole[slots]), slots
    few = [b for b in range(20) if ctx[b] <= 512]
    many = (few * 20)[:17]
    assert torch.equal(c.run(k3, split=128, max_ctx=512, slots=many), whole[many])
    assert torch.equal(c.run(k3, split=128, max_ctx=512, slots=many[:9]), whole[many[:9]])


@pytest.mark.parametrize("exponent", [-130, -40, 0, 30])
def test_queries_of_very_different_sizes(gpu_lib, exponent):
    """Heads 2^-18 to 2^18 apart, the entries of a head too, about 2^exponent (bf16's smallest among them)."""
    c = Case([70, 260], seed=15)
    g = np.random.default_rng(15)
    q = g.standard_normal((2, H, ROW)) * 2.0 ** (exponent + g.uniform(-9, 9, (2, H, 1)) + g.uniform(-9, 9, (2, H, ROW)))
    c.q = torch.from_numpy(q.astype(np.float32)).cuda().bfloat16()
    c.check(c.run(gpu_lib))


def test_planned_splits(gpu_lib):
    c = Case([900, 1, 400, 130, 257, 64] * 3, seed=16)
    c.check(c.run(gpu_lib, split=gpu_lib.quant_split_tokens(18, 900, MOST)))


def test_captured_and_replayed_with_new_lengths_on_another_stream(gpu_lib):
    k3 = gpu_lib
    c = Case([500, 130, 64, 0], seed=14).stale()
    slab, table = torch.from_numpy(c.blocks).cuda(), torch.from_numpy(c.table).cuda()
    ctx = torch.tensor(c.ctx, dtype=torch.int32).cuda()
    ws = torch.full((k3.quant_decode_workspace_bytes(4, 500, MOST, 0, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(4, H, V, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: k3.quant_decode(c.q, slab, c.layer, table, ctx, c.w, SCALE_BITS, out, ws, 500, MOST, 0, 128)  # noqa: E731
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    for lens in ([500, 130, 64, 0], [1, 0, 333, 0], [65, 128, 2, 0]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        c.ctx = lens
        c.check(out)
        assert torch.equal(out, c.run(k3, split=128, max_ctx=500))


def test_two_streams_at_once_with_workspaces_of_their_own(gpu_lib):
    k3 = gpu_lib
    a, b = Case([900, 40], seed=15).stale(), Case([300] * 3, seed=16).stale()
    want = [a.run(k3, split=128), b.run(k3, 50, 4)]
    work = []
    for c, window, sink, split in ((a, MOST, 0, 128), (b, 50, 4, 0)):
        B, most = len(c.ctx), max(c.ctx)
        args = (c.q, torch.from_numpy(c.blocks).cuda(), c.layer, torch.from_numpy(c.table).cuda(),
                torch.tensor(c.ctx, dtype=torch.int32).cuda(), c.w, SCALE_BITS,
                torch.empty(B, H, V, dtype=torch.bfloat16, device="cuda"),
                torch.empty(k3.quant_decode_workspace_bytes(B, most, window, sink, split), dtype=torch.uint8, device="cuda"), most,
                window, sink, split)
        work.append((torch.cuda.Stream(), args))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, args in work:
            with torch.cuda.stream(s):
                k3.quant_decode(*args)
    torch.cuda.synchronize()
    for (_, args), w in zip(work, want):
        assert torch.equal(args[7], w)


def test_an_appended_token_is_attended_to_and_read_back(gpu_lib):
    """A decode step as a server runs it: the step's row is quantised into its page, then the slot attends to it; a prefill
    that goes on from the cache reads the pages back and gets the same attention from the bf16 kernels."""
    k3 = gpu_lib
    c = Case([129, 64, 200], seed=17)
    slab, table = torch.from_numpy(c.blocks).cuda(), torch.from_numpy(c.table).cuda()
    ctx = torch.tensor(c.ctx, dtype=torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(17)
    q = torch.randn(3, H, 192, generator=g, device="cuda").bfloat16()
    kv = torch.randn(3, ROW, generator=g, device="cuda").bfloat16()
    inv = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
    k3.quant_norm_rope_append(q, q, slab, c.layer, table, ctx - 1, None, kv[:, :LORA], kv[:, LORA:], inv_freq=inv)
    k3.absorb_q(q, c.w, c.q)
    ws = torch.empty(k3.quant_decode_workspace_bytes(3, 200, 200), dtype=torch.uint8, device="cuda")
    out = torch.empty(3, H, V, dtype=torch.bfloat16, device="cuda")
    k3.quant_decode(c.q, slab, c.layer, table, ctx, c.w, SCALE_BITS, out, ws, 200)
    torch.cuda.synchronize()
    assert not np.array_equal(c.blocks, slab.cpu().numpy())
    c.blocks = slab.cpu().numpy()
    c.check(out)
    back = torch.zeros(slab.shape[0], 2, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(slab.shape[0], dtype=torch.int32, device="cuda")
    k3.quant_read_pages(back, slab, ids, ids)
    ws = torch.empty(k3.window_decode_workspace_bytes(3, 200, 200), dtype=torch.uint8, device="cuda")
    other = torch.empty_like(out)
    k3.window_decode(c.q, back, c.layer, table, ctx, c.w, SCALE_BITS, other, ws, 200, 200)
    torch.cuda.synchronize()
    c.check(other)
