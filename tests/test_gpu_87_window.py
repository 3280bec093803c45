"""Attention over a sliding window and the first tokens (k3mla_window_decode, k3mla_window_chunk_decode)
against the definition in 64 bits; the bound of every element is worked out in window_ref.out_tolerance."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla, synth
from tests import window_ref as ref

pytestmark = pytest.mark.gpu

PAGE, H, V, ROW = 64, 96, 128, 576
SCALE_BITS, SCALE = 0x3D94, 0.072265625


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Case:
    """Slots of lens[b] cached tokens in shuffled pages of a two-layer slab (layer 1 is used)."""

    def __init__(self, seed, lens, n_rows, L=2, spare=2, layer=1):
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        pages = [(max(n, 0) + PAGE - 1) // PAGE for n in lens]
        self.n_pages, self.cols, self.layer = sum(pages) + spare, max(1, max(pages)), layer
        ids = self.rng.permutation(self.n_pages)
        self.table = np.full((len(lens), self.cols), -1, np.int32)
        k = 0
        for b, m in enumerate(pages):
            self.table[b, :m] = ids[k:k + m]
            k += m
        self.lens = np.array(lens, np.int32)
        self.slab = torch.randn(self.n_pages, L, PAGE, ROW, generator=self.g, device="cuda").bfloat16()
        self.q = torch.randn(n_rows, H, ROW, generator=self.g, device="cuda")
        self.q[:, :, :512] *= 0.5
        self.q = self.q.bfloat16()
        self.w = (torch.randn(H * 256, 512, generator=self.g, device="cuda") * 512 ** -0.5).bfloat16()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.max_ctx = self.cols * PAGE

    def poison(self, seen):
        """NaN or infinity into every cached row that no token row sees (seen: per slot a set of positions),
        the rows past each slot's tokens and the pages of no slot among them; pages without a seen token leave
        the table."""
        bad = torch.tensor([float("nan"), float("inf"), float("-inf")]).bfloat16().cuda()
        keep = torch.zeros(self.n_pages, PAGE, dtype=torch.bool)
        for b, s in enumerate(seen):
            for t in s:
                page = self.table[b, t // PAGE]
                if 0 <= page < self.n_pages:
                    keep[page, t % PAGE] = True
            for lp in range(self.cols):
                if not any(t // PAGE == lp for t in s):
                    self.table[b, lp] = -1
        where = (~keep).nonzero()
        pick = bad[torch.randint(3, (len(where), ROW), generator=self.g, device="cuda")]
        self.slab[where[:, 0].cuda(), self.layer, where[:, 1].cuda()] = pick

    def decode(self, window, sink, split=0, table=None, q=None, ctx=None, max_ctx=None, ws=None, slots=None):
        slots = np.arange(len(self.lens)) if slots is None else np.asarray(slots)
        ctx = self.lens if ctx is None else ctx
        table = self.table if table is None else table
        B, max_ctx = len(slots), max_ctx or self.max_ctx
        out = torch.full((B, H, V), float("nan"), dtype=torch.bfloat16, device="cuda")
        need = k3mla.window_decode_workspace_bytes(B, max_ctx, window, sink, split)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda") if ws is None else ws
        q = (self.q if q is None else q)[torch.from_numpy(slots).cuda()].contiguous()
        k3mla.window_decode(q, self.slab, self.layer, torch.from_numpy(table[slots]).cuda(),
                            torch.from_numpy(np.asarray(ctx, np.int32)[slots]).cuda(), self.w, SCALE_BITS, out, ws, max_ctx,
                            window, sink, split, dev_err=self.err)
        torch.cuda.synchronize()
        return out

    def chunk(self, pos0, start, window, sink, max_ctx=None):
        R, B, max_ctx = self.q.shape[0], len(pos0), max_ctx or self.max_ctx
        out = torch.full((R, H, V), float("nan"), dtype=torch.bfloat16, device="cuda")
        ws = torch.full((k3mla.window_chunk_decode_workspace_bytes(B, R, max_ctx),), 0xFF, dtype=torch.uint8, device="cuda")
        k3mla.window_chunk_decode(self.q, self.slab, self.layer, torch.from_numpy(self.table).cuda(),
                                  torch.from_numpy(np.asarray(pos0, np.int32)).cuda(),
                                  torch.from_numpy(np.asarray(start, np.int32)).cuda(), self.w, SCALE_BITS, out, ws, max_ctx,
                                  window, sink, dev_err=self.err)
        torch.cuda.synchronize()
        return out

    def check(self, got, slot_of, n_of, window, sink, rows=None):
        """Every listed row r of `got`: slot slot_of[r], context n_of[r]."""
        got, q, w = f64(got), f64(self.q), f64(self.w)
        slab = f64(self.slab[:, self.layer:self.layer + 1])
        worst = 0.0
        for r in range(len(slot_of)) if rows is None else rows:
            out, o, p, kept = ref.attend(q[r], slab, 0, self.table[max(slot_of[r], 0)], n_of[r], window, sink, w, SCALE)
            if n_of[r] <= 0:
                assert np.all(got[r] == 0), r
                continue
            tol = ref.out_tolerance(out, o, p, kept, w, np.abs(q[r]) @ np.abs(kept).T * SCALE)
            e = np.abs(got[r] - out)
            assert np.all(e <= tol), (r, slot_of[r], n_of[r], float(np.nanmax(e / tol)), bool(np.isnan(got[r]).any()))
            worst = max(worst, float((e / tol).max()))
        return worst


def seen_sets(lens, window, sink):
    return [set(ref.visible(int(n), window, sink).tolist()) for n in lens]


@pytest.mark.parametrize("window,sink", [(1, 0), (64, 4), (100, 0), (63, 64), (65, 65), (128, 1), (7, 200), (1000, 0),
                                         (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("lens", [[1], [130], [5, 64, 65, 0, 200, 129, 333]])
def test_decode_small(gpu_lib, lens, window, sink):
    c = Case(len(lens) + window % 1000, lens, len(lens))
    c.poison(seen_sets(lens, window, sink))
    got = c.decode(window, sink)
    c.check(got, list(range(len(lens))), lens, window, sink)
    assert c.err.item() == 0


@pytest.mark.parametrize("split", [128, 256, 0])
@pytest.mark.parametrize("window,sink", [(700, 70), (64, 1), (1024, 0), (300, 128)])
def test_decode_splits(gpu_lib, window, sink, split):
    lens = [1200, 700, 1, 0, 64, 129, 1025]
    c = Case(7 + window, lens, len(lens))
    c.poison(seen_sets(lens, window, sink))
    got = c.decode(window, sink, split)
    c.check(got, list(range(len(lens))), lens, window, sink)
    assert c.err.item() == 0


def test_decode_more_units_than_clusters(gpu_lib):
    # 200 slots of 0 .. 300 tokens, up to three units a cluster, single and several splits side by side
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 300, 200)]
    for window, sink, split in ((150, 3, 0), (290, 0, 128)):
        c = Case(3 + split, lens, len(lens))
        c.poison(seen_sets(lens, window, sink))
        got = c.decode(window, sink, split)
        c.check(got, list(range(200)), lens, window, sink, rows=range(0, 200, 3))
        assert c.err.item() == 0


def test_many_units_of_one_cluster(gpu_lib):
    # 900 slots of one to three pages: a cluster's roles pass a dozen units, one or two pages each
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(1, 190, 900)]
    c = Case(69, lens, len(lens))
    got = c.decode(60, 3)
    c.check(got, list(range(900)), lens, 60, 3, rows=range(0, 900, 19))
    for _ in range(5):
        assert torch.equal(c.decode(60, 3), got)
    assert c.err.item() == 0


def test_decode_long(gpu_lib):
    lens = [9000, 5000, 4096]
    c = Case(11, lens, 3)
    window, sink = 4500, 100
    c.poison(seen_sets(lens, window, sink))
    for split in (0, 128, k3mla.window_split_tokens(3, c.max_ctx, window, sink)):
        got = c.decode(window, sink, split)
        c.check(got, [0, 1, 2], lens, window, sink)
    assert c.err.item() == 0


def test_reference_max_that_moves(gpu_lib):
    # scores that rise by far more than the lazy maximum's slack, page after page, and fall again
    lens = [640, 640]
    c = Case(12, lens, 2)
    t = np.arange(640)
    for b, growth in enumerate((np.minimum(t, 500) / 16.0, -t / 16.0)):
        for lp in range(10):
            page = int(c.table[b, lp])
            f = torch.from_numpy(growth[64 * lp:64 * lp + 64]).float().cuda()
            c.slab[page, 1] = (c.slab[page, 1].float() * 0.05).bfloat16()
            c.slab[page, 1, :, 575] = f.bfloat16()
    c.q[:, :, 575] = 40.0
    for split in (0, 128):
        for window, sink in ((640, 0), (300, 70)):
            got = c.decode(window, sink, split)
            c.check(got, [0, 1], lens, window, sink)


def test_holes_and_bad_pages_read_as_zero(gpu_lib):
    lens = [400, 400]
    c = Case(13, lens, 2)
    c.table[0, 2] = -1
    c.table[0, 6] = -1
    c.table[1, 5] = c.n_pages
    got = c.decode(300, 64)
    assert c.err.item() == k3mla.DEV_BAD_PAGE
    c.check(got, [0, 1], lens, 300, 64)


def test_context_beyond_the_table_is_clamped_and_flagged(gpu_lib):
    c = Case(14, [200], 1)
    got = c.decode(100, 4, ctx=[10 ** 6])
    assert c.err.item() == k3mla.DEV_CTX
    c.check(got, [0], [256], 100, 4)
    c.err.zero_()
    got = c.decode(100, 4, max_ctx=150)
    assert c.err.item() == k3mla.DEV_CTX
    c.check(got, [0], [150], 100, 4)
    assert torch.all(c.decode(100, 4, ctx=[-5]) == 0)


def test_a_slots_bits_depend_on_the_slot_alone(gpu_lib):
    lens = [900, 65, 0, 300, 64, 1000]
    c = Case(15, lens, len(lens))
    for split in (0, 256):
        whole = c.decode(500, 10, split)
        for b in range(len(lens)):
            assert torch.equal(c.decode(500, 10, split, slots=[b])[0], whole[b])
        assert torch.equal(c.decode(500, 10, split), whole)
        # the same rows in other pages
        perm = c.rng.permutation(c.n_pages)
        moved = torch.empty_like(c.slab)
        moved[torch.from_numpy(perm).cuda()] = c.slab
        old, c.slab = c.slab, moved
        table = np.where(c.table >= 0, perm[np.maximum(c.table, 0)], -1).astype(np.int32)
        assert torch.equal(c.decode(500, 10, split, table=table), whole)
        c.slab = old


def test_a_slots_bits_do_not_depend_on_who_adds_its_splits_up(gpu_lib):
    # alone, among 5, 16 and 17 slots and with lists of more than eight splits: the sums are one order everywhere
    lens = [900, 65, 0, 300, 64, 1000, 1, 500, 1300, 128, 700, 20, 640, 333, 90, 1100, 800]
    c = Case(68, lens, len(lens))
    for window, split in ((700, 128), (1300, 128), (700, 256)):
        whole = c.decode(window, 10, split)
        c.check(whole, list(range(17)), lens, window, 10)
        for some in ([5], [8, 2, 15], [0, 1, 2, 3, 4], list(range(16))):
            got = c.decode(window, 10, split, slots=some)
            assert torch.equal(got, whole[some])


def test_wide_window_is_the_full_decode(gpu_lib):
    # k3mla_paged_decode lands its scores in bf16, so the two agree within those landings: each score is off by
    # 2^-8 of itself, twice, and an output by at most the largest weight error of its row
    lens = [700, 130]
    c = Case(16, lens, 2)
    got = f64(c.decode(10 ** 6, 0))
    out = torch.empty(2, H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(k3mla.decode_workspace_bytes(2, c.max_ctx), dtype=torch.uint8, device="cuda")
    k3mla.paged_decode(c.q, c.slab, 1, torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda(), c.w, SCALE_BITS, out,
                       ws, c.max_ctx)
    torch.cuda.synchronize()
    full, q, w, slab = f64(out), f64(c.q), f64(c.w), f64(c.slab[:, 1:2])
    for b in range(2):
        o64, o, p, rows = ref.attend(q[b], slab, 0, c.table[b], lens[b], 10 ** 6, 0, w, SCALE)
        s_abs = np.abs(q[b]) @ np.abs(rows).T * SCALE
        tol = ref.out_tolerance(o64, o, p, rows, w, s_abs)
        s = np.abs(q[b] @ rows.T * SCALE)
        d = 2.0 ** -7 * 1.1 * s + 2.0 ** -8
        wuv = np.abs(w.reshape(H, 256, 512)[:, 128:])
        more = np.einsum("hvk,hk->hv", wuv, np.einsum("ht,tk->hk", p * d, np.abs(rows[:, :512])) +
                         (p * d).sum(-1)[:, None] * np.abs(o) + 2.0 ** -8 * np.abs(o)) + 2.0 ** -8 * np.abs(o64)
        assert np.all(np.abs(got[b] - full[b]) <= tol + more)


def test_rows_past_2_31_elements(gpu_lib):
    n_pages, L = 1024, 64
    c = Case(17, [100, 64], 2)
    slab = torch.zeros(n_pages, L, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
    assert slab.numel() > 2 ** 31
    slab[-c.n_pages:, -1] = c.slab[:, 1]
    c.table = np.where(c.table >= 0, c.table + n_pages - c.n_pages, -1).astype(np.int32)
    c.slab, c.layer, c.n_pages = slab, L - 1, n_pages
    got = c.decode(70, 3)
    c.check(got, [0, 1], [100, 64], 70, 3)


def rows_to(start, pos0, R):
    at = ref.rows_of(pos0, start, R)
    return [b for b, _ in at], [p + 1 if b >= 0 else 0 for b, p in at]


@pytest.mark.parametrize("window,sink", [(1, 0), (64, 4), (100, 64), (65, 0), (3, 130), (10 ** 6, 0)])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([130], [130]), ([5, 300, 64, 90, 0], [5, 7, 4, 1, 0]), ([700, 260], [33, 66])])
def test_chunk_small(gpu_lib, lens, new, window, sink):
    R = sum(new)
    c = Case(20 + window % 1000 + len(lens), lens, R)
    pos0 = [n - m for n, m in zip(lens, new)]
    start = np.concatenate([[0], np.cumsum(new)])
    slot, n = rows_to(start, pos0, R)
    seen = [set().union(*[set(ref.visible(n[r], window, sink).tolist()) for r in range(R) if slot[r] == b] or [set()])
            for b in range(len(lens))]
    c.poison(seen)
    got = c.chunk(pos0, start, window, sink)
    c.check(got, slot, n, window, sink, rows=range(0, R, max(1, R // 24)))
    assert c.err.item() == 0


def test_chunk_more_units_than_clusters(gpu_lib):
    new = [200, 1, 63, 0, 130, 5, 77]
    lens = [400, 900, 63, 10, 131, 2000, 300]
    R = sum(new)
    c = Case(31, lens, R)
    pos0 = [n - m for n, m in zip(lens, new)]
    start = np.concatenate([[0], np.cumsum(new)])
    slot, n = rows_to(start, pos0, R)
    for window, sink in ((129, 2), (1500, 0)):
        got = c.chunk(pos0, start, window, sink)
        c.check(got, slot, n, window, sink, rows=range(0, R, 7))
    assert c.err.item() == 0


def test_chunk_of_many_tiles(gpu_lib):
    # enough rows for several CTAs a head in the expansion, the last tile a part of one
    c = Case(71, [1200], 1100)
    got = c.chunk([100], [0, 1100], 30, 2)
    c.check(got, [0] * 1100, [101 + r for r in range(1100)], 30, 2, rows=[*range(0, 1100, 61), 1023, 1024, 1087, 1088, 1099])
    assert c.err.item() == 0


def test_chunk_many_slots(gpu_lib):
    # more slots than one warp scans at once, most of them without new tokens
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 100, 150)]
    new = [int(rng.integers(1, min(6, n) + 1)) if b % 3 == 0 else 0 for b, n in enumerate(lens)]
    R = sum(new)
    c = Case(32, lens, R)
    pos0 = [n - m for n, m in zip(lens, new)]
    start = np.concatenate([[0], np.cumsum(new)])
    slot, n = rows_to(start, pos0, R)
    got = c.chunk(pos0, start, 40, 1)
    c.check(got, slot, n, 40, 1, rows=range(0, R, 4))


def test_chunk_rows_outside_every_slot_and_before_the_first_token(gpu_lib):
    c = Case(33, [200, 90], 14)
    start, pos0 = [2, 8, 12], [190, -2]         # rows 0, 1, 12, 13 are no slot's; slot 1 starts two rows early
    slot, n = rows_to(start, pos0, 14)
    got = c.chunk(pos0, start, 50, 4)
    c.check(got, slot, n, 50, 4)
    assert torch.all(got[[0, 1, 8, 9, 12, 13]] == 0)
    assert c.err.item() == 0


def test_chunk_context_is_clamped_and_flagged(gpu_lib):
    c = Case(34, [128], 6)
    got = c.chunk([125], [0, 6], 60, 0)         # positions 125 .. 130 on a 128-token table
    slot, n = [0] * 6, [126, 127, 128, 128, 128, 128]
    c.check(got, slot, n, 60, 0)
    assert c.err.item() == k3mla.DEV_CTX


def test_chunk_nan_reaches_only_the_rows_that_see_it(gpu_lib):
    # token 200 is row 4's own: rows 0..3 come before it; with a window of 6 rows 10.. no longer see it
    c = Case(35, [220], 24)
    c.slab[int(c.table[0, 200 // PAGE]), 1, 200 % PAGE, 3] = float("nan")
    c.slab[int(c.table[0, 207 // PAGE]), 1, 207 % PAGE] = float("inf")
    got = c.chunk([196], [0, 24], 6, 2)
    bad = torch.isnan(got.float()).flatten(1).all(1).cpu().numpy()
    some = torch.isnan(got.float()).flatten(1).any(1).cpu().numpy()
    want = np.array([any(t in (200, 207) for t in ref.visible(197 + r, 6, 2)) for r in range(24)])
    assert np.array_equal(bad, want) and np.array_equal(some, want)
    clean = c.slab.clone()
    clean[torch.isnan(clean) | torch.isinf(clean)] = 0
    c.slab = clean
    c.check(got, [0] * 24, [197 + r for r in range(24)], 6, 2, rows=np.flatnonzero(~want))


def test_chunk_row_is_its_decode(gpu_lib):
    # a chunk's row against the decode of the same context: both within the bound of the definition
    c = Case(36, [500], 9)
    got = c.chunk([491], [0, 9], 200, 70)
    one = Case(36, [500], 9)
    for r in (0, 3, 8):
        d = one.decode(200, 70, ctx=[492 + r], q=c.q[r:r + 1])
        e = np.abs(f64(d[0]) - f64(got[r]))
        _, o, p, rows = ref.attend(f64(c.q)[r], f64(c.slab[:, 1:2]), 0, c.table[0], 492 + r, 200, 70, f64(c.w), SCALE)
        out = ref.attend(f64(c.q)[r], f64(c.slab[:, 1:2]), 0, c.table[0], 492 + r, 200, 70, f64(c.w), SCALE)[0]
        assert np.all(e <= 2 * ref.out_tolerance(out, o, p, rows, f64(c.w), np.abs(f64(c.q)[r]) @ np.abs(rows).T * SCALE))


def test_two_graphs_on_one_workspace(gpu_lib):
    a, b = Case(40, [700, 100], 2), Case(41, [300, 900], 2)
    split = 256
    need = max(k3mla.window_decode_workspace_bytes(2, x.max_ctx, 500, 5, split) for x in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    eager = [x.decode(500, 5, split) for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        args = [torch.from_numpy(v).cuda() for v in (x.table, x.lens)]
        out = torch.empty(2, H, V, dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            k3mla.window_decode(x.q, x.slab, 1, *args, x.w, SCALE_BITS, out, ws, x.max_ctx, 500, 5, split)
        graphs.append((g, args))
        outs.append(out)
    ws.fill_(0xFF)
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, e) for o, e in zip(outs, eager))


def test_on_another_stream_and_two_calls_in_a_row(gpu_lib):
    c = Case(42, [700, 100, 33], 3)
    want = c.decode(200, 5)
    table, lens = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    ws = torch.empty(k3mla.window_decode_workspace_bytes(3, c.max_ctx, 200, 5), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(3, H, V, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for o in outs:
        k3mla.window_decode(c.q, c.slab, 1, table, lens, c.w, SCALE_BITS, o, ws, c.max_ctx, 200, 5, stream=s)
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_decode_steps_of_a_windowed_layer(gpu_lib):
    """The operators as a decode loop uses them: claim, norms + rotation + append, absorption, windowed
    decode, and pages behind the window given back."""
    window, sink, B = 100, 3, 3
    pool = k3mla.Pool(n_slots=B, max_ctx=512, shuffle_seed=4)
    g = torch.Generator(device="cuda").manual_seed(50)
    slab = torch.full((pool.n_pages, 2, PAGE, ROW), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = (torch.randn(H * 256, 512, generator=g, device="cuda") * 512 ** -0.5).bfloat16()
    wq, wc, wk = [(1 + 0.1 * torch.randn(n, generator=g, device="cuda")).bfloat16() for n in (192, 512, 64)]
    inv = (10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)).float()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(k3mla.window_decode_workspace_bytes(B, 512, window, sink), dtype=torch.uint8, device="cuda")
    cws = torch.empty(k3mla.window_chunk_decode_workspace_bytes(B, 400, 512), dtype=torch.uint8, device="cuda")
    freed, lens = 0, [0] * B
    for new in ([190, 64, 1], [1, 1, 1], [1, 1, 1], [60, 0, 130], [1, 1, 1]):
        decode = new == [1, 1, 1]
        pos0 = np.array(lens, np.int32)
        lens = [n + m for n, m in zip(lens, new)]
        assert pool.ensure_all(lens) == 0
        table = torch.from_numpy(pool.table()).cuda()
        R = sum(new)
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        p0 = torch.from_numpy(pos0).cuda()
        q = torch.randn(R, H, 192, generator=g, device="cuda").bfloat16()
        kv = torch.randn(R, ROW, generator=g, device="cuda").bfloat16()
        q_abs = torch.empty(R, H, ROW, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(R, H, V, dtype=torch.bfloat16, device="cuda")
        k3mla.norm_rope_append(q, q, slab, 1, table, p0, None if decode else start, kv[:, :512], kv[:, 512:], q_weight=wq,
                               c_weight=wc, k_weight=wk, inv_freq=inv, dev_err=err)
        k3mla.absorb_q(q, w, q_abs)
        if decode:
            k3mla.window_decode(q_abs, slab, 1, table, p0 + 1, w, SCALE_BITS, out, ws, 512, window, sink, dev_err=err)
        else:
            k3mla.window_chunk_decode(q_abs, slab, 1, table, p0, start, w, SCALE_BITS, out, cws, 512, window, sink, dev_err=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        c = Case.__new__(Case)
        c.q, c.w, c.slab, c.layer, c.table = q_abs, w, slab, 1, pool.table()
        slot = [b for b in range(B) for _ in range(new[b])]
        n = [int(pos0[b]) + j + 1 for b in range(B) for j in range(new[b])]
        c.check(out, slot, n, window, sink, rows=range(0, R, max(1, R // 15)))
        for b in range(B):
            row = pool.table()[b].copy()
            given = pool.trim(b, lens[b], window, sink)
            assert given >= 0
            for page in row[(row >= 0) & (pool.table()[b] < 0)]:
                slab[int(page)] = float("nan")         # a freed page may hold anything
            freed += given
    assert freed > 0
    pool.close()


def test_refusals_of_the_binding(gpu_lib):
    c = Case(60, [100], 1)
    out = torch.empty(1, H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(k3mla.window_decode_workspace_bytes(1, 128, 10), dtype=torch.uint8, device="cuda")
    table, ctx = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    args = [c.q, c.slab, 1, table, ctx, c.w, SCALE_BITS, out, ws, 128, 10]
    k3mla.window_decode(*args)
    for at, bad in ((0, c.q.float()), (0, c.q[:, :90]), (1, c.slab.cpu()), (2, 2), (3, table.long()), (3, table.repeat(2, 1)),
                    (4, ctx.repeat(2)), (5, c.w[:-1]), (6, 0), (6, 0xBD94), (6, 0x7F80), (7, out.half()), (8, ws[:-256]),
                    (9, 0), (10, 0)):
        wrong = list(args)
        wrong[at] = bad
        with pytest.raises(k3mla.K3mlaError):
            k3mla.window_decode(*wrong)
    with pytest.raises(k3mla.K3mlaError):
        k3mla.window_decode(*args, n_sink=-1)
    with pytest.raises(k3mla.K3mlaError):
        k3mla.window_decode(*args, split_tokens=100)
    torch.cuda.synchronize()


def test_zero_queries_beside_unseen_infinities(gpu_lib):
    # every score is 0, and a zero query times an unseen infinity is the NaN that gives it away
    lens = [200, 77]
    c = Case(61, lens, 2)
    c.q.zero_()
    c.poison(seen_sets(lens, 70, 3))
    for split in (0, 128):
        c.check(c.decode(70, 3, split), [0, 1], lens, 70, 3)
    c = Case(62, [150], 9)
    c.q.zero_()
    n = [142 + r for r in range(9)]
    c.poison([set().union(*[set(ref.visible(x, 40, 3).tolist()) for x in n])])
    c.check(c.chunk([141], [0, 9], 40, 3), [0] * 9, n, 40, 3)


@pytest.mark.parametrize("first,rest", [(0.0, 1.0), (2.0 ** -30, 1.0), (2.0 ** -9, 1.0), (1.0, 2.0 ** -20), (2.0 ** 12, 1.0),
                                        (1.0, 0.0), (0.0, 0.0)])
def test_first_dims_unlike_the_others(gpu_lib, first, rest):
    # the power of two of a row of o_lat starts from its first 32 entries
    lens = [400, 130, 64]
    c = Case(63, lens, 3)
    c.slab[..., :32] *= first
    c.slab[..., 32:512] *= rest
    for split in (0, 128):
        c.check(c.decode(300, 3, split), [0, 1, 2], lens, 300, 3)
    c = Case(64, [300], 7)
    c.slab[..., :32] *= first
    c.slab[..., 32:512] *= rest
    c.check(c.chunk([293], [0, 7], 90, 3), [0] * 7, [294 + r for r in range(7)], 90, 3)


@pytest.mark.parametrize("power", [60, -60])
def test_large_and_small_latents(gpu_lib, power):
    lens = [400, 100]
    c = Case(65, lens, 2)
    c.slab *= 2.0 ** power
    c.q *= 2.0 ** -power
    for split in (0, 128):
        c.check(c.decode(300, 3, split), [0, 1], lens, 300, 3)


def test_two_streams_at_once(gpu_lib):
    # each call has its own workspace and output; they share the cache
    c = Case(66, [900, 400, 1000], 3)
    want = [c.decode(700, 5, split) for split in (0, 128)]
    table, lens = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros(3, H, V, dtype=torch.bfloat16, device="cuda") for _ in range(8)] for _ in range(2)]
    ws = [torch.empty(k3mla.window_decode_workspace_bytes(3, c.max_ctx, 700, 5, split), dtype=torch.uint8, device="cuda")
          for split in (0, 128)]
    torch.cuda.synchronize()
    for i in range(8):
        for s, split in enumerate((0, 128)):
            k3mla.window_decode(c.q, c.slab, 1, table, lens, c.w, SCALE_BITS, outs[s][i], ws[s], c.max_ctx, 700, 5, split,
                                stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[s]) for s in range(2) for o in outs[s])


def test_chunk_replayed_with_other_lengths(gpu_lib):
    # a captured call reads positions and row ranges at its replay
    c = Case(67, [300, 200], 12)
    table = torch.from_numpy(c.table).cuda()
    pos0 = torch.tensor([290, 198], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 10, 12], dtype=torch.int32, device="cuda")
    out = torch.empty(12, H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(k3mla.window_chunk_decode_workspace_bytes(2, 12, c.max_ctx), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        k3mla.window_chunk_decode(c.q, c.slab, 1, table, pos0, start, c.w, SCALE_BITS, out, ws, c.max_ctx, 100, 2)
    for p, s in (([290, 198], [0, 10, 12]), ([0, 191], [0, 3, 12]), ([100, 5], [0, 0, 7])):
        pos0.copy_(torch.tensor(p))
        start.copy_(torch.tensor(s))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.chunk(p, s, 100, 2))
        slot, n = rows_to(s, p, 12)
        c.check(out, slot, n, 100, 2)


def test_tensors_of_another_device_are_refused(gpu_lib, monkeypatch):
    # (one GPU: the current device is made to look like another one)
    c = Case(70, [100], 1)
    out = torch.empty(1, H, V, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    table, ctx = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    rows = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, H, 192, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(1, ROW, dtype=torch.bfloat16, device="cuda")
    calls = (lambda: k3mla.window_decode(c.q, c.slab, 1, table, ctx, c.w, SCALE_BITS, out, ws, 128, 10),
             lambda: k3mla.window_chunk_decode(c.q, c.slab, 1, table, ctx, rows, c.w, SCALE_BITS, out, ws, 128, 10),
             lambda: k3mla.compact_rows(c.slab, table, rows, rows),
             lambda: k3mla.norm_rope_append(q, q, c.slab, 1, table, ctx, None, kv[:, :512], kv[:, 512:]))
    monkeypatch.setattr(k3mla, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(k3mla.K3mlaError, match="is on cuda:0"):
            call()
    with pytest.raises(k3mla.K3mlaError, match="is on cuda:0"):
        k3mla._rows(kv, 1, "c_kv", 512, 1)
    with pytest.raises(k3mla.K3mlaError, match="CUDA tensor"):
        k3mla.window_decode(c.q, c.slab.cpu(), 1, table, ctx, c.w, SCALE_BITS, out, ws, 128, 10)
