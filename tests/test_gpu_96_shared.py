"""Decode for slots that share their first pages, against the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import window_ref as wr

pytestmark = pytest.mark.gpu
H, V, LORA, PAGE, ROW = 96, 128, 512, 64, 576
SCALE_BITS, SCALE = 0x3D94, 0.072265625
MOST = 1 << 30


class Case:
    """Groups [(contexts, shared tokens)], then slots that share nothing; pages scattered over the slab."""

    def __init__(self, groups, alone=(), seed=0, layers=2, layer=1, extra_cols=0):
        g = np.random.default_rng(seed)
        self.layer = layer
        self.ctx = [n for ctx, _ in groups for n in ctx] + list(alone)
        self.start = np.concatenate([[0], np.cumsum([len(ctx) for ctx, _ in groups])]).astype(np.int32)
        self.shared = np.array([s for _, s in groups], np.int32)
        B = len(self.ctx)
        cols = max([1] + [-(-max(n, 0) // PAGE) for n in self.ctx] + [s // PAGE for s in self.shared]) + extra_cols
        pages = sum(s // PAGE for s in self.shared) + sum(-(-max(n, 0) // PAGE) for n in self.ctx) + 2
        ids = list(g.permutation(pages))
        self.table = np.full((B, cols), -1, np.int32)
        self.first = np.zeros(B, int)
        for i, (_, s) in enumerate(groups):
            common = [ids.pop() for _ in range(s // PAGE)]
            for b in range(self.start[i], self.start[i + 1]):
                self.table[b, :len(common)] = common
                self.first[b] = len(common)
        for b, n in enumerate(self.ctx):
            for lp in range(self.first[b], -(-max(n, 0) // PAGE)):
                self.table[b, lp] = ids.pop()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
        self.slab = rand(pages, layers, PAGE, ROW).bfloat16()
        self.q = (rand(B, H, ROW) * 0.7).bfloat16()
        self.w = (rand(H * 256, LORA) * LORA ** -0.5).bfloat16()
        self.max_shared = max([0] + [int(s) for s in self.shared])
        self.max_own = max([1] + [n - PAGE * f for n, f in zip(self.ctx, self.first)])
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def args(self):
        dev = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
        return self.slab, self.layer, dev(self.table), dev(self.ctx), dev(self.start), dev(self.shared), self.w, SCALE_BITS

    def run(self, k3, shared_split=0, own_split=0, max_shared=None, max_own=None):
        B = len(self.ctx)
        ms, mo = self.max_shared if max_shared is None else max_shared, max_own or self.max_own
        ws = torch.full((k3.shared_decode_workspace_bytes(B, ms, mo, shared_split, own_split),), 0xFF, dtype=torch.uint8, device="cuda")
        out = torch.full((B, H, V), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.err.zero_()
        k3.shared_decode(self.q, *self.args(), out, ws, ms, mo, shared_split, own_split, dev_err=self.err)
        torch.cuda.synchronize()
        return out

    def check(self, got, ctx=None):
        q, w, slab = self.q.double().cpu().numpy(), self.w.double().cpu().numpy(), self.slab.double().cpu().numpy()
        for b, n in enumerate(self.ctx if ctx is None else ctx):
            out, o, p, rows = wr.attend(q[b], slab, self.layer, self.table[b], n, MOST, 0, w, SCALE)
            s_abs = np.abs(q[b]) @ np.abs(rows).T * SCALE
            err = np.abs(got[b].double().cpu().numpy() - out)
            tol = wr.out_tolerance(out, o, p, rows, w, s_abs)
            assert (err <= tol).all(), (b, n, float((err / tol).max()))


@pytest.mark.parametrize("shared_split,own_split", [(0, 0), (128, 128), (256, 0), (128, 256), (-1, 0), (-1, 128)])
@pytest.mark.parametrize("size", [1, 2, 3, 4, 5, 9])
def test_one_group(gpu_lib, size, shared_split, own_split):
    c = Case([([300 + 64 + 37 * i for i in range(size)], 330)], seed=size)
    c.check(c.run(gpu_lib, shared_split, own_split))
    assert c.err.item() == 0


@pytest.mark.parametrize("shared_split,own_split", [(0, 0), (128, 128), (512, 128), (-1, 128), (-1, 0)])
def test_many_groups_of_all_kinds(gpu_lib, shared_split, own_split):
    """Sizes 1 to 6 and 0, prefixes of no whole page, of one token, of exact pages; slots without a token of their own; slots
    that share nothing; empty slots."""
    c = Case([([65, 64, 0], 64), ([700] * 6, 640), ([], 100), ([63, 1, 200, 90], 63), ([128], 128), ([129, 192, -3, 500, 128], 130),
              ([10, 0], 0), ([1300, 1281], 1280)], alone=[1, 0, 300, 64], seed=3)
    c.check(c.run(gpu_lib, shared_split, own_split))
    assert c.err.item() == 0


def test_no_groups_and_no_prefix(gpu_lib):
    c = Case([], alone=[200, 1, 0, 640], seed=4)
    c.check(c.run(gpu_lib))
    c.check(c.run(gpu_lib, 128, 128, max_shared=1000))
    d = Case([([100, 20], 40), ([64, 3], 0)], seed=5)
    d.check(d.run(gpu_lib))


def test_a_long_prefix_and_the_planned_splits(gpu_lib):
    k3 = gpu_lib
    c = Case([([4200 + 11 * i for i in range(13)], 4160), ([2200, 2100], 2050)], alone=[77], seed=6)
    split = k3.shared_split_tokens(16, 2, c.max_shared, c.max_own)
    c.check(c.run(k3, *split))
    c.check(c.run(k3))


def test_bounds_may_be_larger_and_a_prefix_beyond_its_bound_is_read_by_each(gpu_lib):
    k3 = gpu_lib
    c = Case([([500, 460], 448), ([130, 140, 64], 64)], alone=[90], seed=7)
    want = c.run(k3)
    assert torch.equal(c.run(k3, max_shared=5000, max_own=3000), want)
    got = c.run(k3, max_shared=130, max_own=400)        # two whole pages shared, the rest read by each slot
    c.check(got)
    assert c.err.item() == 0


def test_alone_is_the_window_decode_of_the_same_tables(gpu_lib):
    k3 = gpu_lib
    c = Case([([700, 650, 641], 640), ([130, 0, 128], 128)], alone=[90], seed=17)
    for split in (0, 128):
        got = c.run(k3, k3.SHARED_NONE, split)
        args = c.args()
        want = torch.empty_like(got)
        ws = torch.empty(k3.window_decode_workspace_bytes(7, 700, MOST, 0, split), dtype=torch.uint8, device="cuda")
        k3.window_decode(c.q, args[0], args[1], args[2], args[3], c.w, SCALE_BITS, want, ws, 700, MOST, 0, split)
        assert torch.equal(got, want)
    c.ctx[1], c.ctx[2] = 639, 5000                       # too few tokens, and more than max_own says
    got = c.run(k3, k3.SHARED_NONE, 128, max_own=60)
    assert c.err.item() == k3.DEV_CTX and (got[1] == 0).all() and not got[1].isnan().any()
    c.check(got, ctx=[700, 0, 700, 130, 0, 128, 60])


def test_too_short_and_too_long_slots_are_flagged(gpu_lib):
    k3 = gpu_lib
    c = Case([([500, 200, 470], 448)], alone=[300], seed=8)
    c.max_own = 300
    got = c.run(k3)
    assert c.err.item() == k3.DEV_CTX
    c.check(got, ctx=[500, 0, 470, 300])
    d = Case([([500, 460], 448)], alone=[300], seed=9)
    got = d.run(k3, max_own=40)
    assert d.err.item() == k3.DEV_CTX
    d.check(got, ctx=[488, 460, 40])


def test_unmapped_and_bad_pages(gpu_lib):
    k3 = gpu_lib
    c = Case([([300, 290, 310, 260, 257], 256)], seed=10)
    c.table[:, 2] = -1
    c.table[1, 4] = -1
    want = c.run(k3)
    c.check(want)
    assert c.err.item() == 0
    c.table[0, 2] = c.slab.shape[0]      # (the group's pages are looked up in its first slot's row)
    assert torch.equal(c.run(k3), want) and c.err.item() == k3.DEV_BAD_PAGE
    c.table[0, 2] = -1
    c.table[1:, :4] = -2 ** 31
    assert torch.equal(c.run(k3), want) and c.err.item() == 0


def test_stale_rows_do_not_matter_and_a_seen_nan_stays_with_those_that_see_it(gpu_lib):
    k3 = gpu_lib
    c = Case([([300, 290, 310], 256), ([200, 130], 128)], alone=[70], seed=11)
    want = c.run(k3)
    for b, n in enumerate(c.ctx):
        if n % PAGE:
            c.slab[int(c.table[b, n // PAGE]), c.layer, n % PAGE:] = float("nan")
    assert torch.equal(c.run(k3), want)
    c.slab[int(c.table[0, 1]), c.layer, 3, 5] = float("nan")       # a shared page of group 0
    c.slab[int(c.table[4, 2]), c.layer, 0, 5] = float("inf")       # slot 4's own page
    got = c.run(k3)
    assert got[:3].isnan().all() and got[4].isnan().all()
    assert torch.equal(got[[3, 5]], want[[3, 5]])


def test_a_slot_does_not_depend_on_its_neighbours(gpu_lib):
    k3 = gpu_lib
    ctx = [1100, 1050, 1025, 1024, 1200, 1090, 1030]
    c = Case([(ctx, 1024)], seed=12)
    whole = c.run(k3, 256, 128)
    assert torch.equal(c.run(k3, 256, 128), whole)
    for keep in ([0], [1, 2], [6, 5, 4, 3, 0], [2, 2, 1]):
        d = Case([([ctx[b] for b in keep], 1024)], seed=12)
        d.slab, d.w, d.q, d.table = c.slab, c.w, c.q[keep].contiguous(), c.table[keep]
        assert torch.equal(d.run(k3, 256, 128), whole[keep]), keep


def test_the_pool_s_shared_pages_as_a_server_runs_them(gpu_lib):
    """A prompt's pages mapped into four slots, a page un-shared before each slot's first write, a step appended, and the four
    decoded together: as each slot by itself with windowed decode over its whole context."""
    k3 = gpu_lib
    pool = k3.Pool(n_slots=5, max_ctx=1024, n_pages=40, shuffle_seed=5)
    prompt = 300
    assert pool.ensure(0, prompt) == 0
    for s in range(1, 4):
        assert pool.share_prefix(s, 0, prompt) == 0
    gen = torch.Generator(device="cuda").manual_seed(13)
    slab = torch.randn(40, 1, PAGE, ROW, generator=gen, device="cuda").bfloat16()
    src, dst = [], []
    for s in range(4):
        assert pool.ensure(s, prompt + 1) == 0
        copied = pool.cow(s, prompt)
        if copied is not None and copied is not False:
            src.append(copied[0]), dst.append(copied[1])
    i32 = dict(dtype=torch.int32, device="cuda")
    if src:
        k3.copy_pages(slab, slab, torch.tensor(src, **i32), torch.tensor(dst, **i32))
    table = torch.from_numpy(pool.table()[:4].copy()).cuda()
    assert (table[:, :prompt // PAGE] == table[0, :prompt // PAGE]).all() and len(set(table[:, prompt // PAGE].tolist())) == 4
    kv = torch.randn(4, ROW, generator=gen, device="cuda").bfloat16()
    k3.append_latent(slab, 0, table, torch.full((4,), prompt, **i32), kv[:, :LORA], kv[:, LORA:])
    q = torch.randn(4, H, 192, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(H * 256, LORA, generator=gen, device="cuda") * LORA ** -0.5).bfloat16()
    q_abs = torch.empty(4, H, ROW, dtype=torch.bfloat16, device="cuda")
    k3.absorb_q(q, w, q_abs)
    ctx, out, other = torch.full((4,), prompt + 1, **i32), *(torch.empty(4, H, V, dtype=torch.bfloat16, device="cuda") for _ in "ab")
    ws = torch.empty(k3.shared_decode_workspace_bytes(4, prompt, 64), dtype=torch.uint8, device="cuda")
    k3.shared_decode(q_abs, slab, 0, table, ctx, torch.tensor([0, 4], **i32), torch.tensor([prompt], **i32), w, SCALE_BITS, out, ws,
                     prompt, 64)
    ws2 = torch.empty(k3.window_decode_workspace_bytes(4, 1024, 1024), dtype=torch.uint8, device="cuda")
    k3.window_decode(q_abs, slab, 0, table, ctx, w, SCALE_BITS, other, ws2, 1024, 1024)
    torch.cuda.synchronize()
    c = Case([([prompt + 1] * 4, prompt)], seed=13)
    c.slab, c.table, c.q, c.w, c.layer = slab, table.cpu().numpy(), q_abs, w, 0
    c.check(out)
    c.check(other)
    pool.close()


def test_captured_and_replayed_with_new_groups_on_another_stream(gpu_lib):
    k3 = gpu_lib
    c = Case([([400, 390, 350], 320), ([200, 150], 128)], alone=[70], seed=14)
    slab, layer, table, ctx, start, shared, w, bits = c.args()
    ws = torch.full((k3.shared_decode_workspace_bytes(6, 320, 512, 128, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(6, H, V, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda: k3.shared_decode(c.q, slab, layer, table, ctx, start, shared, w, bits, out, ws, 320, 512, 128, 128)  # noqa: E731
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    for lens, starts, lens_shared in (([400, 390, 350, 200, 150, 70], [0, 3, 5], [320, 128]),
                                      ([330, 390, 321, 180, 129, 1], [0, 2, 5], [256, 0]), ([0, 0, 350, 200, 0, 64], [0, 3, 3], [64, 9])):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        start.copy_(torch.tensor(starts, dtype=torch.int32))
        shared.copy_(torch.tensor(lens_shared, dtype=torch.int32))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        c.check(out, ctx=lens)


def test_two_streams_at_once_with_workspaces_of_their_own(gpu_lib):
    k3 = gpu_lib
    cases = [Case([([900, 880, 870], 832)], seed=15), Case([([200] * 9, 128)], alone=[300], seed=16)]
    want = [c.run(k3, 128, 128) for c in cases]
    work = []
    for c in cases:
        B = len(c.ctx)
        ws = torch.empty(k3.shared_decode_workspace_bytes(B, c.max_shared, c.max_own, 128, 128), dtype=torch.uint8, device="cuda")
        out = torch.empty(B, H, V, dtype=torch.bfloat16, device="cuda")
        work.append((torch.cuda.Stream(), (c.q, *c.args(), out, ws, c.max_shared, c.max_own, 128, 128), out))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, args, _ in work:
            with torch.cuda.stream(s):
                k3.shared_decode(*args)
    torch.cuda.synchronize()
    for (_, _, out), w in zip(work, want):
        assert torch.equal(out, w)
