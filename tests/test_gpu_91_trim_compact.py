"""Trim, compaction, rotation and windowed attention on one slot, as an eviction uses them together: a trimmed slot gets
pages for its kept rows, the rows move, and the tokens that follow are turned by positions that go on from the old ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests import window_ref as ref
from tests.test_gpu_87_window import SCALE_BITS, Case

pytestmark = pytest.mark.gpu

PAGE, H, V, ROW = 64, 96, 128, 576


@pytest.mark.parametrize("refill", [True, False])
def test_evicting_from_trimmed_slots(gpu_lib, refill):
    window, sink, B = 200, 70, 2
    pool = k3mla.Pool(n_slots=B, max_ctx=1024, shuffle_seed=3)
    g = torch.Generator(device="cuda").manual_seed(60)
    slab = torch.full((pool.n_pages, 2, PAGE, ROW), float("nan"), dtype=torch.bfloat16, device="cuda")
    w = (torch.randn(H * 256, 512, generator=g, device="cuda") * 512 ** -0.5).bfloat16()
    wk = (1 + 0.1 * torch.randn(64, generator=g, device="cuda")).bfloat16()
    inv = (10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)).float()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.from_numpy(np.array(x, np.int32)).cuda()  # noqa: E731
    history = [[] for _ in range(B)]                 # (projection row, position that turned it) of every row in the cache

    def step(new, at, turned):
        """Rows of `new` tokens a slot, written from position at[b] on, turned from turned[b] on; their queries."""
        for b in range(B):
            assert pool.ensure(b, at[b] + new[b]) == 0
        R, start = sum(new), np.concatenate([[0], np.cumsum(new)])
        q = torch.randn(R, H, 192, generator=g, device="cuda").bfloat16()
        kv = torch.randn(R, ROW, generator=g, device="cuda").bfloat16()
        k3mla.norm_rope_append(q, q, slab, 1, i32(pool.table()), i32(at), i32(start), kv[:, :512], kv[:, 512:],
                               k_weight=wk, inv_freq=inv, dev_err=err, rope_pos0=i32(turned))
        for b in range(B):
            history[b] += [(kv[start[b] + j].float().cpu().numpy(), turned[b] + j) for j in range(new[b])]
        q_abs = torch.empty(R, H, ROW, dtype=torch.bfloat16, device="cuda")
        k3mla.absorb_q(q, w, q_abs)
        return q_abs

    lens = [700, 300]
    step(lens, [0, 0], [0, 0])
    freed = [pool.trim(b, lens[b], window, sink) for b in range(B)]
    assert freed == [5, 0]                           # slot 0: pages 2 .. 6 lie between the sinks and token 501
    keep = [np.r_[0:sink, n - window + 1:n] for n in lens]
    kept = [len(k) for k in keep]
    if refill:
        assert [pool.refill(b, kept[b]) for b in range(B)] == [3, 0]
    start = np.concatenate([[0], np.cumsum(kept)])
    k3mla.compact_rows(slab, i32(pool.table()), i32(np.concatenate(keep)), i32(start), dev_err=err)
    torch.cuda.synchronize()
    if not refill:                                   # said, where there is a word to say it in
        assert err.item() == k3mla.DEV_UNMAPPED
        pool.close()
        return
    assert err.item() == 0
    for b in range(B):
        assert pool.truncate(b, kept[b]) == 0
        history[b] = [history[b][int(t)] for t in keep[b]]
    assert pool.stats()[1] == sum(-(-k // PAGE) for k in kept)

    # three decode steps, then a chunk, over all that is left
    n, ws = list(kept), torch.empty(k3mla.window_decode_workspace_bytes(B, 1024, 1024), dtype=torch.uint8, device="cuda")
    for i in range(3):
        q_abs = step([1, 1], n, [lens[b] + i for b in range(B)])
        n = [x + 1 for x in n]
        out = torch.empty(B, H, V, dtype=torch.bfloat16, device="cuda")
        k3mla.window_decode(q_abs, slab, 1, i32(pool.table()), i32(n), w, SCALE_BITS, out, ws, 1024, 1024, dev_err=err)
    new = [9, 70]
    chunk_q = step(new, n, [lens[b] + 3 for b in range(B)])
    chunk_out = torch.empty(sum(new), H, V, dtype=torch.bfloat16, device="cuda")
    cws = torch.empty(k3mla.window_chunk_decode_workspace_bytes(B, sum(new), 1024), dtype=torch.uint8, device="cuda")
    k3mla.window_chunk_decode(chunk_q, slab, 1, i32(pool.table()), i32(n), i32([0, 9, 79]), w, SCALE_BITS, chunk_out, cws,
                              1024, 1024, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == 0

    c = Case.__new__(Case)
    c.w, c.slab, c.layer, c.table = w, slab, 1, pool.table()
    c.q = q_abs
    c.check(out, [0, 1], n, 1024, 0)
    c.q = chunk_q
    c.check(chunk_out, [0] * 9 + [1] * 70, [n[0] + 1 + j for j in range(9)] + [n[1] + 1 + j for j in range(70)], 1024, 0,
            rows=range(0, 79, 6))
    # the cache holds the kept rows and the new ones, each turned by its own position (bounds: test_gpu_85_norm_rope)
    got, wk, inv = slab[:, 1].float().cpu().numpy(), wk.float().cpu().numpy(), inv.cpu().numpy()
    for b in range(B):
        assert len(history[b]) == n[b] + new[b]
        for t, (kv, turn) in enumerate(history[b]):
            y, mag = ref.key_row(kv[:512], kv[512:], turn, None, wk, 1e-6, inv, False)
            x = got[pool.table()[b, t // PAGE], t % PAGE]
            assert np.all(np.abs(x - y) <= 2.0 ** -8 * np.abs(y) * 1.01 + 2.0 ** -18 * mag * 1.01), (b, t, turn)
    pool.close()
