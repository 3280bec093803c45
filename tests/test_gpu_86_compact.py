"""k3mla_compact_rows (bit for bit: it moves rows) with the pool's trim and truncate."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla, synth

pytestmark = pytest.mark.gpu

PAGE = 64


def make(seed, lens, L, extra=1):
    rng = np.random.default_rng(seed)
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    n_pages, cols = sum(pages) + extra, max(1, max(pages))
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), cols), -1, np.int32)
    k = 0
    for b, m in enumerate(pages):
        table[b, :m] = ids[k:k + m]
        k += m
    g = torch.Generator(device="cuda").manual_seed(seed)
    slab = torch.randn(n_pages, L, PAGE, 576, generator=g, device="cuda").bfloat16()
    return rng, table, slab


def expected(bits, table, keep, start):
    L = bits.shape[1]
    out = bits.copy()
    flag = 0
    for b in range(table.shape[0]):
        for layer in range(L):
            ks = keep[layer if keep.shape[0] > 1 else 0][start[b]:start[b + 1]]
            for i, t in enumerate(ks):
                if t == i:
                    continue
                dp = table[b, i // PAGE] if i // PAGE < table.shape[1] else -1
                ok_src = 0 <= t < table.shape[1] * PAGE
                sp = table[b, t // PAGE] if ok_src else -1
                if not ok_src:
                    flag |= k3mla.DEV_CTX
                if sp >= bits.shape[0] or sp < -1:
                    flag |= k3mla.DEV_BAD_PAGE
                    sp = -1
                if not 0 <= dp < bits.shape[0]:
                    flag |= k3mla.DEV_UNMAPPED
                    continue
                out[dp, layer, i % PAGE] = bits[sp, layer, t % PAGE] if sp >= 0 else 0
    return out, flag


def go(slab, table, keep, start):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k3mla.compact_rows(slab, torch.from_numpy(table).cuda(), torch.from_numpy(keep).cuda(),
                       torch.from_numpy(start).cuda(), dev_err=err)
    torch.cuda.synchronize()
    return err.item()


@pytest.mark.parametrize("per_layer", [False, True])
@pytest.mark.parametrize("lens,share,L", [([1], 1.0, 1), ([200, 1, 64, 65, 0], 0.5, 3), ([1500, 700], 0.7, 2), ([900], 0.05, 4),
                                          ([128, 129, 300], 1.0, 2), ([70, 0, 200, 33] * 10, 0.6, 4)])
def test_kept_rows_move_to_the_front(gpu_lib, lens, share, L, per_layer):
    rng, table, slab = make(sum(lens) + L, lens, L)
    kept = [min(n, max(n > 0, int(n * share))) for n in lens]
    start = np.concatenate([[0], np.cumsum(kept)]).astype(np.int32)
    sets = L if per_layer else 1
    keep = np.stack([np.concatenate([np.sort(rng.permutation(n)[:k]) for n, k in zip(lens, kept)]) for _ in range(sets)])
    keep = np.ascontiguousarray(keep.astype(np.int32))
    want, flag = expected(synth.bf16_bits(slab), table, keep, start)
    assert flag == 0 and go(slab, table, keep, start) == 0
    assert np.array_equal(synth.bf16_bits(slab), want)


def test_shift_by_one_across_every_step(gpu_lib):
    # the tightest overlap: every row moves down by one, over many steps and page ends
    n = 1000
    _, table, slab = make(3, [n], 2)
    keep = np.arange(1, n, dtype=np.int32)[None]
    start = np.array([0, n - 1], np.int32)
    want, _ = expected(synth.bf16_bits(slab), table, keep, start)
    assert go(slab, table, keep, start) == 0
    assert np.array_equal(synth.bf16_bits(slab), want)


def test_holes_and_bad_entries(gpu_lib):
    _, table, slab = make(4, [400, 400], 2)
    table[0, 4] = -1                       # a trimmed page reads as zeros
    table[0, 5] = slab.shape[0]            # outside the slab
    table[1, 0] = -1                       # nowhere to write rows 0..63
    keep = np.concatenate([np.arange(2, 400, 3), [10 ** 7], np.arange(1, 400, 2)]).astype(np.int32)[None]
    a = len(np.arange(2, 400, 3)) + 1
    start = np.array([0, a, keep.shape[1]], np.int32)
    want, flag = expected(synth.bf16_bits(slab), table, keep, start)
    assert flag == k3mla.DEV_CTX | k3mla.DEV_BAD_PAGE | k3mla.DEV_UNMAPPED
    assert go(slab, table, keep, start) == flag
    assert np.array_equal(synth.bf16_bits(slab), want)


def test_rows_past_2_31_elements(gpu_lib):
    n_pages, L = 1024, 64                  # 2.4e9 elements
    slab = torch.zeros(n_pages, L, PAGE, 576, dtype=torch.bfloat16, device="cuda")
    assert slab.numel() > 2 ** 31
    slab[n_pages - 1, L - 1, 40] = 3.0
    table = np.array([[n_pages - 1]], np.int32)
    assert go(slab, table, np.array([[40]], np.int32), np.array([0, 1], np.int32)) == 0
    assert torch.all(slab[n_pages - 1, L - 1, 0] == 3.0) and torch.all(slab[n_pages - 1, :L - 1, 0] == 0)


def test_graph_replay_moves_the_rows_of_the_replay(gpu_lib):
    _, table, slab = make(6, [300], 3)
    fresh = slab.clone()
    keep = np.arange(50, 300, 2, dtype=np.int32)[None]
    start = np.array([0, keep.shape[1]], np.int32)
    want, _ = expected(synth.bf16_bits(slab), table, keep, start)
    args = [torch.from_numpy(a).cuda() for a in (table, keep, start)]
    graph = torch.cuda.CUDAGraph()
    k3mla.compact_rows(slab, *args)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        k3mla.compact_rows(slab, *args)
    slab.copy_(fresh)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(synth.bf16_bits(slab), want)


def test_evict_then_truncate_then_append(gpu_lib):
    # a slot's life: 300 tokens, keep 5 first and 60 last, give the pages back, append the next token
    pool = k3mla.Pool(n_slots=1, max_ctx=512, shuffle_seed=9)
    assert pool.ensure(0, 300) == 0
    slab = torch.randn(pool.n_pages, 2, PAGE, 576, device="cuda").bfloat16()
    keep = np.concatenate([np.arange(5), np.arange(240, 300)]).astype(np.int32)[None]
    start = np.array([0, 65], np.int32)
    want, _ = expected(synth.bf16_bits(slab), pool.table(), keep, start)
    assert go(slab, pool.table(), keep, start) == 0
    assert np.array_equal(synth.bf16_bits(slab), want)
    assert pool.truncate(0, 65) == 0 and pool.stats()[1] == 2
    assert pool.ensure(0, 66) == 0 and pool.stats()[1] == 2
    row = torch.randn(1, 576, device="cuda").bfloat16()
    table = torch.from_numpy(pool.table()).cuda()
    k3mla.append_latent(slab, 1, table, torch.tensor([65], dtype=torch.int32, device="cuda"), row[:, :512], row[:, 512:])
    torch.cuda.synchronize()
    want[pool.table()[0, 1], 1, 1] = synth.bf16_bits(row)[0]
    assert np.array_equal(synth.bf16_bits(slab), want)
    pool.close()
