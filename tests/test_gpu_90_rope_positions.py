"""Norms, rotation and append with the angles' positions apart from the cache rows' (a slot whose rows were compacted),
against the definition in 64 bits; the bounds are those of test_gpu_85_norm_rope."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla
from tests import window_ref as ref
from tests.test_gpu_85_norm_rope import PAGE, f32, make

pytestmark = pytest.mark.gpu


def run(d, q_out, slab, row_start, rope_pos0, interleaved=False, weights=None, inv=True):
    w = d["w"] if weights is None else weights
    k3mla.norm_rope_append(
        d["q"], q_out, slab, 1, torch.from_numpy(d["table"]).cuda(), torch.from_numpy(d["pos0"]).cuda(),
        None if row_start is None else torch.from_numpy(row_start).cuda(), d["kv"][:, :512], d["kv"][:, 512:], q_weight=w[0],
        c_weight=w[1], k_weight=w[2], inv_freq=d["inv"] if inv else None, interleaved=interleaved,
        rope_pos0=None if rope_pos0 is None else torch.from_numpy(rope_pos0).cuda())
    torch.cuda.synchronize()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,rows,packed", [([70, 5, 300], [3, 5, 130], True), ([70, 5, 300], [1, 1, 1], False)])
def test_rows_are_turned_by_their_own_positions(gpu_lib, lens, rows, packed, interleaved):
    d = make(21 + interleaved, lens, rows)
    start = d["start"] if packed else None
    rope = np.array([100_003, 4, -7], np.int32)        # far behind the cache row, the row itself, before the first
    before, q_out = f32(d["slab"]), torch.full_like(d["q"], float("nan"))
    run(d, q_out, d["slab"], start, rope, interleaved)
    qw, cw, kw = [f32(w) for w in d["w"]]
    q_in, got, kv, inv = f32(d["q"]), f32(q_out), f32(d["kv"]), f32(d["inv"])
    want, bound = before.astype(np.float64), np.zeros(before.shape)
    for r, (b, p) in enumerate(ref.rows_of(d["pos0"], start, d["R"])):
        turn = int(rope[b]) + p - int(d["pos0"][b])
        y, mag = ref.query_row(q_in[r], turn, qw, 1e-6, inv, interleaved)
        assert np.all(np.abs(got[r] - y) <= 2.0 ** -8 * np.abs(y) * 1.01 + 2.0 ** -18 * mag * 1.01), (r, b, p)
        y, mag = ref.key_row(kv[r, :512], kv[r, 512:], turn, cw, kw, 1e-6, inv, interleaved)
        at = (d["table"][b, p // PAGE], 1, p % PAGE)
        want[at], bound[at] = y, 2.0 ** -8 * np.abs(y) * 1.01 + 2.0 ** -18 * mag * 1.01
    assert np.all(np.abs(f32(d["slab"]) - want) <= bound)


def test_the_same_positions_give_the_same_bits(gpu_lib):
    d = make(23, [70, 0, 300], [3, 0, 130])
    slabs, outs = [d["slab"].clone() for _ in range(2)], [torch.full_like(d["q"], 7.0) for _ in range(2)]
    run(d, outs[0], slabs[0], d["start"], None)
    run(d, outs[1], slabs[1], d["start"], d["pos0"])
    assert torch.equal(outs[0], outs[1]) and torch.equal(slabs[0], slabs[1])
    # without a rotation they are not read
    for i, rope in enumerate((None, d["pos0"] + 5)):
        slabs[i].copy_(d["slab"])
        run(d, outs[i], slabs[i], d["start"], rope, inv=False)
    assert torch.equal(outs[0], outs[1]) and torch.equal(slabs[0], slabs[1])


def test_the_latent_norm_alone_leaves_the_queries(gpu_lib):
    # what a layer without rotation needs: queries in place, untouched (NaN payloads too), the latent normed, the key copied
    d = make(24, [70, 5, 300], [3, 5, 130])
    d["q"][2, 3, 4] = float("nan")
    before, q_in = f32(d["slab"]), d["q"].clone()
    run(d, d["q"], d["slab"], d["start"], None, weights=(None, d["w"][1], None), inv=False)
    assert torch.equal(d["q"].view(torch.int16), q_in.view(torch.int16))
    cw, kv = f32(d["w"][1]), f32(d["kv"])
    want, bound = before.astype(np.float64), np.zeros(before.shape)
    for r, (b, p) in enumerate(ref.rows_of(d["pos0"], d["start"], d["R"])):
        y, mag = ref.key_row(kv[r, :512], kv[r, 512:], p, cw, None, 1e-6, None, False)
        at = (d["table"][b, p // PAGE], 1, p % PAGE)
        want[at], bound[at] = y, 2.0 ** -8 * np.abs(y) * 1.01 + 2.0 ** -18 * mag * 1.01
        bound[at][512:] = 0.0
    assert np.all(np.abs(f32(d["slab"]) - want) <= bound)
