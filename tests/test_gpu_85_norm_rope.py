"""k3mla_norm_rope_append against the definition in 64 bits: norms per head, rotation by position in both
pair orders, rows into mapped pages.

Bound: the f32 work before the last rounding is within 2^-19 relative (a sum of at most 512 squares in a
tree of at most 29 additions, halved by the square root, rsqrtf within 2 ulp, three products), the
rotation within 2^-20 of |a| + |b| (2^-25 turns of angle, sincospif within 2^-22, two products); 2^-18
covers their sum.  The rounding to bf16 adds 2^-8 of the value."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_latent_attention_k3mla_gb300 import k3mla, synth
from tests import window_ref as ref

pytestmark = pytest.mark.gpu

PAGE = 64


def f32(t):
    return t.float().cpu().numpy()


def make(seed, lens, rows, L=2, pool=None):
    """Slots of lens[b] tokens in shuffled pages; rows[b] packed token rows end at position lens[b] - 1."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    n_pages, cols = max(1, sum(pages)) + 2, max(1, max(pages))
    ids = torch.randperm(n_pages, generator=g, device="cuda")[: sum(pages)].cpu().numpy()
    table = np.full((len(lens), cols), -1, np.int32)
    k = 0
    for b, m in enumerate(pages):
        table[b, :m] = ids[k:k + m]
        k += m
    slab = torch.randn(n_pages, L, PAGE, 576, generator=g, device="cuda").bfloat16()
    R = sum(rows)
    q = (torch.randn(R, 96, 192, generator=g, device="cuda") * 3).bfloat16()
    kv = torch.randn(R, 576, generator=g, device="cuda").bfloat16()
    w = [(1 + 0.3 * torch.randn(n, generator=g, device="cuda")).bfloat16() for n in (192, 512, 64)]
    inv = (10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)).float()
    pos0 = np.array([n - m for n, m in zip(lens, rows)], np.int32)
    start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return dict(g=g, slab=slab, table=table, q=q, kv=kv, w=w, inv=inv, pos0=pos0, start=start, R=R)


def check(d, q_in, q_out, slab_before, layer, weights, inv, interleaved, row_start, eps=1e-6):
    qw, cw, kw = [None if w is None else f32(w) for w in weights]
    inv = None if inv is None else f32(inv)
    q_in, got = f32(q_in), f32(q_out)
    kv = f32(d["kv"])
    want = f32(slab_before)
    scale = np.zeros(want.shape, np.float32)
    for r, (b, p) in enumerate(ref.rows_of(d["pos0"], row_start, d["R"])):
        if b < 0:
            continue
        y, mag = ref.query_row(q_in[r], p, qw, eps, inv, interleaved)
        assert np.all(np.abs(got[r] - y) <= 2.0 ** -8 * np.abs(y) * 1.01 + 2.0 ** -18 * mag * 1.01), (r, b, p)
        lp = p // PAGE
        page = d["table"][b, lp] if lp < d["table"].shape[1] else -1
        if 0 <= page < want.shape[0]:
            row, mag = ref.key_row(kv[r, :512], kv[r, 512:], p, cw, kw, eps, inv, interleaved)
            want[page, layer, p % PAGE] = row
            scale[page, layer, p % PAGE] = 2.0 ** -8 * np.abs(row) * 1.01 + 2.0 ** -18 * mag * 1.01
    assert np.all(np.abs(f32(d["slab"]) - want) <= scale)      # rows that no token names: bit for bit as before


def call(d, q, q_out, layer, weights, inv, interleaved, row_start, err=None, table=None, pos0=None):
    k3mla.norm_rope_append(
        q, q_out, d["slab"], layer, torch.from_numpy(d["table"] if table is None else table).cuda(),
        torch.from_numpy(d["pos0"] if pos0 is None else pos0).cuda(),
        None if row_start is None else torch.from_numpy(row_start).cuda(), d["kv"][:, :512], d["kv"][:, 512:],
        q_weight=weights[0], c_weight=weights[1], k_weight=weights[2], inv_freq=inv, interleaved=interleaved, dev_err=err)
    torch.cuda.synchronize()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lens,rows", [([1], [1]), ([130, 64, 1, 65], [3, 64, 1, 0]), ([700], [700]),
                                       ([40] * 37, [1] * 37), ([9] * 1100, [1] * 1100)])
def test_norms_rotation_and_rows(gpu_lib, lens, rows, interleaved):
    d = make(len(lens) * 7 + interleaved, lens, rows)
    before, q_out = d["slab"].clone(), torch.full_like(d["q"], float("nan"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(d, d["q"], q_out, 1, d["w"], d["inv"], interleaved, d["start"], err)
    check(d, d["q"], q_out, before, 1, d["w"], d["inv"], interleaved, d["start"])
    assert err.item() == 0


@pytest.mark.parametrize("have", [(False, False, False), (True, False, False), (False, True, True), (False, False, True)])
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_parts_left_out(gpu_lib, have, rope, in_place):
    d = make(5, [70, 3], [2, 3])
    weights = [w if h else None for w, h in zip(d["w"], have)]
    inv = d["inv"] if rope else None
    before, q_in = d["slab"].clone(), d["q"].clone()
    q_out = d["q"] if in_place else torch.full_like(d["q"], float("nan"))
    call(d, d["q"], q_out, 0, weights, inv, False, d["start"])
    check(d, q_in, q_out, before, 0, weights, inv, False, d["start"])
    if not have[0] and not rope:
        assert torch.equal(q_out, q_in)


def test_far_positions_keep_their_angles(gpu_lib):
    # positions near 2^29 on a one-page table: the cache write is skipped and flagged, the queries are not
    d = make(11, [1, 1, 1], [1, 1, 1])
    pos = np.array([2 ** 29 - 1, 1_000_003, 5], np.int32)
    q_out = torch.empty_like(d["q"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = d["slab"].clone()
    call(d, d["q"], q_out, 0, d["w"], d["inv"], False, d["start"], err, pos0=pos)
    d["pos0"] = pos
    check(d, d["q"], q_out, before, 0, d["w"], d["inv"], False, d["start"])
    assert err.item() == k3mla.DEV_UNMAPPED


def test_decode_form_and_rows_left_alone(gpu_lib):
    d = make(13, [5, 64, 200], [1, 1, 1])
    d["pos0"] = np.array([4, -1, 199], np.int32)               # slot 1 is a padding row
    before, q_out = d["slab"].clone(), torch.full_like(d["q"], 7.0)
    call(d, d["q"], q_out, 1, d["w"], d["inv"], True, None)
    check(d, d["q"], q_out, before, 1, d["w"], d["inv"], True, None)
    assert torch.all(q_out[1] == 7.0)
    # rows before the first and behind the last slot, an empty slot in between, and one that starts before 0
    d = make(14, [5, 64, 200], [3, 0, 6])
    d["start"] = np.array([2, 5, 5, 7], np.int32)
    d["pos0"] = np.array([-1, 0, 190], np.int32)
    before, q_out = d["slab"].clone(), torch.full_like(d["q"], 7.0)
    call(d, d["q"], q_out, 0, d["w"], d["inv"], False, d["start"])
    check(d, d["q"], q_out, before, 0, d["w"], d["inv"], False, d["start"])
    assert torch.all(q_out[[0, 1, 2, 7, 8]] == 7.0)


def test_unmapped_and_bad_pages_are_skipped_and_flagged(gpu_lib):
    d = make(15, [70, 70], [70, 70])
    table = d["table"].copy()
    table[0, 1], table[1, 0] = -1, 10 ** 6
    d["table"] = table
    before, q_out = d["slab"].clone(), torch.empty_like(d["q"])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call(d, d["q"], q_out, 1, d["w"], d["inv"], False, d["start"], err)
    check(d, d["q"], q_out, before, 1, d["w"], d["inv"], False, d["start"])
    assert err.item() == k3mla.DEV_UNMAPPED


def test_zero_rows_extreme_values_and_strides(gpu_lib):
    d = make(16, [64], [5])
    d["q"][0] = 0.0
    d["q"][1] = 2.0 ** 50
    d["kv"][2] = 0.0
    wide = torch.full((5, 640), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:584] = d["kv"]
    d["kv"] = wide[:, 8:584]                                    # row pitch 640, 16 bytes in
    before, q_out = d["slab"].clone(), torch.empty_like(d["q"])
    call(d, d["q"], q_out, 0, d["w"], d["inv"], False, d["start"])
    check(d, d["q"], q_out, before, 0, d["w"], d["inv"], False, d["start"])
    # a NaN stays in its own head and its own row
    d["q"][3, 17, 5] = float("nan")
    call(d, d["q"], q_out, 0, d["w"], d["inv"], False, d["start"])
    bad = torch.isnan(q_out.float()).flatten(2).any(-1)
    assert bad[3, 17] and bad.sum() == 1


def test_graph_replay_is_the_eager_call(gpu_lib):
    d = make(17, [300] * 4, [20] * 4)
    args = (torch.from_numpy(d["table"]).cuda(), torch.from_numpy(d["pos0"]).cuda(), torch.from_numpy(d["start"]).cuda())
    q_out, slab2, q2 = torch.empty_like(d["q"]), d["slab"].clone(), torch.empty_like(d["q"])

    def go(q_out, slab):
        k3mla.norm_rope_append(d["q"], q_out, slab, 1, *args, d["kv"][:, :512], d["kv"][:, 512:], q_weight=d["w"][0],
                               c_weight=d["w"][1], k_weight=d["w"][2], inv_freq=d["inv"])

    go(q_out, d["slab"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        go(q2, slab2)
    torch.cuda.current_stream().wait_stream(s)
    q2.fill_(0)
    with torch.cuda.graph(graph):
        go(q2, slab2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q2, q_out) and torch.equal(slab2, d["slab"])
