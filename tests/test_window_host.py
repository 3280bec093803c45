"""Host-side tests of the windowed latent-cache operators that need no GPU: the pool's trim and truncate, and
argument errors that come back before anything is launched."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from paged_latent_attention_k3mla_gb300 import k3mla


def test_trim_unmaps_what_no_later_token_sees():
    pool = k3mla.Pool(n_slots=2, max_ctx=1024, n_pages=16)
    assert pool.ensure(0, 600) == 0                              # ten pages
    before = pool.table()[0].copy()
    assert pool.trim(0, 600, 1024, 0) == 0                       # the window reaches the first token
    # the next token (position 600) sees 600 - 200 + 1 = 401 and later; with 65 sinks pages 0, 1 stay
    assert pool.trim(0, 600, 200, 65) == 4                       # pages 2..5 hold tokens 128..383
    t = pool.table()[0]
    assert np.all(t[2:6] == -1) and np.array_equal(t[[0, 1, 6, 7, 8, 9]], before[[0, 1, 6, 7, 8, 9]])
    assert pool.stats() == (16, 6)
    assert pool.trim(0, 600, 200, 65) == 0                       # nothing left to give
    assert pool.trim(0, 600, 153, 65) == 1                       # first seen: 448, page 6 ends there
    assert pool.trim(0, 600, 1, 0) == 4                          # pages 0, 1, 7, 8; the next token's page stays
    assert pool.table()[0, 9] == before[9] and pool.stats() == (16, 1)
    assert pool.ensure(0, 641) == 0 and pool.table()[0, 10] >= 0  # growth goes on behind the holes
    assert pool.cow(0, 100) == -4 and pool.cow(0, 640) is None
    assert pool.release(0) == 0 and pool.stats() == (16, 0)
    assert all(pool.refs(p) == 0 for p in range(16))
    pool.close()


def test_every_page_trimmed_is_behind_every_later_window():
    for n in (1, 63, 64, 65, 127, 128, 129, 500, 511, 512):
        for w in (1, 2, 63, 64, 65, 66, 128, 129, 600):
            for s in (0, 1, 64, 65, 130, 10 ** 9):
                pool = k3mla.Pool(n_slots=1, max_ctx=512)
                pool.ensure(0, n)
                full = pool.table()[0].copy()
                given = pool.trim(0, n, w, s)
                t = pool.table()[0]
                seen = {p // 64 for p in range(n) if p < s or p > n - w}     # by the next token, at position n
                for lp in range((n + 63) // 64):
                    assert (t[lp] == full[lp]) == (lp in seen or (n % 64 and lp == n // 64)), (n, w, s, lp)
                assert given == int((t != full).sum())
                pool.close()


def test_trim_of_shared_pages_and_sharing_of_holes():
    pool = k3mla.Pool(n_slots=3, max_ctx=512, n_pages=12)
    assert pool.ensure(0, 320) == 0 and pool.share_prefix(1, 0, 320) == 0
    shared = pool.table()[0, :5].copy()
    assert pool.trim(0, 320, 64, 0) == 4                         # slot 1 still holds them: first seen token 257
    assert pool.stats() == (12, 5) and all(pool.refs(int(p)) == 1 for p in shared[:4])
    assert pool.share_prefix(2, 0, 320) == 0                     # the holes come along
    assert np.all(pool.table()[2, :4] == -1) and pool.table()[2, 4] == shared[4] and pool.refs(int(shared[4])) == 3
    for s in (0, 1, 2):
        assert pool.release(s) == 0
    assert pool.stats() == (12, 0)
    assert pool.ensure(0, 512) == 0 and len(set(pool.table()[0].tolist())) == 8   # no page twice in the free list
    pool.close()


def test_truncate_gives_back_the_pages_behind():
    pool = k3mla.Pool(n_slots=2, max_ctx=512)
    assert pool.ensure(0, 512) == 0
    before = pool.table()[0].copy()
    assert pool.truncate(0, 512) == 0 and pool.stats()[1] == 8
    assert pool.truncate(0, 65) == 0 and pool.stats()[1] == 2
    assert np.array_equal(pool.table()[0, :2], before[:2]) and np.all(pool.table()[0, 2:] == -1)
    assert pool.truncate(0, 2 ** 31 - 1) == 0 and pool.stats()[1] == 2
    assert pool.ensure(0, 512) == 0 and pool.stats()[1] == 8
    assert pool.truncate(0, 0) == 0 and pool.stats()[1] == 0
    pool.close()


def test_pool_refusals():
    pool = k3mla.Pool(n_slots=1, max_ctx=128)
    assert pool.trim(1, 0, 1, 0) == -3 and pool.trim(0, 129, 1, 0) == -4
    assert pool.trim(0, -1, 1, 0) == -1 and pool.trim(0, 1, 0, 0) == -1 and pool.trim(0, 1, 1, -1) == -1
    assert pool.truncate(1, 0) == -3 and pool.truncate(0, -1) == -1
    lib = k3mla.load()
    assert lib.k3mla_pool_trim(None, 0, 0, 1, 0) == -1 and lib.k3mla_pool_truncate(None, 0, 0) == -1
    pool.close()


P = ctypes.c_void_p(256)          # never dereferenced: every call below is refused on the host
ODD = ctypes.c_void_p(264)        # 8-byte aligned only


def norm_rope(lib, **change):
    a = dict(q=P, q_out=P, qw=None, slab=P, n_pages=4, n_layers=2, layer=1, table=P, cols=2, pos0=P, start=P, c=P, cs=576,
             cw=None, k=P, ks=576, kw=None, eps=1e-6, inv=None, inter=0, B=2, R=3, err=None, stream=None)
    a.update(change)
    return lib.k3mla_norm_rope_append(*a.values())


@pytest.mark.parametrize("change", [
    dict(layer=2), dict(layer=-1), dict(n_pages=0), dict(cols=0), dict(cs=511), dict(cs=580), dict(ks=63), dict(ks=68),
    dict(eps=-1.0), dict(eps=float("nan")), dict(B=-1), dict(R=-1), dict(start=None), dict(q=None), dict(q_out=None),
    dict(slab=None), dict(table=None), dict(pos0=None), dict(c=None), dict(k=None), dict(q=ODD), dict(q_out=ODD),
    dict(slab=ODD), dict(c=ODD), dict(k=ODD), dict(qw=ODD), dict(cw=ODD), dict(kw=ODD), dict(inv=ctypes.c_void_p(257)),
    dict(R=2 ** 31 - 1), dict(q=ctypes.c_void_p(512)), dict(q_out=ctypes.c_void_p(256 + 3 * 96 * 192 * 2 - 16))])
def test_norm_rope_refusals(change):
    lib = k3mla.load()
    assert norm_rope(lib, **change) == -1
    assert b"k3mla_norm_rope_append" in lib.k3mla_last_error()


def test_norm_rope_without_rows_does_nothing():
    lib = k3mla.load()
    assert norm_rope(lib, R=0) == 0 and norm_rope(lib, B=0, R=0, start=None) == 0


def compact(lib, **change):
    a = dict(slab=P, n_pages=4, n_layers=2, table=P, cols=2, keep=P, stride=0, n=5, start=P, B=2, err=None, stream=None)
    a.update(change)
    return lib.k3mla_compact_rows(*a.values())


@pytest.mark.parametrize("change", [dict(n_pages=0), dict(n_layers=0), dict(cols=0), dict(n=-1), dict(n=2 ** 30), dict(B=-1), dict(stride=4),
                                    dict(stride=-1), dict(slab=None), dict(slab=ODD), dict(table=None), dict(keep=None),
                                    dict(start=None)])
def test_compact_refusals(change):
    lib = k3mla.load()
    assert compact(lib, **change) == -1
    assert b"k3mla_compact_rows" in lib.k3mla_last_error()


def test_compact_without_rows_does_nothing():
    lib = k3mla.load()
    assert compact(lib, n=0) == 0 and compact(lib, B=0) == 0


def decode(lib, **change):
    a = dict(q=P, slab=P, n_pages=4, n_layers=2, layer=1, table=P, cols=2, ctx=P, w=P, scale=0x3D94, out=P, ws=P,
             ws_bytes=1 << 40, B=2, max_ctx=128, window=100, sink=4, split=0, err=None, stream=None)
    a.update(change)
    return lib.k3mla_window_decode(*a.values())


def chunk(lib, **change):
    a = dict(q=P, slab=P, n_pages=4, n_layers=2, layer=1, table=P, cols=2, pos0=P, start=P, B=2, R=3, w=P, scale=0x3D94,
             out=P, ws=P, ws_bytes=1 << 40, max_ctx=128, window=100, sink=4, err=None, stream=None)
    a.update(change)
    return lib.k3mla_window_chunk_decode(*a.values())


COMMON = [dict(layer=2), dict(layer=-1), dict(n_pages=0), dict(n_layers=0), dict(cols=0), dict(max_ctx=0), dict(window=0),
          dict(window=-1), dict(sink=-1), dict(scale=0), dict(scale=0x8000), dict(scale=0xBD94), dict(scale=0x7F80),
          dict(scale=0x7FC0), dict(B=-1), dict(n_pages=1 << 24, n_layers=4), dict(q=None), dict(q=ODD), dict(slab=None),
          dict(slab=ODD), dict(table=None), dict(w=None), dict(w=ODD), dict(out=None), dict(out=ODD), dict(ws=None), dict(ws=ODD)]


@pytest.mark.parametrize("change", COMMON + [dict(ctx=None), dict(split=-128), dict(split=100), dict(B=70000)])
def test_window_decode_refusals(change):
    lib = k3mla.load()
    assert decode(lib, **change) == -1
    assert b"k3mla_window_decode" in lib.k3mla_last_error()


@pytest.mark.parametrize("change", COMMON + [dict(pos0=None), dict(start=None), dict(R=-1), dict(B=0)])
def test_window_chunk_refusals(change):
    lib = k3mla.load()
    assert chunk(lib, **change) == -1
    assert b"k3mla_window_chunk_decode" in lib.k3mla_last_error()


def test_window_workspaces():
    lib = k3mla.load()
    assert decode(lib, ws_bytes=k3mla.window_decode_workspace_bytes(2, 128, 100, 4) - 1) == -6
    assert chunk(lib, ws_bytes=k3mla.window_chunk_decode_workspace_bytes(2, 3, 128) - 1) == -6
    assert decode(lib, B=0) == 0 and chunk(lib, R=0) == 0 and chunk(lib, R=0, B=0) == 0
    r256 = lambda x: (x + 255) // 256 * 256
    for B, max_ctx, w, s, split in ((1, 128, 100, 4, 0), (64, 4096, 1024, 64, 0), (3, 5000, 1000, 100, 128), (2, 10 ** 6, 9000, 0, 0)):
        # a window covers at most (w + 62) / 64 + 1 pages, the sinks (s + 63) / 64, the context all of its own
        pages = min(-(-max_ctx // 64), -(-min(s, max_ctx) // 64) + (min(w, max_ctx) + 62) // 64 + 1)
        ns = -(-pages * 64 // (split or 4096))
        o_lat = r256(96 * B * 512 * 2) + r256(96 * B * 4)         # f16 rows and a scale each
        rec = B * ns * 96                                       # f16 rows, a scale each, two f32 each
        partial = 0 if ns == 1 else r256(rec * 512 * 2) + r256(rec * 4) + r256(rec * 8)
        assert k3mla.window_decode_workspace_bytes(B, max_ctx, w, s, split) == o_lat + partial
    assert k3mla.window_chunk_decode_workspace_bytes(2, 37, 1000) == r256(96 * 37 * 512 * 2) + r256(96 * 37 * 4)
    for bad in ((0, 1, 1, 0, 0), (1, 0, 1, 0, 0), (1, 1, 0, 0, 0), (1, 1, 1, -1, 0), (1, 1, 1, 0, 64)):
        assert k3mla.window_decode_workspace_bytes(*bad) == 0


def test_window_split_plan():
    for B, max_ctx, w, s in ((1, 32768, 4096, 4), (16, 4096, 1000, 4), (64, 4096, 1024, 64), (500, 4096, 1024, 0), (1, 1, 1, 0),
                             (3, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)):
        split = k3mla.window_split_tokens(B, max_ctx, w, s)
        assert split >= 128 and split % 128 == 0
    assert k3mla.window_split_tokens(500, 4096, 1024, 0) >= 1024      # more slots than SM pairs: a split a slot
    assert k3mla.window_split_tokens(1, 32768, 4096, 4) < k3mla.window_split_tokens(16, 32768, 4096, 4)
    assert k3mla.window_split_tokens(0, 1, 1, 0) == 128


def test_arguments_past_32_bits_are_refused():
    for call in (lambda: k3mla.window_decode_workspace_bytes(1, 2 ** 32 + 64, 1), lambda: k3mla.window_split_tokens(1, 64, 2 ** 40),
                 lambda: k3mla.window_chunk_decode_workspace_bytes(1, 2 ** 31, 64)):
        with pytest.raises(k3mla.K3mlaError, match="32 bits"):
            call()
    pool = k3mla.Pool(n_slots=1, max_ctx=128)
    with pytest.raises(k3mla.K3mlaError, match="32 bits"):
        pool.trim(0, 0, 2 ** 32 + 1)
    with pytest.raises(k3mla.K3mlaError, match="32 bits"):
        pool.truncate(0, 2 ** 32)
    pool.close()
