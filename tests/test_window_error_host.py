"""The bounds of window_error.py: they accept the roundings that the windowed kernels make and reject wrong results that
are within the bound of every element (no GPU needed)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import window_error, window_ref as ref

SCALE = 0.072265625
# contexts and windows of the GPU tests that check with it
LENGTHS = [(1024, 64, 2000), (4500, 100, 9000), (300, 1, 700), (64, 4, 130)]


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def f16_rows(x):
    """f16 with a power of two per row that brings its largest entry to [2^14, 2^15)."""
    up = 2.0 ** (14 - np.floor(np.log2(np.abs(x).max(-1, keepdims=True))))
    return (x * up).astype(np.float16).astype(np.float64) / up


@pytest.fixture(scope="module", params=LENGTHS, ids=str)
def case(request):
    window, sink, n = request.param
    rng = np.random.default_rng(window)
    q = rng.standard_normal((ref.H, ref.ROW))
    q[:, :512] *= 0.5
    slab = bf16(rng.standard_normal((-(-n // 64), 1, 64, ref.ROW)))
    w = bf16(rng.standard_normal((ref.H * 256, 512)) * 512 ** -0.5)
    table = np.arange(slab.shape[0])

    def attend(window=window, sink=sink, scale=SCALE):
        return ref.attend(bf16(q), slab, 0, table, n, window, sink, w, scale)

    return dict(window=window, sink=sink, n=n, w=w.reshape(ref.H, 256, 512)[:, 128:], attend=attend, out=attend()[0])


def test_the_kernels_roundings_are_accepted(case):
    _, o, p, rows = case["attend"]()
    pb = bf16(p / p.max(-1, keepdims=True)) * p.max(-1, keepdims=True)
    whole = np.einsum("hvk,hk->hv", case["w"], f16_rows(pb @ rows[:, :512]))
    half = rows.shape[0] // 2
    parts = f16_rows(pb[:, :half] @ rows[:half, :512]) + f16_rows(pb[:, half:] @ rows[half:, :512])
    for got in (bf16(whole), bf16(np.einsum("hvk,hk->hv", case["w"], f16_rows(parts)))):
        assert window_error.accepts(got, case["out"]), window_error.relative(got, case["out"])[0]
    assert window_error.accepts(bf16(case["out"]), case["out"])


def test_wrong_results_are_rejected(case):
    out, a, window, sink = case["out"], case["attend"], case["window"], case["sink"]
    _, _, p, rows = a()
    last = max(1, rows.shape[0] - 128)                     # the last 128-token split left out, p as it was
    lost = np.einsum("hvk,hk->hv", case["w"], p[:, :last] @ rows[:last, :512])
    wrong = dict(zeros=0 * out, short=a(window=max(1, window - 64))[0], long=a(window=window + 64)[0],
                 one_short=a(window=window - 1)[0] if window <= 1024 else None, no_sink=a(sink=0)[0],
                 scale=a(scale=SCALE * 1.02)[0], lost=lost, one_head=np.where(np.arange(ref.H)[:, None] == 17, 0, out))
    for name, got in wrong.items():
        assert got is None or not window_error.accepts(bf16(got), out), (name, window_error.relative(bf16(got), out)[0])
