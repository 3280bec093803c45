"""The bounds that the decode over the 8-bit cache is held to as a whole (window_error.py): they accept weights as pairs of e4m3
numbers in units of the largest of 32 tokens, and reject what the bound of every element lets pass: pairs in units of the largest of
all tokens, one number where two are meant, rows and heads that are off (no GPU needed)."""
from __future__ import annotations

import numpy as np
import pytest

from tests import quant_ref as qr
from tests import window_error
from tests.test_window_error_host import bf16, f16_rows

H, LORA, ROPE, ROW = 96, 512, 64, 576
SCALE = 0.072265625


def e4m3(x):
    return qr.E4M3[qr.to_codes(np.clip(x, -448, 448))]


def pair(x, second=True):
    """x (at most 256) as a sum of two e4m3 numbers, the second in units of 1 / 32."""
    first = e4m3(x)
    return first + (e4m3((x - first) * 32) / 32 if second else 0)


@pytest.fixture(scope="module", params=[(1000, 0.0), (4096, 0.9), (300, 0.99)], ids=str)
def case(request):
    n, share = request.param
    g = np.random.default_rng(n)
    rows = g.standard_normal((n, ROW))
    if share:
        rows[:, :LORA] += g.standard_normal(LORA)
    rows[:, LORA] = 0
    q = bf16(g.standard_normal((H, ROW)) * 0.5)
    q[:, LORA] = 1
    w = bf16(g.standard_normal((H * 256, LORA)) * LORA ** -0.5)
    if share:    # the first token, with an ordinary scale and nearly nothing to add
        w[:, 0] = 0
        mass = np.log(np.exp(q @ rows.T * SCALE).sum(-1)).mean()
        rows[0, :LORA] *= 2.0 ** -6
        rows[0, 0] = 4
        rows[0, LORA:] = 0
        rows[0, LORA] = (mass + np.log(share / (1 - share))) / SCALE
    codes, scale, rope = qr.quantise(bf16(rows))
    s = qr.bits_value(scale)
    vals = np.concatenate([qr.E4M3[codes], qr.bits_value(rope)], -1) * s[:, None]
    w_uv = w.reshape(H, 256, LORA)[:, 128:]

    def out(p, of=vals):       # weights, not yet divided by their sum: what the kernel makes of them
        return bf16(np.einsum("hvk,hk->hv", w_uv, f16_rows(p @ of[:, :LORA])))

    def weights(q=q):
        x = q @ vals.T * SCALE
        e = np.exp(x - x.max(-1, keepdims=True))
        return e / e.sum(-1, keepdims=True)

    exact = np.einsum("hvk,hk->hv", w_uv, weights() @ vals[:, :LORA])
    return dict(q=q, s=s, vals=vals, share=share, out=out, weights=weights, exact=exact)


def held(p, s, tokens, top=256, second=True):
    """p times the rows' powers of two as pairs, in units that bring the largest of `tokens` tokens to below `top`."""
    x = p * s
    for t in range(0, x.shape[1], tokens):
        most = x[:, t:t + tokens].max(-1, keepdims=True)
        unit = 2.0 ** (np.floor(np.log2(most)) + 1 - np.log2(top))
        x[:, t:t + tokens] = pair(x[:, t:t + tokens] / unit, second) * unit
    return x / s


def test_pairs_by_blocks_are_accepted(case):
    p = case["weights"]()
    got = case["out"](held(p, case["s"], 32))
    assert window_error.accepts(got, case["exact"]), window_error.relative(got, case["exact"])[0]
    assert window_error.accepts(bf16(case["exact"]), case["exact"])


def test_wrong_results_are_rejected(case):
    p, s, q, out = case["weights"](), case["s"], case["q"], case["out"]
    size = np.abs(q[:, :LORA]).max() / 256
    one = np.concatenate([e4m3(q[:, :LORA] / size) * size, q[:, LORA:]], -1)
    wrong = dict(one_number_queries=out(case["weights"](one)), zeros=0 * case["exact"], heads=case["exact"][::-1], unscaled=out(p * s),
                 one_head=np.where(np.arange(H)[:, None] == 17, 0, case["exact"]), lost=out(p[:, :-33], case["vals"][:-33]))
    if not case["share"]:      # (a common mean averages the weights' errors out)
        wrong["one_number"] = out(held(p, s, 32, second=False))
    if case["share"] == 0.9:   # the largest of all at 2, with room for 2^7 above it
        wrong["units_of_the_largest"] = out(held(p, s, p.shape[1], top=2))
    for name, got in wrong.items():
        assert not window_error.accepts(bf16(got), case["exact"]), (name, window_error.relative(bf16(got), case["exact"])[0])
