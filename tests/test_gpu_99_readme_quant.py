"""The README's samples of a layer over the 8-bit cache and of a batch that shares a prompt, run as they stand."""
from __future__ import annotations

import os

import pytest
import torch

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def sample():
    blocks = open(README).read().split("```python\n")[1:]
    block = next(b.split("```")[0] for b in blocks if "quant_decode(" in b.split("```")[0])
    first, second = block.split("\n\n")
    return first, second


def state(k3):
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")
    B, n_prompt, pages = 2, 130, 12
    pool = k3.Pool(n_slots=B, max_ctx=512, n_pages=pages, shuffle_seed=1)
    return dict(k3mla=k3, torch=torch, B=B, pool=pool, layer=0, n_prompt=n_prompt, max_own=64, max_ctx=512, slab=rand(pages, 1, 64, 576),
                slab8=torch.zeros(pages, 1, k3.QUANT_PAGE_BYTES, dtype=torch.uint8, device="cuda"),
                q=rand(B, 96, 192), c_kv=rand(B, 512), k_rope=rand(B, 64), w_kv_b=rand(24576, 512) / 22, wc=rand(512).abs(),
                inv_freq=(10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda(),
                q_abs=torch.full((B, 96, 576), float("nan"), device="cuda").bfloat16(),
                out=torch.full((B, 96, 128), float("nan"), device="cuda").bfloat16(), pos0=torch.full((B,), n_prompt, **i32),
                ctx_len=torch.full((B,), n_prompt + 1, **i32), pages=torch.arange(pages, **i32),
                group_start=torch.tensor([0, B], **i32), shared_len=torch.tensor([n_prompt], **i32),
                ws=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))


def test_a_step_over_the_8_bit_cache(gpu_lib):
    k3, s = gpu_lib, state(gpu_lib)
    for b in range(2):
        assert s["pool"].ensure(b, s["n_prompt"] + 1) == 0
    s["table"] = torch.from_numpy(s["pool"].table()).cuda()
    exec(sample()[0], s)
    torch.cuda.synchronize()
    got = s["out"].clone()
    q_abs = torch.empty_like(s["q_abs"])
    k3.absorb_q(s["q"], s["w_kv_b"], q_abs)               # (q was rotated in place)
    k3.quant_decode(q_abs, s["slab8"], 0, s["table"], s["ctx_len"], s["w_kv_b"], 0x3D94, s["out"], s["ws"], 512)
    assert got.isfinite().all() and got.any() and torch.equal(s["q_abs"], q_abs)
    # (other splits: the outputs' roundings, 2^-8 each)
    assert (got.float() - s["out"].float()).abs().max() <= 2.0 ** -7 * got.float().abs().max()


def test_a_batch_that_shares_a_prompt(gpu_lib):
    k3, s = gpu_lib, state(gpu_lib)
    k3.absorb_q(s["q"], s["w_kv_b"], s["q_abs"])
    assert s["pool"].ensure(0, s["n_prompt"]) == 0
    share, rest = sample()[1].split("\n", 1)
    exec(share, s)
    for b in range(2):
        assert s["pool"].ensure(b, s["n_prompt"] + 1) == 0
    s["table"] = torch.from_numpy(s["pool"].table()).cuda()
    exec(rest, s)
    torch.cuda.synchronize()
    want = torch.empty_like(s["out"])
    k3.window_decode(s["q_abs"], s["slab"], 0, s["table"], s["ctx_len"], s["w_kv_b"], 0x3D94, want, s["ws"], 512, 512)
    assert s["out"].isfinite().all() and s["out"].any()
    # (other splits: p and the outputs rounded to bf16 on both sides, 2^-8 each)
    assert (want.float() - s["out"].float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()
