"""Workloads of the windowed latent-cache operators: what a user's program has in hand before a call
(`prepare`), the call itself (`run`), what it cannot do without (`work`) and its result in 64 bits
(`exact`).

Four operators over the paged latent cache ([page][layer][64 tokens][576] bf16):

  rows     norms of the queries (per head) and of the latent and rope key, the position rotation of both,
           and the write of the cache rows into their mapped pages
  window   decode of one token per slot over the last `window` tokens and the first `sink` tokens
  chunk    the same for a chunk of new tokens per slot, each token with its own window
  compact  an eviction: the kept tokens of every slot move down to the front of its pages

`own` false: elementary torch operations in 32 bits (angles in 64), rounded once at the end; `own` true:
the library's calls.
"""
import math
import random

import torch

own = False

H, NOPE, ROPE, V, LORA, PAGE, ROW = 96, 128, 64, 128, 512, 64, 576
LAYERS, LAYER = 2, 1          # the slab of an attention case holds two layers; the calls work on the second
SCALE_BITS = 0x3D94           # bf16(1 / sqrt(192))
SCALE = 0.072265625
EPS = 1e-6


def listed():
    return [
        # one new token of one slot: a lone stream's decode step, where latency is all there is
        {"name": "rows 1x1", "op": "rows", "slots": 1, "chunk": 1, "ragged": False, "lo": 130, "hi": 130, "lens": 0,
         "norms": True, "rotate": "halves"},
        # the decode step of the 64-slot batch at 4096 tokens
        {"name": "rows 64x1", "op": "rows", "slots": 64, "chunk": 1, "ragged": False, "lo": 4096, "hi": 4096, "lens": 2,
         "norms": True, "rotate": "pairs"},
        # prefill: ragged chunks of 16 slots, some 6 thousand token rows
        {"name": "rows 16x601", "op": "rows", "slots": 16, "chunk": 601, "ragged": True, "lo": 601, "hi": 4096, "lens": 1,
         "norms": True, "rotate": "halves"},
        # a lone stream far into a long context: a short work list on a large machine
        {"name": "window 1 slot", "op": "window", "slots": 1, "lo": 32768, "hi": 32768, "lens": 3, "empty": 0.0,
         "window": 4096, "sink": 4},
        # the ragged 16-slot batch: contexts shorter and longer than the window
        {"name": "window 16 ragged", "op": "window", "slots": 16, "lo": 1, "hi": 4096, "lens": 1, "empty": 0.0,
         "window": 1000, "sink": 4},
        # the steady 64-slot batch
        {"name": "window 64", "op": "window", "slots": 64, "lo": 4096, "hi": 4096, "lens": 2, "empty": 0.0,
         "window": 1024, "sink": 64},
        # the padded bucket: 128 rows, 40 % of them empty, contexts up to 256
        {"name": "window 128 padded", "op": "window", "slots": 128, "lo": 1, "hi": 256, "lens": 4, "empty": 0.4,
         "window": 128, "sink": 1},
        # long contexts with a wide window: the cache read is all there is
        {"name": "window 64 wide", "op": "window", "slots": 64, "lo": 32000, "hi": 32768, "lens": 5, "empty": 0.0,
         "window": 4096, "sink": 4},
        # chunked prefill of the 16-slot batch, 64 tokens each
        {"name": "chunk 16x64", "op": "chunk", "slots": 16, "chunk": 64, "ragged": False, "lo": 4096, "hi": 4096, "lens": 1,
         "window": 1024, "sink": 4},
        # one prompt from its first token on, and a window shorter than it
        {"name": "chunk 1x1000", "op": "chunk", "slots": 1, "chunk": 1000, "ragged": False, "lo": 1000, "hi": 1000, "lens": 2,
         "window": 300, "sink": 1},
        # eviction in a lone slot, every layer keeping the same tokens
        {"name": "compact 1 slot", "op": "compact", "slots": 1, "layers": 24, "lo": 4096, "hi": 4096, "lens": 3, "keep": 1028,
         "per_layer": False},
        # eviction in the ragged batch, every layer keeping tokens of its own
        {"name": "compact 16 ragged", "op": "compact", "slots": 16, "layers": 24, "lo": 1, "hi": 4096, "lens": 1, "keep": 1500,
         "per_layer": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rows", "window", "window", "chunk", "compact"))
    lens = rng.randrange(1 << 20)
    if op == "rows":
        slots = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(1, 6000 // slots))
        hi = max(chunk, _log(rng, 64, 4096))
        return {"op": op, "slots": slots, "chunk": chunk, "ragged": rng.random() < 0.5, "lo": max(chunk, hi // 3), "hi": hi,
                "lens": lens, "norms": rng.random() < 0.8, "rotate": rng.choice(("halves", "pairs", "none"))}
    if op == "window":
        slots, window, hi = _log(rng, 1, 128), _log(rng, 1, 4096), _log(rng, 64, 32768)
        while slots * min(window, hi) > 64 * 4096:
            slots = max(1, slots // 2)
        return {"op": op, "slots": slots, "lo": rng.choice((1, max(1, hi // 2), hi)), "hi": hi, "lens": lens,
                "empty": rng.choice((0.0, 0.0, 0.3)), "window": window, "sink": rng.choice((0, 1, 4, 64, rng.randrange(200)))}
    if op == "chunk":
        slots, window = _log(rng, 1, 16), _log(rng, 16, 1024)
        chunk = _log(rng, 1, 1024 // slots)
        hi = max(chunk, _log(rng, 64, 4096))
        return {"op": op, "slots": slots, "chunk": chunk, "ragged": rng.random() < 0.5, "lo": max(chunk, hi // 2), "hi": hi,
                "lens": lens, "window": window, "sink": rng.choice((0, 1, 4, 64))}
    slots, layers, hi = _log(rng, 1, 16), rng.choice((1, 2, 7, 24)), _log(rng, 64, 4096)
    return {"op": op, "slots": slots, "layers": layers, "lo": rng.choice((hi // 2, hi)), "hi": hi, "lens": lens,
            "keep": _log(rng, 8, max(8, hi * 6 // 10)), "per_layer": rng.random() < 0.5}


# ---- what a case's numbers come to -------------------------------------------------------------


def _lengths(case):
    """Per slot: the context after the call and the new tokens in it."""
    r = random.Random(case["lens"])
    ctx = [r.randint(case["lo"], case["hi"]) for _ in range(case["slots"])]
    for b in range(case["slots"]):
        if r.random() < case.get("empty", 0.0):
            ctx[b] = 0
    chunk = case.get("chunk", 1)
    new = [min(c, r.randint(1, chunk) if case.get("ragged") else chunk) for c in ctx]
    return ctx, new


def _visible(n, window, sink):
    """Tokens that the last of n tokens attends to."""
    first = max(0, n - window)
    return min(n, sink, first) + n - first


def work(case):
    ctx, new = _lengths(case)
    op = case["op"]
    if op == "rows":
        rows = sum(new)
        q = H * (NOPE + ROPE) if case["norms"] else H * (NOPE + ROPE if case["rotate"] == "none" else ROPE)
        return {"bytes": rows * 2 * (2 * q + 2 * ROW), "flops": rows * 6.0 * (q + ROW)}
    if op == "compact":
        moved = sum(max(0, case["keep"] - 4) for c in ctx if c > case["keep"])     # the first four stay in place
        lists = sum(min(c, case["keep"]) for c in ctx) * (case["layers"] if case["per_layer"] else 1)
        return {"bytes": moved * case["layers"] * ROW * 2 * 2 + 4 * lists, "flops": 0.0}
    w, s = case["window"], case["sink"]
    rows = sum(1 for c in ctx if c) if op == "window" else sum(new)
    read = sum(_visible(c, w + n - 1, s) for c, n in zip(ctx, new))                  # cache rows, each once
    pairs = sum(_visible(c - j, w, s) for c, n in zip(ctx, new) for j in range(n))   # (new token, seen token)
    return {"bytes": 2.0 * (read * ROW + rows * H * (ROW + V) + H * V * LORA),
            "flops": 2.0 * H * (pairs * (ROW + LORA) + rows * LORA * V)}


# ---- inputs ------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _paged(g, ctx, layers, first=None):
    """A slab of random latents and a table that maps every slot's tokens to scattered pages; pages of
    tokens before first[b] (and past the sinks first[b] names) have been freed."""
    cols = max(1, max((c + PAGE - 1) // PAGE for c in ctx))
    live = []
    for b, c in enumerate(ctx):
        keep, lo = first[b] if first else (0, 0)
        live += [(b, lp) for lp in range((c + PAGE - 1) // PAGE) if lp * PAGE < keep or (lp + 1) * PAGE > lo]
    n_pages = max(1, len(live))
    table = torch.full((len(ctx), cols), -1, dtype=torch.int32, device="cuda")
    if live:
        at = torch.tensor(live, device="cuda").T
        table[at[0], at[1]] = torch.randperm(n_pages, generator=g, device="cuda")[: len(live)].int()
    return _normal(g, n_pages, layers, PAGE, ROW), table


def prepare(case, seed):
    g = _gen(seed)
    ctx, new = _lengths(case)
    op, B = case["op"], case["slots"]
    st = {"case": case, "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"), "max_ctx": max(1, max(ctx)),
          "pos0": torch.tensor([c - n for c, n in zip(ctx, new)], dtype=torch.int32, device="cuda"),
          "row_start": torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda"),
          "rows": sum(new), "max_new": max(new)}
    if op == "rows":
        R = st["rows"]
        st["slab"], st["table"] = _paged(g, ctx, LAYERS)
        st["q"] = _normal(g, R, H, NOPE + ROPE)
        st["kv"] = _normal(g, R, ROW)             # the projection's rows: latent | rope key, not yet normed
        st["q_out"] = torch.empty_like(st["q"])
        weight = lambda n: (1.0 + 0.2 * torch.randn(n, generator=g, device="cuda")).bfloat16()  # noqa: E731
        st["weights"] = (weight(NOPE + ROPE), weight(LORA), weight(ROPE)) if case["norms"] else (None, None, None)
        st["inv_freq"] = None
        if case["rotate"] != "none":
            st["inv_freq"] = (10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)).float()
        return st
    if op == "compact":
        st["slab"], st["table"] = _paged(g, ctx, case["layers"])
        sets = case["layers"] if case["per_layer"] else 1
        keep = []
        for c in ctx:      # the first tokens, the latest, and in between those that drew the largest scores
            k = min(c, case["keep"])
            score = torch.rand(sets, c, generator=g, device="cuda")
            score[:, :4] += 2
            score[:, c - k // 2:] += 2
            keep.append(score.topk(k, dim=1).indices.sort(dim=1).values.int())
        kept = [k.shape[1] for k in keep]
        st["keep"] = torch.cat(keep, 1).contiguous()
        st["keep_start"] = torch.tensor([sum(kept[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        return st
    w, s = case["window"], case["sink"]
    st["slab"], st["table"] = _paged(g, ctx, LAYERS, [(min(s, c), max(0, c - n + 1 - w)) for c, n in zip(ctx, new)])
    R = B if op == "window" else st["rows"]
    st["q_abs"] = _normal(g, R, H, ROW, std=0.5)   # 128 products with weights of variance 1 / 512
    st["q_abs"][:, :, LORA:] = _normal(g, R, H, ROPE)
    st["w_kv_b"] = _normal(g, H * (NOPE + V), LORA, std=LORA ** -0.5)
    st["out"] = torch.empty(R, H, V, dtype=torch.bfloat16, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------------------------


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st)
    if op == "rows":
        return _rows(st)
    if op == "compact":
        return _compact(st)
    return _attend(st)


def _own(st):
    from paged_latent_attention_k3mla_gb300 import k3mla

    case = st["case"]
    op = case["op"]
    if op == "rows":
        qw, cw, kw = st["weights"]
        k3mla.norm_rope_append(st["q"], st["q_out"], st["slab"], LAYER, st["table"], st["pos0"], st["row_start"],
                               st["kv"][:, :LORA], st["kv"][:, LORA:], q_weight=qw, c_weight=cw, k_weight=kw, eps=EPS,
                               inv_freq=st["inv_freq"], interleaved=case["rotate"] == "pairs")
        return {"q": st["q_out"], "slab": st["slab"]}
    if op == "compact":
        k3mla.compact_rows(st["slab"], st["table"], st["keep"], st["keep_start"])
        return st["slab"]
    w, s, B = case["window"], case["sink"], case["slots"]
    if op == "window":
        if "ws" not in st:   # planned and allocated once, as a serving program does
            st["split"] = k3mla.window_split_tokens(B, st["max_ctx"], w, s)
            st["ws"] = torch.empty(k3mla.window_decode_workspace_bytes(B, st["max_ctx"], w, s, st["split"]),
                                   dtype=torch.uint8, device="cuda")
        k3mla.window_decode(st["q_abs"], st["slab"], LAYER, st["table"], st["ctx"], st["w_kv_b"], SCALE_BITS, st["out"],
                            st["ws"], st["max_ctx"], w, s, st["split"])
        return st["out"]
    if "ws" not in st:
        st["ws"] = torch.empty(k3mla.window_chunk_decode_workspace_bytes(B, st["rows"], st["max_ctx"]),
                               dtype=torch.uint8, device="cuda")
    k3mla.window_chunk_decode(st["q_abs"], st["slab"], LAYER, st["table"], st["pos0"], st["row_start"], st["w_kv_b"],
                              SCALE_BITS, st["out"], st["ws"], st["max_ctx"], w, s)
    return st["out"]


def _slot_of(starts, n):
    """The slot of each of n packed rows, and the row's place in it."""
    r = torch.arange(n, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(starts, r, right=True) - 1
    return b, r - starts[b]


def _norm(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def _rotate(x, cos, sin, pairs):
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., : ROPE // 2], x[..., ROPE // 2:])
    y = (a * cos - b * sin, a * sin + b * cos)
    return torch.stack(y, -1).flatten(-2) if pairs else torch.cat(y, -1)


def _rows(st):
    case = st["case"]
    qw, cw, kw = st["weights"]
    b, j = _slot_of(st["row_start"], st["rows"])
    pos = (st["pos0"][b] + j).long()
    q = _norm(st["q"].float(), qw)
    c = _norm(st["kv"][:, :LORA].float(), cw)
    k = _norm(st["kv"][:, LORA:].float(), kw)
    if st["inv_freq"] is not None:
        angle = pos.double()[:, None] * st["inv_freq"].double()
        cos, sin = angle.cos().float(), angle.sin().float()
        pairs = case["rotate"] == "pairs"
        q = torch.cat([q[..., :NOPE], _rotate(q[..., NOPE:], cos[:, None], sin[:, None], pairs)], -1)
        k = _rotate(k, cos, sin, pairs)
    st["slab"][st["table"][b, pos // PAGE].long(), LAYER, pos % PAGE] = torch.cat([c, k], -1).bfloat16()
    return {"q": q.bfloat16(), "slab": st["slab"]}


def _compact(st):
    slab, table, keep = st["slab"], st["table"], st["keep"].long()
    L = slab.shape[1]
    b, i = _slot_of(st["keep_start"], keep.shape[1])
    i = i.long()
    layer = torch.arange(L, device="cuda")[:, None]
    flat = slab.view(-1, ROW)
    src = (table[b[None, :], keep // PAGE].long() * L + layer) * PAGE + keep % PAGE
    dst = (table[b, i // PAGE].long() * L + layer) * PAGE + i % PAGE
    flat[dst] = flat[src]
    return slab


def _attend(st):
    case, slab, table = st["case"], st["slab"], st["table"]
    w, s, B = case["window"], case["sink"], case["slots"]
    ctx, first = st["ctx"].long()[:, None], (st["pos0"].long() + 1)[:, None]   # contexts of the last and first new token
    if case["op"] == "window":
        first = ctx
    M = 1 if case["op"] == "window" else st["max_new"]
    lo = (first - w).clamp(min=s)
    span = min(st["max_ctx"], w + M - 1)
    t = torch.cat([torch.arange(s, device="cuda").expand(B, s), lo + torch.arange(span, device="cuda")], 1)   # [B, T]
    page = table.gather(1, (t // PAGE).clamp(max=table.shape[1] - 1)).long()
    there = (t < ctx) & (page >= 0)
    rows = slab[page.clamp(min=0), LAYER, t % PAGE].float() * there[..., None]
    if M == 1 and case["op"] == "window":
        q = st["q_abs"].float()[:, None]
        n = ctx
    else:
        r = torch.arange(M, device="cuda")
        at = (st["row_start"][:-1].long()[:, None] + r).clamp(max=st["rows"] - 1)
        q = st["q_abs"][at].float()
        n = first + r                                                          # [B, M]
    seen = (t[:, None] < n[..., None]) & ((t[:, None] < s) | (t[:, None] >= n[..., None] - w)) & (t[:, None] < ctx[..., None])
    score = torch.matmul(q.view(B, M * H, ROW), rows.transpose(1, 2)).view(B, M, H, -1) * SCALE
    score = score.masked_fill(~seen[:, :, None], float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(B, M * H, -1), rows[..., :LORA]).view(B * M, H, LORA)
    w_uv = st["w_kv_b"].view(H, NOPE + V, LORA)[:, NOPE:].float()
    out = torch.matmul(o.transpose(0, 1), w_uv.transpose(1, 2)).transpose(0, 1)
    if case["op"] == "chunk":
        b, j = _slot_of(st["row_start"], st["rows"])
        out = out.reshape(B, M, H, V)[b, j.long()]
    return out.bfloat16()


# ---- the definitions in 64 bits, slot by slot ----------------------------------------------------


def exact(case, seed):
    st = prepare(case, seed)
    ctx, new = _lengths(case)
    table, slab = st["table"].long(), st["slab"].double()

    def address(b, t):
        return table[b, torch.div(t, PAGE, rounding_mode="floor")], t % PAGE

    if case["op"] == "compact":
        L, start = case["layers"], st["keep_start"].tolist()
        result = slab.clone()
        for b in range(case["slots"]):
            kept = st["keep"][:, start[b]:start[b + 1]].long()
            to = address(b, torch.arange(kept.shape[1], device="cuda"))
            for layer in range(L):
                at = address(b, kept[layer if case["per_layer"] else 0])
                result[to[0], layer, to[1]] = slab[at[0], layer, at[1]]
        return result
    if case["op"] == "rows":
        pos = torch.cat([torch.arange(c - n, c, device="cuda", dtype=torch.float64) for c, n in zip(ctx, new)])
        slot = torch.cat([torch.full((n,), b, device="cuda") for b, n in enumerate(new)])
        x = [st["q"].double(), st["kv"][:, :LORA].double(), st["kv"][:, LORA:].double()]
        for i, wt in enumerate(st["weights"]):
            if wt is not None:
                x[i] = wt.double() * x[i] / (x[i].pow(2).sum(-1, keepdim=True) / x[i].shape[-1] + EPS).sqrt()
        q, c, k = x
        if st["inv_freq"] is not None:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None] * st["inv_freq"].double())
            for v, z in ((q, turn[:, None]), (k, turn)):
                part = v[..., -ROPE:]
                if case["rotate"] == "pairs":
                    y = torch.view_as_complex(part.reshape(*part.shape[:-1], ROPE // 2, 2).contiguous()) * z
                    part.copy_(torch.view_as_real(y).reshape(part.shape))
                else:
                    y = torch.complex(part[..., :ROPE // 2].contiguous(), part[..., ROPE // 2:].contiguous()) * z
                    part.copy_(torch.cat([y.real, y.imag], -1))
        for b in range(case["slots"]):
            mine = slot == b
            page, line = address(b, pos[mine].long())
            slab[page, LAYER, line, :LORA] = c[mine]
            slab[page, LAYER, line, LORA:] = k[mine]
        return {"q": q, "slab": slab}
    w, s = case["window"], case["sink"]
    w_uv = st["w_kv_b"].double().view(H, NOPE + V, LORA)[:, NOPE:]
    out, row = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        if not c:
            row += case["op"] == "window"
            continue
        t = torch.arange(c, device="cuda")
        t = t[(t < s) | (t > c - n - w)]
        page, line = address(b, t)
        rows = slab[page.clamp(min=0), LAYER, line] * (page >= 0)[:, None]
        for a in range(0, n, 64):                      # a few query tokens at a time
            m = min(64, n - a)
            own_n = c - n + a + 1 + torch.arange(m, device="cuda")[:, None]
            hide = (t >= own_n) | ((t >= s) & (t < own_n - w))
            score = torch.einsum("mhk,tk->mht", st["q_abs"][row + a:row + a + m].double(), rows) * SCALE
            p = score.masked_fill(hide[:, None], float("-inf")).softmax(-1)
            out[row + a:row + a + m] = torch.einsum("hvk,mhk->mhv", w_uv, torch.einsum("mht,tk->mhk", p, rows[:, :LORA]))
        row += n if case["op"] == "chunk" else 1
    return out
