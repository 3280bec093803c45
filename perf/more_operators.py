"""Workloads of the operators over an 8-bit latent cache and over shared prefixes: what a user's program has in
hand before a call (`prepare`), the call itself (`run`), what it cannot do without (`work`) and its result in 64
bits (`exact`).

Four operators:

  rows    norms and rotation of queries and keys, and the cache rows written as 8-bit latents with a power of two
          per row (e4m3) and a bf16 rope key
  pages   whole bf16 pages into the 8-bit cache ("in"), and back ("back")
  decode  decode of one token per slot over the 8-bit cache: the whole context, or a window and the first tokens
  shared  decode over the bf16 cache for groups of slots whose tables begin with the same pages

An 8-bit page of a layer is 64 rows of 640 bytes (512 e4m3 codes, then 64 bf16 rope entries) and then 64 bf16
scales, one a row; a row stands for its codes, and its rope entries, times its scale.

`own` false: elementary torch operations in 32 bits (angles in 64), rounded once at the end; `own` true: the
library's calls.
"""
import math
import random

import torch

own = False

H, NOPE, ROPE, V, LORA, PAGE, ROW = 96, 128, 64, 128, 512, 64, 576
ROW8 = LORA + 2 * ROPE               # bytes of an 8-bit row without its scale
PAGE8 = PAGE * ROW8 + 2 * PAGE       # bytes of an 8-bit page of a layer
LAYERS, LAYER = 2, 1          # the slab of an attention case holds two layers; the calls work on the second
SCALE_BITS = 0x3D94           # bf16(1 / sqrt(192))
SCALE = 0.072265625
EPS = 1e-6
MOST = 1 << 30                # a window that nothing reaches: the whole context


def listed():
    return [
        # one new token of one slot: a lone stream's decode step, where latency is all there is
        {"name": "rows 1x1", "op": "rows", "slots": 1, "chunk": 1, "ragged": False, "lo": 130, "hi": 130, "lens": 0,
         "norms": True, "rotate": "halves"},
        # prefill: ragged chunks of 16 slots, some 6 thousand token rows
        {"name": "rows 16x601", "op": "rows", "slots": 16, "chunk": 601, "ragged": True, "lo": 601, "hi": 4096, "lens": 1,
         "norms": True, "rotate": "pairs"},
        # a page that has just filled up, all layers of it, moves into the 8-bit cache
        {"name": "pages in 1", "op": "pages", "back": False, "pages": 1, "layers": 24},
        # a prefilled prompt of 4096 tokens is adopted into the 8-bit cache
        {"name": "pages in 64", "op": "pages", "back": False, "pages": 64, "layers": 24},
        # a cached prefix of 4000 tokens is read back for a chunked prefill that goes on from it
        {"name": "pages back 63", "op": "pages", "back": True, "pages": 63, "layers": 24},
        # a lone stream far into a long context: a short work list on a large machine
        {"name": "decode 1 slot", "op": "decode", "slots": 1, "lo": 32768, "hi": 32768, "lens": 3, "empty": 0.0,
         "window": MOST, "sink": 0},
        # the padded bucket: 128 rows, 40 % of them empty, contexts up to 256, a window and the first token
        {"name": "decode 128 padded", "op": "decode", "slots": 128, "lo": 1, "hi": 256, "lens": 4, "empty": 0.4,
         "window": 128, "sink": 1},
        # the steady 64-slot batch
        {"name": "decode 64", "op": "decode", "slots": 64, "lo": 4096, "hi": 4096, "lens": 2, "empty": 0.0,
         "window": MOST, "sink": 0},
        # long contexts: the cache read is all there is
        {"name": "decode 64 long", "op": "decode", "slots": 64, "lo": 15000, "hi": 16384, "lens": 5, "empty": 0.0,
         "window": MOST, "sink": 0},
        # eight samples of one 4096-token prompt, a few tokens in
        {"name": "shared 8", "op": "shared", "groups": 1, "size": 8, "ragged": False, "shared": 4096, "own_lo": 1, "own_hi": 64,
         "lens": 1, "alone": 0},
        # five conversations with branches of their own and some requests that share nothing
        {"name": "shared ragged", "op": "shared", "groups": 5, "size": 7, "ragged": True, "shared": 2500, "own_lo": 1,
         "own_hi": 1000, "lens": 2, "alone": 3},
        # 64 requests behind one long system prompt
        {"name": "shared 64", "op": "shared", "groups": 1, "size": 64, "ragged": False, "shared": 16384, "own_lo": 100,
         "own_hi": 600, "lens": 3, "alone": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("rows", "pages", "decode", "decode", "shared", "shared"))
    lens = rng.randrange(1 << 20)
    if op == "rows":
        slots = _log(rng, 1, 64)
        chunk = _log(rng, 1, max(1, 6000 // slots))
        hi = max(chunk, _log(rng, 64, 4096))
        return {"op": op, "slots": slots, "chunk": chunk, "ragged": rng.random() < 0.5, "lo": max(chunk, hi // 3), "hi": hi,
                "lens": lens, "norms": rng.random() < 0.8, "rotate": rng.choice(("halves", "pairs", "none"))}
    if op == "pages":
        return {"op": op, "back": rng.random() < 0.5, "pages": _log(rng, 1, 64), "layers": _log(rng, 1, 24)}
    if op == "decode":
        slots, hi = _log(rng, 1, 128), _log(rng, 64, 32768)
        while slots * hi > 64 * 15000:
            slots = max(1, slots // 2)
        return {"op": op, "slots": slots, "lo": rng.choice((1, max(1, hi // 2), hi)), "hi": hi, "lens": lens,
                "empty": rng.choice((0.0, 0.0, 0.3)), "window": rng.choice((MOST, MOST, _log(rng, 1, 4096))),
                "sink": rng.choice((0, 1, 4, 64, rng.randrange(200)))}
    groups, size, shared = _log(rng, 1, 8), _log(rng, 1, 64), _log(rng, 64, 16384)
    while groups * size > 64:
        size = max(1, size // 2)
    while groups * size * shared > 64 * 16384:
        shared = max(64, shared // 2)
    own_hi = _log(rng, 1, 1000)
    return {"op": op, "groups": groups, "size": size, "ragged": rng.random() < 0.5, "shared": shared,
            "own_lo": rng.choice((1, own_hi)), "own_hi": own_hi, "lens": lens, "alone": rng.choice((0, 0, 1, 5))}


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


def _groups(case):
    """(slots, shared tokens) of every group, then every slot's context: what it shares and its own tokens."""
    r = random.Random(case["lens"])
    groups = [(r.randint(1, case["size"]) if case["ragged"] else case["size"],
               max(1, case["shared"] - (r.randint(0, case["shared"] // 2) if case["ragged"] else 0)))
              for _ in range(case["groups"])]
    ctx = [shared + r.randint(case["own_lo"], case["own_hi"]) for size, shared in groups for _ in range(size)]
    return groups, ctx + [r.randint(case["own_lo"], case["own_hi"]) for _ in range(case["alone"])]


def _whole(n):
    return n // PAGE * PAGE


def _seen(n, window, sink):
    """How many tokens the last of n tokens attends to."""
    first = max(0, n - window)
    return min(n, sink, first) + n - first


def work(case):
    op = case["op"]
    if op == "rows":
        rows = sum(_lengths(case)[1])
        q = H * (NOPE + ROPE) if case["norms"] else H * (NOPE + ROPE if case["rotate"] == "none" else ROPE)
        return {"bytes": rows * (4 * q + 2 * ROW + ROW8 + 2), "flops": rows * 6.0 * (q + ROW)}
    if op == "pages":
        n = case["pages"] * case["layers"]
        return {"bytes": n * (PAGE * ROW * 2 + PAGE8), "flops": n * PAGE * ROW * 2.0}
    if op == "decode":
        ctx, _ = _lengths(case)
        rows, pairs = sum(1 for c in ctx if c), sum(_seen(c, case["window"], case["sink"]) for c in ctx)
        read = pairs * (ROW8 + 2)
    else:
        groups, ctx = _groups(case)
        rows, pairs = len(ctx), sum(ctx)
        read = 2.0 * ROW * (pairs - sum((size - 1) * _whole(shared) for size, shared in groups))
    return {"bytes": read + 2.0 * (rows * H * (ROW + V) + H * V * LORA),
            "flops": 2.0 * H * (pairs * (ROW + LORA) + rows * LORA * V)}


# ---- inputs ------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape, std=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, std, generator=g)


def _latents(g, *shape):
    """Latent rows as a trained model has them: the norm's weights give every entry a size of its own, and rows differ."""
    x = torch.empty(*shape, LORA, dtype=torch.float32, device="cuda").normal_(generator=g)
    x *= torch.exp(0.5 * torch.randn(LORA, generator=g, device="cuda"))
    x *= torch.exp(0.3 * torch.randn(*shape, 1, generator=g, device="cuda"))
    return x


def _parts(slab8):
    """The three kinds of value that an 8-bit slab [pages][layers][PAGE8] holds: codes, scales, rope entries."""
    rows = slab8[..., : PAGE * ROW8].unflatten(-1, (PAGE, ROW8))
    scale = slab8[..., PAGE * ROW8:].view(torch.bfloat16)
    return rows[..., :LORA].view(torch.float8_e4m3fn), scale, rows[..., LORA:].view(torch.bfloat16)


def _power(n):
    """2^n, to the bit (torch's own powers are off in the last place on the GPU)."""
    return ((n.int() + 127) << 23).view(torch.float32)


def _quantise(c, k):
    """f32 latents and rope keys -> codes, scales, rope entries: the largest finite latent of a row comes to (224, 448]."""
    m = torch.where(c.isfinite(), c.abs(), 0.0).amax(-1)
    r = torch.where(k.isfinite(), k.abs(), 0.0).amax(-1)
    f, e = torch.frexp(m)
    n = torch.where(m > 0, e - 9 + (f > 0.875).int(), 0)
    n = torch.maximum(n, torch.frexp(r)[1] - 120).clamp(-96, 120)
    down = _power(-n)[..., None]
    return (c * down).to(torch.float8_e4m3fn), _power(n).bfloat16(), (k * down).bfloat16()


def _fill(slab8, c, k):
    for part, x in zip(_parts(slab8), _quantise(c, k)):
        part.copy_(x)


def _slab8(g, pages, layers):
    slab8 = torch.empty(pages, layers, PAGE8, dtype=torch.uint8, device="cuda")
    for p in range(0, pages, 512):
        n = min(512, pages - p)
        _fill(slab8[p:p + n], _latents(g, n, layers, PAGE), _normal(g, n, layers, PAGE, ROPE).float())
    return slab8


def _slab16(g, pages, layers):
    slab = _normal(g, pages, layers, PAGE, ROW)
    for p in range(0, pages, 512):
        n = min(512, pages - p)
        slab[p:p + n, ..., :LORA] = _latents(g, n, layers, PAGE).bfloat16()
    return slab


def _table(g, live, slots):
    """A table that maps the listed (slot, logical page) pairs, or lists of them to one page, to scattered pages."""
    cols = max([1] + [lp + 1 for ps in live for _, lp in ps])
    table = torch.full((slots, cols), -1, dtype=torch.int32, device="cuda")
    n = max(1, len(live))
    if live:
        ids = torch.randperm(n, generator=g, device="cuda")[: len(live)].int()
        at = torch.tensor([(b, lp, i) for i, ps in enumerate(live) for b, lp in ps], device="cuda").T
        table[at[0], at[1]] = ids[at[2]]
    return n, table


def _count(c):
    return (c + PAGE - 1) // PAGE


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "pages":
        n, layers = case["pages"], case["layers"]
        st["src"] = torch.randperm(n + 2, generator=g, device="cuda")[:n].int()
        st["dst"] = torch.randperm(n + 3, generator=g, device="cuda")[:n].int()
        if case["back"]:
            st["slab8"] = _slab8(g, n + 2, layers)
            st["slab"] = torch.zeros(n + 3, layers, PAGE, ROW, dtype=torch.bfloat16, device="cuda")
        else:
            st["slab"] = _slab16(g, n + 2, layers)
            st["slab8"] = torch.zeros(n + 3, layers, PAGE8, dtype=torch.uint8, device="cuda")
        return st
    if op == "shared":
        groups, ctx = _groups(case)
        start = [sum(s for s, _ in groups[:i]) for i in range(len(groups) + 1)]
        live = [[(b, lp) for b in range(start[i], start[i + 1])] for i, (_, shared) in enumerate(groups)
                for lp in range(shared // PAGE)]
        first = [shared // PAGE for size, shared in groups for _ in range(size)] + [0] * case["alone"]
        live += [[(b, lp)] for b, c in enumerate(ctx) for lp in range(first[b], _count(c))]
        st["group_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        st["shared_len"] = torch.tensor([s for _, s in groups], dtype=torch.int32, device="cuda")
        st["max_shared"] = max(s for _, s in groups)
        st["max_own"] = max(c - PAGE * f for c, f in zip(ctx, first))
        pages, st["table"] = _table(g, live, len(ctx))
        st["slab"] = _slab16(g, pages, LAYERS)
    else:
        ctx, new = _lengths(case)
        w, s = case.get("window", MOST), case.get("sink", 0)
        # (pages that no token sees have been freed)
        pages, st["table"] = _table(g, [[(b, lp)] for b, c in enumerate(ctx) for lp in range(_count(c))
                                        if lp * PAGE < s or (lp + 1) * PAGE > c - w], len(ctx))
        st["slab8"] = _slab8(g, pages, LAYERS)
    B = len(ctx)
    st["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st["max_ctx"] = max(1, max(ctx))
    if op == "rows":
        R = st["rows"] = sum(new)
        st["pos0"] = torch.tensor([c - n for c, n in zip(ctx, new)], dtype=torch.int32, device="cuda")
        st["row_start"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
        st["q"] = _normal(g, R, H, NOPE + ROPE)
        st["kv"] = _normal(g, R, ROW)             # the projection's rows: latent | rope key, not yet normed
        st["q_out"] = torch.empty_like(st["q"])
        weight = lambda n, s: torch.exp(s * torch.randn(n, generator=g, device="cuda")).bfloat16()  # noqa: E731
        st["weights"] = (weight(NOPE + ROPE, 0.2), weight(LORA, 0.5), weight(ROPE, 0.2)) if case["norms"] else (None, None, None)
        st["inv_freq"] = None
        if case["rotate"] != "none":
            st["inv_freq"] = (10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE)).float()
        return st
    st["q_abs"] = _normal(g, B, H, ROW, std=0.5)   # 128 products with weights of variance 1 / 512
    st["q_abs"][:, :, LORA:] = _normal(g, B, H, ROPE)
    st["w_kv_b"] = _normal(g, H * (NOPE + V), LORA, std=LORA ** -0.5)
    st["out"] = torch.empty(B, H, V, dtype=torch.bfloat16, device="cuda")
    return st


# ---- one pass ----------------------------------------------------------------------------------


def run(st):
    op = st["case"]["op"]
    if own:
        return _own(st)
    if op == "rows":
        return _rows(st)
    if op == "pages":
        return _pages(st)
    return _decode(st) if op == "decode" else _shared(st)


def _named(slab8):
    codes, scale, rope = _parts(slab8)
    return {"codes": codes, "scale": scale, "rope": rope}


def _own(st):
    from paged_latent_attention_k3mla_gb300 import k3mla

    case = st["case"]
    op = case["op"]
    if op == "rows":
        qw, cw, kw = st["weights"]
        k3mla.quant_norm_rope_append(st["q"], st["q_out"], st["slab8"], LAYER, st["table"], st["pos0"], st["row_start"],
                                     st["kv"][:, :LORA], st["kv"][:, LORA:], q_weight=qw, c_weight=cw, k_weight=kw, eps=EPS,
                                     inv_freq=st["inv_freq"], interleaved=case["rotate"] == "pairs")
        return {"q": st["q_out"], **_named(st["slab8"])}
    if op == "pages":
        if case["back"]:
            k3mla.quant_read_pages(st["slab"], st["slab8"], st["src"], st["dst"])
            return st["slab"]
        k3mla.quant_write_pages(st["slab8"], st["slab"], st["src"], st["dst"])
        return _named(st["slab8"])
    B = st["q_abs"].shape[0]
    if op == "decode":
        w, s = case["window"], case["sink"]
        if "ws" not in st:   # planned and allocated once, as a serving program does
            st["split"] = k3mla.quant_split_tokens(B, st["max_ctx"], w, s)
            st["ws"] = torch.empty(k3mla.quant_decode_workspace_bytes(B, st["max_ctx"], w, s, st["split"]),
                                   dtype=torch.uint8, device="cuda")
        k3mla.quant_decode(st["q_abs"], st["slab8"], LAYER, st["table"], st["ctx"], st["w_kv_b"], SCALE_BITS, st["out"],
                           st["ws"], st["max_ctx"], w, s, st["split"])
        return st["out"]
    if "ws" not in st:
        st["split"] = k3mla.shared_split_tokens(B, case["groups"], st["max_shared"], st["max_own"])
        st["ws"] = torch.empty(k3mla.shared_decode_workspace_bytes(B, st["max_shared"], st["max_own"], *st["split"]),
                               dtype=torch.uint8, device="cuda")
    k3mla.shared_decode(st["q_abs"], st["slab"], LAYER, st["table"], st["ctx"], st["group_start"], st["shared_len"],
                        st["w_kv_b"], SCALE_BITS, st["out"], st["ws"], st["max_shared"], st["max_own"], *st["split"])
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
    slab8 = st["slab8"]
    page, line = st["table"][b, pos // PAGE].long(), pos % PAGE
    codes, scale, rope = _quantise(c, k)
    rows = slab8[..., : PAGE * ROW8].unflatten(-1, (PAGE, ROW8))
    rows[page, LAYER, line] = torch.cat([codes.view(torch.uint8), rope.view(torch.uint8)], -1)
    slab8[..., PAGE * ROW8:].view(torch.bfloat16)[page, LAYER, line] = scale
    return {"q": q.bfloat16(), **_named(slab8)}


def _values(slab8, page, layer):
    """f32 rows [..., 64, 576] of the listed pages."""
    codes, scale, rope = _parts(slab8[page, layer])
    return torch.cat([codes.float(), rope.float()], -1) * scale.float()[..., None]


def _pages(st):
    src, dst, slab, slab8 = st["src"].long(), st["dst"].long(), st["slab"], st["slab8"]
    if st["case"]["back"]:
        slab[dst] = _values(slab8, src, slice(None)).bfloat16()
        return slab
    x = slab[src].float()
    codes, scale, rope = _quantise(x[..., :LORA], x[..., LORA:])
    rows = torch.cat([codes.view(torch.uint8), rope.view(torch.uint8)], -1)
    slab8[dst] = torch.cat([rows.flatten(-2), scale.view(torch.uint8)], -1)
    return _named(slab8)


def _softmax(score, seen):
    score = (score * SCALE).masked_fill(~seen, float("-inf"))
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _expand(o, w_kv_b):
    w_uv = w_kv_b.view(H, NOPE + V, LORA)[:, NOPE:].float()
    return torch.matmul(o.transpose(0, 1), w_uv.transpose(1, 2)).transpose(0, 1).bfloat16()


def _decode(st):
    case, table = st["case"], st["table"].long()
    n, cols = st["ctx"].long()[:, None], st["table"].shape[1]
    if case["window"] >= st["max_ctx"]:
        pages = torch.arange(cols, device="cuda").expand(table.shape[0], cols)
    else:   # the sinks' pages, and the window's that are not among them
        few = min(cols, _count(case["sink"]))
        at = ((n - case["window"]).clamp(min=0) // PAGE).clamp(min=few)
        pages = torch.cat([torch.arange(few, device="cuda").expand(table.shape[0], few),
                           at + torch.arange(_count(case["window"]) + 1, device="cuda")], 1)
    page = table.gather(1, pages.clamp(max=cols - 1))
    rows = _values(st["slab8"], page.clamp(min=0), LAYER) * (page >= 0)[..., None, None]
    rows = rows.flatten(1, 2)                                                    # [B, T, 576]
    t = (pages[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)
    seen = (t < n) & ((t < case["sink"]) | (t >= n - case["window"])) & (t < cols * PAGE)
    rows = rows.masked_fill(~seen[..., None], 0.0)
    p = _softmax(torch.matmul(st["q_abs"].float(), rows.transpose(1, 2)), seen[:, None])
    return _expand(torch.matmul(p, rows[..., :LORA]), st["w_kv_b"])


def _shared(st):
    """Scores over the groups' shared pages (a batched product a group) and over every slot's own ones; one softmax of both."""
    table, slab, start = st["table"].long(), st["slab"], st["group_start"].long()
    B, cols = table.shape
    G, size = start.numel() - 1, st["case"]["size"]
    full = st["shared_len"].long() // PAGE                                        # whole pages
    q = st["q_abs"].float()
    slot = start[:-1, None] + torch.arange(size, device="cuda")                   # [G, size]
    member = slot < start[1:, None]
    slot = slot.clamp(max=B - 1)
    S = max(1, st["max_shared"] // PAGE)
    page = table[start[:-1], :S]
    there = torch.arange(page.shape[1], device="cuda") < full[:, None]
    rows = slab[page.clamp(min=0), LAYER].float() * (there & (page >= 0))[..., None, None]
    rows = rows.flatten(1, 2)                                                     # [G, S, 576]
    scores = torch.matmul(q[slot].flatten(1, 2), rows.transpose(1, 2)).unflatten(1, (size, H))
    b, i = slot[member], member.nonzero()
    shared = torch.full((B, H, rows.shape[1]), float("-inf"), device="cuda")
    shared[b] = scores[i[:, 0], i[:, 1]]
    seen = torch.zeros(B, rows.shape[1], dtype=torch.bool, device="cuda")
    seen[b] = there.repeat_interleave(PAGE, 1)[i[:, 0]]
    first = torch.zeros(B, dtype=torch.long, device="cuda")
    first[b] = full[i[:, 0]]
    at = first[:, None] + torch.arange(_count(st["max_own"]), device="cuda")
    page = table.gather(1, at.clamp(max=cols - 1))
    mine = slab[page.clamp(min=0), LAYER].float() * (page >= 0)[..., None, None]
    mine = mine.flatten(1, 2)                                                     # [B, T, 576]
    t = (at[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)
    score = torch.cat([shared, torch.matmul(q, mine.transpose(1, 2))], -1)
    p = _softmax(score, torch.cat([seen, t < st["ctx"][:, None]], 1)[:, None])
    common, rest = p.split([rows.shape[1], mine.shape[1]], -1)
    o = torch.matmul(rest, mine[..., :LORA])
    weights = torch.zeros(G, size, H, rows.shape[1], device="cuda")
    weights[i[:, 0], i[:, 1]] = common[b]
    o[b] += torch.matmul(weights.flatten(1, 2), rows[..., :LORA]).unflatten(1, (size, H))[i[:, 0], i[:, 1]]
    return _expand(o, st["w_kv_b"])


# ---- the definitions in 64 bits, slot by slot ----------------------------------------------------


def _exact_quantise(x):
    """[..., 576] -> codes, scales and rope entries as 64-bit values; a code is the nearest of e4m3's values, ties to even."""
    c, k = x[..., :LORA], x[..., LORA:]
    m, r = c.abs().amax(-1), k.abs().amax(-1)
    n = torch.where(m > 0, torch.ceil(torch.log2(m.clamp(min=1e-300) / 448)), 0.0)
    pow2 = lambda i: ((i.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    n = torch.where(m > 448 * pow2(n), n + 1, torch.where((m > 0) & (m <= 224 * pow2(n)), n - 1, n))
    n = torch.maximum(n, torch.where(r > 0, torch.frexp(r)[1].double(), torch.zeros_like(r)) - 120).clamp(-96, 120)
    scale = pow2(n)[..., None]
    y = c / scale
    step = pow2((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step, scale[..., 0], k / scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "pages":
        src, dst = st["src"].long(), st["dst"].long()
        if case["back"]:
            out = st["slab"].double()
            for s, d in zip(src.tolist(), dst.tolist()):
                codes, scale, rope = _parts(st["slab8"][s])
                out[d] = torch.cat([codes.double(), rope.double()], -1) * scale.double()[..., None]
            return out
        codes, scale, rope = (x.double() for x in _parts(st["slab8"]))
        for s, d in zip(src.tolist(), dst.tolist()):
            codes[d], scale[d], rope[d] = _exact_quantise(st["slab"][s].double())
        return {"codes": codes, "scale": scale, "rope": rope}
    if op == "rows":
        ctx, new = _lengths(case)
        table = st["table"].long()
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
        codes, scale, rope = (v.double() for v in _parts(st["slab8"]))
        page, line = table[slot, pos.long() // PAGE], pos.long() % PAGE
        for to, v in zip((codes, scale, rope), _exact_quantise(torch.cat([c, k], -1))):
            to[page, LAYER, line] = v
        return {"q": q, "codes": codes, "scale": scale, "rope": rope}
    table = st["table"].long()
    w, s = case.get("window", MOST), case.get("sink", 0)
    w_uv = st["w_kv_b"].double().view(H, NOPE + V, LORA)[:, NOPE:]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b, c in enumerate(st["ctx"].tolist()):
        if not c:
            continue
        t = torch.arange(c, device="cuda")
        t = t[(t < s) | (t >= c - w)]
        page, line = table[b, torch.div(t, PAGE, rounding_mode="floor")], t % PAGE
        if op == "decode":
            codes, scale, rope = _parts(st["slab8"][:, LAYER])
            bits = torch.cat([codes.view(torch.uint8)[page, line], rope.view(torch.uint8)[page, line]], -1)
            rows = torch.cat([bits[:, :LORA].contiguous().view(torch.float8_e4m3fn).double(),
                              bits[:, LORA:].contiguous().view(torch.bfloat16).double()], -1)
            rows = rows * scale[page, line].double()[:, None]
        else:
            rows = st["slab"][page, LAYER, line].double()
        p = (torch.einsum("hk,tk->ht", st["q_abs"][b].double(), rows) * SCALE).softmax(-1)
        out[b] = torch.einsum("hvk,hk->hv", w_uv, torch.einsum("ht,tk->hk", p, rows[:, :LORA]))
    return out
