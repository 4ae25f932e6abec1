"""The operators around the int4 projections of a decoder layer, as cases to be timed and compared.

Four operators stand between one int4 matrix product and the next when a model answers:

  extend     the step's new tokens get their places in a paged key-value cache: pages are taken
             from a free list (and given back by requests that ended), the block table grows,
             every token gets its slot and its position
  rope       the joined QKV projection's rows: bias, rotary positions, and the new keys and
             values written into the cache at their slots
  attention  one new token of each request over its pages of the cache
  norm       the projection's output added to the residual stream (normed before, gated and
             scaled where the model has that) and the next block's norm of the sum

`own` chooses who computes them: plain torch operations, or the library's calls.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # One step of a running batch: every request has one more token.
        dict(name="extend-decode-48", op="extend", batch=48, page=16, longest=8192, mode="decode", tight=False),
        # A step that mixes running requests, new prompts and ended requests, with too few pages for the last ones.
        dict(name="extend-mixed-1501", op="extend", batch=1501, page=16, longest=2048, mode="mixed", tight=True),
        # The smallest call: one request's QKV row, 40 query and 8 key-value heads (width 5120), bias, half layout.
        dict(name="rope-one-row", op="rope", rows=1, heads=40, kv_heads=8, dim=128, rot=128, layout="half", type="f16",
             cache="f16", page=16, bias=True, scaled=False, far=30000, pad=0),
        # A long prompt's chunk far into a scaled context, bf16.
        dict(name="rope-prompt-4099", op="rope", rows=4099, heads=40, kv_heads=8, dim=128, rot=128, layout="half",
             type="bf16", cache="bf16", page=16, bias=True, scaled=True, far=1000000, pad=0),
        # Prompts packed into a padded step, 32 query and 2 key-value heads (width 4096), half of each head turned
        # in neighbouring pairs, 8-bit cache.
        dict(name="rope-prompt-16384-e4m3", op="rope", rows=16384, heads=32, kv_heads=2, dim=128, rot=64,
             layout="pairs", type="f16", cache="e4m3", page=32, bias=True, scaled=False, far=131072, pad=301),
        # The smallest attention call: one request, about a thousand tokens.
        dict(name="attention-one-1000", op="attention", batch=1, longest=1000, heads=40, kv_heads=8, dim=128,
             type="f16", cache="f16", page=16, order="tokens", window=0, cap=0.0, empty=False),
        # A batch of requests of different ages, some of them not started.
        dict(name="attention-64-ragged", op="attention", batch=64, longest=8191, heads=40, kv_heads=8, dim=128,
             type="f16", cache="f16", page=16, order="tokens", window=0, cap=0.0, empty=True),
        # A larger batch over an 8-bit cache, 16 query heads to each key-value head.
        dict(name="attention-121-e4m3", op="attention", batch=121, longest=16001, heads=32, kv_heads=2, dim=128,
             type="f16", cache="e4m3", page=32, order="tokens", window=0, cap=0.0, empty=False),
        # Two very long documents: the work has to be split along the cache.
        dict(name="attention-2-long", op="attention", batch=2, longest=200003, heads=32, kv_heads=2, dim=128,
             type="bf16", cache="bf16", page=64, order="heads", window=0, cap=0.0, empty=False),
        # A layer with a window and capped scores, wide heads.
        dict(name="attention-24-window", op="attention", batch=24, longest=6000, heads=16, kv_heads=8, dim=256,
             type="bf16", cache="bf16", page=16, order="tokens", window=1024, cap=50.0, empty=False),
        # One token's row between two projections.
        dict(name="norm-one-row", op="norm", rows=1, width=5120, type="f16", stream="f16", post=False, gate="none",
             alpha=1.0),
        # A prompt's rows, residual stream in 32 bits, normed on both sides, with a gate for each channel.
        dict(name="norm-prompt-8192", op="norm", rows=8192, width=5120, type="bf16", stream="f32", post=True,
             gate="channel", alpha=0.7),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["extend", "rope", "attention", "attention", "norm"])
    if op == "extend":
        return dict(op=op, batch=log(1, 2048), page=rng.choice([1, 8, 16, 32, 48, 64]), longest=log(64, 8192),
                    mode=rng.choice(["decode", "mixed"]), tight=rng.random() < 0.3)
    heads, kv_heads, dim = rng.choice([(40, 8, 128), (32, 2, 128), (32, 8, 128), (16, 16, 64), (24, 8, 96),
                                       (14, 2, 64), (16, 8, 256), (32, 1, 128), (9, 3, 64), (20, 4, 80)])
    kind = rng.choice(["f16", "bf16"])
    cache = rng.choice([kind, kind, "e4m3"])
    if op == "rope":
        rows = log(1, 8192)
        return dict(op=op, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, rot=rng.choice([dim, dim // 2]),
                    layout=rng.choice(["half", "pairs"]), type=kind, cache=cache, page=rng.choice([1, 16, 24, 32, 64]),
                    bias=rng.random() < 0.5, scaled=rng.random() < 0.5, far=log(1000, 1000000),
                    pad=rng.randrange(rows // 8 + 1))
    if op == "norm":
        width = 8 * log(8, 2048)
        return dict(op=op, rows=log(1, max(1, min(16384, 8192 * 2560 // width))), width=width, type=kind,
                    stream=rng.choice([kind, "f32"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "full"]), alpha=rng.choice([1.0, 0.7, 0.25]))
    batch = log(1, 192)
    # At most 260 MB of 16-bit keys and values, so that the widest heads stay below the largest listed case.
    most = max(1, 65_000_000 // (batch * kv_heads * dim))
    return dict(op=op, batch=batch, longest=log(1, min(200000, most)), heads=heads, kv_heads=kv_heads, dim=dim,
                type=kind, cache=cache, page=rng.choice([1, 8, 16, 24, 32, 64, 128]),
                order=rng.choice(["tokens", "heads"]), window=rng.choice([0, 0, log(1, 4096)]),
                cap=rng.choice([0.0, 0.0, 30.0]), empty=rng.random() < 0.3)


# ------------------------------------------------------------------------------ sizes that follow from a case
def _lengths(c):
    """The requests' lengths, as a set that the case alone gives (prepare() orders it by the seed)."""
    r = random.Random("%d %d" % (c["batch"], c["longest"]))
    got = [r.randint(max(1, c["longest"] // 8), c["longest"]) for _ in range(c["batch"])]
    got[0] = c["longest"]
    if c.get("empty") and c["batch"] > 1:
        for i in range(1, c["batch"], 16):
            got[i] = 0
    return got


def _requests(c):
    """(length, new tokens) of each request of an extend case; -1 new tokens: the request has ended."""
    r = random.Random("extend %d %d %d" % (c["batch"], c["longest"], c["page"]))
    most = max(1, min(2048, 65536 // c["batch"] * 8))
    got = []
    for n in _lengths(dict(c, empty=False)):
        kind = r.random() if c["mode"] == "mixed" else 0.0
        if kind < 0.7:
            got.append((n, 1))                       # a running request
        elif kind < 0.8:
            got.append((n, -1))                      # one that has ended
        elif kind < 0.85:
            got.append((n, 0))                       # one that waits
        else:
            got.append((0 if kind < 0.95 else n, r.randint(1, most)))  # a prompt, or the next part of one
    total = 0
    for i, (n, new) in enumerate(got):  # the step's tokens are bounded
        if new > 1 and total + new > 65536 - c["batch"]:
            got[i] = (n, 1)
        total += max(0, got[i][1])
    return got


def _extend_sizes(c):
    page, reqs = c["page"], _requests(c)
    pages = lambda n: -(-n // page)  # noqa: E731
    used = sum(pages(n) for n, _ in reqs)
    given = sum(pages(n) for n, new in reqs if new < 0)
    need = sum(pages(n + new) - pages(n) for n, new in reqs if new > 0)
    tokens = sum(max(0, new) for _, new in reqs)
    width = pages(c["longest"] + 2048 + 1)
    free = max(0, need - given - need // 10) if c["tight"] else need + 64
    return dict(used=used, given=given, need=need, tokens=tokens, slots=-(-tokens // 64) * 64, width=width, free=free,
                pool=used + free)


def work(c):
    if c["op"] == "extend":
        z = _extend_sizes(c)
        # lengths, counts in; lengths, refusals out; pages given and taken; slots and positions out
        return {"bytes": 16 * c["batch"] + 8 * z["given"] + 8 * z["need"] + 12 * z["slots"], "flops": 4 * z["slots"]}
    if c["op"] == "rope":
        e, o, n = SIZE[c["type"]], SIZE[c["cache"]], c["rows"]
        q, kv = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
        read = n * (q + 2 * kv) * e + 12 * n + 2 * c["rot"] + (e * (q + 2 * kv) if c["bias"] else 0)
        return {"bytes": read + n * q * e + 2 * (n - c["pad"]) * kv * o, "flops": 3 * n * (c["heads"] + c["kv_heads"]) * c["rot"]}
    if c["op"] == "attention":
        seen = [min(n, c["window"]) if c["window"] else n for n in _lengths(c)]
        kv = 2 * c["kv_heads"] * c["dim"] * SIZE[c["cache"]]
        rest = c["batch"] * c["heads"] * (2 * c["dim"] * SIZE[c["type"]] + 4) + 4 * c["batch"]
        return {"bytes": sum(seen) * kv + 4 * sum(-(-n // c["page"]) for n in seen) + rest,
                "flops": 4 * c["heads"] * c["dim"] * sum(seen)}
    n, e, h = c["rows"] * c["width"], SIZE[c["type"]], SIZE[c["stream"]]
    small = c["width"] * e * (1 + c["post"] + (c["gate"] == "channel"))
    return {"bytes": n * (2 * e + 2 * h + (e if c["gate"] == "full" else 0)) + small, "flops": n * (10 + 4 * c["post"])}


# ------------------------------------------------------------------------------ the inputs
def prepare(c, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    r = random.Random(seed)
    s = {"extend": _prepare_extend, "rope": _prepare_rope, "attention": _prepare_attention, "norm": _prepare_norm}[c["op"]](c, g, r)
    s["case"] = c
    return s


def _normal(g, shape, kind, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float16)
    return (x * scale + shift if scale != 1.0 or shift else x).to(TYPES[kind])


def _ints(v, kind=torch.int32):
    return torch.tensor(v, dtype=kind, device=DEVICE)


def _shuffled(g, n):
    return torch.randperm(n, generator=g, device=DEVICE)


def _prepare_extend(c, g, r):
    z, reqs = _extend_sizes(c), _requests(c)
    r.shuffle(reqs)
    pages = _shuffled(g, z["pool"]).to(torch.int32)
    lens = _ints([n for n, _ in reqs])
    held = (lens + c["page"] - 1) // c["page"]
    at = (torch.cumsum(held, 0) - held)[:, None] + torch.arange(z["width"], device=DEVICE)
    mine = torch.arange(z["width"], device=DEVICE) < held[:, None]
    table = torch.where(mine, pages[at.clamp(max=z["pool"] - 1).long()], -1).to(torch.int32)
    free = torch.cat([pages[z["used"]:], torch.full((z["used"],), -1, dtype=torch.int32, device=DEVICE)])
    s = dict(lens=lens, new=_ints([n for _, n in reqs]), table=table, free=free, count=_ints([z["free"]]))
    s["slots"] = torch.empty(z["slots"], dtype=torch.int64, device=DEVICE)
    for name, n in (("positions", z["slots"]), ("refused", c["batch"]), ("lens_out", c["batch"]), ("count_out", 1)):
        s[name] = torch.empty(n, dtype=torch.int32, device=DEVICE)
    return s


def _pool(g, pages, c, kind):
    """One side of a cache in the case's order, seen as [pages, page, kv_heads, dim]."""
    inner = (c["kv_heads"], c["page"]) if c.get("order") == "heads" else (c["page"], c["kv_heads"])
    x = _normal(g, (pages, *inner, c["dim"]), kind, 40.0 if kind == "e4m3" else 1.0)
    return x.transpose(1, 2) if c.get("order") == "heads" else x


def _scales(g, c):
    return torch.rand(c["kv_heads"], generator=g, device=DEVICE) * 0.02 + 0.015 if c["cache"] == "e4m3" else None


def _prepare_rope(c, g, r):
    n, h, kv, d = c["rows"], c["heads"], c["kv_heads"], c["dim"]
    qkv = _normal(g, (n, h + 2 * kv, d), c["type"], 2.0)
    pages = -(-(n + n // 4 + 1) // c["page"])
    s = dict(qkv=qkv, q=qkv[:, :h], k=qkv[:, h:h + kv], v=qkv[:, h + kv:])
    s["bias"] = _normal(g, ((h + 2 * kv) * d,), c["type"], 0.5) if c["bias"] else None
    s["k_pool"], s["v_pool"] = _pool(g, pages, c, c["cache"]), _pool(g, pages, c, c["cache"])
    s["k_scale"], s["v_scale"] = _scales(g, c), _scales(g, c)
    slots = _shuffled(g, pages * c["page"])[:n]
    if c["pad"]:
        slots[n - c["pad"]:] = -1
    s["slots"] = slots
    start = r.randrange(max(1, c["far"] - n))
    s["positions"] = torch.arange(start, start + n, device=DEVICE, dtype=torch.int32)
    s["inv_freq"], s["mscale"] = _frequencies(c["rot"], c["scaled"])
    s["q_out"] = torch.empty((n, h, d), dtype=qkv.dtype, device=DEVICE)
    if own:
        import weight_only_int4_repack_gb300 as w4
        s["kv"] = w4.KVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
    return s


def _frequencies(rot, scaled, base=1000000.0, factor=4.0, window=32768):
    """Inverse frequencies; scaled: by `factor` where a turn is longer than the first context, left where it is
    much shorter, with a ramp between, and the rotated values drawn up as the scores get flatter."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = base ** (-i / rot)
    m = 1.0
    if scaled:
        turns = window * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        m = 0.1 * math.log(factor) + 1.0
    return f.to(torch.float32).to(DEVICE), m


def _prepare_attention(c, g, r):
    lens = _lengths(c)
    r.shuffle(lens)
    width = max(1, -(-c["longest"] // c["page"]))
    held = [-(-n // c["page"]) for n in lens]
    pages = sum(held) + 3
    order = _shuffled(g, pages).to(torch.int32)
    held = _ints(held)
    at = (torch.cumsum(held, 0) - held)[:, None] + torch.arange(width, device=DEVICE)
    table = torch.where(torch.arange(width, device=DEVICE) < held[:, None], order[at.clamp(max=pages - 1).long()], -1)
    s = dict(q=_normal(g, (c["batch"], c["heads"], c["dim"]), c["type"], 2.5), table=table.to(torch.int32), lens=_ints(lens))
    s["k_pool"], s["v_pool"] = _pool(g, pages, c, c["cache"]), _pool(g, pages, c, c["cache"])
    s["k_scale"], s["v_scale"] = _scales(g, c), _scales(g, c)
    s["scale"] = c["dim"] ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((c["batch"], c["heads"]), dtype=torch.float32, device=DEVICE)
    if own:
        import weight_only_int4_repack_gb300 as w4
        s["kv"] = w4.KVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        need = w4.w4a16_paged_attention_workspace_bytes(c["batch"], c["heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=DEVICE)
    return s


def _prepare_norm(c, g, r):
    n, k = c["rows"], c["width"]
    s = dict(h=_normal(g, (n, k), c["stream"], 3.0), y=_normal(g, (n, k), c["type"]), eps=1e-5)
    s["gamma"] = _normal(g, (k,), c["type"], 0.2, 1.0)
    s["post"] = _normal(g, (k,), c["type"], 0.2, 1.0) if c["post"] else None
    s["gate"] = None if c["gate"] == "none" else _normal(g, (k,) if c["gate"] == "channel" else (n, k), c["type"], 0.3, 0.5)
    s["h_out"] = torch.empty_like(s["h"])
    s["n_out"] = torch.empty_like(s["y"])
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"extend": _own_extend, "rope": _own_rope, "attention": _own_attention, "norm": _own_norm}[op](s)
    return {"extend": _plain_extend, "rope": _plain_rope, "attention": _plain_attention, "norm": _plain_norm}[op](s)


def _own_extend(s):
    import weight_only_int4_repack_gb300 as w4
    w4.w4a16_kv_extend(s["lens"], s["new"], s["table"], s["free"], s["count"], s["case"]["page"], s["slots"], s["positions"],
                       s["refused"], lens_out=s["lens_out"], count_out=s["count_out"])
    return {k: s[k] for k in ("table", "free", "count_out", "lens_out", "slots", "positions", "refused")}


def _own_rope(s):
    import weight_only_int4_repack_gb300 as w4
    w4.w4a16_rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["kv"], s["slots"],
                         interleaved=s["case"]["layout"] == "pairs", mscale=s["mscale"], bias=s["bias"], out=s["q_out"])
    return {"q": s["q_out"], "k": s["k_pool"], "v": s["v_pool"]}


def _own_attention(s):
    import weight_only_int4_repack_gb300 as w4
    w4.w4a16_paged_attention(s["q"], s["kv"], s["table"], s["lens"], scale=s["scale"], window=s["case"]["window"],
                             softcap=s["case"]["cap"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_norm(s):
    import weight_only_int4_repack_gb300 as w4
    w4.w4a16_residual_rmsnorm(s["h"], s["y"], s["gamma"], s["eps"], post_gamma=s["post"], gate=s["gate"],
                              alpha=s["case"]["alpha"], h_out=s["h_out"], n_out=s["n_out"])
    return {"h": s["h_out"], "n": s["n_out"]}


def _plain_extend(s):
    page, table, lens, new, free = s["case"]["page"], s["table"], s["lens"].long(), s["new"].long(), s["free"]
    width, slots = table.shape[1], s["slots"].numel()
    col = torch.arange(width, device=table.device)
    held = (lens + page - 1) // page
    # pages of ended requests go onto the list, in the order of the requests
    ended = new < 0
    give = torch.where(ended, held, 0)
    giving = col < give[:, None]
    to = s["count"].long() + (torch.cumsum(give, 0) - give)[:, None] + col
    listing = torch.cat([free, free.new_zeros(1)])
    listing = listing.index_put((torch.where(giving, to, free.numel()).reshape(-1),), table.reshape(-1))
    count = s["count"].long() + give.sum()
    # what each request asks for, and who gets it
    add = new.clamp(min=0)
    end = torch.cumsum(add, 0)
    fits = (lens + add <= width * page) & ((end <= slots) | (add == 0))
    need = torch.where(fits, (lens + add + page - 1) // page - held, 0).clamp(min=0)
    need = torch.where(ended, 0, need)
    upto = torch.cumsum(need, 0)
    got = fits & ((need == 0) | (upto <= count)) & ~ended
    take = torch.where(got, need, 0)
    taken = torch.where(got & (need > 0), upto, 0).amax()
    nth = (upto - need)[:, None] + col - held[:, None]
    mine = (col >= held[:, None]) & (col < (held + take)[:, None])
    table = torch.where(mine, listing[torch.where(mine, count - 1 - nth, 0)], table)
    # each token's slot
    tok = torch.arange(slots, device=table.device)
    req = torch.searchsorted(end, tok, right=True).clamp(max=len(lens) - 1)
    real = (tok < end[-1]) & got[req]
    pos = torch.where(real, lens[req] + tok - (end - add)[req], 0)
    slot = torch.where(real, table[req, pos // page].long() * page + pos % page, -1)
    lens_out = torch.where(ended, 0, lens + torch.where(got, add, 0))
    refused = torch.where(ended | got, 0, torch.where(fits, 1, 2))
    return {"table": table, "free": listing[:-1], "count_out": (count - taken).reshape(1).int(), "lens_out": lens_out.int(),
            "slots": slot, "positions": pos.int(), "refused": refused.int()}


def _turn(x, cos, sin, rot, pairs):
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if pairs else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if pairs else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    c = s["case"]
    h, kv = c["heads"], c["kv_heads"]
    x = s["qkv"].float()
    if s["bias"] is not None:
        x = x + s["bias"].float().view(h + 2 * kv, c["dim"])
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos = (angle.cos() * s["mscale"]).float()[:, None]
    sin = (angle.sin() * s["mscale"]).float()[:, None]
    qk = _turn(x[:, :h + kv], cos, sin, c["rot"], c["layout"] == "pairs")
    keep = s["slots"] >= 0
    slots = s["slots"][keep]
    for pool, scale, new in ((s["k_pool"], s["k_scale"], qk[:, h:]), (s["v_pool"], s["v_scale"], x[:, h + kv:])):
        new = new[keep]
        if scale is not None:
            new = (new / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        new = new.to(pool.dtype)
        if pool.dtype == torch.float8_e4m3fn:
            pool, new = pool.view(torch.uint8), new.view(torch.uint8)
        pool[slots // c["page"], slots % c["page"]] = new
    return {"q": qk[:, :h].to(s["qkv"].dtype), "k": s["k_pool"], "v": s["v_pool"]}


def _gathered(pool, scale, table):
    """[batch, tokens, kv_heads, dim] in 32 bits of a cache's pages."""
    at = table.long().clamp(min=0)
    x = pool.view(torch.uint8)[at].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[at]
    x = x.float() if scale is None else x.float() * scale[:, None]
    return x.flatten(1, 2)


def _plain_attention(s):
    c = s["case"]
    b, kv, d = c["batch"], c["kv_heads"], c["dim"]
    k, v = _gathered(s["k_pool"], s["k_scale"], s["table"]), _gathered(s["v_pool"], s["v_scale"], s["table"])
    q = s["q"].float().view(b, kv, c["heads"] // kv, d)
    score = torch.einsum("bhgd,blhd->bhgl", q, k) * s["scale"]
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    at, lens = torch.arange(k.shape[1], device=k.device), s["lens"][:, None]
    seen = at < lens
    if c["window"]:
        seen = seen & (at >= lens - c["window"])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.einsum("bhgl,blhd->bhgd", p, v.masked_fill(~seen[:, :, None, None], 0.0))
    out = torch.where(total > 0, out / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    return {"out": out.to(s["q"].dtype).view(b, c["heads"], d), "lse": lse.view(b, c["heads"])}


def _plain_norm(s):
    y = s["y"].float()
    if s["post"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s["post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["h"].float() + s["case"]["alpha"] * y
    n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["gamma"].float()
    return {"h": h.to(s["h"].dtype), "n": n.to(s["y"].dtype)}


# ------------------------------------------------------------------------------ from the definition, in 64 bits
def exact(c, seed):
    if c["op"] == "extend":
        return None  # whole numbers
    s = prepare(c, seed)
    return {"rope": _exact_rope, "attention": _exact_attention, "norm": _exact_norm}[c["op"]](c, s)


def _exact_rope(c, s):
    h, kv, d, rot = c["heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qkv"].double()
    if s["bias"] is not None:
        x += s["bias"].double().reshape(1, h + 2 * kv, d)
    first = torch.arange(0, rot, 2, device=x.device) if c["layout"] == "pairs" else torch.arange(rot // 2, device=x.device)
    second = first + (1 if c["layout"] == "pairs" else rot // 2)
    z = torch.polar(torch.full((1,), s["mscale"], dtype=torch.float64, device=x.device),
                    torch.outer(s["positions"].double(), s["inv_freq"].double()))
    out = x.clone()
    turned = torch.complex(x[:, :h + kv].index_select(2, first), x[:, :h + kv].index_select(2, second)) * z[:, None, :]
    out[:, :h + kv, first], out[:, :h + kv, second] = turned.real, turned.imag
    pools = []
    for name, lo in (("k", h), ("v", h + kv)):
        pool = s[name + "_pool"].to(torch.float32).double().reshape(-1, kv, d).clone()
        new = out[:, lo:lo + kv]
        if s[name + "_scale"] is not None:
            new = (new / s[name + "_scale"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        real = s["slots"] >= 0
        pool[s["slots"][real]] = new[real]
        pools.append(pool.reshape(s[name + "_pool"].shape))
    return {"q": out[:, :h], "k": pools[0], "v": pools[1]}


def _exact_attention(c, s):
    kv, group, page = c["kv_heads"], c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
    for i, n in enumerate(s["lens"].tolist()):
        low = max(0, n - c["window"]) if c["window"] else 0
        if n <= low:
            continue
        pages = s["table"][i, :-(-n // page)].long()
        side = []
        for name in ("k", "v"):
            pool, scale = s[name + "_pool"], s[name + "_scale"]
            x = pool.view(torch.uint8)[pages].view(pool.dtype).float() if c["cache"] == "e4m3" else pool[pages]
            x = x.reshape(-1, kv, c["dim"])[low:n].double()
            side.append(x if scale is None else x * scale.double()[None, :, None])
        for j in range(kv):
            rows = slice(j * group, (j + 1) * group)
            t = (s["q"][i, rows].double() @ side[0][:, j].T) * s["scale"]
            if c["cap"]:
                t = c["cap"] * torch.tanh(t / c["cap"])
            lse[i, rows] = torch.logsumexp(t, -1)
            out[i, rows] = torch.exp(t - lse[i, rows][:, None]) @ side[1][:, j]
    return {"out": out, "lse": lse}


def _exact_norm(c, s):
    def unit(x):
        return x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"])

    y = s["y"].double()
    if s["post"] is not None:
        y = unit(y) * s["post"].double()
    if s["gate"] is not None:
        y = y * s["gate"].double()
    h = s["h"].double() + c["alpha"] * y
    return {"h": h, "n": unit(h) * s["gamma"].double()}
