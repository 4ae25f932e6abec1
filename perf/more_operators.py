"""Attention of many query rows over a paged cache, and the choice of the next token, as cases to be timed and compared.

Three operators that a server of a decoder with int4 projections runs beside those of perf/operators.py:

  prompt    attention of several new tokens of each request (prompts, parts of prompts, drafts) over its pages and,
            where the request has one, a prefix that it shares with others
  prefix    one new token of each request of a batch whose requests share long prefixes: what the requests of a
            prefix see of it is computed once for all, and joined with their own tokens
  sample    the next token of each request from its logits: temperature, top-k, top-p, min-p, given random numbers

`own` chooses who computes them: plain torch operations, or the library's calls.
"""
import math
import random

import torch

own = False

DEVICE = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # The smallest call: one request checks a draft of 5 tokens behind a short context.
        dict(name="prompt-draft-5", op="prompt", batch=1, tokens=5, before=400, heads=40, kv_heads=8, dim=128, type="f16",
             cache="f16", page=16, order="tokens", window=0, cap=0.0, prefixes=0, shared=0, pad=0),
        # One long prompt from its first token on.
        dict(name="prompt-4099", op="prompt", batch=1, tokens=4099, before=0, heads=40, kv_heads=8, dim=128, type="bf16",
             cache="bf16", page=16, order="tokens", window=0, cap=0.0, prefixes=0, shared=0, pad=0),
        # A step that packs prompts of very different lengths, later parts of long ones among them, behind two shared
        # prefixes; 8-bit cache, 16 query heads to each key-value head, padded rows at the end.
        dict(name="prompt-13-packed", op="prompt", batch=13, tokens=1400, before=6000, heads=32, kv_heads=2, dim=128,
             type="f16", cache="e4m3", page=32, order="tokens", window=0, cap=0.0, prefixes=2, shared=1000, pad=37),
        # A layer with a window and capped scores, wide heads.
        dict(name="prompt-window", op="prompt", batch=4, tokens=1700, before=900, heads=16, kv_heads=8, dim=256, type="bf16",
             cache="bf16", page=16, order="heads", window=1024, cap=50.0, prefixes=0, shared=0, pad=0),
        # A few answers to one question: a small batch behind a prompt of ordinary length.
        dict(name="prefix-8", op="prefix", batch=8, longest=120, shared=2000, prefixes=1, none=0, heads=40, kv_heads=8,
             dim=128, type="f16", cache="f16", page=16, order="tokens", window=0, cap=0.0),
        # A batch behind one long system prompt.
        dict(name="prefix-64", op="prefix", batch=64, longest=1000, shared=16001, prefixes=1, none=0, heads=40, kv_heads=8,
             dim=128, type="f16", cache="f16", page=16, order="tokens", window=0, cap=0.0),
        # A large batch behind several documents, some requests behind none; 8-bit cache.
        dict(name="prefix-301-e4m3", op="prefix", batch=301, longest=700, shared=20000, prefixes=5, none=23, heads=32,
             kv_heads=2, dim=128, type="bf16", cache="e4m3", page=32, order="tokens", window=0, cap=0.0),
        # Small heads, many of them, pages heads first.
        dict(name="prefix-37-heads", op="prefix", batch=37, longest=300, shared=6007, prefixes=2, none=0, heads=16,
             kv_heads=16, dim=64, type="bf16", cache="bf16", page=24, order="heads", window=0, cap=0.0),
        # One request's next token.
        dict(name="sample-one", op="sample", rows=1, vocab=32001, type="f16", params="one", banned=0.0),
        # A batch in which every request has its own settings.
        dict(name="sample-64", op="sample", rows=64, vocab=131072, type="f16", params="mixed", banned=0.01),
        # A large batch and vocabulary, nucleus only, no top-k that would make it small.
        dict(name="sample-256-nucleus", op="sample", rows=256, vocab=150001, type="bf16", params="nucleus", banned=0.0),
        # Logits in 32 bits, most tokens excluded by a grammar.
        dict(name="sample-17-grammar", op="sample", rows=17, vocab=50257, type="f32", params="mixed", banned=0.9),
    ]


HEADS = [(40, 8, 128), (32, 2, 128), (32, 8, 128), (16, 16, 64), (12, 4, 96), (14, 2, 64), (16, 8, 256), (32, 1, 128),
         (9, 3, 64), (20, 4, 80)]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["prompt", "prefix", "sample"])
    if op == "sample":
        vocab = log(1000, 160000)
        return dict(op=op, rows=log(1, min(320, 256 * 150001 // vocab)), vocab=vocab, type=rng.choice(["f16", "bf16", "f32"]),
                    params=rng.choice(["mixed", "mixed", "nucleus", "plain"]), banned=rng.choice([0.0, 0.0, 0.01, 0.9]))
    heads, kv_heads, dim = rng.choice(HEADS)
    kind = rng.choice(["f16", "bf16"])
    c = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, type=kind, cache=rng.choice([kind, kind, "e4m3"]),
             page=rng.choice([1, 8, 16, 24, 32, 64, 128]), order=rng.choice(["tokens", "heads"]),
             window=rng.choice([0, 0, 0, log(16, 4096)]), cap=rng.choice([0.0, 0.0, 0.0, 30.0]))
    if op == "prompt":
        c["batch"] = log(1, 24)
        # Below the pairs of a query and a key that the largest listed cases have, fewer where heads are many and wide.
        c["tokens"] = log(1, min(3000, max(1, 12000 // c["batch"])))
        most = max(1, 25_000_000 * 5120 // (heads * dim * c["batch"] * c["tokens"] * 2))
        c["before"] = log(1, min(20000, most)) if rng.random() < 0.7 else 0
        c["prefixes"] = rng.choice([0, 0, 1, 2])
        c["shared"] = log(1, min(8000, most)) if c["prefixes"] else 0
        c["pad"] = rng.choice([0, 0, rng.randrange(1, 100)])
        return c
    c["batch"] = log(1, 320)
    c["prefixes"] = rng.choice([1, 1, 2, 5])
    c["none"] = rng.choice([0, 0, min(c["batch"] // 4, 20)])
    # At most 65 million elements of keys, in the prefixes and in the requests' own pages.
    c["shared"] = log(16, min(20000, 65_000_000 // (c["prefixes"] * kv_heads * dim)))
    c["longest"] = log(1, min(1500, max(1, 65_000_000 // (c["batch"] * kv_heads * dim))))
    return c


# ------------------------------------------------------------------------------ sizes that follow from a case
def _requests(c):
    """(new tokens, tokens before them) of each request of a prompt case, as a set that the case alone gives."""
    r = random.Random("prompt %d %d %d" % (c["batch"], c["tokens"], c["before"]))
    got = []
    for _ in range(c["batch"]):
        n = max(1, int(c["tokens"] * math.exp(r.uniform(-4.0, 0.0))))  # most are short, some are long
        got.append((n, r.randint(0, c["before"]) if r.random() < 0.7 else 0))
    got[0] = (c["tokens"], c["before"])
    return got


def _owned(c):
    """Own lengths of a prefix case's requests, the new token counted."""
    r = random.Random("own %d %d" % (c["batch"], c["longest"]))
    return [c["longest"]] + [r.randint(1, c["longest"]) for _ in range(c["batch"] - 1)]


def _prefixes(c):
    """Lengths of the shared prefixes, and the prefix of each request (-1: none)."""
    r = random.Random("shared %d %d %d" % (c["batch"], c["shared"], c["prefixes"]))
    if not c["prefixes"]:
        return [], [-1] * c["batch"]
    lens = [c["shared"]] + [r.randint(max(1, c["shared"] // 4), c["shared"]) for _ in range(c["prefixes"] - 1)]
    none = c["none"] if c["op"] == "prefix" else c["batch"] // 3
    return lens, [-1 if i < none else i % c["prefixes"] for i in range(c["batch"])]


def _pairs(c):
    """Visible (query, key) pairs of a case, and the tokens whose keys and values are read once at least."""
    lens, of = _prefixes(c)
    w = c["window"] or 1 << 60
    pairs, tokens, seen = 0, 0, [0] * len(lens)  # of a prefix: its tokens that some request sees
    if c["op"] == "prompt":
        for (n, before), p in zip(_requests(c), of):
            first = (lens[p] if p >= 0 else 0) + before  # tokens in front of the first new one
            whole = min(n, max(0, w - first))       # rows that see all in front of them
            pairs += whole * first + whole * (whole + 1) // 2 + (n - whole) * w
            reach = min(first + n, w + n - 1)       # tokens that some row sees
            tokens += min(reach, before + n)
            if p >= 0:
                seen[p] = max(seen[p], reach - (before + n))
    else:
        for n, p in zip(_owned(c), of):
            tokens += min(n, w)
            mine = max(0, min(lens[p], w - n)) if p >= 0 else 0
            pairs += min(n, w) + mine
            if p >= 0:
                seen[p] = max(seen[p], mine)
    return pairs, tokens + sum(max(0, x) for x in seen)


def work(c):
    if c["op"] == "sample":
        n = c["rows"] * c["vocab"]
        # the logits, settings and random numbers in, tokens out; a difference, a product, an exponential and a sum each
        return {"bytes": n * SIZE[c["type"]] + 32 * c["rows"], "flops": 4 * n}
    pairs, tokens = _pairs(c)
    rows = sum(n for n, _ in _requests(c)) if c["op"] == "prompt" else c["batch"]
    kv = 2 * c["kv_heads"] * c["dim"] * SIZE[c["cache"]]
    rest = rows * c["heads"] * (2 * c["dim"] * SIZE[c["type"]] + 4) + 4 * tokens // c["page"]
    return {"bytes": tokens * kv + rest, "flops": 4 * c["heads"] * c["dim"] * pairs}


# ------------------------------------------------------------------------------ the inputs
def prepare(c, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    r = random.Random(seed)
    s = _prepare_sample(c, g, r) if c["op"] == "sample" else _prepare_attention(c, g, r)
    s["case"] = c
    return s


def _normal(g, shape, kind, scale=1.0):
    x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float16)
    return (x * scale if scale != 1.0 else x).to(TYPES[kind])


def _ints(v, kind=torch.int32):
    return torch.tensor(v, dtype=kind, device=DEVICE)


def _pool(g, pages, c):
    """One side of a cache in the case's order, seen as [pages, page, kv_heads, dim]."""
    inner = (c["kv_heads"], c["page"]) if c["order"] == "heads" else (c["page"], c["kv_heads"])
    x = _normal(g, (pages, *inner, c["dim"]), c["cache"], 40.0 if c["cache"] == "e4m3" else 1.0)
    return x.transpose(1, 2) if c["order"] == "heads" else x


def _table(order, at, lens, page):
    """A block table for these lengths, its pages taken from `order` from entry `at` on."""
    width = max(1, max(-(-n // page) for n in lens))
    held = _ints([-(-n // page) for n in lens])
    place = (torch.cumsum(held, 0) - held)[:, None] + torch.arange(width, device=DEVICE) + at
    mine = torch.arange(width, device=DEVICE) < held[:, None]
    return torch.where(mine, order[place.clamp(max=order.numel() - 1).long()], -1).to(torch.int32), at + int(held.sum())


def _prepare_attention(c, g, r):
    shared, of = _prefixes(c)
    mix = list(range(c["batch"]))
    r.shuffle(mix)
    of = [of[i] for i in mix]
    if c["op"] == "prompt":
        reqs = [_requests(c)[i] for i in mix]
        new = [n for n, _ in reqs]
        lens = [n + before for n, before in reqs]
        rows = sum(new) + c["pad"]
    else:
        lens, rows = [_owned(c)[i] for i in mix], c["batch"]
    pages = sum(-(-n // c["page"]) for n in lens + shared) + 3
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    s = dict(q=_normal(g, (rows, c["heads"], c["dim"]), c["type"], 2.5), lens=_ints(lens), scale=c["dim"] ** -0.5)
    s["table"], at = _table(order, 0, lens, c["page"])
    if shared:
        s["prefix_table"], _ = _table(order, at, shared, c["page"])
        s["prefix_lens"], s["prefix_of"] = _ints(shared), _ints(of)
    else:
        s["prefix_table"] = s["prefix_lens"] = s["prefix_of"] = None
    if c["op"] == "prompt":
        s["starts"] = _ints([sum(new[:i]) for i in range(len(new) + 1)])
    s["k_pool"], s["v_pool"] = _pool(g, pages, c), _pool(g, pages, c)
    for name in ("k_scale", "v_scale"):
        s[name] = torch.rand(c["kv_heads"], generator=g, device=DEVICE) * 0.02 + 0.015 if c["cache"] == "e4m3" else None
    s["out"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros((rows, c["heads"]), dtype=torch.float32, device=DEVICE)
    # What the host knows of the step, as a program has that packs it.
    s["host"] = dict(lens=lens, shared=shared, of=of, new=new if c["op"] == "prompt" else [1] * len(lens))
    if own:
        import weight_only_int4_repack_gb300 as w4
        s["kv"] = w4.KVCache(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        if c["op"] == "prompt":
            need = w4.w4a16_prompt_attention_workspace_bytes(rows, c["heads"], c["kv_heads"], c["dim"])
        else:
            need = w4.w4a16_prefix_attention_workspace_bytes(rows, c["heads"], c["kv_heads"], c["dim"])
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=DEVICE)
    return s


SETTINGS = {
    # temperature, top-k, top-p, min-p: 0, 0, 1 and 0 leave a request alone (temperature 0: the largest logit)
    "one": [(0.8, 50, 0.95, 0.0)],
    "mixed": [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.7, 40, 0.95, 0.0), (1.0, 0, 0.9, 0.0), (1.3, 0, 1.0, 0.05),
              (0.6, 1000, 0.8, 0.02), (1.0, 1, 1.0, 0.0), (0.9, 200, 1.0, 0.0), (1.5, 20, 0.5, 0.1), (0.3, 0, 0.99, 0.0)],
    "nucleus": [(1.0, 0, 0.95, 0.0), (0.8, 0, 0.9, 0.0), (1.2, 0, 0.8, 0.0)],
    "plain": [(1.0, 0, 1.0, 0.0), (0.7, 0, 1.0, 0.0)],
}


def _prepare_sample(c, g, r):
    n, vocab = c["rows"], c["vocab"]
    # A broad floor, and a few hundred tokens that stand out of it, by more in some rows than in others.
    x = torch.randn((n, vocab), generator=g, device=DEVICE, dtype=torch.float16).float() * 2.0
    high = torch.randint(0, vocab, (n, 300), generator=g, device=DEVICE)
    sharp = torch.rand((n, 1), generator=g, device=DEVICE) * 4.0 + 2.0
    x.scatter_add_(1, high, torch.rand((n, 300), generator=g, device=DEVICE).square() * sharp * 2.0)
    if c["banned"]:
        x.masked_fill_(torch.rand((n, vocab), generator=g, device=DEVICE) < c["banned"], -math.inf)
    picks = [SETTINGS[c["params"]][i % len(SETTINGS[c["params"]])] for i in range(n)]
    r.shuffle(picks)
    s = dict(logits=x.to(TYPES[c["type"]]), uniform=torch.rand(n, generator=g, device=DEVICE))
    for i, (name, kind) in enumerate((("temperature", torch.float32), ("top_k", torch.int32), ("top_p", torch.float32),
                                      ("min_p", torch.float32))):
        s[name] = _ints([p[i] for p in picks], kind)
    s["out"] = torch.zeros(n, dtype=torch.int64, device=DEVICE)
    return s


# ------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "prefix": _own_prefix, "sample": _own_sample}[op](s)
    return {"prompt": _plain_attention, "prefix": _plain_attention, "sample": _plain_sample}[op](s)


def _own_prompt(s):
    import weight_only_int4_repack_gb300 as w4
    w4.w4a16_prompt_attention(s["q"], s["kv"], s["table"], s["starts"], s["lens"], scale=s["scale"],
                              window=s["case"]["window"], softcap=s["case"]["cap"], prefix_table=s["prefix_table"],
                              prefix_lens=s["prefix_lens"], prefix_of=s["prefix_of"], out=s["out"], lse=s["lse"],
                              workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_prefix(s):
    import weight_only_int4_repack_gb300 as w4
    w4.w4a16_prefix_attention(s["q"], s["kv"], s["table"], s["lens"], s["prefix_table"], s["prefix_lens"], s["prefix_of"],
                              scale=s["scale"], window=s["case"]["window"], softcap=s["case"]["cap"], out=s["out"],
                              lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_sample(s):
    import weight_only_int4_repack_gb300 as w4
    return w4.w4a16_sample(s["logits"], s["uniform"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], out=s["out"])


def _gathered(pool, scale, pages):
    """[tokens, kv_heads, dim] in 32 bits of a list of pages."""
    x = pool.view(torch.uint8)[pages].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[pages]
    x = x.float() if scale is None else x.float() * scale[:, None]
    return x.flatten(0, 1)


def _part(s, q, k, v, first, lo):
    """Sums over some of the keys: q [n, kv, group, dim], k, v [m, kv, dim]; row i sees keys lo[i] <= j < first[i].
    Returns the maximum, the sum of the weights and the weighted sum of the values."""
    c = s["case"]
    score = torch.einsum("nhgd,mhd->hgnm", q, k) * s["scale"]
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    at = torch.arange(k.shape[0], device=k.device)
    score = score.masked_fill((at >= first[:, None]) | (at < lo[:, None]), -math.inf)
    top = score.amax(-1) if k.shape[0] else score.new_full(score.shape[:3], -math.inf)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top)[..., None])
    return top, p.sum(-1), torch.einsum("hgnm,mhd->hgnd", p, v)


def _joined(a, b):
    top = torch.maximum(a[0], b[0])
    base = torch.where(top == -math.inf, 0.0, top)
    x, y = torch.exp(a[0] - base), torch.exp(b[0] - base)
    return top, a[1] * x + b[1] * y, a[2] * x[..., None] + b[2] * y[..., None]


def _plain_attention(s):
    """Request after request over its own tokens; a prefix once for all rows that are behind it."""
    c, host = s["case"], s["host"]
    kv, group, page = c["kv_heads"], c["heads"] // c["kv_heads"], c["page"]
    q = s["q"].float().unflatten(1, (kv, group))
    window = c["window"] or 1 << 30
    starts = [sum(host["new"][:i]) for i in range(len(host["new"]) + 1)]
    rows = starts[-1]
    top = q.new_full((kv, group, rows), -math.inf)
    total, out = torch.zeros_like(top), q.new_zeros((kv, group, rows, c["dim"]))
    place = torch.zeros(rows, dtype=torch.int64, device=q.device)  # each row's position among its own tokens
    for b, n in enumerate(host["lens"]):
        at = slice(starts[b], starts[b + 1])
        pages = s["table"][b, :-(-n // page)].long()
        pos = torch.arange(n - host["new"][b], n, device=q.device)
        place[at] = pos
        k, v = (_gathered(s[x + "_pool"], s[x + "_scale"], pages)[:n] for x in ("k", "v"))
        top[:, :, at], total[:, :, at], out[:, :, at] = _part(s, q[at], k, v, pos + 1, pos + 1 - window)
    for p, n in enumerate(host["shared"]):
        mine = [i for b, x in enumerate(host["of"]) if x == p for i in range(starts[b], starts[b + 1])]
        if not mine:
            continue
        at = torch.tensor(mine, device=q.device)
        pages = s["prefix_table"][p, :-(-n // page)].long()
        k, v = (_gathered(s[x + "_pool"], s[x + "_scale"], pages)[:n] for x in ("k", "v"))
        got = _part(s, q[at], k, v, torch.full_like(at, n), place[at] + n + 1 - window)
        top[:, :, at], total[:, :, at], out[:, :, at] = _joined((top[:, :, at], total[:, :, at], out[:, :, at]), got)
    some = total > 0
    out = torch.where(some[..., None], out / total[..., None], 0.0)
    lse = torch.where(some, top + torch.log(total), -math.inf)
    s["out"][:rows] = out.permute(2, 0, 1, 3).flatten(1, 2).to(s["out"].dtype)
    s["lse"][:rows] = lse.permute(2, 0, 1).flatten(1, 2)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_sample(s):
    x = s["logits"].double()
    vocab = x.shape[1]
    order = torch.arange(vocab, device=x.device)
    most = x.amax(1, keepdim=True)
    greedy = torch.where(x == most, order, vocab).amin(1)
    heat = s["temperature"].double()[:, None]
    by, index = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((by - most) / torch.where(heat > 0, heat, 1.0))
    k = torch.where(s["top_k"] > 0, s["top_k"], vocab)[:, None]
    kept = order < k
    w = torch.where(kept, w, 0.0)
    upto = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
    top_p = s["top_p"].double()[:, None]
    kept = kept & ((top_p >= 1) | (before < top_p * upto[:, -1:]) | (order == 0)) & (w >= s["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, index, torch.where(kept, w, 0.0))  # in the order of the tokens again
    upto = torch.cumsum(w, 1)
    drawn = (upto <= s["uniform"].double()[:, None] * upto[:, -1:]).sum(1).clamp(max=vocab - 1)
    return torch.where(heat[:, 0] > 0, drawn, greedy)


# ------------------------------------------------------------------------------ from the definition, in 64 bits
def exact(c, seed):
    if c["op"] == "sample":
        return None  # whole numbers
    s = prepare(c, seed)
    host, kv, group, page = s["host"], c["kv_heads"], c["heads"] // c["kv_heads"], c["page"]
    out, lse = s["out"].double(), s["lse"].double()
    row = 0
    for b, own_len in enumerate(host["lens"]):
        n, p = host["new"][b], host["of"][b]
        lists = [(s["table"][b], own_len)]
        if p >= 0:
            lists.insert(0, (s["prefix_table"][p], host["shared"][p]))
        side = {}
        for name in ("k", "v"):
            got = []
            for table, length in lists:
                pool, pages = s[name + "_pool"], table[:(length + page - 1) // page].long()
                x = pool.view(torch.uint8)[pages].view(pool.dtype).float() if c["cache"] == "e4m3" else pool[pages]
                got.append(x.reshape(-1, kv, c["dim"])[:length].double())
            side[name] = torch.cat(got)
            if s[name + "_scale"] is not None:
                side[name] *= s[name + "_scale"].double()[None, :, None]
        seen = side["k"].shape[0]
        for i in range(0, n, 512):  # some rows at a time
            m = min(512, n - i)
            last = torch.arange(seen - n + i, seen - n + i + m, device=out.device)[:, None]
            j = torch.arange(seen, device=out.device)[None]
            hidden = j > last
            if c["window"]:
                hidden |= j <= last - c["window"]
            for h in range(c["heads"]):
                t = (s["q"][row + i:row + i + m, h].double() @ side["k"][:, h // group].T) * s["scale"]
                if c["cap"]:
                    t = c["cap"] * torch.tanh(t / c["cap"])
                t[hidden] = -math.inf
                lse[row + i:row + i + m, h] = torch.logsumexp(t, 1)
                out[row + i:row + i + m, h] = torch.softmax(t, 1) @ side["v"][:, h // group]
        row += n
    return {"out": out, "lse": lse}
