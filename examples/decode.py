"""A decoder with int4 weights, answering: every operator of the library in the order in which a step runs them.

    python examples/decode.py                      # a small model, random weights
    python examples/decode.py --width 5120 --heads 40 --kv-heads 8 --ffn 13824 --layers 4 --batch 8
    python examples/decode.py --prefix 64 --prompt 100 --temperature 0.8 --top-p 0.95

A step takes one token of each request: its place in the paged cache (kv_extend), then for each layer the QKV
projection, rotary positions and the cache (rope_append), attention over the cache's pages (paged_attention), the
output projection, the residual stream and the next norm (residual_rmsnorm), the SwiGLU and down projections, and
again residual stream and norm. Nothing in it allocates or waits for the GPU, so the whole step is captured into one
CUDA graph and replayed; requests grow, end and start anew inside the graph, because lengths, block table and free
list live on the GPU.

Prompts come in by the same layers, all their tokens at once (prompt_attention). What many requests begin with can be
kept once, as a prefix that they share: their own tokens stand behind it, and a step computes what they see of it for
all of them together (prefix_attention). The next token is the likeliest one or, with a temperature, drawn (sample).
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int4_repack_gb300 as w4  # noqa: E402

GROUP, PAGE, EPS = 128, 16, 1e-5


def int4_weight(n: int, k: int, generator):
    """Random packed weights of an n x k projection, scaled to keep a row's variance: (repacked, scales, zero points)."""
    q = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=generator)
    scales = (torch.rand(n, k // GROUP, device="cuda", generator=generator) * 0.4 + 0.8) * (0.2 / k**0.5)
    zp = torch.randint(0x66, 0x9A, (n, (k // GROUP + 1) // 2), dtype=torch.uint8, device="cuda", generator=generator)
    return q, scales.half(), zp


class Decoder:
    """Weights, cache and buffers of a decoder, and step()."""

    def __init__(self, width=1024, heads=8, kv_heads=2, dim=128, ffn=2048, layers=2, vocab=4096, batch=8, context=512,
                 pages=None, cache=torch.float16, seed=0, prefixes=0, prefix_context=0, sampling=None):
        """prefixes, prefix_context: how many prefixes can be shared, of how many tokens at most. sampling: temperature,
        top_k, top_p, min_p (numbers) of the next tokens; None takes the likeliest."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.batch, self.max_pages = heads, kv_heads, dim, batch, -(-context // PAGE)
        pages = pages or batch * self.max_pages
        prefix_pages = -(-prefix_context // PAGE)
        new = lambda *s, dtype=torch.float16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        qkv = (heads + 2 * kv_heads) * dim
        self.raw = [dict(qkv=int4_weight(qkv, width, g), o=int4_weight(width, heads * dim, g), gate=int4_weight(ffn, width, g),
                         up=int4_weight(ffn, width, g), down=int4_weight(width, ffn, g)) for _ in range(layers)]
        self.raw_head = int4_weight(vocab, width, g)
        ready = lambda w: (w4.w4a16_repack(w[0]), w[1], w[2])  # noqa: E731
        self.layers = [{n: ready(w) for n, w in layer.items()} for layer in self.raw]
        self.head = ready(self.raw_head)
        norm = lambda: (1 + 0.1 * torch.randn(width, device="cuda", generator=g)).half()  # noqa: E731
        for layer in self.layers:
            layer["norm_in"], layer["norm_ffn"] = norm(), norm()
            layer["bias"] = (0.1 * torch.randn(qkv, device="cuda", generator=g)).half()
            pools = [new(pages + prefixes * prefix_pages, PAGE, kv_heads, dim).to(cache) for _ in range(2)]
            scale = torch.full((kv_heads,), 0.05, device="cuda") if cache == torch.float8_e4m3fn else None
            layer["cache"] = w4.KVCache(*pools, scale, scale)
        self.norm_out = norm()
        self.embedding = torch.randn(vocab, width, device="cuda", generator=g).half()
        self.inv_freq = w4.w4a16_rope_frequencies(dim, 10000.0).cuda()
        # The requests: lengths, what they get next (1: a token, 0: nothing, -1: ended), pages.
        i32 = torch.int32
        self.lens, self.new = new(batch, dtype=i32), torch.ones(batch, dtype=i32, device="cuda")
        self.table = new(batch, self.max_pages, dtype=i32)
        self.free = torch.randperm(pages, device="cuda", generator=g).to(i32)
        self.free_count = torch.full((1,), pages, dtype=i32, device="cuda")
        self.refused, self.slots, self.positions = new(batch, dtype=i32), new(batch, dtype=torch.int64), new(batch, dtype=i32)
        # Shared prefixes: their pages, lengths, each request's prefix (-1: none) and the tokens in front of its own.
        self.shared = prefixes > 0
        self.prefix_table = (pages + torch.arange(prefixes * prefix_pages, dtype=i32, device="cuda")).view(prefixes, prefix_pages)
        self.prefix_lens = new(prefixes, dtype=i32)
        self.prefix_of = torch.full((batch,), -1, dtype=i32, device="cuda")
        self.behind, self.places = new(batch, dtype=i32), new(batch, dtype=i32)
        # What sampling goes by (its random numbers are the caller's, anew before each step and each prompt).
        kinds = dict(temperature=torch.float32, top_k=i32, top_p=torch.float32, min_p=torch.float32)
        self.sampling = sampling and {n: torch.full((batch,), x, dtype=kinds[n], device="cuda") for n, x in sampling.items()}
        # The step's buffers. tokens: what each request goes on with; -1 where logits that are none left nothing to draw
        # (the request goes on with token 0 unless the caller ends it).
        self.tokens, self.words = torch.randint(0, vocab, (batch,), device="cuda", generator=g), new(batch, dtype=torch.int64)
        self.uniform = torch.rand(batch, device="cuda", generator=g)
        self.zero, self.h = new(batch, width, dtype=torch.float32), new(batch, width, dtype=torch.float32)
        self.x, self.n, self.y = new(batch, width), new(batch, width), new(batch, width)
        self.qkv, self.q, self.o = new(batch, qkv), new(batch, heads, dim), new(batch, heads, dim)
        self.act, self.logits = new(batch, ffn), new(batch, vocab)
        need = w4.w4a16_prefix_attention_workspace_bytes if self.shared else w4.w4a16_paged_attention_workspace_bytes
        self.workspace = new(need(batch, heads, kv_heads, dim), dtype=torch.uint8)

    def step(self):
        """One token of each request; tokens are replaced by the next ones."""
        w4.w4a16_kv_extend(self.lens, self.new, self.table, self.free, self.free_count, PAGE, self.slots, self.positions,
                           self.refused, spacing=1)  # row b of everything stays request b's
        places = torch.add(self.positions, self.behind, out=self.places) if self.shared else self.positions
        words = self.tokens if self.sampling is None else torch.clamp(self.tokens, min=0, out=self.words)
        torch.index_select(self.embedding, 0, words, out=self.x)
        self.rows(self.__dict__, places, self.slots, self.attend)
        w4.w4a16_gemm(self.n, *self.head, GROUP, out=self.logits)
        self.pick(self.logits, self.uniform, self.sampling, self.tokens)

    def attend(self, cache):
        """Each request's one token over its pages, and over those of its prefix."""
        if self.shared:
            w4.w4a16_prefix_attention(self.q, cache, self.table, self.lens, self.prefix_table, self.prefix_lens,
                                      self.prefix_of, out=self.o, workspace=self.workspace)
        else:
            w4.w4a16_paged_attention(self.q, cache, self.table, self.lens, out=self.o, workspace=self.workspace)

    def rows(self, at, positions, slots, attend):
        """The layers over the rows of at["x"], in the buffers of `at`; at["n"] is what the head reads."""
        rows = at["x"].shape[0]
        h, y = at["zero"], at["x"]  # the residual stream begins as the embedding
        q, k, v = at["qkv"].view(rows, -1, self.dim).split([self.heads, self.kv_heads, self.kv_heads], 1)
        for layer in self.layers:
            w4.w4a16_residual_rmsnorm(h, y, layer["norm_in"], EPS, h_out=at["h"], n_out=at["n"])
            h, y = at["h"], at["y"]
            w4.w4a16_gemm(at["n"], *layer["qkv"], GROUP, out=at["qkv"])
            w4.w4a16_rope_append(q, k, v, positions, self.inv_freq, layer["cache"], slots, bias=layer["bias"], out=at["q"])
            attend(layer["cache"])
            w4.w4a16_gemm(at["o"].view(rows, -1), *layer["o"], GROUP, out=y)
            w4.w4a16_residual_rmsnorm(h, y, layer["norm_ffn"], EPS, h_out=h, n_out=at["n"])
            w4.w4a16_gemm_swiglu(at["n"], *layer["gate"], *layer["up"], GROUP, out=at["act"])
            w4.w4a16_gemm(at["act"], *layer["down"], GROUP, out=y)
        w4.w4a16_residual_rmsnorm(h, y, self.norm_out, EPS, h_out=h, n_out=at["n"])

    def pick(self, logits, uniform, sampling, out):
        if sampling is None:
            torch.argmax(logits, 1, out=out)
        else:
            w4.w4a16_sample(logits, uniform, **sampling, out=out)

    def many(self, tokens, positions, slots, table, starts, lens, **prefix):
        """The layers over many tokens of some requests; returns the rows that the head reads."""
        like = ("zero", "h", "x", "n", "y", "qkv", "q", "o", "act")
        at = {n: torch.zeros(len(tokens), *self.__dict__[n].shape[1:], dtype=self.__dict__[n].dtype, device="cuda") for n in like}
        torch.index_select(self.embedding, 0, tokens, out=at["x"])
        size = w4.w4a16_prompt_attention_workspace_bytes(len(tokens), self.heads, self.kv_heads, self.dim)
        workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.rows(at, positions, slots, lambda cache: w4.w4a16_prompt_attention(
            at["q"], cache, table, starts, lens, out=at["o"], workspace=workspace, **prefix))
        return at["n"]

    def share(self, number, tokens):
        """Makes `tokens` (int64) prefix `number`, which requests name in prefix_of when they begin."""
        n, table = len(tokens), self.prefix_table[number:number + 1]
        assert 0 < n <= table.shape[1] * PAGE
        positions = torch.arange(n, dtype=torch.int32, device="cuda")
        slots = table[0].long().repeat_interleave(PAGE)[:n] * PAGE + positions % PAGE
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.many(tokens, positions, slots, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"), lens)
        self.prefix_lens[number] = n

    def prompt(self, prompts, prefix_of=None):
        """New tokens (int64) of some requests, {request: tokens}, behind what they have, or behind a shared prefix,
        {request: number}, where they begin; their next tokens are in `tokens` then. Returns their last rows' logits."""
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        for b, number in (prefix_of or {}).items():
            self.prefix_of[b], self.behind[b] = number, self.prefix_lens[number]
        new = [len(prompts.get(b, ())) for b in range(self.batch)]
        tokens = torch.cat([prompts[b] for b in range(self.batch) if new[b]])
        slots, positions = torch.zeros(len(tokens), dtype=torch.int64, device="cuda"), i32([0] * len(tokens))
        w4.w4a16_kv_extend(self.lens, i32(new), self.table, self.free, self.free_count, PAGE, slots, positions, self.refused)
        if self.refused.any():
            raise RuntimeError(f"no pages for the requests {self.refused.nonzero().flatten().tolist()}")
        ends = torch.tensor(new, device="cuda").cumsum(0)
        starts = torch.cat([ends.new_zeros(1), ends]).int()
        prefix = {}
        if self.shared:
            positions += self.behind.repeat_interleave(torch.tensor(new, device="cuda"))
            prefix = dict(prefix_table=self.prefix_table, prefix_lens=self.prefix_lens, prefix_of=self.prefix_of)
        n = self.many(tokens, positions, slots, self.table, starts, self.lens, **prefix)
        who = torch.tensor([b for b in range(self.batch) if new[b]], device="cuda")
        logits = w4.w4a16_gemm(n[ends[who] - 1], *self.head, GROUP)
        picked = torch.empty(len(who), dtype=torch.int64, device="cuda")
        self.pick(logits, self.uniform[who], self.sampling and {n: t[who] for n, t in self.sampling.items()}, picked)
        self.tokens[who] = picked
        return logits

    def capture(self):
        """The step as a CUDA graph (call step() once before)."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            self.step()
        torch.cuda.current_stream().wait_stream(stream)
        return graph


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in dict(width=1024, heads=8, kv_heads=2, dim=128, ffn=2048, layers=2, vocab=4096, batch=8, context=512,
                            steps=100).items():
        ap.add_argument("--" + name.replace("_", "-"), type=int, default=value)
    ap.add_argument("--cache", choices=("f16", "e4m3"), default="f16")
    ap.add_argument("--prompt", type=int, default=0, help="tokens that each request begins with")
    ap.add_argument("--prefix", type=int, default=0, help="tokens in front of these that all requests share")
    for name, kind in dict(temperature=float, top_k=int, top_p=float, min_p=float).items():
        ap.add_argument("--" + name.replace("_", "-"), type=kind, help="draws the next tokens")
    a = vars(ap.parse_args())
    steps, cache, prompt, prefix = (a.pop(n) for n in ("steps", "cache", "prompt", "prefix"))
    sampling = {n: x for n in ("temperature", "top_k", "top_p", "min_p") if (x := a.pop(n)) is not None}
    model = Decoder(cache=torch.float8_e4m3fn if cache == "e4m3" else torch.float16, **a, prefixes=int(prefix > 0),
                    prefix_context=prefix, sampling=sampling or None)

    def timed(step, n):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            if sampling:
                model.uniform.uniform_()
            step()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6

    some = lambda n: torch.randint(0, a["vocab"], (n,), device="cuda")  # noqa: E731
    if prefix:
        model.share(0, some(prefix))
        model.prefix_of.zero_()
        model.behind.fill_(prefix)
    if prompt:
        model.prompt({b: some(prompt) for b in range(a["batch"])})
        model.uniform.uniform_()  # the prompts' draws have had theirs
    model.step()
    n = min(steps, (a["context"] - prompt) // 4)
    print(f"eager: {timed(model.step, n):.1f} us a step")
    graph = model.capture()
    print(f"graph: {timed(graph.replay, n):.1f} us a step")
    w4.w4a16_set_launch_overlap(True)
    graph = model.capture()
    print(f"graph with launch overlap: {timed(graph.replay, n):.1f} us a step")
    w4.w4a16_set_launch_overlap(False)
    assert w4.w4a16_device_error() == w4.W4A16_OK and int(model.tokens.min()) >= 0
    print(f"{a['batch']} requests of {int(model.lens[0])} tokens, {int(model.free_count)} pages free; "
          f"next tokens {model.tokens.tolist()}")


if __name__ == "__main__":
    main()
