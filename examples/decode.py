"""A decoder with int4 weights, answering: every operator of the library in the order in which a step runs them.

    python examples/decode.py                      # a small model, random weights
    python examples/decode.py --width 5120 --heads 40 --kv-heads 8 --ffn 13824 --layers 4 --batch 8

A step takes one token of each request: its place in the paged cache (kv_extend), then for each layer the QKV
projection, rotary positions and the cache (rope_append), attention over the cache's pages (paged_attention), the
output projection, the residual stream and the next norm (residual_rmsnorm), the SwiGLU and down projections, and
again residual stream and norm. Nothing in it allocates or waits for the GPU, so the whole step is captured into one
CUDA graph and replayed; requests grow, end and start anew inside the graph, because lengths, block table and free
list live on the GPU.
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
                 pages=None, cache=torch.float16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.batch, self.max_pages = heads, kv_heads, dim, batch, -(-context // PAGE)
        pages = pages or batch * self.max_pages
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
            pools = [new(pages, PAGE, kv_heads, dim).to(cache) for _ in range(2)]
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
        # The step's buffers.
        self.tokens = torch.randint(0, vocab, (batch,), device="cuda", generator=g)
        self.zero, self.h = new(batch, width, dtype=torch.float32), new(batch, width, dtype=torch.float32)
        self.x, self.n, self.y = new(batch, width), new(batch, width), new(batch, width)
        self.qkv, self.q, self.o = new(batch, qkv), new(batch, heads, dim), new(batch, heads, dim)
        self.act, self.logits = new(batch, ffn), new(batch, vocab)
        self.workspace = new(w4.w4a16_paged_attention_workspace_bytes(batch, heads, kv_heads, dim), dtype=torch.uint8)

    def step(self):
        """One token of each request; tokens are replaced by the next ones."""
        w4.w4a16_kv_extend(self.lens, self.new, self.table, self.free, self.free_count, PAGE, self.slots, self.positions,
                           self.refused, spacing=1)  # row b of everything stays request b's
        torch.index_select(self.embedding, 0, self.tokens, out=self.x)
        h, y = self.zero, self.x  # the residual stream begins as the embedding
        q, k, v = self.qkv.view(self.batch, -1, self.dim).split([self.heads, self.kv_heads, self.kv_heads], 1)
        for layer in self.layers:
            w4.w4a16_residual_rmsnorm(h, y, layer["norm_in"], EPS, h_out=self.h, n_out=self.n)
            h, y = self.h, self.y
            w4.w4a16_gemm(self.n, *layer["qkv"], GROUP, out=self.qkv)
            w4.w4a16_rope_append(q, k, v, self.positions, self.inv_freq, layer["cache"], self.slots, bias=layer["bias"],
                                 out=self.q)
            w4.w4a16_paged_attention(self.q, layer["cache"], self.table, self.lens, out=self.o, workspace=self.workspace)
            w4.w4a16_gemm(self.o.view(self.batch, -1), *layer["o"], GROUP, out=y)
            w4.w4a16_residual_rmsnorm(h, y, layer["norm_ffn"], EPS, h_out=h, n_out=self.n)
            w4.w4a16_gemm_swiglu(self.n, *layer["gate"], *layer["up"], GROUP, out=self.act)
            w4.w4a16_gemm(self.act, *layer["down"], GROUP, out=y)
        w4.w4a16_residual_rmsnorm(h, y, self.norm_out, EPS, h_out=h, n_out=self.n)
        w4.w4a16_gemm(self.n, *self.head, GROUP, out=self.logits)
        torch.argmax(self.logits, 1, out=self.tokens)

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
    a = vars(ap.parse_args())
    steps, cache = a.pop("steps"), a.pop("cache")
    model = Decoder(cache=torch.float8_e4m3fn if cache == "e4m3" else torch.float16, **a)

    def timed(step, n):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            step()
        torch.cuda.synchronize()
        return (time.perf_counter() - t) / n * 1e6

    model.step()
    n = min(steps, a["context"] // 4)
    print(f"eager: {timed(model.step, n):.1f} us a step")
    graph = model.capture()
    print(f"graph: {timed(graph.replay, n):.1f} us a step")
    w4.w4a16_set_launch_overlap(True)
    graph = model.capture()
    print(f"graph with launch overlap: {timed(graph.replay, n):.1f} us a step")
    w4.w4a16_set_launch_overlap(False)
    assert w4.w4a16_device_error() == w4.W4A16_OK
    print(f"{a['batch']} requests of {int(model.lens[0])} tokens, {int(model.free_count)} pages free; "
          f"next tokens {model.tokens.tolist()}")


if __name__ == "__main__":
    main()
