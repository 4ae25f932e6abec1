"""The example decoder (examples/decode.py): steps against a float64 restatement of the whole model, requests that
end and start anew, and the captured step against the eager one."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import decode_ops as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = dict(width=256, heads=4, kv_heads=2, dim=64, ffn=512, layers=2, vocab=512, batch=3, context=64)


@pytest.fixture
def ex(gpu_lib):
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    yield mod
    gpu_lib.w4a16_set_launch_overlap(False)
    assert gpu_lib.w4a16_device_error() == gpu_lib.W4A16_OK


def f64(t):
    return t.detach().float().cpu().double().numpy()


class Plain:
    """The model in float64, a list of keys and values for each request and layer; values are rounded to fp16 nowhere."""

    def __init__(self, m, ex):
        self.m, self.ex = m, ex
        w = lambda r: oracle.dequant(r[0].cpu().numpy(), r[1].cpu().numpy(), r[2].cpu().numpy(), 2 * r[0].shape[1], ex.GROUP)  # noqa: E731
        self.layers = [{n: w(r) for n, r in layer.items()} for layer in m.raw]
        self.head = w(m.raw_head)
        self.kv = [[([], []) for _ in range(m.batch)] for _ in m.raw]
        self.pos = np.zeros(m.batch, dtype=np.int64)

    def forget(self, b):
        self.pos[b] = 0
        for layer in self.kv:
            layer[b] = ([], [])

    def logits(self, tokens, rows):
        m = self.m
        rms = lambda x, g: x / np.sqrt(np.mean(x * x, 1, keepdims=True) + self.ex.EPS) * f64(g)  # noqa: E731
        h = f64(m.embedding)[tokens]
        for i, (layer, raw) in enumerate(zip(m.layers, self.layers)):
            x = rms(h, layer["norm_in"]) @ raw["qkv"].T + f64(layer["bias"])
            x = x.reshape(m.batch, -1, m.dim)
            turned, _ = ref.rope(x[:, :m.heads + m.kv_heads], self.pos, f64(m.inv_freq), m.dim, False, 1.0)
            o = np.zeros((m.batch, m.heads, m.dim))
            g = m.heads // m.kv_heads
            for b in rows:
                ks, vs = self.kv[i][b]
                ks.append(turned[b, m.heads:])
                vs.append(x[b, m.heads + m.kv_heads:])
                k, v = np.stack(ks), np.stack(vs)
                for j in range(m.kv_heads):
                    o[b, j * g:(j + 1) * g] = ref.attention(turned[b, j * g:(j + 1) * g], k[:, j], v[:, j], m.dim**-0.5)[0]
            h = h + o.reshape(m.batch, -1) @ raw["o"].T
            x = rms(h, layer["norm_ffn"])
            gate, up = x @ raw["gate"].T, x @ raw["up"].T
            h = h + (gate / (1 + np.exp(-gate)) * up) @ raw["down"].T
        self.pos[rows] += 1
        return rms(h, m.norm_out) @ self.head.T


def test_steps_match_the_model_in_float64(ex):
    m = ex.Decoder(**SIZES, pages=7)
    plain = Plain(m, ex)
    rng = np.random.default_rng(0)
    for step in range(40):
        tokens = torch.from_numpy(rng.integers(0, SIZES["vocab"], m.batch)).cuda()
        m.tokens.copy_(tokens)
        new = [1, 1, 1]
        if step in (17, 30):  # a request ends, gives its pages back and begins anew in the next step
            new[step % 3] = -1
            plain.forget(step % 3)
        m.new.copy_(torch.tensor(new, dtype=torch.int32))
        m.step()
        rows = [b for b in range(m.batch) if new[b] > 0]
        want = plain.logits(tokens.cpu().numpy(), rows)[rows]
        got = f64(m.logits)[rows]
        assert m.lens.tolist() == plain.pos.tolist() and not m.refused.any()
        # Some thirty roundings to fp16 (2^-11 each) lie between a token and its logits, and the int4 product's own
        # (of the dequantised weights): well inside the bound that the product alone is held to.
        assert np.abs(got - want).max() <= 2e-2 * np.abs(want).max()


def test_refused_request_leaves_the_others_alone(ex):
    m, few = ex.Decoder(**SIZES), ex.Decoder(**SIZES, pages=3)
    for step in range(17):  # the fourth page is not there
        m.step()
        few.step()
    torch.cuda.synchronize()
    assert m.lens.tolist() == [17] * 3
    assert few.lens.tolist() == [16] * 3 and few.refused.tolist() == [1] * 3 and few.slots.tolist() == [-1] * 3


@pytest.mark.parametrize("cache", [torch.float16, torch.float8_e4m3fn])
@pytest.mark.parametrize("overlap", [False, True])
def test_captured_steps_equal_eager_ones(ex, gpu_lib, cache, overlap):
    a, b = ex.Decoder(**SIZES, cache=cache), ex.Decoder(**SIZES, cache=cache)
    a.step()
    b.step()
    gpu_lib.w4a16_set_launch_overlap(overlap)
    torch.cuda.synchronize()
    graph = b.capture()
    for _ in range(30):
        a.step()
        graph.replay()
    torch.cuda.synchronize()
    assert a.lens.tolist() == b.lens.tolist() == [31] * 3
    for name in ("logits", "tokens", "h", "table", "slots", "free_count"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
