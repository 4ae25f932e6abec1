"""The operators as a server runs them (examples/decode.py): shared prefixes, prompts and parts of prompts, steps and drawn
tokens, against a float64 restatement of the whole model and of the draw; captured steps against eager ones."""
import numpy as np
import pytest
import torch

from oracle import wide_ops
from test_gpu_decode_example import SIZES, Plain, ex, f64  # noqa: F401

pytestmark = pytest.mark.gpu
SAMPLING = dict(temperature=0.7, top_k=50, top_p=0.9, min_p=0.01)


def words(rng, n):
    return torch.from_numpy(rng.integers(0, SIZES["vocab"], n)).cuda()


def feed(plain, b, tokens):
    """Request b's tokens one by one; the last one's logits."""
    for t in tokens.tolist():
        row = np.zeros(plain.m.batch, dtype=np.int64)
        row[b] = t
        got = plain.logits(row, [b])[b]
    return got


def check(got, want):
    # The bound of the steps' test (test_gpu_decode_example.py): the layers and their roundings are the same.
    assert np.abs(f64(got) - want).max() <= 2e-2 * np.abs(want).max()


def drawn(m, logits, uniform, tokens):
    """The tokens are those that the definition draws from the logits that the model has come to."""
    for row, u, token in zip(f64(logits), f64(uniform), tokens.tolist()):
        want, near = wide_ops.sample(row, u, **{n: float(np.float32(x)) if n != "top_k" else x for n, x in SAMPLING.items()})
        assert token == want or near < 1e-6


def test_prompts_prefixes_and_steps_match_the_model_in_float64(ex):  # noqa: F811
    m = ex.Decoder(**SIZES, prefixes=2, prefix_context=40, sampling=SAMPLING)
    plain, rng = Plain(m, ex), np.random.default_rng(1)
    first, second = words(rng, 21), words(rng, 40)
    m.share(0, first)
    m.share(1, second)
    prompts = {b: words(rng, n) for b, n in ((0, 17), (1, 1), (2, 30))}
    # Request 0 behind the first prefix, 2 behind the second, 1 behind none.
    own = {0: first, 2: second}
    want = {b: feed(plain, b, torch.cat([own[b], t]) if b in own else t) for b, t in prompts.items()}
    logits = m.prompt(prompts, {0: 0, 2: 1})
    assert m.lens.tolist() == [17, 1, 30] and m.behind.tolist() == [21, 0, 40]
    for i, b in enumerate(prompts):
        check(logits[i], want[b])
    drawn(m, logits, m.uniform, m.tokens)
    for step in range(12):
        if step == 5:  # some requests get several tokens more, one of them just one
            more = {1: words(rng, 7), 2: words(rng, 1)}
            logits = m.prompt(more)
            for i, (b, t) in enumerate(more.items()):
                check(logits[i], feed(plain, b, t))
        tokens = m.tokens.cpu().numpy()
        m.uniform.copy_(torch.from_numpy(rng.random(m.batch, dtype=np.float32)))
        m.step()
        want = plain.logits(tokens, [0, 1, 2])
        check(m.logits, want)
        drawn(m, m.logits, m.uniform, m.tokens)
    assert m.lens.tolist() == [29, 20, 43] and plain.pos.tolist() == [50, 20, 83] and not m.refused.any()


def test_a_prompt_without_pages_is_refused(ex):  # noqa: F811
    m = ex.Decoder(**SIZES, pages=3)
    with pytest.raises(RuntimeError, match=r"\[1\]"):
        m.prompt({0: torch.zeros(20, dtype=torch.int64, device="cuda"), 1: torch.zeros(20, dtype=torch.int64, device="cuda")})
    assert m.lens.tolist() == [20, 0, 0]


@pytest.mark.parametrize("cache", [torch.float16, torch.float8_e4m3fn])
@pytest.mark.parametrize("overlap", [False, True])
def test_captured_steps_equal_eager_ones(ex, gpu_lib, cache, overlap):  # noqa: F811
    both = [ex.Decoder(**SIZES, cache=cache, prefixes=1, prefix_context=33, sampling=SAMPLING) for _ in range(2)]
    rng = np.random.default_rng(2)
    prefix, prompts = words(rng, 33), {b: words(rng, n) for b, n in ((0, 5), (2, 18))}
    numbers = torch.from_numpy(rng.random((20, 3), dtype=np.float32)).cuda()
    for m in both:
        m.share(0, prefix)
        m.prompt(prompts, {0: 0, 1: 0, 2: 0})
        m.step()
    gpu_lib.w4a16_set_launch_overlap(overlap)
    torch.cuda.synchronize()
    a, b = both
    graph = b.capture()
    for u in numbers:
        for m, run in ((a, a.step), (b, graph.replay)):
            m.uniform.copy_(u)
            run()
    torch.cuda.synchronize()
    assert a.lens.tolist() == b.lens.tolist() == [26, 21, 39]
    for name in ("logits", "tokens", "h", "table", "slots", "free_count"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
