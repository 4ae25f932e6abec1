"""What the example decoder (examples/decode.py) tells its caller where nothing can be drawn, and what its draws go by."""
import math
import sys

import pytest
import torch

from test_gpu_decode_example import SIZES, ex  # noqa: F401
from test_gpu_serving import SAMPLING

pytestmark = pytest.mark.gpu


def test_nothing_to_draw_from_is_seen(ex):  # noqa: F811
    m = ex.Decoder(**SIZES, sampling=SAMPLING)
    prompts = {b: torch.arange(5 + b, device="cuda") for b in range(3)}
    norm = m.norm_out.clone()
    m.norm_out.fill_(math.nan)
    m.prompt(prompts)
    assert m.tokens.tolist() == [-1, -1, -1]
    m.step()
    assert m.tokens.tolist() == [-1, -1, -1]
    graph = m.capture()
    graph.replay()
    assert m.tokens.tolist() == [-1, -1, -1]
    m.norm_out.copy_(norm)  # the layers and the cache have had token 0, and go on
    graph.replay()
    assert bool((m.tokens >= 0).all()) and bool(torch.isfinite(m.logits).all())
    assert m.lens.tolist() == [8, 9, 10]


def test_every_draw_of_the_example_has_random_numbers_of_its_own(ex, monkeypatch):  # noqa: F811
    had = []
    pick = ex.Decoder.pick

    def look(self, logits, uniform, sampling, out):
        if not torch.cuda.is_current_stream_capturing():
            had.append(uniform.tolist())
        pick(self, logits, uniform, sampling, out)

    monkeypatch.setattr(ex.Decoder, "pick", look)
    monkeypatch.setattr(sys, "argv", ["decode.py", "--prompt", "9", "--prefix", "5", "--steps", "4", "--temperature", "0.8", "--width", "256",
                                      "--heads", "4", "--dim", "64", "--ffn", "512", "--vocab", "512", "--batch", "3", "--context", "64"])
    ex.main()
    assert len(had) == 1 + 1 + 4  # the prompts', a step, the timed eager ones
    for b in range(3):
        assert len({u[b] for u in had}) == len(had)
