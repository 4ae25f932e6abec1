"""What the example decoder (examples/decode.py) tells its caller where nothing can be drawn, and what its draws go by."""
import math

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
