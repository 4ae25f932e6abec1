"""Sampling where it is hardest to get right: steps of a cluster that follow each other closely, weights that are taken by
differences of logits of any size, random numbers next to a border between two tokens."""
import pytest
import torch

from oracle.wide_ops import sample

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture
def w4(gpu_lib):
    yield gpu_lib
    assert gpu_lib.w4a16_device_error() == gpu_lib.W4A16_OK


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [4104, 9000, 33001])
def test_a_border_among_equal_logits_again_and_again(w4, dtype, vocab):
    # The border lies among more equal tokens than are gathered: it is looked for by their numbers, and the draw, which is
    # the next step of the cluster, begins at once. CTAs have few tokens, so one that is ahead is soon there.
    rows = 8
    x = torch.full((rows, vocab), -2.5, dtype=dtype, device="cuda")
    u = (torch.arange(rows, device="cuda", dtype=F32) + 0.37) / rows
    k = torch.tensor([vocab - 1, vocab // 2, 0, 0, 2000, 3000, 1500, vocab - 7], dtype=torch.int32, device="cuda")
    p = torch.tensor([1.0, 1.0, 0.5, 0.9375, 1.0, 0.75, 1.0, 0.25], device="cuda")
    # All weights are alike: sums are whole multiples of one number on both sides.
    want = [sample(x[r].double().cpu().numpy(), float(u[r]), 1.0, int(k[r]), float(p[r]))[0] for r in range(rows)]
    out = torch.full((400, rows), -7, dtype=torch.int64, device="cuda")
    for i in range(400):
        w4.w4a16_sample(x, u, top_k=k, top_p=p, out=out[i])
    assert bool((out == torch.tensor(want, device="cuda")).all())
