"""GPU parity of w4a16_sample with its float64 statement: the same token, unless the random number or top-p is nearer to a
border between two tokens than the weights' precision.

A weight is off by less than 2^-30 of itself. A border F is a quotient of two sums, which errors e and f of what is in front
of it and behind move by F (1 - F) |e - f|, less than 2^-31; the float64 statement is off by n 2^-53: answers may differ where
a border is nearer than 2^-30 of the sum. Rows where one is (none of the seeds here) would be left out, not accepted.
"""
import math

import numpy as np
import pytest
import torch

from oracle.wide_ops import sample

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NEAR = 2.0**-30


@pytest.fixture
def w4(gpu_lib):
    yield gpu_lib
    assert gpu_lib.w4a16_device_error() == gpu_lib.W4A16_OK


def logits(rows, vocab, dtype, seed=0, spread=2.0, high=20, banned=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * spread
    if high:
        at = torch.randint(0, vocab, (rows, high), generator=g)
        x.scatter_add_(1, at, torch.rand(rows, high, generator=g) * 8)
    if banned:
        x[torch.rand(rows, vocab, generator=g) < banned] = -math.inf
    return x.to(dtype).cuda()


def check(w4, x, u, temperature=None, top_k=None, top_p=None, min_p=None, exact=False):
    rows = x.shape[0]
    per = lambda v, d: [d] * rows if v is None else list(v)  # noqa: E731
    dev = lambda v, kind: None if v is None else torch.tensor(list(v), dtype=kind, device="cuda")  # noqa: E731
    args = (dev(temperature, F32), dev(top_k, torch.int32), dev(top_p, F32), dev(min_p, F32))
    uu = torch.tensor(list(u), dtype=F32, device="cuda")
    got = w4.w4a16_sample(x, uu, *args).tolist()
    assert w4.w4a16_sample(x, uu, *args).tolist() == got
    values = x.float().cpu().double().numpy()
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    left_out = 0
    for r in range(rows):
        want, near = sample(values[r], f32(u[r]), f32(per(temperature, 1.0)[r]), per(top_k, 0)[r], f32(per(top_p, 1.0)[r]),
                            f32(per(min_p, 0.0)[r]))
        if near < NEAR and not exact:
            left_out += 1
            continue
        assert got[r] == want, f"row {r}: {got[r]}, not {want} (near {near})"
    assert left_out <= rows // 20
    return got


def spread(rows, seed):
    return np.random.RandomState(seed).rand(rows).astype(np.float32)


SETTINGS = [dict(), dict(temperature=0.7), dict(top_k=40), dict(top_k=1000), dict(top_k=5000), dict(top_p=0.9), dict(top_p=0.05),
            dict(top_p=0.999), dict(min_p=0.05), dict(temperature=1.5, top_k=30, top_p=0.8, min_p=0.02),
            dict(temperature=0.3, top_k=3000, top_p=0.95), dict(temperature=3.0, top_k=4000, top_p=0.5), dict(temperature=0.0),
            dict(top_k=1), dict(top_p=0.0), dict(temperature=1e-6), dict(temperature=1e6, top_p=0.7), dict(temperature=math.inf, min_p=1.0)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("s", SETTINGS, ids=str)
def test_settings(w4, dtype, s):
    for rows, vocab, high in ((6, 9001, 20), (3, 40000, 0)):
        x = logits(rows, vocab, dtype, seed=vocab, high=high)
        check(w4, x, spread(rows, vocab), **{k: [v] * rows for k, v in s.items()})


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 31, 511, 512, 513, 4096, 32001, 65537, 131072, 262144])
@pytest.mark.parametrize("dtype", [F16, F32])
def test_vocabularies(w4, vocab, dtype):
    rows = 5
    x = logits(rows, vocab, dtype, seed=vocab, banned=0.2)
    x[:, vocab // 2] = 1.0
    check(w4, x, spread(rows, vocab), top_p=[1.0, 0.9, 0.5, 1.0, 0.7], top_k=[0, 0, 7, 3, vocab], temperature=[1.0, 0.8, 1.0, 2.0, 1.0])


def test_many_rows_with_settings_of_their_own(w4):
    rows, vocab = 400, 5003
    x = logits(rows, vocab, BF16, seed=5, banned=0.1)
    r = np.random.RandomState(3)
    check(w4, x, spread(rows, 1), temperature=r.choice([0.0, 0.5, 1.0, 1.7], rows), top_k=[int(v) for v in r.choice([0, 1, 5, 50, 2000], rows)],
          top_p=r.choice([1.0, 0.9, 0.3], rows), min_p=r.choice([0.0, 0.1, 0.01], rows))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_equal_logits(w4, dtype):
    # All alike: the first k, the first p of them, in the order of their numbers, far more than are gathered. Every weight is
    # the same number, so sums are whole multiples of it on both sides, and borders that are met exactly are met by both.
    rows, vocab = 8, 30000
    x = torch.full((rows, vocab), 1.5, dtype=dtype, device="cuda")
    check(w4, x, spread(rows, 2), top_k=[0, 5000, 20000, 0, 0, 9, 0, 1200], top_p=[1.0, 1.0, 0.3, 0.501, 0.25, 1.0, 0.9999, 0.5],
          exact=True)
    # A few values only; the border lies among thousands of equal ones (in the last row among the largest ones alone).
    g = torch.Generator().manual_seed(0)
    x = (torch.randint(0, 6, (rows, vocab), generator=g) * 0.25).to(dtype).cuda()
    check(w4, x, spread(rows, 3), top_k=[0, 7000, 25000, 0, 0, 12000, 0, 4000], top_p=[1.0, 1.0, 0.3, 0.501, 0.25, 0.7, 0.9999, 0.5],
          exact=True)
    # Values so near each other that they share a bin of weights, all different in 32 bits.
    if dtype == F32:
        x = (1.0 + torch.rand(rows, vocab, generator=g) * 0.01).cuda()
        check(w4, x, spread(rows, 4), top_k=[0, 7000, 25000, 0, 0, 12000, 0, 4000], top_p=[1.0, 1.0, 0.3, 0.501, 0.25, 0.7, 0.9999, 0.5])


def test_zeros_of_either_sign_are_equal(w4):
    x = torch.zeros(4, 3000, dtype=F16, device="cuda")
    x[:, ::2] = -0.0
    check(w4, x, [0.0, 0.3, 0.7, 0.99], top_k=[10, 11, 1500, 0])


def test_infinities_and_nan(w4):
    x = logits(7, 2000, F32, seed=1)
    x[0] = -math.inf
    x[1, :] = math.nan
    x[2, ::3] = math.nan
    x[3, 17] = x[3, 900] = math.inf
    x[4] = -math.inf
    x[4, 1234] = -5e37
    x[5, 100:] = -math.inf
    got = check(w4, x, [0.5, 0.5, 0.3, 0.7, 0.9, 1.0, 0.0], top_p=[0.9, 0.9, 0.9, 0.9, 1.0, 1.0, 1.0])
    assert got[0] == got[1] == -1 and got[3] == 900 and got[4] == 1234
    got = w4.w4a16_sample(x, torch.zeros(7, device="cuda"), torch.zeros(7, device="cuda")).tolist()
    assert got[0] == -1 and got[3] == 17 and got[4] == 1234


def test_random_numbers_at_the_ends(w4):
    x = logits(6, 12000, BF16, seed=2, banned=0.3)
    check(w4, x, [0.0, 1.0, 0.0, 1.0, 1.0 - 2**-24, 2**-30], top_p=[1.0, 1.0, 0.9, 0.9, 1.0, 1.0], top_k=[0, 0, 50, 50, 0, 0])


def test_out_of_range_settings(w4):
    x, n = logits(4, 500, F16), math.nan
    f = lambda *v: torch.tensor(v, dtype=F32, device="cuda")  # noqa: E731
    half, one, none = f(0.5, 0.5, 0.5, 0.5), f(1, 1, 1, 1), f(0, 0, 0, 0)
    for u, t, p, m, same in ((f(0.5, -0.1, 0.5, 0.5), one, one, none, (f(0.5, 0, 0.5, 0.5), one, one, none)),
                             (f(0.5, 1.5, n, 0.5), one, one, none, (f(0.5, 1, 0, 0.5), one, one, none)),
                             (half, f(1, -1, n, 1), one, none, (half, f(1, 0, 0, 1), one, none)),
                             (half, one, f(1, n, 1, 1), f(0, 0, n, 0), (half, one, one, none))):
        got = w4.w4a16_sample(x, u, t, None, p, m).tolist()
        assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
        assert got == w4.w4a16_sample(x, same[0], same[1], None, same[2], same[3]).tolist()


def test_views_streams_and_graphs(w4):
    wide = torch.full((9, 7013), 50.0, dtype=F16, device="cuda")
    x = wide[:, 3:7004]
    x.copy_(logits(9, 7001, F16, seed=7))
    u = spread(9, 9)
    want = check(w4, x, u, top_p=[0.9] * 9)
    uu, p = torch.tensor(u, device="cuda"), torch.full((9,), 0.9, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = w4.w4a16_sample(x, uu, top_p=p, stream=stream)
    stream.synchronize()
    assert got.tolist() == want
    out = torch.zeros(9, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        w4.w4a16_sample(x, uu, top_p=p, out=out)
    for _ in range(3):
        out.fill_(-5)
        graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == want


def test_draws_have_their_probabilities(w4):
    # 2000 evenly spaced random numbers: each token gets its share to within one of them.
    x = logits(1, 40, F32, seed=3).expand(2000, 40).contiguous()
    u = (torch.arange(2000, device="cuda", dtype=F32) + 0.5) / 2000
    got = torch.bincount(w4.w4a16_sample(x, u), minlength=40).double() / 2000
    want = torch.softmax(x[0].double(), 0)
    assert float((got - want).abs().max()) <= 1 / 2000 + 1e-6


def test_more_rows_than_fit_the_gpu_at_once(w4):
    r = np.random.RandomState(5)
    x = torch.from_numpy(r.randn(3001, 700).astype(np.float32) * 3).cuda()
    check(w4, x.half(), spread(3001, 6), top_p=[float(v) for v in r.rand(3001)], top_k=[int(v) for v in r.randint(0, 300, 3001)])
