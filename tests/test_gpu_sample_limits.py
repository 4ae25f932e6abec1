"""Sampling where it is hardest to get right: steps of a cluster that follow each other closely, weights that are taken by
differences of logits of any size, random numbers next to a border between two tokens."""
import numpy as np
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


# A weight is off by less than 2^-30 of itself and 2^-44 of the largest. A border F between two tokens is a quotient of two
# sums, which errors of e and f of what is in front of it and behind move by F (1 - F) |e - f| < 2^-31; the second part adds
# 2^-44 for each token, the sum being the largest weight at least. The float64 statement is off by n 2^-53.
def bound(n):
    return 2.0**-31 + n * (2.0**-44 + 2.0**-53)


def next_to_a_border(upto):
    """The float32 number that is nearest to one of the borders `upto` (float64, from 0 to 1), but not nearer than twice the
    bound; None if there is none within 2^-28."""
    near = upto[:-1].astype(np.float32)
    u = np.stack([near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(1))])
    far = np.abs(u.astype(np.float64) - upto[:-1])
    far[(far <= 2 * bound(len(upto))) | (u <= 0) | (u >= 1)] = 1
    at = np.unravel_index(far.argmin(), far.shape)
    return float(u[at]) if far[at] < 2.0**-28 else None


def rows_of(kind, n, dtype, g):
    """Logits whose largest is smaller than the others' magnitudes, so that differences to it need more bits than 32."""
    x = -torch.rand(n, generator=g) * 6 - 0.3
    if kind == "negative":       # all but the largest a little beyond a power of two
        x = -4.0 - torch.rand(n, generator=g) * 1e-2
        x[int(torch.randint(0, n, (1,), generator=g))] = -1.0 - float(torch.rand(1, generator=g)) * 0.7
    elif kind == "tiny largest":
        x[int(torch.randint(0, n, (1,), generator=g))] = 2.0**-24 * float(torch.randint(1, 512, (1,), generator=g))
    else:
        x = torch.log_softmax(x, 0)
    return x.to(dtype)


@pytest.mark.parametrize("kind,dtype", [("log-probabilities", F32), ("tiny largest", F32), ("tiny largest", F16), ("negative", F32),
                                        ("log-probabilities", BF16)])
@pytest.mark.parametrize("n", [7, 60, 2500])
def test_next_to_a_border(w4, kind, dtype, n):
    g = torch.Generator().manual_seed(n)
    rows, us, ps = [], [], []
    while len(rows) < 48:
        x = rows_of(kind, n, dtype, g)
        v = x.double().numpy()
        if len(rows) % 2:  # a border of the draw
            w = np.exp(v - v.max())
            u, p = next_to_a_border(np.cumsum(w) / w.sum()), 1.0
        else:              # of top-p: the last random number that is not 1 draws the last token that is left, or one near it
            w = np.sort(np.exp(v - v.max()))[::-1]
            u, p = 1.0, next_to_a_border(np.cumsum(w) / w.sum())
        if u is not None and p is not None:
            rows.append(x), us.append(u), ps.append(p)
    x = torch.stack(rows)
    got = w4.w4a16_sample(x.cuda(), torch.tensor(us, device="cuda"), top_p=torch.tensor(ps, device="cuda")).tolist()
    for r in range(len(rows)):
        assert got[r] == sample(x[r].double().numpy(), us[r], 1.0, 0, ps[r])[0], f"row {r}, u {us[r]}, top-p {ps[r]}"


@pytest.mark.parametrize("down", [20.0, 26.0, 29.5])
def test_many_small_weights(w4, down):
    # One token of weight 1 and 200000 far below it: whichever of these is drawn, its borders are next to u.
    n, rows = 200001, 16
    g = torch.Generator().manual_seed(1)
    x = -down - torch.rand(n, generator=g)
    x[77] = 0.0
    w = np.exp(x.double().numpy())
    upto = np.cumsum(w)
    u = torch.from_numpy(np.float32(1) - np.float32(2.0**-24) * np.arange(rows, dtype=np.float32))
    got = w4.w4a16_sample(x.expand(rows, n).contiguous().cuda(), u.cuda()).tolist()
    for token, at in zip(got, u.double().tolist()):
        before = upto[token - 1] if token else 0.0
        assert before / upto[-1] - bound(n) <= at <= upto[token] / upto[-1] + bound(n), (token, at)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,n", [(12, 50), (12, 3000)])
def test_logits_further_apart_than_the_largest_float(w4, dtype, rows, n):
    # With temperatures of their size they have weights all the same: e^-2 for the lowest at 3e38, all alike at infinity.
    g = torch.Generator().manual_seed(n)
    x = ((torch.rand(rows, n, generator=g) * 2 - 1) * 3.3e38).to(dtype)
    x[:, 5] = 3.3e38
    x[:, n - 3] = -3.3e38
    heat = torch.tensor([3e38, float("inf"), 1e38, 3e37] * 3)
    k = torch.tensor([0] * 8 + [n // 2] * 4, dtype=torch.int32)
    p = torch.tensor([1.0] * 4 + [0.9] * 8)
    m = torch.tensor([0.0] * 11 + [0.05])
    u = (torch.arange(rows) + 0.4) / rows
    got = w4.w4a16_sample(x.cuda(), u.cuda(), heat.cuda(), k.cuda(), p.cuda(), m.cuda()).tolist()
    for r in range(rows):
        want, near = sample(x[r].double().numpy(), float(u[r]), float(heat[r]), int(k[r]), float(p[r]), float(m[r]))
        # At infinity every weight is the same number, so that sums are whole multiples of it on both sides (the product of u,
        # 24 bits, and n is exact in 64): a border may be as near as it likes.
        assert near > 2 * bound(n) or heat[r] == float("inf")
        assert got[r] == want, r


def test_settings_that_leave_the_largest_logit_only(w4):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(6, 5000, generator=g)
    x[:, 4321] = x[:, 1234] = 9.0
    f = lambda *v: torch.tensor(v, dtype=F32, device="cuda")  # noqa: E731
    got = w4.w4a16_sample(x.cuda(), f(*[0.99] * 6), f(0, 1, 1, 1, 1, 1), torch.tensor([0, 1, 0, 0, 0, 0], dtype=torch.int32, device="cuda"),
                          f(1, 1, 0, -2, 1, 1), f(0, 0, 0, 0, 1.5, 1))
    assert got.tolist() == [1234] * 5 + [4321]  # of weights of 1 the second one, too, is at least 1
