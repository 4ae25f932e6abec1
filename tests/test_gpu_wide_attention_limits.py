"""Attention of many rows at its limits: what lies in shared memory where a call begins, rows of a tile that are nobody's,
what only other rows see, large caps and windows, prompts of many thousand tokens."""
import math

import numpy as np
import pytest
import torch

from oracle.wide_ops import rows_attention
from test_gpu_wide_attention import BF16, E, E4M3, F16, Setup, U, f64, w4  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F16)])
def test_queries_and_keys_come_where_the_plan_has_been(w4, dim, dtype):  # noqa: F811
    # The plan of many requests lies where the first boxes of queries and keys are brought, in every call.
    n = 3000
    s = Setup(w4, [2] * n, [2 + 11 * i % 40 for i in range(n)], heads=2, kv=1, dim=dim, dtype=dtype, page=16)
    s.prompt()
    s.check(only=range(0, n, 41))
    first = s.out.clone(), s.lse.clone()
    for _ in range(30):
        s.prompt()
        assert torch.equal(s.out, first[0]) and torch.equal(s.lse, first[1])


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, F16)])
@pytest.mark.parametrize("new,pad", [(3, 40), (49, 0)])
def test_rows_that_are_nobody_s_change_nothing(w4, dim, dtype, new, pad):  # noqa: F811
    # 5 heads to a kv head: a box of queries does not fill a tile, and holds rows of other requests and of none behind a
    # request's last one. So many keys that every CTA has several units of them.
    s = Setup(w4, [new, 20], [50000, 300], heads=10, kv=2, dim=dim, dtype=dtype, q_scale=0.4, pad=pad, page=64)
    loud = Setup(w4, [300], [300], heads=8, kv=2, dim=dim, dtype=dtype, q_scale=1.0)
    for x in (loud.q, loud.k, loud.v):
        x.fill_(200.0)
    mine = slice(0, new)
    s.prompt()
    first = s.out[mine].clone(), s.lse[mine].clone()
    for level in (0.0, 1.0, 30.0, -30.0):
        loud.q.fill_(200.0 + level)
        loud.prompt()  # leaves its numbers in shared memory
        s.q[new:] = level * torch.sign(torch.randn(s.q[new:].shape, device="cuda"))
        s.prompt()
        same = torch.equal(s.out[mine], first[0]), torch.equal(s.lse[mine], first[1])
        assert same == (True, True), level


def check_scores_to_their_own_size(s, expected, rows=None):
    """As Setup.check, for scores that are off by a few roundings of themselves and nothing that goes by a cap: of all rows, or
    of those named for each request (from its first one on)."""
    torch.cuda.synchronize()
    u, out, lse = U[s.dtype], f64(s.out), f64(s.lse)
    for i, (at, (want, want_lse, mag, top), n) in enumerate(expected):
        # products' sum, then scale, quotient by the cap, tanh (2), product with the cap, difference, exponential
        eps = (s.dim + 24) * E * top + (n + 8) * E + 2.0**-22
        bound = u * np.abs(want) + 2 * (u + eps)[..., None] * mag + n * 2.0**-36 * (mag.max() + 1) + 2.0**-24
        some = slice(0, rows[i]) if rows else slice(None)
        assert (np.abs(out[at] - want) <= bound)[some].all()
        assert (np.abs(lse[at] - want_lse) <= eps + 2 * E * np.abs(want_lse))[some].all()


@pytest.mark.parametrize("dim,dtype,cache", [(64, F16, F16), (128, BF16, BF16), (128, BF16, E4M3), (256, F16, F16)])
@pytest.mark.parametrize("softcap", [129.0, 1000.0, 1e4, 1e6, 1e20, 3e38])
def test_large_caps(w4, softcap, dim, dtype, cache):  # noqa: F811
    s = Setup(w4, [3, 70], [200, 300], [100], [0, -1], heads=6, kv=2, dim=dim, dtype=dtype, cache=cache)
    s.prompt(softcap=softcap)
    check_scores_to_their_own_size(s, s.want(dim**-0.5, 0, softcap))
    s = Setup(w4, [1] * 20, [1 + 7 * i for i in range(20)], [400], [-(i % 2) for i in range(20)], heads=6, kv=2, dim=dim, dtype=dtype,
              cache=cache)
    s.prefix(softcap=softcap)
    check_scores_to_their_own_size(s, s.want(dim**-0.5, 0, softcap))


def test_the_largest_window_of_rows_in_front_of_the_first_token(w4):  # noqa: F811
    # A length below a request's rows: the first ones see nothing, the others what there is, with any window.
    s = Setup(w4, [9, 4], [9, 4], heads=4, kv=2, dim=64)
    s.len_t = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    s.prompt()
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    assert bool((s.out[:7] == 0).all()) and bool((s.out[7:] != 0).all())
    want = s.out.clone(), s.lse.clone()
    s.prompt(window=2**31 - 1)
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    assert torch.equal(s.out, want[0]) and torch.equal(s.lse, want[1])


@pytest.mark.parametrize("cache,junk", [(F16, math.nan), (F16, math.inf), (F16, -math.inf), (F16, 65504.0), (F16, -65504.0),
                                        (BF16, math.nan), (BF16, -math.inf), (E4M3, math.nan), (E4M3, -448.0)])
@pytest.mark.parametrize("dim", [128, 256])
def test_what_only_other_rows_see_is_not_seen(w4, cache, junk, dim):  # noqa: F811
    # As test_what_is_not_visible, every set of it with something to find, and no error named.
    s = Setup(w4, [40, 7], [300, 130], [70], [0, -1], heads=10, kv=2, dim=dim, dtype=BF16 if cache == BF16 else F16, cache=cache)
    expected = s.want(dim**-0.5)
    hidden = torch.ones(s.pages, s.page, dtype=torch.bool)
    for row, n in ((s.table[0], 297), (s.table[1], 129), (s.ptable[0], 70)):  # all but the last 3 and the last 1 tokens
        for j in range(n):
            hidden[int(row[j // 16]), j % 16] = False
    for pool in (s.k, s.v):
        x = pool.float()
        x[hidden.cuda()] = junk
        pool.copy_(x.to(cache))
    s.prompt()
    check_scores_to_their_own_size(s, expected, rows=(37, 6))


@pytest.mark.parametrize("dim,dtype,cache,window", [(64, F16, F16, 0), (128, BF16, BF16, 0), (128, BF16, E4M3, 5000), (256, F16, F16, 0)])
def test_prompts_of_many_thousand_tokens(w4, dim, dtype, cache, window):  # noqa: F811
    n, before = 20011, 3000
    s = Setup(w4, [n], [n + before], heads=4, kv=2, dim=dim, dtype=dtype, cache=cache, page=32)
    s.prompt(window=window)
    k, v = s.tokens(0)
    rows = [0, 1, 127, 128, n - 2, n - 1, *np.random.RandomState(dim).randint(0, n, 60).tolist()]
    got = s.out, s.lse, s.q
    s.out, s.lse, s.q = (x[rows] for x in got)
    check_scores_to_their_own_size(s, [
        (slice(i, i + 1), rows_attention(f64(s.q[i:i + 1]), k[:before + r + 1], v[:before + r + 1], before + r, dim**-0.5, window),
         before + r + 1) for i, r in enumerate(rows)])
    assert bool((got[0] != 77.0).any(2).all()) and bool((got[1] != 55.0).all())
