"""GPU tests of the operators between the projections at the limits of what they take: infinities beside finite
values, heads of very different size, weights far below the largest, values on a rounding border, strides beyond
31 bits, streams of the caller's."""
import math

import numpy as np
import pytest
import torch

from test_gpu_decode_ops import (BF16, E, E4M3, F16, U, attention_expect, build, check_attention, f64, i32, make_cache,
                                 normal, w4, within)  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ paged_attention: strides
@pytest.mark.parametrize("page,stride", [(16, 2**29), (4, 2**31 - 16)])
@pytest.mark.parametrize("window", [0, 21])
def test_attention_token_strides_beyond_32_bits(w4, page, stride, window):
    # Tokens outermost: those of a page `stride` elements apart, so that a page's last one begins beyond 2^32 elements.
    # The window begins inside a group of 16 tokens.
    pages, kv, D = 20, 2, 16
    flat = torch.empty((page - 1) * stride + 2 * pages * kv * D, dtype=torch.uint8, device="cuda").view(E4M3)
    pools = [flat[x * pages * kv * D:].as_strided((pages, page, kv, D), (kv * D, stride, D, 1)) for x in (0, 1)]
    for seed, pool in enumerate(pools):
        new = normal((pages, page, kv, D), F16, seed, 40.0).to(E4M3)
        for t in range(page):
            pool[:, t].copy_(new[:, t])
    scales = [torch.full((kv,), 0.02, device="cuda") for _ in (0, 1)]
    lens = [8 * page - 3, 37, 1] if page == 16 else [17 * page - 3, 38, 1]
    width = -(-lens[0] // page)
    table = np.random.default_rng(page).permutation(pages * 3).reshape(3, -1)[:, :width] % pages
    q = normal((3, 4, D), F16, 7, 2.5)
    cache = w4.KVCache(*pools, *scales)
    assert cache.k_token == cache.v_token == stride
    check_attention(w4, q, cache, pools, scales, table, lens, page, window=window)
    del flat, pools, cache
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ paged_attention: the softmax's weights
def few_large(w4, dtype, cdtype, score, large, small, requests=912, n=640, page=16):
    """Requests over the same pages: keys 0, 16, .. 112 have a score of `score` and the value `large`, the others a score
    of 0 and the values `small` [kv_heads, D] (8-bit caches: one value for each head). So many requests that a CTA has
    some from end to end: its weights are relative to the largest, which comes first. Returns outputs [requests, kv_heads,
    D] and the part that the others have of the sum of weights."""
    kv, D = small.shape
    cache, pools, scales = make_cache(w4, n // page, page, kv, D, cdtype, 5)
    first = (torch.arange(n, device="cuda").view(n // page, page, 1, 1) % 16 == 0)
    first &= torch.arange(n, device="cuda").view(n // page, page, 1, 1) < 128
    one = torch.ones(n // page, page, kv, D, device="cuda")
    unit = small if cdtype != E4M3 else torch.ones_like(small)
    pools[0].copy_(torch.where(first, one * (score / math.sqrt(D)), one * 0).to(cdtype))
    pools[1].copy_(torch.where(first, one * large, one * unit.cuda()).to(cdtype))
    if cdtype == E4M3:
        scales[0].fill_(1.0)
        scales[1].copy_(small[:, 0])
    table = np.arange(n // page)[None].repeat(requests, 0)
    q = torch.ones(requests, kv, D, dtype=dtype, device="cuda")
    out = w4.w4a16_paged_attention(q, cache, i32(table), i32([n] * requests))
    w = (n - 8) * math.exp(-score)
    return f64(out), w / (8 + w)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_over_one_value_returns_it(w4, dtype):
    # All values of the 8-bit cache stand for 2047/1024. Weights of exp(-3.25) are rounded up by 3.5e-4 each, more than
    # the output's half step there; the sums of 640 weights and products differ by 704 e = 4.2e-5 at most.
    small = torch.full((1, 64), 2047 / 1024)
    got, _ = few_large(w4, dtype, E4M3, 3.25, 1.0, small)
    assert (got == f64(small.to(dtype))).all()


@pytest.mark.parametrize("score", [14.0, 18.0, 20.0])
@pytest.mark.parametrize("dtype,cdtype", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
def test_attention_weights_far_below_the_largest(w4, dtype, cdtype, score):
    # The largest weights' values are 0, so the output is made of weights of 2^-20 to 2^-29 of them. As fp16 operands
    # each is off by 2^-35 of the largest, besides their rounding (half a step with 8-bit caches, 2^-16 otherwise).
    got, share = few_large(w4, dtype, cdtype, score, 0.0, torch.full((2, 64), 28672.0))
    want = 28672.0 * share
    rounding = U[F16] if cdtype == E4M3 else 2.0**-16
    bound = (U[dtype] + rounding + 704 * E) * want + 632 / 8 * 2.0**-35 * 28672.0
    assert np.abs(got - want).max() <= bound


def test_attention_sums_values_as_large_as_fp32_does(w4):
    # 640 values of 2^118 with weights of 1 at most: sums stay below 2^128.
    got, _ = few_large(w4, BF16, BF16, 0.0, 2.0**118, torch.full((1, 64), 2.0**118))
    assert (got == 2.0**118).all()


@pytest.mark.parametrize("dtype,cdtype", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
@pytest.mark.parametrize("scale", [3000.0, 7.3e6, -1.9e12, 1.1e20])
def test_attention_scores_beyond_24_bits(w4, dtype, cdtype, scale):
    # Exact products far apart: the best key's value is the output, and its score the lse, however large it is.
    lens, page, heads = [700, 3, 90], 16, 6
    q, cache, pools, scales, table = build(w4, lens, heads, 2, 64, dtype, cdtype, page, "tokens", 3)
    for s in scales:
        if s is not None:
            s.fill_(1.0)
    q.fill_(3.0)
    g = torch.Generator().manual_seed(1)
    pools[0].copy_(torch.randint(-8, 8, pools[0].shape, generator=g).float().cuda().to(cdtype))
    lse = torch.empty(3, heads, device="cuda")
    out = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens), scale=scale, lse=lse)
    for b, n in enumerate(lens):
        pages = torch.as_tensor(table[b, :-(-n // page)]).cuda()
        k, v = (f64(p.float()[pages]).reshape(-1, 2, 64)[:n] for p in pools)
        score = 3.0 * k.sum(2) * scale
        for h in range(heads):
            mine = score[:, h // 3]
            best = mine == mine.max()
            want = v[best, h // 3].mean(0)
            assert np.abs(f64(out[b, h]) - want).max() <= U[dtype] * np.abs(want).max() + 2.0**-16 * np.abs(v).max()
            assert abs(float(lse[b, h]) - mine.max()) <= 8 * E * abs(mine.max())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("lens", [[50, 300, 1], [20000, 3]])
def test_attention_infinite_values_stay_infinite(w4, dtype, lens):
    page = 16
    q, cache, pools, scales, table = build(w4, lens, 8, 2, 64, dtype, dtype, page, "tokens", 8, q_scale=1.0)
    clean = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens))
    inf = float("inf")
    for b, n in enumerate(lens):
        for j in range(0, n, 7):  # elements 3 and 9: one sign; element 20: one such value; 33: both signs
            pools[1][int(table[b, j // page]), j % page, 1, 3] = inf
            pools[1][int(table[b, j // page]), j % page, 1, 9] = -inf
        at = n // 2
        pools[1][int(table[b, at // page]), at % page, 1, 20] = inf
        pools[1][int(table[b, 0]), 0, 1, 33] = -inf
        pools[1][int(table[b, (n - 1) // page]), (n - 1) % page, 1, 33] = inf
    out = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens))
    want = clean.clone()
    want[:, 4:, 3], want[:, 4:, 9], want[:, 4:, 20] = inf, -inf, inf
    want[:, 4:, 33] = torch.tensor([inf if n == 1 else math.nan for n in lens], device="cuda")[:, None]
    np.testing.assert_array_equal(f64(out), f64(want))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_weights_are_not_rounded_to_the_operands_type(w4, dtype):
    # Weights of exp(-3.25), of which one in 16 bits is 3.5e-4 (fp16) or 1.1e-3 (bf16) too large. As two operands they are
    # exact to 2^-16, sums of 640 terms to 704 e: all outputs but those near a border have to be the correctly rounded
    # ones.
    small = (torch.rand(8, 64, generator=torch.Generator().manual_seed(3)) + 1.0).to(dtype).float()
    got, share = few_large(w4, dtype, dtype, 3.25, 0.0, small)
    half = lambda x: f64(torch.as_tensor(x, dtype=torch.float64).to(dtype))  # noqa: E731
    want, off = f64(small) * share, 2.0**-16 + 704 * E
    sure = half(want * (1 - off)) == half(want * (1 + off))
    once = float(torch.tensor(math.exp(-3.25), dtype=torch.float64).to(dtype)) * math.exp(3.25)
    assert sure.mean() > 0.8 and (half(want * once) != half(want))[sure].mean() > 0.1  # what is asked for is worth asking
    np.testing.assert_array_equal(got[:, sure], half(want)[None, sure].repeat(len(got), 0))


@pytest.mark.parametrize("heads,kv,D", [(8, 1, 128), (32, 2, 64), (8, 1, 256), (5, 1, 48)])
def test_attention_heads_of_any_size_on_8_bit_keys(w4, heads, kv, D):
    # Each head's queries are brought to fp16 by a power of two of their own: neighbours 2^30 larger take nothing away.
    lens, page = [130, 17, 1], 16
    q, cache, pools, scales, table = build(w4, lens, heads, kv, D, BF16, E4M3, page, "tokens", 8)
    q.mul_(torch.exp2(torch.arange(heads, device="cuda") % 5 * -30.0 + 30.0).to(BF16)[:, None])
    check_attention(w4, q, cache, pools, scales, table, lens, page)
    check_attention(w4, q, cache, pools, scales, table, lens, page, cap=4.0)


def test_attention_infinite_and_nan_queries_stay_in_their_head_on_8_bit_keys(w4):
    lens, page = [50, 130], 16
    q, cache, pools, scales, table = build(w4, lens, 16, 1, 128, BF16, E4M3, page, "tokens", 8)
    q[:, 2] *= 2.0**100
    clean = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens))
    q[0, 5, 7], q[1, 9, 3] = float("inf"), float("nan")
    out = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens))
    nan = torch.isnan(out)
    assert nan[0, 5].all() and nan[1, 9].all()
    clean[0, 5], clean[1, 9] = 0, 0
    out[0, 5], out[1, 9] = 0, 0
    assert torch.equal(out, clean)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("k_scale,scale,cap", [(0.0, 0.125, 0.0), (1e-10, 1e-40, 0.0), (0.0, 0.125, 5.0)])
def test_attention_scores_that_vanish_are_all_alike(w4, dtype, k_scale, scale, cap):
    # Keys that stand for 0 (or next to it): the mean of the visible values, in a slice that is not full too.
    lens, page = [21, 1, 300], 16
    q, cache, pools, scales, table = build(w4, lens, 8, 2, 64, dtype, E4M3, page, "tokens", 8)
    scales[0].fill_(k_scale)
    check_attention(w4, q, cache, pools, scales, table, lens, page, scale=scale, cap=cap)


# ------------------------------------------------------------------ rope_append
@pytest.mark.parametrize("rot", [16, 12])
def test_rope_append_divides_by_the_scale(w4, rot):
    # x / scale lies exactly between two e4m3 values: the even one is stored. A product with the rounded reciprocal
    # leaves the border, one way or the other, in 38 of these 256.
    odd = torch.arange(3, 67, 2, dtype=torch.float32)                     # one scale for each head
    cache, pools, scales = make_cache(w4, 1, 16, odd.numel(), 16, E4M3, 1)
    ties = torch.arange(17, 33, 2, dtype=torch.float32).repeat(2) * torch.tensor([1.0, -1.0]).repeat_interleave(8)
    for s in scales:
        s.copy_(odd * 2.0**-8)
    kv = (odd[:, None] * 2.0**-8 * ties).to(F16)[None].cuda()
    assert torch.equal(kv.float().cpu()[0], odd[:, None] * 2.0**-8 * ties)
    q = torch.zeros(1, 32, 16, dtype=F16, device="cuda")
    w4.w4a16_rope_append(q, kv, kv, i32([0]), torch.ones(rot // 2, device="cuda"), cache, torch.tensor([3], device="cuda"))
    want = f64(ties.to(E4M3))[None].repeat(odd.numel(), 0)
    assert set(np.abs(want[0])) == {16, 20, 24, 28, 32}
    for pool in pools:
        np.testing.assert_array_equal(f64(pool)[0, 3], want)


@pytest.mark.parametrize("rot", [16, 12])
def test_rope_append_stores_the_rounded_quotient_of_every_value(w4, rot):
    # Every finite fp16 value as a value of the cache, over scales of different mantissas and sizes.
    x = torch.arange(2**16, dtype=torch.int32).to(torch.int16).view(F16)
    x = x[torch.isfinite(x)]
    rows = x.numel() // 16
    scale = torch.tensor([1.0, 1 / 3, 0.0213, 2 - 2.0**-23, 1 + 2.0**-23, 7.7e4, 3.1e-7, 2.0**-60 * 1.7])
    cache, pools, scales = make_cache(w4, -(-rows // 16), 16, scale.numel(), 16, E4M3, 1)
    for s in scales:
        s.copy_(scale)
    kv = x.view(rows, 1, 16).expand(rows, scale.numel(), 16).contiguous().cuda()
    q = torch.zeros(rows, 8, 16, dtype=F16, device="cuda")
    w4.w4a16_rope_append(q, kv, kv, i32(np.zeros(rows)), torch.ones(rot // 2, device="cuda"), cache, torch.arange(rows, device="cuda"))
    want = f64((kv.float().cpu() / scale[:, None]).clamp(-448, 448).to(E4M3))
    for pool in pools:
        np.testing.assert_array_equal(f64(pool).reshape(-1, scale.numel(), 16)[:rows], want)


@pytest.mark.parametrize("rot", [32, 28])
@pytest.mark.parametrize("pairs", [False, True])
def test_rope_append_frequencies_that_are_no_numbers(w4, rot, pairs):
    cache, pools, _ = make_cache(w4, 1, 16, 2, 64, F16, 1)
    qkv = normal((3, 8, 64), F16, 2)
    freq = w4.w4a16_rope_frequencies(rot, 1e4)
    args = i32([0, 5, -7]), cache, torch.arange(3, device="cuda")
    run = lambda f: w4.w4a16_rope_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], args[0], f.cuda(), *args[1:], interleaved=pairs)  # noqa: E731
    clean = [run(freq)] + [p[0, :3].clone() for p in pools]
    freq[2], freq[5], freq[6] = float("inf"), float("nan"), -float("inf")
    got = [run(freq)] + [p[0, :3] for p in pools]
    gone = [x for i in (2, 5, 6) for x in ((2 * i, 2 * i + 1) if pairs else (i, i + rot // 2))]
    for x, y in zip(got[:2], clean[:2]):
        assert torch.isnan(x[..., gone]).all()
        rest = [i for i in range(64) if i not in gone]
        assert torch.equal(x[..., rest], y[..., rest])
    assert torch.equal(got[2], clean[2])


# ------------------------------------------------------------------ kv_extend
def extend(w4, lens, new, table, free, count, page=4, n=16, spacing=0):
    t = [i32(x) for x in (lens, new, table, free, [count])]
    slots = torch.full((n,), 77, dtype=torch.int64, device="cuda")
    positions, refused = i32(np.full(n, 77)), i32(np.full(len(lens), 77))
    w4.w4a16_kv_extend(*t, page, slots, positions, refused, spacing=spacing)
    return t, slots.tolist(), positions.tolist(), refused.tolist()


def test_kv_extend_names_pages_that_are_none(w4):
    ok, bad = w4.W4A16_OK, w4.W4A16_ERR_INVALID_ARG
    # A page of -1 in a running request's row, which its next token would go to.
    t, slots, positions, refused = extend(w4, [5, 5], [1, 1], [[0, -1], [2, 3]], [9, 9], 0, n=4)
    assert w4.w4a16_device_error() == bad
    assert slots == [-1, 13, -1, -1] and positions[:2] == [5, 5] and refused == [0, 0]
    # One that an ended request gives back, and that goes on to the next: both calls say so.
    t, slots, _, _ = extend(w4, [6, 0], [-1, 0], [[1, -3], [0, 0]], [9, 9, 9], 1, n=4)
    assert w4.w4a16_device_error() == bad and t[3].tolist() == [9, 1, -3] and t[4].tolist() == [3]
    t, slots, _, refused = extend(w4, [0], [6], [[0, 0]], [9, 1, -3], 3, n=8)
    assert w4.w4a16_device_error() == bad and refused == [0]
    assert slots == [-1] * 4 + [4, 5, -1, -1] and t[2].tolist() == [[-3, 1]]
    # Pages that no token of the step goes to are not looked at.
    extend(w4, [5, 5], [1, 0], [[-1, 1], [-1, -1]], [-1, -1], 0, n=4)
    assert w4.w4a16_device_error() == ok


def test_kv_extend_names_lengths_of_ended_requests_out_of_range(w4):
    ok, bad = w4.W4A16_OK, w4.W4A16_ERR_INVALID_ARG
    for length, status in ((-1, bad), (9, bad), (8, ok), (0, ok), (2**31 - 1, bad)):
        t, _, _, refused = extend(w4, [length, 3], [-1, 1], [[1, 2], [3, 4]], [9] * 4, 1)
        assert w4.w4a16_device_error() == status
        held = 0 if length <= 0 else 2
        assert t[0].tolist() == [0, 4] and t[4].tolist() == [1 + held] and refused == [0, 0]
    # Running requests' are answered by `refused` alone.
    extend(w4, [-1, 9], [1, 1], [[1, 2], [3, 4]], [9] * 4, 1)
    assert w4.w4a16_device_error() == ok


# ------------------------------------------------------------------ strides that step over nothing
def test_strides_of_single_entries_say_nothing(w4):
    # One request, one head, a cache of one page: strides between entries that there are none of may be anything.
    odd = lambda t, *steps: torch.as_strided(t, t.shape, (*steps, 1))  # noqa: E731
    pools = [normal((1, 16, 1, 64), F16, s) for s in (1, 2)]
    cache, same = w4.KVCache(*[odd(p, 1027, 64, 13) for p in pools]), w4.KVCache(*pools)
    q, k, v = (normal((1, 1, 64), F16, s) for s in (3, 4, 5))
    args = i32([7]), torch.ones(32, device="cuda")
    slot = torch.tensor([9], device="cuda")
    out = torch.zeros(1, 1, 64, dtype=F16, device="cuda")
    want = w4.w4a16_rope_append(q, k, v, *args, same, slot)
    kept = [p.clone() for p in pools]
    w4.w4a16_rope_append(odd(q, 77, 3), odd(k, 5, 9), odd(v, 1, 1), *args, cache, slot, out=odd(out, 65, 67))
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(pools, kept))
    table, lens = i32([[0]]), i32([10])
    want = w4.w4a16_paged_attention(q, same, table, lens)
    w4.w4a16_paged_attention(odd(q, 77, 3), cache, table, lens, out=odd(out, 65, 67))
    assert torch.equal(out, want)


# ------------------------------------------------------------------ streams of the caller's
def on_side_stream(call, as_number):
    """call(stream) while the current stream is busy and its free memory holds ones; the result."""
    torch.cuda.synchronize()
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (1 << 24, 1 << 23, 1 << 20, 1 << 14)]
    side = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)
    del junk
    out = call(side.cuda_stream if as_number else side)
    side.synchronize()
    early = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert early, "the current stream was to be busy all the while"
    return out


@pytest.mark.parametrize("as_number", [False, True])
def test_calls_on_another_stream_than_the_current_one(w4, as_number):
    lens, page = [3000, 9, 777], 16
    q, cache, pools, scales, table = build(w4, lens, 8, 2, 64, F16, F16, page, "tokens", 8)
    t, n = i32(table), i32(lens)
    want = w4.w4a16_paged_attention(q, cache, t, n)
    assert torch.equal(on_side_stream(lambda s: w4.w4a16_paged_attention(q, cache, t, n, stream=s), as_number), want)
    h, y, gm = normal((5, 64), F16, 1), normal((5, 64), F16, 2), normal((64,), F16, 3)
    want = w4.w4a16_residual_rmsnorm(h, y, gm)
    got = on_side_stream(lambda s: w4.w4a16_residual_rmsnorm(h, y, gm, stream=s), as_number)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    args = i32([5, 6, 7]), torch.ones(32, device="cuda"), cache, torch.tensor([0, 1, 2], device="cuda")
    want = w4.w4a16_rope_append(q, q[:, :2], q[:, 2:4], *args)
    assert torch.equal(on_side_stream(lambda s: w4.w4a16_rope_append(q, q[:, :2], q[:, 2:4], *args, stream=s), as_number), want)
    g = torch.Generator(device="cuda").manual_seed(1)
    weight = torch.randint(0, 256, (256, 128), dtype=torch.uint8, device="cuda", generator=g)
    scale = torch.full((256, 2), 0.01, dtype=F16, device="cuda")
    rep, a, gm = w4.w4a16_repack(weight), normal((5, 256), F16, 4), normal((256,), F16, 5)
    side = lambda s: {"stream": s}  # noqa: E731
    for call in (lambda kw: w4.w4a16_repack(weight, **kw),
                 lambda kw: w4.w4a16_gemm(a, rep, scale, None, 128, **kw),
                 lambda kw: w4.w4a16_gemm_swiglu(a, rep, scale, None, rep, scale, None, 128, **kw),
                 lambda kw: w4.w4a16_gemm_swiglu(a, rep, scale, None, rep, scale, None, 128, fused=False, **kw),
                 lambda kw: w4.w4a16_gemm_rmsnorm(a, gm, 1e-5, rep, scale, None, 128, **kw),
                 lambda kw: w4.w4a16_gemm_swiglu_rmsnorm(a, gm, 1e-5, rep, scale, None, rep, scale, None, 128, **kw),
                 lambda kw: w4.w4a16_gemm_swiglu_unfused_static(a, rep, scale, None, rep, scale, None, 128, **kw)):
        want = call({})
        assert torch.equal(on_side_stream(lambda s: call(side(s)), as_number), want)
