"""GPU parity of the operators between the projections (kv_extend, rope_append,
paged_attention, residual_rmsnorm) with their float64 statements.

Error bounds are counted in half steps of the output's type (u: fp16 2^-11, bf16
2^-8, e4m3 2^-4 and half the subnormal step) and in fp32 roundings (e = 2^-24) of
the sums of magnitudes that the oracle returns:
  rope       u |x'| + 16 e (|x_a| + |x_b|): two products, a sum, a bias, cos and sin
             of an angle that is itself rounded to fp32 (up to pi e, and 2 ulp each)
  attention  a score is off by (D + 8) e max_j scale sum |q k|, which turns into the
             same relative error of every weight; the weights are rounded to the
             operands' type at most once (u_p = u), and sums over n tokens add n e
  norm       the sum of squares (a tree over at most 64 serial terms) 96 e, halved
             by the root; 8 further roundings
"""
import math

import numpy as np
import pytest
import torch

from oracle import decode_ops as ref

pytestmark = pytest.mark.gpu
E = 2.0**-24
U = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture
def w4(gpu_lib):
    yield gpu_lib
    gpu_lib.w4a16_set_launch_overlap(False)
    assert gpu_lib.w4a16_device_error() == gpu_lib.W4A16_OK


def f64(t):
    return t.float().cpu().double().numpy() if t.dtype != torch.float64 else t.cpu().numpy()


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


def within(got, want, bound, label):
    got, want = f64(got) if torch.is_tensor(got) else got, np.asarray(want)
    both = np.isfinite(want)
    assert np.array_equal(got[~both], want[~both], equal_nan=True), label
    off = np.abs(got[both] - want[both]) - np.broadcast_to(bound, want.shape)[both]
    worst = off.max() if off.size else 0.0
    assert worst <= 0, f"{label}: {worst} over the bound"


# ------------------------------------------------------------------ kv_extend
def run_extend(w4, lens, new, table, free, count, page, n_slots, in_place=False, spacing=0):
    t = dict(lens=i32(lens), new=i32(new), table=i32(table), free=i32(free), count=i32([count]))
    batch = len(lens)
    slots = torch.full((n_slots,), 77, dtype=torch.int64, device="cuda")
    positions, refused = i32(np.full(n_slots, 77)), i32(np.full(batch, 77))
    lens_out, count_out = (t["lens"], t["count"]) if in_place else (i32(np.full(batch, 77)), i32([77]))
    w4.w4a16_kv_extend(t["lens"], t["new"], t["table"], t["free"], t["count"], page, slots, positions, refused,
                       lens_out=lens_out, count_out=count_out, spacing=spacing)
    torch.cuda.synchronize()
    return dict(table=t["table"], free_pages=t["free"], free_count_out=count_out[0], lens_out=lens_out, refused=refused,
                slots=slots, positions=positions)


def check_extend(w4, lens, new, table, free, count, page, n_slots, in_place=False, spacing=0):
    want = ref.kv_extend(lens, new, table, free, count, page, n_slots, spacing)
    got = run_extend(w4, lens, new, table, free, count, page, n_slots, in_place, spacing)
    for name, x in want.items():
        np.testing.assert_array_equal(got[name].cpu().numpy(), x, err_msg=name)
    return want


def draw_extend(rng, batch, page, max_pages, share, tight=False):
    """Requests, their table and the free list; `share` of them get one token each, the others end, wait or
    get a prompt."""
    room = max_pages * page
    lens = rng.integers(0, room, batch)
    kind = rng.random(batch)
    prompt = rng.integers(0, room // 2 + 2, batch)
    new = np.where(kind < share, 1, np.where(kind < share + 0.1, -1, np.where(kind < share + 0.15, 0, prompt)))
    if tight:  # few end, and only they give pages
        new = np.where((new < 0) & (np.arange(batch) % 8 > 0), 1, new)
    held = -(-lens // page)
    pool = int(held.sum() + (-(-prompt // page) + 1).sum()) + 8
    order = rng.permutation(pool)
    table = np.full((batch, max_pages), -1, dtype=np.int64)
    at = 0
    for b in range(batch):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(pool, -1, dtype=np.int64)
    free[:pool - at] = order[at:]
    return lens, new, table, free, 0 if tight else pool - at


@pytest.mark.parametrize("batch,page,max_pages,share,tight", [
    (1, 16, 4, 1.0, False), (1, 1, 3, 0.0, False), (7, 1, 40, 0.5, False), (33, 16, 9, 0.9, False),
    (200, 24, 12, 0.4, True), (1023, 16, 6, 0.7, False), (1025, 8, 6, 0.8, True), (3001, 16, 4, 0.6, True),
    (8192, 16, 3, 0.9, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_kv_extend(w4, batch, page, max_pages, share, tight, in_place):
    rng = np.random.default_rng(batch + page)
    a = draw_extend(rng, batch, page, max_pages, share, tight)
    n = int(np.maximum(a[1], 0).sum())
    want = check_extend(w4, *a, page, n + 5, in_place)
    if tight:
        assert (want["refused"] == 1).any()


@pytest.mark.parametrize("batch,spacing,short", [(1, 1, 0), (50, 1, 0), (50, 3, 7), (700, 64, 0), (8192, 2, 100)])
def test_kv_extend_with_spacing(w4, batch, spacing, short):
    rng = np.random.default_rng(batch + spacing)
    a = draw_extend(rng, batch, 16, 5, 0.7)
    want = check_extend(w4, *a, 16, batch * spacing - short, spacing=spacing)
    assert spacing < 2 or (want["refused"] == 2).any()


def test_kv_extend_refuses_what_does_not_fit(w4):
    # Table rows of 3 pages of 4 tokens; a negative and an overlong length; a slots buffer that ends early.
    table = np.arange(24).reshape(8, 3)
    lens, new = [12, -5, 40, 11, 0, 3, 13, 2], [1, 1, 1, 2, 12, 1, 0, 1]
    want = check_extend(w4, lens, new, table, np.arange(100, 130), 30, 4, 17)
    assert want["refused"].tolist() == [2, 2, 2, 2, 0, 2, 2, 2]
    check_extend(w4, lens, new, table, np.arange(100, 130), 30, 4, 64)
    check_extend(w4, lens, new, table, np.arange(100, 130), 30, 4, 0)


def test_kv_extend_counts_out_of_range(w4):
    table = np.arange(8).reshape(2, 4)
    check_extend(w4, [4, 6], [1, -1], table, np.arange(10, 16), -3, 4, 4)       # nothing but what is given back
    check_extend(w4, [4, 6], [1, -1], table, np.arange(10, 16), 99, 4, 4)       # more than the list holds
    check_extend(w4, [16, 16], [-1, -1], table, np.arange(10, 16), 3, 4, 4)     # more given back than it holds
    check_extend(w4, [0, 0], [2**31 - 1, 2**31 - 1], table, np.arange(10, 16), 3, 4, 4)


def test_kv_extend_steps_reuse_pages(w4):
    # A small server in place: requests grow, end and start again; no page ever has two owners.
    rng = np.random.default_rng(5)
    batch, page, max_pages, pool = 9, 4, 8, 40
    lens, table = i32(np.zeros(batch)), i32(np.full((batch, max_pages), -1))
    free, count = i32(rng.permutation(pool)), i32([pool])
    slots = torch.empty(64, dtype=torch.int64, device="cuda")
    positions, refused = i32(np.zeros(64)), i32(np.zeros(batch))
    for step in range(40):
        new = np.where(rng.random(batch) < 0.15, -1, rng.integers(0, 6, batch))
        want = ref.kv_extend(lens.tolist(), new, table.cpu().numpy(), free.cpu().numpy(), int(count), page, 64)
        w4.w4a16_kv_extend(lens, i32(new), table, free, count, page, slots, positions, refused)
        torch.cuda.synchronize()
        for name, x in dict(table=table, free_pages=free, lens_out=lens, slots=slots, refused=refused).items():
            np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=f"step {step}: {name}")
        owned = [int(p) for b in range(batch) for p in table[b, :-(-int(lens[b]) // page)]]
        owned += free[:int(count)].tolist()
        assert sorted(owned) == list(range(pool))


# ------------------------------------------------------------------ rope_append
def make_cache(w4, pages, page, kv, D, dtype, seed, order="tokens", scale_seed=None):
    inner = (kv, page) if order == "heads" else (page, kv)
    pools = [normal((pages, *inner, D), F16, seed + i, 40.0 if dtype == E4M3 else 1.0).to(dtype) for i in (0, 1)]
    if order == "heads":
        pools = [x.transpose(1, 2) for x in pools]
    if order == "joined":  # keys and values side by side in one allocation
        both = normal((pages, page, 2, kv, D), F16, seed, 40.0 if dtype == E4M3 else 1.0).to(dtype)
        pools = [both[:, :, 0], both[:, :, 1]]
    scales = [None, None]
    if dtype == E4M3:
        scales = [torch.rand(kv, generator=torch.Generator().manual_seed(seed + 7 + i)).cuda() * 0.02 + 0.015
                  for i in (0, 1)]
    return w4.KVCache(*pools, *scales), pools, scales


ROPE = [  # rows, heads, kv_heads, D, rot, pairs, type, cache, bias
    (1, 40, 8, 128, 128, False, F16, F16, True), (3, 32, 2, 128, 64, True, F16, E4M3, True),
    (67, 40, 8, 128, 128, False, BF16, BF16, False), (5, 9, 3, 64, 64, True, BF16, E4M3, False),
    (4, 20, 4, 80, 40, False, F16, F16, True), (4, 20, 4, 80, 20, True, BF16, BF16, True),
    (2, 16, 8, 256, 256, False, F16, E4M3, False), (2, 6, 1, 96, 0, False, F16, F16, True),
    (9, 1, 1, 8, 8, False, F16, F16, False), (9, 3, 3, 24, 4, True, BF16, BF16, True),
    (300, 14, 2, 64, 64, False, F16, F16, False)]


def rope_expect(qkv, bias, heads, kv, positions, freq, rot, pairs, m):
    x = f64(qkv) + (0 if bias is None else f64(bias).reshape(1, -1, qkv.shape[2]))
    turned, mag = ref.rope(x[:, :heads + kv], positions.cpu().numpy(), freq.cpu().numpy(), rot, pairs, m)
    return turned[:, :heads], turned[:, heads:], x[:, heads + kv:], mag[:, :heads], mag[:, heads:]


def cache_bound(want, mag, dtype):
    return (2.0**-4 * np.abs(want) + 2.0**-10 if dtype == E4M3 else U[dtype] * np.abs(want)) + 20 * E * mag


@pytest.mark.parametrize("rows,heads,kv,D,rot,pairs,dtype,cdtype,bias", ROPE)
@pytest.mark.parametrize("overlap", [False, True])
def test_rope_append(w4, rows, heads, kv, D, rot, pairs, dtype, cdtype, bias, overlap):
    w4.w4a16_set_launch_overlap(overlap)
    page, pages, m = 16, rows // 8 + 2, 1.25
    cache, pools, scales = make_cache(w4, pages, page, kv, D, cdtype, 3, "heads" if rows % 2 else "joined")
    qkv = normal((rows, heads + 2 * kv, D), dtype, 11, 2.0)
    b = normal(((heads + 2 * kv) * D,), dtype, 12, 0.5) if bias else None
    freq = w4.w4a16_rope_frequencies(rot, 10000.0).cuda() if rot else torch.empty(0, device="cuda")
    rng = np.random.default_rng(rows)
    positions = i32(rng.integers(0, 200000, rows))
    slots = torch.from_numpy(rng.permutation(pages * page)[:rows]).cuda()
    if rows > 2:
        slots[1] = -1
    before = [f64(p).copy() for p in pools]
    out = w4.w4a16_rope_append(qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], positions, freq, cache, slots,
                               interleaved=pairs, mscale=m, bias=b)
    torch.cuda.synchronize()
    q, k, v, q_mag, k_mag = rope_expect(qkv, b, heads, kv, positions, freq, rot, pairs, m)
    within(out, q, U[dtype] * np.abs(q) + 16 * E * q_mag, "q")
    at = slots.cpu().numpy()
    for pool, old, new, mag, scale in ((pools[0], before[0], k, k_mag, scales[0]), (pools[1], before[1], v, np.abs(v), scales[1])):
        if scale is not None:
            s = f64(scale)[None, :, None]
            new, mag = np.clip(new / s, -ref.E4M3_MAX, ref.E4M3_MAX), mag / s
        got = f64(pool)
        real = at >= 0
        rowsel = (at[real] // page, at[real] % page)
        within(got[rowsel], new[real], cache_bound(new[real], mag[real], cdtype), "cache")
        old[rowsel] = got[rowsel]
        np.testing.assert_array_equal(got, old, err_msg="other slots")


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [128, 36])
def test_rope_append_in_place_and_repeatable(w4, pairs, rot):
    cache, _, _ = make_cache(w4, 4, 16, 2, 128, F16, 1)
    qkv = normal((5, 8, 128), F16, 2)
    freq = w4.w4a16_rope_frequencies(rot, 10000.0).cuda()
    positions, slots = i32(np.arange(5) * 1000), torch.arange(5, device="cuda")
    args = (positions, freq, cache, slots)
    out = [w4.w4a16_rope_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], *args, interleaved=pairs) for _ in (0, 1)]
    q = qkv[:, :4].clone()
    w4.w4a16_rope_append(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], *args, interleaved=pairs, out=qkv[:, :4])
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], qkv[:, :4]) and not torch.equal(q, out[0])


def test_rope_append_far_positions(w4):
    # The product of position and frequency is reduced exactly; a frequency above a turn and a negative one too.
    cache, _, _ = make_cache(w4, 4, 16, 1, 64, F16, 1)
    positions = i32([0, 1, 2**20 - 1, 2**24 + 1, 2**31 - 1, -1, -(2**31)])
    n = positions.numel()
    qkv = normal((n, 3, 64), F16, 4)
    freq = w4.w4a16_rope_frequencies(64, 1e6)
    freq[1], freq[2], freq[3] = 7.3, -0.61, 0.0
    freq = freq.cuda()
    out = w4.w4a16_rope_append(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], positions, freq, cache, torch.arange(n, device="cuda"))
    q, _, _, mag, _ = rope_expect(qkv, None, 1, 1, positions, freq, 64, False, 1.0)
    # 2^-53 of a turn (times 7.3 / 2 pi) at a distance of 2^31 is 2^-21.8 turns
    within(out, q, U[F16] * np.abs(q) + (16 * E + 2 * math.pi * 2.0**-21.7) * mag, "q")


def test_rope_append_scale_saturates_and_nan_stays(w4):
    cache, pools, _ = make_cache(w4, 1, 16, 1, 16, E4M3, 1)
    qkv = torch.zeros(2, 3, 16, dtype=F16, device="cuda")
    qkv[0, 1], qkv[0, 2, 0], qkv[0, 2, 1], qkv[1, 2, 2] = 60000.0, -60000.0, float("inf"), float("nan")
    w4.w4a16_rope_append(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], i32([0, 0]), torch.ones(8, device="cuda"), cache,
                         torch.arange(2, device="cuda"))
    got = f64(pools[0])[0, 0, 0], f64(pools[1])[0, 0, 0], f64(pools[1])[0, 1, 0]
    assert (got[0] == 448).all() and got[1][0] == -448 and got[1][1] == 448
    assert np.isnan(got[2][2]) and not np.isnan(np.delete(got[2], 2)).any()


def test_rope_append_slot_beyond_the_cache_is_an_error(w4):
    cache, pools, _ = make_cache(w4, 2, 16, 1, 64, F16, 1)
    before = [p.clone() for p in pools]
    qkv = normal((3, 3, 64), F16, 4)
    slots = torch.tensor([32, 2**40, -5], device="cuda")
    w4.w4a16_rope_append(qkv[:, :1], qkv[:, 1:2], qkv[:, 2:], i32([0, 0, 0]), torch.ones(32, device="cuda"), cache, slots)
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, pools))


# ------------------------------------------------------------------ paged_attention
def build(w4, lens, heads, kv, D, dtype, cdtype, page, order, seed, q_scale=2.5, spare=3):
    """Queries, a cache with shuffled pages, the table (with garbage behind each request's pages)."""
    rng = np.random.default_rng(seed)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    cache, pools, scales = make_cache(w4, pages, page, kv, D, cdtype, seed, order)
    perm = rng.permutation(pages)
    width = max(1, max(held)) + 1
    table = rng.integers(-5, pages + 5, (len(lens), width))
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    q = normal((len(lens), heads, D), dtype, seed + 100, q_scale)
    return q, cache, pools, scales, table


def tokens(pool, scale, table, b, n, page):
    x = f64(pool[torch.as_tensor(table[b, :-(-n // page)]).cuda()] if pool.dtype != E4M3 else
            pool.view(torch.uint8)[torch.as_tensor(table[b, :-(-n // page)]).cuda()].view(E4M3))
    x = x.reshape(-1, *x.shape[2:])[:n]
    return x if scale is None else x * f64(scale)[None, :, None]


def attention_expect(q, pools, scales, table, lens, page, scale, window=0, cap=0.0, drop=None):
    """drop(b, j): whether token j is left out. Returns out, lse, bound of out, bound of lse."""
    B, H, D = q.shape
    kv = pools[0].shape[2]
    g, u = H // kv, U[q.dtype]
    out, lse, bo, bl = np.zeros((B, H, D)), np.full((B, H), -np.inf), np.zeros((B, H, D)), np.zeros((B, H))
    qd = f64(q)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = (tokens(p, s, table, b, n, page) for p, s in zip(pools, scales))
        keep = np.arange(n) >= (max(0, n - window) if window else 0)
        if drop is not None:
            keep &= ~np.array([drop(b, j) for j in range(n)])
        k, v = k[keep], v[keep]
        for h in range(kv):
            r = slice(h * g, (h + 1) * g)
            out[b, r], lse[b, r], mean, size = ref.attention(qd[b, r], k[:, h], v[:, h], scale, cap)
            ds = ((D + 8) * E * size)[:, None]
            bo[b, r] = u * np.abs(out[b, r]) + (u + 2 * ds + (len(k) + 64) * E) * mean
            bl[b, r] = ds[:, 0] + (len(k) + 64) * E + 8 * E * np.abs(lse[b, r])
    return out, lse, bo, bl


def check_attention(w4, q, cache, pools, scales, table, lens, page, scale=None, window=0, cap=0.0, **kw):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    lse = torch.full(q.shape[:2], 77.0, device="cuda")
    out = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens), scale=scale, window=window, softcap=cap, lse=lse, **kw)
    torch.cuda.synchronize()
    want, want_lse, bo, bl = attention_expect(q, pools, scales, table, lens, page, scale, window, cap)
    within(lse, want_lse, bl, "lse")
    within(out, want, bo, "out")
    return out, lse


HEADS = [(40, 8, 128), (32, 2, 128), (8, 8, 64), (24, 1, 64), (16, 8, 256), (6, 2, 96), (20, 4, 80), (71, 1, 64),
         (3, 3, 8), (2, 1, 16)]
LENS = [1, 0, 15, 16, 17, 63, 64, 65, 130, 257, 0, 1000]


@pytest.mark.parametrize("heads,kv,D", HEADS)
@pytest.mark.parametrize("dtype,cdtype", [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3)])
def test_paged_attention(w4, heads, kv, D, dtype, cdtype):
    if cdtype == E4M3 and D % 16:
        pytest.skip("8-bit heads are multiples of 16")
    a = build(w4, LENS, heads, kv, D, dtype, cdtype, 16, "tokens", heads + D)
    check_attention(w4, *a, LENS, 16)


@pytest.mark.parametrize("page,order", [(1, "tokens"), (3, "heads"), (8, "joined"), (24, "tokens"), (64, "heads"),
                                        (128, "tokens"), (1024, "joined")])
@pytest.mark.parametrize("cdtype", [F16, E4M3])
def test_paged_attention_pages(w4, page, order, cdtype):
    lens = [5, 129, 0, 700, 64]
    a = build(w4, lens, 10, 2, 128, F16, cdtype, page, order, page)
    check_attention(w4, *a, lens, page)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 100, 5000])
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_paged_attention_window_and_cap(w4, window, cap):
    lens = [0, 1, 2, 16, 18, 64, 65, 300, 1111]
    a = build(w4, lens, 8, 4, 64, BF16, BF16, 16, "tokens", window)
    check_attention(w4, *a, lens, 16, window=window, cap=cap)


@pytest.mark.parametrize("n,heads,kv,cdtype", [(40000, 4, 1, F16), (70001, 16, 1, E4M3), (200003, 2, 1, F16)])
def test_paged_attention_long(w4, n, heads, kv, cdtype):
    lens = [n, 3]
    a = build(w4, lens, heads, kv, 128, F16, cdtype, 64, "tokens", 9)
    check_attention(w4, *a, lens, 64)


def test_paged_attention_many_requests(w4):
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    a = build(w4, lens, 4, 2, 64, F16, F16, 16, "heads", 4)
    check_attention(w4, *a, lens, 16)


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.3, 40.0])
def test_paged_attention_scores_of_any_size(w4, scale):
    lens = [300, 33, 1]
    a = build(w4, lens, 8, 2, 64, F16, F16, 16, "tokens", 21)
    check_attention(w4, *a, lens, 16, scale=scale)


def test_paged_attention_one_key_far_above_many(w4):
    # One score far above thousands of equal ones: their small weights still add up.
    lens, page = [8000], 16
    q, cache, pools, scales, table = build(w4, lens, 1, 1, 64, F16, F16, page, "tokens", 3)
    pools[0].zero_()
    pools[1].fill_(1.0)
    q.fill_(1.0)
    t = int(table[0, 100])
    pools[0][t, 5] = 9.0 / 8.0  # score 9 with scale 1/8
    pools[1][t, 5] = 0.0
    out, _ = check_attention(w4, q, cache, pools, scales, table, lens, page)
    want = 7999 / (7999 + math.exp(9.0))
    assert abs(float(out.float().mean()) - want) < 2 * 2.0**-11


@pytest.mark.parametrize("dtype,cdtype", [(F16, F16), (BF16, BF16), (F16, E4M3)])
@pytest.mark.parametrize("window", [0, 40])
def test_paged_attention_ignores_what_is_not_visible(w4, dtype, cdtype, window):
    lens, page = [37, 1, 100, 0, 64], 16
    q, cache, pools, scales, table = build(w4, lens, 8, 2, 64, dtype, cdtype, page, "tokens", 8)
    clean = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens), window=window).clone()
    bad = [float("nan")] if cdtype == E4M3 else [float("nan"), float("inf"), -float("inf"), float(torch.finfo(dtype).min)]
    for x in bad:
        for pool in pools:
            seen = torch.zeros(pool.shape[:2], dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(max(0, n - window) if window else 0, n):
                    seen[int(table[b, j // page]), j % page] = True
            raw = pool.view(torch.uint8) if cdtype == E4M3 else pool
            raw[~seen.cuda()] = 0x7F if cdtype == E4M3 else x
        got = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens), window=window)
        torch.cuda.synchronize()
        assert torch.equal(got, clean)


def test_paged_attention_nan_stays_in_its_request_and_head(w4):
    lens, page = [50, 50], 16
    q, cache, pools, scales, table = build(w4, lens, 8, 2, 64, F16, F16, page, "tokens", 8)
    pools[0][int(table[0, 1]), 3, 1, 7] = float("nan")
    out = w4.w4a16_paged_attention(q, cache, i32(table), i32(lens))
    nan = torch.isnan(out).cpu()
    assert nan[0, 4:].all() and not nan[0, :4].any() and not nan[1].any()


def test_paged_attention_bad_pages_and_lengths(w4):
    lens, page = [100, 40, 33], 16
    q, cache, pools, scales, table = build(w4, lens, 4, 2, 64, F16, F16, page, "tokens", 8)
    bad = table.copy()
    bad[0, 2], bad[1, 0], bad[2, 2] = pools[0].shape[0], -1, 2**31 - 1
    lse = torch.empty(3, 4, device="cuda")
    out = w4.w4a16_paged_attention(q, cache, i32(bad), i32(lens), lse=lse)
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    gone = {0: 2, 1: 0, 2: 2}
    want, want_lse, bo, bl = attention_expect(q, pools, scales, table, lens, page, 0.125, drop=lambda b, j: j // page == gone[b])
    within(lse, want_lse, bl, "lse")
    within(out, want, bo, "out")
    # lengths: negative counts as none, one beyond the table as the table's room
    full = table[:, :3].copy()
    out = w4.w4a16_paged_attention(q, cache, i32(full), i32([10**9, -1, 33]))
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    same = w4.w4a16_paged_attention(q, cache, i32(full), i32([48, 0, 33]))
    torch.cuda.synchronize()
    assert torch.equal(out, same) and not out[1].any()


def test_paged_attention_views_streams_and_workspaces(w4):
    lens, page = [200, 9, 77], 16
    q, cache, pools, scales, table = build(w4, lens, 8, 2, 64, F16, F16, page, "joined", 8)
    wide = torch.zeros(3, 20, 72, dtype=F16, device="cuda")
    wide[:, 5:13, :64] = q
    ws = torch.zeros(w4.w4a16_paged_attention_workspace_bytes(8, 64, 1, 256), dtype=torch.uint8, device="cuda")
    out = torch.zeros(3, 20, 72, dtype=F16, device="cuda")
    t, n = i32(table), i32(lens)
    want, _ = check_attention(w4, q, cache, pools, scales, table, lens, page)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.w4a16_paged_attention(wide[:, 5:13, :64], cache, t, n, out=out[:, 5:13, :64], workspace=ws)
        # the same workspace, not cleared, for other shapes
        big = build(w4, [3000] * 5, 12, 1, 128, BF16, BF16, 16, "tokens", 2)
        check_attention(w4, *big, [3000] * 5, 16, workspace=ws)
        w4.w4a16_paged_attention(wide[:, 5:13, :64], cache, t, n, out=wide[:, 5:13, :64], workspace=ws)  # in place
    torch.cuda.synchronize()
    assert torch.equal(out[:, 5:13, :64], want) and torch.equal(wide[:, 5:13, :64], want)
    out[:, 5:13, :64] = 0
    assert not out.any()


def test_paged_attention_offsets_beyond_32_bits(w4):
    # Pages 2^25 elements apart: page 99 begins beyond 2^31 elements (and 2^32 bytes).
    page, D, pages = 16, 64, 100
    flat = torch.zeros((pages - 1) * 2**25 + page * D, dtype=F16, device="cuda")
    k = flat.as_strided((pages, page, 1, D), (2**25, D, D, 1))
    v = torch.empty(pages, page, 1, D, dtype=F16, device="cuda")
    k.copy_(normal((pages, page, 1, D), F16, 1))
    v.copy_(normal((pages, page, 1, D), F16, 2))
    cache = w4.KVCache(k, v)
    table, lens = np.array([[99, 3, 64, 98]]), [60]
    check_attention(w4, normal((1, 4, D), F16, 3), cache, [k, v], [None, None], table, lens, page)
    del flat, k
    torch.cuda.empty_cache()


def test_paged_attention_repeats_bit_for_bit_with_and_without_overlap(w4):
    lens = [5000, 1, 300, 0, 9000]
    a = build(w4, lens, 10, 2, 128, F16, F16, 16, "tokens", 8)
    ws = torch.zeros(w4.w4a16_paged_attention_workspace_bytes(5, 10, 2, 128), dtype=torch.uint8, device="cuda")
    t, n = i32(a[4]), i32(lens)
    outs = []
    for i in range(6):
        w4.w4a16_set_launch_overlap(i >= 3)
        outs.append(w4.w4a16_paged_attention(a[0], a[1], t, n, workspace=ws))
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs)


# ------------------------------------------------------------------ residual_rmsnorm
NORM = [  # M, K, type, stream, post, gate, gamma, alpha
    (1, 5120, F16, F16, False, None, True, 1.0), (3, 8, F16, F32, True, "channel", True, 0.5),
    (7, 4096, BF16, BF16, True, "full", True, -2.0), (300, 5120, BF16, F32, True, "channel", True, 0.7),
    (5, 4104, F16, F32, False, "full", True, 1.0), (2, 32768, F16, F16, True, None, True, 1.0),
    (2, 13824, BF16, F32, False, None, False, 0.0), (33, 264, F16, F16, True, "channel", False, 1.0),
    (5000, 128, F16, F16, False, None, True, 1.0), (1, 8192, BF16, F32, True, "full", True, 1.0)]


@pytest.mark.parametrize("M,K,dtype,stream,post,gate,gamma,alpha", NORM)
@pytest.mark.parametrize("overlap", [False, True])
def test_residual_rmsnorm(w4, M, K, dtype, stream, post, gate, gamma, alpha, overlap):
    w4.w4a16_set_launch_overlap(overlap)
    h, y = normal((M, K), stream, 1, 3.0), normal((M, K), dtype, 2)
    pg = (normal((K,), dtype, 3, 0.3).float() + 1).to(dtype) if post else None
    gm = (normal((K,), dtype, 4, 0.3).float() + 1).to(dtype) if gamma else None
    gt = None if gate is None else normal((K,) if gate == "channel" else (M, K), dtype, 5, 0.6)
    ho, no = w4.w4a16_residual_rmsnorm(h, y, gm, 1e-5, post_gamma=pg, gate=gt, alpha=alpha)
    torch.cuda.synchronize()
    x = lambda t: None if t is None else f64(t)  # noqa: E731
    want, wn, mag, mn = ref.residual_rmsnorm(x(h), x(y), x(gm), 1e-5, x(pg), x(gt), alpha)
    within(ho, want, U[stream] * np.abs(want) + 60 * E * mag, "h")
    assert (no is None) == (not gamma)
    if gamma:
        within(no, wn, U[dtype] * np.abs(wn) + 120 * E * mn, "n")
    # in place, through wider rows
    hw, yw = torch.zeros(M, K + 16, dtype=stream, device="cuda"), torch.zeros(M, K + 24, dtype=dtype, device="cuda")
    hw[:, 8:K + 8], yw[:, 16:K + 16] = h, y
    w4.w4a16_residual_rmsnorm(hw[:, 8:K + 8], yw[:, 16:K + 16], gm, 1e-5, post_gamma=pg, gate=gt, alpha=alpha,
                              h_out=hw[:, 8:K + 8], n_out=yw[:, 16:K + 16] if gamma else None)
    torch.cuda.synchronize()
    assert torch.equal(hw[:, 8:K + 8], ho) and not hw[:, :8].any() and not hw[:, K + 8:].any()
    assert torch.equal(yw[:, 16:K + 16], no if gamma else y) and not yw[:, :16].any() and not yw[:, K + 16:].any()


def test_residual_rmsnorm_zero_rows_and_zero_values(w4):
    h, y, gm = torch.zeros(2, 64, dtype=F16, device="cuda"), torch.zeros(2, 64, dtype=F16, device="cuda"), normal((64,), F16, 1)
    ho, no = w4.w4a16_residual_rmsnorm(h[:0], y[:0], gm)
    assert ho.shape == no.shape == (0, 64)
    ho, no = w4.w4a16_residual_rmsnorm(h, y, gm, 1e-6, post_gamma=gm)
    torch.cuda.synchronize()
    assert not ho.any() and not no.any()


# ------------------------------------------------------------------ together
def test_no_rows(w4):
    cache, _, _ = make_cache(w4, 2, 16, 1, 64, F16, 1)
    e = lambda *s, d=F16: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    w4.w4a16_rope_append(e(0, 2, 64), e(0, 1, 64), e(0, 1, 64), e(0, d=torch.int32), torch.ones(32, device="cuda"), cache,
                         e(0, d=torch.int64))
    assert w4.w4a16_paged_attention(e(0, 2, 64), cache, e(0, 4, d=torch.int32), e(0, d=torch.int32),
                                    workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda")).shape == (0, 2, 64)
    z = e(0, d=torch.int32)
    w4.w4a16_kv_extend(z, z, e(0, 4, d=torch.int32), i32([1]), i32([1]), 16, e(0, d=torch.int64), z, z)


@pytest.mark.parametrize("overlap", [False, True])
def test_captured_step_equals_the_eager_one(w4, overlap):
    """extend, rope_append, attention and norm of a step, captured; replays continue the sequence."""
    w4.w4a16_set_launch_overlap(overlap)
    B, H, KV, D, page, pages = 5, 8, 2, 64, 16, 60

    def state():
        rng = np.random.default_rng(2)
        k, v = (torch.zeros(pages, page, KV, D, dtype=F16, device="cuda") for _ in (0, 1))
        s = dict(k=k, v=v, cache=w4.KVCache(k, v), lens=i32(np.zeros(B)), new=i32(np.ones(B)), free=i32(rng.permutation(pages)),
                 count=i32([pages]), table=i32(np.zeros((B, 10))), slots=torch.zeros(8, dtype=torch.int64, device="cuda"),
                 pos=i32(np.zeros(8)), refused=i32(np.zeros(B)), x=normal((B, H * D), F16, 3),
                 w=normal((H * D, (H + 2 * KV) * D), F16, 4, 0.05), freq=w4.w4a16_rope_frequencies(D, 1e4).cuda(),
                 gamma=normal((H * D,), F16, 5), q=torch.zeros(B, H, D, dtype=F16, device="cuda"),
                 o=torch.zeros(B, H, D, dtype=F16, device="cuda"), qkv=torch.zeros(B, H + 2 * KV, D, dtype=F16, device="cuda"),
                 n=normal((B, H * D), F16, 6),
                 ws=torch.zeros(w4.w4a16_paged_attention_workspace_bytes(B, H, KV, D), dtype=torch.uint8, device="cuda"))
        return s

    def step(s):
        w4.w4a16_kv_extend(s["lens"], s["new"], s["table"], s["free"], s["count"], page, s["slots"], s["pos"], s["refused"])
        torch.matmul(s["n"], s["w"], out=s["qkv"].view(B, -1))
        q, k, v = s["qkv"].split([H, KV, KV], 1)
        w4.w4a16_rope_append(q, k, v, s["pos"][:B], s["freq"], s["cache"], s["slots"][:B], out=s["q"])
        w4.w4a16_paged_attention(s["q"], s["cache"], s["table"], s["lens"], out=s["o"], workspace=s["ws"])
        w4.w4a16_residual_rmsnorm(s["x"], s["o"].view(B, -1), s["gamma"], h_out=s["x"], n_out=s["n"])

    a, b = state(), state()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(b)
        step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream, capture_error_mode="global"):
        step(b)
    with torch.cuda.stream(stream):
        for _ in range(36):
            step(a)
            g.replay()
    torch.cuda.synchronize()
    for name in ("x", "n", "o", "k", "v", "table", "lens", "count", "slots"):
        assert torch.equal(a[name], b[name]), name
    assert a["lens"].tolist() == [37] * B and int(a["count"]) == pages - 3 * B
