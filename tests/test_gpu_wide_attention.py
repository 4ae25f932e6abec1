"""GPU parity of the attention of many rows (prompt_attention, prefix_attention) with its
float64 statement.

Error bounds are counted in half steps of the output's type (u: fp16 2^-11, bf16 2^-8) and
in fp32 roundings (e = 2^-24). A score is off by (D + 16) e max_j scale sum |q k|: the
products' sum, the difference to the reference, its product with the scale, the exponential.
That is also the relative error of a weight, which is then rounded once as an operand (u);
outputs are a mean under these weights, so each counts twice (once in the sum they are divided
by), of the mean of |v|; sums over n keys add n e; the output is rounded once (u). fp16
operands end at 2^-36 of the reference.
"""
import math

import numpy as np
import pytest
import torch

from oracle.wide_ops import rows_attention

pytestmark = pytest.mark.gpu
E = 2.0**-24
U = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
F16, BF16, F32, E4M3 = torch.float16, torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture
def w4(gpu_lib):
    yield gpu_lib
    gpu_lib.w4a16_set_launch_overlap(False)
    assert gpu_lib.w4a16_device_error() == gpu_lib.W4A16_OK


def f64(t):
    return t.float().cpu().double().numpy()


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


class Setup:
    """Requests with `new` tokens of `lens`, prefixes, a cache with shuffled pages, queries."""

    def __init__(self, w4, new, lens, shared=(), of=None, heads=8, kv=2, dim=64, dtype=F16, cache=None, page=16,
                 order="tokens", seed=0, pad=0, q_scale=2.0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.w4, self.new, self.lens, self.shared, self.page = w4, list(new), list(lens), list(shared), page
        self.of = list(of) if of is not None else [-1] * len(self.lens)
        self.heads, self.kv, self.dim, self.dtype, self.cache_type = heads, kv, dim, dtype, cache or dtype
        held = [-(-n // page) for n in self.lens + self.shared]
        self.pages = sum(held) + 2
        perm = torch.randperm(self.pages, generator=g)
        self.width = max(1, max(held[:len(self.lens)], default=1)) + 1
        self.pwidth = max(1, max(held[len(self.lens):], default=1))
        table = torch.full((len(self.lens), self.width), -7, dtype=torch.int32)
        ptable = torch.full((max(1, len(self.shared)), self.pwidth), -7, dtype=torch.int32)
        at = 0
        for i, n in enumerate(held):
            row = table[i] if i < len(self.lens) else ptable[i - len(self.lens)]
            row[:n] = perm[at:at + n]
            at += n
        self.table, self.ptable = table.cuda(), ptable.cuda()
        shape = (self.pages, kv, page, dim) if order == "heads" else (self.pages, page, kv, dim)
        amount = 60.0 if self.cache_type == E4M3 else spread
        make = lambda: (torch.randn(shape, generator=g) * amount).to(self.cache_type).cuda()  # noqa: E731
        self.k, self.v = make(), make()
        if order == "heads":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.k_scale = self.v_scale = None
        if self.cache_type == E4M3:
            self.k_scale = (torch.rand(kv, generator=g) * 0.01 + 0.01).cuda()
            self.v_scale = (torch.rand(kv, generator=g) * 0.01 + 0.01).cuda()
        self.rows = sum(self.new) + pad
        self.q = (torch.randn(self.rows, heads, dim, generator=g) * q_scale).to(dtype).cuda()
        self.starts = i32(np.cumsum([0] + self.new))
        self.len_t, self.of_t = i32(self.lens), i32(self.of)
        self.plens = i32(self.shared or [0])
        self.kv_cache()

    def kv_cache(self):
        self.kvc = self.w4.KVCache(self.k, self.v, self.k_scale, self.v_scale)

    def prefix_args(self):
        return dict(prefix_table=self.ptable, prefix_lens=self.plens, prefix_of=self.of_t) if self.shared else {}

    def tokens(self, b):
        """Keys and values of request b in float64, its prefix in front."""
        parts = []
        lists = [(self.table[b], self.lens[b])]
        if self.of[b] >= 0:
            lists.insert(0, (self.ptable[self.of[b]], self.shared[self.of[b]]))
        for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            got = []
            for row, n in lists:
                pages = row[:-(-n // self.page)].cpu().long()
                x = pool.float().cpu()[pages].reshape(-1, self.kv, self.dim)[:n].double().numpy()
                got.append(x)
            x = np.concatenate(got)
            parts.append(x if scale is None else x * scale.cpu().double().numpy()[None, :, None])
        return parts

    def want(self, scale, window=0, softcap=0.0, only=None):
        outs = []
        for b in range(len(self.lens)) if only is None else only:
            k, v = self.tokens(b)
            first = int(np.sum(self.new[:b]))
            outs.append((slice(first, first + self.new[b]), rows_attention(
                f64(self.q[first:first + self.new[b]]), k, v, len(k) - self.new[b], scale, window, softcap), len(k)))
        return outs

    def prompt(self, **kw):
        self.out = torch.full_like(self.q, 77.0)
        self.lse = torch.full((self.rows, self.heads), 55.0, device="cuda")
        return self.w4.w4a16_prompt_attention(self.q, self.kvc, self.table, self.starts, self.len_t, out=self.out,
                                              lse=self.lse, **self.prefix_args(), **kw)

    def prefix(self, **kw):
        self.out = torch.full_like(self.q, 77.0)
        self.lse = torch.full((self.rows, self.heads), 55.0, device="cuda")
        return self.w4.w4a16_prefix_attention(self.q, self.kvc, self.table, self.len_t, self.ptable, self.plens, self.of_t,
                                              out=self.out, lse=self.lse, **kw)

    def check(self, scale=None, window=0, softcap=0.0, only=None):
        torch.cuda.synchronize()
        scale = self.dim**-0.5 if scale is None else scale
        u = U[self.dtype]
        out, lse = f64(self.out), f64(self.lse)
        for at, (want, want_lse, mag, top), n in self.want(scale, window, softcap, only):
            if want.size == 0:
                continue
            eps = (self.dim + 16) * E * (np.minimum(top, softcap) + 1 if softcap else top) + (n + 8) * E + 2.0**-22
            if softcap:
                eps = eps + (self.dim + 16) * E * top + 8 * E * softcap
            bound = u * np.abs(want) + 2 * (u + eps)[..., None] * mag + n * 2.0**-36 * (mag[np.isfinite(mag)].max() + 1) + 2.0**-24
            finite = np.isfinite(want)
            assert np.array_equal(out[at][~finite], want[~finite], equal_nan=True), "what is not finite"
            off = (np.abs(out[at] - want) - bound)[finite]
            assert off.size == 0 or off.max() <= 0, f"out: {off.max()} over the bound, rows {at}"
            some = np.isfinite(want_lse)
            assert np.array_equal(lse[at][~some], want_lse[~some], equal_nan=True), "lse of nothing"
            off = np.abs(lse[at] - want_lse)[some] - (eps + 2 * E * np.abs(want_lse))[some]
            assert off.size == 0 or off.max() <= 0, f"lse: {off.max()} over the bound, rows {at}"


SHAPES = [  # heads, kv heads, dim, type, cache, page, order
    (8, 2, 64, F16, F16, 16, "tokens"), (10, 2, 128, BF16, BF16, 16, "tokens"), (4, 2, 256, F16, F16, 16, "heads"),
    (8, 2, 128, F16, E4M3, 32, "tokens"), (16, 1, 64, BF16, E4M3, 8, "heads"), (6, 2, 256, BF16, E4M3, 16, "tokens"),
    (9, 3, 80, F16, F16, 24, "tokens"), (4, 4, 96, BF16, BF16, 1, "heads"), (3, 1, 8, F16, F16, 16, "tokens"),
    (71, 1, 72, F16, F16, 64, "tokens"), (5, 5, 16, BF16, E4M3, 128, "tokens"), (2, 1, 192, BF16, BF16, 40, "tokens"),
]


@pytest.mark.parametrize("heads,kv,dim,dtype,cache,page,order", SHAPES)
def test_prompt_shapes(w4, heads, kv, dim, dtype, cache, page, order):
    s = Setup(w4, [1, 37, 5, 130], [1, 37, 300, 401], heads=heads, kv=kv, dim=dim, dtype=dtype, cache=cache, page=page,
              order=order, pad=3)
    s.prompt()
    s.check()
    assert bool((s.out[-3:] == 77.0).all()) and bool((s.lse[-3:] == 55.0).all())


@pytest.mark.parametrize("new,before", [(1, 0), (1, 127), (1, 128), (1, 129), (2, 126), (25, 0), (26, 0), (51, 0), (52, 3),
                                        (127, 0), (128, 0), (129, 0), (255, 1), (256, 0), (257, 255), (33, 1000), (600, 0)])
def test_prompt_lengths(w4, new, before):
    s = Setup(w4, [new], [new + before], heads=5, kv=1, dim=64, seed=new)
    s.prompt()
    s.check()


@pytest.mark.parametrize("heads,kv,dim,dtype,cache,page,order", SHAPES)
def test_prefix_shapes(w4, heads, kv, dim, dtype, cache, page, order):
    n = 70 // heads + 9
    s = Setup(w4, [1] * n, [1 + 13 * i % 90 for i in range(n)], [333, 128, 1], [i % 4 - 1 for i in range(n)], heads=heads,
              kv=kv, dim=dim, dtype=dtype, cache=cache, page=page, order=order)
    s.prefix()
    s.check()


@pytest.mark.parametrize("batch,shared", [(1, 1), (1, 5000), (2, 127), (25, 128), (26, 129), (51, 1000), (52, 300), (103, 700)])
def test_prefix_lengths(w4, batch, shared):
    s = Setup(w4, [1] * batch, [1 + i % 40 for i in range(batch)], [shared], [0] * batch, heads=5, kv=1, dim=64, seed=batch)
    s.prefix()
    s.check()


@pytest.mark.parametrize("dim,cache", [(64, F16), (128, E4M3), (256, F16)])
@pytest.mark.parametrize("window,softcap,scale", [(1, 0.0, None), (50, 0.0, None), (200, 30.0, None), (0, 5.0, 0.3),
                                                  (0, 0.0, -0.2), (64, 2.0, -0.2), (0, 0.0, 0.0), (0, 0.0, 40.0)])
def test_windows_caps_scales(w4, dim, cache, window, softcap, scale):
    kw = dict(window=window, softcap=softcap, scale=scale)
    s = Setup(w4, [3, 150, 1], [40, 150, 333], [100, 260], [1, -1, 0], heads=6, kv=2, dim=dim, cache=cache, page=16)
    s.prompt(**kw)
    s.check(**kw)
    s = Setup(w4, [1] * 40, [1 + 7 * i % 300 for i in range(40)], [100, 260], [i % 3 - 1 for i in range(40)], heads=6, kv=2,
              dim=dim, cache=cache, page=16)
    s.prefix(**kw)
    s.check(**kw)


def test_prompts_behind_prefixes(w4):
    s = Setup(w4, [5, 0, 60, 1, 128], [5, 3, 260, 1, 128], [77, 500, 16], [1, 0, 0, 2, -1], heads=10, kv=2, dim=128, dtype=BF16)
    s.prompt()
    s.check()


def test_many_requests(w4):
    r = np.random.RandomState(0)
    new = [int(x) for x in r.randint(0, 4, 900)]
    lens = [n + int(x) for n, x in zip(new, r.randint(0, 60, 900))]
    s = Setup(w4, new, lens, [40], [int(x) for x in r.randint(-1, 1, 900)], heads=2, kv=1, dim=16, page=8)
    s.prompt()
    s.check()
    of = [int(x) for x in r.randint(-1, 300, 900)]
    s = Setup(w4, [1] * 900, [max(1, n) for n in lens], [int(x) for x in r.randint(0, 200, 300)], of, heads=2, kv=1, dim=16, page=8)
    s.prefix()
    s.check()


def test_rows_without_keys(w4):
    # A length below the rows is an error: the rows in front of the first token see nothing.
    s = Setup(w4, [6, 4], [6, 4], heads=4, kv=2, dim=64)
    s.len_t = i32([2, 4])
    s.prompt()
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    assert bool((s.out[:4] == 0).all()) and bool(torch.isneginf(s.lse[:4]).all())
    assert bool(torch.isfinite(s.lse[4:]).all())
    # Requests without tokens of their own, prefixes without tokens.
    s = Setup(w4, [1] * 4, [3, 3, 3, 3], [50, 0], [0, 1, 0, 1], heads=4, kv=2, dim=64)
    s.len_t = i32([3, 3, 0, 0])
    s.prefix()
    s.check(only=[0])
    assert bool((s.out[2:] == 0).all()) and bool(torch.isneginf(s.lse[2:]).all())
    s.of, s.shared = [0, -1, 0, -1], [50]
    s.check(only=[1])


@pytest.mark.parametrize("cache", [F16, E4M3])
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_what_is_not_visible(w4, junk, cache):
    if cache == E4M3 and junk != junk or cache == F16:
        new, lens = [40, 7], [300, 130]
        s = Setup(w4, new, lens, [70], [0, -1], heads=10, kv=2, dim=128, cache=cache, page=16)
        s.prompt()
        torch.cuda.synchronize()
        clean = s.out.clone(), s.lse.clone()
        # Everything that no row sees; and the last tokens' keys and values, which only the last rows see.
        used = torch.zeros(s.pages, s.page, dtype=torch.bool)
        for row, n in [(s.table[0], 300), (s.table[1], 130), (s.ptable[0], 70)]:
            for j in range(n):
                used[int(row[j // 16]), j % 16] = True
        for j in (297, 298, 299):
            used[int(s.table[0][j // 16]), j % 16] = False
        used[int(s.table[1][129 // 16]), 129 % 16] = False
        for pool in (s.k, s.v):
            x = pool.float()
            x[~used.cuda()] = junk
            pool.copy_(x.to(cache))
        s.prompt()
        torch.cuda.synchronize()
        for rows in (slice(0, 37), slice(40, 46)):
            # Rows of a tile that has been spoilt are summed anew, key by key.
            a, b = s.out[rows].float(), clean[0][rows].float()
            assert bool((a - b).abs().max() <= 4 * 2.0**-11 * b.abs().max())
            assert bool(((s.lse[rows] - clean[1][rows]).abs() <= 2e-5).all())
        w4.w4a16_device_error()


def test_visible_infinities(w4):
    s = Setup(w4, [30], [200], heads=4, kv=2, dim=64)
    page, at = int(s.table[0, 100 // 16]), 100 % 16
    s.v[page, at, 0, 3], s.v[page, at, 1, 5], s.v[page, at, 1, 6] = math.inf, -math.inf, math.nan
    s.prompt()
    s.check()
    s = Setup(w4, [1] * 5, [20] * 5, [200], [0, 0, -1, 0, 0], heads=4, kv=2, dim=64)
    page = int(s.ptable[0, 100 // 16])
    s.v[page, at, 0, 3], s.v[page, at, 1, 5], s.v[page, at, 1, 6] = math.inf, -math.inf, math.nan
    s.prefix()
    s.check()


def test_values_out_of_range(w4):
    def errors(s, call):
        call()
        torch.cuda.synchronize()
        assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG

    # Bad pages are left out.
    for bad in (-1, 10**6):
        s = Setup(w4, [20], [70], [40], [0], heads=4, kv=2, dim=64)
        good = s.tokens(0)
        s.table[0, 1], s.ptable[0, 0] = bad, bad
        errors(s, s.prompt)
        keep = [j for j in range(110) if not (j < 16 or 56 <= j < 72)]
        k, v = good[0][keep], good[1][keep]
        want, lse, mag, _ = rows_attention(f64(s.q), k, v, len(k) - 20, 64**-0.5)
        assert np.abs(f64(s.out) - want).max() <= 8 * 2.0**-11 * mag.max() and np.abs(f64(s.lse) - lse).max() < 1e-4
        s = Setup(w4, [1] * 3, [20] * 3, [40], [0, 0, -1], heads=4, kv=2, dim=64)
        good = s.tokens(1)
        s.ptable[0, 1] = bad
        errors(s, s.prefix)
        keep = [j for j in range(60) if not 16 <= j < 32]
        k, v = good[0][keep], good[1][keep]
        want, lse, mag, _ = rows_attention(f64(s.q[1:2]), k, v, len(k) - 1, 64**-0.5)
        assert np.abs(f64(s.out[1:2]) - want).max() <= 8 * 2.0**-11 * mag.max()
    # Starts that fall or leave the rows; prefix numbers and lengths beyond the table.
    for starts in ([0, 5, 3, 9], [0, 4, 8, 10**6], [-4, 3, 6, 9]):
        s = Setup(w4, [3, 3, 3], [30, 30, 30], heads=4, kv=2, dim=64)
        s.starts = i32(starts)
        errors(s, s.prompt)
    s = Setup(w4, [3, 3], [30, 30], [20], [0, -1], heads=4, kv=2, dim=64)
    s.of_t = i32([0, 1])
    errors(s, s.prompt)
    s.check()
    s = Setup(w4, [1, 1], [30, 30], [32], [0, -1], heads=4, kv=2, dim=64)
    s.of_t, s.plens = i32([0, 9]), i32([10**9])
    errors(s, s.prefix)
    s.check()
    s = Setup(w4, [3], [30], heads=4, kv=2, dim=64)
    s.len_t = i32([10**9])  # counts as the table's row
    errors(s, s.prompt)
    s.len_t = i32([-5])
    errors(s, s.prompt)
    assert bool((s.out == 0).all())


def test_views_strides_and_streams(w4):
    s = Setup(w4, [17, 60], [100, 60], heads=6, kv=2, dim=64, page=16)
    wide = torch.full((s.rows, 6 + 4, 64 + 8), math.nan, dtype=F16, device="cuda")
    wide[:, :6, :64] = s.q
    s.q = wide[:, :6, :64]
    # Tokens outermost, then heads, then pages.
    for name in ("k", "v"):
        pool = getattr(s, name)
        big = torch.full((s.page, s.kv, s.pages + 1, s.dim), math.nan, dtype=F16, device="cuda")
        view = big.permute(2, 0, 1, 3)[:s.pages]
        view.copy_(pool)
        setattr(s, name, view)
    s.kv_cache()
    keep = torch.full((s.rows, 8, 64), 33.0, dtype=F16, device="cuda")
    s.out = keep[:, :6]
    s.lse = torch.zeros(s.rows, 6, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = w4.w4a16_prompt_attention(s.q, s.kvc, s.table, s.starts, s.len_t, out=s.out, lse=s.lse, stream=stream)
    stream.synchronize()
    assert got is s.out and bool((keep[:, 6:] == 33.0).all())
    s.check()


def test_one_workspace_for_calls_and_graphs(w4):
    a = Setup(w4, [40, 3], [140, 300], [200], [0, 0], heads=10, kv=2, dim=128)
    b = Setup(w4, [500], [700], heads=10, kv=2, dim=128, seed=1)
    c = Setup(w4, [1] * 30, [9 + i for i in range(30)], [900], [0] * 30, heads=10, kv=2, dim=128, seed=2)
    ws = torch.full((w4.w4a16_prompt_attention_workspace_bytes(700, 10, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    wsp = torch.zeros(w4.w4a16_prefix_attention_workspace_bytes(30, 10, 2, 128), dtype=torch.uint8, device="cuda")
    first = []
    for s, call in ((a, lambda: a.prompt(workspace=ws)), (b, lambda: b.prompt(workspace=ws)), (c, lambda: c.prefix(workspace=wsp))):
        call()
        s.check()
        first.append((s.out.clone(), s.lse.clone()))
    for overlap in (False, True):
        w4.w4a16_set_launch_overlap(overlap)
        graphs = []
        for s, call in ((a, "prompt"), (b, "prompt"), (c, "prefix")):
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                if call == "prompt":
                    w4.w4a16_prompt_attention(s.q, s.kvc, s.table, s.starts, s.len_t, out=s.out, lse=s.lse, workspace=ws,
                                              **s.prefix_args())
                else:
                    w4.w4a16_prefix_attention(s.q, s.kvc, s.table, s.len_t, s.ptable, s.plens, s.of_t, out=s.out, lse=s.lse,
                                              workspace=wsp)
            torch.cuda.current_stream().wait_stream(stream)
            graphs.append(graph)
        for _ in range(3):
            for s in (a, b, c):
                s.out.fill_(1.0), s.lse.fill_(1.0)
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for s, (out, lse) in zip((a, b, c), first):
            assert torch.equal(s.out, out) and torch.equal(s.lse, lse)


def test_a_wait_that_runs_out(w4):
    s = Setup(w4, [400], [900], [100], [0], heads=8, kv=2, dim=128)
    w4.w4a16_set_wait_limit_ns(0)
    try:
        s.prompt()
        torch.cuda.synchronize()
        assert w4.w4a16_device_error() == w4.W4A16_ERR_TIMEOUT
    finally:
        w4.w4a16_set_wait_limit_ns(w4.WAIT_LIMIT_DEFAULT_NS)
    s.prompt()
    s.check()


def test_offsets_beyond_32_bits(w4):
    # Pages 2^30 elements apart: the third one is beyond 2^31 elements, 2^32 bytes.
    s = Setup(w4, [20], [48], heads=4, kv=1, dim=64, page=16)
    big = torch.empty(3 * 2**30 + 16 * 64 * 2, dtype=F16, device="cuda")
    pools = [torch.as_strided(big, (4, 16, 1, 64), (2**30, 64, 64, 1), 16 * 64 * i) for i in range(2)]
    pages = s.table[0, :3].long()
    for new, old in zip(pools, (s.k, s.v)):
        new[1:] = old[pages]
    s.k, s.v, s.pages = pools[0], pools[1], 4
    s.table[0, :3] = i32([3, 1, 2])
    for pool in (s.k, s.v):
        x = pool[1:].clone()
        pool[3], pool[1], pool[2] = x[0], x[1], x[2]
    s.kv_cache()
    s.prompt()
    k = [f64(torch.stack([pool[3], pool[1], pool[2]])).reshape(48, 1, 64) for pool in (s.k, s.v)]
    want, lse, mag, _ = rows_attention(f64(s.q), k[0], k[1], 28, 0.125)
    assert np.abs(f64(s.out) - want).max() <= 4 * 2.0**-11 * mag.max() and np.abs(f64(s.lse) - lse).max() < 1e-4


def test_starts_that_fall_again_and_again(w4):
    # Requests that all have all rows would be more work than the rows could need: nothing is done.
    n = 600
    s = Setup(w4, [1] * n, [30] * n, heads=256, kv=1, dim=16)  # a tile has one token
    s.starts = i32([0, n] * (n // 2) + [0])
    s.prompt()
    torch.cuda.synchronize()
    assert w4.w4a16_device_error() == w4.W4A16_ERR_INVALID_ARG
    assert bool((s.out == 77).all()) and bool((s.lse == 55).all())


def test_tiny_softcap(w4):
    s = Setup(w4, [20], [60], heads=4, kv=2, dim=64)
    s.q[:, 0] = 0.0  # scores of 0 stay 0, all others are the cap, which is as good as 0
    s.prompt(softcap=1e-40)
    s.check(softcap=1e-40)


def test_workspace_of_a_larger_batch_serves_smaller_ones_in_between(w4):
    big = Setup(w4, [1] * 40, [50] * 40, [300], [0] * 40, heads=8, kv=2, dim=64)
    small = Setup(w4, [1] * 3, [700, 5, 90], [20], [0, -1, 0], heads=4, kv=4, dim=256, seed=1)
    ws = torch.zeros(max(w4.w4a16_prefix_attention_workspace_bytes(40, 8, 2, 64), w4.w4a16_prefix_attention_workspace_bytes(3, 4, 4, 256)),
                     dtype=torch.uint8, device="cuda")
    for s in (big, small, big, small):
        s.prefix(workspace=ws)
        s.check()


def test_two_calls_at_once(w4):
    a = Setup(w4, [700, 90], [1500, 90], [200], [0, 0], heads=8, kv=2, dim=128)
    b = Setup(w4, [1] * 50, [40 + i for i in range(50)], [2000], [0] * 50, heads=8, kv=2, dim=128, dtype=BF16, seed=1)
    logits = torch.randn(70, 50257, device="cuda")
    u, p = torch.rand(70, device="cuda"), torch.full((70,), 0.9, device="cuda")
    a.prompt(), b.prefix()
    first = (a.out.clone(), b.out.clone(), w4.w4a16_sample(logits, u, top_p=p))
    a.check(), b.check()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        outs = []
        torch.cuda.synchronize()
        for stream, call in zip(streams, (a.prompt, b.prefix, lambda: w4.w4a16_sample(logits, u, top_p=p))):
            with torch.cuda.stream(stream):
                outs.append(call())
        torch.cuda.synchronize()
        for x, y in zip(first, outs):
            assert torch.equal(x, y)


def test_most_requests_and_prefixes(w4):
    r = np.random.RandomState(3)
    n = 8192
    s = Setup(w4, [1] * n, [int(x) for x in r.randint(1, 6, n)], heads=2, kv=1, dim=16, page=8)
    s.prompt()
    s.check()
    of = [int(x) for x in r.randint(-1, 2048, n)]
    s = Setup(w4, [1] * n, [int(x) for x in r.randint(1, 4, n)], [int(x) for x in r.randint(1, 20, 2048)], of, heads=2, kv=1, dim=16, page=8)
    s.prefix()
    s.check()
