"""CPU-only checks of the operators between the projections: refusals of the C ABI
(fake addresses, nothing is launched) and of the binding, the frequency helper
against its formulas, and the oracle on worked examples."""
import ctypes
import struct

import numpy as np
import pytest
import torch

from oracle import decode_ops as ref

A, BAD4, BAD16 = 0x10000, 0x10002, 0x10008
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def w4():
    import weight_only_int4_repack_gb300 as w4
    return w4


def cache(w4, **kw):
    c = w4.KVCache(torch.empty(1, 1, 1, 16, dtype=torch.float16), torch.empty(1, 1, 1, 16, dtype=torch.float16))
    base = dict(k=A, v=A, k_scale=None, v_scale=None, k_page=16 * 8 * 128, k_token=8 * 128, k_head=128,
                v_page=16 * 8 * 128, v_token=8 * 128, v_head=128, type=0, pages=100, page_size=16, kv_heads=8,
                head_dim=128)
    for n, x in {**base, **kw}.items():
        setattr(c, n, x)
    return c


CACHE_REFUSALS = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=BAD16), INVALID), (dict(pages=0), INVALID),
    (dict(page_size=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(type=3), INVALID),
    (dict(type=9), INVALID), (dict(k_token=1028), INVALID), (dict(v_page=-8), INVALID), (dict(k_scale=A), INVALID),
    (dict(type=2, k_head=136), INVALID), (dict(type=2, k_scale=BAD4), INVALID), (dict(head_dim=132), UNSUPPORTED),
    (dict(head_dim=264), UNSUPPORTED), (dict(type=2, head_dim=72), UNSUPPORTED), (dict(v_page=2**31), UNSUPPORTED),
]


def extend(w4, **kw):
    a = dict(lens=A, new=A, table=A, stride=64, batch=4, max_pages=64, page=16, free=A, pool=100, count=A, lens_out=A,
             count_out=A, slots=A, positions=A, n=64, refused=A, spacing=0)
    a.update(kw)
    return w4.lib.w4a16_kv_extend(a["lens"], a["new"], a["table"], a["stride"], a["batch"], a["max_pages"], a["page"],
                                  a["free"], a["pool"], a["count"], a["lens_out"], a["count_out"], a["slots"],
                                  a["positions"], a["n"], a["refused"], a["spacing"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(max_pages=0), INVALID), (dict(page=0), INVALID), (dict(pool=0), INVALID),
    (dict(n=-1), INVALID), (dict(spacing=-1), INVALID), (dict(n=2**31 - 1), UNSUPPORTED), (dict(stride=63), INVALID), (dict(batch=8193), UNSUPPORTED), (dict(lens=None), INVALID),
    (dict(new=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID), (dict(count=None), INVALID),
    (dict(lens_out=None), INVALID), (dict(count_out=None), INVALID), (dict(slots=None), INVALID),
    (dict(positions=None), INVALID), (dict(refused=None), INVALID), (dict(lens=BAD4), INVALID),
    (dict(slots=0x10004), INVALID), (dict(batch=0), 0),
])
def test_kv_extend_refusals(w4, kw, status):
    assert extend(w4, **kw) == status


def rope(w4, c=None, **kw):
    a = dict(q=A, k=A, v=A, type=0, q_row=7168, q_head=128, k_row=7168, k_head=128, v_row=7168, v_head=128, bias=None,
             positions=A, freq=A, rot=128, inter=0, m=1.0, out=A, o_row=5120, o_head=128, slots=A, rows=3, heads=40)
    a.update(kw)
    return w4.lib.w4a16_rope_append(a["q"], a["k"], a["v"], a["type"], a["q_row"], a["q_head"], a["k_row"],
                                    a["k_head"], a["v_row"], a["v_head"], a["bias"], a["positions"], a["freq"],
                                    a["rot"], a["inter"], a["m"], a["out"], a["o_row"], a["o_head"],
                                    c or cache(w4), a["slots"], a["rows"], a["heads"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(type=3), INVALID), (dict(type=1), UNSUPPORTED), (dict(rows=-1), INVALID),
    (dict(heads=0), INVALID), (dict(inter=2), INVALID), (dict(rot=-4), INVALID), (dict(rot=132), INVALID),
    (dict(rot=6), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(out=None), INVALID), (dict(positions=None), INVALID), (dict(freq=None), INVALID), (dict(slots=None), INVALID),
    (dict(q=BAD4), INVALID), (dict(bias=BAD4), INVALID), (dict(slots=0x10004), INVALID), (dict(positions=BAD4), INVALID),
    (dict(q_row=7167), INVALID), (dict(v_head=-128), INVALID), (dict(rows=0), 0),
])
def test_rope_append_refusals(w4, kw, status):
    assert rope(w4, **kw) == status


def attention(w4, c=None, **kw):
    a = dict(q=A, type=0, q_row=5120, q_head=128, table=A, stride=64, max_pages=64, lens=A, batch=3, heads=40,
             scale=0.1, window=0, cap=0.0, out=A, o_row=5120, o_head=128, lse=None, ws=A * 16, ws_bytes=1 << 40)
    a.update(kw)
    return w4.lib.w4a16_paged_attention(a["q"], a["type"], a["q_row"], a["q_head"], c or cache(w4), a["table"],
                                        a["stride"], a["max_pages"], a["lens"], a["batch"], a["heads"], a["scale"],
                                        a["window"], a["cap"], a["out"], a["o_row"], a["o_head"], a["lse"], a["ws"],
                                        a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(type=1), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(heads=0), INVALID),
    (dict(heads=41), INVALID), (dict(max_pages=0), INVALID), (dict(stride=63), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(cap=-1.0), INVALID),
    (dict(cap=float("inf")), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(table=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=BAD16), INVALID), (dict(out=BAD16), INVALID), (dict(lens=BAD4), INVALID),
    (dict(lse=BAD4), INVALID), (dict(q_row=5124), INVALID), (dict(o_head=-128), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws=A * 16 + 16), WORKSPACE), (dict(ws_bytes=0), WORKSPACE), (dict(batch=1 << 20), UNSUPPORTED),
    (dict(batch=100, max_pages=1 << 27, stride=1 << 27), UNSUPPORTED),
    (dict(batch=0), 0),
])
def test_paged_attention_refusals(w4, kw, status):
    assert attention(w4, **kw) == status


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refusals(w4, kw, status):
    assert rope(w4, cache(w4, **kw), rot=0) == status
    assert attention(w4, cache(w4, **kw)) == status


def test_workspace_bytes(w4):
    f = w4.w4a16_paged_attention_workspace_bytes
    assert f(1, 40, 8, 128) > 0
    assert f(0, 40, 8, 128) == 0 and f(1, 41, 8, 128) == 0 and f(1, 40, 0, 128) == 0 and f(1, 8, 8, 0) == 0
    assert attention(w4, ws_bytes=f(3, 40, 8, 128) - 1) == WORKSPACE


def norm(w4, **kw):
    a = dict(h=A, h_type=0, h_row=5120, y=A, type=0, y_row=5120, post=None, gate=None, gate_row=0, alpha=1.0, gamma=A,
             eps=1e-5, h_out=A, ho_row=5120, n_out=A, no_row=5120, M=3, K=5120)
    a.update(kw)
    return w4.lib.w4a16_residual_rmsnorm(a["h"], a["h_type"], a["h_row"], a["y"], a["type"], a["y_row"], a["post"],
                                         a["gate"], a["gate_row"], a["alpha"], a["gamma"], a["eps"], a["h_out"],
                                         a["ho_row"], a["n_out"], a["no_row"], a["M"], a["K"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(K=5124), UNSUPPORTED), (dict(K=32776), UNSUPPORTED),
    (dict(type=2), INVALID), (dict(type=3), INVALID), (dict(h_type=1), UNSUPPORTED), (dict(h_type=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(alpha=float("nan")), INVALID), (dict(gamma=None), INVALID), (dict(n_out=None), INVALID),
    (dict(h=None), INVALID), (dict(y=None), INVALID), (dict(h_out=None), INVALID), (dict(h=BAD16), INVALID),
    (dict(post=BAD16), INVALID), (dict(gate=BAD16), INVALID), (dict(h_row=5112), INVALID), (dict(y_row=5124), INVALID),
    (dict(gate=A, gate_row=8), INVALID), (dict(no_row=5112), INVALID), (dict(M=0), 0),
])
def test_residual_rmsnorm_refusals(w4, kw, status):
    assert norm(w4, **kw) == status


# ------------------------------------------------------------------ the calls with their arguments in one block
class Blocks:
    """Stands for the library where a call's arguments go as the block of its parameters, in their order."""

    def __init__(self, w4):
        self.w4, self.lib, self.KVCache = w4, self, w4.KVCache

    def __getattr__(self, name):
        def call(*args):
            flat = [0 if a is None else ctypes.addressof(a) if isinstance(a, ctypes.Structure) else a for a in args]
            return getattr(self.w4.lib, name + "_block")(struct.pack(self.w4._blocks[name], *flat))
        return call


@pytest.mark.parametrize("call,kw,status", [
    (extend, dict(batch=8193), UNSUPPORTED), (extend, dict(refused=None), INVALID), (extend, dict(spacing=-1), INVALID),
    (extend, dict(slots=0x10004), INVALID), (extend, dict(n=-1), INVALID), (extend, dict(batch=0), 0),
    (rope, dict(rot=6), UNSUPPORTED), (rope, dict(bias=BAD4), INVALID), (rope, dict(v_head=-128), INVALID),
    (rope, dict(slots=0x10004), INVALID), (rope, dict(heads=0), INVALID), (rope, dict(rows=0), 0),
    (attention, dict(heads=41), INVALID), (attention, dict(cap=-1.0), INVALID), (attention, dict(lse=BAD4), INVALID),
    (attention, dict(ws_bytes=0), WORKSPACE), (attention, dict(type=1), UNSUPPORTED), (attention, dict(batch=0), 0),
    (norm, dict(K=5124), UNSUPPORTED), (norm, dict(eps=-1.0), INVALID), (norm, dict(no_row=5112), INVALID),
    (norm, dict(h_type=2), INVALID), (norm, dict(gate=A, gate_row=8), INVALID), (norm, dict(M=0), 0)])
def test_blocks_are_read_in_order(w4, call, kw, status):
    assert call(w4, **kw) == status and call(Blocks(w4), **kw) == status


def test_blocks_refuse_none(w4):
    for name in w4._blocks:
        assert getattr(w4.lib, name + "_block")(None) == INVALID


# ------------------------------------------------------------------ binding
def test_binding_refusals(w4):
    half = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    with pytest.raises(ValueError):
        w4.KVCache(half(2, 16, 2, 64), half(2, 16, 2, 32))
    with pytest.raises(TypeError):
        w4.KVCache(torch.zeros(2, 16, 2, 64), torch.zeros(2, 16, 2, 64))
    with pytest.raises(ValueError):
        w4.KVCache(half(2, 16, 64, 2).transpose(2, 3), half(2, 16, 64, 2).transpose(2, 3))
    with pytest.raises(TypeError):
        w4.KVCache(half(2, 16, 2, 64), half(2, 16, 2, 64), half(2))
    c = w4.KVCache(half(2, 16, 2, 64), half(2, 16, 2, 64))
    i32, i64 = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    q, k, f = half(3, 4, 64), half(3, 2, 64), torch.ones(32)
    with pytest.raises(TypeError):
        w4.w4a16_rope_append(q, k, k, i64, f, c, i64, out=q, stream=0)
    with pytest.raises(ValueError):
        w4.w4a16_rope_append(q, k[:, :1], k, i32, f, c, i64, out=q, stream=0)
    with pytest.raises(TypeError):
        w4.w4a16_rope_append(q, k.float(), k, i32, f, c, i64, out=q, stream=0)
    with pytest.raises(ValueError):
        w4.w4a16_rope_append(q, k, k, i32, f, c, i64, bias=half(5), out=q, stream=0)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError):
        w4.w4a16_paged_attention(q, c, torch.zeros(2, 4, dtype=torch.int32), i32, out=q, workspace=ws, stream=0)
    with pytest.raises(TypeError):
        w4.w4a16_paged_attention(q, c, torch.zeros(3, 4), i32, out=q, workspace=ws, stream=0)
    with pytest.raises(ValueError):
        w4.w4a16_residual_rmsnorm(half(3, 64), half(3, 32), half(64))
    with pytest.raises(TypeError):
        w4.w4a16_residual_rmsnorm(half(3, 64), half(3, 64), torch.ones(64))
    with pytest.raises(ValueError):
        w4.w4a16_kv_extend(i32, i32, torch.zeros(2, 4, dtype=torch.int32), i32, i32, 16, i64, i32, i32, stream=0)


def test_cache_strides_follow_the_view(w4):
    pool = torch.zeros(5, 2, 16, 64, dtype=torch.float16)  # heads first
    c = w4.KVCache(pool.transpose(1, 2), pool.transpose(1, 2))
    assert (c.k_page, c.k_token, c.k_head) == (2 * 16 * 64, 64, 16 * 64)
    assert (c.pages, c.page_size, c.kv_heads, c.head_dim) == (5, 16, 2, 64)


# ------------------------------------------------------------------ frequencies
def test_rope_frequencies(w4):
    rot, base, factor, context = 64, 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2, dtype=np.float64)
    plain = base ** (-2 * i / rot)
    got = lambda **kw: w4.w4a16_rope_frequencies(rot, base, **kw).numpy()  # noqa: E731
    half_step = 2.0**-24
    np.testing.assert_allclose(got(), plain, rtol=2 * half_step)
    np.testing.assert_allclose(got(scaling=1, factor=factor), plain / factor, rtol=2 * half_step)
    two = got(scaling=2, factor=factor)
    assert two[0] == 1.0
    np.testing.assert_allclose(two[-1], plain[-1] / factor, rtol=2 * half_step)
    three = got(scaling=3, factor=factor, context=context, low=1.0, high=32.0)
    turns = context * plain / (2 * np.pi)
    np.testing.assert_allclose(three[turns >= 32], plain[turns >= 32], rtol=2 * half_step)
    np.testing.assert_allclose(three[turns <= 1], plain[turns <= 1] / factor, rtol=2 * half_step)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all(three[mid] < plain[mid]) and np.all(three[mid] > plain[mid] / factor)


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(base=0.0), dict(base=float("nan")), dict(scaling=4),
                                dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, rot=2, factor=2.0),
                                dict(scaling=3, factor=2.0, context=0.0), dict(scaling=3, factor=2.0, context=64.0,
                                                                                low=4.0, high=4.0)])
def test_rope_frequencies_refusals(w4, kw):
    a = dict(rot=64, base=1e4, scaling=0, factor=1.0, context=0.0, low=1.0, high=32.0)
    a.update(kw)
    buf = (ctypes.c_float * 64)()
    assert w4.lib.w4a16_rope_frequencies(buf, a["rot"], a["base"], a["scaling"], a["factor"], a["context"], a["low"],
                                         a["high"]) == INVALID


# ------------------------------------------------------------------ oracle on worked examples
def test_oracle_kv_extend_worked_example():
    # Pages of 4 tokens; request 0 ends and gives 7, 8 back; request 1 (5 tokens, page 3, 2 held) gets 4 more and
    # needs one page; request 2 starts with 3 tokens; request 3 wants 9 pages, which are not there.
    table = np.array([[7, 8, -1, -1], [3, 2, -1, -1], [-1] * 4, [-1] * 4])
    got = ref.kv_extend([6, 5, 0, 0], [-1, 4, 3, 16], table, np.array([1, 9, 0, 0, 0]), 2, 4, 32)
    assert got["table"].tolist() == [[7, 8, -1, -1], [3, 2, 8, -1], [7, -1, -1, -1], [-1] * 4]
    assert got["free_pages"].tolist() == [1, 9, 7, 8, 0] and got["free_count_out"] == 2
    assert got["lens_out"].tolist() == [0, 9, 3, 0] and got["refused"].tolist() == [0, 0, 0, 1]
    assert got["slots"][:8].tolist() == [9, 10, 11, 32, 28, 29, 30, -1]
    assert got["positions"][:8].tolist() == [5, 6, 7, 8, 0, 1, 2, 0]


def test_oracle_kv_extend_spacing():
    table = np.array([[7, 8], [3, 2], [4, 5]])
    got = ref.kv_extend([6, 5, 2], [0, 2, 3], table, np.array([1]), 0, 4, 6, spacing=2)
    assert got["slots"].tolist() == [-1, -1, 9, 10, -1, -1] and got["refused"].tolist() == [0, 0, 2]


def test_oracle_rope_quarter_turn():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    f = np.array([np.pi / 2, np.pi])
    half, _ = ref.rope(x, [1], f, 4, False, 2.0)
    np.testing.assert_allclose(half, [[[-6, -4, 2, -8, 5]]], atol=1e-12)
    pairs, _ = ref.rope(x, [1], f, 4, True, 1.0)
    np.testing.assert_allclose(pairs, [[[-2, 1, -3, -4, 5]]], atol=1e-12)


def test_oracle_attention_two_tokens():
    q = np.array([[1.0, 0.0]])
    k = np.array([[np.log(3.0), 0.0], [0.0, 9.0]])
    v = np.array([[4.0, 0.0], [0.0, 8.0]])
    out, lse, mag, _ = ref.attention(q, k, v, 1.0)
    np.testing.assert_allclose(out, [[3.0, 2.0]])
    np.testing.assert_allclose(lse, [np.log(4.0)])
    np.testing.assert_allclose(mag, out)
    out, lse, _, _ = ref.attention(q, k[:0], v[:0], 1.0)
    assert not out.any() and lse[0] == -np.inf


def test_oracle_residual_rmsnorm_worked_example():
    h, n, _, _ = ref.residual_rmsnorm(np.array([[1.0, 1.0]]), np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0,
                                      post_gamma=np.array([1.0, 1.0]), gate=np.array([[1.0, 0.0]]), alpha=2.0)
    a = 1 + 2 * 3 / np.sqrt(12.5)
    np.testing.assert_allclose(h, [[a, 1.0]])
    np.testing.assert_allclose(n, np.array([[a, 2.0]]) / np.sqrt((a * a + 1) / 2))
