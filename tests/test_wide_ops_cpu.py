"""CPU-only checks of the attention of many rows, of shared prefixes and of the choice of tokens: refusals of the C ABI
(fake addresses, nothing is launched) and of the binding, and the oracle on worked examples."""
import ctypes
import re
import os
import struct

import numpy as np
import pytest
import torch

from oracle import wide_ops as ref

A, BAD4, BAD16 = 0x10000, 0x10002, 0x10008
OUT = 0x40000
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


class Direct:
    """The call with its arguments one by one."""

    def __init__(self, w4):
        self.w4 = w4

    def __call__(self, name, *args):
        return getattr(self.w4.lib, name)(*args)


class Block(Direct):
    """The same with the arguments in one block, in their order."""

    def __call__(self, name, *args):
        flat = [0 if a is None else ctypes.addressof(a) if isinstance(a, ctypes.Structure) else a for a in args]
        return getattr(self.w4.lib, name + "_block")(struct.pack(self.w4._wide_blocks[name], *flat))


def prompt(call, c=None, **kw):
    a = dict(q=A, type=0, q_row=5120, q_head=128, table=A, stride=64, max_pages=64, starts=A, lens=A, rows=70, batch=3,
             heads=40, ptable=A, pstride=32, ppages=32, plens=A, pof=A, prefixes=2, scale=0.1, window=0, cap=0.0, out=OUT,
             o_row=5120, o_head=128, lse=None, ws=A * 16, ws_bytes=1 << 40)
    a.update(kw)
    return call("w4a16_prompt_attention", a["q"], a["type"], a["q_row"], a["q_head"], c or cache(call.w4), a["table"],
                a["stride"], a["max_pages"], a["starts"], a["lens"], a["rows"], a["batch"], a["heads"], a["ptable"],
                a["pstride"], a["ppages"], a["plens"], a["pof"], a["prefixes"], a["scale"], a["window"], a["cap"], a["out"],
                a["o_row"], a["o_head"], a["lse"], a["ws"], a["ws_bytes"], None)


def prefix(call, c=None, **kw):
    a = dict(q=A, type=0, q_row=5120, q_head=128, table=A, stride=64, max_pages=64, lens=A, batch=3, heads=40, ptable=A,
             pstride=32, ppages=32, plens=A, pof=A, prefixes=2, scale=0.1, window=0, cap=0.0, out=OUT, o_row=5120, o_head=128,
             lse=None, ws=A * 16, ws_bytes=1 << 40)
    a.update(kw)
    return call("w4a16_prefix_attention", a["q"], a["type"], a["q_row"], a["q_head"], c or cache(call.w4), a["table"],
                a["stride"], a["max_pages"], a["lens"], a["batch"], a["heads"], a["ptable"], a["pstride"], a["ppages"],
                a["plens"], a["pof"], a["prefixes"], a["scale"], a["window"], a["cap"], a["out"], a["o_row"], a["o_head"],
                a["lse"], a["ws"], a["ws_bytes"], None)


def sample(call, **kw):
    a = dict(logits=A, type=0, row=50257, rows=3, vocab=50257, u=A, t=A, k=A, p=A, m=A, out=A)
    a.update(kw)
    return call("w4a16_sample", a["logits"], a["type"], a["row"], a["rows"], a["vocab"], a["u"], a["t"], a["k"], a["p"],
                a["m"], a["out"], None)


@pytest.fixture(params=[Direct, Block])
def call(request, w4):
    return request.param(w4)


BOTH = [
    (dict(type=2), INVALID), (dict(type=3), INVALID), (dict(type=1), UNSUPPORTED), (dict(batch=-1), INVALID),
    (dict(heads=0), INVALID), (dict(heads=41), INVALID), (dict(max_pages=0), INVALID), (dict(stride=63), INVALID),
    (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(cap=-1.0), INVALID), (dict(cap=float("inf")), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(q=BAD16), INVALID), (dict(out=BAD16), INVALID),
    (dict(lens=BAD4), INVALID), (dict(table=BAD4), INVALID), (dict(lse=BAD4), INVALID), (dict(q_row=5124), INVALID),
    (dict(q_head=-8), INVALID), (dict(o_row=5124), INVALID), (dict(o_head=-128), INVALID), (dict(out=A), INVALID),
    (dict(prefixes=-1), INVALID), (dict(ppages=0), INVALID), (dict(pstride=31), INVALID), (dict(ptable=None), INVALID),
    (dict(plens=None), INVALID), (dict(pof=None), INVALID), (dict(ptable=BAD4), INVALID), (dict(plens=BAD4), INVALID),
    (dict(pof=BAD4), INVALID), (dict(prefixes=2049), UNSUPPORTED), (dict(batch=8193), UNSUPPORTED),
    (dict(max_pages=1 << 27, stride=1 << 27), UNSUPPORTED),
    (dict(max_pages=1 << 26, stride=1 << 26, ppages=1 << 26, pstride=1 << 26), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws=A * 16 + 16), WORKSPACE), (dict(ws_bytes=0), WORKSPACE), (dict(batch=0), 0),
]


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(rows=-1), INVALID), (dict(starts=None), INVALID), (dict(starts=BAD4), INVALID), (dict(rows=(1 << 24) // 40 + 1), UNSUPPORTED),
    (dict(rows=200000, batch=8000, max_pages=1 << 26, stride=1 << 26, prefixes=0), UNSUPPORTED), (dict(rows=0), 0)])
def test_prompt_attention_refusals(call, kw, status):
    assert prompt(call, **kw) == status


@pytest.mark.parametrize("kw,status", BOTH + [(dict(prefixes=0), INVALID), (dict(heads=8 << 12, batch=1000), UNSUPPORTED)])
def test_prefix_attention_refusals(call, kw, status):
    assert prefix(call, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=BAD16), INVALID), (dict(pages=0), INVALID),
    (dict(page_size=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(type=3), INVALID),
    (dict(k_token=1028), INVALID), (dict(v_page=-8), INVALID), (dict(k_scale=A), INVALID), (dict(type=2, k_head=136), INVALID),
    (dict(type=2, k_scale=BAD4), INVALID), (dict(head_dim=132), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED),
    (dict(type=2, head_dim=72), UNSUPPORTED)])
def test_cache_refusals(call, kw, status):
    assert prompt(call, cache(call.w4, **kw)) == status and prefix(call, cache(call.w4, **kw)) == status
    assert prompt(call, cache(call.w4, **kw), rows=0) == status  # whatever there is to do


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(type=9), INVALID), (dict(rows=-1), INVALID), (dict(vocab=0), INVALID),
    (dict(vocab=-5), INVALID), (dict(row=-1), INVALID), (dict(row=50256), INVALID), (dict(vocab=(1 << 18) + 1, row=1 << 20), UNSUPPORTED),
    (dict(rows=(1 << 20) + 1), UNSUPPORTED), (dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(out=None), INVALID),
    (dict(logits=A + 1), INVALID), (dict(type=3, logits=A + 2), INVALID), (dict(out=A + 4), INVALID), (dict(u=BAD4), INVALID),
    (dict(t=BAD4), INVALID), (dict(k=BAD4), INVALID), (dict(p=BAD4), INVALID), (dict(m=BAD4), INVALID), (dict(rows=0), 0),
    (dict(rows=0, logits=None, u=None, out=None), 0)])
def test_sample_refusals(call, kw, status):
    assert sample(call, **kw) == status


def test_workspace_bytes(w4):
    for name, run in (("prompt", prompt), ("prefix", prefix)):
        f = getattr(w4, f"w4a16_{name}_attention_workspace_bytes")
        assert f(1, 40, 8, 128) > 0
        assert f(0, 40, 8, 128) == f(1, 41, 8, 128) == f(1, 40, 0, 128) == f(1, 8, 8, 0) == f(1, 8, 8, 264) == f(1 << 22, 8, 8, 64) == 0
        assert run(Direct(w4), ws_bytes=f(70 if name == "prompt" else 3, 40, 8, 128) - 1) == WORKSPACE


# Types of the header's blocks, as struct.pack names them.
KINDS = {"int": "i", "float": "f", "long long": "q", "size_t": "N"}


def test_blocks_are_laid_out_as_the_header_says(w4):
    text = open(os.path.join(ROOT, "include", "w4a16.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, form in w4._wide_blocks.items():
        fields = re.search(r"typedef struct \{([^}]*)\} %s_args;" % name, text).group(1)
        got = ""
        for line in fields.split(";"):
            if line := re.sub(r"\bconst\b", "", line).strip():
                kind, names = re.match(r"(long long|\w+)\s+(.*)", line, re.S).groups()
                for one in names.split(","):
                    got += "P" if "*" in one or "*" in names.split(",")[0] and "*" in one else KINDS[kind]
        assert got == form, name
        assert getattr(w4.lib, name + "_block")(None) == INVALID


# ------------------------------------------------------------------ binding
def test_binding_refusals(w4):
    half = lambda *s: torch.zeros(*s, dtype=torch.float16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    c = w4.KVCache(half(2, 16, 2, 64), half(2, 16, 2, 64))
    q, table, lens, starts, ws = half(5, 4, 64), i32(3, 4), i32(3), i32(4), torch.zeros(1 << 20, dtype=torch.uint8)

    def no(error, f, *args, **kw):
        with pytest.raises(error):
            f(*args, stream=0, **kw)

    run, shared = w4.w4a16_prompt_attention, w4.w4a16_prefix_attention
    kw = dict(out=torch.zeros_like(q), workspace=ws)
    no(ValueError, run, q, c, table, i32(3), lens, **kw)                    # starts
    no(ValueError, run, q, c, table, starts, i32(2), **kw)                  # lens
    no(ValueError, run, q[:, :, :32], c, table, starts, lens, **kw)         # head_dim
    no(ValueError, run, q, c, i32(12), starts, lens, **kw)                  # table
    no(ValueError, run, q, c, i32(4, 3).T, starts, lens, **kw)              # its rows have gaps
    no(ValueError, run, half(5, 64, 4).transpose(1, 2), c, table, starts, lens, **kw)
    no(TypeError, run, q, c, table.long(), starts, lens, **kw)
    no(TypeError, run, q, c, table, starts.long(), lens, **kw)
    no(TypeError, run, q.bfloat16(), c, table, starts, lens, **kw)          # out has another type
    no(TypeError, run, q, c, table, starts, lens, lse=half(5, 4), **kw)
    no(ValueError, run, q, c, table, starts, lens, lse=torch.zeros(5, 3), **kw)
    no(ValueError, run, q, c, table, starts, lens, prefix_of=lens, **kw)    # without a table
    no(ValueError, run, q, c, table, starts, lens, prefix_table=table, prefix_lens=lens, **kw)
    no(ValueError, run, q, c, table, starts, lens, prefix_table=table, prefix_lens=i32(2), prefix_of=lens, **kw)
    no(TypeError, run, q, c, table, starts, lens, prefix_table=table, prefix_lens=lens.long(), prefix_of=lens, **kw)
    no(ValueError, run, q, c, table, starts, lens, **kw)                    # not on a GPU
    for broadcast in (half(1, 4, 64).expand(5, 4, 64), half(5, 1, 64).expand(5, 4, 64)):
        with pytest.raises(ValueError, match="one place"):
            run(q, c, table, starts, lens, out=broadcast, workspace=ws, stream=0)
    one = q[:3]
    kw = dict(out=torch.zeros_like(one), workspace=ws)
    no(ValueError, shared, one, c, table, i32(2), table, lens, lens, **kw)
    no(ValueError, shared, one, c, i32(2, 4), lens, table, lens, lens, **kw)
    no(ValueError, shared, one, c, table, lens, table, lens, i32(2), **kw)
    no(TypeError, shared, one, c, table, lens, table, lens, lens.float(), **kw)
    no(ValueError, shared, one, c, table, lens, table, lens, lens, **kw)
    pick, x, u = w4.w4a16_sample, half(3, 40), torch.zeros(3)
    kw = dict(out=torch.zeros(3, dtype=torch.int64))
    no(ValueError, pick, half(40), u, **kw)
    no(ValueError, pick, half(40, 3).T, u, **kw)
    no(ValueError, pick, x, torch.zeros(2), **kw)
    no(TypeError, pick, x, u.half(), **kw)
    no(TypeError, pick, x, u, out=i32(3))
    no(TypeError, pick, x, u, top_k=torch.zeros(3), **kw)
    no(ValueError, pick, x, u, temperature=torch.ones(2), **kw)
    no(TypeError, pick, x, u, top_p=torch.ones(6)[::2], **kw)
    no(ValueError, pick, x, u, **kw)


# ------------------------------------------------------------------ oracle on worked examples
def test_oracle_rows_attention_sees_up_to_itself():
    k = np.array([[[0.0, 0.0]], [[np.log(3.0), 0.0]], [[0.0, np.log(2.0)]]])
    v = np.array([[[4.0, 0.0]], [[0.0, 8.0]], [[12.0, 4.0]]])
    q = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])
    out, lse, _, _ = ref.rows_attention(q, k, v, 1, 1.0)
    np.testing.assert_allclose(out[:, 0], [[1.0, 6.0], [7.0, 4.0]])  # weights 1, 3; then 1, 1, 2
    np.testing.assert_allclose(lse[:, 0], [np.log(4.0), np.log(4.0)])
    out, _, _, _ = ref.rows_attention(q, k, v, 1, 1.0, window=1)
    np.testing.assert_allclose(out[:, 0], v[1:, 0])


@pytest.mark.parametrize("kw,u,token", [
    (dict(), 0.0, 0), (dict(), 0.24, 0), (dict(), 0.26, 1), (dict(), 0.74, 1), (dict(), 0.76, 2), (dict(), 1.0, 3),
    (dict(top_k=2), 0.3, 0), (dict(top_k=2), 0.34, 1),        # 2/8 and 4/8 are left; of two equal ones the first
    # 0.75 (8 + 1e-9) is more than the first two's 6: three are left, and 0.3 of their 8 lies in the second.
    (dict(top_p=0.75), 0.3, 1), (dict(top_p=0.75), 0.99, 2), (dict(top_p=0.74), 0.3, 0), (dict(top_p=0.74), 0.99, 1),
    (dict(top_p=0.76), 0.99, 2),
    (dict(min_p=0.5), 0.99, 2), (dict(min_p=0.51), 0.0, 1), (dict(temperature=0.0), 0.9, 1), (dict(temperature=0.5), 0.16, 0),
    (dict(temperature=0.5), 0.2, 1)])
def test_oracle_sample_worked_example(kw, u, token):
    weights = [2.0, 4.0, 2.0, 1e-9]  # at temperature 0.5 4, 16, 4 of 24
    assert ref.sample(np.log(weights), u, **kw)[0] == token


def test_oracle_sample_odd_rows():
    inf = np.inf
    assert ref.sample([-inf, -inf], 0.5)[0] == -1 and ref.sample([np.nan, -inf, -3.0], 0.0)[0] == 2
    assert [ref.sample([1.0, inf, 2.0, inf], u)[0] for u in (0.2, 0.8)] == [1, 3]
