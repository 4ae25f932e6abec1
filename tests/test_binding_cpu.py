"""CPU checks of what the Python binding refuses before it hands addresses to the library, and of the argument blocks'
layout."""
import ctypes
import os
import re

import pytest
import torch


@pytest.fixture(scope="module")
def w4():
    import weight_only_int4_repack_gb300 as w4
    return w4


def projections(w4, a, out, gamma):
    """Every call of an int4 projection, over activations a [M, 256] and out [M, 256]."""
    q, s = torch.zeros(256, 128, dtype=torch.uint8), torch.ones(256, 2, dtype=torch.float16)
    w, kw = (q, s, None), dict(out=out, stream=0)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    return [lambda: w4.w4a16_gemm(a, *w, 128, **kw),
            lambda: w4.w4a16_gemm_swiglu(a, *w, *w, 128, workspace=ws, **kw),
            lambda: w4.w4a16_gemm_rmsnorm(a, gamma, 1e-5, *w, 128, workspace=ws, **kw),
            lambda: w4.w4a16_gemm_swiglu_rmsnorm(a, gamma, 1e-5, *w, *w, 128, workspace=ws, **kw),
            lambda: w4.w4a16_gemm_swiglu_unfused_static(a, *w, *w, 128, **kw),
            lambda: w4.w4a16_gemm_host_io(a, a, *w, 128, out, out, stream=0)]


@pytest.mark.parametrize("wrong", ["activations", "out", "strided activations", "strided out"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_projections_take_contiguous_fp16_only(w4, wrong, dtype):
    # The operators between them also work in bf16 and on views, whose bits mean something else here.
    good, wide = torch.zeros(3, 256, dtype=torch.float16), torch.zeros(3, 300, dtype=torch.float16)
    bad = wide[:, :256] if "strided" in wrong else good.to(dtype)
    a, out = (bad, good) if "activations" in wrong else (good, bad)
    for call in projections(w4, a, out, good[0]):
        with pytest.raises(TypeError):
            call()


def test_rmsnorm_projections_take_fp16_gamma_only(w4):
    good = torch.zeros(3, 256, dtype=torch.float16)
    for call in projections(w4, good, good, torch.ones(256, dtype=torch.bfloat16))[2:4]:
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ the argument blocks against the header
def header_struct(name):
    """(field, type) of a struct of include/w4a16.h, in its order; "*" for every pointer."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "w4a16.h")) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    body = re.search(r"typedef struct \{([^{}]*)\} %s;" % name, text).group(1)
    fields = []
    for line in filter(None, (part.strip() for part in body.split(";"))):
        kind, names = re.match(r"((?:const )?(?:long long|\w+))\s+(.*)", line, flags=re.S).groups()
        for n in names.split(","):
            fields.append((n.strip().lstrip("*").strip(), "*" if "*" in n else kind))
    return fields


LETTERS = {"*": "P", "int": "i", "long long": "q", "float": "f", "size_t": "N"}


def test_blocks_are_laid_out_as_in_the_header(w4):
    assert len(w4._blocks) == 4
    for name, letters in w4._blocks.items():
        assert "".join(LETTERS[kind] for _, kind in header_struct(name + "_args")) == letters, name


def test_cache_is_laid_out_as_in_the_header(w4):
    kinds = {ctypes.c_void_p: "*", ctypes.c_longlong: "long long", ctypes.c_int: "int"}
    assert [(n, kinds[t]) for n, t in w4.KVCache._fields_] == header_struct("w4a16_kv_cache")
