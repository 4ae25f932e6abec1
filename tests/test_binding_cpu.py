"""CPU checks of what the Python binding refuses before it hands addresses to the library, and of the argument blocks'
layout."""
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
