"""Python binding of libw4a16.so (fp16 x int4 group-quantized GEMM for GB300, and
the operators between two such GEMMs of a decoder layer).

Argument marshalling only: every step of the computation runs in the CUDA
library. PyTorch supplies device memory and the current stream. The functions
carry the C ABI's names (include/w4a16.h); `lib` is the raw ctypes handle. A call with
`stream` runs there; outputs and workspaces that it makes belong to that stream, inputs
have to be ready on it.

Importing fails loudly when the compiled library is missing: there is no CPU or
PyTorch fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a16.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                      f"g.build()'` (needs nvcc); there is no fallback implementation")

# torch first: the library links the shared CUDA runtime by soname, so it must
# resolve to the runtime torch already loaded (one runtime per process).
import torch  # noqa: E402,F401

lib = ctypes.CDLL(LIB_PATH)

# Status codes and enums (mirror include/w4a16.h).
W4A16_OK = 0
W4A16_ERR_INVALID_ARG = 1
W4A16_ERR_UNSUPPORTED = 2
W4A16_ERR_WORKSPACE = 3
W4A16_ERR_CUDA = 4
W4A16_ERR_TIMEOUT = 5
W4A16_SCALE_F16 = 0
W4A16_SCALE_F32 = 1
W4A16_PATH_SMALL_M = 0
W4A16_PATH_TCGEN05 = 1
W4A16_TYPE_F16 = 0
W4A16_TYPE_BF16 = 1
W4A16_TYPE_E4M3 = 2
W4A16_TYPE_F32 = 3

EXPORTS = (
    "w4a16_status_string", "w4a16_repacked_bytes", "w4a16_repack", "w4a16_unpack_host",
    "w4a16_gemm_workspace_bytes", "w4a16_gemm_plan", "w4a16_gemm",
    "w4a16_swiglu_workspace_bytes", "w4a16_gemm_swiglu", "w4a16_set_tuning", "w4a16_set_launch_overlap",
    "w4a16_device_error", "w4a16_swiglu_static_scratch_bytes", "w4a16_gemm_swiglu_unfused_static",
    "w4a16_set_wait_limit_ns", "w4a16_rmsnorm_workspace_bytes", "w4a16_gemm_rmsnorm",
    "w4a16_gemm_swiglu_rmsnorm", "w4a16_gemm_launch_info", "w4a16_gemm_host_io",
    "w4a16_kv_extend", "w4a16_rope_frequencies", "w4a16_rope_append",
    "w4a16_paged_attention_workspace_bytes", "w4a16_paged_attention", "w4a16_residual_rmsnorm",
    "w4a16_kv_extend_block", "w4a16_rope_append_block", "w4a16_paged_attention_block",
    "w4a16_residual_rmsnorm_block",
    "w4a16_prompt_attention_workspace_bytes", "w4a16_prompt_attention", "w4a16_prompt_attention_block",
    "w4a16_prefix_attention_workspace_bytes", "w4a16_prefix_attention", "w4a16_prefix_attention_block",
    "w4a16_sample", "w4a16_sample_block",
)

_vp, _ci, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_ll, _cf, _cd = ctypes.c_longlong, ctypes.c_float, ctypes.c_double


class LaunchInfo(ctypes.Structure):
    """w4a16_launch_info: launch shape of the kernel a call would run."""
    _fields_ = [("path", _ci), ("split", _ci), ("ctas", _ci), ("threads", _ci), ("smem_bytes", _ci),
                ("stages", _ci)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


_int32, _int64, _float32 = torch.int32, torch.int64, torch.float32
_TYPES = {torch.float16: W4A16_TYPE_F16, torch.bfloat16: W4A16_TYPE_BF16,
          torch.float8_e4m3fn: W4A16_TYPE_E4M3, torch.float32: W4A16_TYPE_F32}


class KVCache(ctypes.Structure):
    """w4a16_kv_cache over two pools of pages, CUDA tensors [pages, page_size, kv_heads,
    head_dim] of float16, bfloat16 or float8_e4m3fn. Any order of the first three
    dimensions will do (pass a transposed view of pools that are laid out heads first);
    head_dim is contiguous. k_scale, v_scale: float32 [kv_heads], float8_e4m3fn only.
    Made once for a cache and passed to every call; holds on to its tensors."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp),
                ("k_page", _ll), ("k_token", _ll), ("k_head", _ll),
                ("v_page", _ll), ("v_token", _ll), ("v_head", _ll),
                ("type", _ci), ("pages", _ci), ("page_size", _ci), ("kv_heads", _ci), ("head_dim", _ci)]

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v are two pools [pages, page_size, kv_heads, head_dim] of one type")
        if k.dtype not in _TYPES or k.dtype == torch.float32:
            raise TypeError("a cache is float16, bfloat16 or float8_e4m3fn")
        if k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("head_dim must be contiguous")
        for s in (k_scale, v_scale):
            if s is not None:
                _expect(s, torch.float32, "k_scale, v_scale")
                if s.numel() != k.shape[2]:
                    raise ValueError("one scale for each kv head")
        super().__init__(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), *_steps(k), *_steps(v),
                         _TYPES[k.dtype], *k.shape)
        self.tensors = (k, v, k_scale, v_scale)
        self.address = ctypes.addressof(self)


def _steps(t):
    """Strides of all dimensions but the last; 0 where there is one entry only, whose stride says nothing."""
    n, step = t.shape, t.stride()
    return [step[i] if n[i] > 1 else 0 for i in range(len(n) - 1)]


def _expect(t, dtype, what):
    if t.dtype is not dtype or not t.is_contiguous():
        raise TypeError(f"{what}: contiguous {dtype} expected")


_kv = ctypes.POINTER(KVCache)

_sig = {
    "w4a16_status_string": (ctypes.c_char_p, [_ci]),
    "w4a16_repacked_bytes": (_sz, [_ci, _ci]),
    "w4a16_repack": (_ci, [_vp, _vp, _ci, _ci, _vp]),
    "w4a16_unpack_host": (_ci, [_vp, _vp, _ci, _ci]),
    "w4a16_gemm_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci]),
    "w4a16_gemm_plan": (_ci, [_ci, _ci, _ci, _ci, _ci, ctypes.POINTER(_ci), ctypes.POINTER(_ci)]),
    "w4a16_gemm_launch_info": (_ci, [_ci, _ci, _ci, _ci, _ci, _ci, ctypes.POINTER(LaunchInfo)]),
    "w4a16_gemm": (_ci, [_vp, _vp, _vp, _ci, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _vp, _sz, _vp]),
    "w4a16_gemm_host_io": (_ci, [_vp, _vp, _vp, _vp, _ci, _vp, _vp, _vp, _ci, _ci, _ci, _ci, _ci, _vp]),
    "w4a16_swiglu_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci]),
    "w4a16_gemm_swiglu": (_ci, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _vp,
                                _ci, _ci, _ci, _ci, _ci, _vp, _sz, _vp]),
    "w4a16_set_tuning": (_ci, [_ci]),
    "w4a16_set_launch_overlap": (_ci, [_ci]),
    "w4a16_device_error": (_ci, [_vp]),
    "w4a16_set_wait_limit_ns": (_ci, [ctypes.c_ulonglong]),
    "w4a16_rmsnorm_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci, _ci]),
    "w4a16_gemm_rmsnorm": (_ci, [_vp, _vp, ctypes.c_float, _vp, _vp, _ci, _vp, _vp, _ci, _ci, _ci, _ci, _ci,
                                 _vp, _sz, _vp]),
    "w4a16_gemm_swiglu_rmsnorm": (_ci, [_vp, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _vp,
                                        _ci, _ci, _ci, _ci, _ci, _vp, _sz, _vp]),
    "w4a16_swiglu_static_scratch_bytes": (_sz, []),
    "w4a16_gemm_swiglu_unfused_static": (_ci, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _ci, _vp,
                                               _ci, _ci, _ci, _ci, _vp]),
    "w4a16_kv_extend": (_ci, [_vp, _vp, _vp, _ll, _ci, _ci, _ci, _vp, _ci, _vp, _vp, _vp, _vp, _vp, _ci, _vp,
                              _ci, _vp]),
    "w4a16_rope_frequencies": (_ci, [_vp, _ci, _cd, _ci, _cd, _cd, _cd, _cd]),
    "w4a16_rope_append": (_ci, [_vp, _vp, _vp, _ci, _ll, _ll, _ll, _ll, _ll, _ll, _vp, _vp, _vp, _ci, _ci, _cf,
                                _vp, _ll, _ll, _kv, _vp, _ci, _ci, _vp]),
    "w4a16_paged_attention_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci]),
    "w4a16_paged_attention": (_ci, [_vp, _ci, _ll, _ll, _kv, _vp, _ll, _ci, _vp, _ci, _ci, _cf, _ci, _cf, _vp,
                                    _ll, _ll, _vp, _vp, _sz, _vp]),
    "w4a16_residual_rmsnorm": (_ci, [_vp, _ci, _ll, _vp, _ci, _ll, _vp, _vp, _ll, _cf, _vp, _cf, _vp, _ll, _vp,
                                     _ll, _ci, _ci, _vp]),
}
# The same calls with their arguments in one block: packed by `struct` in the parameters' order (native alignment, as
# the C structs of include/w4a16.h), which costs a fifth of what ctypes takes to convert them one by one.
_blocks = {
    "w4a16_kv_extend": "PPPqiiiPiPPPPPiPiP",
    "w4a16_rope_append": "PPPiqqqqqqPPPiifPqqPPiiP",
    "w4a16_paged_attention": "PiqqPPqiPiififPqqPPNP",
    "w4a16_residual_rmsnorm": "PiqPiqPPqfPfPqPqiiP",
}
# Those of the attention of many rows, and of sampling.
_wide_blocks = {
    "w4a16_prompt_attention": "PiqqPPqiPPiiiPqiPPififPqqPPNP",
    "w4a16_prefix_attention": "PiqqPPqiPiiPqiPPififPqqPPNP",
    "w4a16_sample": "PiqiiPPPPPPP",
}
_sig.update({
    "w4a16_prompt_attention_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci]),
    "w4a16_prompt_attention": (_ci, [_vp, _ci, _ll, _ll, _kv, _vp, _ll, _ci, _vp, _vp, _ci, _ci, _ci, _vp, _ll, _ci, _vp,
                                     _vp, _ci, _cf, _ci, _cf, _vp, _ll, _ll, _vp, _vp, _sz, _vp]),
    "w4a16_prefix_attention_workspace_bytes": (_sz, [_ci, _ci, _ci, _ci]),
    "w4a16_prefix_attention": (_ci, [_vp, _ci, _ll, _ll, _kv, _vp, _ll, _ci, _vp, _ci, _ci, _vp, _ll, _ci, _vp, _vp, _ci,
                                     _cf, _ci, _cf, _vp, _ll, _ll, _vp, _vp, _sz, _vp]),
    "w4a16_sample": (_ci, [_vp, _ci, _ll, _ci, _ci, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
})
_sig.update({_name + "_block": (_ci, [ctypes.c_char_p]) for _name in (*_blocks, *_wide_blocks)})
for _name, (_res, _args) in _sig.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args
_pack_extend, _pack_rope, _pack_attention, _pack_norm = (struct.Struct(_blocks[_name]).pack for _name in _blocks)
_extend, _rope, _attention, _norm = (getattr(lib, _name + "_block") for _name in _blocks)
_pack_prompt, _pack_prefix, _pack_sample = (struct.Struct(_wide_blocks[_name]).pack for _name in _wide_blocks)
_prompt, _prefix, _sample = (getattr(lib, _name + "_block") for _name in _wide_blocks)


class W4A16Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {w4a16_status_string(status)} (status {status})")


def w4a16_status_string(status: int) -> str:
    return lib.w4a16_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != W4A16_OK:
        raise W4A16Error(status, where)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The current stream as a number. torch.cuda.current_stream() builds a Stream object for it, about 3 us a call on the
# host, as long as a small kernel runs; the getter behind it takes 0.1.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None and _current_device is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _new(shape, dtype, like, stream, make=torch.empty):
    """A tensor on `like`'s device for a call on `stream`. Made under that stream: it is cleared there, if at all, and its
    memory is not given to work of another stream while the call may still use it."""
    if stream is None or _stream(stream) == _stream(None):
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, like.device) if isinstance(stream, int) else stream):
        return make(shape, dtype=dtype, device=like.device)


def _placed(where, *tensors):
    """Refuses tensors that the call's kernels, which run on the current device, cannot be given."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"{where}: tensors on different devices")
    if device < 0 or device != (torch.cuda.current_device() if _current_device is None else _current_device()):
        raise ValueError(f"{where}: tensors on the current CUDA device expected")


def _expect_half(*tensors):
    """The projections read and write contiguous float16 and are handed addresses only."""
    for t in tensors:
        if t is not None and (t.dtype is not torch.float16 or not t.is_contiguous()):
            raise TypeError(f"activations, gamma and out: contiguous torch.float16 expected, got {t.dtype}"
                            f"{'' if t.is_contiguous() else ' with gaps'}")


def w4a16_repacked_bytes(N: int, K: int) -> int:
    return int(lib.w4a16_repacked_bytes(N, K))


def w4a16_repack(q, out=None, stream=None):
    """q: uint8 CUDA tensor [N, K/2] -> repacked uint8 CUDA tensor [N*K/2]."""
    import torch
    N, K = q.shape[0], 2 * q.shape[1]
    if out is None:
        out = _new(w4a16_repacked_bytes(N, K), torch.uint8, q, stream)
    _check(lib.w4a16_repack(_ptr(q), _ptr(out), N, K, _stream(stream)), "w4a16_repack")
    return out


def w4a16_unpack_host(q_rep, N: int, K: int):
    """Host inverse of the repack (numpy in, numpy out)."""
    import numpy as np
    src = np.ascontiguousarray(np.asarray(q_rep, dtype=np.uint8).reshape(-1))
    if src.size != N * K // 2:
        raise ValueError("q_rep has the wrong size")
    dst = np.empty((N, K // 2), dtype=np.uint8)
    _check(lib.w4a16_unpack_host(src.ctypes.data, dst.ctypes.data, N, K), "w4a16_unpack_host")
    return dst


def w4a16_gemm_workspace_bytes(M, N, K, group, split_k=0) -> int:
    return int(lib.w4a16_gemm_workspace_bytes(M, N, K, group, split_k))


def w4a16_gemm_plan(M, N, K, group, split_k=0) -> Tuple[int, int]:
    path, split = _ci(), _ci()
    _check(lib.w4a16_gemm_plan(M, N, K, group, split_k, ctypes.byref(path), ctypes.byref(split)),
           "w4a16_gemm_plan")
    return path.value, split.value


def w4a16_gemm_launch_info(M, N, K, group, split_k=0, swiglu_fused=False) -> dict:
    """Launch shape of w4a16_gemm (or fused w4a16_gemm_swiglu): path, split, ctas,
    threads, smem_bytes, stages."""
    info = LaunchInfo()
    _check(lib.w4a16_gemm_launch_info(M, N, K, group, split_k, int(bool(swiglu_fused)), ctypes.byref(info)),
           "w4a16_gemm_launch_info")
    return info.as_dict()


def _scale_dtype(scales) -> int:
    import torch
    if scales.dtype == torch.float16:
        return W4A16_SCALE_F16
    if scales.dtype == torch.float32:
        return W4A16_SCALE_F32
    raise TypeError("scales must be float16 or float32")


def w4a16_gemm(A, q_rep, scales, zp, group: int, out=None, split_k: int = 0, workspace=None,
               stream=None):
    """Y[M, N] = A[M, K] . dequant(q_rep)^T (all CUDA tensors; zp may be None)."""
    _expect_half(A, out)
    M, K = A.shape
    N = scales.shape[0]
    if out is None:
        out = _new((M, N), torch.float16, A, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.w4a16_gemm(_ptr(A), _ptr(q_rep), _ptr(scales), _scale_dtype(scales), _ptr(zp),
                          _ptr(out), M, N, K, group, split_k, _ptr(workspace), ws_bytes,
                          _stream(stream)), "w4a16_gemm")
    return out


def w4a16_gemm_host_io(A_host, A_dev, q_rep, scales, zp, group: int, Y_dev, Y_host, split_k: int = 0,
                       stream=None):
    """Copy A_host (pinned CPU fp16 [M, K]) into A_dev, run the GEMM into Y_dev and
    copy it into Y_host (pinned CPU fp16 [M, N]), all enqueued on the stream; no
    synchronisation (Y_host is valid once the stream has passed the call)."""
    _expect_half(A_host, A_dev, Y_dev, Y_host)
    M, K = A_host.shape
    N = scales.shape[0]
    _check(lib.w4a16_gemm_host_io(_ptr(A_host), _ptr(A_dev), _ptr(q_rep), _ptr(scales), _scale_dtype(scales),
                                  _ptr(zp), _ptr(Y_dev), _ptr(Y_host), M, N, K, group, split_k,
                                  _stream(stream)), "w4a16_gemm_host_io")
    return Y_host


def w4a16_swiglu_workspace_bytes(M, N, K, group, fused) -> int:
    return int(lib.w4a16_swiglu_workspace_bytes(M, N, K, group, int(bool(fused))))


def w4a16_gemm_swiglu(A, qg_rep, sg, zg, qu_rep, su, zu, group: int, fused: bool = True,
                      out=None, workspace=None, stream=None):
    """Y = silu(A . Wg^T) * (A . Wu^T); fused or the unfused three-kernel chain."""
    _expect_half(A, out)
    M, K = A.shape
    N = sg.shape[0]
    if out is None:
        out = _new((M, N), torch.float16, A, stream)
    need = w4a16_swiglu_workspace_bytes(M, N, K, group, fused)
    if workspace is None and need:
        workspace = _new(need, torch.uint8, A, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.w4a16_gemm_swiglu(_ptr(A), _ptr(qg_rep), _ptr(sg), _ptr(zg), _ptr(qu_rep),
                                 _ptr(su), _ptr(zu), _scale_dtype(sg), _ptr(out), M, N, K, group,
                                 int(bool(fused)), _ptr(workspace), ws_bytes, _stream(stream)),
           "w4a16_gemm_swiglu")
    return out


def w4a16_rmsnorm_workspace_bytes(M, N, K, group, mode) -> int:
    return int(lib.w4a16_rmsnorm_workspace_bytes(M, N, K, group, mode))


def w4a16_gemm_rmsnorm(A, gamma, eps: float, q_rep, scales, zp, group: int, out=None, split_k: int = 0,
                       workspace=None, stream=None):
    """Y = rmsnorm(A; gamma, eps) . dequant(q_rep)^T (normalised A staged in the workspace)."""
    _expect_half(A, gamma, out)
    M, K = A.shape
    N = scales.shape[0]
    if out is None:
        out = _new((M, N), torch.float16, A, stream)
    if workspace is None:
        workspace = _new(w4a16_rmsnorm_workspace_bytes(M, N, K, group, 0), torch.uint8, A, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.w4a16_gemm_rmsnorm(_ptr(A), _ptr(gamma), float(eps), _ptr(q_rep), _ptr(scales),
                                  _scale_dtype(scales), _ptr(zp), _ptr(out), M, N, K, group, split_k,
                                  _ptr(workspace), ws_bytes, _stream(stream)), "w4a16_gemm_rmsnorm")
    return out


def w4a16_gemm_swiglu_rmsnorm(A, gamma, eps: float, qg_rep, sg, zg, qu_rep, su, zu, group: int,
                              fused: bool = True, out=None, workspace=None, stream=None):
    """Y = silu(An . Wg^T) * (An . Wu^T), An = rmsnorm(A; gamma, eps)."""
    _expect_half(A, gamma, out)
    M, K = A.shape
    N = sg.shape[0]
    if out is None:
        out = _new((M, N), torch.float16, A, stream)
    if workspace is None:
        workspace = _new(w4a16_rmsnorm_workspace_bytes(M, N, K, group, 1 if fused else 2), torch.uint8, A, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.w4a16_gemm_swiglu_rmsnorm(_ptr(A), _ptr(gamma), float(eps), _ptr(qg_rep), _ptr(sg), _ptr(zg),
                                         _ptr(qu_rep), _ptr(su), _ptr(zu), _scale_dtype(sg), _ptr(out),
                                         M, N, K, group, int(bool(fused)), _ptr(workspace), ws_bytes,
                                         _stream(stream)), "w4a16_gemm_swiglu_rmsnorm")
    return out


def w4a16_swiglu_static_scratch_bytes() -> int:
    return int(lib.w4a16_swiglu_static_scratch_bytes())


def w4a16_gemm_swiglu_unfused_static(A, qg_rep, sg, zg, qu_rep, su, zu, group: int, out=None,
                                     stream=None):
    """Unfused SwiGLU whose intermediates live in the library's fixed device
    array: for callers that cannot allocate device memory (see include/w4a16.h)."""
    _expect_half(A, out)
    M, K = A.shape
    N = sg.shape[0]
    if out is None:
        out = _new((M, N), torch.float16, A, stream)
    _check(lib.w4a16_gemm_swiglu_unfused_static(_ptr(A), _ptr(qg_rep), _ptr(sg), _ptr(zg),
                                                _ptr(qu_rep), _ptr(su), _ptr(zu),
                                                _scale_dtype(sg), _ptr(out), M, N, K, group,
                                                _stream(stream)),
           "w4a16_gemm_swiglu_unfused_static")
    return out


def w4a16_kv_extend(lens, new_tokens, table, free_pages, free_count, page_size: int, slots, positions, refused,
                    lens_out=None, count_out=None, spacing: int = 0, stream=None):
    """Places for a step's new tokens: pages taken from (and, where new_tokens is negative,
    given back to) the free list, the block table grown, a slot and a position for every
    token (packed, or request b's from entry b*spacing on). All int32 CUDA tensors but
    slots (int64); see include/w4a16.h. lens and
    free_count are updated in place unless lens_out / count_out are given. Returns lens."""
    lens_out = lens if lens_out is None else lens_out
    count_out = free_count if count_out is None else count_out
    batch, max_pages = table.shape
    if not (lens.dtype is new_tokens.dtype is free_pages.dtype is free_count.dtype is positions.dtype is refused.dtype
            is lens_out.dtype is count_out.dtype is table.dtype is _int32) or slots.dtype is not _int64:
        raise TypeError("w4a16_kv_extend: slots is int64, everything else int32")
    n_slots = slots.numel()
    if (not (lens.is_contiguous() and new_tokens.is_contiguous() and free_pages.is_contiguous() and slots.is_contiguous()
             and positions.is_contiguous() and refused.is_contiguous() and (lens_out is lens or lens_out.is_contiguous()))
            or (max_pages > 1 and table.stride(1) != 1)
            or not lens.numel() == new_tokens.numel() == refused.numel() == lens_out.numel() == batch
            or positions.numel() != n_slots):
        raise ValueError("w4a16_kv_extend: table is [batch, max_pages], the others are contiguous with one entry for "
                         "each request or slot")
    status = _extend(_pack_extend(
        lens.data_ptr(), new_tokens.data_ptr(), table.data_ptr(), table.stride(0) if batch > 1 else max_pages, batch,
        max_pages, page_size, free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(), lens_out.data_ptr(),
        count_out.data_ptr(), slots.data_ptr(), positions.data_ptr(), n_slots, refused.data_ptr(), spacing,
        _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_kv_extend")
    return lens_out


def w4a16_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = 0, factor: float = 1.0,
                           context: float = 0.0, low: float = 1.0, high: float = 32.0):
    """The rot_dim/2 inverse frequencies as a CPU float32 tensor; scaling 0..3 as in include/w4a16.h (3 goes from one
    to the other linearly in turns within the context, from `low` to `high` of them)."""
    out = torch.empty(max(0, rot_dim) // 2, dtype=torch.float32)
    _check(lib.w4a16_rope_frequencies(out.data_ptr() or None, rot_dim, base, scaling, factor, context, low, high),
           "w4a16_rope_frequencies")
    return out


def w4a16_rope_append(q, k, v, positions, inv_freq, cache, slots, interleaved: bool = False, mscale: float = 1.0,
                      bias=None, out=None, stream=None):
    """Rotary positions for q [rows, heads, D] and k [rows, kv_heads, D] (their first
    2*len(inv_freq) elements), k and v into the cache at `slots`; returns the turned q.
    q, k, v may be views of one joined projection; out may be q."""
    rows, heads, D = q.shape
    if out is None:
        out = _new((rows, heads, D), q.dtype, q, stream)
    if (positions.dtype is not _int32 or slots.dtype is not _int64 or inv_freq.dtype is not _float32
            or not (positions.is_contiguous() and slots.is_contiguous() and inv_freq.is_contiguous())):
        raise TypeError("w4a16_rope_append: positions int32, slots int64, inv_freq float32, contiguous")
    sq, sk, sv, so = q.stride(), k.stride(), v.stride(), out.stride()
    if (k.shape != (rows, cache.kv_heads, D) or v.shape != k.shape or out.shape != q.shape or D != cache.head_dim
            or positions.numel() != rows or slots.numel() != rows or sq[2] != 1 or sk[2] != 1 or sv[2] != 1
            or so[2] != 1):
        raise ValueError("w4a16_rope_append: q, out [rows, heads, D], k, v [rows, kv_heads, D], positions and slots "
                         "[rows], D contiguous and the cache's")
    if not q.dtype is k.dtype is v.dtype is out.dtype:
        raise TypeError("w4a16_rope_append: q, k, v and out have one type")
    if bias is not None:
        _expect(bias, q.dtype, "bias")
        if bias.numel() != (heads + 2 * cache.kv_heads) * D:
            raise ValueError("bias: (heads + 2*kv_heads) * head_dim elements")
    many, kv = rows > 1, cache.kv_heads > 1  # strides over one entry say nothing
    status = _rope(_pack_rope(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _TYPES.get(q.dtype, -1), sq[0] if many else 0,
        sq[1] if heads > 1 else 0, sk[0] if many else 0, sk[1] if kv else 0, sv[0] if many else 0, sv[1] if kv else 0,
        0 if bias is None else bias.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), 2 * inv_freq.numel(),
        interleaved, mscale, out.data_ptr(), so[0] if many else 0, so[1] if heads > 1 else 0, cache.address,
        slots.data_ptr(), rows, heads, _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_rope_append")
    return out


def w4a16_paged_attention_workspace_bytes(batch: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib.w4a16_paged_attention_workspace_bytes(batch, heads, kv_heads, head_dim))


def w4a16_paged_attention(q, cache, table, lens, scale: Optional[float] = None, window: int = 0,
                          softcap: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token of each request, q [batch, heads, D], over its pages of
    the cache (table int32 [batch, max_pages], lens int32 [batch], the new token counted).
    scale defaults to D ** -0.5; lse (float32 [batch, heads]) is written if given.
    workspace: w4a16_paged_attention_workspace_bytes() of uint8, zeroed once before its
    first use and then kept for further calls; made here if it is not given."""
    batch, heads, D = q.shape
    max_pages = table.shape[1]
    if out is None:
        out = _new((batch, heads, D), q.dtype, q, stream)
    if workspace is None:
        need = w4a16_paged_attention_workspace_bytes(batch, heads, cache.kv_heads, D)
        workspace = _new(need, torch.uint8, q, stream, torch.zeros)
    sq, so = q.stride(), out.stride()
    if (D != cache.head_dim or table.shape[0] != batch or lens.numel() != batch or out.shape != q.shape
            or sq[2] != 1 or so[2] != 1 or (max_pages > 1 and table.stride(1) != 1)):
        raise ValueError("w4a16_paged_attention: q, out [batch, heads, D], table [batch, max_pages], lens [batch], D "
                         "contiguous and the cache's")
    if (q.dtype is not out.dtype or not table.dtype is lens.dtype is _int32 or not lens.is_contiguous()):
        raise TypeError("w4a16_paged_attention: q and out have one type, table and lens are int32, lens contiguous")
    if lse is not None:
        _expect(lse, torch.float32, "lse")
        if lse.numel() != batch * heads:
            raise ValueError("lse: [batch, heads]")
    many = batch > 1  # strides over one entry say nothing
    status = _attention(_pack_attention(
        q.data_ptr(), _TYPES.get(q.dtype, -1), sq[0] if many else 0, sq[1] if heads > 1 else 0, cache.address,
        table.data_ptr(), table.stride(0) if many else max_pages, max_pages, lens.data_ptr(), batch, heads,
        D ** -0.5 if scale is None else scale, window, softcap, out.data_ptr(), so[0] if many else 0,
        so[1] if heads > 1 else 0,
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_paged_attention")
    return out


def _prefixes(where, batch, prefix_table, prefix_lens, prefix_of):
    """The arguments of shared prefixes as they go into a block: (table, stride, pages, lens, of, prefixes)."""
    if prefix_table is None:
        if prefix_lens is not None or prefix_of is not None:
            raise ValueError(f"{where}: prefix_lens and prefix_of come with prefix_table")
        return 0, 0, 0, 0, 0, 0
    if prefix_lens is None or prefix_of is None or prefix_table.dim() != 2:
        raise ValueError(f"{where}: prefix_table [prefixes, pages] comes with prefix_lens and prefix_of")
    n, pages = prefix_table.shape
    if not (prefix_table.dtype is prefix_lens.dtype is prefix_of.dtype is _int32):
        raise TypeError(f"{where}: prefix_table, prefix_lens and prefix_of are int32")
    if (prefix_lens.numel() != n or prefix_of.numel() != batch or not prefix_lens.is_contiguous()
            or not prefix_of.is_contiguous() or (pages > 1 and prefix_table.stride(1) != 1)):
        raise ValueError(f"{where}: prefix_table [prefixes, pages], prefix_lens [prefixes], prefix_of [batch]")
    return (prefix_table.data_ptr(), prefix_table.stride(0) if n > 1 else pages, pages, prefix_lens.data_ptr(),
            prefix_of.data_ptr(), n)


def _attention_tensors(where, q, cache, table, out, lse, *ints):
    """What prompt and prefix attention expect alike of their tensors. Returns q's and out's strides."""
    if q.dim() != 3 or table.dim() != 2 or out.shape != q.shape or q.shape[2] != cache.head_dim:
        raise ValueError(f"{where}: q, out [rows, heads, D], D the cache's, table [batch, max_pages]")
    if q.dtype is not out.dtype or table.dtype is not _int32:
        raise TypeError(f"{where}: q and out have one type, table is int32")
    sq, so = q.stride(), out.stride()
    if sq[2] != 1 or so[2] != 1 or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"{where}: D and the table's rows are contiguous")
    for t in ints:
        _expect(t, _int32, f"{where}: starts, lens")
    if lse is not None:
        _expect(lse, _float32, "lse")
        if lse.numel() != q.shape[0] * q.shape[1]:
            raise ValueError("lse: [rows, heads]")
    rows, heads = q.shape[0] > 1, q.shape[1] > 1  # strides over one entry say nothing
    if (rows and so[0] == 0) or (heads and so[1] == 0):
        raise ValueError(f"{where}: rows of out lie in one place")
    return sq[0] if rows else 0, sq[1] if heads else 0, so[0] if rows else 0, so[1] if heads else 0


def w4a16_prompt_attention_workspace_bytes(rows: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib.w4a16_prompt_attention_workspace_bytes(rows, heads, kv_heads, head_dim))


def w4a16_prompt_attention(q, cache, table, starts, lens, scale: Optional[float] = None, window: int = 0,
                           softcap: float = 0.0, prefix_table=None, prefix_lens=None, prefix_of=None, out=None, lse=None,
                           workspace=None, stream=None):
    """Attention of several new tokens of each request, q [rows, heads, D]: request b's are the rows from starts[b] up
    to starts[b + 1] (int32 [batch + 1]), the newest of its lens[b] tokens in the cache; each sees the keys up to its
    own. With prefix_table (int32 [prefixes, pages]), prefix_lens and prefix_of (int32 [batch], negative: none) the
    tokens of a shared prefix come in front of the request's own. Rows of no request are left as they are in `out` (and
    as torch.empty gives them where it is made here). lse: float32 [rows, heads], written if given.
    workspace: w4a16_prompt_attention_workspace_bytes() of uint8; made here if it is not given."""
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    q_row, q_head, o_row, o_head = _attention_tensors("w4a16_prompt_attention", q, cache, table, out, lse, starts, lens)
    rows, heads, D = q.shape
    batch, max_pages = table.shape
    if starts.numel() != batch + 1 or lens.numel() != batch:
        raise ValueError("w4a16_prompt_attention: starts [batch + 1], lens [batch]")
    prefixes = _prefixes("w4a16_prompt_attention", batch, prefix_table, prefix_lens, prefix_of)
    if workspace is None:
        workspace = _new(w4a16_prompt_attention_workspace_bytes(rows, heads, cache.kv_heads, D), torch.uint8, q, stream)
    _placed("w4a16_prompt_attention", q, out, table, starts, lens, lse, workspace, prefix_table, prefix_lens, prefix_of,
            *cache.tensors)
    status = _prompt(_pack_prompt(
        q.data_ptr(), _TYPES.get(q.dtype, -1), q_row, q_head, cache.address, table.data_ptr(),
        table.stride(0) if batch > 1 else max_pages, max_pages, starts.data_ptr(), lens.data_ptr(), rows, batch, heads,
        *prefixes, D ** -0.5 if scale is None else scale, window, softcap, out.data_ptr(), o_row, o_head,
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_prompt_attention")
    return out


def w4a16_prefix_attention_workspace_bytes(batch: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib.w4a16_prefix_attention_workspace_bytes(batch, heads, kv_heads, head_dim))


def w4a16_prefix_attention(q, cache, table, lens, prefix_table, prefix_lens, prefix_of, scale: Optional[float] = None,
                           window: int = 0, softcap: float = 0.0, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token of each request, q [batch, heads, D], as w4a16_paged_attention, where request b's own
    tokens (table, lens) come behind those of prefix prefix_of[b] (int32 [batch], negative: none; prefix_table int32
    [prefixes, pages], prefix_lens int32 [prefixes]). What is shared is computed once for all requests of a prefix.
    workspace: w4a16_prefix_attention_workspace_bytes() of uint8, zeroed once before its first use and then kept for
    further calls; made here if it is not given."""
    if out is None:
        out = _new(q.shape, q.dtype, q, stream)
    q_row, q_head, o_row, o_head = _attention_tensors("w4a16_prefix_attention", q, cache, table, out, lse, lens)
    batch, heads, D = q.shape
    max_pages = table.shape[1]
    if table.shape[0] != batch or lens.numel() != batch:
        raise ValueError("w4a16_prefix_attention: table [batch, max_pages], lens [batch]")
    prefixes = _prefixes("w4a16_prefix_attention", batch, prefix_table, prefix_lens, prefix_of)
    if workspace is None:
        workspace = _new(w4a16_prefix_attention_workspace_bytes(batch, heads, cache.kv_heads, D), torch.uint8, q, stream,
                         torch.zeros)
    _placed("w4a16_prefix_attention", q, out, table, lens, lse, workspace, prefix_table, prefix_lens, prefix_of,
            *cache.tensors)
    status = _prefix(_pack_prefix(
        q.data_ptr(), _TYPES.get(q.dtype, -1), q_row, q_head, cache.address, table.data_ptr(),
        table.stride(0) if batch > 1 else max_pages, max_pages, lens.data_ptr(), batch, heads, *prefixes,
        D ** -0.5 if scale is None else scale, window, softcap, out.data_ptr(), o_row, o_head,
        0 if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_prefix_attention")
    return out


def w4a16_residual_rmsnorm(h, y, gamma=None, eps: float = 1e-5, post_gamma=None, gate=None, alpha: float = 1.0,
                           h_out=None, n_out=None, stream=None):
    """h + alpha * [gate *] [rmsnorm(y; post_gamma) | y], and its rmsnorm with gamma: returns
    (h_out, n_out), n_out None without gamma. h [M, K] is y's type or float32; gate is [K]
    or [M, K]; h_out may be h."""
    M, K = h.shape
    if h_out is None:
        h_out = _new((M, K), h.dtype, h, stream)
    if gamma is not None and n_out is None:
        n_out = _new((M, K), y.dtype, y, stream)
    shape = h.shape
    if (y.shape != shape or h_out.shape != shape or (n_out is not None and n_out.shape != shape)
            or (gate is not None and gate.shape != shape and gate.shape != (K,))):
        raise ValueError("w4a16_residual_rmsnorm: h, y, h_out, n_out [M, K], gate [K] or [M, K]")
    if K > 1 and (h.stride(1) != 1 or y.stride(1) != 1 or h_out.stride(1) != 1
                  or (n_out is not None and n_out.stride(1) != 1) or (gate is not None and gate.stride(-1) != 1)):
        raise ValueError("w4a16_residual_rmsnorm: rows must be contiguous")
    for t in (gamma, post_gamma):
        if t is not None:
            if t.dtype is not y.dtype:
                raise TypeError("gamma and post_gamma have y's type")
            if t.numel() != K or not t.is_contiguous():
                raise ValueError("gamma, post_gamma: [K], contiguous")
    if h_out.dtype is not h.dtype or (n_out is not None and n_out.dtype is not y.dtype) or (
            gate is not None and gate.dtype is not y.dtype):
        raise TypeError("w4a16_residual_rmsnorm: h_out has h's type, n_out and gate have y's")
    gate_row = 0 if gate is None or gate.dim() == 1 else gate.stride(0) if M > 1 else K
    status = _norm(_pack_norm(
        h.data_ptr(), _TYPES.get(h.dtype, -1), h.stride(0) if M > 1 else K, y.data_ptr(), _TYPES.get(y.dtype, -1),
        y.stride(0) if M > 1 else K, 0 if post_gamma is None else post_gamma.data_ptr(),
        0 if gate is None else gate.data_ptr(), gate_row, alpha, 0 if gamma is None else gamma.data_ptr(), eps,
        h_out.data_ptr(), h_out.stride(0) if M > 1 else K, 0 if n_out is None else n_out.data_ptr(),
        0 if n_out is None else n_out.stride(0) if M > 1 else K, M, K, _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_residual_rmsnorm")
    return h_out, n_out


def w4a16_sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, out=None, stream=None):
    """The next token of each row of logits [rows, vocab] (float16, bfloat16 or float32) for the random numbers uniform
    (float32 [rows], from 0 to 1): int64 [rows], -1 where every logit is minus infinity. temperature, top_p, min_p
    (float32 [rows]) and top_k (int32 [rows]) may be None; temperature 0, top_p <= 0 and min_p > 1 take the largest logit,
    top_k <= 0, top_p >= 1 and min_p <= 0 leave a row alone. See include/w4a16.h."""
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("w4a16_sample: logits [rows, vocab], rows contiguous")
    rows, vocab = logits.shape
    if out is None:
        out = _new((rows,), _int64, logits, stream)
    _expect(uniform, _float32, "uniform")
    _expect(out, _int64, "out")
    for t, kind, name in ((temperature, _float32, "temperature"), (top_k, _int32, "top_k"), (top_p, _float32, "top_p"),
                          (min_p, _float32, "min_p")):
        if t is not None:
            _expect(t, kind, name)
            if t.numel() != rows:
                raise ValueError(f"{name}: one entry for each row")
    if uniform.numel() != rows or out.numel() != rows:
        raise ValueError("w4a16_sample: uniform, out: one entry for each row")
    _placed("w4a16_sample", logits, uniform, temperature, top_k, top_p, min_p, out)
    status = _sample(_pack_sample(
        logits.data_ptr(), _TYPES.get(logits.dtype, -1), logits.stride(0) if rows > 1 else vocab, rows, vocab,
        uniform.data_ptr(), 0 if temperature is None else temperature.data_ptr(), 0 if top_k is None else top_k.data_ptr(),
        0 if top_p is None else top_p.data_ptr(), 0 if min_p is None else min_p.data_ptr(), out.data_ptr(), _stream(stream)))
    if status:
        raise W4A16Error(status, "w4a16_sample")
    return out


def w4a16_set_tuning(smallm_max: int) -> None:
    _check(lib.w4a16_set_tuning(smallm_max), "w4a16_set_tuning")


def w4a16_set_launch_overlap(enable: bool) -> None:
    """Let small-M GEMM calls start while the work before them finishes
    (weights must not be written by that work); see include/w4a16.h."""
    _check(lib.w4a16_set_launch_overlap(int(enable)), "w4a16_set_launch_overlap")


WAIT_LIMIT_DEFAULT_NS = 2_000_000_000


def w4a16_set_wait_limit_ns(limit_ns: int) -> None:
    """Limit of every bounded device-side wait (tests of the failure path)."""
    _check(lib.w4a16_set_wait_limit_ns(int(limit_ns)), "w4a16_set_wait_limit_ns")


def w4a16_device_error(stream=None) -> int:
    return int(lib.w4a16_device_error(_stream(stream)))
