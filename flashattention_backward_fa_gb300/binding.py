"""Thin ctypes binding over libfa.so (the C ABI declared in include/fa.h).

Argument marshalling only: shapes, strides and pointers of torch tensors are
passed to the C entry points, which validate them and launch the CUDA kernels
on the caller's current stream. torch supplies device memory and streams;
every step of the computation runs in the library's kernels. There is no
fallback: if the library is missing or the tensors are not on a CUDA device,
these functions raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from functools import lru_cache
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libfa.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "fa.h")

FA_F32, FA_F16, FA_BF16 = 0, 1, 2
FA_BWD_PREPROCESS, FA_BWD_DKDV, FA_BWD_DQ = 0, 1, 2
# dQ algorithms (the `deterministic` argument of the backward calls, fa.h FA_DQ_*)
FA_DQ_ATOMIC, FA_DQ_DETERMINISTIC, FA_DQ_RECOMPUTE, FA_DQ_ORDERED = 0, 1, 2, 3


def _dq_mode(deterministic) -> int:
    """A `deterministic` argument as the C ABI's dQ mode: True / False are
    FA_DQ_DETERMINISTIC / FA_DQ_ATOMIC; integers pass through (FA_DQ_*)."""
    if isinstance(deterministic, bool):
        return FA_DQ_DETERMINISTIC if deterministic else FA_DQ_ATOMIC
    mode = int(deterministic)
    if mode not in (FA_DQ_ATOMIC, FA_DQ_DETERMINISTIC, FA_DQ_RECOMPUTE, FA_DQ_ORDERED):
        raise ValueError(f"deterministic must be a bool or one of FA_DQ_* (0..3), not {deterministic!r}")
    return mode
ERROR_CODES = {
    0: "FA_OK", -1: "FA_ERR_INVALID_ARG", -2: "FA_ERR_UNSUPPORTED", -3: "FA_ERR_ALIGNMENT",
    -4: "FA_ERR_WORKSPACE", -5: "FA_ERR_CUDA", -6: "FA_ERR_TIMEOUT",
}
_TORCH_TO_FA = {torch.float32: FA_F32, torch.float16: FA_F16, torch.bfloat16: FA_BF16}


class FaStrides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("n", ctypes.c_int64), ("h", ctypes.c_int64)]


class _Kv8CacheArg(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("H", ctypes.c_int), ("d", ctypes.c_int), ("strides", FaStrides)]


class _Kv8SeqsArg(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("seq_lens", ctypes.c_void_p),
                ("new_lens", ctypes.c_void_p), ("B", ctypes.c_int), ("max_pages", ctypes.c_int)]


class FaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_CODES.get(code, code)}: {msg}")
        self.code = code


_lib = None


def load_library(path: str = LIB_PATH):
    """Load libfa.so and declare the C signatures; raises if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libfa.so not found at {path}: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i, f, u64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint64, ctypes.c_size_t
    lib.fa_version.argtypes, lib.fa_version.restype = [], i
    lib.fa_strerror.argtypes, lib.fa_strerror.restype = [i], ctypes.c_char_p
    lib.fa_bwd_workspace_size.argtypes = [i, i, i, i, i, i]
    lib.fa_bwd_workspace_size.restype = sz
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, vp]
    lib.fa_fwd.restype = i
    bwd_args = [vp] * 9 + [i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, i, vp, sz, vp]
    lib.fa_bwd.argtypes, lib.fa_bwd.restype = bwd_args, i
    lib.fa_bwd_stage.argtypes, lib.fa_bwd_stage.restype = [i] + bwd_args, i
    lib.fa_get_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i]
    lib.fa_get_device_status.restype = i
    lib.fa_selftest_timeout.argtypes, lib.fa_selftest_timeout.restype = [vp, vp], i
    lib.fa_bwd_noalloc.argtypes = [vp] * 9 + [i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, vp]
    lib.fa_bwd_noalloc.restype = i
    i64 = ctypes.c_int64
    lib.fa_varlen_bwd_workspace_size.argtypes = [i, i, i, i, i, i, i]
    lib.fa_varlen_bwd_workspace_size.restype = sz
    lib.fa_varlen_fwd.argtypes = [vp] * 6 + [i, i, i, i, i, i64, i64, i, f, i, i, vp, i64, vp]
    lib.fa_varlen_fwd.restype = i
    lib.fa_varlen_bwd.argtypes = [vp] * 10 + [i, i, i, i, i, i64, i64, i, f, i, i, vp, i64, i, vp, sz, vp]
    lib.fa_varlen_bwd.restype = i
    lib.fa_bwd_host_buffer_size.argtypes = [i, i, i, i, i, i]
    lib.fa_bwd_host_buffer_size.restype = sz
    lib.fa_bwd_host.argtypes = bwd_args
    lib.fa_bwd_host.restype = i
    lib.fa_fwd_bias.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, vp, FaStrides,
                                vp]
    lib.fa_fwd_bias.restype = i
    lib.fa_bwd_bias.argtypes = [vp] * 9 + [i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, vp, FaStrides, i, vp,
                                           sz, vp]
    lib.fa_bwd_bias.restype = i
    lib.fa_fwd_alibi.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, vp, i64, vp]
    lib.fa_fwd_alibi.restype = i
    lib.fa_bwd_alibi.argtypes = [vp] * 9 + [i, i, i, i, FaStrides, i, f, i, i, f, u64, u64, vp, i64, i, vp, sz,
                                            vp]
    lib.fa_bwd_alibi.restype = i
    st = FaStrides
    lib.fa_qk_norm_rope_fwd.argtypes = [vp] * 9 + [i64] + [i] * 8 + [st] * 4 + [i, i, f, vp]
    lib.fa_qk_norm_rope_fwd.restype = i
    lib.fa_qk_norm_rope_bwd_workspace_size.argtypes = [i]
    lib.fa_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.fa_qk_norm_rope_bwd.argtypes = [vp] * 13 + [i64] + [i] * 8 + [st] * 6 + [i, i, f, vp, sz, vp]
    lib.fa_qk_norm_rope_bwd.restype = i
    cache, seqs = ctypes.POINTER(_Kv8CacheArg), ctypes.POINTER(_Kv8SeqsArg)
    lib.fa_kv8_append.argtypes = [cache, seqs, vp, vp, i, st, st, i, vp]
    lib.fa_kv8_append.restype = i
    lib.fa_kv8_norm_rope_append.argtypes = [cache, seqs] + [vp] * 8 + [i] * 5 + [st] * 4 + [i, i, f, vp]
    lib.fa_kv8_norm_rope_append.restype = i
    lib.fa_kv8_attn_workspace_size.argtypes = [i] * 10
    lib.fa_kv8_attn_workspace_size.restype = sz
    lib.fa_kv8_attn.argtypes = [cache, seqs, vp, vp, vp, i, i, i, st, st, i, f, i, i, vp, i64, vp, sz, vp]
    lib.fa_kv8_attn.restype = i
    _lib = lib
    return lib


def header_functions(path: str = HEADER_PATH):
    """Names of the functions include/fa.h declares (used to check the exports)."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(fa_[a-z_0-9]+)\s*\(", text)))


def fa_strerror(code: int) -> str:
    return load_library().fa_strerror(int(code)).decode()


def _check(code: int):
    if code != 0:
        raise FaError(code, fa_strerror(code))


def _layout(t: torch.Tensor):
    if t.dim() != 4:
        raise ValueError("attention tensors are [B, N, H, d]")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if t.stride(3) != 1:
        raise ValueError("the head dimension must be contiguous")
    B, N, H, d = t.shape
    return (B, N, H, d), FaStrides(t.stride(0), t.stride(1), t.stride(2))


def _same_layout(ref: torch.Tensor, *others: torch.Tensor):
    shp, st = _layout(ref)
    for o in others:
        s2, st2 = _layout(o)
        if s2 != shp or (st2.b, st2.n, st2.h) != (st.b, st.n, st.h) or o.dtype != ref.dtype:
            raise ValueError("all [B, N, H, d] tensors must share shape, strides and dtype")
        if o.device != ref.device:
            raise ValueError("all tensors must live on the same CUDA device")
    if ref.device.index is not None and ref.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors live on {ref.device} but the current device is cuda:{torch.cuda.current_device()}"
                         " (use torch.cuda.device(...))")
    return shp, st


def _on_device(t: torch.Tensor, ref: torch.Tensor, name: str):
    if not t.is_cuda or t.device != ref.device:
        raise ValueError(f"{name} must be a CUDA tensor on {ref.device}")


def _stream(stream):
    if stream is None:
        # the handle alone: building a torch.cuda.Stream object costs about 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _alibi(slopes, lead: int, H: int, device):
    """(pointer, lead stride) of ALiBi slopes shaped [H] or [lead, H] (fp32 CUDA), or (None, 0)."""
    if slopes is None:
        return None, 0
    if slopes.dtype != torch.float32 or not slopes.is_cuda or slopes.device != device:
        raise ValueError("alibi_slopes must be a float32 tensor on the tensors' device")
    if slopes.dim() == 1 and slopes.shape[0] == H and slopes.stride(0) == 1:
        return slopes.data_ptr(), 0
    if slopes.dim() == 2 and tuple(slopes.shape) == (lead, H) and slopes.stride(1) == 1:
        return slopes.data_ptr(), slopes.stride(0)
    raise ValueError(f"alibi_slopes must be [H] or [{lead}, H] with a contiguous head dimension")


def _bias(bias, q):
    """(pointer, FaStrides(b, n, h)) of an attention bias shaped [B or 1, H or 1, N, N]."""
    B, N, H, _ = q.shape
    if bias.dtype != q.dtype or not bias.is_cuda or bias.device != q.device:
        raise ValueError("attn_bias must be a CUDA tensor of the tensors' dtype on their device")
    if bias.dim() != 4 or bias.shape[0] not in (1, B) or bias.shape[1] not in (1, H) or \
            tuple(bias.shape[2:]) != (N, N) or bias.stride(3) != 1:
        raise ValueError(f"attn_bias must be [B or 1, H or 1, {N}, {N}] with contiguous keys")
    sb = bias.stride(0) if bias.shape[0] > 1 else 0
    sh = bias.stride(1) if bias.shape[1] > 1 else 0
    return bias.data_ptr(), FaStrides(sb, bias.stride(2), sh)


@lru_cache(maxsize=None)
def default_scale(d: int) -> float:
    return float(torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32))


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int, dtype, deterministic: bool = True) -> int:
    code = _TORCH_TO_FA[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().fa_bwd_workspace_size(B, H, N, d, code, _dq_mode(deterministic)))


def fa_fwd(q, k, v, o, lse, scale=None, causal=False, window=0, dropout_p=0.0, seed=0, offset=0, stream=None,
           alibi_slopes=None, attn_bias=None):
    """Forward through the C ABI: fills o ([B,N,H,d]) and lse ([B,H,N] fp32).

    ``alibi_slopes`` (fp32 [H] or [B, H]) adds -m|i - j| to the scaled scores (fa_fwd_alibi).
    """
    (B, N, H, d), st = _same_layout(q, k, v, o)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    _on_device(lse, q, "lse")
    lib = load_library()
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d, st,
            _TORCH_TO_FA[q.dtype], default_scale(d) if scale is None else float(scale), int(causal), int(window),
            float(dropout_p), int(seed), int(offset))
    if alibi_slopes is not None and attn_bias is not None:
        raise ValueError("pass either alibi_slopes or attn_bias (fold ALiBi into the bias to combine them)")
    if attn_bias is not None:
        _check(lib.fa_fwd_bias(*args, *_bias(attn_bias, q), _stream(stream)))
    elif alibi_slopes is None:
        _check(lib.fa_fwd(*args, _stream(stream)))
    else:
        _check(lib.fa_fwd_alibi(*args, *_alibi(alibi_slopes, B, H, q.device), _stream(stream)))


def _bwd_args(q, k, v, o, do, lse, dq, dk, dv, scale, causal, window, dropout_p, seed, offset, deterministic,
              workspace, stream):
    (B, N, H, d), st = _same_layout(q, k, v, o, do, dq, dk, dv)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    _on_device(lse, q, "lse")
    _on_device(workspace, q, "workspace")
    return (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), B, H, N, d, st, _TORCH_TO_FA[q.dtype],
            default_scale(d) if scale is None else float(scale), int(causal), int(window), float(dropout_p),
            int(seed), int(offset), _dq_mode(deterministic), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(stream))


def fa_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, scale=None, causal=False, window=0, dropout_p=0.0,
           seed=0, offset=0, deterministic=True, stream=None, alibi_slopes=None, attn_bias=None):
    """Backward through the C ABI: fills dq, dk, dv. ``workspace`` is a uint8 CUDA tensor.

    ``alibi_slopes`` as for :func:`fa_fwd` (fa_bwd_alibi)."""
    a = _bwd_args(q, k, v, o, do, lse, dq, dk, dv, scale, causal, window, dropout_p, seed, offset, deterministic,
                  workspace, stream)
    if alibi_slopes is not None and attn_bias is not None:
        raise ValueError("pass either alibi_slopes or attn_bias (fold ALiBi into the bias to combine them)")
    if attn_bias is not None:
        _check(load_library().fa_bwd_bias(*a[:21], *_bias(attn_bias, q), *a[21:]))
    elif alibi_slopes is None:
        _check(load_library().fa_bwd(*a))
    else:
        # fa_bwd_alibi takes the slopes before `deterministic`
        _check(load_library().fa_bwd_alibi(*a[:21], *_alibi(alibi_slopes, q.shape[0], q.shape[2], q.device),
                                           *a[21:]))


def fa_bwd_stage(stage, q, k, v, o, do, lse, dq, dk, dv, workspace, scale=None, causal=False, window=0,
                 dropout_p=0.0, seed=0, offset=0, deterministic=True, stream=None):
    """One of the three backward steps (FA_BWD_PREPROCESS, FA_BWD_DKDV, FA_BWD_DQ)."""
    _check(load_library().fa_bwd_stage(int(stage), *_bwd_args(q, k, v, o, do, lse, dq, dk, dv, scale, causal,
                                                              window, dropout_p, seed, offset, deterministic,
                                                              workspace, stream)))


def fa_bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, scale=None, causal=False, window=0, dropout_p=0.0, seed=0,
                   offset=0, stream=None):
    """Deterministic backward with the library's fixed internal scratch instead of a workspace.

    For callers that cannot allocate device memory when they run the backward.
    Limit B*H*roundup(N,128) <= 1048576; calls sharing a device must not overlap.
    """
    (B, N, H, d), st = _same_layout(q, k, v, o, do, dq, dk, dv)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    _on_device(lse, q, "lse")
    _check(load_library().fa_bwd_noalloc(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), B, H, N, d, st, _TORCH_TO_FA[q.dtype],
        default_scale(d) if scale is None else float(scale), int(causal), int(window), float(dropout_p), int(seed),
        int(offset), _stream(stream)))


def _host_layout(ref: torch.Tensor, *others: torch.Tensor):
    if ref.dim() != 4 or ref.is_cuda or ref.stride(3) != 1:
        raise ValueError("host tensors are CPU [B, N, H, d] with a contiguous head dimension")
    for o in others:
        if o.is_cuda or tuple(o.shape) != tuple(ref.shape) or o.stride() != ref.stride() or o.dtype != ref.dtype:
            raise ValueError("all host [B, N, H, d] tensors must share shape, strides and dtype")
    B, N, H, d = ref.shape
    return (B, N, H, d), FaStrides(ref.stride(0), ref.stride(1), ref.stride(2))


def fa_bwd_host_buffer_size(B: int, H: int, N: int, d: int, dtype, deterministic: bool = True) -> int:
    code = _TORCH_TO_FA[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().fa_bwd_host_buffer_size(B, H, N, d, code, _dq_mode(deterministic)))


def fa_bwd_host(q, k, v, o, do, lse, dq, dk, dv, dev_buf, scale=None, causal=False, window=0, dropout_p=0.0,
                seed=0, offset=0, deterministic=True, stream=None):
    """Backward from host (CPU) tensors through fa_bwd_host: uploads, computes and downloads
    on ``stream`` with the copies overlapped; pin the host tensors for that overlap.
    ``dev_buf`` is a uint8 CUDA tensor of fa_bwd_host_buffer_size(...) bytes. The outputs
    are ready once the stream has completed the work."""
    (B, N, H, d), st = _host_layout(q, k, v, o, do, dq, dk, dv)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous() or lse.is_cuda:
        raise ValueError("lse must be a contiguous float32 CPU [B, H, N] tensor")
    if not dev_buf.is_cuda or dev_buf.device.index not in (None, torch.cuda.current_device()):
        raise ValueError("dev_buf must be device memory of the current device")
    _check(load_library().fa_bwd_host(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), B, H, N, d, st, _TORCH_TO_FA[q.dtype],
        default_scale(d) if scale is None else float(scale), int(causal), int(window), float(dropout_p), int(seed),
        int(offset), _dq_mode(deterministic), dev_buf.data_ptr(), dev_buf.numel() * dev_buf.element_size(),
        _stream(stream)))


def fa_get_device_status(clear: bool = True) -> int:
    """Raw device status bits of the current device (synchronises it)."""
    s = ctypes.c_uint(0)
    code = load_library().fa_get_device_status(ctypes.byref(s), int(clear))
    if code not in (0, -6):
        _check(code)
    return int(s.value)


def fa_selftest_timeout(device=None, stream=None) -> int:
    """Run the bounded-wait self-test kernel (about 8 s) and return its outcome bits.

    Bit w is set when warp w's wait gave up (3 = both). The device status word
    then carries the timeout bit: read and clear it with fa_get_device_status().
    """
    outcome = torch.zeros(1, dtype=torch.int32, device=device if device is not None else "cuda")
    _check(load_library().fa_selftest_timeout(outcome.data_ptr(), _stream(stream)))
    return int(outcome.item())


def alloc_workspace(q: torch.Tensor, deterministic: bool = True) -> torch.Tensor:
    B, N, H, d = q.shape
    nbytes = fa_bwd_workspace_size(B, H, N, d, q.dtype, deterministic)
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device)


def attention_forward(q, k, v, scale=None, causal=False, window=0, dropout_p=0.0, seed=0, offset=0,
                      alibi_slopes=None, attn_bias=None):
    """Allocate O and L and run the forward; returns (o, lse)."""
    B, N, H, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fa_fwd(q, k, v, o, lse, scale, causal, window, dropout_p, seed, offset, alibi_slopes=alibi_slopes,
           attn_bias=attn_bias)
    return o, lse


def attention_backward(q, k, v, o, do, lse, scale=None, causal=False, window=0, dropout_p=0.0, seed=0, offset=0,
                       deterministic=True, workspace=None, alibi_slopes=None, attn_bias=None):
    """Allocate dQ, dK, dV (and the workspace unless given) and run the backward."""
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = alloc_workspace(q, deterministic)
    fa_bwd(q, k, v, o, do, lse, dq, dk, dv, workspace, scale, causal, window, dropout_p, seed, offset,
           deterministic, alibi_slopes=alibi_slopes, attn_bias=attn_bias)
    return dq, dk, dv


# ----------------------- packed variable-length input -----------------------
def _varlen_layout(ref: torch.Tensor, cu_seqlens: torch.Tensor, *others: torch.Tensor):
    """Checks packed [total, H, d] tensors and the int32 cu_seqlens; returns (total, H, d, sn, sh, nseq)."""
    if ref.dim() != 3 or not ref.is_cuda or ref.stride(2) != 1:
        raise ValueError("packed tensors are CUDA [total, H, d] with a contiguous head dimension")
    for o in others:
        if tuple(o.shape) != tuple(ref.shape) or o.stride() != ref.stride() or o.dtype != ref.dtype:
            raise ValueError("all packed tensors must share shape, strides and dtype")
        _on_device(o, ref, "every packed tensor")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_cuda \
            or not cu_seqlens.is_contiguous() or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor of nseq + 1 offsets")
    _on_device(cu_seqlens, ref, "cu_seqlens")
    total, H, d = ref.shape
    return total, H, d, ref.stride(0), ref.stride(1), cu_seqlens.numel() - 1


def _varlen_lse_check(lse, H, total):
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, total) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [H, total] tensor")


def fa_varlen_bwd_workspace_size(nseq: int, max_seqlen: int, total: int, H: int, d: int, dtype,
                                 deterministic: bool = True) -> int:
    code = _TORCH_TO_FA[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().fa_varlen_bwd_workspace_size(nseq, max_seqlen, total, H, d, code,
                                                           _dq_mode(deterministic)))


def fa_varlen_fwd(q, k, v, o, lse, cu_seqlens, max_seqlen, scale=None, causal=False, window=0, stream=None,
                  alibi_slopes=None):
    """Forward over packed sequences: fills o ([total, H, d]) and lse ([H, total] fp32).

    ``alibi_slopes``: fp32 [H] or [nseq, H], or None."""
    total, H, d, sn, sh, nseq = _varlen_layout(q, cu_seqlens, k, v, o)
    _varlen_lse_check(lse, H, total)
    _check(load_library().fa_varlen_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), cu_seqlens.data_ptr(), nseq,
        int(max_seqlen), total, H, d, sn, sh, _TORCH_TO_FA[q.dtype], default_scale(d) if scale is None else
        float(scale), int(causal), int(window), *_alibi(alibi_slopes, nseq, H, q.device), _stream(stream)))


def fa_varlen_bwd(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, max_seqlen, workspace, scale=None, causal=False,
                  window=0, deterministic=True, stream=None, alibi_slopes=None):
    """Backward over packed sequences: fills dq, dk, dv. ``workspace`` is a uint8 CUDA tensor."""
    total, H, d, sn, sh, nseq = _varlen_layout(q, cu_seqlens, k, v, o, do, dq, dk, dv)
    _varlen_lse_check(lse, H, total)
    _check(load_library().fa_varlen_bwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), cu_seqlens.data_ptr(), nseq, int(max_seqlen), total, H, d, sn, sh,
        _TORCH_TO_FA[q.dtype], default_scale(d) if scale is None else float(scale), int(causal), int(window),
        *_alibi(alibi_slopes, nseq, H, q.device), _dq_mode(deterministic), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def varlen_attention_forward(q, k, v, cu_seqlens, max_seqlen, scale=None, causal=False, window=0,
                             alibi_slopes=None):
    """Allocate O and L and run the packed forward; returns (o, lse)."""
    total, H, _ = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((H, total), dtype=torch.float32, device=q.device)
    fa_varlen_fwd(q, k, v, o, lse, cu_seqlens, max_seqlen, scale, causal, window, alibi_slopes=alibi_slopes)
    return o, lse


def varlen_attention_backward(q, k, v, o, do, lse, cu_seqlens, max_seqlen, scale=None, causal=False, window=0,
                              deterministic=True, alibi_slopes=None):
    """Allocate dQ, dK, dV and the workspace and run the packed backward."""
    total, H, d = q.shape
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = fa_varlen_bwd_workspace_size(cu_seqlens.numel() - 1, max_seqlen, total, H, d, q.dtype, deterministic)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    fa_varlen_bwd(q, k, v, o, do, lse, dq, dk, dv, cu_seqlens, max_seqlen, ws, scale, causal, window,
                  deterministic, alibi_slopes=alibi_slopes)
    return dq, dk, dv


class _FlashAttnFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, scale, causal, window, dropout_p, seed, offset, deterministic, alibi_slopes, attn_bias):
        o, lse = attention_forward(q, k, v, scale, causal, window, dropout_p, seed, offset, alibi_slopes, attn_bias)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.cfg = (scale, causal, window, dropout_p, seed, offset, deterministic, alibi_slopes, attn_bias)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        scale, causal, window, dropout_p, seed, offset, deterministic, alibi_slopes, attn_bias = ctx.cfg
        if do.stride() != q.stride():
            do = _match_layout(do, q)
        dq, dk, dv = attention_backward(q, k, v, o, do, lse, scale, causal, window, dropout_p, seed, offset,
                                        deterministic, alibi_slopes=alibi_slopes, attn_bias=attn_bias)
        return dq, dk, dv, None, None, None, None, None, None, None, None, None


def _match_layout(t: torch.Tensor, ref: torch.Tensor) -> torch.Tensor:
    out = torch.empty_strided(ref.shape, ref.stride(), dtype=ref.dtype, device=ref.device)
    out.copy_(t)
    return out


def flash_attn_func(q, k, v, causal=False, window=0, dropout_p=0.0, softmax_scale=None, seed=0, offset=0,
                    deterministic=True, alibi_slopes=None, attn_bias=None):
    """Attention on [B, S, H, D] tensors with autograd (forward fa_fwd, backward fa_bwd).

    ``alibi_slopes`` (fp32 [H] or [B, H]) adds -m|i - j| to the scaled scores; ``attn_bias``
    ([B or 1, H or 1, S, S], the tensors' dtype, -inf masks) adds itself. Neither is differentiated."""
    k = k if k.stride() == q.stride() else _match_layout(k, q)
    v = v if v.stride() == q.stride() else _match_layout(v, q)
    return _FlashAttnFunc.apply(q, k, v, softmax_scale, causal, window, dropout_p, seed, offset, deterministic,
                                alibi_slopes, attn_bias)


class _FlashAttnVarlenFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, max_seqlen, scale, causal, window, deterministic, alibi_slopes):
        o, lse = varlen_attention_forward(q, k, v, cu_seqlens, max_seqlen, scale, causal, window, alibi_slopes)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.cfg = (max_seqlen, scale, causal, window, deterministic, alibi_slopes)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, cu_seqlens = ctx.saved_tensors
        max_seqlen, scale, causal, window, deterministic, alibi_slopes = ctx.cfg
        if do.stride() != q.stride():
            do = _match_layout(do, q)
        dq, dk, dv = varlen_attention_backward(q, k, v, o, do, lse, cu_seqlens, max_seqlen, scale, causal, window,
                                               deterministic, alibi_slopes)
        return dq, dk, dv, None, None, None, None, None, None, None


def flash_attn_varlen_func(q, k, v, cu_seqlens, max_seqlen, causal=False, window=0, softmax_scale=None,
                           deterministic=True, alibi_slopes=None):
    """Attention over packed sequences ([total, H, D] tensors, int32 cu_seqlens on the
    device) with autograd (forward fa_varlen_fwd, backward fa_varlen_bwd)."""
    k = k if k.stride() == q.stride() else _match_layout(k, q)
    v = v if v.stride() == q.stride() else _match_layout(v, q)
    return _FlashAttnVarlenFunc.apply(q, k, v, cu_seqlens, int(max_seqlen), softmax_scale, causal, window,
                                      deterministic, alibi_slopes)


# ---------------- norm of queries and keys, and their rotation ----------------
# A serving loop makes these calls once a layer and token, where the GPU's work is a few
# microseconds: the checks below fetch every tensor property once, and the structs of
# strides that recur from call to call are built once.
@lru_cache(maxsize=1024)
def _strides(b: int, n: int, h: int) -> FaStrides:
    return FaStrides(b, n, h)


def _rows_layout(t: torch.Tensor, shape, dtype, dev: int, name: str) -> FaStrides:
    """Strides of a [B, N, H, d] CUDA tensor of that shape, dtype and device index."""
    s = t.stride()
    if t.shape != shape or s[3] != 1:
        raise ValueError(f"{name} must be {list(shape)} with a contiguous head dimension")
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {dtype} on cuda:{dev}, as the call's other tensors")
    return _strides(s[0], s[1], s[2])


def _new_tensor(t: torch.Tensor, name: str):
    """(shape, dtype, device index) of a [B, N, H, d] tensor on the current device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must live on a CUDA device")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} lives on cuda:{dev} but the current device is "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device(...))")
    if t.dim() != 4:
        raise ValueError(f"{name} must be four-dimensional: [B, N, H, d]")
    dtype = t.dtype
    if dtype not in _TORCH_TO_FA:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, not {dtype}")
    return t.shape, dtype, dev


def _int32(t, shape, dev: int, name: str):
    """Pointer of an int32 tensor of that shape with contiguous rows (None passes through)."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.get_device() != dev or t.shape != shape or \
            (shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be an int32 tensor {list(shape)} with contiguous rows on cuda:{dev}")
    return t.data_ptr()


def _weight(w, d: int, dtype, dev: int, name: str):
    if w is None:
        return None
    if w.shape != (d,) or (d > 1 and w.stride(0) != 1) or w.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous [{d}] tensor on cuda:{dev}")
    if w.dtype is not dtype and w.dtype is not torch.float32:
        raise ValueError(f"{name} must be float32 or of the tensors' dtype")
    return w.data_ptr()


def _rope_args(d: int, dtype, dev: int, q_weight, k_weight, cos, sin):
    """Weights and tables of the norm-and-rotation calls: (rot_dim, max_pos, weight dtype code, four pointers)."""
    qw, kw = _weight(q_weight, d, dtype, dev, "q_weight"), _weight(k_weight, d, dtype, dev, "k_weight")
    wt = dtype if qw is kw is None else (k_weight if qw is None else q_weight).dtype
    if qw is not None and kw is not None and k_weight.dtype is not wt:
        raise ValueError("q_weight and k_weight must have the same dtype")
    if cos is None or sin is None:
        if cos is not sin:
            raise ValueError("pass both tables or neither")
        return 0, 0, _TORCH_TO_FA[wt], (qw, kw, None, None)
    shape = cos.shape
    for name, t in (("cos", cos), ("sin", sin)):
        if len(shape) != 2 or t.shape != shape or t.dtype is not torch.float32 or t.get_device() != dev or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 [max_pos, rot_dim / 2] tensor on cuda:{dev}")
    rows, half = shape
    if 2 * half > d:
        raise ValueError(f"the tables rotate {2 * half} values of heads of {d}")
    return 2 * half, rows, _TORCH_TO_FA[wt], (qw, kw, cos.data_ptr(), sin.data_ptr())


def _positions(positions, B: int, N: int, dev: int):
    """(pointer, stride) of int32 positions [N] or [B, N], or (None, 0)."""
    if positions is None:
        return None, 0
    if positions.dim() == 1:
        return _int32(positions, (N,), dev, "positions"), 0
    return _int32(positions, (B, N), dev, "positions"), positions.stride(0)


def rope_tables(max_pos: int, rot_dim: int, base: float = 10000.0, device="cuda"):
    """cos and sin tables [max_pos, rot_dim / 2] (fp32) of the angles pos * base^(-2i / rot_dim),
    computed in float64 (in fp32 the angles of far positions lose their fraction)."""
    if max_pos < 1 or rot_dim < 2 or rot_dim % 2:
        raise ValueError("max_pos must be positive and rot_dim positive and even")
    freq = base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float(), angle.sin().float()


def _norm_rope_fwd(q, k, q_out, k_out, q_weight, k_weight, cos, sin, positions, eps, interleaved, stream):
    shape, dtype, dev = _new_tensor(q, "q")
    B, N, Hq, d = shape
    kshape = k.shape
    if len(kshape) != 4 or kshape[0] != B or kshape[1] != N or kshape[3] != d:
        raise ValueError(f"k must be [{B}, {N}, Hk, {d}] as q is {list(shape)}")
    Hk = kshape[2]
    rot, rows, wt, ptrs = _rope_args(d, dtype, dev, q_weight, k_weight, cos, sin)
    eps, interleaved = float(eps), bool(interleaved)
    q_st, k_st = _rows_layout(q, shape, dtype, dev, "q"), _rows_layout(k, kshape, dtype, dev, "k")
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        qo_st, ko_st = _strides(N * Hq * d, Hq * d, d), _strides(N * Hk * d, Hk * d, d)
    else:
        qo_st = _rows_layout(q_out, shape, dtype, dev, "q_out")
        ko_st = _rows_layout(k_out, kshape, dtype, dev, "k_out")
    _check((_lib or load_library()).fa_qk_norm_rope_fwd(
        q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), *ptrs, *_positions(positions, B, N, dev), B,
        N, Hq, Hk, d, rot, interleaved, rows, q_st, k_st, qo_st, ko_st, _TORCH_TO_FA[dtype], wt, eps,
        _stream(stream)))
    return q_out, k_out


def fa_qk_norm_rope_fwd(q, k, q_out, k_out, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                        eps=1e-6, interleaved=False, stream=None):
    """Per-head RMS norm and rotation through the C ABI: fills q_out and k_out (shaped as q and k)."""
    _norm_rope_fwd(q, k, q_out, k_out, q_weight, k_weight, cos, sin, positions, eps, interleaved, stream)


def qk_norm_rope_forward(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                         interleaved=False):
    """Allocate the outputs and run the norm and rotation; returns (q_out, k_out), contiguous.

    q [B, N, Hq, d], k [B, N, Hk, d]; weights [d] (None: ones); tables as from rope_tables (None: no
    rotation); positions int32 [N] or [B, N] (None: 0 .. N - 1)."""
    return _norm_rope_fwd(q, k, None, None, q_weight, k_weight, cos, sin, positions, eps, interleaved, None)


@lru_cache(maxsize=None)
def fa_qk_norm_rope_bwd_workspace_size(d: int) -> int:
    return int(load_library().fa_qk_norm_rope_bwd_workspace_size(int(d)))


def _weight_grad(g, w, dev: int, name: str):
    if g is None or w is None:
        if g is not w:
            raise ValueError(f"{name} must be None exactly where its weight is")
        return None
    if g.dtype is not w.dtype or g.shape != w.shape or g.get_device() != dev or not g.is_contiguous():
        raise ValueError(f"{name} must match its weight")
    return g.data_ptr()


def _norm_rope_bwd(q, k, dq_out, dk_out, outs, q_weight, k_weight, cos, sin, positions, eps, interleaved, stream):
    """``outs``: (dq, dk, dq_weight, dk_weight, workspace) of the caller, or None to allocate them."""
    shape, dtype, dev = _new_tensor(q, "q")
    B, N, Hq, d = shape
    kshape = k.shape
    if len(kshape) != 4 or kshape[0] != B or kshape[1] != N or kshape[3] != d:
        raise ValueError(f"k must be [{B}, {N}, Hk, {d}] as q is {list(shape)}")
    Hk = kshape[2]
    rot, rows, wt, (qw, kw, cp, sp) = _rope_args(d, dtype, dev, q_weight, k_weight, cos, sin)
    q_st, k_st = _rows_layout(q, shape, dtype, dev, "q"), _rows_layout(k, kshape, dtype, dev, "k")
    gq_st = _rows_layout(dq_out, shape, dtype, dev, "dq_out")
    gk_st = _rows_layout(dk_out, kshape, dtype, dev, "dk_out")
    if outs is None:
        dq = torch.empty_like(q, memory_format=torch.contiguous_format)
        dk = torch.empty_like(k, memory_format=torch.contiguous_format)
        dqw = None if q_weight is None else torch.empty_like(q_weight)
        dkw = None if k_weight is None else torch.empty_like(k_weight)
        size = fa_qk_norm_rope_bwd_workspace_size(d)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        dq_st, dk_st = _strides(N * Hq * d, Hq * d, d), _strides(N * Hk * d, Hk * d, d)
        dqw_ptr, dkw_ptr = (None if dqw is None else dqw.data_ptr()), (None if dkw is None else dkw.data_ptr())
    else:
        dq, dk, dqw, dkw, workspace = outs
        dq_st, dk_st = _rows_layout(dq, shape, dtype, dev, "dq"), _rows_layout(dk, kshape, dtype, dev, "dk")
        dqw_ptr = _weight_grad(dqw, q_weight, dev, "dq_weight")
        dkw_ptr = _weight_grad(dkw, k_weight, dev, "dk_weight")
        if workspace.get_device() != dev:
            raise ValueError(f"workspace must be a CUDA tensor on cuda:{dev}")
        size = workspace.numel() * workspace.element_size()
    _check((_lib or load_library()).fa_qk_norm_rope_bwd(
        q.data_ptr(), k.data_ptr(), dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), qw, kw, dqw_ptr,
        dkw_ptr, cp, sp, *_positions(positions, B, N, dev), B, N, Hq, Hk, d, rot, bool(interleaved), rows, q_st, k_st,
        gq_st, gk_st, dq_st, dk_st, _TORCH_TO_FA[dtype], wt, float(eps), workspace.data_ptr(), size, _stream(stream)))
    return dq, dk, dqw, dkw


def fa_qk_norm_rope_bwd(q, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, q_weight=None, k_weight=None,
                        cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, stream=None):
    """Its backward through the C ABI: fills dq, dk and, where there are weights, dq_weight and dk_weight.
    ``workspace`` is a uint8 CUDA tensor of fa_qk_norm_rope_bwd_workspace_size(d) bytes."""
    _norm_rope_bwd(q, k, dq_out, dk_out, (dq, dk, dq_weight, dk_weight, workspace), q_weight, k_weight, cos, sin,
                   positions, eps, interleaved, stream)


def qk_norm_rope_backward(q, k, dq_out, dk_out, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                          eps=1e-6, interleaved=False):
    """Allocate the gradients and the workspace and run the backward; returns
    (dq, dk, dq_weight, dk_weight), contiguous, None for a weight that is None."""
    return _norm_rope_bwd(q, k, dq_out, dk_out, None, q_weight, k_weight, cos, sin, positions, eps, interleaved, None)


class _QkNormRopeFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.cfg = (eps, interleaved)
        return qk_norm_rope_forward(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        grads = qk_norm_rope_backward(q, k, _readable(dq_out), _readable(dk_out), q_weight, k_weight, cos, sin,
                                      positions, *ctx.cfg)
        return (*grads, None, None, None, None, None)


def _readable(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels read it: a copy where its strides (an expanded one's zeros,
    unaligned rows) or its base do not allow reading it in place."""
    s = t.stride()
    if len(s) != 4:
        return t  # refused by the call's own checks
    unit = 8 if t.element_size() == 2 else 1
    if s[3] != 1 or min(s) < 1 or any(x % unit for x in s[:3]) or t.data_ptr() % 16:
        return t.clone(memory_format=torch.contiguous_format)
    return t


def qk_norm_rope_func(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps=1e-6,
                      interleaved=False):
    """Per-head RMS norm and rotation of q [B, N, Hq, d] and k [B, N, Hk, d] with autograd
    (forward fa_qk_norm_rope_fwd, backward fa_qk_norm_rope_bwd): (q_out, k_out), as
    flash_attn_func takes them. Gradients reach q, k and the weights."""
    return _QkNormRopeFunc.apply(_readable(q), _readable(k), q_weight, k_weight, cos, sin, positions, float(eps),
                                 bool(interleaved))


# ---------------------------- 8-bit key/value cache ----------------------------
class Kv8Cache(NamedTuple):
    """A paged cache: k and v float8_e4m3fn [num_pages, page_size, H, d], k_scale and v_scale
    float32 [num_pages, H]; the values held are ``k.float() * k_scale[:, None, :, None]``."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv8_cache_alloc(num_pages: int, page_size: int, H: int, d: int, device="cuda") -> Kv8Cache:
    """An empty cache; each head's part of a page is contiguous, which reads fastest."""
    k, v = (torch.zeros((num_pages, H, page_size, d), dtype=torch.uint8, device=device)
            .view(torch.float8_e4m3fn).transpose(1, 2) for _ in range(2))
    k_scale, v_scale = (torch.ones((num_pages, H), dtype=torch.float32, device=device) for _ in range(2))
    return Kv8Cache(k, v, k_scale, v_scale)


def _kv8_args(cache: Kv8Cache, B: int, d: int, dtype, dev: int, block_table, seq_lens, new_lens):
    """The two C structs of a cache and its sequences, for new tokens [B, T, *, d]."""
    if dtype is torch.float32:
        raise ValueError("the 8-bit cache takes float16 or bfloat16 tensors")
    k, v, ks, vs = cache
    shape, st = k.shape, k.stride()
    if len(shape) != 4 or k.dtype is not torch.float8_e4m3fn or v.dtype is not torch.float8_e4m3fn or \
            v.shape != shape or v.stride() != st or st[3] != 1:
        raise ValueError("cache.k and cache.v must be float8_e4m3fn [num_pages, page_size, H, d] of the same "
                         "strides with a contiguous head dimension")
    P, page, H, dc = shape
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"the cache must live on cuda:{dev}")
    for s in (ks, vs):
        if s.dtype is not torch.float32 or s.shape != (P, H) or not s.is_contiguous() or s.get_device() != dev:
            raise ValueError(f"the cache's scales must be contiguous float32 [{P}, {H}] tensors on cuda:{dev}")
    if dc != d:
        raise ValueError(f"the cache holds heads of {dc}, the new tokens' tensors of {d}")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    pages = block_table.shape[1]
    return (_Kv8CacheArg(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), P, page, H, d,
                         _strides(st[0], st[1], st[2])),
            _Kv8SeqsArg(_int32(block_table, (B, pages), dev, "block_table"), block_table.stride(0),
                        _int32(seq_lens, (B,), dev, "seq_lens"), _int32(new_lens, (B,), dev, "new_lens"), B, pages))


def kv8_append(cache: Kv8Cache, k, v, block_table, seq_lens, new_lens=None, stream=None):
    """Write new keys and values [B, T, H, d] into the cache (fa_kv8_append). Not differentiable.

    ``seq_lens`` (int32 [B]) counts the new tokens already; they are the last ``new_lens``
    (int32 [B], None: T) of each sequence, further rows of k and v are padding. Token j of
    sequence b lies in page ``block_table[b, j // page_size]`` (int32 [B, max_pages])."""
    shape, dtype, dev = _new_tensor(k, "k")
    B, T, _, d = shape
    c, s = _kv8_args(cache, B, d, dtype, dev, block_table, seq_lens, new_lens)
    shape = (B, T, c.H, d)
    _check((_lib or load_library()).fa_kv8_append(
        c, s, k.data_ptr(), v.data_ptr(), T, _rows_layout(k, shape, dtype, dev, "k"),
        _rows_layout(v, shape, dtype, dev, "v"), _TORCH_TO_FA[dtype], _stream(stream)))


def _norm_rope_append(cache, q, k, v, q_out, q_weight, k_weight, cos, sin, block_table, seq_lens, new_lens, eps,
                      interleaved, stream):
    shape, dtype, dev = _new_tensor(q, "q")
    B, T, Hq, d = shape
    c, s = _kv8_args(cache, B, d, dtype, dev, block_table, seq_lens, new_lens)
    rot, rows, wt, ptrs = _rope_args(d, dtype, dev, q_weight, k_weight, cos, sin)
    eps, interleaved = float(eps), bool(interleaved)
    kshape = (B, T, c.H, d)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        qo_st = _strides(T * Hq * d, Hq * d, d)
    else:
        qo_st = _rows_layout(q_out, shape, dtype, dev, "q_out")
    _check((_lib or load_library()).fa_kv8_norm_rope_append(
        c, s, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), *ptrs, T, Hq, rot, interleaved, rows,
        _rows_layout(q, shape, dtype, dev, "q"), _rows_layout(k, kshape, dtype, dev, "k"),
        _rows_layout(v, kshape, dtype, dev, "v"), qo_st, _TORCH_TO_FA[dtype], wt, eps, _stream(stream)))
    return q_out


def fa_kv8_norm_rope_append(cache: Kv8Cache, q, k, v, q_out, q_weight, k_weight, cos, sin, block_table, seq_lens,
                            new_lens=None, eps=1e-6, interleaved=False, stream=None):
    """Norm and rotation of new q and k, then k and v into the cache, through the C ABI: fills q_out."""
    _norm_rope_append(cache, q, k, v, q_out, q_weight, k_weight, cos, sin, block_table, seq_lens, new_lens, eps,
                      interleaved, stream)


def kv8_norm_rope_append(cache: Kv8Cache, q, k, v, q_weight, k_weight, cos, sin, block_table, seq_lens, new_lens=None,
                         eps=1e-6, interleaved=False):
    """qk_norm_rope_forward of new q and k at their positions and kv8_append of the result in one
    launch; returns the normed and rotated q (zeros in padding rows)."""
    return _norm_rope_append(cache, q, k, v, None, q_weight, k_weight, cos, sin, block_table, seq_lens, new_lens, eps,
                             interleaved, None)


@lru_cache(maxsize=1024)
def fa_kv8_attn_workspace_size(B: int, T: int, Hq: int, H: int, d: int, page_size: int, max_pages: int,
                               max_seqlen: int, causal: bool = True, window: int = 0) -> int:
    return load_library().fa_kv8_attn_workspace_size(B, T, Hq, H, d, page_size, max_pages, int(max_seqlen),
                                                     int(causal), int(window))


def _kv8_attn(q, cache, o, lse, block_table, seq_lens, max_seqlen, workspace, new_lens, scale, causal, window,
              alibi_slopes, stream):
    shape, dtype, dev = _new_tensor(q, "q")
    B, T, Hq, d = shape
    c, s = _kv8_args(cache, B, d, dtype, dev, block_table, seq_lens, new_lens)
    lib = _lib or load_library()
    max_seqlen, causal, window = int(max_seqlen), bool(causal), int(window)
    q_st = _rows_layout(q, shape, dtype, dev, "q")
    if o is None:
        size = fa_kv8_attn_workspace_size(B, T, Hq, c.H, d, c.page_size, s.max_pages, max_seqlen, causal, window)
        device = q.device
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((B, Hq, T), dtype=torch.float32, device=device)
        workspace = torch.empty(size, dtype=torch.uint8, device=device) if size else None
        o_st = _strides(T * Hq * d, Hq * d, d)
    else:
        o_st = _rows_layout(o, shape, dtype, dev, "o")
        if lse.dtype is not torch.float32 or lse.shape != (B, Hq, T) or not lse.is_contiguous() or \
                lse.get_device() != dev:
            raise ValueError(f"lse must be a contiguous float32 [B, Hq, T] tensor on cuda:{dev}")
        size = 0
        if workspace is not None:
            if workspace.get_device() != dev:
                raise ValueError(f"workspace must be a CUDA tensor on cuda:{dev}")
            size = workspace.numel() * workspace.element_size()
    slopes, per_seq = (None, 0) if alibi_slopes is None else _alibi(alibi_slopes, B, Hq, q.device)
    _check(lib.fa_kv8_attn(
        c, s, q.data_ptr(), o.data_ptr(), lse.data_ptr(), T, Hq, max_seqlen, q_st, o_st, _TORCH_TO_FA[dtype],
        default_scale(d) if scale is None else float(scale), causal, window, slopes, per_seq,
        None if workspace is None else workspace.data_ptr(), size, _stream(stream)))
    return o, lse


def fa_kv8_attn(q, cache: Kv8Cache, o, lse, block_table, seq_lens, max_seqlen, workspace, new_lens=None, scale=None,
                causal=True, window=0, alibi_slopes=None, stream=None):
    """Attention over the cache through the C ABI: fills o ([B, T, Hq, d]) and lse ([B, Hq, T] fp32).
    ``workspace`` is a uint8 CUDA tensor of fa_kv8_attn_workspace_size(...) bytes (None where that is 0)."""
    _kv8_attn(q, cache, o, lse, block_table, seq_lens, max_seqlen, workspace, new_lens, scale, causal, window,
              alibi_slopes, stream)


def kv8_attention(q, cache: Kv8Cache, block_table, seq_lens, max_seqlen, new_lens=None, scale=None, causal=True,
                  window=0, alibi_slopes=None):
    """Attention of the newest tokens' queries [B, T, Hq, d] over the cache; returns (o, lse).

    The queries belong to the last ``new_lens`` tokens of each sequence (as for kv8_append, which
    comes first: a token attends to itself through the cache). Hq must be a multiple of the
    cache's heads. ``max_seqlen`` is an upper bound of ``seq_lens``. Not differentiable."""
    return _kv8_attn(q, cache, None, None, block_table, seq_lens, max_seqlen, None, new_lens, scale, causal, window,
                     alibi_slopes, None)
