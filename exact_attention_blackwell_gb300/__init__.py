"""Fused exact attention for NVIDIA GB300 (sm_103a): Python binding.

The compute lives in ``libfa_gb300.so`` (hand-written CUDA, C ABI declared in
``include/fa.h``).  This module only marshals arguments: every function with a
C name calls the C entry point of the same name and returns its status code;
the ``attention_*`` helpers allocate outputs with torch and raise
:class:`FaError` on a non-zero status.  There is no fallback: if the library is
missing the first call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa_gb300.so")

FA_OK = 0
FA_ERR_INVALID_ARG = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_ALIGNMENT = -3
FA_ERR_WORKSPACE = -4
FA_ERR_CUDA = -5
FA_ERR_TIMEOUT = -6

# name -> (restype, argtypes) for every symbol include/fa.h declares
_P, _I, _F, _LL, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong, ctypes.c_size_t
SIGNATURES = {
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_fwd_fp8_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_fwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_bwd_varlen": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_bwd_fused_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_bwd_fused": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_bwd_prepare": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "fa_bwd_dkdv": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_bwd_dq": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_bwd_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd_noalloc_scratch_bytes": (_SZ, []),
    "fa_cache_append": (_I, [_P] * 7 + [_I] * 7 + [_P]),
    "fa_fwd_paged_workspace_bytes": (_SZ, [_I] * 5),
    "fa_fwd_paged": (_I, [_P] * 7 + [_I, _P, _P] + [_I] * 9 + [_F, _P, _SZ, _P]),
    "fa_cache_compact": (_I, [_P] * 7 + [_I] * 8 + [_P]),
    "fa_cache_fork": (_I, [_P] * 5 + [_I] * 4 + [_P]),
    "fa_cache_resize_workspace_bytes": (_SZ, [_I]),
    "fa_cache_resize": (_I, [_P] * 8 + [_I] * 7 + [_P, _SZ, _P]),
    "fa_exp2_poly": (_I, [_P, _P, _LL, _P]),
    "fa_last_device_status": (_I, [_P]),
    "fa_last_device_status_site": (_I, [_P, _P]),
    "fa_debug_stall": (_I, [_I]),
    "fa_rescale_count": (_I, [_P, _P]),
    "fa_status_string": (ctypes.c_char_p, [_I]),
}

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Loads the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with exact_attention_blackwell_gb300.build.build()")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def status_string(status: int) -> str:
    return lib().fa_status_string(int(status)).decode()


# ------------------------------------------------------------------ C names
def fa_fwd(q, k, v, o, lse, B, H, Hkv, N, d, scale, causal, stream=None) -> int:
    return lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N, d, float(scale),
                        int(bool(causal)), _stream(stream))


def fa_fwd_fp8_workspace_bytes(B, H, Hkv, N, d) -> int:
    return int(lib().fa_fwd_fp8_workspace_bytes(B, H, Hkv, N, d))


def fa_fwd_fp8(q, k, v, rot_signs, o, lse, B, H, Hkv, N, d, scale, causal, workspace, workspace_bytes,
               stream=None) -> int:
    return lib().fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(rot_signs), _ptr(o), _ptr(lse), B, H, Hkv, N, d,
                            float(scale), int(bool(causal)), _ptr(workspace), int(workspace_bytes), _stream(stream))


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, B, max_seqlen, total, H, Hkv, d, scale, causal, stream=None) -> int:
    return lib().fa_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), B, max_seqlen, total,
                               H, Hkv, d, float(scale), int(bool(causal)), _stream(stream))


def fa_bwd_workspace_bytes(B, H, Hkv, N, d) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, H, Hkv, N, d))


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, Hkv, N, d, scale, causal, workspace, workspace_bytes,
           stream=None) -> int:
    return lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), B,
                        H, Hkv, N, d, float(scale), int(bool(causal)), _ptr(workspace), int(workspace_bytes),
                        _stream(stream))


def fa_bwd_fused_workspace_bytes(B, H, Hkv, N, d) -> int:
    return int(lib().fa_bwd_fused_workspace_bytes(B, H, Hkv, N, d))


def fa_bwd_fused(q, k, v, o, lse, dO, dq, dk, dv, B, H, Hkv, N, d, scale, causal, workspace, workspace_bytes,
                 stream=None) -> int:
    return lib().fa_bwd_fused(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
                              B, H, Hkv, N, d, float(scale), int(bool(causal)), _ptr(workspace), int(workspace_bytes),
                              _stream(stream))


def fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens, B, max_seqlen, total, H, Hkv, d, scale, causal,
                  workspace, workspace_bytes, stream=None) -> int:
    return lib().fa_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv),
                               _ptr(cu_seqlens), B, max_seqlen, total, H, Hkv, d, float(scale), int(bool(causal)),
                               _ptr(workspace), int(workspace_bytes), _stream(stream))


def fa_bwd_prepare(o, lse, dO, B, H, Hkv, N, d, workspace, workspace_bytes, stream=None) -> int:
    return lib().fa_bwd_prepare(_ptr(o), _ptr(lse), _ptr(dO), B, H, Hkv, N, d, _ptr(workspace),
                                int(workspace_bytes), _stream(stream))


def fa_bwd_dkdv(q, k, v, dO, dk, dv, B, H, Hkv, N, d, scale, causal, workspace, workspace_bytes,
                stream=None) -> int:
    return lib().fa_bwd_dkdv(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(dk), _ptr(dv), B, H, Hkv, N, d,
                             float(scale), int(bool(causal)), _ptr(workspace), int(workspace_bytes),
                             _stream(stream))


def fa_bwd_dq(q, k, v, dO, dq, B, H, Hkv, N, d, scale, causal, workspace, workspace_bytes, stream=None) -> int:
    return lib().fa_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(dq), B, H, Hkv, N, d, float(scale),
                           int(bool(causal)), _ptr(workspace), int(workspace_bytes), _stream(stream))


def fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B, H, Hkv, N, d, scale, causal, stream=None) -> int:
    """fa_bwd without a workspace: for callers that cannot allocate device
    memory when they run the backward pass (see include/fa.h)."""
    return lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                _ptr(dv), B, H, Hkv, N, d, float(scale), int(bool(causal)), _stream(stream))


def fa_bwd_noalloc_scratch_bytes() -> int:
    """Size of fa_bwd_noalloc's built-in scratch array, as the library was built."""
    return int(lib().fa_bwd_noalloc_scratch_bytes())


def fa_cache_append(k, v, k_pages, v_pages, page_table, cache_lens, cu_seqlens, B, max_pages, num_pages, page_size,
                    total, Hkv, d, stream=None) -> int:
    return lib().fa_cache_append(_ptr(k), _ptr(v), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cache_lens),
                                 _ptr(cu_seqlens), B, max_pages, num_pages, page_size, total, Hkv, d, _stream(stream))


def fa_fwd_paged_workspace_bytes(B, max_new, H, Hkv, d) -> int:
    return int(lib().fa_fwd_paged_workspace_bytes(B, max_new, H, Hkv, d))


def fa_fwd_paged(q, k_pages, v_pages, page_table, cache_lens, cu_seqlens, tree_mask, mask_words, o, lse, B, max_pages,
                 num_pages, page_size, max_new, total, H, Hkv, d, scale, workspace, workspace_bytes,
                 stream=None) -> int:
    return lib().fa_fwd_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cache_lens),
                              _ptr(cu_seqlens), _ptr(tree_mask), mask_words, _ptr(o), _ptr(lse), B, max_pages,
                              num_pages, page_size, max_new, total, H, Hkv, d, float(scale), _ptr(workspace),
                              int(workspace_bytes), _stream(stream))


def fa_cache_compact(k_pages, v_pages, page_table, cache_lens, accepted, n_accepted, lens_out, B, max_accepted,
                     max_pages, num_pages, page_size, layers, Hkv, d, stream=None) -> int:
    return lib().fa_cache_compact(_ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cache_lens), _ptr(accepted),
                                  _ptr(n_accepted), _ptr(lens_out), B, max_accepted, max_pages, num_pages, page_size,
                                  layers, Hkv, d, _stream(stream))


def fa_cache_fork(page_refs, page_table, cache_lens, parents, lens_out, B, max_pages, num_pages, page_size,
                  stream=None) -> int:
    return lib().fa_cache_fork(_ptr(page_refs), _ptr(page_table), _ptr(cache_lens), _ptr(parents), _ptr(lens_out), B,
                               max_pages, num_pages, page_size, _stream(stream))


def fa_cache_resize_workspace_bytes(B) -> int:
    return int(lib().fa_cache_resize_workspace_bytes(B))


def fa_cache_resize(page_refs, k_pages, v_pages, page_table, cache_lens, new_lens, lens_out, status, B, max_pages,
                    num_pages, page_size, layers, Hkv, d, workspace, workspace_bytes, stream=None) -> int:
    return lib().fa_cache_resize(_ptr(page_refs), _ptr(k_pages), _ptr(v_pages), _ptr(page_table), _ptr(cache_lens),
                                 _ptr(new_lens), _ptr(lens_out), _ptr(status), B, max_pages, num_pages, page_size,
                                 layers, Hkv, d, _ptr(workspace), int(workspace_bytes), _stream(stream))


def fa_exp2_poly(x, y, n, stream=None) -> int:
    return lib().fa_exp2_poly(_ptr(x), _ptr(y), int(n), _stream(stream))


def fa_rescale_count(stream=None) -> int:
    """Rescales applied by the forward kernels since the last call (then reset)."""
    c = ctypes.c_uint(0)
    st = lib().fa_rescale_count(_stream(stream), ctypes.addressof(c))
    if st != FA_OK:
        raise FaError(st, "fa_rescale_count")
    return int(c.value)


def fa_last_device_status(stream=None) -> int:
    return lib().fa_last_device_status(_stream(stream))


# ------------------------------------------------------------------ torch helpers
def _check(name, t, dtype, shape):
    """Raise ValueError unless t has this dtype and shape and is contiguous (the C ABI reads dense
    memory and cannot tell); returns (name, t) for the device check that follows all of them."""
    if t is None:
        raise ValueError(f"{name} is None")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return name, t


def _on_cuda(*checked):
    for name, t in checked:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")


def _dims(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, N, H, d] and [B, N, Hkv, d]")
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    return B, N, H, Hkv, d


def _check_fixed(q, k, v, o=None, lse=None, dO=None):
    import torch

    B, N, H, Hkv, d = _dims(q, k)
    c = [_check("q", q, torch.bfloat16, (B, N, H, d)), _check("k", k, torch.bfloat16, (B, N, Hkv, d)),
         _check("v", v, torch.bfloat16, (B, N, Hkv, d))]
    if o is not None:
        c.append(_check("o", o, torch.bfloat16, (B, N, H, d)))
    if dO is not None:
        c.append(_check("dO", dO, torch.bfloat16, (B, N, H, d)))
    if lse is not None:
        c.append(_check("lse", lse, torch.float32, (B, H, N)))
    _on_cuda(*c)
    return B, N, H, Hkv, d


def _check_packed(q, k, v, cu_seqlens, o=None, lse=None, dO=None):
    import torch

    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [total, H, d] and [total, Hkv, d]")
    total, H, d = q.shape
    Hkv = k.shape[1]
    c = [_check("q", q, torch.bfloat16, (total, H, d)), _check("k", k, torch.bfloat16, (total, Hkv, d)),
         _check("v", v, torch.bfloat16, (total, Hkv, d))]
    if cu_seqlens is None or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D int32 tensor of B + 1 offsets")
    c.append(_check("cu_seqlens", cu_seqlens, torch.int32, (cu_seqlens.numel(),)))
    if o is not None:
        c.append(_check("o", o, torch.bfloat16, (total, H, d)))
    if dO is not None:
        c.append(_check("dO", dO, torch.bfloat16, (total, H, d)))
    if lse is not None:
        c.append(_check("lse", lse, torch.float32, (H, total)))
    _on_cuda(*c)
    return total, H, Hkv, d


def attention_fwd(q, k, v, scale=None, causal=False, out=None, lse=None, stream=None):
    """q [B,N,H,d], k/v [B,N,Hkv,d] bf16 CUDA tensors -> (o bf16, lse fp32 [B,H,N])."""
    import torch

    B, N, H, Hkv, d = _check_fixed(q, k, v, o=out, lse=lse)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    st = fa_fwd(q, k, v, o, lse, B, H, Hkv, N, d, scale, causal, stream)
    if st != FA_OK:
        raise FaError(st, "fa_fwd")
    return o, lse


def attention_fwd_fp8(q, k, v, rot_signs=None, scale=None, causal=False, workspace=None, stream=None):
    """FP8 forward (d = 128): q [B,N,H,128], k/v [B,N,Hkv,128] bf16, rot_signs a float32 CUDA tensor of
    +-1 [128] or None -> (o bf16, lse fp32 [B,H,N], workspace holding the e4m3 tensors and scales)."""
    import torch

    if rot_signs is not None:
        _check("rot_signs", rot_signs, torch.float32, (128,))
    B, N, H, Hkv, d = _check_fixed(q, k, v)
    if rot_signs is not None:
        _on_cuda(("rot_signs", rot_signs))
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    nbytes = fa_fwd_fp8_workspace_bytes(B, H, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    st = fa_fwd_fp8(q, k, v, rot_signs, o, lse, B, H, Hkv, N, d, scale, causal, workspace, workspace.numel(), stream)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_fp8")
    return o, lse, workspace


def attention_fwd_varlen(q, k, v, cu_seqlens, max_seqlen, scale=None, causal=False, out=None, lse=None,
                         stream=None):
    """Packed batch: q [total,H,d], k/v [total,Hkv,d] bf16 CUDA tensors, cu_seqlens an int32
    CUDA tensor [B+1] -> (o bf16 [total,H,d], lse fp32 [H,total])."""
    import torch

    total, H, Hkv, d = _check_packed(q, k, v, cu_seqlens, o=out, lse=lse)
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o = torch.empty_like(q) if out is None else out
    lse = torch.empty((H, total), dtype=torch.float32, device=q.device) if lse is None else lse
    st = fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, B, int(max_seqlen), total, H, Hkv, d, scale, causal, stream)
    if st != FA_OK:
        raise FaError(st, "fa_fwd_varlen")
    return o, lse


def attention_bwd_varlen(q, k, v, o, lse, dO, cu_seqlens, max_seqlen, scale=None, causal=False, stream=None):
    """Packed batch backward (layouts of :func:`attention_fwd_varlen`) -> (dq, dk, dv) bf16."""
    import torch

    total, H, Hkv, d = _check_packed(q, k, v, cu_seqlens, o=o, lse=lse, dO=dO)
    B = cu_seqlens.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = fa_bwd_workspace_bytes(B, H, Hkv, int(max_seqlen), d)
    workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    st = fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens, B, int(max_seqlen), total, H, Hkv, d, scale,
                       causal, workspace, nbytes, stream)
    if st != FA_OK:
        raise FaError(st, "fa_bwd_varlen")
    return dq, dk, dv


def attention_bwd_fused(q, k, v, o, lse, dO, scale=None, causal=False, workspace=None, stream=None):
    """The fused CTA-pair backward (head dim 128): (dq, dk, dv) bf16, not bitwise reproducible."""
    import torch

    B, N, H, Hkv, d = _check_fixed(q, k, v, o=o, lse=lse, dO=dO)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = fa_bwd_fused_workspace_bytes(B, H, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    st = fa_bwd_fused(q, k, v, o, lse, dO, dq, dk, dv, B, H, Hkv, N, d, scale, causal, workspace, workspace.numel(),
                      stream)
    if st != FA_OK:
        raise FaError(st, "fa_bwd_fused")
    return dq, dk, dv


def attention_bwd(q, k, v, o, lse, dO, scale=None, causal=False, workspace=None, stream=None):
    """Returns (dq, dk, dv) bf16."""
    import torch

    B, N, H, Hkv, d = _check_fixed(q, k, v, o=o, lse=lse, dO=dO)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    nbytes = fa_bwd_workspace_bytes(B, H, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    st = fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, Hkv, N, d, scale, causal, workspace, workspace.numel(),
                stream)
    if st != FA_OK:
        raise FaError(st, "fa_bwd")
    return dq, dk, dv


# ------------------------------------------------------------------ paged cache
def _same_device(*checked):
    """Raise ValueError unless all tensors are on one CUDA device; returns it."""
    dev = checked[0][1].device
    for name, t in checked:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, {checked[0][0]} on {dev}")
    return dev


class _On:
    """Makes `dev` the current device and `stream` (None: its current stream) the current stream, so
    that what a call allocates belongs to the stream its kernels run on."""

    def __init__(self, dev, stream):
        import torch

        self.device = torch.cuda.device(dev)
        self.stream = None
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
            if stream.device != dev:
                raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
            self.stream = torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        if self.stream is not None:
            self.stream.__enter__()

    def __exit__(self, *exc):
        if self.stream is not None:
            self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _check_pages(k_pages, v_pages, layered):
    import torch

    dims = k_pages.dim()
    if dims != 4 and not (layered and dims == 5):
        raise ValueError("k_pages and v_pages must be [num_pages, page_size, Hkv, d]"
                         + (", or the same with a leading [layers]" if layered else ""))
    c = [_check("k_pages", k_pages, torch.bfloat16, k_pages.shape),
         _check("v_pages", v_pages, torch.bfloat16, k_pages.shape)]
    return c, (1 if dims == 4 else k_pages.shape[0]), *k_pages.shape[-4:]


def _check_table(page_table, cache_lens):
    import torch

    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    return [_check("page_table", page_table, torch.int32, (B, max_pages)),
            _check("cache_lens", cache_lens, torch.int32, (B,))], B, max_pages


# A decoding step makes these calls for every layer.  Their ordinary case (operands as documented, on
# the current device and stream, outputs allocated by the call) is checked and made by a CPython module,
# csrc/paged_binding.cpp; where that returns None, the code below says what is wrong or does the rest.
_fast = None


class _NoBinding:
    """Where no binding fits (none was built, or one for another torch): every call takes the code below,
    which costs some 10 us more on the host."""

    append = attention = compact = fork = resize = staticmethod(lambda *operands: None)


def _paged_binding():
    global _fast
    if _fast is None:
        import importlib.util

        import torch

        from . import build

        l = lib()
        try:
            spec = importlib.util.spec_from_file_location("_paged_binding", build.binding_path(torch))
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
        except ImportError as e:
            import warnings

            warnings.warn(f"paged-cache calls go through ctypes, some 10 us slower on the host: {e}", RuntimeWarning,
                          stacklevel=3)
            module = _NoBinding
        else:
            module.connect(*(ctypes.cast(getattr(l, name), ctypes.c_void_p).value for name in (
                "fa_cache_append", "fa_fwd_paged_workspace_bytes", "fa_fwd_paged", "fa_cache_compact", "fa_cache_fork",
                "fa_cache_resize_workspace_bytes", "fa_cache_resize")))
        _fast = module
    return _fast


def _done(result, what):
    """The result of a call, or FaError where it is a status."""
    if type(result) is int and result != FA_OK:
        raise FaError(result, what)
    return result


def _workspace(given, nbytes, dev):
    import torch

    if given is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev), nbytes
    return given, given.numel() * given.element_size()


def _int32(name, x):
    """x as the C int that the entry points take (ctypes would cut off what does not fit)."""
    x = int(x)
    if not -(2**31) <= x < 2**31:
        raise ValueError(f"{name} must fit 32 bits, is {x}")
    return x


def _check_workspace(workspace):
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return "workspace", workspace


def cache_append(k, v, k_pages, v_pages, page_table, cache_lens, cu_seqlens, stream=None):
    """Writes packed new rows k/v [total,Hkv,d] bf16 into the pages [num_pages,page_size,Hkv,d]: row i of
    sequence b (rows cu_seqlens[b]..cu_seqlens[b+1]) to place cache_lens[b] + i of the cache, i.e. row
    place % page_size of page page_table[b, place // page_size].  page_table int32 [B,max_pages],
    cache_lens int32 [B], cu_seqlens int32 [B+1]."""
    if stream is None:
        st = (_fast or _paged_binding()).append(k, v, k_pages, v_pages, page_table, cache_lens, cu_seqlens)
        if st is not None:
            _done(st, "fa_cache_append")
            return
    import torch

    pages, _, num_pages, page_size, Hkv, d = _check_pages(k_pages, v_pages, False)
    table, B, max_pages = _check_table(page_table, cache_lens)
    if k.dim() != 3:
        raise ValueError("k and v must be [total, Hkv, d]")
    total = k.shape[0]
    dev = _same_device(_check("k", k, torch.bfloat16, (total, Hkv, d)), _check("v", v, torch.bfloat16, (total, Hkv, d)),
                       *pages, *table, _check("cu_seqlens", cu_seqlens, torch.int32, (B + 1,)))
    with _On(dev, stream):
        if total > 0:
            _done(fa_cache_append(k, v, k_pages, v_pages, page_table, cache_lens, cu_seqlens, B, max_pages, num_pages,
                                  page_size, total, Hkv, d), "fa_cache_append")


def attention_fwd_paged(q, k_pages, v_pages, page_table, cache_lens, cu_seqlens, max_new, tree_mask=None, scale=None,
                        out=None, lse=None, workspace=None, stream=None):
    """Attention of new tokens q [total,H,d] bf16 (sequence b: rows cu_seqlens[b]..cu_seqlens[b+1], at most
    max_new <= 256 of them) over the cache, which already holds their own keys and values
    (:func:`cache_append`) -> (o bf16 [total,H,d], lse fp32 [H,total]).  Token i sees the cache_lens[b]
    places before the new ones and, of the new ones, those up to itself, or with tree_mask (int64
    [total, ceil(max_new / 64)]) those whose bits are set in its words.  A token that sees nothing gets
    o = 0 and lse = -inf."""
    if stream is None and out is None and lse is None and workspace is None:
        both = (_fast or _paged_binding()).attention(q, k_pages, v_pages, page_table, cache_lens, cu_seqlens, max_new,
                                                     tree_mask, scale)
        if both is not None:
            return _done(both, "fa_fwd_paged")
    import torch

    pages, _, num_pages, page_size, Hkv, d = _check_pages(k_pages, v_pages, False)
    table, B, max_pages = _check_table(page_table, cache_lens)
    if q.dim() != 3:
        raise ValueError("q must be [total, H, d]")
    total, H, _ = q.shape
    max_new = _int32("max_new", max_new)
    words = (max_new + 63) // 64 if tree_mask is not None else 0
    c = [_check("q", q, torch.bfloat16, (total, H, d)), *pages, *table,
         _check("cu_seqlens", cu_seqlens, torch.int32, (B + 1,))]
    if tree_mask is not None:
        c.append(_check("tree_mask", tree_mask, torch.int64, (total, words)))
    if out is not None:
        c.append(_check("out", out, torch.bfloat16, (total, H, d)))
    if lse is not None:
        c.append(_check("lse", lse, torch.float32, (H, total)))
    if workspace is not None:
        c.append(_check_workspace(workspace))
    dev = _same_device(*c)
    with _On(dev, stream):
        o = torch.empty_like(q) if out is None else out
        lse = torch.empty((H, total), dtype=torch.float32, device=dev) if lse is None else lse
        if total > 0:
            workspace, nbytes = _workspace(workspace, fa_fwd_paged_workspace_bytes(B, max_new, H, Hkv, d), dev)
            _done(fa_fwd_paged(q, k_pages, v_pages, page_table, cache_lens, cu_seqlens, tree_mask, words, o, lse, B,
                               max_pages, num_pages, page_size, max_new, total, H, Hkv, d,
                               1.0 / math.sqrt(d) if scale is None else scale, workspace, nbytes), "fa_fwd_paged")
    return o, lse


def cache_compact(k_pages, v_pages, page_table, cache_lens, accepted, n_accepted, stream=None):
    """Moves the accepted path of each sequence's drafted tokens together, in every layer (k/v_pages
    [num_pages,page_size,Hkv,d], or with a leading [layers]): the rows of place cache_lens[b] +
    accepted[b, i] go to place cache_lens[b] + i for i < n_accepted[b] -> new lengths int32 [B].
    accepted int32 [B,max_accepted] ascends along each path; a path ends before the first entry that
    does not.  Without columns (no token accepted anywhere) the lengths are copied and nothing moves."""
    if stream is None:
        lens = (_fast or _paged_binding()).compact(k_pages, v_pages, page_table, cache_lens, accepted, n_accepted)
        if lens is not None:
            return _done(lens, "fa_cache_compact")
    import torch

    pages, layers, num_pages, page_size, Hkv, d = _check_pages(k_pages, v_pages, True)
    table, B, max_pages = _check_table(page_table, cache_lens)
    if accepted.dim() != 2:
        raise ValueError("accepted must be [B, max_accepted]")
    most = accepted.shape[1]
    dev = _same_device(*pages, *table, _check("accepted", accepted, torch.int32, (B, most)),
                       _check("n_accepted", n_accepted, torch.int32, (B,)))
    with _On(dev, stream):
        if most == 0:  # no path has a token
            return cache_lens.clone()
        lens = torch.empty_like(cache_lens)
        _done(fa_cache_compact(k_pages, v_pages, page_table, cache_lens, accepted, n_accepted, lens, B, most, max_pages,
                               num_pages, page_size, layers, Hkv, d), "fa_cache_compact")
    return lens


def cache_fork(page_refs, page_table, cache_lens, parents, page_size, stream=None):
    """Row b of page_table becomes what row parents[b] was before the call, sharing its pages (-1 empties
    the row; b leaves it alone) -> new lengths int32 [B].  page_refs int32 [num_pages] counts the rows
    that hold each page and is kept in step; no key or value moves."""
    if stream is None:
        lens = (_fast or _paged_binding()).fork(page_refs, page_table, cache_lens, parents, page_size)
        if lens is not None:
            return _done(lens, "fa_cache_fork")
    import torch

    table, B, max_pages = _check_table(page_table, cache_lens)
    if page_refs.dim() != 1:
        raise ValueError("page_refs must be [num_pages]")
    num_pages = page_refs.shape[0]
    page_size = _int32("page_size", page_size)
    dev = _same_device(_check("page_refs", page_refs, torch.int32, (num_pages,)), *table,
                       _check("parents", parents, torch.int32, (B,)))
    with _On(dev, stream):
        lens = torch.empty_like(cache_lens)
        _done(fa_cache_fork(page_refs, page_table, cache_lens, parents, lens, B, max_pages, num_pages, page_size),
              "fa_cache_fork")
    return lens


def cache_resize(page_refs, k_pages, v_pages, page_table, cache_lens, new_lens, workspace=None, stream=None):
    """Makes every row of page_table hold new_lens[b] places: shrinking rows give pages back, growing rows
    take free ones (count 0 in page_refs), lowest first, and a growing row's shared, partly filled last
    page is first copied into one of its own, in every layer -> (lengths int32 [B], status int32 [2]).
    status[0] is the number of pages that were missing (then no row has grown), status[1] the number of
    rows left alone because a length was negative or past the table."""
    if stream is None and workspace is None:
        both = (_fast or _paged_binding()).resize(page_refs, k_pages, v_pages, page_table, cache_lens, new_lens)
        if both is not None:
            return _done(both, "fa_cache_resize")
    import torch

    pages, layers, num_pages, page_size, Hkv, d = _check_pages(k_pages, v_pages, True)
    table, B, max_pages = _check_table(page_table, cache_lens)
    c = [_check("page_refs", page_refs, torch.int32, (num_pages,)), *pages, *table,
         _check("new_lens", new_lens, torch.int32, (B,))]
    if workspace is not None:
        c.append(_check_workspace(workspace))
    dev = _same_device(*c)
    with _On(dev, stream):
        lens = torch.empty_like(cache_lens)
        status = torch.empty(2, dtype=torch.int32, device=dev)
        workspace, nbytes = _workspace(workspace, fa_cache_resize_workspace_bytes(B), dev)
        _done(fa_cache_resize(page_refs, k_pages, v_pages, page_table, cache_lens, new_lens, lens, status, B, max_pages,
                              num_pages, page_size, layers, Hkv, d, workspace, nbytes), "fa_cache_resize")
    return lens, status
