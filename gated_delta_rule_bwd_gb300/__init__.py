"""GB300 (sm_103a) Gated DeltaNet / Kimi Delta Attention token mixer.

Thin ctypes binding over the C ABI in ``include/gdn.h`` (``libgdn.so``).  The
functions here only marshal arguments: they check dtypes and devices, allocate
the outputs and the backward workspace with PyTorch, and pass raw device
pointers and the current CUDA stream to the library.  Every step of the
computation runs in the library's CUDA kernels; there is no other path.  If
the library has not been built, every call raises.

Names follow the ABI: ``gdn_fwd``, ``gdn_bwd``, ``kda_fwd``, ``kda_bwd`` and
``mamba2_fwd``, ``mamba2_bwd`` (the scalar-gated state without the delta rule);
the training pair with a saved context ``gdn_fwd_save`` / ``gdn_bwd_saved``
(and the KDA and Mamba2 pairs), whose forward keeps what the backward would
recompute; and the token-recurrent ``gdn_decode`` / ``kda_decode`` for a few
tokens per sequence.  The mixer's fused neighbours: ``short_conv_fwd`` /
``short_conv_bwd`` (causal depthwise convolution + SiLU, with the per-head
L2 norm for q and k) and ``gated_rmsnorm_fwd`` / ``gated_rmsnorm_bwd``.  The
softmax attention layers between the mixers: ``attn_fwd`` / ``attn_bwd`` (causal,
grouped heads, packed sequences), ``attn_decode`` (a few tokens against a cache
that the call extends), and the pre-norm ``layer_norm_fwd`` / ``layer_norm_bwd``.
In front of them ``qk_norm_rope_fwd`` / ``qk_norm_rope_bwd`` (norm of the query and
key heads and rotation by position), and for serving from pages of 16-bit, fp32 or
4-bit keys and values ``kv_append``, ``attn_paged`` and ``kv_gather``.
Token tensors are ``[B, T, H, D]`` (fp32 or bf16, all the same dtype), ``g``
is ``[B, T, H]`` (GDN) or ``[B, T, H, dk]`` (KDA) fp32, ``beta`` ``[B, T, H]``
fp32, states ``[B, H, dk, dv]`` fp32.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_F32, GDN_BF16, GDN_BF16_G16 = 0, 1, 2
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


class GdnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class ConvShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("D", ctypes.c_int), ("W", ctypes.c_int), ("dtype", ctypes.c_int)]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("D", ctypes.c_int), ("dtype", ctypes.c_int)]


class AttnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Tq", ctypes.c_int), ("Tk", ctypes.c_int),
                ("H", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("q_stride", ctypes.c_longlong * 3),
                ("k_stride", ctypes.c_longlong * 3), ("v_stride", ctypes.c_longlong * 3)]


class AttnDecodeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("S", ctypes.c_int),
                ("H", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("kc_stride", ctypes.c_longlong * 3),
                ("vc_stride", ctypes.c_longlong * 3)]


class QkRopeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("Hkv", ctypes.c_int), ("D", ctypes.c_int), ("R", ctypes.c_int),
                ("P", ctypes.c_int), ("interleaved", ctypes.c_int), ("dtype", ctypes.c_int),
                ("q_stride", ctypes.c_longlong * 3), ("k_stride", ctypes.c_longlong * 3)]


class PagedCacheDesc(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int), ("page", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("format", ctypes.c_int), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("k_stride", ctypes.c_longlong * 3), ("v_stride", ctypes.c_longlong * 3),
                ("k_scale_stride", ctypes.c_longlong * 3), ("v_scale_stride", ctypes.c_longlong * 3)]


class KvAppendShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int), ("R", ctypes.c_int),
                ("P", ctypes.c_int), ("interleaved", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rows", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("table_stride", ctypes.c_longlong), ("q_stride", ctypes.c_longlong * 3),
                ("k_stride", ctypes.c_longlong * 3), ("v_stride", ctypes.c_longlong * 3)]


class AttnPagedShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dtype", ctypes.c_int), ("max_pages", ctypes.c_int),
                ("table_stride", ctypes.c_longlong)]


class GdnError(RuntimeError):
    pass


_lock = threading.Lock()
_lib = None
EXPORTS = ("gdn_fwd", "gdn_bwd", "kda_fwd", "kda_bwd", "gdn_fwd_workspace", "kda_fwd_workspace",
           "gdn_bwd_workspace", "kda_bwd_workspace", "gdn_ctx_bytes", "kda_ctx_bytes",
           "gdn_fwd_save", "kda_fwd_save", "gdn_bwd_saved", "kda_bwd_saved",
           "mamba2_fwd", "mamba2_bwd", "mamba2_fwd_save", "mamba2_bwd_saved",
           "mamba2_fwd_workspace", "mamba2_bwd_workspace", "mamba2_ctx_bytes",
           "gdn_decode", "kda_decode",
           "gdn_status_str", "gdn_last_cuda_error", "gdn_device_status", "gdn_uses_tensor_cores",
           "gdn_wait_selftest", "gdn_attn_wait_selftest", "kda_uses_tensor_cores",
           "gdn_varlen_workspace", "kda_varlen_workspace", "mamba2_varlen_workspace",
           "gdn_fwd_varlen", "gdn_bwd_varlen", "kda_fwd_varlen", "kda_bwd_varlen",
           "mamba2_fwd_varlen", "mamba2_bwd_varlen",
           "gdn_short_conv_fwd", "gdn_short_conv_bwd", "gdn_short_conv_bwd_workspace",
           "gdn_gated_rmsnorm_fwd", "gdn_gated_rmsnorm_bwd", "gdn_gated_rmsnorm_bwd_workspace",
           "gdn_attn_fwd_workspace", "gdn_attn_fwd", "gdn_attn_bwd_workspace", "gdn_attn_bwd",
           "gdn_attn_decode_workspace", "gdn_attn_decode",
           "gdn_layer_norm_fwd", "gdn_layer_norm_bwd", "gdn_layer_norm_bwd_workspace",
           "gdn_qk_norm_rope_fwd", "gdn_qk_norm_rope_bwd", "gdn_qk_norm_rope_bwd_workspace",
           "gdn_kv_append", "gdn_kv_gather", "gdn_attn_paged", "gdn_attn_paged_workspace",
           "gdn_profile_begin", "gdn_profile_end", "gdn_profile_read", "gdn_kernel_name")


def lib():
    """The loaded ``libgdn.so``; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise GdnError(f"{LIB_PATH} is missing: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
            L = ctypes.CDLL(LIB_PATH)
            vp, sz, fp = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p
            sp = ctypes.POINTER(GdnShape)
            for name in ("gdn_fwd_workspace", "kda_fwd_workspace", "gdn_bwd_workspace",
                         "kda_bwd_workspace", "gdn_ctx_bytes", "kda_ctx_bytes",
                         "mamba2_fwd_workspace", "mamba2_bwd_workspace", "mamba2_ctx_bytes"):
                getattr(L, name).argtypes = [sp]
                getattr(L, name).restype = sz
            for name in ("gdn_fwd", "kda_fwd", "gdn_fwd_save", "kda_fwd_save", "mamba2_fwd",
                         "mamba2_fwd_save"):
                getattr(L, name).argtypes = [sp] + [vp] * 8 + [vp, sz, vp]
                getattr(L, name).restype = ctypes.c_int
            for name in ("gdn_bwd", "kda_bwd", "gdn_bwd_saved", "kda_bwd_saved", "mamba2_bwd",
                         "mamba2_bwd_saved"):
                getattr(L, name).argtypes = [sp] + [vp] * 14 + [vp, sz, vp]
                getattr(L, name).restype = ctypes.c_int
            for name in ("gdn_decode", "kda_decode"):
                getattr(L, name).argtypes = [sp] + [vp] * 8 + [vp]
                getattr(L, name).restype = ctypes.c_int
            L.gdn_status_str.argtypes = [ctypes.c_int]
            L.gdn_status_str.restype = ctypes.c_char_p
            L.gdn_last_cuda_error.argtypes = []
            L.gdn_last_cuda_error.restype = ctypes.c_int
            L.gdn_device_status.argtypes = []
            L.gdn_device_status.restype = ctypes.c_int
            for name in ("gdn_varlen_workspace", "kda_varlen_workspace", "mamba2_varlen_workspace"):
                getattr(L, name).argtypes = [sp, ctypes.c_int, ctypes.c_int]
                getattr(L, name).restype = sz
            for name in ("gdn_fwd_varlen", "kda_fwd_varlen", "mamba2_fwd_varlen"):
                getattr(L, name).argtypes = [sp, vp, ctypes.c_int] + [vp] * 8 + [vp, sz, vp]
                getattr(L, name).restype = ctypes.c_int
            for name in ("gdn_bwd_varlen", "kda_bwd_varlen", "mamba2_bwd_varlen"):
                getattr(L, name).argtypes = [sp, vp, ctypes.c_int] + [vp] * 14 + [vp, sz, vp]
                getattr(L, name).restype = ctypes.c_int
            for name in ("gdn_wait_selftest", "gdn_attn_wait_selftest"):
                getattr(L, name).argtypes = [ctypes.c_int, vp]
                getattr(L, name).restype = ctypes.c_int
            for name in ("gdn_uses_tensor_cores", "kda_uses_tensor_cores"):
                getattr(L, name).argtypes = [sp]
                getattr(L, name).restype = ctypes.c_int
            cs, ns, f32, i32 = (ctypes.POINTER(ConvShape), ctypes.POINTER(NormShape),
                                ctypes.c_float, ctypes.c_int)
            L.gdn_short_conv_fwd.argtypes = [cs, vp, vp, vp, i32, f32, f32, vp, i32, vp]
            L.gdn_short_conv_fwd.restype = ctypes.c_int
            L.gdn_short_conv_bwd_workspace.argtypes = [cs]
            L.gdn_short_conv_bwd_workspace.restype = sz
            L.gdn_short_conv_bwd.argtypes = [cs, vp, vp, vp, vp, vp, i32, f32, f32, vp, i32, vp, sz,
                                             vp]
            L.gdn_short_conv_bwd.restype = ctypes.c_int
            L.gdn_gated_rmsnorm_fwd.argtypes = [ns, vp, vp, vp, vp, f32, vp]
            L.gdn_gated_rmsnorm_fwd.restype = ctypes.c_int
            L.gdn_gated_rmsnorm_bwd_workspace.argtypes = [ns]
            L.gdn_gated_rmsnorm_bwd_workspace.restype = sz
            L.gdn_gated_rmsnorm_bwd.argtypes = [ns, vp, vp, vp, vp, vp, vp, vp, f32, vp, sz, vp]
            L.gdn_gated_rmsnorm_bwd.restype = ctypes.c_int
            as_, ds = ctypes.POINTER(AttnShape), ctypes.POINTER(AttnDecodeShape)
            for name in ("gdn_attn_fwd_workspace", "gdn_attn_bwd_workspace"):
                getattr(L, name).argtypes = [as_, i32]
                getattr(L, name).restype = sz
            L.gdn_attn_fwd.argtypes = [as_, vp, vp, vp, f32, vp, vp, i32, vp, vp, vp, sz, vp]
            L.gdn_attn_fwd.restype = ctypes.c_int
            L.gdn_attn_bwd.argtypes = [as_, vp, vp, vp, f32, vp, vp, i32] + [vp] * 7 + [sz, vp]
            L.gdn_attn_bwd.restype = ctypes.c_int
            L.gdn_attn_decode_workspace.argtypes = [ds]
            L.gdn_attn_decode_workspace.restype = sz
            L.gdn_attn_decode.argtypes = [ds] + [vp] * 6 + [f32, vp, vp, sz, vp]
            L.gdn_attn_decode.restype = ctypes.c_int
            L.gdn_layer_norm_fwd.argtypes = [ns, vp, vp, vp, vp, vp, vp, f32, vp]
            L.gdn_layer_norm_fwd.restype = ctypes.c_int
            L.gdn_layer_norm_bwd_workspace.argtypes = [ns]
            L.gdn_layer_norm_bwd_workspace.restype = sz
            L.gdn_layer_norm_bwd.argtypes = [ns] + [vp] * 9 + [sz, vp]
            L.gdn_layer_norm_bwd.restype = ctypes.c_int
            # shapes and caches go in as packed bytes (or by reference to a Structure)
            L.gdn_qk_norm_rope_fwd.argtypes = [vp] * 5 + [f32] + [vp] * 6
            L.gdn_qk_norm_rope_fwd.restype = i32
            L.gdn_qk_norm_rope_bwd_workspace.argtypes = [vp]
            L.gdn_qk_norm_rope_bwd_workspace.restype = sz
            L.gdn_qk_norm_rope_bwd.argtypes = [vp] * 5 + [f32] + [vp] * 10 + [sz, vp]
            L.gdn_qk_norm_rope_bwd.restype = i32
            L.gdn_kv_append.argtypes = [vp] * 12
            L.gdn_kv_append.restype = i32
            L.gdn_kv_gather.argtypes = [vp, vp, i32, i32, ctypes.c_longlong, vp, i32, i32, vp, vp, vp]
            L.gdn_kv_gather.restype = i32
            L.gdn_attn_paged_workspace.argtypes = [vp, vp]
            L.gdn_attn_paged_workspace.restype = sz
            L.gdn_attn_paged.argtypes = [vp] * 5 + [f32, vp, vp, sz, vp]
            L.gdn_attn_paged.restype = i32
            L.gdn_profile_begin.argtypes = [ctypes.c_int]
            L.gdn_profile_begin.restype = ctypes.c_int
            L.gdn_profile_end.argtypes = []
            L.gdn_profile_end.restype = ctypes.c_int
            L.gdn_profile_read.argtypes = [ctypes.POINTER(ctypes.c_int),
                                           ctypes.POINTER(ctypes.c_float), ctypes.c_int]
            L.gdn_profile_read.restype = ctypes.c_int
            L.gdn_kernel_name.argtypes = [ctypes.c_int]
            L.gdn_kernel_name.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _ptr(x):
    return None if x is None else ctypes.c_void_p(x.data_ptr())


def _check(rc):
    if rc != 0:
        L = lib()
        msg = L.gdn_status_str(rc).decode()
        if rc == -6:
            msg += f" (cudaError {L.gdn_last_cuda_error()})"
        raise GdnError(msg)


def make_shape(q, v, chunk, g=None) -> GdnShape:
    """The ABI shape of a call; a bf16 ``g`` (KDA) selects GDN_BF16_G16."""
    B, T, H, dk = q.shape
    dt = _DTYPES[q.dtype]
    if g is not None and g.dtype == torch.bfloat16:
        dt = GDN_BF16_G16
    return GdnShape(B, T, H, dk, v.shape[3], chunk, dt)


def _validate(q, k, v, g, beta, kda, extra=()):
    if q.dtype not in _DTYPES:
        raise GdnError(f"unsupported dtype {q.dtype}")
    dev = q.device
    if dev.type != "cuda":
        raise GdnError("inputs must be CUDA tensors (the library has no CPU path)")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    want = {"k": (k, (B, T, H, dk), q.dtype), "v": (v, (B, T, H, dv), q.dtype),
            "g": (g, (B, T, H, dk) if kda else (B, T, H),
                  torch.bfloat16 if (kda and g is not None and g.dtype == torch.bfloat16
                                     and q.dtype == torch.bfloat16) else torch.float32),
            "beta": (beta, (B, T, H), torch.float32)}
    for name, (x, shape, dt) in list(want.items()) + list(extra):
        if x is None:
            continue
        if tuple(x.shape) != tuple(shape) or x.dtype != dt or x.device != dev:
            raise GdnError(f"{name}: expected {tuple(shape)} {dt} on {dev}, got "
                           f"{tuple(x.shape)} {x.dtype} on {x.device}")
        if not x.is_contiguous():
            raise GdnError(f"{name} must be contiguous")


def _on_current(device):
    """Refuses tensors of a device that is not the current one: the library's kernels
    run on the current device, whatever device a stream or a pointer belongs to."""
    if device.index != torch.cuda.current_device():
        raise GdnError(f"the tensors are on {device}, the current device is "
                       f"cuda:{torch.cuda.current_device()}: call inside torch.cuda.device({device.index})")


def _stream(dev):
    _on_current(dev)
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _mixer(kda, delta):
    if kda and not delta:
        raise GdnError("the per-key-dimension gate is only offered with the delta rule (KDA)")
    return "kda" if kda else ("gdn" if delta else "mamba2")


def _entry(kda, delta, name):
    """The ABI function ``<mixer>_<name>``."""
    return getattr(lib(), f"{_mixer(kda, delta)}_{name}")


def fwd_workspace_bytes(q, v, chunk=64, kda=False, delta=True) -> int:
    s = make_shape(q, v, chunk)
    return int(_entry(kda, delta, "fwd_workspace")(ctypes.byref(s)))


def bwd_workspace_bytes(q, v, chunk=64, kda=False, delta=True) -> int:
    s = make_shape(q, v, chunk)
    return int(_entry(kda, delta, "bwd_workspace")(ctypes.byref(s)))


def ctx_bytes(q, v, chunk=64, kda=False, delta=True) -> int:
    """Bytes of the saved context of ``*_fwd_save`` / ``*_bwd_saved``."""
    s = make_shape(q, v, chunk)
    return int(_entry(kda, delta, "ctx_bytes")(ctypes.byref(s)))


def _workspace(need, given, device):
    if given is not None and (given.device != device or not given.is_contiguous()):
        raise GdnError(f"workspace must be contiguous and on {device}, got one on {given.device}")
    if given is not None and given.numel() >= need:
        return given
    return torch.empty(max(need, 16), dtype=torch.uint8, device=device)


def uses_tensor_cores(q, v, chunk=64, kda=False) -> bool:
    s = make_shape(q, v, chunk)
    fn = lib().kda_uses_tensor_cores if kda else lib().gdn_uses_tensor_cores
    return bool(fn(ctypes.byref(s)))


def _fwd(kda, q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, out=None,
         workspace=None, ctx=None, delta=True):
    B, T, H, dk = q.shape
    dv = v.shape[3]
    _validate(q, k, v, g, beta, kda, [("h0", (h0, (B, H, dk, dv), torch.float32))])
    o = out if out is not None else torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    ht = (torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
          if output_final_state else None)
    if ctx is not None:
        _check_ctx(ctx, ctx_bytes(q, v, chunk, kda, delta), q.device)
        ws = ctx
        fn = _entry(kda, delta, "fwd_save")
    else:
        ws = _workspace(fwd_workspace_bytes(q, v, chunk, kda, delta), workspace, q.device)
        fn = _entry(kda, delta, "fwd")
    s = make_shape(q, v, chunk, g)
    _check(fn(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o),
              _ptr(ht), _ptr(ws), ws.numel(), _stream(q.device)))
    return o, ht


def _check_ctx(ctx, need, device):
    if (not isinstance(ctx, torch.Tensor) or ctx.dtype != torch.uint8 or ctx.device != device
            or not ctx.is_contiguous() or ctx.numel() < need):
        raise GdnError(f"ctx must be a contiguous uint8 tensor of at least {need} bytes "
                       f"on {device} (see new_ctx)")


def _bwd(kda, q, k, v, g, beta, h0, do, dht=None, chunk=64, want_dh0=True, workspace=None,
         ctx=None, delta=True):
    B, T, H, dk = q.shape
    dv = v.shape[3]
    _validate(q, k, v, g, beta, kda, [("h0", (h0, (B, H, dk, dv), torch.float32)),
                                      ("do", (do, (B, T, H, dv), q.dtype)),
                                      ("dht", (dht, (B, H, dk, dv), torch.float32))])
    e = lambda x: torch.empty_like(x)
    dq, dk_, dv_, dg, dbeta = e(q), e(k), e(v), e(g), e(beta)
    dh0 = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_dh0 else None
    if ctx is not None:
        _check_ctx(ctx, ctx_bytes(q, v, chunk, kda, delta), q.device)
        ws = ctx
        fn = _entry(kda, delta, "bwd_saved")
    else:
        ws = _workspace(bwd_workspace_bytes(q, v, chunk, kda, delta), workspace, q.device)
        fn = _entry(kda, delta, "bwd")
    s = make_shape(q, v, chunk, g)
    _check(fn(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(do),
              _ptr(dht), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(dbeta), _ptr(dh0),
              _ptr(ws), ws.numel(), _stream(q.device)))
    return {"dq": dq, "dk": dk_, "dv": dv_, "dg": dg, "dbeta": dbeta, "dh0": dh0}


def gdn_fwd(q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, workspace=None):
    """GDN forward.  Returns ``(o, ht)`` (``ht`` None if not requested).  ``workspace``
    (uint8 CUDA tensor) is used when it holds ``fwd_workspace_bytes`` bytes, else one
    is allocated."""
    return _fwd(False, q, k, v, g, beta, h0, chunk, output_final_state, workspace=workspace)


def kda_fwd(q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, workspace=None):
    """KDA forward (``g`` is ``[B,T,H,dk]``).  Returns ``(o, ht)``."""
    return _fwd(True, q, k, v, g, beta, h0, chunk, output_final_state, workspace=workspace)


def gdn_bwd(q, k, v, g, beta, h0, do, dht=None, chunk=64, want_dh0=True, workspace=None):
    """GDN backward.  Returns a dict ``dq, dk, dv, dg, dbeta, dh0``."""
    return _bwd(False, q, k, v, g, beta, h0, do, dht, chunk, want_dh0, workspace)


def kda_bwd(q, k, v, g, beta, h0, do, dht=None, chunk=64, want_dh0=True, workspace=None):
    """KDA backward.  Returns a dict ``dq, dk, dv, dg, dbeta, dh0``."""
    return _bwd(True, q, k, v, g, beta, h0, do, dht, chunk, want_dh0, workspace)


def new_ctx(q, v, chunk=64, kda=False, delta=True):
    """An uninitialised saved-context buffer for ``q``/``v``'s shape."""
    return torch.empty(max(16, ctx_bytes(q, v, chunk, kda, delta)), dtype=torch.uint8,
                       device=q.device)


def gdn_fwd_save(q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, ctx=None):
    """GDN forward that also leaves the saved context for ``gdn_bwd_saved``.
    Returns ``(o, ht, ctx)``; ``ctx`` (from ``new_ctx``) is allocated if not given."""
    ctx = new_ctx(q, v, chunk) if ctx is None else ctx
    o, ht = _fwd(False, q, k, v, g, beta, h0, chunk, output_final_state, ctx=ctx)
    return o, ht, ctx


def kda_fwd_save(q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, ctx=None):
    """KDA forward that also leaves the saved context for ``kda_bwd_saved``."""
    ctx = new_ctx(q, v, chunk, True) if ctx is None else ctx
    o, ht = _fwd(True, q, k, v, g, beta, h0, chunk, output_final_state, ctx=ctx)
    return o, ht, ctx


def gdn_bwd_saved(q, k, v, g, beta, h0, do, ctx, dht=None, chunk=64, want_dh0=True):
    """GDN backward reading the context ``gdn_fwd_save`` left in ``ctx`` (the same
    q, k, v, g, beta, h0 must be passed).  Returns the dict of ``gdn_bwd``."""
    return _bwd(False, q, k, v, g, beta, h0, do, dht, chunk, want_dh0, ctx=ctx)


def kda_bwd_saved(q, k, v, g, beta, h0, do, ctx, dht=None, chunk=64, want_dh0=True):
    """KDA backward reading the context ``kda_fwd_save`` left in ``ctx``."""
    return _bwd(True, q, k, v, g, beta, h0, do, dht, chunk, want_dh0, ctx=ctx)


def mamba2_fwd(q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, workspace=None):
    """Mamba2 forward (``g`` is ``[B,T,H]``): the scalar-gated state without the
    delta rule, ``H_t = exp(g_t) H_{t-1} + beta_t k_t v_t^T``.  Returns ``(o, ht)``."""
    return _fwd(False, q, k, v, g, beta, h0, chunk, output_final_state, workspace=workspace,
                delta=False)


def mamba2_bwd(q, k, v, g, beta, h0, do, dht=None, chunk=64, want_dh0=True, workspace=None):
    """Mamba2 backward.  Returns a dict ``dq, dk, dv, dg, dbeta, dh0``."""
    return _bwd(False, q, k, v, g, beta, h0, do, dht, chunk, want_dh0, workspace, delta=False)


def mamba2_fwd_save(q, k, v, g, beta, h0=None, chunk=64, output_final_state=True, ctx=None):
    """Mamba2 forward that also leaves the saved context for ``mamba2_bwd_saved``."""
    ctx = new_ctx(q, v, chunk, delta=False) if ctx is None else ctx
    o, ht = _fwd(False, q, k, v, g, beta, h0, chunk, output_final_state, ctx=ctx, delta=False)
    return o, ht, ctx


def mamba2_bwd_saved(q, k, v, g, beta, h0, do, ctx, dht=None, chunk=64, want_dh0=True):
    """Mamba2 backward reading the context ``mamba2_fwd_save`` left in ``ctx``."""
    return _bwd(False, q, k, v, g, beta, h0, do, dht, chunk, want_dh0, ctx=ctx, delta=False)


# ------------------------------------------------------------------ packed sequences

def varlen_workspace_bytes(q, v, nseq, chunk=64, kda=False, delta=True, backward=False) -> int:
    """Workspace bytes of a packed-sequence call (``*_varlen_workspace``)."""
    s = make_shape(q, v, chunk)
    return int(_entry(kda, delta, "varlen_workspace")(ctypes.byref(s), int(nseq), int(backward)))


def _check_cu(cu_seqlens, q):
    if (not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32
            or cu_seqlens.device != q.device or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1
            or not cu_seqlens.is_contiguous()):
        raise GdnError("cu_seqlens must be a contiguous 1-D int32 tensor on the inputs' device")
    if q.shape[0] != 1:
        raise GdnError("packed sequences: the token tensors must be [1, T, H, D]")
    return cu_seqlens.numel() - 1


def _fwd_varlen(kda, delta, q, k, v, g, beta, cu_seqlens, h0, chunk, workspace):
    nseq = _check_cu(cu_seqlens, q)
    _, T, H, dk = q.shape
    dv = v.shape[3]
    _validate(q, k, v, g, beta, kda, [("h0", (h0, (nseq, H, dk, dv), torch.float32))])
    o = torch.empty((1, T, H, dv), dtype=q.dtype, device=q.device)
    ht = torch.empty((nseq, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = _workspace(varlen_workspace_bytes(q, v, nseq, chunk, kda, delta), workspace, q.device)
    s = make_shape(q, v, chunk, g)
    _check(_entry(kda, delta, "fwd_varlen")(ctypes.byref(s), _ptr(cu_seqlens), nseq, _ptr(q), _ptr(k),
                                            _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(ht),
                                            _ptr(ws), ws.numel(), _stream(q.device)))
    return o, ht


def _bwd_varlen(kda, delta, q, k, v, g, beta, cu_seqlens, h0, do, dht, chunk, workspace):
    nseq = _check_cu(cu_seqlens, q)
    _, T, H, dk = q.shape
    dv = v.shape[3]
    _validate(q, k, v, g, beta, kda, [("h0", (h0, (nseq, H, dk, dv), torch.float32)),
                                      ("do", (do, (1, T, H, dv), q.dtype)),
                                      ("dht", (dht, (nseq, H, dk, dv), torch.float32))])
    e = lambda x: torch.empty_like(x)
    dq, dk_, dv_, dg, dbeta = e(q), e(k), e(v), e(g), e(beta)
    dh0 = torch.empty((nseq, H, dk, dv), dtype=torch.float32, device=q.device)
    ws = _workspace(varlen_workspace_bytes(q, v, nseq, chunk, kda, delta, True), workspace, q.device)
    s = make_shape(q, v, chunk, g)
    _check(_entry(kda, delta, "bwd_varlen")(ctypes.byref(s), _ptr(cu_seqlens), nseq, _ptr(q), _ptr(k),
                                            _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(do), _ptr(dht),
                                            _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(dbeta),
                                            _ptr(dh0), _ptr(ws), ws.numel(), _stream(q.device)))
    return {"dq": dq, "dk": dk_, "dv": dv_, "dg": dg, "dbeta": dbeta, "dh0": dh0}


def gdn_fwd_varlen(q, k, v, g, beta, cu_seqlens, h0=None, chunk=64, workspace=None):
    """GDN forward over packed sequences: token tensors ``[1, T, H, D]``,
    ``cu_seqlens`` an int32 device tensor of ``nseq + 1`` offsets, ``h0`` and the
    returned ``ht`` ``[nseq, H, dk, dv]``.  Returns ``(o, ht)``."""
    return _fwd_varlen(False, True, q, k, v, g, beta, cu_seqlens, h0, chunk, workspace)


def gdn_bwd_varlen(q, k, v, g, beta, cu_seqlens, h0, do, dht=None, chunk=64, workspace=None):
    """GDN backward over packed sequences; returns the dict of ``gdn_bwd``."""
    return _bwd_varlen(False, True, q, k, v, g, beta, cu_seqlens, h0, do, dht, chunk, workspace)


def kda_fwd_varlen(q, k, v, g, beta, cu_seqlens, h0=None, chunk=64, workspace=None):
    """KDA forward over packed sequences (``g`` is ``[1, T, H, dk]``)."""
    return _fwd_varlen(True, True, q, k, v, g, beta, cu_seqlens, h0, chunk, workspace)


def kda_bwd_varlen(q, k, v, g, beta, cu_seqlens, h0, do, dht=None, chunk=64, workspace=None):
    """KDA backward over packed sequences."""
    return _bwd_varlen(True, True, q, k, v, g, beta, cu_seqlens, h0, do, dht, chunk, workspace)


def mamba2_fwd_varlen(q, k, v, g, beta, cu_seqlens, h0=None, chunk=64, workspace=None):
    """Mamba2 forward over packed sequences."""
    return _fwd_varlen(False, False, q, k, v, g, beta, cu_seqlens, h0, chunk, workspace)


def mamba2_bwd_varlen(q, k, v, g, beta, cu_seqlens, h0, do, dht=None, chunk=64, workspace=None):
    """Mamba2 backward over packed sequences."""
    return _bwd_varlen(False, False, q, k, v, g, beta, cu_seqlens, h0, do, dht, chunk, workspace)


# ---------------------------------------------------------------- neighbours
NORM_EPS = 1e-6  # the recipe's normalisation epsilon


def _nb_check(name, x, dtype=None, device=None, shape=None):
    if not isinstance(x, torch.Tensor):
        raise GdnError(f"{name} must be a tensor")
    if x.device.type != "cuda":
        raise GdnError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if dtype is not None and x.dtype != dtype:
        raise GdnError(f"{name}: expected {dtype}, got {x.dtype}")
    if device is not None and x.device != device:
        raise GdnError(f"{name}: expected device {device}, got {x.device}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise GdnError(f"{name}: expected shape {tuple(shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise GdnError(f"{name} must be contiguous")


def _conv_args(x, w, H, cu_seqlens):
    _nb_check("x", x)
    if x.dtype not in _DTYPES or x.dim() != 3:
        raise GdnError("x must be [B, T, H*D] fp32 or bf16")
    B, T, CH = x.shape
    if H <= 0 or CH % H:
        raise GdnError(f"H={H} does not divide the {CH} channels of x")
    _nb_check("w", w, torch.float32, x.device)
    if w.dim() != 2 or w.shape[0] != CH:
        raise GdnError(f"w must be [{CH}, W] fp32")
    nseq = 0
    if cu_seqlens is not None:
        if (cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device
                or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous()):
            raise GdnError("cu_seqlens must be a contiguous 1-D int32 tensor on x's device")
        nseq = cu_seqlens.numel() - 1
    return ConvShape(B, T, H, CH // H, w.shape[1], _DTYPES[x.dtype]), nseq


def short_conv_fwd(x, w, H, l2norm=False, scale=1.0, eps=NORM_EPS, cu_seqlens=None):
    """Causal depthwise short convolution + SiLU over ``x [B, T, H*D]`` with
    ``w [H*D, W]`` fp32; with ``l2norm`` each head's D outputs of a token are
    scaled to ``scale * y / sqrt(|y|^2 + eps)`` (the q and k inputs of the
    mixer).  ``cu_seqlens`` (int32, B = 1) restarts the convolution at every
    packed sequence.  Returns ``z`` (layout and dtype of x)."""
    s, nseq = _conv_args(x, w, H, cu_seqlens)
    z = torch.empty_like(x)
    _check(lib().gdn_short_conv_fwd(ctypes.byref(s), _ptr(x), _ptr(w), _ptr(z), int(bool(l2norm)),
                                    float(scale), float(eps), _ptr(cu_seqlens), nseq,
                                    _stream(x.device)))
    return z


def short_conv_bwd(x, w, dz, H, l2norm=False, scale=1.0, eps=NORM_EPS, cu_seqlens=None,
                   workspace=None):
    """Gradients of ``short_conv_fwd``: returns ``(dx, dw)`` (dw fp32, a
    reproducible sum over the tokens)."""
    s, nseq = _conv_args(x, w, H, cu_seqlens)
    _nb_check("dz", dz, x.dtype, x.device, x.shape)
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    need = int(lib().gdn_short_conv_bwd_workspace(ctypes.byref(s)))
    ws = _workspace(need, workspace, x.device)
    _check(lib().gdn_short_conv_bwd(ctypes.byref(s), _ptr(x), _ptr(w), _ptr(dz), _ptr(dx), _ptr(dw),
                                    int(bool(l2norm)), float(scale), float(eps), _ptr(cu_seqlens),
                                    nseq, _ptr(ws), ws.numel(), _stream(x.device)))
    return dx, dw


def _norm_args(o, gate, weight):
    _nb_check("o", o)
    if o.dtype not in _DTYPES or o.dim() < 1:
        raise GdnError("o must be [..., D] fp32 or bf16")
    _nb_check("gate", gate, o.dtype, o.device, o.shape)
    D = o.shape[-1]
    _nb_check("weight", weight, torch.float32, o.device, (D,))
    return NormShape(o.numel() // D if D else 0, D, _DTYPES[o.dtype])


def gated_rmsnorm_fwd(o, gate, weight, eps=NORM_EPS):
    """``o / sqrt(mean(o^2) + eps) * weight * SiLU(gate)`` over the last
    dimension of ``o`` (e.g. the mixer output ``[B, T, H, dv]``); ``weight``
    ``[D]`` fp32.  Returns ``out`` (layout and dtype of o)."""
    s = _norm_args(o, gate, weight)
    out = torch.empty_like(o)
    _check(lib().gdn_gated_rmsnorm_fwd(ctypes.byref(s), _ptr(o), _ptr(gate), _ptr(weight), _ptr(out),
                                       float(eps), _stream(o.device)))
    return out


def gated_rmsnorm_bwd(o, gate, weight, dout, eps=NORM_EPS, workspace=None):
    """Gradients of ``gated_rmsnorm_fwd``: returns ``(do, dgate, dweight)``."""
    s = _norm_args(o, gate, weight)
    _nb_check("dout", dout, o.dtype, o.device, o.shape)
    d_o, dgate = torch.empty_like(o), torch.empty_like(gate)
    dweight = torch.empty_like(weight)
    need = int(lib().gdn_gated_rmsnorm_bwd_workspace(ctypes.byref(s)))
    ws = _workspace(need, workspace, o.device)
    _check(lib().gdn_gated_rmsnorm_bwd(ctypes.byref(s), _ptr(o), _ptr(gate), _ptr(weight), _ptr(dout),
                                       _ptr(d_o), _ptr(dgate), _ptr(dweight), float(eps), _ptr(ws),
                                       ws.numel(), _stream(o.device)))
    return d_o, dgate, dweight


def _decode(kda, q, k, v, g, beta, state=None, inplace=True, chunk=64):
    B, T, H, dk = q.shape
    dv = v.shape[3]
    _validate(q, k, v, g, beta, kda, [("state", (state, (B, H, dk, dv), torch.float32))])
    o = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    ht = state if (inplace and state is not None) else torch.empty(
        (B, H, dk, dv), dtype=torch.float32, device=q.device)
    s = make_shape(q, v, chunk, g)
    fn = lib().kda_decode if kda else lib().gdn_decode
    _check(fn(ctypes.byref(s), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
              _ptr(o), _ptr(ht), _stream(q.device)))
    return o, ht


def gdn_decode(q, k, v, g, beta, state=None, inplace=True):
    """GDN forward run token by token (decode; a few tokens per sequence).
    Returns ``(o, ht)``; with ``inplace`` (and a ``state``) the state tensor is
    updated in place and returned as ``ht``.  ``state`` None is the zero state."""
    return _decode(False, q, k, v, g, beta, state, inplace)


def kda_decode(q, k, v, g, beta, state=None, inplace=True):
    """KDA forward run token by token (``g`` is ``[B,T,H,dk]``); see ``gdn_decode``."""
    return _decode(True, q, k, v, g, beta, state, inplace)


# ---------------------------------------------------------------- attention layers
#
# Small calls are bound by the host: the checks below take one expression per
# tensor, and build their messages only when it fails.

def _same(x, dtype, device, shape):
    return (isinstance(x, torch.Tensor) and x.dtype is dtype and x.shape == shape
            and x.device == device and x.is_contiguous())


def _raw_stream(device):
    _on_current(device)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _addr(x):
    return None if x is None else x.data_ptr()


def _dense(x):
    """x, contiguous and 16-byte aligned: a gradient may be a slice of another's
    memory (of a concatenation's) that starts anywhere."""
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _call(rc):
    if rc:
        _check(rc)


def _attn_tensor(name, x, dtype, device):
    """A [B, T, H, D] tensor whose head rows are contiguous (any other strides)."""
    if not isinstance(x, torch.Tensor):
        raise GdnError(f"{name} must be a tensor")
    if x.device.type != "cuda":
        raise GdnError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if x.dim() != 4 or x.dtype is not dtype or x.device != device:
        raise GdnError(f"{name}: expected a [B, T, H, D] {dtype} tensor on {device}, got "
                       f"{tuple(x.shape)} {x.dtype} on {x.device}")
    st = x.stride()
    if x.shape[3] == 0:
        raise GdnError(f"{name}: a head has no values (D = 0)")
    if st[3] != 1 and x.shape[3] > 1:
        raise GdnError(f"{name}: the D values of a head must be contiguous")
    return st[:3]


def _attn_cu(name, cu, device):
    if (not isinstance(cu, torch.Tensor) or cu.dtype is not torch.int32 or cu.device != device
            or cu.dim() != 1 or cu.numel() < 1 or not cu.is_contiguous()):
        raise GdnError(f"{name} must be a contiguous 1-D int32 tensor on the inputs' device")


def _attn_args(q, k, v, cu_seqlens, cu_seqlens_k, scale):
    """The ABI shape and scale of a prompt call, the offsets and their number."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise GdnError("q must be a fp32 or bf16 tensor")
    dtype, device = q.dtype, q.device
    qs, ks, vs = (_attn_tensor("q", q, dtype, device), _attn_tensor("k", k, dtype, device),
                  _attn_tensor("v", v, dtype, device))
    B, Tq, H, D = q.shape
    Bk, Tk, Hkv, Dk = k.shape
    if v.shape != k.shape or Bk != B or Dk != D:
        raise GdnError(f"k and v: expected [{B}, Tk, Hkv, {D}], got {tuple(k.shape)} and "
                       f"{tuple(v.shape)}")
    if H > 0 and (Hkv == 0 or H % Hkv):
        raise GdnError(f"{Hkv} key heads do not divide the {H} query heads")
    nseq = 0
    if cu_seqlens is not None:
        _attn_cu("cu_seqlens", cu_seqlens, device)
        if cu_seqlens_k is None:
            if Tk != Tq:
                raise GdnError(f"{Tk} keys for {Tq} queries: packed keys of other lengths need "
                               "cu_seqlens_k")
            cu_seqlens_k = cu_seqlens
        else:
            _attn_cu("cu_seqlens_k", cu_seqlens_k, device)
            if cu_seqlens_k.numel() != cu_seqlens.numel():
                raise GdnError("cu_seqlens and cu_seqlens_k must have the same length")
        if B != 1:
            raise GdnError("packed sequences: the token tensors must be [1, T, H, D]")
        nseq = cu_seqlens.numel() - 1
    elif cu_seqlens_k is not None:
        raise GdnError("cu_seqlens_k needs cu_seqlens")
    s = AttnShape(B, Tq, Tk, H, Hkv, D, _DTYPES[dtype], qs, ks, vs)
    return s, D ** -0.5 if scale is None else float(scale), cu_seqlens, cu_seqlens_k, nseq


def attn_fwd(q, k, v, cu_seqlens=None, cu_seqlens_k=None, scale=None, workspace=None):
    """Causal attention of whole prompts with grouped heads: ``q [B, Tq, H, D]``,
    ``k``, ``v`` ``[B, Tk, Hkv, D]`` (views of one projection are taken as they
    are), query i of a sequence seeing the keys ``j <= i + lk - lq``.  Packed
    sequences (``B = 1``): ``cu_seqlens`` int32 device offsets of the queries,
    and ``cu_seqlens_k`` of the keys where they differ.  ``scale`` defaults to
    ``D ** -0.5``.  Returns ``(o [B, Tq, H, D], lse [B, H, Tq] fp32)``; a query
    without keys has o = 0 and lse = -inf."""
    s, scale, cu, cuk, nseq = _attn_args(q, k, v, cu_seqlens, cu_seqlens_k, scale)
    device, L, sp = q.device, lib(), ctypes.byref(s)
    o = torch.empty(q.shape, dtype=q.dtype, device=device)
    lse = torch.empty((s.B, s.H, s.Tq), dtype=torch.float32, device=device)
    need = L.gdn_attn_fwd_workspace(sp, nseq)
    ws = _workspace(need, workspace, device) if need else None
    _call(L.gdn_attn_fwd(sp, q.data_ptr(), k.data_ptr(), v.data_ptr(), scale, _addr(cu), _addr(cuk),
                         nseq, o.data_ptr(), lse.data_ptr(), _addr(ws), need, _raw_stream(device)))
    return o, lse


def attn_bwd(q, k, v, o, lse, do, cu_seqlens=None, cu_seqlens_k=None, scale=None, workspace=None):
    """Gradients of ``attn_fwd`` for the output gradient ``do``, from its inputs
    and its ``o`` and ``lse``: returns ``(dq, dk, dv)`` (contiguous)."""
    s, scale, cu, cuk, nseq = _attn_args(q, k, v, cu_seqlens, cu_seqlens_k, scale)
    dtype, device, L, sp = q.dtype, q.device, lib(), ctypes.byref(s)
    if not (_same(o, dtype, device, q.shape) and _same(do, dtype, device, q.shape)
            and _same(lse, torch.float32, device, (s.B, s.H, s.Tq))):
        _nb_check("o", o, dtype, device, q.shape)
        _nb_check("do", do, dtype, device, q.shape)
        _nb_check("lse", lse, torch.float32, device, (s.B, s.H, s.Tq))
    dq = torch.empty(q.shape, dtype=dtype, device=device)
    dk = torch.empty(k.shape, dtype=dtype, device=device)
    dv = torch.empty(k.shape, dtype=dtype, device=device)
    need = L.gdn_attn_bwd_workspace(sp, nseq)
    ws = _workspace(need, workspace, device) if need else None
    _call(L.gdn_attn_bwd(sp, q.data_ptr(), k.data_ptr(), v.data_ptr(), scale, _addr(cu), _addr(cuk),
                         nseq, o.data_ptr(), lse.data_ptr(), do.data_ptr(), dq.data_ptr(),
                         dk.data_ptr(), dv.data_ptr(), _addr(ws), need, _raw_stream(device)))
    return dq, dk, dv


def attn_decode(q, k, v, k_cache, v_cache, lens, scale=None, workspace=None):
    """Attention of T new tokens per batch row (``q [B, T, H, D]``, ``k``, ``v``
    ``[B, T, Hkv, D]``) against caches ``[B, S, Hkv, D]`` holding ``lens[b]``
    tokens (int32, on the device).  The new k and v are written to the caches'
    slots ``lens[b] ..`` and new token t sees the slots up to ``lens[b] + t``;
    ``lens`` itself is left to the caller.  Returns ``o [B, T, H, D]``."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise GdnError("q must be a fp32 or bf16 tensor")
    dtype, device = q.dtype, q.device
    _attn_tensor("q", q, dtype, device)
    kst = _attn_tensor("k_cache", k_cache, dtype, device)
    vst = _attn_tensor("v_cache", v_cache, dtype, device)
    B, T, H, D = q.shape
    Bc, S, Hkv, Dc = k_cache.shape
    if v_cache.shape != k_cache.shape or Bc != B or Dc != D:
        raise GdnError(f"the caches must be [{B}, S, Hkv, {D}], got {tuple(k_cache.shape)} and "
                       f"{tuple(v_cache.shape)}")
    if H > 0 and (Hkv == 0 or H % Hkv):
        raise GdnError(f"{Hkv} key heads do not divide the {H} query heads")
    if not q.is_contiguous():
        raise GdnError("q must be contiguous")
    new = (B, T, Hkv, D)
    if not (_same(k, dtype, device, new) and _same(v, dtype, device, new)
            and _same(lens, torch.int32, device, (B,))):
        _nb_check("k", k, dtype, device, new)
        _nb_check("v", v, dtype, device, new)
        _nb_check("lens", lens, torch.int32, device, (B,))
    s = AttnDecodeShape(B, T, S, H, Hkv, D, _DTYPES[dtype], kst, vst)
    L, sp = lib(), ctypes.byref(s)
    o = torch.empty_like(q)
    need = L.gdn_attn_decode_workspace(sp)
    ws = _workspace(need, workspace, device) if need else None
    _call(L.gdn_attn_decode(sp, q.data_ptr(), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
                            v_cache.data_ptr(), lens.data_ptr(),
                            D ** -0.5 if scale is None else float(scale), o.data_ptr(), _addr(ws),
                            need, _raw_stream(device)))
    return o


def _ln_args(x, weight):
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype in _DTYPES and x.is_contiguous()
            and x.dim() > 0 and x.shape[-1] > 0):
        _nb_check("x", x)
        raise GdnError("x must be [..., D] fp32 or bf16, D >= 1")
    D = x.shape[-1]
    if not _same(weight, torch.float32, x.device, (D,)):
        _nb_check("weight", weight, torch.float32, x.device, (D,))
    return NormShape(x.numel() // D, D, _DTYPES[x.dtype])


def layer_norm_fwd(x, weight, bias=None, eps=NORM_EPS):
    """``(x - mean) * rstd * weight + bias`` over the last dimension of ``x``
    (``weight``, ``bias`` ``[D]`` fp32).  Returns ``(y, mean, rstd)``, the
    statistics ``[...]`` in fp32 for ``layer_norm_bwd``."""
    s = _ln_args(x, weight)
    device = x.device
    if bias is not None and not _same(bias, torch.float32, device, weight.shape):
        _nb_check("bias", bias, torch.float32, device, weight.shape)
    y = torch.empty_like(x)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=device)
    rstd = torch.empty_like(mean)
    _call(lib().gdn_layer_norm_fwd(ctypes.byref(s), x.data_ptr(), weight.data_ptr(), _addr(bias),
                                   y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), float(eps),
                                   _raw_stream(device)))
    return y, mean, rstd


def layer_norm_bwd(x, weight, mean, rstd, dy, workspace=None):
    """Gradients of ``layer_norm_fwd``: returns ``(dx, dweight, dbias)`` (the last
    two fp32, reproducible sums over the rows)."""
    s = _ln_args(x, weight)
    device, lead, L, sp = x.device, x.shape[:-1], lib(), ctypes.byref(s)
    if not (_same(dy, x.dtype, device, x.shape) and _same(mean, torch.float32, device, lead)
            and _same(rstd, torch.float32, device, lead)):
        _nb_check("dy", dy, x.dtype, device, x.shape)
        _nb_check("mean", mean, torch.float32, device, lead)
        _nb_check("rstd", rstd, torch.float32, device, lead)
    dx = torch.empty_like(x)
    dweight, dbias = torch.empty_like(weight), torch.empty_like(weight)
    ws = _workspace(L.gdn_layer_norm_bwd_workspace(sp), workspace, device)
    _call(L.gdn_layer_norm_bwd(sp, x.data_ptr(), weight.data_ptr(), mean.data_ptr(),
                               rstd.data_ptr(), dy.data_ptr(), dx.data_ptr(), dweight.data_ptr(),
                               dbias.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(device)))
    return dx, dweight, dbias


# ---------------------------------------------------------------- positions and pages

def rope_table(n, R, base=10000.0, device="cuda"):
    """``(cos, sin)`` fp32 ``[n, R / 2]`` of the angles ``position * base ** (-2 i / R)``,
    made in 64 bits (an fp32 angle of a far position is off by more than its cosine
    may be).  Any other tables of that shape serve as well."""
    if R < 0 or R % 2:
        raise GdnError(f"R = {R}: an even number of rotated values")
    f = float(base) ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / max(R, 1))
    angle = torch.arange(n, dtype=torch.float64, device=device)[:, None] * f
    return angle.cos().float(), angle.sin().float()


# A decode step calls these once per layer with little for the GPU to do, so their
# checks are few expressions on what every call has, and build their messages only
# when one fails; shapes go to the library as packed bytes.
_QK_ROPE = struct.Struct("@9i6q")      # gdn_qk_rope_shape
_CACHE = struct.Struct("@5i4P12q")     # gdn_paged_cache
_APPEND = struct.Struct("@9i10q")      # gdn_kv_append_shape
_PAGED = struct.Struct("@5iq")         # gdn_attn_paged_shape
_MOST = 1 << 30                        # tokens, rows and pages of a row that the library takes


def _pack(form, *values):
    try:
        return form.pack(*values)
    except struct.error:
        raise GdnError(f"a size of the call does not fit the library's integers: {values}") from None


def _f32(name, x, device, shape):
    if not _same(x, torch.float32, device, shape):
        _nb_check(name, x, torch.float32, device, shape)


def _i32(name, x, device, shape):
    if not _same(x, torch.int32, device, shape):
        _nb_check(name, x, torch.int32, device, shape)


def _empty(x, dtype, device):
    """A contiguous tensor of x's shape."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=dtype, device=device)


def _heads(name, x, dtype, device):
    """x's strides, a [B, T, H, D] tensor whose head rows are contiguous."""
    st = x.stride() if isinstance(x, torch.Tensor) else ()
    if len(st) == 4 and st[3] == 1 and x.dtype is dtype and x.device == device and x.is_cuda and x.shape[3] > 0:
        return st
    _attn_tensor(name, x, dtype, device)
    return st


def _tables(cos, sin, D, device):
    """R and P of the tables (0, 0: none)."""
    if cos is None and sin is None:
        return 0, 0
    if not isinstance(cos, torch.Tensor) or not isinstance(sin, torch.Tensor) or cos.dim() != 2:
        raise GdnError("cos and sin must be fp32 tables [positions, R / 2], both or neither")
    _f32("cos", cos, device, cos.shape)
    _f32("sin", sin, device, cos.shape)
    P, half = cos.shape
    if not 0 < 2 * half <= D:
        raise GdnError(f"tables of {half} pairs for heads of {D} values")
    return 2 * half, P


def _table_ok(cos, sin, D, device):
    """Whether the angles are tables that a call takes (most calls' case, in one look)."""
    shape = cos.shape
    return (len(shape) == 2 and 0 < 2 * shape[1] <= D and cos.dtype is torch.float32
            and sin.dtype is torch.float32 and sin.shape == shape and cos.device == device
            and sin.device == device and cos.is_contiguous() and sin.is_contiguous())


def _qk_args(q, k, q_weight, k_weight, cos, sin, positions, interleaved):
    """The ABI shape of a call, packed.  First the looks that every good call passes,
    then, if one did not, the slow ones that say why."""
    try:
        dtype, device, qs, ks = q.dtype, q.device, q.stride(), k.stride()
        B, T, H, D = q.shape
        Bk, Tk, Hkv, Dk = k.shape
        half = cos.shape[1]
        if (k.dtype is dtype and k.device == device and q.is_cuda and Bk == B and Tk == T and Dk == D
                and qs[3] == 1 and ks[3] == 1 and _table_ok(cos, sin, D, device)
                and (positions is None or (positions.dtype is torch.int32 and positions.shape == (B, T)
                                           and positions.device == device and positions.is_contiguous()))
                and (q_weight is k_weight is None
                     or (q_weight.dtype is torch.float32 and k_weight.dtype is torch.float32
                         and q_weight.shape == (D,) and k_weight.shape == (D,)
                         and q_weight.device == device and k_weight.device == device
                         and q_weight.is_contiguous() and k_weight.is_contiguous()))):
            return _QK_ROPE.pack(B, T, H, Hkv, D, 2 * half, cos.shape[0], bool(interleaved),
                                 _DTYPES[dtype], qs[0], qs[1], qs[2], ks[0], ks[1], ks[2])
    except (AttributeError, KeyError, TypeError, ValueError, IndexError, struct.error):
        pass
    return _qk_args_slow(q, k, q_weight, k_weight, cos, sin, positions, interleaved)


def _qk_args_slow(q, k, q_weight, k_weight, cos, sin, positions, interleaved):
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise GdnError("q must be a fp32 or bf16 tensor")
    dtype, device = q.dtype, q.device
    qs, ks = _heads("q", q, dtype, device), _heads("k", k, dtype, device)
    B, T, H, D = q.shape
    Bk, Tk, Hkv, Dk = k.shape
    if Bk != B or Tk != T or Dk != D:
        raise GdnError(f"k: expected [{B}, {T}, Hkv, {D}], got {tuple(k.shape)}")
    if (q_weight is None) != (k_weight is None):
        raise GdnError("q_weight and k_weight: both or neither")
    if q_weight is not None:
        _f32("q_weight", q_weight, device, (D,))
        _f32("k_weight", k_weight, device, (D,))
    R, P = _tables(cos, sin, D, device)
    if R == 0 and q_weight is None:
        raise GdnError("neither weights nor tables: nothing to do")
    if positions is not None:
        if R == 0:
            raise GdnError("positions need cos and sin")
        _i32("positions", positions, device, (B, T))
    return _pack(_QK_ROPE, B, T, H, Hkv, D, R, P, bool(interleaved), _DTYPES[dtype], qs[0], qs[1], qs[2],
                 ks[0], ks[1], ks[2])


def qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                     interleaved=False, eps=NORM_EPS):
    """RMS norm of every head of ``q [B, T, H, D]`` and ``k [B, T, Hkv, D]`` (views of
    one projection are taken as they are) with weights ``[D]`` fp32, then rotation of
    its first R values by position: ``cos``, ``sin`` ``[P, R / 2]`` fp32 (see
    ``rope_table``), ``positions`` int32 ``[B, T]`` (default: token t has position t; a
    token with a negative one is not in use and gets zeros).  Pairs are ``(i, i + R / 2)``, or ``(2 i, 2 i + 1)`` with ``interleaved``.  Weights
    or tables may be left out.  Returns ``(qo, ko)``, contiguous."""
    s = _qk_args(q, k, q_weight, k_weight, cos, sin, positions, interleaved)
    dtype, device = q.dtype, q.device
    qo, ko = _empty(q, dtype, device), _empty(k, dtype, device)
    _call((_lib or lib()).gdn_qk_norm_rope_fwd(
        s, q.data_ptr(), k.data_ptr(), _addr(q_weight), _addr(k_weight), float(eps), _addr(cos),
        _addr(sin), _addr(positions), qo.data_ptr(), ko.data_ptr(), _raw_stream(device)))
    return qo, ko


def qk_norm_rope_bwd(q, k, dqo, dko, q_weight=None, k_weight=None, cos=None, sin=None,
                     positions=None, interleaved=False, eps=NORM_EPS, workspace=None):
    """Gradients of ``qk_norm_rope_fwd`` from its inputs and those of its outputs:
    returns ``(dq, dk, dq_weight, dk_weight)`` (contiguous; the last two fp32,
    reproducible sums over all tokens and heads, None without weights)."""
    s = _qk_args(q, k, q_weight, k_weight, cos, sin, positions, interleaved)
    dtype, device, L = q.dtype, q.device, _lib or lib()
    if not (_same(dqo, dtype, device, q.shape) and _same(dko, dtype, device, k.shape)):
        _nb_check("dqo", dqo, dtype, device, q.shape)
        _nb_check("dko", dko, dtype, device, k.shape)
    dq, dk = torch.empty_like(dqo), torch.empty_like(dko)
    dwq = dwk = ws = None
    need = 0
    if q_weight is not None:
        dwq, dwk = torch.empty_like(q_weight), torch.empty_like(k_weight)
        need = L.gdn_qk_norm_rope_bwd_workspace(s)
        ws = _workspace(need, workspace, device)
    _call(L.gdn_qk_norm_rope_bwd(
        s, q.data_ptr(), k.data_ptr(), _addr(q_weight), _addr(k_weight), float(eps), _addr(cos),
        _addr(sin), _addr(positions), dqo.data_ptr(), dko.data_ptr(), dq.data_ptr(), dk.data_ptr(),
        _addr(dwq), _addr(dwk), _addr(ws), need, _raw_stream(device)))
    return dq, dk, dwq, dwk


class PagedCache(NamedTuple):
    """Pages of keys and values: ``k``, ``v`` ``[pages, page, Hkv, D]`` in fp32 or bf16,
    or in 4 bits, codes ``[pages, page, Hkv, D / 2]`` uint8 and the steps of every 32
    values ``[pages, page, Hkv, D / 32]`` bf16 (see gdn.h).  The calls take any tuple of
    these two or four tensors, with any strides between tokens, heads and pages."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def new_paged_cache(pages, page, Hkv, D, dtype=torch.bfloat16, bits=None, device="cuda"):
    """An empty cache of ``pages`` pages of ``page`` tokens (a power of two), in
    ``dtype`` or with ``bits=4`` in 4 bits.  A page's tokens of one head lie together
    in memory, which is how attention reads them."""
    if bits not in (None, 4):
        raise GdnError(f"bits = {bits}: None (the dtype's own) or 4")
    if page < 1 or page & (page - 1):
        raise GdnError(f"a page of {page} tokens: not a power of two")
    if dtype not in _DTYPES:
        raise GdnError(f"unsupported dtype {dtype}")

    def make(n, dt):
        return torch.zeros(pages, Hkv, page, n, dtype=dt, device=device).transpose(1, 2)
    if bits is None:
        return PagedCache(make(D, dtype), make(D, dtype))
    if D % 32:
        raise GdnError(f"4 bits: heads of {D} values are no multiple of 32")
    return PagedCache(make(D // 2, torch.uint8), make(D // 2, torch.uint8),
                      make(D // 32, torch.bfloat16), make(D // 32, torch.bfloat16))


def _cache_args(cache, device):
    """The ABI's view of a cache (packed), and its heads, values per head and format."""
    try:
        k, v = cache[0], cache[1]
        shape, dtype, a, b = k.shape, k.dtype, k.stride(), v.stride()
        pages, page, Hkv, D = shape
        if (v.shape == shape and v.dtype is dtype and k.device == device and v.device == device
                and a[3] == 1 and b[3] == 1 and D > 0):
            if dtype is torch.uint8:
                ks, vs = cache[2], cache[3]
                c, d, steps = ks.stride(), vs.stride(), (pages, page, Hkv, D // 16)
                if (len(cache) == 4 and D % 16 == 0 and ks.dtype is torch.bfloat16
                        and vs.dtype is torch.bfloat16 and ks.shape == steps and vs.shape == steps
                        and ks.device == device and vs.device == device and c[3] == 1 and d[3] == 1):
                    return _CACHE.pack(pages, page, Hkv, 2 * D, 2, k.data_ptr(), v.data_ptr(),
                                       ks.data_ptr(), vs.data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2],
                                       c[0], c[1], c[2], d[0], d[1], d[2]), Hkv, 2 * D, 2
            elif len(cache) == 2:
                form = _DTYPES[dtype]
                return _CACHE.pack(pages, page, Hkv, D, form, k.data_ptr(), v.data_ptr(), 0, 0, a[0],
                                   a[1], a[2], b[0], b[1], b[2], 0, 0, 0, 0, 0, 0), Hkv, D, form
    except (AttributeError, KeyError, TypeError, ValueError, IndexError, struct.error):
        pass
    return _cache_args_slow(cache, device)


def _cache_args_slow(cache, device):
    n = 4 if len(cache) == 4 and cache[2] is not None else 2
    if n == 2 and any(x is not None for x in cache[2:]) or len(cache) < 2 or len(cache) > 4:
        raise GdnError("the cache must be (k, v) or (k, v, k_scale, v_scale)")
    for x in cache[:n]:
        if not isinstance(x, torch.Tensor) or x.dim() != 4 or x.device != device:
            raise GdnError(f"the cache must be [pages, page, Hkv, .] tensors on {device}, "
                           f"(k, v) or (k, v, k_scale, v_scale)")
    k, v = cache[0], cache[1]
    shape, dtype, kst, vst = k.shape, k.dtype, k.stride(), v.stride()
    if v.shape != shape or v.dtype is not dtype:
        raise GdnError(f"the cache's k and v differ: {tuple(shape)} {dtype}, {tuple(v.shape)} {v.dtype}")
    pages, page, Hkv, D = shape
    if D == 0:
        raise GdnError("the cache's heads have no values (D = 0)")
    if (kst[3] != 1 or vst[3] != 1) and D > 1:
        raise GdnError("the values of a head must be contiguous in the cache")
    if n == 2:
        if dtype not in _DTYPES:
            raise GdnError(f"a cache of {dtype}: fp32, bf16, or uint8 codes with scales")
        form = _DTYPES[dtype]
        return _pack(_CACHE, pages, page, Hkv, D, form, k.data_ptr(), v.data_ptr(), 0, 0, *kst[:3],
                     *vst[:3], 0, 0, 0, 0, 0, 0), Hkv, D, form
    ks, vs = cache[2], cache[3]
    steps = (pages, page, Hkv, D // 16)
    if (dtype is not torch.uint8 or D % 16 or ks.dtype is not torch.bfloat16
            or vs.dtype is not torch.bfloat16 or ks.shape != steps or vs.shape != steps):
        raise GdnError(f"a 4-bit cache: uint8 codes [pages, page, Hkv, D / 2] and bf16 scales [pages, page, "
                       f"Hkv, D / 32], D a multiple of 32, got {[(tuple(x.shape), x.dtype) for x in cache]}")
    kss, vss = ks.stride(), vs.stride()
    if (kss[3] != 1 or vss[3] != 1) and steps[3] > 1:
        raise GdnError("the scales of a head must be contiguous in the cache")
    return _pack(_CACHE, pages, page, Hkv, 2 * D, 2, k.data_ptr(), v.data_ptr(), ks.data_ptr(),
                 vs.data_ptr(), *kst[:3], *vst[:3], *kss[:3], *vss[:3]), Hkv, 2 * D, 2


def _block_table(table, rows, device):
    """Entries per row of a block table, and its row stride."""
    if (not isinstance(table, torch.Tensor) or table.dtype is not torch.int32 or table.dim() != 2
            or table.device != device or table.shape[0] != rows
            or (table.stride(1) != 1 and table.shape[1] > 1)):
        raise GdnError(f"block_table must be int32 [{rows}, max_pages] on {device}, the entries of a row "
                       "contiguous")
    return table.shape[1], table.stride(0)


_NO_STRIDES = (0, 0, 0)


def _append_args(k, v, cache, block_table, lens, q, cos, sin, cu_seqlens):
    if not isinstance(k, torch.Tensor) or k.dtype not in _DTYPES:
        raise GdnError("k must be a fp32 or bf16 tensor")
    dtype, device = k.dtype, k.device
    kst, vst = _heads("k", k, dtype, device), _heads("v", v, dtype, device)
    shape = k.shape
    B, T, Hkv, D = shape
    if v.shape != shape:
        raise GdnError(f"k and v differ: {tuple(shape)}, {tuple(v.shape)}")
    H, qst = 0, _NO_STRIDES
    if q is not None:
        qst = _heads("q", q, dtype, device)
        Bq, Tq, H, Dq = q.shape
        if Bq != B or Tq != T or Dq != D:
            raise GdnError(f"q: expected [{B}, {T}, H, {D}], got {tuple(q.shape)}")
    c, heads, values, form = _cache_args(cache, device)
    if heads != Hkv or values != D or form not in (2, _DTYPES[dtype]):
        raise GdnError(f"the cache holds {heads} heads of {values} values ({cache[0].dtype}), k is "
                       f"{tuple(shape)} {dtype}")
    R, P = _tables(cos, sin, D, device)
    rows = B
    if cu_seqlens is not None:
        _attn_cu("cu_seqlens", cu_seqlens, device)
        if B != 1:
            raise GdnError("packed sequences: the token tensors must be [1, T, H, D]")
        rows = cu_seqlens.numel() - 1
    _i32("lens", lens, device, (rows,))
    most, stride = _block_table(block_table, rows, device)
    return c, B, T, H, R, P, _DTYPES[dtype], rows, most, stride, qst, kst, vst


def kv_append(k, v, cache, block_table, lens, q=None, cos=None, sin=None, interleaved=False,
              cu_seqlens=None):
    """Stores new keys and values ``[B, T, Hkv, D]`` in a paged cache: token t of row b
    in slot ``lens[b] + t`` (``lens`` int32, on the device, left to the caller), which
    is place ``slot % page`` of page ``block_table[b, slot // page]`` (int32).  With
    ``cos``, ``sin`` (see ``qk_norm_rope_fwd``) k is rotated by its slot on the way,
    and so is ``q [B, T, H, D]``, if given; returns the rotated q, or None.

    Packed new tokens: ``k``, ``v``, ``q`` ``[1, T, ...]`` and ``cu_seqlens`` int32
    ``[rows + 1]``; tokens behind ``cu_seqlens[-1]`` belong to no row.  A row whose
    ``lens`` is negative is not in use: its tokens are not stored, and their q is 0."""
    rows = None
    try:  # the looks that every good call passes
        dtype, device, kst, vst = k.dtype, k.device, k.stride(), v.stride()
        shape = k.shape
        B, T, Hkv, D = shape
        H, qst, R, P = 0, _NO_STRIDES, 0, 0
        good = (v.shape == shape and v.dtype is dtype and v.device == device and k.is_cuda
                and kst[3] == 1 and vst[3] == 1)
        if q is not None:
            Bq, Tq, H, Dq = q.shape
            qst = q.stride()
            good = (good and q.dtype is dtype and q.device == device and Bq == B and Tq == T and Dq == D
                    and qst[3] == 1)
        if cos is not None or sin is not None:
            good = good and _table_ok(cos, sin, D, device)
            P, R = cos.shape[0], 2 * cos.shape[1]
        if good and cu_seqlens is None:
            c, heads, values, form = _cache_args(cache, device)
            most, stride = _block_table(block_table, B, device)
            if (heads == Hkv and values == D and (form == 2 or form == _DTYPES[dtype])
                    and lens.dtype is torch.int32 and lens.shape == (B,) and lens.device == device
                    and lens.is_contiguous()):
                rows, code = B, _DTYPES[dtype]
    except (AttributeError, KeyError, TypeError, ValueError, IndexError):
        pass
    if rows is None:  # packed tokens, or a call that one of these says no to
        c, B, T, H, R, P, code, rows, most, stride, qst, kst, vst = _append_args(
            k, v, cache, block_table, lens, q, cos, sin, cu_seqlens)
        dtype, device = k.dtype, k.device
    s = _pack(_APPEND, B, T, H, R, P, bool(interleaved), code, rows, most, stride, qst[0], qst[1], qst[2],
              kst[0], kst[1], kst[2], vst[0], vst[1], vst[2])
    qo = None if q is None else _empty(q, dtype, device)
    _call((_lib or lib()).gdn_kv_append(
        s, c, k.data_ptr(), v.data_ptr(), _addr(q), _addr(cos), _addr(sin), block_table.data_ptr(),
        lens.data_ptr(), _addr(cu_seqlens), _addr(qo), _raw_stream(device)))
    return qo


def kv_gather(cache, block_table, cu_seqlens, total, dtype=None):
    """Reads rows of a paged cache back as packed ``k``, ``v`` ``[1, total, Hkv, D]``,
    as ``attn_fwd`` takes them with ``cu_seqlens_k``: the first ``cu_seqlens[b + 1] -
    cu_seqlens[b]`` tokens of row b.  ``total`` is ``cu_seqlens[-1]``, known to the
    host.  ``dtype`` is the cache's own; a 4-bit cache gives bf16 (exact) or fp32."""
    device = cache[0].device
    if device.type != "cuda":
        raise GdnError("the cache must be CUDA tensors (the library has no CPU path)")
    c, Hkv, D, form = _cache_args(cache, device)
    if dtype is None:
        dtype = torch.bfloat16 if form == 2 else cache[0].dtype
    if dtype not in _DTYPES or form not in (2, _DTYPES[dtype]):
        raise GdnError(f"a cache of {cache[0].dtype} does not give {dtype}")
    _attn_cu("cu_seqlens", cu_seqlens, device)
    rows = cu_seqlens.numel() - 1
    most, stride = _block_table(block_table, rows, device)
    if total < 0 or max(total, rows, most) > _MOST:
        raise GdnError(f"{total} tokens of {rows} rows of {most} pages: at most {_MOST}")
    k = torch.empty((1, total, Hkv, D), dtype=dtype, device=device)
    v = torch.empty_like(k)
    _call((_lib or lib()).gdn_kv_gather(
        c, block_table.data_ptr(), rows, most, stride, cu_seqlens.data_ptr(), total, _DTYPES[dtype],
        k.data_ptr(), v.data_ptr(), _raw_stream(device)))
    return k, v


def attn_paged(q, cache, block_table, lens, scale=None, workspace=None):
    """Attention of T new tokens per row, ``q [B, T, H, D]``, against a paged cache
    that holds them already (``kv_append`` with the same ``lens``, the tokens before
    the new ones): token t sees the slots up to ``lens[b] + t``.  ``scale`` defaults
    to ``D ** -0.5``.  A row whose ``lens`` is negative is not in use and gets 0.
    Returns ``o [B, T, H, D]``."""
    if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPES:
        raise GdnError("q must be a fp32 or bf16 tensor")
    dtype, device = q.dtype, q.device
    _heads("q", q, dtype, device)
    if not q.is_contiguous():
        raise GdnError("q must be contiguous")
    B, T, H, D = q.shape
    c, Hkv, values, form = _cache_args(cache, device)
    if values != D or form not in (2, _DTYPES[dtype]):
        raise GdnError(f"the cache holds heads of {values} values ({cache[0].dtype}), q is {tuple(q.shape)} {dtype}")
    if H > 0 and (Hkv == 0 or H % Hkv):
        raise GdnError(f"{Hkv} key heads do not divide the {H} query heads")
    _i32("lens", lens, device, (B,))
    most, stride = _block_table(block_table, B, device)
    s = _pack(_PAGED, B, T, H, _DTYPES[dtype], most, stride)
    L = _lib or lib()
    o = torch.empty_like(q)
    need = L.gdn_attn_paged_workspace(s, c)
    ws = _workspace(need, workspace, device) if need else None
    _call(L.gdn_attn_paged(s, c, q.data_ptr(), block_table.data_ptr(), lens.data_ptr(),
                           D ** -0.5 if scale is None else float(scale), o.data_ptr(), _addr(ws), need,
                           _raw_stream(device)))
    return o


class Attention(torch.autograd.Function):
    """Autograd wrapper of ``attn_fwd`` / ``attn_bwd``."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, cu_seqlens_k, scale):
        o, lse = attn_fwd(q, k, v, cu_seqlens, cu_seqlens_k, scale)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, cu_seqlens_k)
        ctx.scale = scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu, cuk = ctx.saved_tensors
        return (*attn_bwd(q, k, v, o, lse, _dense(do), cu, cuk, ctx.scale), None, None, None)


def attention(q, k, v, cu_seqlens=None, cu_seqlens_k=None, scale=None):
    """Differentiable ``attn_fwd``: returns ``o``."""
    return Attention.apply(q, k, v, cu_seqlens, cu_seqlens_k, scale)


class QkNormRope(torch.autograd.Function):
    """Autograd wrapper of ``qk_norm_rope_fwd`` / ``qk_norm_rope_bwd``."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.interleaved, ctx.eps = interleaved, eps
        return qk_norm_rope_fwd(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko):
        q, k, wq, wk, cos, sin, positions = ctx.saved_tensors
        return (*qk_norm_rope_bwd(q, k, _dense(dqo), _dense(dko), wq, wk, cos, sin, positions,
                                  ctx.interleaved, ctx.eps), None, None, None, None, None)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None,
                 interleaved=False, eps=NORM_EPS):
    """Differentiable ``qk_norm_rope_fwd`` (in q, k and the weights): returns ``(qo, ko)``."""
    return QkNormRope.apply(q, k, q_weight, k_weight, cos, sin, positions, interleaved, eps)


class LayerNorm(torch.autograd.Function):
    """Autograd wrapper of ``layer_norm_fwd`` / ``layer_norm_bwd``."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = _dense(x)
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layer_norm_bwd(x, weight, mean, rstd, _dense(dy))
        return dx, dw, db if ctx.has_bias else None, None


def layer_norm(x, weight, bias=None, eps=NORM_EPS):
    """Differentiable ``layer_norm_fwd``: returns ``y``."""
    return LayerNorm.apply(x, weight, bias, eps)


def wait_selftest(max_tries=5):
    """Runs the device-side timeout path once (see gdn_wait_selftest in gdn.h)."""
    _check(lib().gdn_wait_selftest(max_tries, _stream(torch.device("cuda", torch.cuda.current_device()))))


def attn_wait_selftest(clocks=1 << 22):
    """The same for the attention kernels' waits (see gdn_attn_wait_selftest in gdn.h)."""
    _check(lib().gdn_attn_wait_selftest(clocks, _stream(torch.device("cuda", torch.cuda.current_device()))))


def device_status() -> int:
    """Reads and clears the device status word (0 = OK, else a ``gdn_status``: a
    wait that timed out, bad sequence offsets)."""
    return int(lib().gdn_device_status())


class KernelTimer:
    """Times every kernel the library launches from this thread with CUDA
    events recorded on the launch stream (the ABI's gdn_profile_* hook).

    ``with KernelTimer(cap) as t: ...`` then ``t.records()`` gives a list of
    ``(kernel_name, ms)`` in launch order and ``t.launches`` the launch count."""

    def __init__(self, cap=4096):
        self.cap = cap
        self.launches = 0

    def __enter__(self):
        _check(lib().gdn_profile_begin(self.cap))
        return self

    def __exit__(self, *exc):
        self.launches = int(lib().gdn_profile_end())
        return False

    def records(self):
        ids = (ctypes.c_int * self.cap)()
        ms = (ctypes.c_float * self.cap)()
        n = lib().gdn_profile_read(ids, ms, self.cap)
        if n < 0:
            _check(n)
        return [(lib().gdn_kernel_name(ids[i]).decode(), float(ms[i])) for i in range(n)]


class GatedDeltaRule(torch.autograd.Function):
    """Autograd wrapper: forward via ``*_fwd`` (``*_fwd_save`` with
    ``save_context``), backward via ``*_bwd`` (``*_bwd_saved``).  The inputs
    are saved; with ``save_context`` the forward also keeps the per-chunk
    entry states and solve results (``ctx_bytes``) instead of the backward
    recomputing them."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0, chunk, kda, save_context, delta=True):
        saved = new_ctx(q, v, chunk, kda, delta) if save_context else None
        o, ht = _fwd(kda, q, k, v, g, beta, h0, chunk, True, ctx=saved, delta=delta)
        ctx.save_for_backward(q, k, v, g, beta, h0)
        ctx.chunk, ctx.kda, ctx.saved, ctx.delta = chunk, kda, saved, delta
        return o, ht

    @staticmethod
    def backward(ctx, do, dht):
        q, k, v, g, beta, h0 = ctx.saved_tensors
        gr = _bwd(ctx.kda, q, k, v, g, beta, h0, _dense(do),
                  None if dht is None else _dense(dht), ctx.chunk, h0 is not None,
                  ctx=ctx.saved, delta=ctx.delta)
        ctx.saved = None
        return (gr["dq"], gr["dk"], gr["dv"], gr["dg"], gr["dbeta"], gr["dh0"], None, None,
                None, None)


def gated_delta_rule(q, k, v, g, beta, h0=None, chunk=64, kda=False, save_context=True,
                     delta=True):
    """Differentiable mixer: returns ``(o, final_state)``.  ``save_context``
    trades ``ctx_bytes`` of device memory per call for a faster backward;
    ``delta=False`` selects the Mamba2 mixer (no delta rule, scalar gate)."""
    _mixer(kda, delta)
    return GatedDeltaRule.apply(q, k, v, g, beta, h0, chunk, kda, save_context, delta)
