"""Python binding of libfp4 (block-scaled FP4 on MI355X / gfx950).

Argument marshalling only: every function checks that each tensor has the
dtype, device and layout the C side reads it with, passes device pointers,
sizes and the current HIP stream to the C ABI declared in include/fp4.h, and
raises on a non-zero status.  All computation happens in the library's HIP kernels; there
is no fallback.  Tensors are torch tensors used as device memory.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import NamedTuple

import torch

__all__ = [
    "lib", "Fp4Error", "FMT_MX", "FMT_NV", "DT_BF16", "DT_F32",
    "fp4_quantize_mx", "fp4_quantize_nv", "fp4_quantize_nv_workspace_bytes", "fp4_quantize_nv_noalloc", "fp4_remap_mx_to_nv",
    "fp4_scale_max_workspace_bytes",
    "fp4_dequant", "fp4_gemm", "fp4_quantize_mxfp8", "fp4_mx_to_mxfp8", "fp4_mx_dequant_fp8", "fp4_gemm_w4a8", "fp4_fake_quant",
    "fp4_ste_backward", "fp4_kv_append_mx", "fp4_moe_grouped_gemm", "fp4_moe_workspace_bytes", "MoeDebug",
    "fp4_qk_norm_rope", "KvCache", "KvPages", "fp4_kv_reserve", "fp4_kv_reserve_workspace_bytes", "fp4_kv_fork",
    "fp4_kv_free", "fp4_kv_compact", "fp4_kv_copy_pages", "fp4_attn_tree_mx", "fp4_attn_tree_workspace_bytes",
    "fp4_attn_prompt",
    "fp4_abi_version", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp4.so")
FMT_MX, FMT_NV = 0, 1
DT_BF16, DT_F32 = 0, 1

_c = ctypes
_vp, _i64, _i32, _sz = _c.c_void_p, _c.c_int64, _c.c_int, _c.c_size_t


class MoeDebug(_c.Structure):
    """Mirror of struct fp4_moe_debug (all members nullable device pointers)."""
    _fields_ = [("x_codes", _vp), ("x_scales", _vp), ("counts", _vp), ("offsets", _vp), ("perm", _vp), ("gate_up", _vp),
                ("h_bf16", _vp), ("h_codes", _vp), ("h_scales", _vp), ("y", _vp),
                ("gate_up_in", _vp), ("h_codes_in", _vp), ("h_scales_in", _vp), ("stage_events", _vp * 6)]


# struct fp4_kv_cache (k_codes, k_scales, v_codes, v_scales, num_pages, d, page_size) and
# struct fp4_kv_pages (page_table, page_counts, seq_lens, page_refs, batch, max_pages,
# num_pages): four pointers and three int64, passed as bytes.
_pack_kv = struct.Struct("=4Q3q").pack


_SIGS = {
    "fp4_abi_version": (_i32, []),
    "fp4_status_string": (_c.c_char_p, [_i32]),
    "fp4_last_error": (_c.c_char_p, []),
    "fp4_quantize_mx": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "fp4_quantize_nv": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _sz, _vp]),
    "fp4_quantize_nv_workspace_bytes": (_sz, [_i64, _i64]),
    "fp4_quantize_nv_noalloc": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp]),
    "fp4_remap_mx_to_nv": (_i32, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fp4_scale_max_workspace_bytes": (_sz, [_i64, _i64]),
    "fp4_dequant": (_i32, [_i32, _vp, _vp, _vp, _i64, _i64, _vp, _i32, _i64, _vp]),
    "fp4_gemm": (_i32, [_i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _i64, _vp]),
    "fp4_kv_append_mx": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "fp4_fake_quant": (_i32, [_i32, _vp, _i64, _i64, _i64, _vp, _i32, _i64, _vp, _i32, _vp, _sz, _vp]),
    "fp4_ste_backward": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _i32, _vp]),
    "fp4_quantize_mxfp8": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "fp4_mx_to_mxfp8": (_i32, [_vp, _i64, _i64, _vp, _vp]),
    "fp4_mx_dequant_fp8": (_i32, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "fp4_gemm_w4a8": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32, _i64, _vp]),
    "fp4_moe_grouped_gemm": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i64, _vp, _vp, _vp,
                                     _vp, _vp, _vp, _vp, _vp, _vp, _sz, _c.POINTER(MoeDebug), _vp]),
    "fp4_moe_workspace_bytes": (_sz, [_i32, _i64, _i64, _i32, _i32, _i64]),
    "fp4_qk_norm_rope": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _i64, _i64, _vp, _vp, _i32, _c.c_float, _vp, _i64, _i32,
                                _i32, _vp, _vp, _i64, _vp, _i64, _vp]),
    "fp4_kv_reserve": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]),
    "fp4_kv_reserve_workspace_bytes": (_sz, [_i64, _i64]),
    "fp4_kv_fork": (_i32, [_vp, _vp, _i64, _i64, _vp]),
    "fp4_kv_free": (_i32, [_vp, _vp, _i64, _vp, _i64, _vp]),
    "fp4_kv_compact": (_i32, [_vp, _vp, _vp, _i64, _vp, _vp]),
    "fp4_kv_copy_pages": (_i32, [_vp, _vp, _vp, _vp, _i64, _vp]),
    "fp4_attn_tree_mx": (_i32, [_vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _c.c_float, _vp,
                                _i64, _vp, _sz, _vp]),
    "fp4_attn_tree_workspace_bytes": (_sz, [_i64, _i32, _i32, _i32, _i32]),
    "fp4_attn_prompt": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _i64, _i64, _i64, _c.c_float, _vp, _i64,
                               _vp]),
}


ABI_VERSION = 2          # the signatures below


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    h = _c.CDLL(LIB_PATH)
    h.fp4_abi_version.restype = _i32
    if h.fp4_abi_version() != ABI_VERSION:
        raise ImportError(f"{LIB_PATH} has ABI version {h.fp4_abi_version()}, this binding needs {ABI_VERSION}: "
                          "rebuild it")
    for name, (res, args) in _SIGS.items():
        f = getattr(h, name)
        f.restype, f.argtypes = res, args
    return h


lib = _load()


class Fp4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = lib.fp4_last_error().decode() or lib.fp4_status_string(status).decode()
        super().__init__(f"{fn} failed with status {status} ({lib.fp4_status_string(status).decode()}): {msg}")


def _ptr(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


_U8, _I32, _I64, _F32, _BF16 = (torch.uint8,), (torch.int32,), (torch.int64,), (torch.float32,), (torch.bfloat16,)
_OUT = (torch.bfloat16, torch.float32)


class _Args:
    """Collects a call's tensor arguments and rejects what the C side would
    misread: a non-tensor, another dtype, elements not contiguous along the
    last axis, gaps between rows (dense=True: arguments without a
    leading-dimension parameter), then a tensor not on the GPU.  Dtype and
    layout are checked for every argument before any device check."""

    __slots__ = ("fn", "items")

    def __init__(self, fn):
        self.fn, self.items = fn, []

    def __call__(self, name, t, dtypes, dense=True, optional=False):
        if t is None and optional:
            return self
        fn = self.fn
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a torch tensor, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{fn}: {name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
        if not t.is_contiguous() and t.numel():
            if t.dim() and t.size(-1) > 1 and t.stride(-1) != 1:
                raise ValueError(f"{fn}: {name} must be contiguous along its last axis")
            if dense:
                raise ValueError(f"{fn}: {name} must be contiguous")
        self.items.append((name, t))
        return self

    def on_device(self):
        for name, t in self.items:
            if t.device.type != "cuda":
                raise ValueError(f"{self.fn}: {name} must be on the GPU, got a {t.device.type} tensor")


def _check_all(fn, tensors):
    """Checks (name, tensor, dtypes, dense) of a call as _Args does, in one pass.
    Returns the GPU that all of them are on, or -1 (which _go reports, so that a
    caller's own checks come before any device check)."""
    dev = tensors[0][1].get_device() if isinstance(tensors[0][1], torch.Tensor) else -1
    for name, t, dtypes, dense in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{fn}: {name} must be a torch tensor, got {type(t).__name__}")
        if t.dtype not in dtypes:
            raise TypeError(f"{fn}: {name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
        if not t.is_contiguous():
            if t.stride(-1) != 1 and t.size(-1) > 1 and t.numel():
                raise ValueError(f"{fn}: {name} must be contiguous along its last axis")
            if dense and t.numel():
                raise ValueError(f"{fn}: {name} must be contiguous")
        if t.get_device() != dev:
            dev = -1
    return dev


def _go(fn, dev, tensors, stream, *args):
    """Calls the C entry point with args and the stream (by default the current
    one of the tensors' GPU), with that GPU as the current device."""
    if dev < 0:
        for name, t, _, _ in tensors:
            if t.device.type != "cuda":
                raise ValueError(f"{fn}: {name} must be on the GPU, got a {t.device.type} tensor")
        raise ValueError(f"{fn}: the tensors are on several GPUs: "
                         + ", ".join(f"{name} on {t.device}" for name, t, _, _ in tensors))
    if stream is None:
        stream = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    f = getattr(lib, fn)
    if torch.cuda.current_device() == dev:
        status = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = f(*args, stream)
    if status:
        raise Fp4Error(fn, status)


# The current stream's handle of a GPU by index, without a Stream object where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _shape(fn, name, t, shape, rows_at_least=False):
    """t must have the given shape; with rows_at_least, a 2-D t may hold more
    rows than are read.  Nothing is read when the shape is empty."""
    shape = tuple(int(v) for v in shape)
    if 0 in shape:
        return
    got = tuple(t.shape)
    ok = got == shape or (rows_at_least and len(got) == 2 and got[1] == shape[1] and got[0] >= shape[0])
    if not ok:
        raise ValueError(f"{fn}: {name} has shape {got}, expected {shape}")


def _stream(stream):
    if stream is None:
        return _raw_stream(torch.cuda.current_device()) if torch.cuda.is_initialized() else None
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(fn, status):
    if status != 0:
        raise Fp4Error(fn, status)


def fp4_abi_version() -> int:
    return lib.fp4_abi_version()


def fp4_quantize_mx(x, codes, scales, rows=None, k=None, ld_x=None, stream=None):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    ld_x = x.stride(0) if ld_x is None else ld_x
    fn = "fp4_quantize_mx"
    a = _Args(fn)
    a("x", x, _BF16, dense=False)
    a("codes", codes, _U8)
    a("scales", scales, _U8)
    a.on_device()
    _check("fp4_quantize_mx", lib.fp4_quantize_mx(_ptr(x), rows, k, ld_x, _ptr(codes), _ptr(scales), _stream(stream)))


def fp4_quantize_nv_workspace_bytes(rows: int, k: int) -> int:
    return lib.fp4_quantize_nv_workspace_bytes(rows, k)


def fp4_quantize_nv(x, codes, scales, tensor_scale, tensor_scale_is_input=False, workspace=None,
                    rows=None, k=None, ld_x=None, stream=None):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    ld_x = x.stride(0) if ld_x is None else ld_x
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fn = "fp4_quantize_nv"
    a = _Args(fn)
    a("x", x, _BF16, dense=False)
    a("codes", codes, _U8)
    a("scales", scales, _U8)
    a("tensor_scale", tensor_scale, _F32)
    a.on_device()
    _check("fp4_quantize_nv", lib.fp4_quantize_nv(_ptr(x), rows, k, ld_x, _ptr(codes), _ptr(scales),
                                                  _ptr(tensor_scale), int(bool(tensor_scale_is_input)),
                                                  _ptr(workspace), wsb, _stream(stream)))


def fp4_quantize_nv_noalloc(x, codes, scales, tensor_scale, tensor_scale_is_input=False, rows=None, k=None,
                            ld_x=None, stream=None):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    ld_x = x.stride(0) if ld_x is None else ld_x
    fn = "fp4_quantize_nv_noalloc"
    a = _Args(fn)
    a("x", x, _BF16, dense=False)
    a("codes", codes, _U8)
    a("scales", scales, _U8)
    a("tensor_scale", tensor_scale, _F32)
    a.on_device()
    _check(fn, lib.fp4_quantize_nv_noalloc(_ptr(x), rows, k, ld_x, _ptr(codes), _ptr(scales), _ptr(tensor_scale),
                                           int(bool(tensor_scale_is_input)), _stream(stream)))


def fp4_scale_max_workspace_bytes(rows: int, k: int) -> int:
    return lib.fp4_scale_max_workspace_bytes(rows, k)


def fp4_remap_mx_to_nv(codes, scales_e8m0, scales_e4m3, tensor_scale, n_inexact, workspace=None, rows=None, k=None,
                       stream=None):
    rows = codes.shape[0] if rows is None else rows
    k = codes.shape[1] * 2 if k is None else k
    fn = "fp4_remap_mx_to_nv"
    a = _Args(fn)
    for nm, t in (("codes", codes), ("scales_e8m0", scales_e8m0), ("scales_e4m3", scales_e4m3)):
        a(nm, t, _U8)
    a("tensor_scale", tensor_scale, _F32)
    a("n_inexact", n_inexact, _I32)
    a("workspace", workspace, _U8, optional=True)
    wsb = 0 if workspace is None else workspace.numel()
    a.on_device()
    _check("fp4_remap_mx_to_nv", lib.fp4_remap_mx_to_nv(_ptr(codes), _ptr(scales_e8m0), rows, k, _ptr(scales_e4m3),
                                                        _ptr(tensor_scale), _ptr(n_inexact), _ptr(workspace), wsb,
                                                        _stream(stream)))


def fp4_dequant(fmt, codes, scales, tensor_scale, out, rows=None, k=None, ld_out=None, stream=None):
    rows = codes.shape[0] if rows is None else rows
    k = codes.shape[1] * 2 if k is None else k
    ld_out = out.stride(0) if ld_out is None else ld_out
    dt = DT_F32 if out.dtype == torch.float32 else DT_BF16
    fn = "fp4_dequant"
    a = _Args(fn)
    a("codes", codes, _U8)
    a("scales", scales, _U8)
    a("tensor_scale", tensor_scale, _F32, optional=fmt == FMT_MX)
    a("out", out, _OUT, dense=False)
    a.on_device()
    _check("fp4_dequant", lib.fp4_dequant(fmt, _ptr(codes), _ptr(scales), _ptr(tensor_scale), rows, k, _ptr(out), dt,
                                          ld_out, _stream(stream)))


def fp4_gemm(fmt, a_codes, a_scales, b_codes, b_scales, c, a_tensor_scale=None, b_tensor_scale=None,
             m=None, n=None, k=None, ldc=None, stream=None):
    m = a_codes.shape[0] if m is None else m
    n = b_codes.shape[0] if n is None else n
    k = a_codes.shape[1] * 2 if k is None else k
    ldc = c.stride(0) if ldc is None else ldc
    dt = DT_F32 if c.dtype == torch.float32 else DT_BF16
    fn = "fp4_gemm"
    a = _Args(fn)
    for nm, t in (("a_codes", a_codes), ("a_scales", a_scales), ("b_codes", b_codes), ("b_scales", b_scales)):
        a(nm, t, _U8)
    a("a_tensor_scale", a_tensor_scale, _F32, optional=fmt == FMT_MX)
    a("b_tensor_scale", b_tensor_scale, _F32, optional=fmt == FMT_MX)
    a("c", c, _OUT, dense=False)
    blk = 32 if fmt == FMT_MX else 16
    _shape(fn, "a_codes", a_codes, (m, k // 2), rows_at_least=True)
    _shape(fn, "b_codes", b_codes, (n, k // 2), rows_at_least=True)
    _shape(fn, "a_scales", a_scales, (m, k // blk), rows_at_least=True)
    _shape(fn, "b_scales", b_scales, (n, k // blk), rows_at_least=True)
    a.on_device()
    _check("fp4_gemm", lib.fp4_gemm(fmt, _ptr(a_codes), _ptr(a_scales), _ptr(a_tensor_scale), _ptr(b_codes),
                                    _ptr(b_scales), _ptr(b_tensor_scale), m, n, k, _ptr(c), dt, ldc,
                                    _stream(stream)))


def fp4_kv_append_mx(x, slots, cache_codes, cache_scales, tokens=None, d=None, ld_x=None, stream=None):
    tokens = x.shape[0] if tokens is None else tokens
    d = x.shape[1] if d is None else d
    ld_x = x.stride(0) if ld_x is None else ld_x
    fn = "fp4_kv_append_mx"
    tensors = (("x", x, _BF16, False), ("slots", slots, _I32, True), ("cache_codes", cache_codes, _U8, True),
               ("cache_scales", cache_scales, _U8, True))
    dev = _check_all(fn, tensors)
    _go(fn, dev, tensors, stream, x.data_ptr(), tokens, d, ld_x, slots.data_ptr(), cache_codes.data_ptr(),
        cache_scales.data_ptr(), cache_codes.shape[0])


def fp4_fake_quant(fmt, x, out, tensor_scale=None, tensor_scale_is_input=False, workspace=None, rows=None, k=None,
                   ld_x=None, ld_out=None, stream=None):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    ld_x = x.stride(0) if ld_x is None else ld_x
    ld_out = out.stride(0) if ld_out is None else ld_out
    dt = DT_F32 if out.dtype == torch.float32 else DT_BF16
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    fn = "fp4_fake_quant"
    a = _Args(fn)
    a("x", x, _BF16, dense=False)
    a("out", out, _OUT, dense=False)
    a("tensor_scale", tensor_scale, _F32, optional=True)
    a.on_device()
    _check("fp4_fake_quant", lib.fp4_fake_quant(fmt, _ptr(x), rows, k, ld_x, _ptr(out), dt, ld_out, _ptr(tensor_scale),
                                                int(bool(tensor_scale_is_input)), _ptr(workspace), wsb,
                                                _stream(stream)))


def fp4_ste_backward(grad, grad_master, accumulate=True, rows=None, k=None, ld_grad=None, ld_master=None,
                     stream=None):
    rows = grad.shape[0] if rows is None else rows
    k = grad.shape[1] if k is None else k
    ld_grad = grad.stride(0) if ld_grad is None else ld_grad
    ld_master = grad_master.stride(0) if ld_master is None else ld_master
    dt = DT_F32 if grad.dtype == torch.float32 else DT_BF16
    fn = "fp4_ste_backward"
    a = _Args(fn)
    a("grad", grad, _OUT, dense=False)
    a("grad_master", grad_master, _F32, dense=False)
    a.on_device()
    _check("fp4_ste_backward", lib.fp4_ste_backward(_ptr(grad), dt, rows, k, ld_grad, _ptr(grad_master), ld_master,
                                                    int(bool(accumulate)), _stream(stream)))


def fp4_quantize_mxfp8(x, codes8, scales, rows=None, k=None, ld_x=None, stream=None):
    rows = x.shape[0] if rows is None else rows
    k = x.shape[1] if k is None else k
    ld_x = x.stride(0) if ld_x is None else ld_x
    fn = "fp4_quantize_mxfp8"
    a = _Args(fn)
    a("x", x, _BF16, dense=False)
    a("codes8", codes8, _U8)
    a("scales", scales, _U8)
    a.on_device()
    _check("fp4_quantize_mxfp8", lib.fp4_quantize_mxfp8(_ptr(x), rows, k, ld_x, _ptr(codes8), _ptr(scales),
                                                        _stream(stream)))


def fp4_mx_to_mxfp8(codes, codes8, rows=None, k=None, stream=None):
    rows = codes.shape[0] if rows is None else rows
    k = codes.shape[1] * 2 if k is None else k
    a = _Args("fp4_mx_to_mxfp8")("codes", codes, _U8)("codes8", codes8, _U8)
    a.on_device()
    _check("fp4_mx_to_mxfp8", lib.fp4_mx_to_mxfp8(_ptr(codes), rows, k, _ptr(codes8), _stream(stream)))


def fp4_mx_dequant_fp8(codes, scales_e8m0, values_e4m3, tensor_scale, n_inexact, block_scales_e4m3=None,
                       workspace=None, rows=None, k=None, stream=None):
    rows = codes.shape[0] if rows is None else rows
    k = codes.shape[1] * 2 if k is None else k
    fn = "fp4_mx_dequant_fp8"
    a = _Args(fn)
    for nm, t in (("codes", codes), ("scales_e8m0", scales_e8m0), ("values_e4m3", values_e4m3)):
        a(nm, t, _U8)
    a("block_scales_e4m3", block_scales_e4m3, _U8, optional=True)
    a("tensor_scale", tensor_scale, _F32)
    a("n_inexact", n_inexact, _I32)
    a("workspace", workspace, _U8, optional=True)
    wsb = 0 if workspace is None else workspace.numel()
    _shape(fn, "scales_e8m0", scales_e8m0, (rows, k // 32), rows_at_least=True)
    _shape(fn, "values_e4m3", values_e4m3, (rows, k), rows_at_least=True)
    a.on_device()
    _check("fp4_mx_dequant_fp8", lib.fp4_mx_dequant_fp8(_ptr(codes), _ptr(scales_e8m0), rows, k, _ptr(values_e4m3),
                                                        _ptr(block_scales_e4m3), _ptr(tensor_scale), _ptr(n_inexact),
                                                        _ptr(workspace), wsb, _stream(stream)))


def fp4_gemm_w4a8(a_codes8, a_scales, b_codes, b_scales, c, m=None, n=None, k=None, ldc=None, stream=None):
    m = a_codes8.shape[0] if m is None else m
    n = b_codes.shape[0] if n is None else n
    k = a_codes8.shape[1] if k is None else k
    ldc = c.stride(0) if ldc is None else ldc
    dt = DT_F32 if c.dtype == torch.float32 else DT_BF16
    fn = "fp4_gemm_w4a8"
    a = _Args(fn)
    for nm, t in (("a_codes8", a_codes8), ("a_scales", a_scales), ("b_codes", b_codes), ("b_scales", b_scales)):
        a(nm, t, _U8)
    a("c", c, _OUT, dense=False)
    _shape(fn, "a_codes8", a_codes8, (m, k), rows_at_least=True)
    _shape(fn, "b_codes", b_codes, (n, k // 2), rows_at_least=True)
    _shape(fn, "a_scales", a_scales, (m, k // 32), rows_at_least=True)
    _shape(fn, "b_scales", b_scales, (n, k // 32), rows_at_least=True)
    a.on_device()
    _check("fp4_gemm_w4a8", lib.fp4_gemm_w4a8(_ptr(a_codes8), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), m, n, k,
                                              _ptr(c), dt, ldc, _stream(stream)))


def fp4_moe_workspace_bytes(fmt, tokens, hidden, topk, num_experts, inter) -> int:
    return lib.fp4_moe_workspace_bytes(fmt, tokens, hidden, topk, num_experts, inter)


def fp4_moe_grouped_gemm(fmt, x, topk_ids, topk_weights, num_experts, inter, w13_codes, w13_scales, w2_codes,
                         w2_scales, out, workspace, w13_tensor_scales=None, w2_tensor_scales=None,
                         act_tensor_scales=None, debug: MoeDebug | None = None, stream=None):
    fn = "fp4_moe_grouped_gemm"
    a = _Args(fn)
    a("x", x, _BF16)
    a("topk_ids", topk_ids, _I32)
    a("topk_weights", topk_weights, _F32)
    for nm, t in (("w13_codes", w13_codes), ("w13_scales", w13_scales), ("w2_codes", w2_codes),
                  ("w2_scales", w2_scales), ("workspace", workspace)):
        a(nm, t, _U8)
    for nm, t in (("w13_tensor_scales", w13_tensor_scales), ("w2_tensor_scales", w2_tensor_scales),
                  ("act_tensor_scales", act_tensor_scales)):
        a(nm, t, _F32, optional=fmt == FMT_MX)
    a("out", out, _BF16)
    tokens, hidden = x.shape
    topk = topk_ids.shape[1]
    blk = 32 if fmt == FMT_MX else 16
    _shape(fn, "topk_ids", topk_ids, (tokens, topk))
    _shape(fn, "topk_weights", topk_weights, (tokens, topk))
    _shape(fn, "out", out, (tokens, hidden))
    _shape(fn, "w13_codes", w13_codes, (num_experts, 2 * inter, hidden // 2))
    _shape(fn, "w13_scales", w13_scales, (num_experts, 2 * inter, hidden // blk))
    _shape(fn, "w2_codes", w2_codes, (num_experts, hidden, inter // 2))
    _shape(fn, "w2_scales", w2_scales, (num_experts, hidden, inter // blk))
    wsb = workspace.numel() * workspace.element_size()
    dbg = _c.byref(debug) if debug is not None else None
    a.on_device()
    _check("fp4_moe_grouped_gemm", lib.fp4_moe_grouped_gemm(
        fmt, _ptr(x), tokens, hidden, _ptr(topk_ids), _ptr(topk_weights), topk, num_experts, inter,
        _ptr(w13_codes), _ptr(w13_scales), _ptr(w13_tensor_scales), _ptr(w2_codes), _ptr(w2_scales),
        _ptr(w2_tensor_scales), _ptr(act_tensor_scales), _ptr(out), _ptr(workspace), wsb, dbg, _stream(stream)))


def _heads(fn, name, t):
    """The leading dimension of a [tokens, heads, head_dim] tensor, whose heads
    must lie one after another; tokens may be any number of elements apart."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{fn}: {name} must be [tokens, heads, head_dim], got shape {tuple(shape)}")
    tokens, heads, d = shape
    ld, head, _ = t.stride()
    if head != d and heads > 1 and tokens and d:
        raise ValueError(f"{fn}: the heads of {name} must be contiguous")
    return ld if tokens > 1 else heads * d


def fp4_qk_norm_rope(q, k, q_out, k_out, positions=None, cos_sin=None, q_weight=None, k_weight=None, eps=1e-6,
                     interleaved=False, stream=None):
    """q [tokens, q_heads, head_dim], k [tokens, kv_heads, head_dim]: their rms
    norms and rotation into q_out and k_out (which may be q and k).  cos_sin:
    fp32 [max_positions, rot_dim]; None: norms only."""
    fn = "fp4_qk_norm_rope"
    tensors = [("q", q, _BF16, False), ("k", k, _BF16, False), ("q_out", q_out, _BF16, False), ("k_out", k_out, _BF16, False)]
    weight = q_weight if q_weight is not None else k_weight
    if q_weight is not None:
        tensors.append(("q_weight", q_weight, _OUT, True))
    if k_weight is not None:
        tensors.append(("k_weight", k_weight, _OUT if q_weight is None else (q_weight.dtype,), True))
    if cos_sin is not None:
        tensors += (("cos_sin", cos_sin, _F32, True), ("positions", positions, _I32, True))
    dev = _check_all(fn, tensors)
    ld_q, ld_k, ld_qo, ld_ko = _heads(fn, "q", q), _heads(fn, "k", k), _heads(fn, "q_out", q_out), _heads(fn, "k_out", k_out)
    tokens, q_heads, head_dim = shape = q.shape
    k_tokens, kv_heads, k_dim = k_shape = k.shape
    if k_tokens != tokens or k_dim != head_dim:
        raise ValueError(f"{fn}: k has shape {tuple(k_shape)}, q {tuple(shape)}")
    if q_out.shape != shape or k_out.shape != k_shape:
        raise ValueError(f"{fn}: q_out and k_out must have the shapes of q and k")
    for nm, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and w.shape != (head_dim,):
            raise ValueError(f"{fn}: {nm} has shape {tuple(w.shape)}, expected {(head_dim,)}")
    places = rot_dim = 0
    table = where = None
    if cos_sin is not None:
        if cos_sin.dim() != 2 or positions.shape != (tokens,):
            raise ValueError(f"{fn}: cos_sin must be [max_positions, rot_dim] and positions [tokens]")
        places, rot_dim = cos_sin.shape
        table, where = cos_sin.data_ptr(), positions.data_ptr()
    _go(fn, dev, tensors, stream, q.data_ptr(), k.data_ptr(), tokens, q_heads, kv_heads, head_dim, ld_q, ld_k,
        _ptr(q_weight), _ptr(k_weight), DT_BF16 if weight is None or weight.dtype is torch.bfloat16 else DT_F32, eps, table,
        places, rot_dim, 1 if interleaved else 0, where, q_out.data_ptr(), ld_qo, k_out.data_ptr(), ld_ko)


class KvCache(NamedTuple):
    """A paged MXFP4 cache in fp4_kv_append_mx's layout: uint8 codes
    [num_pages * page_size, d/2] and scales [num_pages * page_size, d/32] of the
    keys and of the values (both None: a keys-only cache)."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor | None
    v_scales: torch.Tensor | None
    page_size: int


class KvPages(NamedTuple):
    """The pages that the sequences of a batch hold: int32 page_table
    [batch, max_pages] (-1 = none), page_counts [batch], seq_lens [batch]
    (committed tokens) and page_refs [num_pages] (holders; 0 = free)."""
    page_table: torch.Tensor
    page_counts: torch.Tensor
    seq_lens: torch.Tensor
    page_refs: torch.Tensor


def _cache_tensors(cache, name=""):
    kc, ks, vc, vs, _ = cache
    tensors = [(name + "k_codes", kc, _U8, True), (name + "k_scales", ks, _U8, True)]
    if vc is not None:
        tensors.append((name + "v_codes", vc, _U8, True))
    if vs is not None:
        tensors.append((name + "v_scales", vs, _U8, True))
    return tensors


def _pages_tensors(pages):
    table, counts, lens, refs = pages
    return [("page_table", table, _I32, True), ("page_counts", counts, _I32, True), ("seq_lens", lens, _I32, True),
            ("page_refs", refs, _I32, True)]


def _cache_struct(fn, cache):
    """Checks the shapes of a KvCache's (checked) tensors; its C struct and d."""
    kc, ks, vc, vs, page_size = cache
    if (vc is None) != (vs is None):
        raise ValueError(f"{fn}: v_codes and v_scales must both be given or both be None")
    if kc.dim() != 2 or page_size <= 0 or len(kc) % page_size:
        raise ValueError(f"{fn}: k_codes must be [num_pages * {page_size}, d/2], got {tuple(kc.shape)}")
    rows, half = shape = kc.shape
    scales = ks.shape
    if scales != (rows, half // 16):
        raise ValueError(f"{fn}: k_scales has shape {tuple(scales)}, expected {(rows, half // 16)}")
    if vc is None:
        return _pack_kv(kc.data_ptr(), ks.data_ptr(), 0, 0, rows // page_size, 2 * half, page_size), 2 * half
    if vc.shape != shape or vs.shape != scales:
        raise ValueError(f"{fn}: the cache's values must have the shapes of its keys")
    return _pack_kv(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), rows // page_size, 2 * half, page_size), 2 * half


def _pages_struct(fn, pages):
    """Checks the shapes of a KvPages' (checked) tensors; its C struct and batch."""
    table, counts, lens, refs = pages
    shape = table.shape
    if len(shape) != 2 or counts.shape != shape[:1] or lens.shape != shape[:1] or refs.dim() != 1:
        raise ValueError(f"{fn}: page_table must be [batch, max_pages], page_counts and seq_lens [batch], "
                         "page_refs [num_pages]")
    batch, width = shape
    return _pack_kv(table.data_ptr(), counts.data_ptr(), lens.data_ptr(), refs.data_ptr(), batch, width, len(refs)), batch


def _per_seq(fn, name, t, n):
    if t is not None and t.shape != (n,):
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {(n,)}")


def fp4_kv_reserve_workspace_bytes(batch: int, num_pages: int) -> int:
    return lib.fp4_kv_reserve_workspace_bytes(batch, num_pages)


def fp4_kv_reserve(cache: KvCache, pages: KvPages, new_tokens, slots, n_short, workspace, stream=None):
    """Room for new_tokens[b] tokens behind every sequence; their cache rows in
    slots [batch, max_new] (None: not wanted), -1 past new_tokens[b]."""
    fn = "fp4_kv_reserve"
    tensors = _cache_tensors(cache) + _pages_tensors(pages)
    tensors += (("new_tokens", new_tokens, _I32, True), ("n_short", n_short, _I32, True), ("workspace", workspace, _U8, True))
    if slots is not None:
        tensors.append(("slots", slots, _I32, True))
    dev = _check_all(fn, tensors)
    c, _ = _cache_struct(fn, cache)
    p, batch = _pages_struct(fn, pages)
    _per_seq(fn, "new_tokens", new_tokens, batch)
    _per_seq(fn, "n_short", n_short, 1)
    max_new = 0
    if slots is not None:
        if slots.dim() != 2 or slots.shape[0] != batch:
            raise ValueError(f"{fn}: slots has shape {tuple(slots.shape)}, expected [{batch}, max_new]")
        max_new = slots.shape[1]
    _go(fn, dev, tensors, stream, c, p, new_tokens.data_ptr(), _ptr(slots), max_new, n_short.data_ptr(), workspace.data_ptr(),
        workspace.numel())


def fp4_kv_fork(pages: KvPages, pairs, page_size: int, stream=None):
    """pairs int32 [n, 2]: (source, target) sequences."""
    fn = "fp4_kv_fork"
    tensors = _pages_tensors(pages)
    tensors.append(("pairs", pairs, _I32, True))
    dev = _check_all(fn, tensors)
    p, _ = _pages_struct(fn, pages)
    if pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError(f"{fn}: pairs has shape {tuple(pairs.shape)}, expected [n, 2]")
    _go(fn, dev, tensors, stream, p, pairs.data_ptr(), pairs.shape[0], page_size)


def fp4_kv_free(pages: KvPages, seqs, page_size: int, keep_lens=None, stream=None):
    """Cuts the sequences seqs int32 [n] back to keep_lens int32 [n] tokens (None: none)."""
    fn = "fp4_kv_free"
    tensors = _pages_tensors(pages)
    tensors.append(("seqs", seqs, _I32, True))
    if keep_lens is not None:
        tensors.append(("keep_lens", keep_lens, _I32, True))
    dev = _check_all(fn, tensors)
    p, _ = _pages_struct(fn, pages)
    if seqs.dim() != 1:
        raise ValueError(f"{fn}: seqs has shape {tuple(seqs.shape)}, expected [n]")
    _per_seq(fn, "keep_lens", keep_lens, len(seqs))
    _go(fn, dev, tensors, stream, p, seqs.data_ptr(), len(seqs), _ptr(keep_lens), page_size)


def fp4_kv_compact(cache: KvCache, pages: KvPages, accepted, accepted_lens, stream=None):
    """Commits the drafted tokens accepted[b, :accepted_lens[b]] (None: the first
    accepted_lens[b] reserved ones) behind every sequence."""
    fn = "fp4_kv_compact"
    tensors = _cache_tensors(cache) + _pages_tensors(pages)
    tensors.append(("accepted_lens", accepted_lens, _I32, True))
    if accepted is not None:
        tensors.append(("accepted", accepted, _I32, True))
    dev = _check_all(fn, tensors)
    c, _ = _cache_struct(fn, cache)
    p, batch = _pages_struct(fn, pages)
    _per_seq(fn, "accepted_lens", accepted_lens, batch)
    most = 0
    if accepted is not None:
        if accepted.dim() != 2 or accepted.shape[0] != batch:
            raise ValueError(f"{fn}: accepted has shape {tuple(accepted.shape)}, expected [{batch}, max_accepted]")
        most = accepted.shape[1]
        if most == 0:
            return                                                    # nothing can be accepted
    _go(fn, dev, tensors, stream, c, p, _ptr(accepted), most, accepted_lens.data_ptr())


def fp4_kv_copy_pages(src: KvCache, dst: KvCache, src_pages, dst_pages, stream=None):
    """Page src_pages[i] of src to page dst_pages[i] of dst (int32 [n] each)."""
    fn = "fp4_kv_copy_pages"
    tensors = _cache_tensors(src, "src.") + _cache_tensors(dst, "dst.")
    tensors += (("src_pages", src_pages, _I32, True), ("dst_pages", dst_pages, _I32, True))
    dev = _check_all(fn, tensors)
    (s, _), (d, _) = _cache_struct(fn, src), _cache_struct(fn, dst)
    if src_pages.dim() != 1:
        raise ValueError(f"{fn}: src_pages has shape {tuple(src_pages.shape)}, expected [n]")
    _per_seq(fn, "dst_pages", dst_pages, len(src_pages))
    _go(fn, dev, tensors, stream, s, d, src_pages.data_ptr(), dst_pages.data_ptr(), len(src_pages))


def fp4_attn_tree_workspace_bytes(batch: int, drafts: int, q_heads: int, head_dim: int, kv_heads: int) -> int:
    return lib.fp4_attn_tree_workspace_bytes(batch, drafts, q_heads, head_dim, kv_heads)


def _drafted(fn, name, t):
    """The pitch of the tokens of a [batch, drafts, q_heads, head_dim] tensor, which must be one."""
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{fn}: {name} must be [batch, drafts, q_heads, head_dim], got shape {tuple(shape)}")
    batch, drafts, heads, d = shape
    seq, token, head, _ = t.stride()
    empty = not (batch and drafts and heads and d)
    if heads > 1 and head != d and not empty:
        raise ValueError(f"{fn}: the heads of {name} must be contiguous")
    ld = token if drafts > 1 else seq if batch > 1 else heads * d
    if batch > 1 and seq != drafts * ld and not empty:
        raise ValueError(f"{fn}: the tokens of {name} must be one pitch apart")
    return ld


def fp4_attn_tree_mx(q, cache: KvCache, page_table, seq_lens, out, workspace, draft_lens=None, tree_mask=None, scale=None,
                     stream=None):
    """q, out [batch, drafts, q_heads, head_dim]; tree_mask int64 [batch, drafts]
    (bit j: sees drafted token j; None: tokens up to itself); scale None: head_dim ** -0.5."""
    fn = "fp4_attn_tree_mx"
    tensors = [("q", q, _BF16, False), ("out", out, _BF16, False)]
    tensors += _cache_tensors(cache)
    tensors += (("page_table", page_table, _I32, True), ("seq_lens", seq_lens, _I32, True), ("workspace", workspace, _U8, True))
    if draft_lens is not None:
        tensors.append(("draft_lens", draft_lens, _I32, True))
    if tree_mask is not None:
        tensors.append(("tree_mask", tree_mask, _I64, True))
    dev = _check_all(fn, tensors)
    ld_q, ld_out = _drafted(fn, "q", q), _drafted(fn, "out", out)
    batch, drafts, q_heads, head_dim = shape = q.shape
    if out.shape != shape:
        raise ValueError(f"{fn}: out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    c, d = _cache_struct(fn, cache)
    if cache.v_codes is None:
        raise ValueError(f"{fn}: the cache has no values")
    if not head_dim or not d or d % head_dim:
        raise ValueError(f"{fn}: the cache's rows hold {d} values, not a multiple of head_dim {head_dim}")
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError(f"{fn}: page_table has shape {tuple(page_table.shape)}, expected [{batch}, max_pages]")
    _per_seq(fn, "seq_lens", seq_lens, batch)
    _per_seq(fn, "draft_lens", draft_lens, batch)
    if tree_mask is not None and tree_mask.shape != (batch, drafts):
        raise ValueError(f"{fn}: tree_mask has shape {tuple(tree_mask.shape)}, expected {(batch, drafts)}")
    _go(fn, dev, tensors, stream, q.data_ptr(), ld_q, c, page_table.data_ptr(), page_table.shape[1], seq_lens.data_ptr(),
        _ptr(draft_lens), _ptr(tree_mask), batch, drafts, q_heads, d // head_dim, head_dim,
        head_dim ** -0.5 if scale is None else scale, out.data_ptr(), ld_out, workspace.data_ptr(), workspace.numel())


def fp4_attn_prompt(q, k, v, cu_seqlens, out, scale=None, stream=None):
    """q, out [tokens, q_heads, head_dim], k, v [tokens, kv_heads, head_dim]:
    causal attention inside each sequence [cu_seqlens[s], cu_seqlens[s + 1])
    (int32 [seqs + 1]); scale None: head_dim ** -0.5."""
    fn = "fp4_attn_prompt"
    tensors = (("q", q, _BF16, False), ("k", k, _BF16, False), ("v", v, _BF16, False), ("out", out, _BF16, False),
               ("cu_seqlens", cu_seqlens, _I32, True))
    dev = _check_all(fn, tensors)
    ld_q, ld_k, ld_v, ld_out = _heads(fn, "q", q), _heads(fn, "k", k), _heads(fn, "v", v), _heads(fn, "out", out)
    tokens, q_heads, head_dim = shape = q.shape
    k_tokens, kv_heads, k_dim = k_shape = k.shape
    if k_tokens != tokens or k_dim != head_dim or v.shape != k_shape:
        raise ValueError(f"{fn}: k and v have shapes {tuple(k_shape)} and {tuple(v.shape)}, q {tuple(shape)}")
    if out.shape != shape:
        raise ValueError(f"{fn}: out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if cu_seqlens.dim() != 1 or len(cu_seqlens) < 1:
        raise ValueError(f"{fn}: cu_seqlens has shape {tuple(cu_seqlens.shape)}, expected [seqs + 1]")
    _go(fn, dev, tensors, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), len(cu_seqlens) - 1, tokens,
        q_heads, kv_heads, head_dim, ld_q, ld_k, ld_v, head_dim ** -0.5 if scale is None else scale, out.data_ptr(), ld_out)
