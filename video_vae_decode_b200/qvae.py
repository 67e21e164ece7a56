"""ctypes binding of libqvae (declarations in include/qvae.h).

Argument marshalling only: every step of the layer runs in the CUDA library.
Tensors are torch CUDA tensors (device memory and streams come from PyTorch);
their data pointers are handed to the C entry points of the same names.
Each wrapper raises ``QvaeError`` on a non-zero status.  ``lib()`` raises if
``libqvae.so`` has not been built: there is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# QVAE_LIBRARY names another build of the same ABI (libqvae_debug.so: the
# bounds-checked kernels); the default is the in-tree release library.
LIB_PATH = os.environ.get("QVAE_LIBRARY") or os.path.join(HERE, "libqvae.so")

QVAE_OK, QVAE_ERR_ARG, QVAE_ERR_SHAPE, QVAE_ERR_ALIGN = 0, 1, 2, 3
QVAE_ERR_CUDA, QVAE_ERR_TIMEOUT, QVAE_ERR_UNSUPPORTED, QVAE_ERR_BOUNDS = 4, 5, 6, 7

# Every symbol include/qvae.h declares.
EXPORTS = (
    "qvae_status_string", "qvae_last_error_message", "qvae_packed_weight_bytes",
    "qvae_quantize_weights", "qvae_act_workspace_bytes", "qvae_act_absmax_quant",
    "qvae_causal_conv3d_w8a8", "qvae_causal_conv3d_w8a8_acc32", "qvae_decode_workspace_bytes",
    "qvae_decode_layers", "qvae_get_error", "qvae_set_wait_limit_ns",
    "qvae_selftest_wait_timeout", "qvae_build_flags", "qvae_set_conv_tiling", "qvae_get_conv_tiling", "qvae_set_conv_cta_limit",
    "qvae_act_absmax_quant_noalloc",
    "qvae_causal_conv3d_w8a8_carry", "qvae_causal_conv3d_w8a8_carry_acc32",
    "qvae_act_absmax", "qvae_act_quant_from_absmax",
    "qvae_causal_conv3d_w8a8_band", "qvae_causal_conv3d_w8a8_band_acc32",
    "qvae_packed_weight_bytes_bf16", "qvae_pack_weights_bf16", "qvae_causal_conv3d_bf16",
    "qvae_causal_conv3d_bf16_acc32", "qvae_causal_conv3d_w8a8_fused", "qvae_causal_conv3d_w8a8_fused_acc32",
    "qvae_set_fused_quant",
    "qvae_fp8_packed_weight_bytes", "qvae_fp8_weight_scale_bytes", "qvae_fp8_quantize_weights",
    "qvae_fp8_code_bytes", "qvae_fp8_scale_bytes", "qvae_fp8_workspace_bytes", "qvae_fp8_quant_act",
    "qvae_linear_fp8", "qvae_linear_fp8_grouped", "qvae_linear_fp8_fused", "qvae_linear_fp8_grouped_fused",
    "qvae_set_linear_tiling", "qvae_get_linear_tiling", "qvae_get_linear_footprint",
)

# qvae_fp8_op: what a linear layer quantises of its rows
QVAE_FP8_PLAIN, QVAE_FP8_SILU_MUL = 0, 1


class QvaeError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed: {message} (status {status})")
        self.status = status


class qvae_shape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("W", ctypes.c_int64), ("Cin", ctypes.c_int32), ("Cout", ctypes.c_int32)]


class qvae_layer(ctypes.Structure):
    _fields_ = [("shape", qvae_shape), ("quantized", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("wq_packed", ctypes.c_void_p),
                ("w_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libqvae.so; raises when it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m video_vae_decode_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, i64, u64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                ctypes.c_size_t)
        sig = {
            "qvae_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "qvae_last_error_message": ([], ctypes.c_char_p),
            "qvae_packed_weight_bytes": ([i32, i32], sz),
            "qvae_quantize_weights": ([i32, i32, p, p, p, p, p], ctypes.c_int),
            "qvae_act_workspace_bytes": ([i64], sz),
            "qvae_act_absmax_quant": ([p, i64, p, p, p, sz, p], ctypes.c_int),
            "qvae_act_absmax_quant_noalloc": ([p, i64, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8": ([ctypes.POINTER(qvae_shape), p, p, p, p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8_acc32": ([ctypes.POINTER(qvae_shape), p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8_carry": ([ctypes.POINTER(qvae_shape), p, p, p, p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8_carry_acc32": ([ctypes.POINTER(qvae_shape), p, p, p, p], ctypes.c_int),
            "qvae_act_absmax": ([p, i64, p, p], ctypes.c_int),
            "qvae_act_quant_from_absmax": ([p, i64, p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8_band": ([ctypes.POINTER(qvae_shape), i32, i32, p, p, p, p, p, p, p],
                                             ctypes.c_int),
            "qvae_causal_conv3d_w8a8_band_acc32": ([ctypes.POINTER(qvae_shape), i32, i32, p, p, p, p],
                                                   ctypes.c_int),
            "qvae_packed_weight_bytes_bf16": ([i32, i32], sz),
            "qvae_pack_weights_bf16": ([i32, i32, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_bf16": ([ctypes.POINTER(qvae_shape), p, p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_bf16_acc32": ([ctypes.POINTER(qvae_shape), p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8_fused": ([ctypes.POINTER(qvae_shape), p, p, p, p, p, p, p, p], ctypes.c_int),
            "qvae_causal_conv3d_w8a8_fused_acc32": ([ctypes.POINTER(qvae_shape), p, p, p, p, p], ctypes.c_int),
            "qvae_decode_workspace_bytes": ([ctypes.POINTER(qvae_layer), i32], sz),
            "qvae_decode_layers": ([ctypes.POINTER(qvae_layer), i32, p, sz, p], ctypes.c_int),
            "qvae_get_error": ([p], ctypes.c_int),
            "qvae_set_wait_limit_ns": ([u64], ctypes.c_int),
            "qvae_selftest_wait_timeout": ([u64, p], ctypes.c_int),
            "qvae_build_flags": ([], ctypes.c_int),
            "qvae_set_conv_tiling": ([i32, i32, i32, i32, i32, i32], ctypes.c_int),
            "qvae_set_conv_cta_limit": ([i32], ctypes.c_int),
            "qvae_set_fused_quant": ([i32], ctypes.c_int),
            "qvae_get_conv_tiling": ([ctypes.POINTER(qvae_shape), i32, ctypes.POINTER(i32)], ctypes.c_int),
            "qvae_fp8_packed_weight_bytes": ([i32, i32, i32], sz),
            "qvae_fp8_weight_scale_bytes": ([i32, i32, i32], sz),
            "qvae_fp8_quantize_weights": ([i32, i32, i32, p, p, p, p], ctypes.c_int),
            "qvae_fp8_code_bytes": ([i64, i32], sz),
            "qvae_fp8_scale_bytes": ([i64, i32], sz),
            "qvae_fp8_workspace_bytes": ([i64, i32], sz),
            "qvae_fp8_quant_act": ([i64, i32, i32, p, i64, p, p, p], ctypes.c_int),
            "qvae_linear_fp8": ([i64, i32, i32, p, p, p, p, p, p, i64, p], ctypes.c_int),
            "qvae_linear_fp8_grouped": ([i32, i64, i32, i32, p, p, p, p, p, p, p, i64, p], ctypes.c_int),
            "qvae_linear_fp8_fused": ([i64, i32, i32, i32, p, i64, p, p, p, p, i64, p, sz, p], ctypes.c_int),
            "qvae_set_linear_tiling": ([i32, i32, i32, i32], ctypes.c_int),
            "qvae_get_linear_tiling": ([i32, i64, i32, i32, ctypes.POINTER(i32)], ctypes.c_int),
            "qvae_get_linear_footprint": ([i32, i64, i32, i32, i32, ctypes.POINTER(i32)], ctypes.c_int),
            "qvae_linear_fp8_grouped_fused": ([i32, i64, i32, i32, i32, p, i64, p, p, p, p, p, i64, p, sz, p],
                                              ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(name: str, status: int):
    if status != QVAE_OK:
        L = lib()
        msg = L.qvae_status_string(status).decode()
        extra = L.qvae_last_error_message().decode()
        raise QvaeError(name, status, msg + (f": {extra}" if extra and status == QVAE_ERR_CUDA else ""))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA tensors"
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_shape(N, T, H, W, Cin, Cout) -> qvae_shape:
    return qvae_shape(int(N), int(T), int(H), int(W), int(Cin), int(Cout))


def shape_of(x: torch.Tensor, Cout: int) -> qvae_shape:
    N, T, H, W, Cin = x.shape
    return make_shape(N, T, H, W, Cin, Cout)


# ---------------------------------------------------------------- weights

def qvae_packed_weight_bytes(Cin: int, Cout: int) -> int:
    return int(lib().qvae_packed_weight_bytes(Cin, Cout))


def qvae_quantize_weights(w: torch.Tensor, wq_packed: torch.Tensor, w_scale: torch.Tensor,
                          wq_plain: Optional[torch.Tensor] = None, stream=None) -> None:
    Cout, Cin = int(w.shape[0]), int(w.shape[1])
    _check("qvae_quantize_weights",
           lib().qvae_quantize_weights(Cin, Cout, _ptr(w), _ptr(wq_packed), _ptr(w_scale),
                                       _ptr(wq_plain), _stream(stream)))


def quantize_weights(w: torch.Tensor, plain: bool = False, stream=None):
    """Allocate and fill (wq_packed, w_scale[, wq_plain [Cout, 27, Cin]]) for a bf16 weight."""
    Cout, Cin = int(w.shape[0]), int(w.shape[1])
    packed = torch.empty(qvae_packed_weight_bytes(Cin, Cout), dtype=torch.int8, device=w.device)
    scale = torch.empty(Cout, dtype=torch.float32, device=w.device)
    pl = torch.zeros((Cout, 27, Cin), dtype=torch.int8, device=w.device) if plain else None
    qvae_quantize_weights(w, packed, scale, pl, stream)
    return (packed, scale, pl) if plain else (packed, scale)


# ------------------------------------------------------------ activations

def qvae_act_workspace_bytes(numel: int) -> int:
    return int(lib().qvae_act_workspace_bytes(numel))


def qvae_act_absmax_quant(x: torch.Tensor, xq: torch.Tensor, x_scale: torch.Tensor,
                          workspace: torch.Tensor, stream=None) -> None:
    _check("qvae_act_absmax_quant",
           lib().qvae_act_absmax_quant(_ptr(x), x.numel(), _ptr(xq), _ptr(x_scale), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


def qvae_act_absmax_quant_noalloc(x: torch.Tensor, xq: torch.Tensor, x_scale: torch.Tensor,
                                  stream=None) -> None:
    """Same as qvae_act_absmax_quant with the library's fixed scratch (no workspace)."""
    _check("qvae_act_absmax_quant_noalloc",
           lib().qvae_act_absmax_quant_noalloc(_ptr(x), x.numel(), _ptr(xq), _ptr(x_scale), _stream(stream)))


def act_absmax_quant(x: torch.Tensor, stream=None, workspace: Optional[torch.Tensor] = None):
    xq = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    s = torch.empty(1, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(qvae_act_workspace_bytes(x.numel()), dtype=torch.uint8, device=x.device)
    qvae_act_absmax_quant(x, xq, s, workspace, stream)
    return xq, s


# ------------------------------------------------------------ convolution

def qvae_causal_conv3d_w8a8(xq: torch.Tensor, x_scale: torch.Tensor, wq_packed: torch.Tensor,
                            w_scale: torch.Tensor, bias: Optional[torch.Tensor], out: torch.Tensor,
                            stream=None) -> None:
    shp = shape_of(xq, int(out.shape[-1]))
    _check("qvae_causal_conv3d_w8a8",
           lib().qvae_causal_conv3d_w8a8(ctypes.byref(shp), _ptr(xq), _ptr(x_scale), _ptr(wq_packed),
                                         _ptr(w_scale), _ptr(bias), _ptr(out), _stream(stream)))


def qvae_causal_conv3d_w8a8_acc32(xq: torch.Tensor, wq_packed: torch.Tensor, acc: torch.Tensor,
                                  stream=None) -> None:
    shp = shape_of(xq, int(acc.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_acc32",
           lib().qvae_causal_conv3d_w8a8_acc32(ctypes.byref(shp), _ptr(xq), _ptr(wq_packed), _ptr(acc),
                                               _stream(stream)))


def causal_conv3d_w8a8(xq, x_scale, wq_packed, w_scale, bias, Cout: int, stream=None):
    out = torch.empty(tuple(xq.shape[:-1]) + (Cout,), dtype=torch.bfloat16, device=xq.device)
    qvae_causal_conv3d_w8a8(xq, x_scale, wq_packed, w_scale, bias, out, stream)
    return out


def _chunk_shape(xq_ext: torch.Tensor, Cout: int) -> qvae_shape:
    """Shape of a streamed chunk: xq_ext holds two carried frames before the chunk's."""
    N, T2, H, W, Cin = xq_ext.shape
    if T2 < 2:
        raise ValueError("a streamed chunk's input holds two carried frames before its own")
    return make_shape(N, T2 - 2, H, W, Cin, Cout)


def qvae_causal_conv3d_w8a8_carry(xq_ext: torch.Tensor, x_scale: torch.Tensor, wq_packed: torch.Tensor,
                                  w_scale: torch.Tensor, bias: Optional[torch.Tensor], out: torch.Tensor,
                                  stream=None) -> None:
    shp = _chunk_shape(xq_ext, int(out.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_carry",
           lib().qvae_causal_conv3d_w8a8_carry(ctypes.byref(shp), _ptr(xq_ext), _ptr(x_scale), _ptr(wq_packed),
                                               _ptr(w_scale), _ptr(bias), _ptr(out), _stream(stream)))


def qvae_causal_conv3d_w8a8_carry_acc32(xq_ext: torch.Tensor, wq_packed: torch.Tensor, acc: torch.Tensor,
                                        stream=None) -> None:
    shp = _chunk_shape(xq_ext, int(acc.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_carry_acc32",
           lib().qvae_causal_conv3d_w8a8_carry_acc32(ctypes.byref(shp), _ptr(xq_ext), _ptr(wq_packed),
                                                     _ptr(acc), _stream(stream)))


def conv_carry(xq_ext, x_scale, wq_packed, w_scale, bias, Cout: int, stream=None):
    _chunk_shape(xq_ext, Cout)
    N, T2, H, W, _ = xq_ext.shape
    out = torch.empty((N, T2 - 2, H, W, Cout), dtype=torch.bfloat16, device=xq_ext.device)
    qvae_causal_conv3d_w8a8_carry(xq_ext, x_scale, wq_packed, w_scale, bias, out, stream)
    return out


def conv_carry_acc32(xq_ext, wq_packed, Cout: int, stream=None):
    _chunk_shape(xq_ext, Cout)
    N, T2, H, W, _ = xq_ext.shape
    acc = torch.empty((N, T2 - 2, H, W, Cout), dtype=torch.int32, device=xq_ext.device)
    qvae_causal_conv3d_w8a8_carry_acc32(xq_ext, wq_packed, acc, stream)
    return acc


def qvae_act_absmax(x: torch.Tensor, amax: torch.Tensor, stream=None) -> None:
    """amax: a 4-byte device tensor (int32 or uint32) that receives max |x| as bf16 magnitude bits."""
    _check("qvae_act_absmax", lib().qvae_act_absmax(_ptr(x), x.numel(), _ptr(amax), _stream(stream)))


def qvae_act_quant_from_absmax(x: torch.Tensor, amax: torch.Tensor, xq: torch.Tensor, x_scale: torch.Tensor,
                               stream=None) -> None:
    _check("qvae_act_quant_from_absmax",
           lib().qvae_act_quant_from_absmax(_ptr(x), x.numel(), _ptr(amax), _ptr(xq), _ptr(x_scale),
                                            _stream(stream)))


def _band_shape(xq_band: torch.Tensor, halo_top: int, halo_bot: int, Cout: int) -> qvae_shape:
    N, T, Hin, W, Cin = xq_band.shape
    H = Hin - halo_top - halo_bot
    if H < 0:
        raise ValueError("a band holds its halo rows and its own")
    return make_shape(N, T, H, W, Cin, Cout)


def qvae_causal_conv3d_w8a8_band(xq_band: torch.Tensor, halo_top: int, halo_bot: int, x_scale: torch.Tensor,
                                 wq_packed: torch.Tensor, w_scale: torch.Tensor, bias: Optional[torch.Tensor],
                                 out: torch.Tensor, stream=None) -> None:
    shp = _band_shape(xq_band, halo_top, halo_bot, int(out.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_band",
           lib().qvae_causal_conv3d_w8a8_band(ctypes.byref(shp), int(halo_top), int(halo_bot), _ptr(xq_band),
                                              _ptr(x_scale), _ptr(wq_packed), _ptr(w_scale), _ptr(bias),
                                              _ptr(out), _stream(stream)))


def qvae_causal_conv3d_w8a8_band_acc32(xq_band: torch.Tensor, halo_top: int, halo_bot: int,
                                       wq_packed: torch.Tensor, acc: torch.Tensor, stream=None) -> None:
    shp = _band_shape(xq_band, halo_top, halo_bot, int(acc.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_band_acc32",
           lib().qvae_causal_conv3d_w8a8_band_acc32(ctypes.byref(shp), int(halo_top), int(halo_bot),
                                                    _ptr(xq_band), _ptr(wq_packed), _ptr(acc), _stream(stream)))


def qvae_causal_conv3d_w8a8_fused(x: torch.Tensor, x_amax: torch.Tensor, wq_packed: torch.Tensor,
                                  w_scale: torch.Tensor, bias: Optional[torch.Tensor], out: torch.Tensor,
                                  x_scale_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """x bf16; x_amax a 4-byte device word from qvae_act_absmax (bf16 magnitude bits of max |x|)."""
    shp = shape_of(x, int(out.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_fused",
           lib().qvae_causal_conv3d_w8a8_fused(ctypes.byref(shp), _ptr(x), _ptr(x_amax), _ptr(wq_packed),
                                               _ptr(w_scale), _ptr(bias), _ptr(out), _ptr(x_scale_out),
                                               _stream(stream)))


def qvae_causal_conv3d_w8a8_fused_acc32(x: torch.Tensor, x_amax: torch.Tensor, wq_packed: torch.Tensor,
                                        acc: torch.Tensor, stream=None) -> None:
    shp = shape_of(x, int(acc.shape[-1]))
    _check("qvae_causal_conv3d_w8a8_fused_acc32",
           lib().qvae_causal_conv3d_w8a8_fused_acc32(ctypes.byref(shp), _ptr(x), _ptr(x_amax), _ptr(wq_packed),
                                                     _ptr(acc), _stream(stream)))


def layer_w8a8(x, wq_packed, w_scale, bias, Cout: int, stream=None, amax=None, scale=None):
    """One quantised layer the fused way: qvae_act_absmax, then the convolution quantising x itself.
    Returns (out, scale)."""
    if amax is None:
        amax = torch.empty(1, dtype=torch.int32, device=x.device)
    if scale is None:
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    out = torch.empty(tuple(x.shape[:-1]) + (Cout,), dtype=torch.bfloat16, device=x.device)
    qvae_act_absmax(x, amax, stream)
    qvae_causal_conv3d_w8a8_fused(x, amax, wq_packed, w_scale, bias, out, scale, stream)
    return out, scale


def conv_acc32(xq, wq_packed, Cout: int, stream=None):
    acc = torch.empty(tuple(xq.shape[:-1]) + (Cout,), dtype=torch.int32, device=xq.device)
    qvae_causal_conv3d_w8a8_acc32(xq, wq_packed, acc, stream)
    return acc


# ------------------------------------------------- native-precision layer

def qvae_packed_weight_bytes_bf16(Cin: int, Cout: int) -> int:
    return int(lib().qvae_packed_weight_bytes_bf16(Cin, Cout))


def qvae_pack_weights_bf16(w: torch.Tensor, w_packed: torch.Tensor, stream=None) -> None:
    Cout, Cin = int(w.shape[0]), int(w.shape[1])
    _check("qvae_pack_weights_bf16",
           lib().qvae_pack_weights_bf16(Cin, Cout, _ptr(w), _ptr(w_packed), _stream(stream)))


def pack_weights_bf16(w: torch.Tensor, stream=None) -> torch.Tensor:
    """Allocate and fill the packed bf16 weights of a native-precision layer."""
    Cout, Cin = int(w.shape[0]), int(w.shape[1])
    packed = torch.empty(qvae_packed_weight_bytes_bf16(Cin, Cout), dtype=torch.uint8, device=w.device)
    qvae_pack_weights_bf16(w, packed, stream)
    return packed


def qvae_causal_conv3d_bf16(x: torch.Tensor, w_packed: torch.Tensor, bias: Optional[torch.Tensor],
                            out: torch.Tensor, stream=None) -> None:
    shp = shape_of(x, int(out.shape[-1]))
    _check("qvae_causal_conv3d_bf16",
           lib().qvae_causal_conv3d_bf16(ctypes.byref(shp), _ptr(x), _ptr(w_packed), _ptr(bias), _ptr(out),
                                         _stream(stream)))


def qvae_causal_conv3d_bf16_acc32(x: torch.Tensor, w_packed: torch.Tensor, acc: torch.Tensor,
                                  stream=None) -> None:
    shp = shape_of(x, int(acc.shape[-1]))
    _check("qvae_causal_conv3d_bf16_acc32",
           lib().qvae_causal_conv3d_bf16_acc32(ctypes.byref(shp), _ptr(x), _ptr(w_packed), _ptr(acc),
                                               _stream(stream)))


def causal_conv3d_bf16(x, w_packed, bias, Cout: int, stream=None):
    out = torch.empty(tuple(x.shape[:-1]) + (Cout,), dtype=torch.bfloat16, device=x.device)
    qvae_causal_conv3d_bf16(x, w_packed, bias, out, stream)
    return out


def conv_bf16_acc32(x, w_packed, Cout: int, stream=None):
    acc = torch.empty(tuple(x.shape[:-1]) + (Cout,), dtype=torch.float32, device=x.device)
    qvae_causal_conv3d_bf16_acc32(x, w_packed, acc, stream)
    return acc


# ------------------------------------------------------------ layer chain

def make_layers(specs: Sequence[dict]):
    """specs: dicts with x, out, wq_packed, w_scale, bias (tensors), quantized (bool).

    A native-precision layer (quantized=False) carries the output of
    pack_weights_bf16 as wq_packed (the library runs it), or no weights (the
    library skips it)."""
    arr = (qvae_layer * len(specs))()
    for i, s in enumerate(specs):
        x, out = s["x"], s["out"]
        N, T, H, W, Cin = x.shape
        arr[i].shape = make_shape(N, T, H, W, Cin, out.shape[-1])
        arr[i].quantized = 1 if s.get("quantized", True) else 0
        arr[i].reserved = 0
        arr[i].x = x.data_ptr()
        arr[i].out = out.data_ptr()
        arr[i].wq_packed = s["wq_packed"].data_ptr() if s.get("wq_packed") is not None else None
        arr[i].w_scale = s["w_scale"].data_ptr() if s.get("w_scale") is not None else None
        arr[i].bias = s["bias"].data_ptr() if s.get("bias") is not None else None
    return arr


def qvae_decode_workspace_bytes(layers) -> int:
    return int(lib().qvae_decode_workspace_bytes(layers, len(layers)))


def qvae_decode_layers(layers, workspace: torch.Tensor, stream=None) -> None:
    _check("qvae_decode_layers",
           lib().qvae_decode_layers(layers, len(layers), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))


# --------------------------------- 8-bit floating-point linear layers
#
# Tensors on another device than the current one run on their own device (its
# current stream by default).  What a wrapper allocates is allocated on the
# stream that the call runs on.  Inference only, as everywhere in this library:
# no call records a gradient, and the outputs of tensors that require one do
# not.

class Fp8Weights:
    """Packed e4m3 weights of E matrices [N, K] (qvae_fp8_quantize_weights): wq, uint8 of
    qvae_fp8_packed_weight_bytes(E, N, K) bytes, and w_scale, uint8 of qvae_fp8_weight_scale_bytes(E, N, K).
    Checked here, once; the tensors are not to be resized."""

    __slots__ = ("wq", "w_scale", "E", "N", "K", "device")

    def __init__(self, wq: torch.Tensor, w_scale: torch.Tensor, E: int, N: int, K: int):
        self.wq, self.w_scale, self.E, self.N, self.K = wq, w_scale, int(E), int(N), int(K)
        self.device = _device(wq, "wq")  # index
        if self.E < 1 or self.N < 1 or self.K < 1:
            raise ValueError("E, N and K are at least 1")
        blocks = self.E * -(-self.N // 128)
        _buffer(wq, torch.uint8, blocks * -(-self.K // 128) * 16384, self.device, "wq")
        _buffer(w_scale, torch.uint8, blocks * -(-self.K // 512) * 4, self.device, "w_scale")


def _i32(v: int) -> int:
    """A size as the library takes it.  ctypes drops the bits beyond 32; sizes out of range stay out of range here, for
    the library to refuse."""
    return min(max(int(v), -2 ** 31), 2 ** 31 - 1)


def qvae_fp8_packed_weight_bytes(E: int, N: int, K: int) -> int:
    return int(lib().qvae_fp8_packed_weight_bytes(_i32(E), _i32(N), _i32(K)))


def qvae_fp8_weight_scale_bytes(E: int, N: int, K: int) -> int:
    return int(lib().qvae_fp8_weight_scale_bytes(_i32(E), _i32(N), _i32(K)))


def qvae_fp8_code_bytes(M: int, K: int) -> int:
    return int(lib().qvae_fp8_code_bytes(M, _i32(K)))


def qvae_fp8_scale_bytes(M: int, K: int) -> int:
    return int(lib().qvae_fp8_scale_bytes(M, _i32(K)))


def qvae_fp8_workspace_bytes(M: int, K: int) -> int:
    return int(lib().qvae_fp8_workspace_bytes(M, _i32(K)))


def _buffer(t: torch.Tensor, dtype: torch.dtype, count: int, device: int, name: str) -> int:
    """Address of a contiguous tensor of at least `count` elements on a device."""
    if t.get_device() != device or t.dtype != dtype or not t.is_contiguous() or t.numel() < count:
        raise ValueError(f"{name}: a contiguous {dtype} tensor of {count} elements on cuda:{device} is needed")
    return t.data_ptr()


_bf16 = torch.bfloat16


def _rows(t: torch.Tensor, columns: int, device: int, name: str):
    """(rows, elements between them) of a bf16 matrix whose columns are adjacent."""
    if t.get_device() != device or t.dtype is not _bf16 or t.dim() != 2:
        raise ValueError(f"{name}: a bf16 matrix on cuda:{device} is needed")
    m, n = t.shape
    ld, step = t.stride()
    if m < 2:
        ld = n  # (one row: its stride says nothing)
    if n != columns or ld < n or (step != 1 and n > 1):
        raise ValueError(f"{name}: rows of {columns} adjacent columns that do not overlap are needed")
    return m, ld


def _device(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is needed")
    return t.get_device()


@contextlib.contextmanager
def _elsewhere(device: int, stream):
    """A device that is not the current one, or a stream that is not its current one: the call's handle."""
    if stream is None:
        with torch.cuda.device(device):
            yield torch.cuda.current_stream().cuda_stream
        return
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream),
                                           torch.device("cuda", device))
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{device}")
    with torch.cuda.stream(stream):
        yield stream.cuda_stream


# The current stream's handle without a Stream object around it (1.3 us less a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)

# (a CUDA tensor is at hand: torch has initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(device: int, stream, call, *args):
    """call(handle, *args) on `device` and `stream` (None: the device's current stream)."""
    if stream is None and device == _current_device():
        return call(_raw_stream(device), *args)
    with _elsewhere(device, stream) as handle:
        return call(handle, *args)


def fp8_quantize_weights(w: torch.Tensor, stream=None) -> Fp8Weights:
    """Quantise and pack bf16 weights [N, K] or, one matrix to an expert, [E, N, K]: their values as they are now; later
    changes of w, an optimizer's too, do not reach the packed ones."""
    device = _device(w, "w")
    if w.dtype != torch.bfloat16 or w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w: contiguous bf16 weights [N, K] or [E, N, K] are needed")
    E, N, K = (1, *w.shape) if w.dim() == 2 else w.shape

    def call(handle):
        wq = torch.empty(qvae_fp8_packed_weight_bytes(E, N, K), dtype=torch.uint8, device=w.device)
        ws = torch.empty(qvae_fp8_weight_scale_bytes(E, N, K), dtype=torch.uint8, device=w.device)
        _check("qvae_fp8_quantize_weights",
               lib().qvae_fp8_quantize_weights(_i32(E), _i32(N), _i32(K), w.data_ptr(), wq.data_ptr(), ws.data_ptr(), handle))
        return Fp8Weights(wq, ws, E, N, K)

    return _run(device, stream, call)


def fp8_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    """Scratch of the _fused layers for M rows of K input channels."""
    return torch.empty(max(16, qvae_fp8_workspace_bytes(M, K)), dtype=torch.uint8, device=device)


def fp8_quant_act(x: torch.Tensor, silu_mul: bool = False, stream=None):
    """Codes (uint8 [ceil(K/128), M, 128]) and scale words (int32 [ceil(K/512), M]) of bf16 rows x [M, K]
    (silu_mul: [M, 2 K], of which silu(x[:, :K]) * x[:, K:] is quantised)."""
    device = _device(x, "x")
    if x.dim() != 2 or x.shape[1] < 1 or (silu_mul and x.shape[1] % 2):
        raise ValueError("x: a matrix is needed, with an even number of columns for silu_mul")
    columns = x.shape[1]
    K = columns // 2 if silu_mul else columns
    M, ld = _rows(x, columns, device, "x")

    def call(handle):
        xq = torch.empty((-(-K // 128), M, 128), dtype=torch.uint8, device=x.device)
        xs = torch.empty((-(-K // 512), M), dtype=torch.int32, device=x.device)
        _check("qvae_fp8_quant_act",
               lib().qvae_fp8_quant_act(M, _i32(K), QVAE_FP8_SILU_MUL if silu_mul else QVAE_FP8_PLAIN, x.data_ptr(), ld,
                                        xq.data_ptr(), xs.data_ptr(), handle))
        return xq, xs

    return _run(device, stream, call)


def _extras(weights: Fp8Weights, bias, offsets):
    """Addresses of the bias and the offsets (None: none), checked."""
    E, N, device = weights.E, weights.N, weights.device
    po = pb = None
    if offsets is not None:
        po = _buffer(offsets, torch.int32, E + 1, device, "offsets")
    elif E != 1:
        raise ValueError(f"the weights hold {E} experts: use the grouped product")
    if bias is not None:
        if tuple(bias.shape) != (E, N) and (E != 1 or tuple(bias.shape) != (N,)):
            raise ValueError(f"bias: [N] or [E, N] is needed, N = {N}, E = {E}")
        pb = _buffer(bias, torch.bfloat16, E * N, device, "bias")
    return pb, po


def _out(out, M: int, N: int, device: int):
    """(out, elements between its rows); a new one for None."""
    if out is None:
        return torch.empty((M, N), dtype=torch.bfloat16, device=torch.device("cuda", device)), N
    rows, ldo = _rows(out, N, device, "out")
    if rows != M:
        raise ValueError(f"out: {M} rows are needed")
    return out, ldo


def _product(handle, name, xq, x_scale, weights, bias, out, offsets):
    N, K, device = weights.N, weights.K, weights.device
    if xq.dim() != 3 or xq.shape[0] != -(-K // 128) or xq.shape[2] != 128:
        raise ValueError(f"xq: codes [{-(-K // 128)}, rows, 128] of {K} input channels are needed")
    M = xq.shape[1]
    _buffer(xq, torch.uint8, xq.numel(), device, "xq")
    groups = -(-K // 512)
    _buffer(x_scale, torch.int32, M * groups, device, "x_scale")
    if groups > 1 and x_scale.dim() > 1 and x_scale.shape[-1] != M:  # (one group: the first M words are the rows')
        raise ValueError(f"x_scale: scale words [{groups}, {M}] of the {M} rows of xq are needed")
    pb, po = _extras(weights, bias, offsets)
    out, ldo = _out(out, M, N, device)
    if po is None:
        status = lib().qvae_linear_fp8(M, N, K, xq.data_ptr(), x_scale.data_ptr(), weights.wq.data_ptr(),
                                       weights.w_scale.data_ptr(), pb, out.data_ptr(), ldo, handle)
    else:
        status = lib().qvae_linear_fp8_grouped(weights.E, M, N, K, xq.data_ptr(), x_scale.data_ptr(), po,
                                               weights.wq.data_ptr(), weights.w_scale.data_ptr(), pb, out.data_ptr(),
                                               ldo, handle)
    if status:
        _check(name, status)
    return out


def linear_fp8(xq: torch.Tensor, x_scale: torch.Tensor, weights: Fp8Weights, bias: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """bf16 [M, N] of quantised rows (fp8_quant_act) and one weight matrix.  Records no gradient."""
    return _run(weights.device, stream, _product, "qvae_linear_fp8", xq, x_scale, weights, bias, out, None)


def linear_fp8_grouped(xq: torch.Tensor, x_scale: torch.Tensor, offsets: torch.Tensor, weights: Fp8Weights,
                       bias: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """bf16 [M, N] of quantised rows sorted by expert: rows offsets[e]..offsets[e+1]-1 (int32, on the device) meet
    expert e's matrix; other rows of out are left as they are."""
    if offsets is None:
        raise ValueError("offsets: an int32 tensor is needed")
    return _run(weights.device, stream, _product, "qvae_linear_fp8_grouped", xq, x_scale, weights, bias, out, offsets)


def _fused(handle, name, x, weights, bias, silu_mul, out, workspace, offsets):
    N, K, device = weights.N, weights.K, weights.device
    M, ldx = _rows(x, 2 * K if silu_mul else K, device, "x")
    # (one layer without a bias has nothing to check there: a small layer's time is the host's, 6.5 us a call here)
    pb, po = (None, None) if bias is None and offsets is None and weights.E == 1 else _extras(weights, bias, offsets)
    out, ldo = _out(out, M, N, device)
    if workspace is None:
        workspace = fp8_workspace(M, K, x.device)
    pk = _buffer(workspace, torch.uint8, 0, device, "workspace")
    op = QVAE_FP8_SILU_MUL if silu_mul else QVAE_FP8_PLAIN
    if po is None:
        status = lib().qvae_linear_fp8_fused(M, N, K, op, x.data_ptr(), ldx, weights.wq.data_ptr(),
                                             weights.w_scale.data_ptr(), pb, out.data_ptr(), ldo, pk, workspace.numel(),
                                             handle)
    else:
        status = lib().qvae_linear_fp8_grouped_fused(weights.E, M, N, K, op, x.data_ptr(), ldx, po,
                                                     weights.wq.data_ptr(), weights.w_scale.data_ptr(), pb,
                                                     out.data_ptr(), ldo, pk, workspace.numel(), handle)
    if status:
        _check(name, status)
    return out


def linear_fp8_fused(x: torch.Tensor, weights: Fp8Weights, bias: Optional[torch.Tensor] = None, silu_mul: bool = False,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """bf16 [M, N] of bf16 rows x [M, K] (silu_mul: [M, 2 K] = [gate | up]), quantised on the way.  Records no gradient."""
    return _run(weights.device, stream, _fused, "qvae_linear_fp8_fused", x, weights, bias, silu_mul, out, workspace,
                None)


def linear_fp8_grouped_fused(x: torch.Tensor, offsets: torch.Tensor, weights: Fp8Weights,
                             bias: Optional[torch.Tensor] = None, silu_mul: bool = False,
                             out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """linear_fp8_grouped of bf16 rows, quantised on the way.  Records no gradient."""
    if offsets is None:
        raise ValueError("offsets: an int32 tensor is needed")
    return _run(weights.device, stream, _fused, "qvae_linear_fp8_grouped_fused", x, weights, bias, silu_mul, out,
                workspace, offsets)


# ---------------------------------------------------------------- control

def qvae_get_error(stream=None) -> int:
    return int(lib().qvae_get_error(_stream(stream)))


def qvae_set_wait_limit_ns(limit_ns: int) -> None:
    _check("qvae_set_wait_limit_ns", lib().qvae_set_wait_limit_ns(int(limit_ns)))


def qvae_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    _check("qvae_selftest_wait_timeout", lib().qvae_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def qvae_set_conv_tiling(MS=0, NT=0, SA=0, SB=0, mode=0, G=0) -> None:
    _check("qvae_set_conv_tiling", lib().qvae_set_conv_tiling(MS, NT, SA, SB, mode, G))


def qvae_set_fused_quant(on: int = 0) -> None:
    _check("qvae_set_fused_quant", lib().qvae_set_fused_quant(int(on)))


def qvae_set_conv_cta_limit(max_ctas: int = 0) -> None:
    _check("qvae_set_conv_cta_limit", lib().qvae_set_conv_cta_limit(int(max_ctas)))


def qvae_get_conv_tiling(N, T, H, W, Cin, Cout, variant: int = 0) -> dict:
    """variant 0: convolution of INT8 codes; 1: fused (bf16 input quantised in the kernel); 2: native bf16."""
    shp = make_shape(N, T, H, W, Cin, Cout)
    out = (ctypes.c_int32 * 8)()
    _check("qvae_get_conv_tiling", lib().qvae_get_conv_tiling(ctypes.byref(shp), int(variant), out))
    return dict(zip(("MS", "NT", "SA", "SB", "acc_buffers", "ctas", "mode", "G"), list(out)))


def qvae_set_linear_tiling(NT=0, mode=0, split=0, max_ctas=0) -> None:
    _check("qvae_set_linear_tiling", lib().qvae_set_linear_tiling(_i32(NT), _i32(mode), _i32(split), _i32(max_ctas)))


def qvae_get_linear_tiling(E, M, N, K) -> dict:
    """E = 0: a single layer; else grouped by E experts."""
    out = (ctypes.c_int32 * 3)()
    _check("qvae_get_linear_tiling", lib().qvae_get_linear_tiling(_i32(E), M, _i32(N), _i32(K), out))
    return dict(zip(("NT", "mode", "split"), list(out)))


def qvae_get_linear_footprint(E, M, N, K, fused=True) -> dict:
    """What a CTA of that product takes: bytes of shared memory, TMEM columns, CTAs of its cluster."""
    out = (ctypes.c_int32 * 3)()
    _check("qvae_get_linear_footprint", lib().qvae_get_linear_footprint(_i32(E), M, _i32(N), _i32(K), 1 if fused else 0, out))
    return dict(zip(("smem", "tmem_cols", "cluster"), list(out)))
