"""ctypes binding of libqs.so.

The functions named like the C entry points (``qs_pack_weights``,
``qs_quant_act``, ``qs_qlinear``, ``qs_qlinear_mixed``, ``qs_qgemm_s32``,
``qs_gelu_bf16``, ...) take torch
CUDA tensors and only marshal their pointers, sizes and the stream into the C
call; every step of the computation runs in the library's kernels.  The
lower-case helpers (``pack_weights``, ``quant_act``, ``qlinear``, ...) allocate
the output tensors with torch and call those.

There is no fallback: if libqs.so has not been built, or a call returns an
error status, a ``QSError`` is raised.
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqs.so")

QS_FLAG_NO_ROTATE = 1
QS_FLAG_BYTE_CODES = 2
QS_MAX_K = 65536
STATUS = {0: "QS_OK", 1: "QS_ERR_NULL", 2: "QS_ERR_SHAPE", 3: "QS_ERR_BITS", 4: "QS_ERR_ALIGN",
          5: "QS_ERR_RANGE", 6: "QS_ERR_CUDA", 7: "QS_ERR_TIMEOUT", 8: "QS_ERR_PTR",
          9: "QS_ERR_DTYPE", 10: "QS_ERR_OVERLAP"}
EXPORTS = ("qs_pack_weights", "qs_quant_act", "qs_qlinear", "qs_qlinear_mixed", "qs_qgemm_s32",
           "qs_qgemm_s32_mixed", "qs_gelu_bf16", "qs_linear_workspace_bytes", "qs_linear",
           "qs_linear_mixed", "qs_linear_ex", "qs_linear_noalloc", "qs_pack_weights_bgr",
           "qs_quant_act_rowsum", "qs_qlinear_asym", "qs_qgemm_s32_asym",
           "qs_linear_bgr_workspace_bytes", "qs_linear_bgr", "qs_sd4_quant", "qs_sd4_quant_e4m3",
           "qs_sd4_linear", "qs_sd4_decode", "qs_sd4_linear_wdec", "qs_sd4_decode_e4m3",
           "qs_sd4_linear_e4m3w", "qs_sd4_linear_e4m3", "qs_sd4_scale_tiles_bytes",
           "qs_sd4_scale_tiles", "qs_sd4_linear_e4m3_tiles", "qs_sd4_quant_decomp",
           "qs_sd4_linear_decomp", "qs_gbs_reset", "qs_gbs_update", "qs_linear_gbs",
           "qs_selftest_timeout", "qs_device_error", "qs_status_str", "qs_version", "qs_rope",
           "qs_lora_workspace_bytes", "qs_lora_add", "qs_block_means",
           "qs_block_select_workspace_bytes", "qs_block_select",
           "qs_block_attention_workspace_bytes", "qs_block_attention")
QS_ROPE_INTERLEAVED, QS_ROPE_INVERSE = 1, 2
QS_ATTN_CAUSAL = 1
QS_BLOCK_Q, QS_BLOCK_K = 128, 64
QS_BF16, QS_F16, QS_F32 = 0, 1, 2
_DTYPES = {torch.bfloat16: QS_BF16, torch.float16: QS_F16, torch.float32: QS_F32}
BITS = (4, 6, 8)
QS_GBS_MAX_BLOCKS = 1024
# sizeof(qs_gbs_state): acc, last_d (f64), bits, step, blocks_done, reserved (i32), partials
QS_GBS_STATE_BYTES = 8 + 8 + 4 * 4 + 2 * QS_GBS_MAX_BLOCKS * 8
QS_NOALLOC_SCRATCH_BYTES = 8 << 20


class _Strides(ctypes.Structure):
    """qs_strides: strides of a [batch, row, head, dim] view in elements."""
    _fields_ = [("batch", ctypes.c_int64), ("row", ctypes.c_int64), ("head", ctypes.c_int64)]


class QSError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({_status_str(status)})")


_lib = None


def load() -> ctypes.CDLL:
    """Loads libqs.so (once) and declares the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m bit_quantized_linear_hadamard_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, u32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint, ctypes.c_float
    L.qs_pack_weights.argtypes = [vp, i64, i64, i32, u32, vp, vp, vp]
    L.qs_quant_act.argtypes = [vp, i64, i64, i32, f32, u32, vp, vp, vp]
    L.qs_qlinear.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, vp]
    L.qs_qlinear_mixed.argtypes = [vp, vp, i32, vp, vp, i32, vp, i64, i64, i64, vp, vp]
    L.qs_qgemm_s32.argtypes = [vp, vp, i64, i64, i64, i32, vp, vp]
    L.qs_qgemm_s32_mixed.argtypes = [vp, i32, vp, i32, i64, i64, i64, vp, vp]
    L.qs_gelu_bf16.argtypes = [vp, i64, vp, vp]
    L.qs_linear_workspace_bytes.argtypes = [i64, i64, i32]
    L.qs_linear_workspace_bytes.restype = i64
    L.qs_linear.argtypes = [vp, i64, i64, f32, vp, vp, vp, i64, i32, vp, i64, vp, vp]
    L.qs_linear_mixed.argtypes = [vp, i64, i64, f32, i32, vp, vp, i32, vp, i64, vp, i64, vp, vp]
    L.qs_linear_ex.argtypes = [vp, i64, i64, f32, i32, u32, vp, vp, i32, vp, i64, vp, i64, vp, vp]
    L.qs_linear_noalloc.argtypes = [vp, i64, i64, f32, vp, vp, vp, i64, i32, vp, vp]
    f64 = ctypes.c_double
    L.qs_pack_weights_bgr.argtypes = [vp, i64, i64, i32, u32, i32, i32, vp, vp, vp, vp]
    L.qs_quant_act_rowsum.argtypes = [vp, i64, i64, i32, f32, u32, vp, vp, vp, vp]
    L.qs_qlinear_asym.argtypes = [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, vp]
    L.qs_qgemm_s32_asym.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, vp]
    L.qs_linear_bgr_workspace_bytes.argtypes = [i64, i64, i32]
    L.qs_linear_bgr_workspace_bytes.restype = i64
    L.qs_linear_bgr.argtypes = [vp, i64, i64, f32, vp, vp, vp, vp, i64, i32, vp, i64, vp, vp]
    L.qs_sd4_quant.argtypes = [vp, i64, i64, vp, vp, vp]
    L.qs_sd4_linear.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.qs_sd4_decode.argtypes = [vp, vp, i64, i64, vp, vp]
    L.qs_sd4_linear_wdec.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.qs_sd4_quant_decomp.argtypes = [vp, i64, i64, vp, i64, vp, vp, vp]
    L.qs_sd4_linear_decomp.argtypes = [vp, vp, vp, i64, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.qs_sd4_decode_e4m3.argtypes = [vp, vp, i64, i64, vp, vp]
    L.qs_sd4_linear_e4m3w.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.qs_sd4_quant_e4m3.argtypes = [vp, i64, i64, vp, vp, vp]
    L.qs_sd4_linear_e4m3.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.qs_sd4_scale_tiles_bytes.argtypes = [i64, i64, i32]
    L.qs_sd4_scale_tiles_bytes.restype = i64
    L.qs_sd4_scale_tiles.argtypes = [vp, i64, i64, i32, vp, i64, vp]
    L.qs_sd4_linear_e4m3_tiles.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp]
    L.qs_gbs_reset.argtypes = [vp, vp]
    L.qs_gbs_update.argtypes = [vp, vp, i64, f64, vp, vp]
    L.qs_linear_gbs.argtypes = [vp, i64, i64, f32, vp, vp, vp, vp, vp, i64, vp, vp, i64, vp, vp]
    st = ctypes.POINTER(_Strides)
    L.qs_rope.argtypes = [vp, i64, i64, i64, i64, i64, i64, vp, i32, vp, vp, f64, u32, i32, vp, i64,
                          i64, vp]
    L.qs_lora_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.qs_lora_workspace_bytes.restype = i64
    L.qs_lora_add.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, i64, i64, vp, vp, i64, vp, i64, vp,
                              vp]
    L.qs_block_means.argtypes = [vp, st, i64, i64, i64, i64, i32, vp, i64, vp, vp]
    L.qs_block_select_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.qs_block_select_workspace_bytes.restype = i64
    L.qs_block_select.argtypes = [vp, st, i64, i64, i64, i64, i32, vp, i64, i64, vp, vp, i64, i64,
                                  i64, u32, vp, i64, vp, vp]
    L.qs_block_attention_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    L.qs_block_attention_workspace_bytes.restype = i64
    L.qs_block_attention.argtypes = [vp, st, vp, st, vp, st, i64, i64, i64, i64, i64, i64, i32, vp,
                                     i64, vp, vp, f32, u32, vp, i64, vp, st, vp, vp]
    L.qs_selftest_timeout.argtypes = [i64, vp]
    L.qs_device_error.argtypes = [vp]
    L.qs_status_str.argtypes = [i32]
    L.qs_status_str.restype = ctypes.c_char_p
    L.qs_version.restype = ctypes.c_char_p
    for name in ("qs_pack_weights", "qs_quant_act", "qs_qlinear", "qs_qlinear_mixed",
                 "qs_qgemm_s32", "qs_qgemm_s32_mixed", "qs_gelu_bf16", "qs_linear",
                 "qs_linear_mixed", "qs_linear_ex", "qs_linear_noalloc", "qs_pack_weights_bgr",
                 "qs_quant_act_rowsum", "qs_qlinear_asym", "qs_qgemm_s32_asym", "qs_linear_bgr",
                 "qs_sd4_quant", "qs_sd4_quant_e4m3", "qs_sd4_linear", "qs_sd4_decode",
                 "qs_sd4_linear_wdec", "qs_sd4_decode_e4m3", "qs_sd4_linear_e4m3w",
                 "qs_sd4_linear_e4m3", "qs_sd4_scale_tiles", "qs_sd4_linear_e4m3_tiles",
                 "qs_sd4_quant_decomp", "qs_sd4_linear_decomp",
                 "qs_gbs_reset", "qs_gbs_update", "qs_linear_gbs", "qs_selftest_timeout",
                 "qs_device_error", "qs_rope", "qs_lora_add", "qs_block_means", "qs_block_select",
                 "qs_block_attention"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _status_str(status: int) -> str:
    try:
        return load().qs_status_str(status).decode()
    except Exception:  # noqa: BLE001 - only used to decorate an error message
        return "?"


def _check(status: int, where: str) -> None:
    if status != 0:
        raise QSError(status, where)


def _p(t):
    return None if t is None else t.data_ptr()


# torch.cuda.current_stream(device).cuda_stream without the objects around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream):
    if stream is None:
        device = torch.cuda.current_device()  # initialises CUDA, or says why it cannot
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _cuda(t, dtype, name):
    if t is None:
        return
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# --------------------------------------------------------------------------- C mirrors

def qs_pack_weights(w, N, K, bits, flags, w_packed, w_scale, stream=None):
    _cuda(w, torch.bfloat16, "w")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(w_scale, torch.float32, "w_scale")
    _check(load().qs_pack_weights(_p(w), N, K, bits, flags, _p(w_packed), _p(w_scale), _s(stream)),
           "qs_pack_weights")


def qs_quant_act(x, M, K, bits, alpha, flags, x_packed, x_scale, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(x_packed, torch.uint8, "x_packed")
    _cuda(x_scale, torch.float32, "x_scale")
    _check(load().qs_quant_act(_p(x), M, K, bits, float(alpha), flags, _p(x_packed), _p(x_scale),
                               _s(stream)), "qs_quant_act")


def qs_qlinear(x_packed, x_scale, w_packed, w_scale, bias, M, N, K, bits, out, stream=None):
    _cuda(x_packed, torch.uint8, "x_packed")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(x_scale, torch.float32, "x_scale")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_qlinear(_p(x_packed), _p(x_scale), _p(w_packed), _p(w_scale), _p(bias),
                             M, N, K, bits, _p(out), _s(stream)), "qs_qlinear")


def qs_qlinear_mixed(x_packed, x_scale, bits_x, w_packed, w_scale, bits_w, bias, M, N, K, out,
                     stream=None):
    _cuda(x_packed, torch.uint8, "x_packed")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(x_scale, torch.float32, "x_scale")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_qlinear_mixed(_p(x_packed), _p(x_scale), bits_x, _p(w_packed), _p(w_scale),
                                   bits_w, _p(bias), M, N, K, _p(out), _s(stream)),
           "qs_qlinear_mixed")


def qs_qgemm_s32_mixed(x_packed, bits_x, w_packed, bits_w, M, N, K, acc, stream=None):
    _cuda(x_packed, torch.uint8, "x_packed")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(acc, torch.int32, "acc")
    _check(load().qs_qgemm_s32_mixed(_p(x_packed), bits_x, _p(w_packed), bits_w, M, N, K, _p(acc),
                                     _s(stream)), "qs_qgemm_s32_mixed")


def qs_qgemm_s32(x_packed, w_packed, M, N, K, bits, acc, stream=None):
    _cuda(x_packed, torch.uint8, "x_packed")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(acc, torch.int32, "acc")
    _check(load().qs_qgemm_s32(_p(x_packed), _p(w_packed), M, N, K, bits, _p(acc), _s(stream)),
           "qs_qgemm_s32")


def qs_gelu_bf16(x, n, y, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(y, torch.bfloat16, "y")
    _check(load().qs_gelu_bf16(_p(x), n, _p(y), _s(stream)), "qs_gelu_bf16")


def qs_linear_workspace_bytes(M, K, bits) -> int:
    return int(load().qs_linear_workspace_bytes(M, K, bits))


def qs_linear(x, M, K, alpha, w_packed, w_scale, bias, N, bits, workspace, workspace_bytes, out,
              stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(workspace, torch.uint8, "workspace")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_linear(_p(x), M, K, float(alpha), _p(w_packed), _p(w_scale), _p(bias), N, bits,
                            _p(workspace), workspace_bytes, _p(out), _s(stream)), "qs_linear")


def qs_linear_mixed(x, M, K, alpha, bits_x, w_packed, w_scale, bits_w, bias, N, workspace,
                    workspace_bytes, out, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(workspace, torch.uint8, "workspace")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_linear_mixed(_p(x), M, K, float(alpha), bits_x, _p(w_packed), _p(w_scale),
                                  bits_w, _p(bias), N, _p(workspace), workspace_bytes, _p(out),
                                  _s(stream)), "qs_linear_mixed")


def qs_linear_ex(x, M, K, alpha, bits_x, x_flags, w_packed, w_scale, bits_w, bias, N, workspace,
                 workspace_bytes, out, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(workspace, torch.uint8, "workspace")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_linear_ex(_p(x), M, K, float(alpha), bits_x, x_flags, _p(w_packed),
                               _p(w_scale), bits_w, _p(bias), N, _p(workspace), workspace_bytes,
                               _p(out), _s(stream)), "qs_linear_ex")


def qs_linear_noalloc(x, M, K, alpha, w_packed, w_scale, bias, N, bits, out, stream=None):
    """qs_linear on the library's own fixed scratch buffer (for callers that
    cannot allocate device memory when they run the layer); nothing is allocated."""
    _cuda(x, torch.bfloat16, "x")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_linear_noalloc(_p(x), M, K, float(alpha), _p(w_packed), _p(w_scale), _p(bias),
                                    N, bits, _p(out), _s(stream)), "qs_linear_noalloc")


def qs_pack_weights_bgr(w, N, K, bits, flags, candidates, iterations, w_packed, w_scale,
                        w_offset, stream=None):
    _cuda(w, torch.bfloat16, "w")
    _cuda(w_packed, torch.uint8, "w_packed")
    _cuda(w_scale, torch.float32, "w_scale")
    _cuda(w_offset, torch.int32, "w_offset")
    _check(load().qs_pack_weights_bgr(_p(w), N, K, bits, flags, candidates, iterations,
                                      _p(w_packed), _p(w_scale), _p(w_offset), _s(stream)),
           "qs_pack_weights_bgr")


def qs_quant_act_rowsum(x, M, K, bits, alpha, flags, x_packed, x_scale, x_rowsum, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(x_packed, torch.uint8, "x_packed")
    _cuda(x_scale, torch.float32, "x_scale")
    _cuda(x_rowsum, torch.int32, "x_rowsum")
    _check(load().qs_quant_act_rowsum(_p(x), M, K, bits, float(alpha), flags, _p(x_packed),
                                      _p(x_scale), _p(x_rowsum), _s(stream)),
           "qs_quant_act_rowsum")


def qs_qlinear_asym(x_packed, x_scale, x_rowsum, w_packed, w_scale, w_offset, bias, M, N, K,
                    bits, out, stream=None):
    for t, name, dt in ((x_packed, "x_packed", torch.uint8), (w_packed, "w_packed", torch.uint8),
                        (x_scale, "x_scale", torch.float32), (w_scale, "w_scale", torch.float32),
                        (x_rowsum, "x_rowsum", torch.int32), (w_offset, "w_offset", torch.int32),
                        (bias, "bias", torch.bfloat16), (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_qlinear_asym(_p(x_packed), _p(x_scale), _p(x_rowsum), _p(w_packed),
                                  _p(w_scale), _p(w_offset), _p(bias), M, N, K, bits, _p(out),
                                  _s(stream)), "qs_qlinear_asym")


def qs_qgemm_s32_asym(x_packed, x_rowsum, w_packed, w_offset, M, N, K, bits, acc, stream=None):
    for t, name, dt in ((x_packed, "x_packed", torch.uint8), (w_packed, "w_packed", torch.uint8),
                        (x_rowsum, "x_rowsum", torch.int32), (w_offset, "w_offset", torch.int32),
                        (acc, "acc", torch.int32)):
        _cuda(t, dt, name)
    _check(load().qs_qgemm_s32_asym(_p(x_packed), _p(x_rowsum), _p(w_packed), _p(w_offset), M, N,
                                    K, bits, _p(acc), _s(stream)), "qs_qgemm_s32_asym")


def qs_linear_bgr_workspace_bytes(M, K, bits) -> int:
    return int(load().qs_linear_bgr_workspace_bytes(M, K, bits))


def qs_linear_bgr(x, M, K, alpha, w_packed, w_scale, w_offset, bias, N, bits, workspace,
                  workspace_bytes, out, stream=None):
    for t, name, dt in ((x, "x", torch.bfloat16), (w_packed, "w_packed", torch.uint8),
                        (w_scale, "w_scale", torch.float32), (w_offset, "w_offset", torch.int32),
                        (bias, "bias", torch.bfloat16), (workspace, "workspace", torch.uint8),
                        (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_linear_bgr(_p(x), M, K, float(alpha), _p(w_packed), _p(w_scale),
                                _p(w_offset), _p(bias), N, bits, _p(workspace), workspace_bytes,
                                _p(out), _s(stream)), "qs_linear_bgr")


def qs_sd4_quant(x, rows, K, codes, meta, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(codes, torch.uint8, "codes")
    _cuda(meta, torch.int16, "meta")
    _check(load().qs_sd4_quant(_p(x), rows, K, _p(codes), _p(meta), _s(stream)), "qs_sd4_quant")


def qs_sd4_linear(x_codes, x_meta, w_codes, w_meta, bias, M, N, K, out, stream=None):
    for t, name, dt in ((x_codes, "x_codes", torch.uint8), (w_codes, "w_codes", torch.uint8),
                        (x_meta, "x_meta", torch.int16), (w_meta, "w_meta", torch.int16),
                        (bias, "bias", torch.bfloat16), (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_sd4_linear(_p(x_codes), _p(x_meta), _p(w_codes), _p(w_meta), _p(bias), M, N,
                                K, _p(out), _s(stream)), "qs_sd4_linear")


def sd4_linear(x_codes, x_meta, w_codes, w_meta, bias, K: int, stream=None, out=None):
    M, N = x_codes.shape[0], w_codes.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x_codes.device)
    qs_sd4_linear(x_codes, x_meta, w_codes, w_meta, bias, M, N, K, out, stream)
    return out


def qs_sd4_decode(codes, meta, rows, K, out, stream=None):
    _cuda(codes, torch.uint8, "codes")
    _cuda(meta, torch.int16, "meta")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_sd4_decode(_p(codes), _p(meta), rows, K, _p(out), _s(stream)), "qs_sd4_decode")


def qs_sd4_linear_wdec(x_codes, x_meta, w, bias, M, N, K, out, stream=None):
    for t, name, dt in ((x_codes, "x_codes", torch.uint8), (x_meta, "x_meta", torch.int16),
                        (w, "w", torch.bfloat16), (bias, "bias", torch.bfloat16),
                        (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_sd4_linear_wdec(_p(x_codes), _p(x_meta), _p(w), _p(bias), M, N, K, _p(out),
                                     _s(stream)), "qs_sd4_linear_wdec")


def sd4_decode(codes, meta, stream=None):
    R, K = codes.shape[0], codes.shape[1] * 2
    out = torch.empty((R, K), dtype=torch.bfloat16, device=codes.device)
    qs_sd4_decode(codes, meta, R, K, out, stream)
    return out


def sd4_quant(x: torch.Tensor, stream=None):
    """x bf16 [R, K] -> (codes uint8 [R, K/2], meta int16 [R, K/32]: e | d << 8)."""
    R, K = x.shape
    codes = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
    meta = torch.empty((R, K // 32), dtype=torch.int16, device=x.device)
    qs_sd4_quant(x, R, K, codes, meta, stream)
    return codes, meta


def qs_sd4_quant_decomp(x, M, K, rows, S, codes2, meta2, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(rows, torch.int32, "rows")
    _cuda(codes2, torch.uint8, "codes2")
    _cuda(meta2, torch.int16, "meta2")
    _check(load().qs_sd4_quant_decomp(_p(x), M, K, _p(rows), S, _p(codes2), _p(meta2),
                                      _s(stream)), "qs_sd4_quant_decomp")


def qs_sd4_linear_decomp(codes2, meta2, rows, S, w_codes, w_meta, w_e4m3, bias, M, N, K, out,
                         stream=None):
    for t, name, dt in ((codes2, "codes2", torch.uint8), (meta2, "meta2", torch.int16),
                        (rows, "rows", torch.int32), (w_codes, "w_codes", torch.uint8),
                        (w_meta, "w_meta", torch.int16), (w_e4m3, "w_e4m3", torch.uint8),
                        (bias, "bias", torch.bfloat16), (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_sd4_linear_decomp(_p(codes2), _p(meta2), _p(rows), S, _p(w_codes),
                                       _p(w_meta), _p(w_e4m3), _p(bias), M, N, K, _p(out),
                                       _s(stream)), "qs_sd4_linear_decomp")


def qs_sd4_decode_e4m3(codes, meta, rows, K, out, stream=None):
    _cuda(codes, torch.uint8, "codes")
    _cuda(meta, torch.int16, "meta")
    _cuda(out, torch.uint8, "out")
    _check(load().qs_sd4_decode_e4m3(_p(codes), _p(meta), rows, K, _p(out), _s(stream)),
           "qs_sd4_decode_e4m3")


def sd4_decode_e4m3(codes, meta, stream=None):
    """SD4 codes [R, K/2] + block words -> e4m3 bytes uint8 [R, K] (the block
    scales stay in the words)."""
    R, K = codes.shape[0], codes.shape[1] * 2
    out = torch.empty((R, K), dtype=torch.uint8, device=codes.device)
    qs_sd4_decode_e4m3(codes, meta, R, K, out, stream)
    return out


def qs_sd4_linear_e4m3w(x_codes, x_meta, w_e4m3, w_meta, bias, M, N, K, out, stream=None):
    for t, name, dt in ((x_codes, "x_codes", torch.uint8), (x_meta, "x_meta", torch.int16),
                        (w_e4m3, "w_e4m3", torch.uint8), (w_meta, "w_meta", torch.int16),
                        (bias, "bias", torch.bfloat16), (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_sd4_linear_e4m3w(_p(x_codes), _p(x_meta), _p(w_e4m3), _p(w_meta), _p(bias),
                                      M, N, K, _p(out), _s(stream)), "qs_sd4_linear_e4m3w")


def sd4_quant_decomp(x: torch.Tensor, rows: torch.Tensor, stream=None):
    """Salient rows `rows` (int32 [S]) of x bf16 [M, K] -> (codes2 uint8 [S, K],
    meta2 int16 [S, K/16]): [Q(x) | Q(x - x_hat)] per row."""
    M, K = x.shape
    S = rows.shape[0]
    codes2 = torch.empty((S, K), dtype=torch.uint8, device=x.device)
    meta2 = torch.empty((S, K // 16), dtype=torch.int16, device=x.device)
    qs_sd4_quant_decomp(x, M, K, rows, S, codes2, meta2, stream)
    return codes2, meta2


def sd4_linear_decomp(x_codes, x_meta, codes2, meta2, rows, w_codes, w_meta, bias, K: int,
                      w_e4m3=None, stream=None, out=None):
    """The SD4 layer with the salient rows decomposed: qs_sd4_linear (or the
    e4m3-weight form when w_e4m3 is given) over all rows, then
    qs_sd4_linear_decomp over the salient ones."""
    M, N = x_codes.shape[0], w_meta.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x_codes.device)
    if w_e4m3 is not None:
        qs_sd4_linear_e4m3w(x_codes, x_meta, w_e4m3, w_meta, bias, M, N, K, out, stream)
    else:
        qs_sd4_linear(x_codes, x_meta, w_codes, w_meta, bias, M, N, K, out, stream)
    qs_sd4_linear_decomp(codes2, meta2, rows, rows.shape[0],
                         None if w_e4m3 is not None else w_codes, w_meta, w_e4m3, bias, M, N, K,
                         out, stream)
    return out


def qs_sd4_quant_e4m3(x, rows, K, out, meta, stream=None):
    _cuda(x, torch.bfloat16, "x")
    _cuda(out, torch.uint8, "out")
    _cuda(meta, torch.int16, "meta")
    _check(load().qs_sd4_quant_e4m3(_p(x), rows, K, _p(out), _p(meta), _s(stream)),
           "qs_sd4_quant_e4m3")


def sd4_quant_e4m3(x: torch.Tensor, stream=None):
    """x bf16 [R, K] -> (e4m3 bytes uint8 [R, K], meta int16 [R, K/32])."""
    R, K = x.shape
    out = torch.empty((R, K), dtype=torch.uint8, device=x.device)
    meta = torch.empty((R, K // 32), dtype=torch.int16, device=x.device)
    qs_sd4_quant_e4m3(x, R, K, out, meta, stream)
    return out, meta


def qs_sd4_linear_e4m3(x_e4m3, x_meta, w_e4m3, w_meta, bias, M, N, K, out, stream=None):
    for t, name, dt in ((x_e4m3, "x_e4m3", torch.uint8), (x_meta, "x_meta", torch.int16),
                        (w_e4m3, "w_e4m3", torch.uint8), (w_meta, "w_meta", torch.int16),
                        (bias, "bias", torch.bfloat16), (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_sd4_linear_e4m3(_p(x_e4m3), _p(x_meta), _p(w_e4m3), _p(w_meta), _p(bias),
                                     M, N, K, _p(out), _s(stream)), "qs_sd4_linear_e4m3")


def qs_sd4_scale_tiles_bytes(rows: int, K: int, weights: int) -> int:
    return int(load().qs_sd4_scale_tiles_bytes(rows, K, weights))


def qs_sd4_scale_tiles(meta, rows, K, weights, tiles, stream=None):
    _cuda(meta, torch.int16, "meta")
    _cuda(tiles, torch.uint8, "tiles")
    _check(load().qs_sd4_scale_tiles(_p(meta), rows, K, weights, _p(tiles), tiles.numel(),
                                     _s(stream)), "qs_sd4_scale_tiles")


def sd4_scale_tiles(meta: torch.Tensor, weights: bool, stream=None) -> torch.Tensor:
    """Block words [rows, K/32] -> the GEMM's pre-arranged scale tiles (uint8)."""
    rows, K = meta.shape[0], meta.shape[1] * 32
    need = qs_sd4_scale_tiles_bytes(rows, K, int(weights))
    if need < 0:
        raise QSError(2, f"qs_sd4_scale_tiles_bytes({rows}, {K})")
    tiles = torch.empty((need,), dtype=torch.uint8, device=meta.device)
    qs_sd4_scale_tiles(meta, rows, K, int(weights), tiles, stream)
    return tiles


def qs_sd4_linear_e4m3_tiles(x_e4m3, x_tiles, w_e4m3, w_tiles, bias, M, N, K, out, stream=None):
    for t, name, dt in ((x_e4m3, "x_e4m3", torch.uint8), (x_tiles, "x_tiles", torch.uint8),
                        (w_e4m3, "w_e4m3", torch.uint8), (w_tiles, "w_tiles", torch.uint8),
                        (bias, "bias", torch.bfloat16), (out, "out", torch.bfloat16)):
        _cuda(t, dt, name)
    _check(load().qs_sd4_linear_e4m3_tiles(_p(x_e4m3), _p(x_tiles), _p(w_e4m3), _p(w_tiles),
                                           _p(bias), M, N, K, _p(out), _s(stream)),
           "qs_sd4_linear_e4m3_tiles")


def qs_gbs_reset(state, stream=None):
    _cuda(state, torch.uint8, "state")
    _check(load().qs_gbs_reset(_p(state), _s(stream)), "qs_gbs_reset")


def qs_gbs_update(y_cur, y_prev, n, delta, state, stream=None):
    _cuda(y_cur, torch.bfloat16, "y_cur")
    _cuda(y_prev, torch.bfloat16, "y_prev")
    _cuda(state, torch.uint8, "state")
    _check(load().qs_gbs_update(_p(y_cur), _p(y_prev), n, float(delta), _p(state), _s(stream)),
           "qs_gbs_update")


def qs_linear_gbs(x, M, K, alpha, w4_packed, w4_scale, w8_packed, w8_scale, bias, N, state,
                  workspace, workspace_bytes, out, stream=None):
    _cuda(x, torch.bfloat16, "x")
    for t, name in ((w4_packed, "w4_packed"), (w8_packed, "w8_packed"), (state, "state"),
                    (workspace, "workspace")):
        _cuda(t, torch.uint8, name)
    _cuda(w4_scale, torch.float32, "w4_scale")
    _cuda(w8_scale, torch.float32, "w8_scale")
    _cuda(bias, torch.bfloat16, "bias")
    _cuda(out, torch.bfloat16, "out")
    _check(load().qs_linear_gbs(_p(x), M, K, float(alpha), _p(w4_packed), _p(w4_scale),
                                _p(w8_packed), _p(w8_scale), _p(bias), N, _p(state),
                                _p(workspace), workspace_bytes, _p(out), _s(stream)),
           "qs_linear_gbs")


_16BIT = (torch.bfloat16, torch.float16)


def _view(t, name, dtypes=_16BIT, dims=4):
    """A CUDA view of `dims` dimensions whose last one is contiguous; its strides."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {', '.join(map(str, dtypes))}, got {t.dtype}")
    st = t.stride()
    if len(st) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {len(st)}")
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return st


def _shape(t, shape, name):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must be of shape {tuple(shape)}, got {tuple(t.shape)}")


_ROPE_DTYPES = tuple(_DTYPES)


def qs_rope(x, positions, inv_freq, y, pair_axis=None, scale=1.0, flags=0, stream=None):
    """x, y: [rows, heads, head_dim] views (y may be x); sizes and strides are theirs."""
    xs = _view(x, "x", _ROPE_DTYPES, 3)
    ys = xs if y is x else _view(y, "y", (x.dtype,), 3)
    _shape(y, x.shape, "y")
    _cuda(positions, torch.int64, "positions")
    _cuda(inv_freq, torch.float64, "inv_freq")
    _cuda(pair_axis, torch.int32, "pair_axis")
    rows, heads, dim = x.shape
    ps = positions.shape
    if len(ps) not in (1, 2) or ps[0] != rows:
        raise ValueError("positions must be [rows] or [rows, axes]")
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be [rot_dim / 2]")
    _shape(pair_axis, inv_freq.shape, "pair_axis")
    _check(load().qs_rope(_p(x), xs[0], xs[1], rows, heads, dim, 2 * inv_freq.numel(), _p(positions),
                          ps[1] if len(ps) == 2 else 1, _p(pair_axis), _p(inv_freq), scale, flags,
                          _DTYPES[x.dtype], _p(y), ys[0], ys[1], _s(stream)), "qs_rope")


def qs_lora_workspace_bytes(M, K, R, requests) -> int:
    return int(load().qs_lora_workspace_bytes(M, K, R, requests))


def qs_lora_add(x, y, M, K, N, a, b, scale, adapters, R, seg_start, seg_adapter, requests,
                workspace, workspace_bytes, out, stream=None):
    for t, name in ((x, "x"), (y, "y"), (a, "a"), (b, "b"), (out, "out")):
        _cuda(t, torch.bfloat16, name)
    _cuda(scale, torch.float32, "scale")
    _cuda(seg_start, torch.int32, "seg_start")
    _cuda(seg_adapter, torch.int32, "seg_adapter")
    _cuda(workspace, torch.uint8, "workspace")
    _check(load().qs_lora_add(_p(x), _p(y), M, K, N, _p(a), _p(b), _p(scale), adapters, R,
                              _p(seg_start), _p(seg_adapter), requests, _p(workspace),
                              workspace_bytes, _p(out), _s(stream)), "qs_lora_add")


def qs_block_means(x, lens, first_block, means, stream=None):
    """x: [B, L, H, D] view; means: float32 [B, H, ceil(L / 64), D]."""
    xs = _view(x, "x")
    B, L, H, D = x.shape
    _cuda(means, torch.float32, "means")
    _shape(means, (B, H, -(-L // QS_BLOCK_K), D), "means")
    _cuda(lens, torch.int32, "lens")
    _shape(lens, (B,), "lens")
    _check(load().qs_block_means(_p(x), _Strides(*xs[:3]), B, L, H, D, _DTYPES[x.dtype], _p(lens),
                                 first_block, _p(means), _s(stream)), "qs_block_means")


def qs_block_select_workspace_bytes(B, Lq, Hq, D) -> int:
    return int(load().qs_block_select_workspace_bytes(B, Lq, Hq, D))


def qs_block_select(q, means, Lk, q_len, k_len, T, keep_first, keep_last, flags, workspace, blocks,
                    stream=None):
    """q: [B, Lq, Hq, D] view; means: float32 [B, Hkv, ceil(Lk / 64), D]; blocks: int32
    [B, Hq, ceil(Lq / 128), T]."""
    st = _view(q, "q")
    B, Lq, Hq, D = q.shape
    _cuda(means, torch.float32, "means")
    if means.dim() != 4:
        raise ValueError("means must be [B, Hkv, blocks, D]")
    Hkv = means.shape[1]
    _shape(means, (B, Hkv, -(-Lk // QS_BLOCK_K), D), "means")
    _cuda(blocks, torch.int32, "blocks")
    _shape(blocks, (B, Hq, -(-Lq // QS_BLOCK_Q), T), "blocks")
    _cuda(workspace, torch.uint8, "workspace")
    for t, name in ((q_len, "q_len"), (k_len, "k_len")):
        if t is not None:
            _cuda(t, torch.int32, name)
            _shape(t, (B,), name)
    _check(load().qs_block_select(_p(q), _Strides(*st[:3]), B, Lq, Hq, D, _DTYPES[q.dtype],
                                  _p(means), Lk, Hkv, _p(q_len), _p(k_len), T, keep_first, keep_last,
                                  flags, _p(workspace), 0 if workspace is None else workspace.numel(),
                                  _p(blocks), _s(stream)), "qs_block_select")


def qs_block_attention_workspace_bytes(B, Lq, Hq, D, T) -> int:
    return int(load().qs_block_attention_workspace_bytes(B, Lq, Hq, D, T))


def qs_block_attention(q, k, v, blocks, q_len, k_len, scale, flags, workspace, out, lse,
                       stream=None):
    """q, out: [B, Lq, Hq, D], k, v: [B, Lk, Hkv, D] views; blocks: int32
    [B, Hq, ceil(Lq / 128), T]; lse: float32 [B, Hq, Lq] or None."""
    dtype = (q.dtype,)
    qst, kst, vst, ost = _view(q, "q"), _view(k, "k", dtype), _view(v, "v", dtype), _view(out, "out", dtype)
    B, Lq, Hq, D = q.shape
    _, Lk, Hkv, _ = k.shape
    _shape(k, (B, Lk, Hkv, D), "k")
    _shape(v, k.shape, "v")
    _shape(out, q.shape, "out")
    _cuda(blocks, torch.int32, "blocks")
    if blocks.dim() != 4:
        raise ValueError("blocks must be [B, Hq, query blocks, T]")
    T = blocks.shape[3]
    _shape(blocks, (B, Hq, -(-Lq // QS_BLOCK_Q), T), "blocks")
    for t, name in ((q_len, "q_len"), (k_len, "k_len")):
        if t is not None:
            _cuda(t, torch.int32, name)
            _shape(t, (B,), name)
    _cuda(workspace, torch.uint8, "workspace")
    _cuda(lse, torch.float32, "lse")
    _shape(lse, (B, Hq, Lq), "lse")
    _check(load().qs_block_attention(_p(q), _Strides(*qst[:3]), _p(k), _Strides(*kst[:3]), _p(v),
                                     _Strides(*vst[:3]), B, Lq, Lk, Hq, Hkv, D, _DTYPES[q.dtype],
                                     _p(blocks), T, _p(q_len), _p(k_len), scale, flags,
                                     _p(workspace), 0 if workspace is None else workspace.numel(),
                                     _p(out), _Strides(*ost[:3]), _p(lse), _s(stream)),
           "qs_block_attention")


def qs_selftest_timeout(timeout_us: int, stream=None) -> None:
    _check(load().qs_selftest_timeout(timeout_us, _s(stream)), "qs_selftest_timeout")


def qs_device_error(stream=None) -> int:
    return int(load().qs_device_error(_s(stream)))


def qs_version() -> str:
    return load().qs_version().decode()


# --------------------------------------------------------------------------- helpers

def packed_cols(K: int, bits: int, flags: int = 0) -> int:
    """Bytes of one packed row of K codes: nibbles for 4 bits (bytes with
    QS_FLAG_BYTE_CODES), bytes for 6 and 8."""
    return K // 2 if bits == 4 and not (flags & QS_FLAG_BYTE_CODES) else K


def storage_bits(bits: int, flags: int = 0) -> int:
    """The width the GEMM calls take for codes of `bits` written with `flags`."""
    return 8 if (flags & QS_FLAG_BYTE_CODES) else bits


def pack_weights(w: torch.Tensor, bits: int, flags: int = 0, stream=None):
    """w bf16 [N, K] -> (w_packed uint8 [N, packed_cols(K, bits)], w_scale float32 [N])."""
    N, K = w.shape
    wp = torch.empty((N, packed_cols(K, bits, flags)), dtype=torch.uint8, device=w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    qs_pack_weights(w, N, K, bits, flags, wp, ws, stream)
    return wp, ws


def pack_weights_bgr(w: torch.Tensor, bits: int, candidates: int = 64, iterations: int = 8,
                     flags: int = 0, stream=None):
    """w bf16 [N, K] -> (signed codes on BGR grids, scales float32 [N], offsets int32 [N])."""
    N, K = w.shape
    wp = torch.empty((N, packed_cols(K, bits)), dtype=torch.uint8, device=w.device)
    ws = torch.empty((N,), dtype=torch.float32, device=w.device)
    wo = torch.empty((N,), dtype=torch.int32, device=w.device)
    qs_pack_weights_bgr(w, N, K, bits, flags, candidates, iterations, wp, ws, wo, stream)
    return wp, ws, wo


def quant_act_rowsum(x: torch.Tensor, bits: int, alpha: float = 1.0, flags: int = 0,
                     stream=None):
    """x bf16 [M, K] -> (packed codes, scales, per-token code sums int32 [M])."""
    M, K = x.shape
    xp = torch.empty((M, packed_cols(K, bits)), dtype=torch.uint8, device=x.device)
    xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    xr = torch.empty((M,), dtype=torch.int32, device=x.device)
    qs_quant_act_rowsum(x, M, K, bits, alpha, flags, xp, xs, xr, stream)
    return xp, xs, xr


def quant_act(x: torch.Tensor, bits: int, alpha: float = 1.0, flags: int = 0, stream=None,
              out=None):
    """x bf16 [M, K] -> (x_packed uint8 [M, packed_cols(K, bits)], x_scale float32 [M])."""
    M, K = x.shape
    if out is None:
        xp = torch.empty((M, packed_cols(K, bits, flags)), dtype=torch.uint8, device=x.device)
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    else:
        xp, xs = out
    qs_quant_act(x, M, K, bits, alpha, flags, xp, xs, stream)
    return xp, xs


def qlinear(x_packed, x_scale, w_packed, w_scale, bias, bits: int, K: int, stream=None, out=None,
            bits_w: int | None = None):
    """Packed activations (``bits``) and weights (``bits_w``, default ``bits``) -> bf16 [M, N]."""
    M, N = x_packed.shape[0], w_packed.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x_packed.device)
    if bits_w is None or bits_w == bits:
        qs_qlinear(x_packed, x_scale, w_packed, w_scale, bias, M, N, K, bits, out, stream)
    else:
        qs_qlinear_mixed(x_packed, x_scale, bits, w_packed, w_scale, bits_w, bias, M, N, K, out,
                         stream)
    return out


def qgemm_s32(x_packed, w_packed, bits: int, K: int, stream=None, bits_w: int | None = None):
    M, N = x_packed.shape[0], w_packed.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=x_packed.device)
    if bits_w is None or bits_w == bits:
        qs_qgemm_s32(x_packed, w_packed, M, N, K, bits, acc, stream)
    else:
        qs_qgemm_s32_mixed(x_packed, bits, w_packed, bits_w, M, N, K, acc, stream)
    return acc


def gelu(x: torch.Tensor, stream=None, out=None):
    y = torch.empty_like(x) if out is None else out
    qs_gelu_bf16(x, x.numel(), y, stream)
    return y


def linear(x, w_packed, w_scale, bias, bits: int, alpha: float = 1.0, workspace=None,
           stream=None, out=None, bits_w: int | None = None, x_flags: int = 0):
    """bf16 activations [M, K] -> bf16 [M, N] through one C call; ``bits`` is
    the activation width, ``bits_w`` the weights' storage width (default
    ``bits``), ``x_flags`` the activation quantisation flags."""
    M, K = x.shape
    N = w_packed.shape[0]
    need = qs_linear_workspace_bytes(M, K, storage_bits(bits, x_flags))
    if need < 0:
        raise QSError(2, "qs_linear_workspace_bytes")
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if x_flags:
        qs_linear_ex(x, M, K, alpha, bits, x_flags, w_packed, w_scale,
                     bits if bits_w is None else bits_w, bias, N, workspace, workspace.numel(),
                     out, stream)
    elif bits_w is None or bits_w == bits:
        qs_linear(x, M, K, alpha, w_packed, w_scale, bias, N, bits, workspace, workspace.numel(),
                  out, stream)
    else:
        qs_linear_mixed(x, M, K, alpha, bits, w_packed, w_scale, bits_w, bias, N, workspace,
                        workspace.numel(), out, stream)
    return out


def _empty_like(t, stream):
    """A contiguous tensor of t's shape and type, as `_empty`."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _empty(t.shape, t.dtype, t.device, stream)


def _empty(shape, dtype, device, stream):
    """A tensor for a kernel on `stream` (None: the current one), allocated on that stream: memory
    that is freed while the kernel runs then goes to later work of the same stream only."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def rope_frequencies(rot_dim: int, theta: float = 10000.0, axes=None, scaling: str | None = None,
                     factor: float = 1.0, trained_length: int = 4096, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cuda"):
    """Frequencies for `rope`: (inv_freq float64 [rot_dim/2], pair_axis int32 [rot_dim/2] or None,
    scale).

    axes     sizes of the sections of a head that turn with each position axis (they sum to
             rot_dim; a video's time, height, width): section of size s has the frequencies
             theta^(-2i/s)
    scaling  how positions beyond `trained_length` are handled (one axis):
             "linear"  all frequencies divided by `factor`
             "ntk"     theta raised to theta * factor^(d/(d-2)): the slowest pair is divided by
                       factor, the fastest stays
             "yarn"    pairs that turn more than beta_fast times over the trained length stay,
                       those below beta_slow turns are divided by factor, a linear ramp between;
                       scale = 0.1 ln(factor) + 1
    """
    sizes = [rot_dim] if axes is None else list(axes)
    if rot_dim < 2 or any(s < 2 or s % 2 for s in sizes) or sum(sizes) != rot_dim:
        raise ValueError("rot_dim and the axes' sizes are even, and the sizes sum to rot_dim")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError("scaling is None, 'linear', 'ntk' or 'yarn'")
    if scaling is not None and (len(sizes) > 1 or factor < 1.0):
        raise ValueError("scaling takes one axis and a factor of at least 1")
    scale = 1.0
    if scaling == "ntk" and rot_dim > 2:
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    inv = torch.cat([theta ** (-torch.arange(0, s, 2, dtype=torch.float64) / s) for s in sizes])
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        # the (fractional) pair that makes `turns` full turns over the trained length
        def pair(turns):
            return rot_dim * math.log(trained_length / (turns * 2 * math.pi)) / (2 * math.log(theta))

        lo = max(math.floor(pair(beta_fast)), 0)
        hi = min(math.ceil(pair(beta_slow)), rot_dim - 1)
        ramp = (torch.arange(rot_dim // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)
        ramp = ramp.clamp(0, 1)
        inv = inv * (1 - ramp) + inv / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    axis = None
    if len(sizes) > 1:
        axis = torch.cat([torch.full((s // 2,), i, dtype=torch.int32) for i, s in enumerate(sizes)])
        axis = axis.to(device)
    return inv.to(device), axis, scale


def rope(x, positions, inv_freq, pair_axis=None, interleaved: bool = True, scale: float = 1.0,
         inverse: bool = False, out=None, stream=None):
    """Rotary positions on x [rows, heads, head_dim] (bf16, fp16 or fp32; a view such as the query
    and key columns of a qkv projection's output): ``positions`` int64 [rows] or [rows, axes],
    ``inv_freq`` float64 [rot_dim/2] and ``pair_axis`` (`rope_frequencies`).  ``out`` may be x (in
    place); by default a new contiguous tensor."""
    if out is None:
        _view(x, "x", _ROPE_DTYPES, 3)
        out = _empty_like(x, stream)
    flags = (QS_ROPE_INTERLEAVED if interleaved else 0) | (QS_ROPE_INVERSE if inverse else 0)
    qs_rope(x, positions, inv_freq, out, pair_axis, scale, flags, stream)
    return out


def lora_add(y, x, a, b, seg_start, seg_adapter, scale=None, out=None, workspace=None, stream=None):
    """y + scale_i * (x A_i^T) B_i^T with i the adapter of each row's request: y bf16 [M, N] (a
    projection's output), x bf16 [M, K], a bf16 [adapters, R, K], b bf16 [adapters, N, R],
    ``seg_start`` int32 [requests + 1], ``seg_adapter`` int32 [requests] (-1: none).  In place
    unless ``out`` is given; rows outside every request are left as they were."""
    M, K = x.shape
    adapters, R, _ = a.shape
    N, requests = y.shape[1], seg_adapter.shape[0]
    out = y if out is None else out
    for t, name, shape in ((y, "y", (M, N)), (a, "a", (adapters, R, K)), (b, "b", (adapters, N, R)),
                           (out, "out", (M, N)), (scale, "scale", (adapters,)),
                           (seg_start, "seg_start", (requests + 1,)),
                           (seg_adapter, "seg_adapter", (requests,))):
        _shape(t, shape, name)
    if workspace is None:
        need = qs_lora_workspace_bytes(M, K, R, requests)
        if need < 0:
            raise QSError(2, f"qs_lora_workspace_bytes({M}, {K}, {R}, {requests})")
        workspace = _empty((need,), torch.uint8, x.device, stream)
    qs_lora_add(x, y, M, K, N, a, b, scale, adapters, R, seg_start, seg_adapter, requests,
                workspace, workspace.numel(), out, stream)
    return out


def block_means(x, lens=None, first_block: int = 0, out=None, stream=None):
    """Means of the 64-row blocks of x [B, L, H, D] (keys): float32 [B, H, ceil(L / 64), D].  With
    ``out`` and ``first_block`` only the blocks from that one on are formed (a cache that grew)."""
    _view(x, "x")
    B, L, H, D = x.shape
    if out is None:
        if first_block:
            raise ValueError("first_block needs the means so far (out)")
        out = _empty((B, H, -(-L // QS_BLOCK_K), D), torch.float32, x.device, stream)
    qs_block_means(x, lens, first_block, out, stream)
    return out


def block_select(q, means, count: int, keys: int, first: int = 0, last: int = 0,
                 causal: bool = False, q_len=None, k_len=None, out=None, workspace=None,
                 stream=None):
    """The ``count`` key blocks that each block of 128 queries of q [B, Lq, Hq, D] attends to, by
    the product of block means (``means`` from `block_means` of ``keys`` keys): int32
    [B, Hq, ceil(Lq / 128), count], ascending, -1 behind the last.  The ``first`` and ``last``
    visible blocks are always among them."""
    _view(q, "q")
    B, Lq, Hq, D = q.shape
    if out is None:
        out = _empty((B, Hq, -(-Lq // QS_BLOCK_Q), count), torch.int32, q.device, stream)
    if workspace is None:
        need = qs_block_select_workspace_bytes(B, Lq, Hq, D)
        if need > 0:
            workspace = _empty((need,), torch.uint8, q.device, stream)
    qs_block_select(q, means, keys, q_len, k_len, count, first, last,
                    QS_ATTN_CAUSAL if causal else 0, workspace, out, stream)
    return out


def block_attention(q, k, v, blocks, scale: float | None = None, causal: bool = False, q_len=None,
                    k_len=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [B, Lq, Hq, D] over the listed 64-key blocks of k, v [B, Lk, Hkv, D] (bf16 or
    fp16, D 64 or 128): (out, lse float32 [B, Hq, Lq]).  ``blocks`` as from `block_select`;
    ``scale`` defaults to D^-1/2.  Rows at and behind ``q_len`` keep what ``out`` and ``lse`` held."""
    _view(q, "q")
    B, Lq, Hq, D = q.shape
    if out is None:
        out = _empty_like(q, stream)
    if lse is None:
        lse = _empty((B, Hq, Lq), torch.float32, q.device, stream)
    if workspace is None:
        need = qs_block_attention_workspace_bytes(B, Lq, Hq, D, blocks.shape[-1])
        if need > 0:
            workspace = _empty((need,), torch.uint8, q.device, stream)
    qs_block_attention(q, k, v, blocks, q_len, k_len, D ** -0.5 if scale is None else scale,
                       QS_ATTN_CAUSAL if causal else 0, workspace, out, lse, stream)
    return out, lse


class LoraBatch:
    """The adapters of one batch beside a projection: stacked factors a [adapters, R, K] and
    b [adapters, N, R], a scale for each, and which rows belong to which request (`lora_add`)."""

    def __init__(self, a, b, seg_start, seg_adapter, scale=None):
        self.a, self.b, self.scale = a, b, scale
        self.seg_start, self.seg_adapter = seg_start, seg_adapter

    def add(self, y, x, stream=None):
        return lora_add(y, x, self.a, self.b, self.seg_start, self.seg_adapter, self.scale,
                        stream=stream)


class QuantLinear:
    """A Hadamard-rotated quantized linear layer (W4A4, W8A8, or mixed such as
    W4A8 / W4A6 with ``bits_x``): weights packed once; each call runs the
    one-call layer (the activation kernel, then the GEMM) on a workspace the
    layer keeps and grows as needed.  ``act_codes`` stores 4-bit activation
    codes two per byte ("packed", packed int4 widened in the GEMM's shared
    memory; the faster form with the GEMM's 256 x 512 tiles) or one per byte
    ("bytes", loaded by TMA straight into the operand tiles); the codes, and
    so the outputs, are the same.  ``lora`` adds the batch's low-rank adapters
    to the output of a call."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None, bits: int,
                 alpha: float = 1.0, bits_x: int | None = None, act_codes: str = "packed"):
        if act_codes not in ("bytes", "packed"):
            raise ValueError("act_codes is 'bytes' or 'packed'")
        self.N, self.K = weight.shape
        self.bits = bits
        self.bits_x = bits if bits_x is None else bits_x
        self.alpha = alpha
        self.x_flags = QS_FLAG_BYTE_CODES if (self.bits_x == 4 and act_codes == "bytes") else 0
        self.w_packed, self.w_scale = pack_weights(weight, bits)
        self.bias = bias
        self.workspace = None

    def __call__(self, x: torch.Tensor, stream=None, out=None, lora: LoraBatch | None = None) -> torch.Tensor:
        need = qs_linear_workspace_bytes(x.shape[0], self.K, storage_bits(self.bits_x, self.x_flags))
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty((max(need, 0),), dtype=torch.uint8, device=x.device)
        y = linear(x, self.w_packed, self.w_scale, self.bias, self.bits_x, self.alpha,
                   self.workspace, stream=stream, out=out, bits_w=self.bits, x_flags=self.x_flags)
        return y if lora is None else lora.add(y, x, stream)


def gbs_state_host(state) -> dict:
    """Copies the header of a qs_gbs_state to the host (synchronises)."""
    import struct
    raw = bytes(state[:32].cpu().numpy().tobytes())
    acc, last_d, bits, step, blocks_done, _ = struct.unpack("<ddiiII", raw)
    return {"acc": acc, "last_d": last_d, "bits": bits, "step": step, "blocks_done": blocks_done}


class GbsLinear:
    """A layer under δ-guided bit switching: weights quantised at 4 bits (codes
    stored one per byte, the form qs_linear_gbs takes) and at 8 bits, one
    device-side state; each call runs the layer at the width the state holds
    and then measures the change of its output against the previous call's,
    choosing the next width on the device (no host synchronisation)."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None, delta: float,
                 alpha: float = 1.0, stream=None):
        self.N, self.K = weight.shape
        self.delta, self.alpha = float(delta), alpha
        self.w4, self.s4 = pack_weights(weight, 4, QS_FLAG_BYTE_CODES, stream=stream)
        self.w8, self.s8 = pack_weights(weight, 8, stream=stream)
        self.bias = bias
        self.state = torch.zeros((QS_GBS_STATE_BYTES,), dtype=torch.uint8, device=weight.device)
        qs_gbs_reset(self.state, stream)
        self.workspace = None
        self.prev = None
        self.buffers = []  # two outputs used in turn when the caller passes none

    def __call__(self, x: torch.Tensor, stream=None, out=None) -> torch.Tensor:
        M = x.shape[0]
        need = qs_linear_workspace_bytes(M, self.K, 8)
        if self.workspace is None or self.workspace.numel() < need:
            self.workspace = torch.empty((max(need, 0),), dtype=torch.uint8, device=x.device)
        if out is None:
            if not self.buffers or self.buffers[0].shape != (M, self.N):
                self.buffers = [torch.empty((M, self.N), dtype=torch.bfloat16, device=x.device)
                                for _ in range(2)]
            self.buffers.reverse()
            out = self.buffers[0]
        if self.prev is not None and out.data_ptr() == self.prev.data_ptr():
            raise ValueError("out must not be the previous step's output")
        qs_linear_gbs(x, M, self.K, self.alpha, self.w4, self.s4, self.w8, self.s8, self.bias,
                      self.N, self.state, self.workspace, self.workspace.numel(), out, stream)
        prev = self.prev if self.prev is not None and self.prev.shape == out.shape else None
        qs_gbs_update(out, prev, out.numel(), self.delta, self.state, stream)
        self.prev = out
        return out
