"""MI355X (gfx950) TTT sequence layer (forward, and the TTT-Linear backward), linear
attention with a decay per head, and rotary positions -- Python binding.

Thin ctypes layer over libttt.so (C ABI in include/ttt.h).  It only checks and
marshals arguments: torch supplies device memory and the current HIP stream,
and every step of the computation runs in the library's HIP kernels.  There is
no CPU or PyTorch fallback: if libttt.so is missing, importing the ops raises.

    import test_sequence_layer_amd as ttt
    z, w_final = ttt.linear_fwd(q, k, v, w0, eta, b=16)
    z, w1_final, w2_final = ttt.mlp_fwd(q, k, v, w1, w2, eta, b=16)
    z, w_final, e = ttt.linear_fwd_save(q, k, v, w0, eta, b=16)          # training
    dq, dk, dv, deta, dw0 = ttt.linear_bwd(q, k, eta, w_final, e, dz, b=16)
    q, k = ttt.rotary(q, k, pos=0, freqs=freqs)
    z, w_final = ttt.linear_attn_fwd(q, k, v, log_decay)
    z = ttt.linear_attn_decode(q1, k1, v1, log_decay, w_final, rope=(pos, freqs))

Pages: [TTT] = news article "大模型最强架构TTT问世！斯坦福UCSD等5年磨一剑，一夜推翻Transformer"
(aharts.cn / itmax.cn), part 03 §1-§9 (the TTT layer, mini-batch GD, the dual
form, TTT-Linear and TTT-MLP).
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libttt.so")

TTT_OK = 0
TTT_F32, TTT_BF16 = 0, 1
TTT_FLAG_GENERIC = 1
TTT_FLAG_PRIMAL = 2
TTT_FLAG_INVERSE = 1  # ttt_rotary
TTT_FLAG_ROWS = {1: 4, 2: 8, 4: 16}  # row blocks per (sequence, head) -> TTT_FLAG_ROWS1/2/4


def _rows_flag(rows) -> int:
    """flag bits forcing ``rows`` row blocks of the matrix-core forward (None: the library's choice)"""
    if rows is None:
        return 0
    if rows not in TTT_FLAG_ROWS:
        raise ValueError(f"rows must be None, 1, 2 or 4, not {rows!r}")
    return TTT_FLAG_ROWS[rows]

STATUS_NAMES = {
    0: "TTT_OK", 1: "TTT_ERR_NULL", 2: "TTT_ERR_SHAPE", 3: "TTT_ERR_DTYPE", 4: "TTT_ERR_UNSUPPORTED",
    5: "TTT_ERR_ALIAS", 6: "TTT_ERR_ALIGN", 7: "TTT_ERR_HIP", 8: "TTT_ERR_STRIDE", 9: "TTT_ERR_FLAGS",
    10: "TTT_ERR_POS", 11: "TTT_ERR_WORKSPACE", 12: "TTT_ERR_SCRATCH",
}
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # TTT_NOALLOC_SCRATCH_BYTES

# Every symbol include/ttt.h declares.
EXPORTS = (
    "ttt_linear_fwd", "ttt_linear_validate", "ttt_linear_kernel_name",
    "ttt_linear_decode", "ttt_linear_decode_validate",
    "ttt_linear_fwd_chunked", "ttt_linear_chunked_workspace_bytes", "ttt_linear_fwd_chunked_noalloc",
    "ttt_linear_ln_fwd", "ttt_linear_ln_fwd_save", "ttt_linear_ln_bwd", "ttt_linear_ln_bwd_validate",
    "ttt_linear_ln_bwd_kernel_name", "ttt_linear_ln_kernel_name", "ttt_linear_ln_decode",
    "ttt_linear_ln_decode_validate",
    "ttt_linear_fwd_save", "ttt_linear_bwd", "ttt_linear_bwd_validate", "ttt_linear_bwd_kernel_name",
    "ttt_mlp_fwd", "ttt_mlp_validate", "ttt_mlp_kernel_name", "ttt_mlp_ln_fwd",
    "ttt_mlp_decode", "ttt_mlp_decode_validate", "ttt_mlp_ln_decode", "ttt_mlp_ln_decode_validate",
    "ttt_mlp_ln_kernel_name", "ttt_mlp_bwd", "ttt_mlp_bwd_validate", "ttt_mlp_bwd_workspace_bytes",
    "ttt_mlp_bwd_kernel_name", "ttt_mlp_ln_bwd", "ttt_mlp_ln_bwd_validate", "ttt_mlp_ln_bwd_kernel_name",
    "ttt_linear_attn_fwd", "ttt_linear_attn_fwd_validate", "ttt_linear_attn_bwd", "ttt_linear_attn_bwd_validate",
    "ttt_linear_attn_workspace_bytes", "ttt_linear_attn_decode", "ttt_linear_attn_decode_validate",
    "ttt_rotary", "ttt_rotary_validate", "ttt_rotary_kernel_name",
    "ttt_status_str", "ttt_abi_version",
)


class LinearDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d", ctypes.c_int32), ("b", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("w0_batch_stride", ctypes.c_int64),
        ("eta_stride_b", ctypes.c_int64), ("eta_stride_h", ctypes.c_int64), ("eta_stride_t", ctypes.c_int64),
    ]


class MlpDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dh", ctypes.c_int32), ("b", ctypes.c_int32),
        ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32),
        ("w_batch_stride", ctypes.c_int64),
        ("eta_stride_b", ctypes.c_int64), ("eta_stride_h", ctypes.c_int64), ("eta_stride_t", ctypes.c_int64),
    ]


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("t", ctypes.c_int64)]


class LinearAttnDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("scale", ctypes.c_float), ("reserved", ctypes.c_int32), ("w0_batch_stride", ctypes.c_int64),
        ("q", Strides), ("k", Strides), ("v", Strides), ("z", Strides),
        ("dq", Strides), ("dk", Strides), ("dv", Strides),
    ]


class Rope(ctypes.Structure):
    _fields_ = [
        ("pos", ctypes.c_void_p), ("pos_stride_b", ctypes.c_int64), ("pos_stride_t", ctypes.c_int64),
        ("pos_offset", ctypes.c_int64), ("freqs", ctypes.c_void_p), ("rot", ctypes.c_int32),
        ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
    ]


class RotaryDesc(ctypes.Structure):
    _fields_ = [
        ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("T", ctypes.c_int32),
        ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("reserved", ctypes.c_int32),
        ("q", Strides), ("k", Strides), ("q_out", Strides), ("k_out", Strides),
    ]


_lib = None


class TTTError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_str(status)})")


def lib() -> ctypes.CDLL:
    """The loaded libttt.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    # torch ships its own HIP runtime under the soname libamdhip64.so.7, which
    # libttt.so also needs.  Loaded after torch, libttt.so binds to torch's
    # runtime; loaded first, it would bind to the system's and torch would then
    # load a second runtime whose device memory the first cannot use.  So torch
    # (when installed) is imported first.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    vp, fp = ctypes.c_void_p, ctypes.c_void_p
    L.ttt_linear_fwd.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, vp, fp, vp]
    L.ttt_linear_fwd.restype = ctypes.c_int
    L.ttt_linear_validate.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, vp, fp]
    L.ttt_linear_validate.restype = ctypes.c_int
    L.ttt_linear_decode.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, vp, fp, fp, ctypes.c_int64, vp]
    L.ttt_linear_decode.restype = ctypes.c_int
    L.ttt_linear_decode_validate.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, vp, fp, fp, ctypes.c_int64]
    L.ttt_linear_decode_validate.restype = ctypes.c_int
    L.ttt_linear_fwd_chunked.argtypes = [ctypes.POINTER(LinearDesc), ctypes.c_int32, vp, vp, vp, fp, fp, vp, fp,
                                         vp, ctypes.c_int64, vp]
    L.ttt_linear_fwd_chunked.restype = ctypes.c_int
    L.ttt_linear_fwd_chunked_noalloc.argtypes = [ctypes.POINTER(LinearDesc), ctypes.c_int32, vp, vp, vp, fp, fp,
                                                 vp, fp, vp]
    L.ttt_linear_fwd_chunked_noalloc.restype = ctypes.c_int
    L.ttt_linear_chunked_workspace_bytes.argtypes = [ctypes.POINTER(LinearDesc), ctypes.c_int32]
    L.ttt_linear_chunked_workspace_bytes.restype = ctypes.c_int64
    L.ttt_linear_ln_fwd.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float, fp, vp, fp,
                                    vp]
    L.ttt_linear_ln_fwd.restype = ctypes.c_int
    L.ttt_linear_ln_fwd_save.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float, fp, vp,
                                         fp, fp, vp]
    L.ttt_linear_ln_fwd_save.restype = ctypes.c_int
    L.ttt_linear_ln_bwd.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float, fp, fp, vp,
                                    fp, vp, vp, vp, fp, fp, fp, fp, vp]
    L.ttt_linear_ln_bwd.restype = ctypes.c_int
    L.ttt_linear_ln_bwd_validate.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float,
                                             fp, fp, vp, fp, vp, vp, vp, fp, fp, fp, fp]
    L.ttt_linear_ln_bwd_validate.restype = ctypes.c_int
    L.ttt_linear_ln_bwd_kernel_name.argtypes = [ctypes.POINTER(LinearDesc)]
    L.ttt_linear_ln_bwd_kernel_name.restype = ctypes.c_char_p
    L.ttt_linear_ln_kernel_name.argtypes = [ctypes.POINTER(LinearDesc)]
    L.ttt_linear_ln_kernel_name.restype = ctypes.c_char_p
    L.ttt_linear_ln_decode.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float, vp, fp,
                                       fp, ctypes.c_int64, vp]
    L.ttt_linear_ln_decode.restype = ctypes.c_int
    L.ttt_linear_ln_decode_validate.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float,
                                                vp, fp, fp, ctypes.c_int64]
    L.ttt_linear_ln_decode_validate.restype = ctypes.c_int
    L.ttt_linear_fwd_save.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, vp, fp, fp, vp, fp, fp, vp]
    L.ttt_linear_fwd_save.restype = ctypes.c_int
    L.ttt_linear_bwd.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, fp, fp, fp, vp, fp, vp, vp, vp, fp, fp, vp]
    L.ttt_linear_bwd.restype = ctypes.c_int
    L.ttt_linear_bwd_validate.argtypes = [ctypes.POINTER(LinearDesc), vp, vp, fp, fp, fp, vp, fp, vp, vp, vp, fp,
                                          fp]
    L.ttt_linear_bwd_validate.restype = ctypes.c_int
    L.ttt_linear_bwd_kernel_name.argtypes = [ctypes.POINTER(LinearDesc)]
    L.ttt_linear_bwd_kernel_name.restype = ctypes.c_char_p
    L.ttt_linear_kernel_name.argtypes = [ctypes.POINTER(LinearDesc)]
    L.ttt_linear_kernel_name.restype = ctypes.c_char_p
    L.ttt_mlp_fwd.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, vp, fp, fp, vp]
    L.ttt_mlp_decode.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, vp, fp, fp, fp, fp, ctypes.c_int64, vp]
    L.ttt_mlp_decode.restype = ctypes.c_int
    L.ttt_mlp_decode_validate.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, vp, fp, fp, fp, fp,
                                          ctypes.c_int64]
    L.ttt_mlp_decode_validate.restype = ctypes.c_int
    L.ttt_mlp_fwd.restype = ctypes.c_int
    L.ttt_mlp_ln_fwd.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, fp, ctypes.c_float, fp, vp, fp,
                                 fp, vp]
    L.ttt_mlp_ln_fwd.restype = ctypes.c_int
    L.ttt_mlp_validate.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, vp, fp, fp]
    L.ttt_mlp_validate.restype = ctypes.c_int
    L.ttt_mlp_kernel_name.argtypes = [ctypes.POINTER(MlpDesc)]
    L.ttt_mlp_kernel_name.restype = ctypes.c_char_p
    L.ttt_mlp_ln_kernel_name.argtypes = [ctypes.POINTER(MlpDesc)]
    L.ttt_mlp_ln_kernel_name.restype = ctypes.c_char_p
    L.ttt_mlp_bwd.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, fp, fp, fp, vp, ctypes.c_int64,
                              fp, fp, fp, fp, fp, fp, vp]
    L.ttt_mlp_bwd.restype = ctypes.c_int
    L.ttt_mlp_bwd_validate.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, fp, fp, fp, vp,
                                       ctypes.c_int64, fp, fp, fp, fp, fp, fp]
    L.ttt_mlp_bwd_validate.restype = ctypes.c_int
    L.ttt_mlp_bwd_workspace_bytes.argtypes = [ctypes.POINTER(MlpDesc)]
    L.ttt_mlp_bwd_workspace_bytes.restype = ctypes.c_int64
    L.ttt_mlp_bwd_kernel_name.argtypes = [ctypes.POINTER(MlpDesc)]
    L.ttt_mlp_bwd_kernel_name.restype = ctypes.c_char_p
    L.ttt_mlp_ln_bwd.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, fp, ctypes.c_float, fp, fp, fp, fp,
                                 vp, ctypes.c_int64, fp, fp, fp, fp, fp, fp, fp, fp, vp]
    L.ttt_mlp_ln_bwd.restype = ctypes.c_int
    L.ttt_mlp_ln_bwd_validate.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, fp, ctypes.c_float, fp,
                                          fp, fp, fp, vp, ctypes.c_int64, fp, fp, fp, fp, fp, fp, fp, fp]
    L.ttt_mlp_ln_bwd_validate.restype = ctypes.c_int
    L.ttt_mlp_ln_bwd_kernel_name.argtypes = [ctypes.POINTER(MlpDesc)]
    L.ttt_mlp_ln_bwd_kernel_name.restype = ctypes.c_char_p
    L.ttt_mlp_ln_decode.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float, vp, fp, fp, fp,
                                    fp, ctypes.c_int64, vp]
    L.ttt_mlp_ln_decode.restype = ctypes.c_int
    L.ttt_mlp_ln_decode_validate.argtypes = [ctypes.POINTER(MlpDesc), vp, vp, vp, fp, fp, fp, ctypes.c_float, vp,
                                             fp, fp, fp, fp, ctypes.c_int64]
    L.ttt_mlp_ln_decode_validate.restype = ctypes.c_int
    ad, i64 = ctypes.POINTER(LinearAttnDesc), ctypes.c_int64
    L.ttt_linear_attn_fwd.argtypes = [ad, vp, vp, vp, fp, fp, vp, vp, fp, vp, i64, vp]
    L.ttt_linear_attn_fwd.restype = ctypes.c_int
    L.ttt_linear_attn_fwd_validate.argtypes = [ad, vp, vp, vp, fp, fp, vp, vp, fp, vp, i64]
    L.ttt_linear_attn_fwd_validate.restype = ctypes.c_int
    L.ttt_linear_attn_bwd.argtypes = [ad, vp, vp, vp, fp, fp, vp, vp, fp, vp, vp, vp, fp, fp, vp, i64, vp]
    L.ttt_linear_attn_bwd.restype = ctypes.c_int
    L.ttt_linear_attn_bwd_validate.argtypes = [ad, vp, vp, vp, fp, fp, vp, vp, fp, vp, vp, vp, fp, fp, vp, i64]
    L.ttt_linear_attn_bwd_validate.restype = ctypes.c_int
    L.ttt_linear_attn_workspace_bytes.argtypes = [ad, ctypes.c_int32]
    L.ttt_linear_attn_workspace_bytes.restype = i64
    L.ttt_linear_attn_decode.argtypes = [ad, vp, vp, vp, fp, vp, ctypes.POINTER(Rope), vp, fp, vp]
    L.ttt_linear_attn_decode.restype = ctypes.c_int
    L.ttt_linear_attn_decode_validate.argtypes = [ad, vp, vp, vp, fp, vp, ctypes.POINTER(Rope), vp, fp]
    L.ttt_linear_attn_decode_validate.restype = ctypes.c_int
    L.ttt_rotary.argtypes = [ctypes.POINTER(RotaryDesc), ctypes.POINTER(Rope), vp, vp, vp, vp, vp]
    L.ttt_rotary.restype = ctypes.c_int
    L.ttt_rotary_validate.argtypes = [ctypes.POINTER(RotaryDesc), ctypes.POINTER(Rope), vp, vp, vp, vp]
    L.ttt_rotary_validate.restype = ctypes.c_int
    L.ttt_rotary_kernel_name.argtypes = [ctypes.POINTER(RotaryDesc), ctypes.POINTER(Rope), vp, vp, vp, vp]
    L.ttt_rotary_kernel_name.restype = ctypes.c_char_p
    L.ttt_status_str.argtypes = [ctypes.c_int]
    L.ttt_status_str.restype = ctypes.c_char_p
    L.ttt_abi_version.argtypes = []
    L.ttt_abi_version.restype = ctypes.c_int
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().ttt_status_str(int(status)).decode()


def abi_version() -> int:
    return int(lib().ttt_abi_version())


# ----------------------------------------------------------------- helpers --

def _torch():
    import torch
    return torch


def _done(status: int, what: str) -> None:
    """Raise on a non-OK status.  With TTT_DEBUG_SYNC=1 in the environment, also
    wait for the launched work and let torch raise any asynchronous kernel fault
    here, at the call that caused it, rather than at a later synchronization."""
    if status != TTT_OK:
        raise TTTError(status, what)
    if os.environ.get("TTT_DEBUG_SYNC") == "1":
        _torch().cuda.synchronize()


def _dtype_code(dt) -> int:
    torch = _torch()
    if dt == torch.float32:
        return TTT_F32
    if dt == torch.bfloat16:
        return TTT_BF16
    raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


_raw_stream = None


def _stream_handle(stream, dev: Optional[int] = None) -> Optional[int]:
    """hipStream_t of ``stream``, else of torch's current stream on device ``dev``
    (default: the current device).  torch's raw-stream query is used when it
    exists: building a Stream object costs ~3 us per call, which matters for
    one-token decode calls."""
    torch = _torch()
    if stream is not None:
        return stream.cuda_stream
    global _raw_stream
    if _raw_stream is None:
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", False)
    if _raw_stream:
        return _raw_stream(torch.cuda.current_device() if dev is None else dev)
    return torch.cuda.current_stream().cuda_stream


def _check_dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("every tensor must be on the GPU")
            if not t.is_contiguous():
                raise ValueError("every tensor must be contiguous")


def eta_layout(eta, B: int, H: int, T: int, device):
    """eta as (device fp32 tensor, (stride_b, stride_h, stride_t)).

    float / 1-element tensor -> scalar; [H] -> per head; [B, H, T] -> per token.
    """
    torch = _torch()
    if not torch.is_tensor(eta):
        return torch.tensor([float(eta)], dtype=torch.float32, device=device), (0, 0, 0)
    if eta.dtype != torch.float32:
        raise TypeError("eta must be float32")
    if eta.numel() == 1:
        return eta.reshape(1), (0, 0, 0)
    if tuple(eta.shape) == (H,):
        return eta, (0, 1, 0)
    if tuple(eta.shape) == (B, H, T):
        return eta, (H * T, T, 1)
    raise ValueError(f"eta shape {tuple(eta.shape)}: expected scalar, [H] or [B, H, T]")


# ------------------------------------------------------------- TTT-Linear --

def linear_desc(B, H, T, d, b, in_dtype, out_dtype, w0_batch_stride, eta_strides, flags=0) -> LinearDesc:
    return LinearDesc(B, H, T, d, b, in_dtype, out_dtype, flags, w0_batch_stride, *eta_strides)


def linear_fwd(q, k, v, w0, eta, b: int, out_dtype=None, w_final=None, z=None,
               generic: bool = False, primal: bool = False, rows=None, stream=None) -> Tuple["object", "object"]:
    """TTT-Linear forward (dual form) on the GPU.

    q, k, v : [B, H, T, d] bfloat16 or float32 (same dtype), contiguous, on the GPU
    w0      : [H, d, d] (shared over the batch) or [B, H, d, d] float32; z = W q
    eta     : float, [H] or [B, H, T] float32
    b       : mini-batch size (T % b == 0)
    returns (Z [B, H, T, d] of out_dtype (default float32), W_final [B, H, d, d] float32).
    ``w_final`` may be ``w0`` itself (in-place carry) when w0 is [B, H, d, d].
    ``generic`` forces the portable fp32 kernel; ``primal`` computes token by
    token (the primal form) instead of with the dual form; ``rows`` (1, 2, 4)
    forces the number of row-block workgroups per sequence and head of the
    matrix-core kernel (default 1).
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if w0.dtype != torch.float32:
        raise TypeError("w0 must be float32")
    if tuple(w0.shape) == (H, d, d):
        wstride = 0
    elif tuple(w0.shape) == (B, H, d, d):
        wstride = H * d * d
    else:
        raise ValueError(f"w0 shape {tuple(w0.shape)}: expected [H,d,d] or [B,H,d,d]")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if w_final is None:
        w_final = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    _check_dev(q, k, v, w0, eta_t, z, w_final)
    flags = (TTT_FLAG_GENERIC if generic else 0) | (TTT_FLAG_PRIMAL if primal else 0) | _rows_flag(rows)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), wstride, est, flags)
    st = lib().ttt_linear_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(eta_t),
                              _ptr(z), _ptr(w_final), _stream_handle(stream))
    _done(st, "ttt_linear_fwd")
    return z, w_final


def linear_fwd_save(q, k, v, w0, eta, b: int, out_dtype=None, w_final=None, z=None, e_saved=None,
                    generic: bool = False, rows=None, stream=None):
    """TTT-Linear forward for training: :func:`linear_fwd` plus the saved
    reconstruction errors E [B, H, T, d] float32 (e_t = W k_t - v_t at the
    mini-batch-start W) that :func:`linear_bwd` needs.

    returns (Z, W_final, E).
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if w0.dtype != torch.float32:
        raise TypeError("w0 must be float32")
    wstride = _w0_stride(w0, B, H, d)
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if w_final is None:
        w_final = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    if e_saved is None:
        e_saved = torch.empty((B, H, T, d), dtype=torch.float32, device=q.device)
    _check_dev(q, k, v, w0, eta_t, z, w_final, e_saved)
    flags = (TTT_FLAG_GENERIC if generic else 0) | _rows_flag(rows)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), wstride, est, flags)
    st = lib().ttt_linear_fwd_save(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(eta_t),
                                   _ptr(z), _ptr(w_final), _ptr(e_saved), _stream_handle(stream))
    _done(st, "ttt_linear_fwd_save")
    return z, w_final, e_saved


def linear_bwd(q, k, eta, w_final, e_saved, dz, b: int, dw_final=None, generic: bool = False, out=None,
               stream=None):
    """TTT-Linear backward (dual form).

    q, k     : the forward's [B, H, T, d] inputs (v is not needed)
    eta      : as given to the forward
    w_final, e_saved : from :func:`linear_fwd_save`
    dz       : [B, H, T, d] gradient of the loss with respect to Z (its dtype
               is the dtype of dq, dk, dv)
    dw_final : [B, H, d, d] float32 gradient with respect to W_final, or None (zero)
    out      : optional (dq, dk, dv, deta, dw0) preallocated outputs
    returns (dq, dk, dv, deta [B, H, T] per token, dw0 [B, H, d, d] per sequence).
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or k.dtype != q.dtype:
        raise ValueError("q, k must have the same shape and dtype")
    if dz.shape != q.shape or tuple(e_saved.shape) != tuple(q.shape) or tuple(w_final.shape) != (B, H, d, d):
        raise ValueError("dz, e_saved must be [B, H, T, d] and w_final [B, H, d, d]")
    if e_saved.dtype != torch.float32 or w_final.dtype != torch.float32:
        raise TypeError("e_saved and w_final must be float32")
    if dw_final is not None and (tuple(dw_final.shape) != (B, H, d, d) or dw_final.dtype != torch.float32):
        raise ValueError("dw_final must be [B, H, d, d] float32")
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if out is None:
        dev = q.device
        out = (torch.empty((B, H, T, d), dtype=dz.dtype, device=dev),
               torch.empty((B, H, T, d), dtype=dz.dtype, device=dev),
               torch.empty((B, H, T, d), dtype=dz.dtype, device=dev),
               torch.empty((B, H, T), dtype=torch.float32, device=dev),
               torch.empty((B, H, d, d), dtype=torch.float32, device=dev))
    dq, dk, dv, deta, dw0 = out
    _check_dev(q, k, eta_t, w_final, e_saved, dz, dw_final, dq, dk, dv, deta, dw0)
    flags = TTT_FLAG_GENERIC if generic else 0
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(dz.dtype), 0, est, flags)
    st = lib().ttt_linear_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(eta_t), _ptr(w_final), _ptr(e_saved),
                              _ptr(dz), _ptr(dw_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(deta), _ptr(dw0),
                              _stream_handle(stream))
    _done(st, "ttt_linear_bwd")
    return dq, dk, dv, deta, dw0


def linear_bwd_kernel_name(B, H, T, d, b, in_dtype=TTT_BF16, out_dtype=TTT_F32, eta_strides=(0, 0, 0),
                           generic=False) -> Optional[str]:
    desc = linear_desc(B, H, T, d, b, in_dtype, out_dtype, 0, eta_strides, TTT_FLAG_GENERIC if generic else 0)
    name = lib().ttt_linear_bwd_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def _w0_stride(w0, B, H, d) -> int:
    if tuple(w0.shape) == (H, d, d):
        return 0
    if tuple(w0.shape) == (B, H, d, d):
        return H * d * d
    raise ValueError(f"w0 shape {tuple(w0.shape)}: expected [H,d,d] or [B,H,d,d]")


def linear_kernel_name(B, H, T, d, b, in_dtype=TTT_BF16, out_dtype=TTT_F32, eta_strides=(0, 0, 0),
                       generic=False, primal=False, rows=None) -> Optional[str]:
    flags = (TTT_FLAG_GENERIC if generic else 0) | (TTT_FLAG_PRIMAL if primal else 0) | _rows_flag(rows)
    desc = linear_desc(B, H, T, d, b, in_dtype, out_dtype, 0, eta_strides, flags)
    name = lib().ttt_linear_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def linear_fwd_chunked(q, k, v, w0, eta, b: int, nchunks: int, workspace=None, out_dtype=None,
                       w_final=None, z=None, rows=None, stream=None):
    """TTT-Linear forward with the sequence split into ``nchunks`` chunks run in parallel.

    Same arguments and result as :func:`linear_fwd` (to rounding).  ``workspace``
    is a uint8 device tensor of at least :func:`linear_chunked_workspace_bytes`
    bytes; one is allocated when omitted.
    """
    torch = _torch()
    B, H, T, d = q.shape
    if tuple(w0.shape) == (H, d, d):
        wstride = 0
    elif tuple(w0.shape) == (B, H, d, d):
        wstride = H * d * d
    else:
        raise ValueError(f"w0 shape {tuple(w0.shape)}: expected [H,d,d] or [B,H,d,d]")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if w_final is None:
        w_final = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), wstride, est, _rows_flag(rows))
    need = int(lib().ttt_linear_chunked_workspace_bytes(ctypes.byref(desc), int(nchunks)))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _check_dev(q, k, v, w0, eta_t, z, w_final, workspace)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().ttt_linear_fwd_chunked(ctypes.byref(desc), int(nchunks), _ptr(q), _ptr(k), _ptr(v), _ptr(w0),
                                      _ptr(eta_t), _ptr(z), _ptr(w_final), _ptr(workspace), wbytes,
                                      _stream_handle(stream))
    _done(st, "ttt_linear_fwd_chunked")
    return z, w_final


def linear_fwd_chunked_noalloc(q, k, v, w0, eta, b: int, nchunks: int, out_dtype=None, w_final=None, z=None,
                               rows=None, stream=None):
    """:func:`linear_fwd_chunked` with the library's static scratch in place of a
    workspace (ttt_linear_fwd_chunked_noalloc: the call allocates no device
    memory; calls that overlap on one GPU race).  ``z`` and ``w_final`` are
    allocated here when omitted; pass them to keep the call allocation-free."""
    torch = _torch()
    B, H, T, d = q.shape
    wstride = _w0_stride(w0, B, H, d)
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if w_final is None:
        w_final = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    _check_dev(q, k, v, w0, eta_t, z, w_final)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), wstride, est, _rows_flag(rows))
    st = lib().ttt_linear_fwd_chunked_noalloc(ctypes.byref(desc), int(nchunks), _ptr(q), _ptr(k), _ptr(v), _ptr(w0),
                                              _ptr(eta_t), _ptr(z), _ptr(w_final), _stream_handle(stream))
    _done(st, "ttt_linear_fwd_chunked_noalloc")
    return z, w_final


def linear_ln_fwd(q, k, v, w0, gamma, beta, eta, b: int, eps: float = 1e-6, out_dtype=None, w_final=None,
                  z=None, stream=None, g_saved=None, save: bool = False, primal: bool = False):
    """TTT-Linear with layer norm and residual inside f: f(x) = x + LN(W x).

    gamma, beta : [H, d] float32 (per head).  Other arguments as :func:`linear_fwd`.
    save / g_saved : also write G [B, H, T, d] float32, each token's update
    factor -eta delta as the forward applied it (delta the gradient of the
    token's loss with respect to W k at its mini-batch-start W), the input of
    :func:`linear_ln_bwd`; then returns (Z, W_final, G).
    primal : compute token by token (the primal form; any b, d in {16, 32, 64}).
    """
    torch = _torch()
    B, H, T, d = q.shape
    if tuple(gamma.shape) != (H, d) or tuple(beta.shape) != (H, d):
        raise ValueError("gamma and beta must be [H, d]")
    if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("gamma and beta must be float32")
    wstride = _w0_stride(w0, B, H, d)
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if w_final is None:
        w_final = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    save = save or g_saved is not None
    if save and g_saved is None:
        g_saved = torch.empty((B, H, T, d), dtype=torch.float32, device=q.device)
    _check_dev(q, k, v, w0, gamma, beta, eta_t, z, w_final, g_saved)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), wstride, est,
                       TTT_FLAG_PRIMAL if primal else 0)
    if save:
        st = lib().ttt_linear_ln_fwd_save(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(gamma),
                                          _ptr(beta), float(eps), _ptr(eta_t), _ptr(z), _ptr(w_final),
                                          _ptr(g_saved), _stream_handle(stream))
        _done(st, "ttt_linear_ln_fwd_save")
        return z, w_final, g_saved
    st = lib().ttt_linear_ln_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w0), _ptr(gamma),
                                 _ptr(beta), float(eps), _ptr(eta_t), _ptr(z), _ptr(w_final), _stream_handle(stream))
    _done(st, "ttt_linear_ln_fwd")
    return z, w_final


def linear_ln_bwd(q, k, v, eta, gamma, beta, w_final, g_saved, dz, b: int, eps: float = 1e-6,
                  dw_final=None, out=None, stream=None, generic: bool = False):
    """Backward of :func:`linear_ln_fwd`.

    q, k, v, eta, gamma, beta, eps : as given to the forward
    w_final, g_saved : from :func:`linear_ln_fwd` with save=True
    dz       : [B, H, T, d] gradient with respect to Z (its dtype is that of dq, dk, dv)
    dw_final : [B, H, d, d] float32 gradient with respect to W_final, or None (zero)
    out      : optional (dq, dk, dv, deta, dw0, dgamma, dbeta) preallocated outputs
    generic  : run the fp32 kernel (the cross-check) instead of the matrix-core one
    returns (dq, dk, dv, deta [B, H, T], dw0 [B, H, d, d], dgamma [B, H, d], dbeta [B, H, d]),
    the last three per sequence.
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if tuple(gamma.shape) != (H, d) or tuple(beta.shape) != (H, d):
        raise ValueError("gamma and beta must be [H, d]")
    if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("gamma and beta must be float32")
    if dz.shape != q.shape or tuple(g_saved.shape) != tuple(q.shape) or tuple(w_final.shape) != (B, H, d, d):
        raise ValueError("dz, g_saved must be [B, H, T, d] and w_final [B, H, d, d]")
    if g_saved.dtype != torch.float32 or w_final.dtype != torch.float32:
        raise TypeError("g_saved and w_final must be float32")
    if dw_final is not None and (tuple(dw_final.shape) != (B, H, d, d) or dw_final.dtype != torch.float32):
        raise ValueError("dw_final must be [B, H, d, d] float32")
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if out is None:
        dev = q.device
        out = (torch.empty((B, H, T, d), dtype=dz.dtype, device=dev),
               torch.empty((B, H, T, d), dtype=dz.dtype, device=dev),
               torch.empty((B, H, T, d), dtype=dz.dtype, device=dev),
               torch.empty((B, H, T), dtype=torch.float32, device=dev),
               torch.empty((B, H, d, d), dtype=torch.float32, device=dev),
               torch.empty((B, H, d), dtype=torch.float32, device=dev),
               torch.empty((B, H, d), dtype=torch.float32, device=dev))
    dq, dk, dv, deta, dw0, dgamma, dbeta = out
    _check_dev(q, k, v, eta_t, gamma, beta, w_final, g_saved, dz, dw_final, *out)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(dz.dtype), 0, est,
                       TTT_FLAG_GENERIC if generic else 0)
    st = lib().ttt_linear_ln_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta_t), _ptr(gamma),
                                 _ptr(beta), float(eps), _ptr(w_final), _ptr(g_saved), _ptr(dz),
                                 _ptr(dw_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(deta), _ptr(dw0),
                                 _ptr(dgamma), _ptr(dbeta), _stream_handle(stream))
    _done(st, "ttt_linear_ln_bwd")
    return dq, dk, dv, deta, dw0, dgamma, dbeta


def linear_ln_bwd_kernel_name(B, H, T, d, b, in_dtype=TTT_BF16, out_dtype=TTT_F32,
                              eta_strides=(0, 0, 0), generic: bool = False) -> Optional[str]:
    desc = linear_desc(B, H, T, d, b, in_dtype, out_dtype, 0, eta_strides, TTT_FLAG_GENERIC if generic else 0)
    name = lib().ttt_linear_ln_bwd_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def linear_ln_kernel_name(B, H, T, d, b, in_dtype=TTT_BF16, out_dtype=TTT_F32, eta_strides=(0, 0, 0),
                          primal: bool = False) -> Optional[str]:
    desc = linear_desc(B, H, T, d, b, in_dtype, out_dtype, 0, eta_strides, TTT_FLAG_PRIMAL if primal else 0)
    name = lib().ttt_linear_ln_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def linear_chunked_workspace_bytes(B, H, T, d, b, nchunks) -> int:
    desc = linear_desc(B, H, T, d, b, TTT_BF16, TTT_F32, 0, (0, 0, 0), 0)
    return int(lib().ttt_linear_chunked_workspace_bytes(ctypes.byref(desc), int(nchunks)))


def linear_decode(q, k, v, eta, w, wb, pos: int, b: int, out_dtype=None, z=None, stream=None):
    """Continue B*H sequences by T new tokens (primal form), state carried in place.

    q, k, v : [B, H, T, d];  w, wb : [B, H, d, d] float32 -- the state and the
    mini-batch-start state after ``pos`` tokens, both updated in place.
    eta     : float, [H] or [B, H, T] (indexed by the new tokens).
    returns Z [B, H, T, d].
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if tuple(w.shape) != (B, H, d, d) or tuple(wb.shape) != (B, H, d, d):
        raise ValueError("w and wb must be [B, H, d, d]")
    if w.dtype != torch.float32 or wb.dtype != torch.float32:
        raise TypeError("w and wb must be float32")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    _check_dev(q, k, v, eta_t, z, w, wb)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), 0, est, 0)
    st = lib().ttt_linear_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta_t), _ptr(z),
                                 _ptr(w), _ptr(wb), int(pos), _stream_handle(stream))
    _done(st, "ttt_linear_decode")
    return z


def linear_ln_decode(q, k, v, eta, gamma, beta, w, wb, pos: int, b: int, eps: float = 1e-6, out_dtype=None,
                     z=None, stream=None):
    """:func:`linear_decode` with f(x) = x + LN(W x); gamma, beta [H, d] float32."""
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if tuple(w.shape) != (B, H, d, d) or tuple(wb.shape) != (B, H, d, d):
        raise ValueError("w and wb must be [B, H, d, d]")
    if w.dtype != torch.float32 or wb.dtype != torch.float32:
        raise TypeError("w and wb must be float32")
    if tuple(gamma.shape) != (H, d) or tuple(beta.shape) != (H, d):
        raise ValueError("gamma and beta must be [H, d]")
    if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("gamma and beta must be float32")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    _check_dev(q, k, v, eta_t, gamma, beta, z, w, wb)
    desc = linear_desc(B, H, T, d, b, _dtype_code(q.dtype), _dtype_code(z.dtype), 0, est, 0)
    st = lib().ttt_linear_ln_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta_t), _ptr(gamma),
                                    _ptr(beta), float(eps), _ptr(z), _ptr(w), _ptr(wb), int(pos),
                                    _stream_handle(stream))
    _done(st, "ttt_linear_ln_decode")
    return z


# ---------------------------------------------------------------- TTT-MLP --

def mlp_desc(B, H, T, d, dh, b, in_dtype, out_dtype, w_batch_stride, eta_strides, flags=0) -> MlpDesc:
    return MlpDesc(B, H, T, d, dh, b, in_dtype, out_dtype, flags, 0, w_batch_stride, *eta_strides)


def mlp_fwd(q, k, v, w1, w2, eta, b: int, out_dtype=None, w1_final=None, w2_final=None, z=None,
            stream=None, primal: bool = False):
    """TTT-MLP forward: f(x) = W2 GELU(W1 x).

    w1 : [H, dh, d] or [B, H, dh, d] float32;  w2 : [H, d, dh] or [B, H, d, dh] float32
    primal : compute token by token (the primal form) instead of the dual form
    returns (Z, W1_final [B,H,dh,d], W2_final [B,H,d,dh]).
    """
    return _mlp_call(q, k, v, w1, w2, eta, b, out_dtype, w1_final, w2_final, z, stream,
                     flags=TTT_FLAG_PRIMAL if primal else 0)


def mlp_ln_fwd(q, k, v, w1, w2, gamma, beta, eta, b: int, eps: float = 1e-6, out_dtype=None, w1_final=None,
               w2_final=None, z=None, stream=None, primal: bool = False):
    """TTT-MLP with layer norm and residual inside f: f(x) = x + LN(W2 GELU(W1 x)).

    gamma, beta : [H, d] float32 (per head).  Other arguments as :func:`mlp_fwd`.
    primal : compute token by token (the primal form) instead of the dual form.
    """
    torch = _torch()
    H, d = q.shape[1], q.shape[3]
    if tuple(gamma.shape) != (H, d) or tuple(beta.shape) != (H, d):
        raise ValueError("gamma and beta must be [H, d]")
    if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("gamma and beta must be float32")
    return _mlp_call(q, k, v, w1, w2, eta, b, out_dtype, w1_final, w2_final, z, stream, ln=(gamma, beta, eps),
                     flags=TTT_FLAG_PRIMAL if primal else 0)


def _mlp_call(q, k, v, w1, w2, eta, b, out_dtype, w1_final, w2_final, z, stream, ln=None, flags=0):
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    dh = w1.shape[-2]
    if w1.dtype != torch.float32 or w2.dtype != torch.float32:
        raise TypeError("w1, w2 must be float32")
    if tuple(w1.shape) == (H, dh, d) and tuple(w2.shape) == (H, d, dh):
        wstride = 0
    elif tuple(w1.shape) == (B, H, dh, d) and tuple(w2.shape) == (B, H, d, dh):
        wstride = H * dh * d
    else:
        raise ValueError("w1/w2 shapes: expected [H,dh,d]/[H,d,dh] or [B,H,dh,d]/[B,H,d,dh]")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    if w1_final is None:
        w1_final = torch.empty((B, H, dh, d), dtype=torch.float32, device=q.device)
    if w2_final is None:
        w2_final = torch.empty((B, H, d, dh), dtype=torch.float32, device=q.device)
    _check_dev(q, k, v, w1, w2, eta_t, z, w1_final, w2_final, *(ln[:2] if ln else ()))
    desc = mlp_desc(B, H, T, d, dh, b, _dtype_code(q.dtype), _dtype_code(z.dtype), wstride, est, flags)
    if ln is None:
        st = lib().ttt_mlp_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(w2), _ptr(eta_t),
                               _ptr(z), _ptr(w1_final), _ptr(w2_final), _stream_handle(stream))
        _done(st, "ttt_mlp_fwd")
    else:
        gamma, beta, eps = ln
        st = lib().ttt_mlp_ln_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(w2), _ptr(gamma),
                                  _ptr(beta), float(eps), _ptr(eta_t), _ptr(z), _ptr(w1_final), _ptr(w2_final),
                                  _stream_handle(stream))
        _done(st, "ttt_mlp_ln_fwd")
    return z, w1_final, w2_final


def mlp_kernel_name(B, H, T, d, dh, b, in_dtype=TTT_BF16, out_dtype=TTT_F32, eta_strides=(0, 0, 0),
                    primal: bool = False):
    desc = mlp_desc(B, H, T, d, dh, b, in_dtype, out_dtype, 0, eta_strides, TTT_FLAG_PRIMAL if primal else 0)
    name = lib().ttt_mlp_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def mlp_ln_kernel_name(B, H, T, d, dh, b, in_dtype=TTT_BF16, out_dtype=TTT_F32, eta_strides=(0, 0, 0),
                       primal: bool = False):
    desc = mlp_desc(B, H, T, d, dh, b, in_dtype, out_dtype, 0, eta_strides, TTT_FLAG_PRIMAL if primal else 0)
    name = lib().ttt_mlp_ln_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def mlp_bwd_workspace_bytes(B, H, T, d, dh, b) -> int:
    return int(lib().ttt_mlp_bwd_workspace_bytes(ctypes.byref(mlp_desc(B, H, T, d, dh, b, TTT_BF16, TTT_F32, 0,
                                                                         (0, 0, 0)))))


def mlp_bwd_kernel_name(B, H, T, d, dh, b, in_dtype=TTT_BF16, primal: bool = False) -> Optional[str]:
    """ttt_mlp_bwd_d64h256b16 (dual form, matrix cores) or ttt_mlp_bwd_d64h256 (primal form)."""
    desc = mlp_desc(B, H, T, d, dh, b, in_dtype, TTT_F32, 0, (0, 0, 0), TTT_FLAG_PRIMAL if primal else 0)
    name = lib().ttt_mlp_bwd_kernel_name(ctypes.byref(desc))
    return None if name is None else name.decode()


def mlp_bwd(q, k, v, w1, w2, eta, b: int, dz, dw1_final=None, dw2_final=None, workspace=None, out=None,
            stream=None, primal: bool = False):
    """Backward of :func:`mlp_fwd`: the gradients of L with respect to every
    input, given dz = dL/dZ and dw1_final, dw2_final = dL/dW1_final, dL/dW2_final
    (None for zero).  dz and the gradients are float32.  The dual form on the
    matrix cores runs where it applies (b = 16, T a multiple of 16, bf16
    inputs); primal=True, or any other shape, runs the primal form.

    workspace : uint8 device tensor of at least mlp_bwd_workspace_bytes bytes
    (allocated when omitted).  out : optional preallocated
    (dq, dk, dv, deta, dw1, dw2).
    returns (dq [B,H,T,d], dk, dv, deta [B,H,T], dw1 [B,H,dh,d], dw2 [B,H,d,dh]).
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if tuple(dz.shape) != (B, H, T, d) or dz.dtype != torch.float32:
        raise ValueError("dz must be float32 [B, H, T, d]")
    dh = w1.shape[-2]
    if w1.dtype != torch.float32 or w2.dtype != torch.float32:
        raise TypeError("w1, w2 must be float32")
    if tuple(w1.shape) == (H, dh, d) and tuple(w2.shape) == (H, d, dh):
        wstride = 0
    elif tuple(w1.shape) == (B, H, dh, d) and tuple(w2.shape) == (B, H, d, dh):
        wstride = H * dh * d
    else:
        raise ValueError("w1/w2 shapes: expected [H,dh,d]/[H,d,dh] or [B,H,dh,d]/[B,H,d,dh]")
    for x, shape in ((dw1_final, (B, H, dh, d)), (dw2_final, (B, H, d, dh))):
        if x is not None and (tuple(x.shape) != shape or x.dtype != torch.float32):
            raise ValueError(f"final-state gradients must be float32 {shape}")
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    desc = mlp_desc(B, H, T, d, dh, b, _dtype_code(q.dtype), TTT_F32, wstride, est,
                    TTT_FLAG_PRIMAL if primal else 0)
    need = int(lib().ttt_mlp_bwd_workspace_bytes(ctypes.byref(desc)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        f = dict(dtype=torch.float32, device=q.device)
        out = (torch.empty((B, H, T, d), **f), torch.empty((B, H, T, d), **f), torch.empty((B, H, T, d), **f),
               torch.empty((B, H, T), **f), torch.empty((B, H, dh, d), **f), torch.empty((B, H, d, dh), **f))
    dq, dk, dv, deta, dw1, dw2 = out
    _check_dev(q, k, v, w1, w2, eta_t, dz, dw1_final, dw2_final, workspace, *out)
    st = lib().ttt_mlp_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(w2), _ptr(eta_t), _ptr(dz),
                           _ptr(dw1_final), _ptr(dw2_final), _ptr(workspace), workspace.numel(), _ptr(dq), _ptr(dk),
                           _ptr(dv), _ptr(deta), _ptr(dw1), _ptr(dw2), _stream_handle(stream))
    _done(st, "ttt_mlp_bwd")
    return dq, dk, dv, deta, dw1, dw2


def mlp_ln_bwd_kernel_name(B, H, T, d, dh, b, in_dtype=TTT_BF16) -> Optional[str]:
    name = lib().ttt_mlp_ln_bwd_kernel_name(ctypes.byref(mlp_desc(B, H, T, d, dh, b, in_dtype, TTT_F32, 0, (0, 0, 0))))
    return None if name is None else name.decode()


def mlp_ln_bwd(q, k, v, w1, w2, gamma, beta, eps: float, eta, b: int, dz, dw1_final=None, dw2_final=None,
               workspace=None, out=None, stream=None):
    """Backward of :func:`mlp_ln_fwd` (f(x) = x + LN(W2 GELU(W1 x))): as
    :func:`mlp_bwd`, with gamma, beta [H, d] float32 and eps the forward's.
    out : optional preallocated (dq, dk, dv, deta, dw1, dw2, dgamma, dbeta).
    returns (dq, dk, dv, deta, dw1, dw2, dgamma [B,H,d], dbeta [B,H,d]).
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    if tuple(dz.shape) != (B, H, T, d) or dz.dtype != torch.float32:
        raise ValueError("dz must be float32 [B, H, T, d]")
    dh = w1.shape[-2]
    if w1.dtype != torch.float32 or w2.dtype != torch.float32:
        raise TypeError("w1, w2 must be float32")
    if tuple(w1.shape) == (H, dh, d) and tuple(w2.shape) == (H, d, dh):
        wstride = 0
    elif tuple(w1.shape) == (B, H, dh, d) and tuple(w2.shape) == (B, H, d, dh):
        wstride = H * dh * d
    else:
        raise ValueError("w1/w2 shapes: expected [H,dh,d]/[H,d,dh] or [B,H,dh,d]/[B,H,d,dh]")
    if tuple(gamma.shape) != (H, d) or tuple(beta.shape) != (H, d):
        raise ValueError("gamma and beta must be [H, d]")
    if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("gamma and beta must be float32")
    for x, shape in ((dw1_final, (B, H, dh, d)), (dw2_final, (B, H, d, dh))):
        if x is not None and (tuple(x.shape) != shape or x.dtype != torch.float32):
            raise ValueError(f"final-state gradients must be float32 {shape}")
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    desc = mlp_desc(B, H, T, d, dh, b, _dtype_code(q.dtype), TTT_F32, wstride, est)
    need = int(lib().ttt_mlp_bwd_workspace_bytes(ctypes.byref(desc)))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    if out is None:
        f = dict(dtype=torch.float32, device=q.device)
        out = (torch.empty((B, H, T, d), **f), torch.empty((B, H, T, d), **f), torch.empty((B, H, T, d), **f),
               torch.empty((B, H, T), **f), torch.empty((B, H, dh, d), **f), torch.empty((B, H, d, dh), **f),
               torch.empty((B, H, d), **f), torch.empty((B, H, d), **f))
    dq, dk, dv, deta, dw1, dw2, dg, db = out
    _check_dev(q, k, v, w1, w2, gamma, beta, eta_t, dz, dw1_final, dw2_final, workspace, *out)
    st = lib().ttt_mlp_ln_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(w1), _ptr(w2), _ptr(gamma),
                              _ptr(beta), float(eps), _ptr(eta_t), _ptr(dz), _ptr(dw1_final), _ptr(dw2_final),
                              _ptr(workspace), workspace.numel(), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(deta),
                              _ptr(dw1), _ptr(dw2), _ptr(dg), _ptr(db), _stream_handle(stream))
    _done(st, "ttt_mlp_ln_bwd")
    return dq, dk, dv, deta, dw1, dw2, dg, db


def mlp_decode(q, k, v, eta, w1, w2, w1b, w2b, pos: int, b: int, out_dtype=None, z=None, stream=None, ln=None):
    """Continue B*H TTT-MLP sequences by T new tokens (primal form), state carried in place.

    q, k, v : [B, H, T, d];  w1, w1b : [B, H, dh, d], w2, w2b : [B, H, d, dh]
    float32 -- the state and the mini-batch-start state after ``pos`` tokens,
    all updated in place.  eta : float, [H] or [B, H, T] (indexed by the new tokens).
    ln : (gamma, beta, eps) for f(x) = x + LN(W2 GELU(W1 x)) (ttt_mlp_ln_decode),
    gamma and beta [H, d] float32.
    returns Z [B, H, T, d].
    """
    torch = _torch()
    B, H, T, d = q.shape
    if k.shape != q.shape or v.shape != q.shape or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same shape and dtype")
    dh = w1.shape[-2]
    if (tuple(w1.shape) != (B, H, dh, d) or tuple(w1b.shape) != (B, H, dh, d) or
            tuple(w2.shape) != (B, H, d, dh) or tuple(w2b.shape) != (B, H, d, dh)):
        raise ValueError("w1, w1b must be [B, H, dh, d] and w2, w2b [B, H, d, dh]")
    if any(x.dtype != torch.float32 for x in (w1, w2, w1b, w2b)):
        raise TypeError("the states must be float32")
    out_dtype = torch.float32 if out_dtype is None else out_dtype
    eta_t, est = eta_layout(eta, B, H, T, q.device)
    if z is None:
        z = torch.empty((B, H, T, d), dtype=out_dtype, device=q.device)
    desc = mlp_desc(B, H, T, d, dh, b, _dtype_code(q.dtype), _dtype_code(z.dtype), 0, est)
    if ln is not None:
        gamma, beta, eps = ln
        if tuple(gamma.shape) != (H, d) or tuple(beta.shape) != (H, d):
            raise ValueError("gamma and beta must be [H, d]")
        if gamma.dtype != torch.float32 or beta.dtype != torch.float32:
            raise TypeError("gamma and beta must be float32")
        _check_dev(q, k, v, eta_t, z, w1, w2, w1b, w2b, gamma, beta)
        st = lib().ttt_mlp_ln_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta_t), _ptr(gamma),
                                     _ptr(beta), float(eps), _ptr(z), _ptr(w1), _ptr(w2), _ptr(w1b), _ptr(w2b),
                                     int(pos), _stream_handle(stream))
        _done(st, "ttt_mlp_ln_decode")
        return z
    _check_dev(q, k, v, eta_t, z, w1, w2, w1b, w2b)
    st = lib().ttt_mlp_decode(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(eta_t), _ptr(z), _ptr(w1),
                              _ptr(w2), _ptr(w1b), _ptr(w2b), int(pos), _stream_handle(stream))
    _done(st, "ttt_mlp_decode")
    return z


# --------------------------------- linear attention with a decay per head --

def _on(x, stream):
    """Context in which a call's tensors are made and its kernels launched: the given
    stream, else the current stream of the device that ``x`` is on (None: it is current)."""
    torch = _torch()
    if stream is not None:
        if stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {x.device}")
        return torch.cuda.stream(stream)
    if x.get_device() != torch._C._cuda_getDevice():
        return torch.cuda.device(x.device)
    return None


def _check_same_dev(x, *ts):
    dev = x.get_device()
    if dev < 0:
        raise ValueError("every tensor must be on the GPU")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on one GPU ({t.device} and {x.device})")


def _strides(t) -> Strides:
    """(b, h, t) element strides of a [B, H, T, d] tensor whose rows are contiguous."""
    b, h, s, e = t.stride()
    if e != 1 and t.shape[3] > 1:
        raise ValueError("the last dimension must be contiguous")
    return Strides(b, h, s)


def _check_sizes(*shapes):
    """ttt_linear_attn_desc and ttt_rotary_desc hold sizes in 32 bits."""
    for shape in shapes:
        if any(n >= 1 << 31 for n in shape):
            raise ValueError(f"{tuple(shape)}: sizes must be below 2^31")


def _like(x, dtype):
    """An empty tensor of x's shape and, where x is dense, its layout."""
    return _torch().empty_like(x, dtype=dtype)


# Checked descriptors by what they were checked from (shapes, strides, types): a call's checks and its
# descriptor take as long as its launch.  Nothing in them belongs to a tensor's memory.
_attn_descs = {}


def _layout(x):
    return None if x is None else (x.shape, x.stride(), x.dtype)


def _attn_desc(q, k, v, log_decay, w0, lens, scale, z, grads=()):
    """(descriptor, forward workspace bytes, backward workspace bytes) of a linear-attention call; z: Z or dZ,
    grads: dq, dk, dv."""
    scale = float(scale)  # (a tensor's value at this call: as a key it would stand for itself)
    key = (q.shape, q.stride(), q.dtype, k.shape, k.stride(), k.dtype, v.shape, v.stride(), v.dtype, log_decay.shape,
           log_decay.stride(), log_decay.dtype, _layout(w0), _layout(lens), scale, z.shape, z.stride(), z.dtype,
           *map(_layout, grads))
    got = _attn_descs.get(key)
    if got is None:
        _check_sizes(q.shape, k.shape)
        B, H, Hkv, T, d, wstride = _attn_args(q, k, v, log_decay, w0, lens)
        if z.shape != q.shape:
            raise ValueError(f"z or dz {tuple(z.shape)}: expected {tuple(q.shape)}")
        desc = LinearAttnDesc(B, H, Hkv, T, d, _dtype_code(q.dtype), _dtype_code(z.dtype), 0, scale, 0, wstride,
                              _strides(q), _strides(k), _strides(v), _strides(z), *map(_strides, grads))
        got = (desc, *(int(lib().ttt_linear_attn_workspace_bytes(ctypes.byref(desc), b)) for b in (0, 1)))
        if len(_attn_descs) >= 1024:
            _attn_descs.clear()
        _attn_descs[key] = got
    return got


def _attn_args(q, k, v, log_decay, w0, lens):
    """Checks what every linear-attention call takes; returns (B, H, Hkv, T, d, w0 batch stride)."""
    torch = _torch()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k, v must be [B, H, T, d]")
    B, H, T, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, T, d) or v.shape != k.shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}: expected [B, H, T, d] and "
                         "twice [B, Hkv, T, d]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must have the same dtype")
    if H and (Hkv == 0 or H % Hkv):
        raise ValueError(f"{H} query heads do not share {Hkv} key / value heads evenly")
    if tuple(log_decay.shape) != (H,):
        raise ValueError(f"log_decay shape {tuple(log_decay.shape)}: expected [H]")
    if log_decay.dtype != torch.float32:
        raise TypeError("log_decay must be float32")
    if lens is not None:
        if tuple(lens.shape) != (B,):
            raise ValueError(f"lens shape {tuple(lens.shape)}: expected [B]")
        if lens.dtype != torch.int32:
            raise TypeError("lens must be int32")
    wstride = 0
    if w0 is not None:
        if w0.dtype != torch.float32:
            raise TypeError("w0 must be float32")
        wstride = _w0_stride(w0, B, H, d)
    for x in (log_decay, lens, w0):
        if x is not None and not x.is_contiguous():
            raise ValueError("log_decay, lens and w0 must be contiguous")
    return B, H, Hkv, T, d, wstride


def _want(x, shape, dtype, what):
    if tuple(x.shape) != tuple(shape) or x.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} {tuple(shape)}, not {x.dtype} {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{what} must be contiguous")


def _attn_workspace(need, workspace, dev):
    if workspace is None:
        return (_torch().empty(need, dtype=_torch().uint8, device=dev), need) if need > 0 else (None, 0)
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def linear_attn_workspace_bytes(q, k, out_dtype=None, backward: bool = False) -> int:
    """Bytes of workspace that a call on inputs like q [B, H, T, d] and k [B, Hkv, T, d] takes."""
    _check_sizes(q.shape, k.shape)
    B, H, T, d = q.shape
    desc = LinearAttnDesc(B, H, k.shape[1], T, d, _dtype_code(q.dtype), _dtype_code(out_dtype or q.dtype))
    return int(lib().ttt_linear_attn_workspace_bytes(ctypes.byref(desc), int(backward)))


def linear_attn_fwd(q, k, v, log_decay, w0=None, scale: float = 1.0, lens=None, out_dtype=None, w_final=None, z=None,
                    workspace=None, stream=None):
    """Linear attention with a decay per head, forward: W_t = exp(log_decay) W_{t-1} + v_t k_t^T, z_t = scale W_t q_t.

    q         : [B, H, T, d] bfloat16 or float32; k, v : [B, Hkv, T, d] of the same dtype, H a multiple of Hkv
                (query head h reads head h // (H // Hkv)).  d in {16, 32, 64, 128}.  Rows contiguous, 16-byte aligned;
                any strides between them (transposed or sliced projections need no copy)
    log_decay : [H] float32, the logarithm of each head's decay (0 keeps everything)
    w0        : initial state [H, d, d] or [B, H, d, d] float32 (z = W q), or None (zero)
    lens      : [B] int32, the tokens of each sequence, or None (T each).  Rows behind them are not read and give
                zero rows of Z; W_final is the state after the last token
    returns (Z [B, H, T, d] of out_dtype (default float32), W_final [B, H, d, d] float32).
    ``w_final`` may be ``w0`` itself when w0 is [B, H, d, d].  ``workspace``: uint8 tensor of
    :func:`linear_attn_workspace_bytes` (allocated when omitted); calls that may overlap need one each.
    """
    if not q.is_cuda:
        _attn_args(q, k, v, log_decay, w0, lens)
    _check_same_dev(q, k, v, log_decay, w0, lens, z, w_final, workspace)
    on = _on(q, stream)
    if on is not None:
        with on:
            return _attn_fwd(q, k, v, log_decay, w0, scale, lens, out_dtype, w_final, z, workspace, stream)
    return _attn_fwd(q, k, v, log_decay, w0, scale, lens, out_dtype, w_final, z, workspace, None)


def _attn_fwd(q, k, v, log_decay, w0, scale, lens, out_dtype, w_final, z, workspace, stream):
    torch = _torch()
    dev = q.device
    if z is None:
        z = _like(q, torch.float32 if out_dtype is None else out_dtype)
    elif out_dtype is not None and z.dtype != out_dtype:
        raise ValueError(f"z is {z.dtype}, out_dtype {out_dtype}")
    desc, need, _ = _attn_desc(q, k, v, log_decay, w0, lens, scale, z)
    shape = (desc.B, desc.H, desc.d, desc.d)
    if w_final is None:
        w_final = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _want(w_final, shape, torch.float32, "w_final")
    if need or workspace is not None:
        workspace, need = _attn_workspace(need, workspace, dev)
    st = lib().ttt_linear_attn_fwd(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                   _ptr(w0), _ptr(lens), z.data_ptr(), w_final.data_ptr(), _ptr(workspace), need,
                                   _stream_handle(stream, dev.index))
    _done(st, "ttt_linear_attn_fwd")
    return z, w_final


def linear_attn_bwd(q, k, v, log_decay, dz, w0=None, dw_final=None, scale: float = 1.0, lens=None, workspace=None,
                    out=None, stream=None):
    """Backward of :func:`linear_attn_fwd`, from its inputs alone.

    q, k, v, log_decay, w0, scale, lens : as given to the forward
    dz        : [B, H, T, d] gradient of the loss with respect to Z (its dtype is that of dq, dk, dv)
    dw_final  : [B, H, d, d] float32 gradient with respect to W_final, or None (zero)
    workspace : uint8 tensor of linear_attn_workspace_bytes(..., out_dtype=dz.dtype, backward=True), or None
    out       : optional (dq, dk, dv, dlog_decay, dw0) preallocated outputs
    returns (dq [B, H, T, d], dk, dv [B, Hkv, T, d] (summed over the query heads that share them),
    dlog_decay [B, H] float32 and dw0 [B, H, d, d] float32, both per sequence: sum them over B for shared parameters).
    """
    if not q.is_cuda:
        _attn_args(q, k, v, log_decay, w0, lens)
    _check_same_dev(q, k, v, log_decay, dz, w0, dw_final, lens, workspace, *(out or ()))
    on = _on(q, stream)
    if on is not None:
        with on:
            return _attn_bwd(q, k, v, log_decay, dz, w0, dw_final, scale, lens, workspace, out, stream)
    return _attn_bwd(q, k, v, log_decay, dz, w0, dw_final, scale, lens, workspace, out, None)


def _attn_bwd(q, k, v, log_decay, dz, w0, dw_final, scale, lens, workspace, out, stream):
    torch = _torch()
    dev = q.device
    if out is None:
        dq, dk, dv = _like(q, dz.dtype), _like(k, dz.dtype), _like(v, dz.dtype)
    else:
        dq, dk, dv, dg, dw0 = out
        for x, like, what in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
            if x.shape != like.shape or x.dtype != dz.dtype:
                raise ValueError(f"{what} must be {dz.dtype} {tuple(like.shape)}, not {x.dtype} {tuple(x.shape)}")
    desc, _, need = _attn_desc(q, k, v, log_decay, w0, lens, scale, dz, (dq, dk, dv))
    shape = (desc.B, desc.H, desc.d, desc.d)
    if dw_final is not None:
        _want(dw_final, shape, torch.float32, "dw_final")
    if out is None:
        dg = torch.empty(shape[:2], dtype=torch.float32, device=dev)
        dw0 = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _want(dg, shape[:2], torch.float32, "dlog_decay")
        _want(dw0, shape, torch.float32, "dw0")
    if need or workspace is not None:
        workspace, need = _attn_workspace(need, workspace, dev)
    st = lib().ttt_linear_attn_bwd(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                   _ptr(w0), _ptr(lens), dz.data_ptr(), _ptr(dw_final), dq.data_ptr(), dk.data_ptr(),
                                   dv.data_ptr(), dg.data_ptr(), dw0.data_ptr(), _ptr(workspace), need,
                                   _stream_handle(stream, dev.index))
    _done(st, "ttt_linear_attn_bwd")
    return dq, dk, dv, dg, dw0


def linear_attn_decode(q, k, v, log_decay, w, scale: float = 1.0, lens=None, rope=None, out_dtype=None, z=None,
                       stream=None):
    """Continue B*H sequences of :func:`linear_attn_fwd` by T new tokens (often 1), the state carried in place.

    q, k, v : [B, H or Hkv, T, d] as for the forward (any alignment);  w : [B, H, d, d] float32, updated in place
    lens    : [B] int32, the new tokens of each sequence (0: its state stays), or None (T each)
    rope    : (pos, freqs[, layout[, scale]]) to turn q and k as :func:`rotary` would, in the same launch, or None
    returns Z [B, H, T, d].
    """
    if not q.is_cuda:
        _attn_args(q, k, v, log_decay, None, lens)
    _check_same_dev(q, k, v, log_decay, w, lens, z)
    on = _on(q, stream)
    if on is not None:
        with on:
            return _attn_decode(q, k, v, log_decay, w, scale, lens, rope, out_dtype, z, stream)
    return _attn_decode(q, k, v, log_decay, w, scale, lens, rope, out_dtype, z, None)


def _attn_decode(q, k, v, log_decay, w, scale, lens, rope, out_dtype, z, stream):
    torch = _torch()
    if z is None:
        z = _like(q, torch.float32 if out_dtype is None else out_dtype)
    elif out_dtype is not None and z.dtype != out_dtype:
        raise ValueError(f"z is {z.dtype}, out_dtype {out_dtype}")
    desc, _, _ = _attn_desc(q, k, v, log_decay, None, lens, scale, z)
    _want(w, (desc.B, desc.H, desc.d, desc.d), torch.float32, "w")
    turn = None if rope is None else ctypes.byref(_rope(q, *rope))
    st = lib().ttt_linear_attn_decode(ctypes.byref(desc), q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
                                      _ptr(lens), turn, z.data_ptr(), w.data_ptr(), _stream_handle(stream, q.device.index))
    _done(st, "ttt_linear_attn_decode")
    return z


# ------------------------------------------------------- rotary positions --

def rotary_freqs(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                 original: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Frequencies for :func:`rotary`: (freqs [rot / 2] float64, scale).

    Plain: base^(-2i / rot) radians per position, scale 1.  For contexts ``factor`` times longer than the ``original``
    one: "linear" divides the positions by factor; "ntk" raises the base, so that the slowest pair is slowed by factor
    and the fastest not at all; "yarn" (Peng et al., arXiv 2309.00071) divides the frequencies of pairs that turn less
    than beta_slow times within the original context, keeps those that turn more than beta_fast times, blends between
    them by the number of turns, and scales q and k by 0.1 ln(factor) + 1.
    """
    torch = _torch()
    if rot < 0 or rot % 2:
        raise ValueError(f"rot must be even and >= 0, not {rot}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be None, 'linear', 'ntk' or 'yarn', not {scaling!r}")
    if factor < 1.0 or (scaling is None and factor != 1.0):
        raise ValueError("factor must be >= 1, and 1 without scaling")
    if scaling == "yarn" and not beta_fast > beta_slow:
        raise ValueError("beta_fast must be greater than beta_slow")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / rot) if rot else i
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        turns = original * f / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rope(x, pos, freqs, layout: str = "half", scale: float = 1.0) -> Rope:
    """The ttt_rope of positions ``pos`` for rows like x [B, H, T, d]."""
    torch = _torch()
    B, _, T, _ = x.shape
    if layout not in ("half", "interleaved"):
        raise ValueError(f"layout must be 'half' or 'interleaved', not {layout!r}")
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous float64 vector")
    r = Rope(None, 0, 0, 0, freqs.data_ptr(), 2 * freqs.shape[0], layout == "interleaved", scale, 0)
    if torch.is_tensor(pos):
        if pos.dtype != torch.int64:
            raise TypeError("positions must be int64")
        if tuple(pos.shape) == (B, T):
            r.pos_stride_b, r.pos_stride_t = pos.stride()
            if T > 1 and r.pos_stride_t == 0:
                raise ValueError("positions of one sequence must not be expanded along T")
        elif tuple(pos.shape) == (B,):
            r.pos_stride_b = pos.stride(0)
        else:
            raise ValueError(f"positions {tuple(pos.shape)}: expected an int, [B] (of the first token) or [B, T]")
        _check_same_dev(x, pos, freqs)
        r.pos = pos.data_ptr()
    else:
        if pos != int(pos) or not -(1 << 63) <= pos < 1 << 63:
            raise ValueError(f"position {pos}: expected a whole number of 64 bits")
        r.pos_offset = int(pos)
        _check_same_dev(x, freqs)
    return r


_rotary_descs = {}  # as _attn_descs


def _rotary_desc(q, k, qo, ko, flags):
    key = (q.shape, q.stride(), q.dtype, _layout(k), _layout(qo), _layout(ko), flags)
    desc = _rotary_descs.get(key)
    if desc is None:
        _check_sizes(q.shape, *(() if k is None else (k.shape,)))
        B, H, T, d = q.shape
        if (ko is None) != (k is None):
            raise ValueError("out must hold an output for k exactly where k is given")
        for x, like, name in ((qo, q, "out[0]"), (ko, k, "out[1]")):
            if x is not None and (x.shape != like.shape or x.dtype != like.dtype):
                raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)}, not {x.dtype} {tuple(x.shape)}")
        none = Strides()
        desc = RotaryDesc(B, H, 0 if k is None else k.shape[1], T, d, _dtype_code(q.dtype), flags, 0, _strides(q),
                          none if k is None else _strides(k), _strides(qo), none if k is None else _strides(ko))
        if len(_rotary_descs) >= 1024:
            _rotary_descs.clear()
        _rotary_descs[key] = desc
    return desc


def _rotary_call(q, k, pos, freqs, layout, scale, out, stream, flags, what):
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    if k is not None:
        if k.dim() != 4 or k.shape[0] != q.shape[0] or k.shape[2:] != q.shape[2:]:
            raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)}: expected [B, H, T, d] and [B, Hkv, T, d]")
        if k.dtype != q.dtype:
            raise ValueError("q and k must have the same dtype")
    _check_same_dev(q, k, *(out or ()))
    on = _on(q, stream)
    if on is not None:
        with on:
            return _rotary_launch(q, k, pos, freqs, layout, scale, out, stream, flags, what)
    return _rotary_launch(q, k, pos, freqs, layout, scale, out, None, flags, what)


def _rotary_launch(q, k, pos, freqs, layout, scale, out, stream, flags, what):
    qo, ko = out if out is not None else (_like(q, q.dtype), None if k is None else _like(k, k.dtype))
    desc = _rotary_desc(q, k, qo, ko, flags)
    rope = _rope(q, pos, freqs, layout, scale)
    st = lib().ttt_rotary(ctypes.byref(desc), ctypes.byref(rope), q.data_ptr(), _ptr(k), qo.data_ptr(), _ptr(ko),
                          _stream_handle(stream, q.device.index))
    _done(st, what)
    return qo, ko


def rotary(q, k, pos, freqs, layout: str = "half", scale: float = 1.0, out=None, stream=None):
    """Rotary positions: each pair of the first 2 len(freqs) elements of q's and k's rows turned by position * freqs[i].

    q      : [B, H, T, d], k : [B, Hkv, T, d] or None; bfloat16 or float32, any strides between contiguous rows
    pos    : int (position of every sequence's first token), int64 [B] (of each one's) or int64 [B, T] (of each token)
    freqs  : float64 vector on the GPU, from :func:`rotary_freqs` (angles are computed in 64 bits)
    layout : "half" pairs (i, i + len(freqs)), "interleaved" pairs (2i, 2i + 1)
    scale  : factor on the turned elements (the second result of :func:`rotary_freqs`); the others are passed on
    out    : optional (q_out, k_out), which may be q and k themselves
    returns (q_out, k_out).
    """
    return _rotary_call(q, k, pos, freqs, layout, scale, out, stream, 0, "ttt_rotary")


def rotary_bwd(dq, dk, pos, freqs, layout: str = "half", scale: float = 1.0, out=None, stream=None):
    """Backward of :func:`rotary`: the gradients with respect to its q and k, given those with respect to its outputs."""
    return _rotary_call(dq, dk, pos, freqs, layout, scale, out, stream, TTT_FLAG_INVERSE, "ttt_rotary")
