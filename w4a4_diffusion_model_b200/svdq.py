"""Python binding of the SVDQuant W4A4 C ABI (include/svdq.h).

Argument marshalling only: every step of the layer runs in the CUDA library
``libsvdq.so`` built in this directory. Tensors are torch CUDA tensors; calls
are issued on torch's current CUDA stream. There is no CPU fallback: if the
library is missing or the device is not sm_100, calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvdq.so")

SVDQ_FUSED = 0
SVDQ_UNFUSED = 1
SVDQ_PREPARE_GIVEN_FACTORS = 1
SVDQ_NEXT_FUSE_LOWRANK = 1
SVDQ_NORM_ADD_ONE = 1
SVDQ_ROPE_HALVES = 1
SVDQ_ROPE_INVERSE = 2

# svdq_dtype
DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int32: 3}

STATUS = {
    0: "SVDQ_OK", 1: "SVDQ_ERR_INVALID_ARG", 2: "SVDQ_ERR_UNSUPPORTED_SHAPE", 3: "SVDQ_ERR_MISALIGNED",
    4: "SVDQ_ERR_BUFFER_TOO_SMALL", 5: "SVDQ_ERR_NO_DEVICE", 6: "SVDQ_ERR_CUDA", 7: "SVDQ_ERR_TIMEOUT",
    8: "SVDQ_ERR_INTERNAL",
}

# Every symbol the header declares, with its ctypes signature.
EXPORTS = [
    "svdq_status_string", "svdq_last_error", "svdq_version", "svdq_act_sizes", "svdq_weight_sizes",
    "svdq_channel_amax", "svdq_prepare_weights", "svdq_prepare_weights_static", "svdq_quantize_act",
    "svdq_linear", "svdq_linear_quantize_next", "svdq_linear_quantize_next_workspace", "svdq_append_lowrank",
    "svdq_selftest_timeout", "svdq_scales_to_canonical", "svdq_check",
    "svdq_int4_act_sizes", "svdq_int4_weight_sizes", "svdq_int4_quantize_residual", "svdq_int4_quantize_act",
    "svdq_int4_linear", "svdq_deltaquant_sizes", "svdq_deltaquant_encode",
    "svdq_int8_quantize_act", "svdq_int8_quantize_weight", "svdq_int8_linear", "svdq_layernorm",
    "svdq_int8_layernorm_quantize", "svdq_layernorm_backward_workspace", "svdq_layernorm_backward", "svdq_rope",
]


class Shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("rank", ctypes.c_int32)]


class SvdqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m w4a4_diffusion_model_b200.build`")
    lib = ctypes.CDLL(path)
    vp, sz, i64, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int
    P = ctypes.POINTER
    lib.svdq_status_string.argtypes, lib.svdq_status_string.restype = [ctypes.c_int], ctypes.c_char_p
    lib.svdq_last_error.argtypes, lib.svdq_last_error.restype = [], ctypes.c_char_p
    lib.svdq_version.argtypes, lib.svdq_version.restype = [], ctypes.c_int
    lib.svdq_act_sizes.argtypes, lib.svdq_act_sizes.restype = [Shape, P(sz), P(sz), P(sz)], st
    lib.svdq_weight_sizes.argtypes = [Shape, P(sz), P(sz), P(sz), P(sz), P(sz)]
    lib.svdq_weight_sizes.restype = st
    lib.svdq_channel_amax.argtypes, lib.svdq_channel_amax.restype = [i64, i64, vp, vp, vp], st
    lib.svdq_prepare_weights.argtypes = [Shape, vp, vp, ctypes.c_float, ctypes.c_uint, vp, vp, vp, vp, vp, vp,
                                         vp, sz, vp]
    lib.svdq_prepare_weights.restype = st
    lib.svdq_prepare_weights_static.argtypes = [Shape, vp, vp, ctypes.c_float, ctypes.c_uint, vp, vp, vp, vp, vp,
                                                vp, vp]
    lib.svdq_prepare_weights_static.restype = st
    lib.svdq_append_lowrank.argtypes = [Shape, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp]
    lib.svdq_append_lowrank.restype = st
    lib.svdq_selftest_timeout.argtypes = [vp]
    lib.svdq_selftest_timeout.restype = st
    lib.svdq_quantize_act.argtypes = [Shape, vp, vp, vp, vp, vp, vp, ctypes.c_int, vp]
    lib.svdq_quantize_act.restype = st
    lib.svdq_linear.argtypes = [Shape, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, vp]
    lib.svdq_linear.restype = st
    lib.svdq_scales_to_canonical.argtypes, lib.svdq_scales_to_canonical.restype = [i64, i64, vp, vp, vp], st
    lib.svdq_check.argtypes, lib.svdq_check.restype = [vp], st
    lib.svdq_linear_quantize_next.argtypes = [Shape, vp, vp, vp, vp, vp, vp, ctypes.c_int32, vp, vp, vp, vp, vp, vp,
                                              vp, sz, ctypes.c_uint, vp]
    lib.svdq_linear_quantize_next.restype = st
    lib.svdq_linear_quantize_next_workspace.argtypes = [Shape, ctypes.c_int32, ctypes.c_uint, P(sz)]
    lib.svdq_linear_quantize_next_workspace.restype = st
    lib.svdq_int4_act_sizes.argtypes, lib.svdq_int4_act_sizes.restype = [Shape, P(sz), P(sz), P(sz)], st
    lib.svdq_int4_weight_sizes.argtypes, lib.svdq_int4_weight_sizes.restype = [Shape, P(sz), P(sz)], st
    lib.svdq_int4_quantize_residual.argtypes = [Shape, vp, vp, vp, vp, vp, vp, vp]
    lib.svdq_int4_quantize_residual.restype = st
    lib.svdq_int4_quantize_act.argtypes, lib.svdq_int4_quantize_act.restype = [Shape, vp, vp, vp, vp, vp, vp, vp], st
    lib.svdq_int4_linear.argtypes, lib.svdq_int4_linear.restype = [Shape, vp, vp, vp, vp, vp, vp, vp, vp], st
    lib.svdq_deltaquant_sizes.argtypes = [i64, i64, i64, i64, P(sz), P(sz), P(sz)]
    lib.svdq_deltaquant_sizes.restype = st
    lib.svdq_deltaquant_encode.argtypes = [i64, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.svdq_deltaquant_encode.restype = st
    i32, u32, f32 = ctypes.c_int32, ctypes.c_uint, ctypes.c_float
    for name in ("svdq_int8_quantize_act", "svdq_int8_quantize_weight"):
        getattr(lib, name).argtypes, getattr(lib, name).restype = [i64, i64, st, vp, i64, vp, vp, vp, vp], st
    lib.svdq_int8_linear.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, st, vp, i64, vp]
    lib.svdq_int8_linear.restype = st
    lib.svdq_layernorm.argtypes = [i64, i64, st, st, vp, i64, vp, vp, i64, f32, u32, vp, i64, vp, vp, vp]
    lib.svdq_layernorm.restype = st
    lib.svdq_int8_layernorm_quantize.argtypes = [i64, i64, st, st, vp, i64, vp, vp, i64, f32, u32, vp, vp, vp, vp]
    lib.svdq_int8_layernorm_quantize.restype = st
    lib.svdq_layernorm_backward_workspace.argtypes = [i64, i64, i64, P(sz)]
    lib.svdq_layernorm_backward_workspace.restype = st
    lib.svdq_layernorm_backward.argtypes = [i64, i64, st, st, vp, i64, vp, i64, vp, vp, vp, i64, u32, vp, i64, vp, vp,
                                            vp, sz, vp]
    lib.svdq_layernorm_backward.restype = st
    lib.svdq_rope.argtypes = [i64, i32, i32, st, vp, i64, i64, vp, i64, i64, vp, st, i64, i32, P(i32), vp, u32, vp]
    lib.svdq_rope.restype = st
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        raise SvdqError(status, load().svdq_last_error().decode())


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@dataclass(frozen=True)
class LayerShape:
    M: int
    K: int
    N: int
    rank: int

    def c(self) -> Shape:
        return Shape(self.M, self.K, self.N, self.rank)


def svdq_act_sizes(shape: LayerShape) -> tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().svdq_act_sizes(shape.c(), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def svdq_weight_sizes(shape: LayerShape) -> tuple[int, int, int, int, int]:
    v = [ctypes.c_size_t() for _ in range(5)]
    _check(load().svdq_weight_sizes(shape.c(), *[ctypes.byref(x) for x in v]))
    return tuple(x.value for x in v)


def svdq_channel_amax(X: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    M, K = X.shape
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=X.device)
    _check(load().svdq_channel_amax(M, K, _ptr(X), _ptr(out), _stream()))
    return out


@dataclass
class PreparedWeights:
    shape: LayerShape          # M is unused (0)
    Qr: torch.Tensor
    Sr: torch.Tensor
    L1p: torch.Tensor | None
    L2t: torch.Tensor | None
    lam: torch.Tensor
    inv_lam: torch.Tensor


def svdq_prepare_weights(W_lin: torch.Tensor, act_amax: torch.Tensor, alpha: float, rank: int,
                         L1p: torch.Tensor | None = None, L2t: torch.Tensor | None = None) -> PreparedWeights:
    """Smoothing, top-rank split and residual NVFP4 encoding of W_lin [N][K].
    Pass both L1p [rank][K] and L2t [N][rank] (bf16) to use given factors."""
    N, K = W_lin.shape
    shape = LayerShape(0, K, N, rank)
    qr, sr, l1, l2, ws = svdq_weight_sizes(shape)
    dev = W_lin.device
    given = L1p is not None and L2t is not None
    if not given:
        L1p = torch.empty(rank, K, dtype=torch.bfloat16, device=dev) if rank else None
        L2t = torch.empty(N, rank, dtype=torch.bfloat16, device=dev) if rank else None
    Qr = torch.empty(qr, dtype=torch.uint8, device=dev)
    Sr = torch.empty(sr, dtype=torch.uint8, device=dev)
    lam = torch.empty(K, dtype=torch.float32, device=dev)
    inv = torch.empty(K, dtype=torch.float32, device=dev)
    work = torch.empty(ws, dtype=torch.uint8, device=dev) if (ws and not given) else None
    _check(load().svdq_prepare_weights(
        shape.c(), _ptr(W_lin), _ptr(act_amax), ctypes.c_float(alpha),
        SVDQ_PREPARE_GIVEN_FACTORS if given else 0, _ptr(L1p), _ptr(L2t), _ptr(Qr), _ptr(Sr), _ptr(lam), _ptr(inv),
        _ptr(work), ws if work is not None else 0, _stream()))
    return PreparedWeights(shape, Qr.view(N, K // 2), Sr, L1p, L2t, lam, inv)


def svdq_quantize_act(X: torch.Tensor, inv_lambda: torch.Tensor, L1p: torch.Tensor | None, rank: int, N: int = 128,
                      variant: int = SVDQ_FUSED, out: tuple | None = None):
    """Returns (Qx [M][K/2] uint8, Sx native uint8, T [M][rank] bf16 or None)."""
    M, K = X.shape
    shape = LayerShape(M, K, N, rank)
    if out is None:
        qx, sx, _ = svdq_act_sizes(shape)
        Qx = torch.empty(M, K // 2, dtype=torch.uint8, device=X.device)
        Sx = torch.empty(sx, dtype=torch.uint8, device=X.device)
        T = torch.empty(M, rank, dtype=torch.bfloat16, device=X.device) if rank else None
    else:
        Qx, Sx, T = out
    _check(load().svdq_quantize_act(shape.c(), _ptr(X), _ptr(inv_lambda), _ptr(L1p), _ptr(Qx), _ptr(Sx), _ptr(T),
                                    variant, _stream()))
    return Qx, Sx, T


def svdq_linear(Qx: torch.Tensor, Sx: torch.Tensor, T: torch.Tensor | None, W: PreparedWeights,
                variant: int = SVDQ_FUSED, out: torch.Tensor | None = None) -> torch.Tensor:
    M = Qx.shape[0]
    K, N, rank = W.shape.K, W.shape.N, W.shape.rank
    shape = LayerShape(M, K, N, rank)
    Y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=Qx.device)
    _check(load().svdq_linear(shape.c(), _ptr(Qx), _ptr(Sx), _ptr(T), _ptr(W.Qr), _ptr(W.Sr), _ptr(W.L2t), _ptr(Y),
                              variant, _stream()))
    return Y


def svdq_linear_quantize_next_workspace(shape: LayerShape, next_rank: int, flags: int = 0) -> int:
    v = ctypes.c_size_t()
    _check(load().svdq_linear_quantize_next_workspace(shape.c(), next_rank, flags, ctypes.byref(v)))
    return v.value


def svdq_linear_quantize_next(Qx: torch.Tensor, Sx: torch.Tensor, T: torch.Tensor | None, W: PreparedWeights,
                              next_inv_lambda: torch.Tensor, next_L1p: torch.Tensor | None, next_rank: int,
                              store_y: bool = False, out: tuple | None = None, workspace: torch.Tensor | None = None,
                              flags: int = 0):
    """svdq_linear whose epilogue also quantizes Y for the next layer (K' = N).
    Returns (next_Qx [M][N/2] uint8, next_Sx native uint8, next_T [M][next_rank] bf16 or None,
    Y [M][N] bf16 or None)."""
    M = Qx.shape[0]
    K, N, rank = W.shape.K, W.shape.N, W.shape.rank
    shape = LayerShape(M, K, N, rank)
    dev = Qx.device
    if out is None:
        _, sxb, _ = svdq_act_sizes(LayerShape(M, N, 128, next_rank))
        Qn = torch.empty(M, N // 2, dtype=torch.uint8, device=dev)
        Sn = torch.empty(sxb, dtype=torch.uint8, device=dev)
        Tn = torch.empty(M, next_rank, dtype=torch.bfloat16, device=dev) if next_rank else None
        Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev) if store_y else None
    else:
        Qn, Sn, Tn, Y = out
    need = svdq_linear_quantize_next_workspace(shape, next_rank, flags)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _check(load().svdq_linear_quantize_next(
        shape.c(), _ptr(Qx), _ptr(Sx), _ptr(T), _ptr(W.Qr), _ptr(W.Sr), _ptr(W.L2t), next_rank, _ptr(next_inv_lambda),
        _ptr(next_L1p), _ptr(Qn), _ptr(Sn), _ptr(Tn), _ptr(Y), _ptr(workspace), workspace.numel(), flags, _stream()))
    return Qn, Sn, Tn, Y


def svdq_scales_to_canonical(native: torch.Tensor, rows: int, K: int) -> torch.Tensor:
    out = torch.empty(rows, K // 16, dtype=torch.uint8, device=native.device)
    _check(load().svdq_scales_to_canonical(rows, K, _ptr(native), _ptr(out), _stream()))
    return out


def svdq_append_lowrank(W: PreparedWeights, A: torch.Tensor, B: torch.Tensor) -> PreparedWeights:
    """Prepared weights whose low-rank branch also carries the LoRA update
    X A^T B^T: A bf16 [extra][K], B bf16 [N][extra]. Qr/Sr are shared."""
    K, N, r = W.shape.K, W.shape.N, W.shape.rank
    extra = A.shape[0]
    L1p = torch.empty(r + extra, K, dtype=torch.bfloat16, device=A.device)
    L2t = torch.empty(N, r + extra, dtype=torch.bfloat16, device=A.device)
    _check(load().svdq_append_lowrank(W.shape.c(), extra, _ptr(W.L1p), _ptr(W.L2t), _ptr(A), _ptr(B), _ptr(L1p),
                                      _ptr(L2t), _stream()))
    return PreparedWeights(LayerShape(0, K, N, r + extra), W.Qr, W.Sr, L1p, L2t, W.lam, W.inv_lam)


# ---------------------------------------------------------------- INT4 variant

def svdq_int4_act_sizes(shape: LayerShape) -> tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().svdq_int4_act_sizes(shape.c(), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def svdq_int4_weight_sizes(shape: LayerShape) -> tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().svdq_int4_weight_sizes(shape.c(), ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


@dataclass
class Int4Weights:
    shape: LayerShape          # M is unused (0)
    Qr: torch.Tensor           # uint8 [N][K]: E4M3 bytes of the INT4 codes
    Sr: torch.Tensor           # fp32 [K/64][N]
    L2t: torch.Tensor | None   # shared with the NVFP4 preparation
    L1p: torch.Tensor | None
    inv_lam: torch.Tensor


def svdq_int4_prepare_weights(W_lin: torch.Tensor, P: PreparedWeights) -> Int4Weights:
    """INT4 encoding of the residual of an NVFP4-prepared layer (same smoothing
    and low-rank factors)."""
    N, K = W_lin.shape
    shape = LayerShape(0, K, N, P.shape.rank)
    qr, sr = svdq_int4_weight_sizes(shape)
    Qr = torch.empty(N, K, dtype=torch.uint8, device=W_lin.device)
    Sr = torch.empty(K // 64, N, dtype=torch.float32, device=W_lin.device)
    assert Qr.numel() == qr and Sr.numel() * 4 == sr
    _check(load().svdq_int4_quantize_residual(shape.c(), _ptr(W_lin), _ptr(P.lam), _ptr(P.L1p), _ptr(P.L2t), _ptr(Qr),
                                              _ptr(Sr), _stream()))
    return Int4Weights(shape, Qr, Sr, P.L2t, P.L1p, P.inv_lam)


def svdq_int4_quantize_act(X: torch.Tensor, inv_lambda: torch.Tensor, L1p: torch.Tensor | None, rank: int,
                           N: int = 128, out: tuple | None = None):
    """Returns (Qx [M][K] uint8 E4M3 bytes, Sx fp32 [K/64][ceil(M/128)*128], T [M][rank] bf16 or None)."""
    M, K = X.shape
    shape = LayerShape(M, K, N, rank)
    if out is None:
        Qx = torch.empty(M, K, dtype=torch.uint8, device=X.device)
        Sx = torch.empty(K // 64, (M + 127) // 128 * 128, dtype=torch.float32, device=X.device)
        T = torch.empty(M, rank, dtype=torch.bfloat16, device=X.device) if rank else None
    else:
        Qx, Sx, T = out
    _check(load().svdq_int4_quantize_act(shape.c(), _ptr(X), _ptr(inv_lambda), _ptr(L1p), _ptr(Qx), _ptr(Sx), _ptr(T),
                                         _stream()))
    return Qx, Sx, T


def svdq_int4_linear(Qx: torch.Tensor, Sx: torch.Tensor, T: torch.Tensor | None, W: Int4Weights,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    M = Qx.shape[0]
    K, N, rank = W.shape.K, W.shape.N, W.shape.rank
    shape = LayerShape(M, K, N, rank)
    Y = out if out is not None else torch.empty(M, N, dtype=torch.bfloat16, device=Qx.device)
    _check(load().svdq_int4_linear(shape.c(), _ptr(Qx), _ptr(Sx), _ptr(T), _ptr(W.Qr), _ptr(W.Sr), _ptr(W.L2t),
                                   _ptr(Y), _stream()))
    return Y


# ---------------------------------------------------------------- DeltaQuant

def svdq_deltaquant_sizes(F: int, H: int, W: int, C: int) -> tuple[int, int, int]:
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().svdq_deltaquant_sizes(F, H, W, C, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)))
    return a.value, b.value, c.value


def svdq_deltaquant_encode(X: torch.Tensor, dims: tuple[int, int, int], out: tuple | None = None):
    """Core + delta encoding of video tokens X bf16 [F*H*W][C] (2 x 2 x 2 blocks).
    Returns (core uint8 [blocks][C], delta codes uint8 [F*H*W][C/2], delta scales native uint8)."""
    F, H, W = dims
    C = X.shape[1]
    if out is None:
        cb, _, sb = svdq_deltaquant_sizes(F, H, W, C)
        core = torch.empty(cb // C, C, dtype=torch.uint8, device=X.device)
        Qd = torch.empty(F * H * W, C // 2, dtype=torch.uint8, device=X.device)
        Sd = torch.empty(sb, dtype=torch.uint8, device=X.device)
    else:
        core, Qd, Sd = out
    _check(load().svdq_deltaquant_encode(F, H, W, C, _ptr(X), _ptr(core), _ptr(Qd), _ptr(Sd), _stream()))
    return core, Qd, Sd


# ---------------------------------------------------------------- around the 4-bit linear layer
# W8A8 linear, layer norm and rotary positions. Rows may have a stride; every
# tensor of a call lives on one CUDA device, which need not be the current one.
# Parameters, positions, codes and statistics are contiguous, and every address is a
# multiple of 16 bytes; tensors that are not are refused.
# As everywhere in this module the calls stand outside autograd: results carry no
# graph, whatever the inputs require, and gradients come from calls of their own
# (svdq_layernorm_backward; svdq_rope with inverse=True).

_FLOAT_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _float_type(t: torch.Tensor, what: str) -> int:
    code = _FLOAT_TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bf16, fp16 or fp32, not {t.dtype}")
    return code


def _device(X: torch.Tensor, *others: torch.Tensor | None) -> int:
    """Index of the CUDA device that holds all the tensors of a call."""
    index = X.get_device()
    if index < 0:
        raise ValueError("tensors must live on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {X.device} and {t.device}: all must live on one CUDA device")
    return index


def _rows(t: torch.Tensor, what: str) -> tuple[int, int]:
    """(address, row stride) of a matrix whose rows are contiguous."""
    stride = t.stride()
    if len(stride) != 2 or (stride[1] != 1 and t.shape[1] > 1):
        raise ValueError(f"{what} must be a matrix with contiguous rows")
    return t.data_ptr(), stride[0]


def _dense(t: torch.Tensor | None, shape: tuple, dtype: torch.dtype, what: str) -> int | None:
    """Address of a contiguous tensor of this shape and type (None: no tensor)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"not {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _call(index: int, fn, *args) -> None:
    """fn(*args, stream) on the device's current stream, with the device current."""
    if index == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status)


@dataclass
class Int8Weights:
    """A W8A8 layer: codes and scales of lambda * W_lin per output channel, and
    what its calls multiply and add."""
    N: int
    K: int
    Qw: torch.Tensor                    # int8 [N][K]
    Sw: torch.Tensor                    # fp32 [N]
    inv_lam: torch.Tensor | None = None  # fp32 [K]: the activation's smoothing factors
    bias: torch.Tensor | None = None    # fp32 [N]


def svdq_int8_prepare_weights(W_lin: torch.Tensor, lam: torch.Tensor | None = None,
                              inv_lam: torch.Tensor | None = None, bias: torch.Tensor | None = None) -> Int8Weights:
    """8-bit codes of W_lin [N][K] (bf16, fp16 or fp32), one scale per output channel. lam and
    inv_lam fp32 [K]: smoothing factors, as svdq_prepare_weights returns them (both or neither)."""
    if (lam is None) != (inv_lam is None):
        raise ValueError("lam and inv_lam come together")
    dev = _device(W_lin, lam, inv_lam, bias)
    wt = _float_type(W_lin, "W_lin")
    wp, ldw = _rows(W_lin, "W_lin")
    N, K = W_lin.shape
    lp = _dense(lam, (K,), torch.float32, "lam")
    _dense(inv_lam, (K,), torch.float32, "inv_lam")
    if bias is not None:
        if bias.shape != (N,):
            raise ValueError(f"bias must have {N} values")
        bias = bias.float().contiguous()
    Qw = W_lin.new_empty(N, K, dtype=torch.int8)
    Sw = W_lin.new_empty(N, dtype=torch.float32)
    _call(dev, load().svdq_int8_quantize_weight, N, K, wt, wp, ldw, lp, Qw.data_ptr(), Sw.data_ptr())
    return Int8Weights(N, K, Qw, Sw, inv_lam, bias)


def svdq_int8_quantize_act(X: torch.Tensor, inv_lambda: torch.Tensor | None = None, out: tuple | None = None):
    """8-bit codes of X [M][K] (bf16, fp16 or fp32; rows may be strided), one scale per token.
    Returns (Qx int8 [M][K], Sx fp32 [M])."""
    dev = _device(X, inv_lambda)
    xt = _float_type(X, "X")
    xp, ldx = _rows(X, "X")
    M, K = X.shape
    lp = _dense(inv_lambda, (K,), torch.float32, "inv_lambda")
    if out is None:
        Qx = X.new_empty(M, K, dtype=torch.int8)
        Sx = X.new_empty(M, dtype=torch.float32)
        qp, sp = Qx.data_ptr(), Sx.data_ptr()
    else:
        Qx, Sx = out
        _device(X, Qx, Sx)
        qp, sp = _dense(Qx, (M, K), torch.int8, "Qx"), _dense(Sx, (M,), torch.float32, "Sx")
    _call(dev, load().svdq_int8_quantize_act, M, K, xt, xp, ldx, lp, qp, sp)
    return Qx, Sx


def svdq_int8_linear(Qx: torch.Tensor, Sx: torch.Tensor, W: Int8Weights, dtype: torch.dtype = torch.bfloat16,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Y [M][N] = Sx Sw (Qx Qw^T) + bias of a W8A8 layer, in dtype (or out's: rows may be strided)."""
    dev = _device(Qx, Sx, W.Qw, W.Sw, W.bias, out)
    M, K, N = Qx.shape[0], W.K, W.N
    Y = Qx.new_empty(M, N, dtype=dtype) if out is None else out
    if Y.shape != (M, N):
        raise ValueError(f"out must be [{M}][{N}]")
    yt = _float_type(Y, "out")
    yp, ldy = _rows(Y, "out")
    _call(dev, load().svdq_int8_linear, M, K, N, _dense(Qx, (M, K), torch.int8, "Qx"),
          _dense(Sx, (M,), torch.float32, "Sx"), _dense(W.Qw, (N, K), torch.int8, "Qw"),
          _dense(W.Sw, (N,), torch.float32, "Sw"), _dense(W.bias, (N,), torch.float32, "bias"), yt, yp, ldy)
    return Y


def _norm_params(X: torch.Tensor, weight: torch.Tensor | None, bias: torch.Tensor | None, rows_per_group: int | None):
    """(w_dtype, weight address, bias address, rows per group, groups) of a norm over X. weight and bias are [C], or
    [groups][C] for groups of rows_per_group rows (default: M / groups, which must be whole)."""
    M, C = X.shape
    first = weight if weight is not None else bias
    if first is None:
        rows = rows_per_group or 0
        if rows < 0:
            raise ValueError("rows_per_group must not be negative")
        return _FLOAT_TYPES[X.dtype], None, None, rows, -(-M // rows) if rows and M else 1
    dtype, shape = first.dtype, first.shape
    if dtype is not X.dtype and dtype is not torch.float32:
        raise ValueError(f"weight and bias must be {X.dtype} or torch.float32")
    if len(shape) == 1:
        if rows_per_group:
            raise ValueError("weight and bias of row groups are [groups][C]")
        rows, groups, want = 0, 1, (C,)
    else:
        groups = shape[0]
        want = (groups, C)
        rows = rows_per_group
        if rows is None:
            if groups < 1 or M % groups:
                raise ValueError(f"{M} rows do not divide into {groups} groups: give rows_per_group")
            rows = M // groups
        if M and (rows < 0 or groups != (-(-M // rows) if rows else 1)):
            raise ValueError(f"{M} rows in groups of {rows} do not have {groups} rows of weight and bias")
    return _FLOAT_TYPES[dtype], _dense(weight, want, dtype, "weight"), _dense(bias, want, dtype, "bias"), rows, groups


def svdq_layernorm(X: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                   eps: float = 1e-6, rows_per_group: int | None = None, add_one: bool = False,
                   out: torch.Tensor | None = None, stats: bool = True):
    """Layer norm of X's rows [M][C] (bf16, fp16 or fp32). weight and bias: [C], or [groups][C] for a modulated norm
    whose rows share them in groups of rows_per_group (default: M / groups); X's type or fp32. add_one: the weight is
    1 + weight. Returns (Y, mean, rstd): mean and rstd fp32 [M] for the backward pass (None with stats=False)."""
    dev = _device(X, weight, bias, out)
    xt = _float_type(X, "X")
    xp, ldx = _rows(X, "X")
    M, C = X.shape
    wt, wp, bp, rows, _ = _norm_params(X, weight, bias, rows_per_group)
    if out is None:
        out = X.new_empty(M, C)
        yp, ldy = out.data_ptr(), C
    else:
        if out.shape != X.shape or out.dtype != X.dtype:
            raise ValueError("out must have X's shape and type")
        yp, ldy = _rows(out, "out")
    mean = rstd = mp = rp = None
    if stats:
        mean = X.new_empty(M, dtype=torch.float32)
        rstd = X.new_empty(M, dtype=torch.float32)
        mp, rp = mean.data_ptr(), rstd.data_ptr()
    _call(dev, load().svdq_layernorm, M, C, xt, wt, xp, ldx, wp, bp, rows, eps, SVDQ_NORM_ADD_ONE if add_one else 0,
          yp, ldy, mp, rp)
    return out, mean, rstd


def svdq_int8_layernorm_quantize(X: torch.Tensor, weight: torch.Tensor | None = None,
                                 bias: torch.Tensor | None = None, inv_lambda: torch.Tensor | None = None,
                                 eps: float = 1e-6, rows_per_group: int | None = None, add_one: bool = False,
                                 out: tuple | None = None):
    """svdq_layernorm straight to the 8-bit codes of the next product: (Qx int8 [M][C], Sx fp32 [M]). The norm is not
    rounded to X's type before it is quantized."""
    dev = _device(X, weight, bias, inv_lambda)
    xt = _float_type(X, "X")
    xp, ldx = _rows(X, "X")
    M, C = X.shape
    wt, wp, bp, rows, _ = _norm_params(X, weight, bias, rows_per_group)
    lp = _dense(inv_lambda, (C,), torch.float32, "inv_lambda")
    if out is None:
        out = (X.new_empty(M, C, dtype=torch.int8), X.new_empty(M, dtype=torch.float32))
    Qx, Sx = out
    _device(X, Qx, Sx)
    _call(dev, load().svdq_int8_layernorm_quantize, M, C, xt, wt, xp, ldx, wp, bp, rows, eps,
          SVDQ_NORM_ADD_ONE if add_one else 0, lp, _dense(Qx, (M, C), torch.int8, "Qx"),
          _dense(Sx, (M,), torch.float32, "Sx"))
    return Qx, Sx


def svdq_layernorm_backward_workspace(M: int, C: int, rows_per_group: int = 0) -> int:
    v = ctypes.c_size_t()
    _check(load().svdq_layernorm_backward_workspace(M, C, rows_per_group, ctypes.byref(v)))
    return v.value


@functools.lru_cache(maxsize=1024)
def _backward_workspace(index: int, M: int, C: int, rows_per_group: int) -> int:
    with torch.cuda.device(index):
        return svdq_layernorm_backward_workspace(M, C, rows_per_group)


def svdq_layernorm_backward(dY: torch.Tensor, X: torch.Tensor, weight: torch.Tensor | None, mean: torch.Tensor,
                            rstd: torch.Tensor, rows_per_group: int | None = None, add_one: bool = False,
                            out: torch.Tensor | None = None, params: bool = True):
    """Gradients of svdq_layernorm: (dX in X's type, dweight, dbias). dweight and dbias are fp32, of weight's shape
    ([C] without a weight), or None with params=False."""
    dev = _device(X, dY, weight, mean, rstd, out)
    xt = _float_type(X, "X")
    xp, ldx = _rows(X, "X")
    M, C = X.shape
    if dY.shape != X.shape or dY.dtype != X.dtype:
        raise ValueError("dY must have X's shape and type")
    gp, ldg = _rows(dY, "dY")
    wt, wp, _, rows, groups = _norm_params(X, weight, None, rows_per_group)
    mp, rp = _dense(mean, (M,), torch.float32, "mean"), _dense(rstd, (M,), torch.float32, "rstd")
    if out is None:
        out = X.new_empty(M, C)
        op, ldo = out.data_ptr(), C
    else:
        if out.shape != X.shape or out.dtype != X.dtype:
            raise ValueError("out must have X's shape and type")
        op, ldo = _rows(out, "out")
    dw = db = dwp = dbp = work = kp = None
    ws = 0
    if params:
        shape = weight.shape if weight is not None else (C,) if groups == 1 else (groups, C)
        new = X.new_empty if M else X.new_zeros
        dw = new(shape, dtype=torch.float32)
        db = new(shape, dtype=torch.float32)
        dwp, dbp = dw.data_ptr(), db.data_ptr()
        ws = _backward_workspace(dev, M, C, rows)
        if ws:
            work = X.new_empty(ws, dtype=torch.uint8)
            kp = work.data_ptr()
    _call(dev, load().svdq_layernorm_backward, M, C, xt, wt, gp, ldg, xp, ldx, wp, mp, rp, rows,
          SVDQ_NORM_ADD_ONE if add_one else 0, op, ldo, dwp, dbp, kp, ws)
    return out, dw, db


class RopeTable:
    """The rotary frequencies of a head, laid out once: axis_dims (the elements of a head that each axis turns) and
    freqs fp64 [sum(axis_dims) / 2] on the device, pair by pair."""

    def __init__(self, axis_dims, freqs: torch.Tensor):
        self.axis_dims = tuple(int(d) for d in axis_dims)
        self.freqs = freqs
        if any(d < 2 or d % 2 for d in self.axis_dims):
            raise ValueError("every axis needs an even number of elements, at least 2")
        _dense(freqs, (sum(self.axis_dims) // 2,), torch.float64, "freqs")
        self._dims = (ctypes.c_int32 * len(self.axis_dims))(*self.axis_dims)


def svdq_rope_table(axis_dims, theta: float = 10000.0, device="cuda") -> RopeTable:
    """Frequencies theta^(-2i/d) for pair i of an axis of d elements."""
    freqs = [theta ** (-2.0 * i / d) for d in axis_dims for i in range(d // 2)]
    return RopeTable(axis_dims, torch.tensor(freqs, dtype=torch.float64, device=device))


def svdq_rope(X: torch.Tensor, positions: torch.Tensor, table: RopeTable, interleaved: bool = True,
              inverse: bool = False, out: torch.Tensor | None = None) -> torch.Tensor:
    """Turns the heads of X [T][heads][D] (bf16, fp16 or fp32; token and head strides are free, so X may be the query
    and key heads inside a merged QKV activation) by their tokens' positions [P][axes] (int32 or fp32; T a multiple
    of P). interleaved: pairs (2i, 2i+1), else (i, i + R/2). inverse: the gradient of the rotation. Returns out, or
    a new contiguous tensor; out may be X."""
    dev = _device(X, positions, table.freqs, out)
    xt = _float_type(X, "X")
    x_stride = X.stride()
    if len(x_stride) != 3 or x_stride[2] != 1:
        raise ValueError("X must be [T][heads][D] with contiguous heads")
    T, H, D = X.shape
    axes = len(table.axis_dims)
    if positions.dim() != 2 or positions.shape[1] != axes or not positions.is_contiguous() or \
            positions.dtype not in (torch.int32, torch.float32):
        raise ValueError(f"positions must be a contiguous int32 or fp32 [P][{axes}] tensor")
    if out is None:
        out = X.new_empty(T, H, D)
    elif out.shape != X.shape or out.dtype != X.dtype or out.stride(2) != 1:
        raise ValueError("out must have X's shape and type, and contiguous heads")
    y_stride = out.stride()
    _call(dev, load().svdq_rope, T, H, D, xt, X.data_ptr(), x_stride[0], x_stride[1], out.data_ptr(), y_stride[0],
          y_stride[1], positions.data_ptr(), DTYPES[positions.dtype], positions.shape[0], axes, table._dims,
          table.freqs.data_ptr(), (0 if interleaved else SVDQ_ROPE_HALVES) | (SVDQ_ROPE_INVERSE if inverse else 0))
    return out


def svdq_selftest_timeout() -> None:
    """Launch the failure-path diagnostic (a bounded wait that gives up after 2 s)."""
    _check(load().svdq_selftest_timeout(_stream()))


def svdq_check() -> None:
    _check(load().svdq_check(_stream()))
