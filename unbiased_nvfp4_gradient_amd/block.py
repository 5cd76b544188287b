"""A feed-forward block's products on MXFP4 operands with what follows them in one kernel, and their
backward pass, through the C ABI of include/nvfp4_block.h.

    f = mxfp4_linear_forward(a, b, bias, activation="gelu", residual=x, keep_z=True)
    f = mxfp4_gated_forward(a, b, activation="silu", keep_z=True)
    g = activation_backward(dy, f.z, "gelu", bias=True)
    g = gated_activation_backward(dy, f.z, "silu")

Element types are float32, bfloat16 and float16.  Work is enqueued on `stream`, by default the
current one.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import MXFP4, _as_mx, _check, _check_buffer, _check_mx_layout, _CMx, _cmx, _mx_dims, lib
from .training import TYPES, _as_rows, _device_tensor, _ptr, _where, _workspace

EXPORTED = ("mxfp4_linear_forward", "activation_backward_workspace_bytes",
            "activation_backward")

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_ready = None


def _lib() -> ctypes.CDLL:
    """The library with this module's entry points declared."""
    global _ready
    if _ready is None:
        h = lib()
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        MP = ctypes.POINTER(_CMx)
        h.mxfp4_linear_forward.argtypes = [MP, MP, i64, i64, i64, i32, i32, i32, i32, i32, P, P, i64,
                                           P, P, P]
        h.activation_backward_workspace_bytes.argtypes = [i32, i32, i64, i64]
        h.activation_backward.argtypes = [i32, i32, i32, i32, P, i64, P, i64, i64, i64, P, P, P,
                                          sz, P]
        for name in EXPORTED:
            getattr(h, name).restype = sz if name.endswith("_bytes") else i32
        _ready = h
    return _ready


class MXLinearForward(NamedTuple):
    y: torch.Tensor
    z: Optional[torch.Tensor]       # what the activation was taken of, if it was to be kept


class ActivationBackward(NamedTuple):
    dz: torch.Tensor
    dbias: Optional[torch.Tensor]


def _activation(kind) -> int:
    if kind not in ACTIVATIONS:
        raise ValueError(f"unknown activation {kind!r}; use one of {tuple(ACTIVATIONS)}")
    return ACTIVATIONS[kind]


def _forward(a, b, bias, activation, residual, gated, rotated_pair, dtype, keep_z,
             stream) -> MXLinearForward:
    kind = _activation(activation)
    if dtype not in TYPES:
        raise ValueError(f"dtype must be one of {tuple(TYPES)}; got {dtype}")
    a, b = _as_mx(a, "a"), _as_mx(b, "b")
    if bool(a.k_tiled) != bool(b.k_tiled):
        raise ValueError("a and b must both be row-major or both K-tiled")
    M, K = _mx_dims(a, "a")
    rows, _ = _mx_dims(b, "b")
    device = a.codes.device
    if device.type != "cuda":
        raise ValueError(f"a and b must be on a GPU; got {device}")
    a, b = _check_mx_layout(a, "a", M, K, device), _check_mx_layout(b, "b", rows, K, device)
    if K % 128:
        raise ValueError(f"K = {K} must be a multiple of 128")
    if gated and rows % 2:
        raise ValueError(f"b must hold as many rows for the gate as for up; got {rows}")
    n = rows // 2 if gated else rows
    if bias is not None:
        _device_tensor(bias, "bias", (dtype,) if dtype is torch.float32 else (dtype, torch.float32))
        _check_buffer(bias, "bias", bias.dtype, (rows,), device)
    r_stride = n
    if residual is not None:
        _device_tensor(residual, "residual", (dtype,))
        if residual.shape != (M, n) or residual.device != device:
            raise ValueError(f"residual must have the shape {(M, n)} on {device}; got "
                             f"{tuple(residual.shape)} on {residual.device}")
        if residual.numel():
            r_stride = _as_rows(residual, "residual")[2]
    L = _lib()
    where, raw = _where(stream, device)
    with where:
        y = torch.empty((M, n), dtype=dtype, device=device)
        z = torch.empty((M, rows), dtype=dtype, device=device) if keep_z else None
        _check("mxfp4_linear_forward", L.mxfp4_linear_forward(
            _cmx(a), _cmx(b), M, n, K, int(bool(rotated_pair)), int(gated), kind, TYPES[dtype],
            TYPES[dtype if bias is None else bias.dtype], _ptr(bias), _ptr(residual), r_stride,
            y.data_ptr(), _ptr(z), raw))
    return MXLinearForward(y, z)


def mxfp4_linear_forward(a: MXFP4, b: MXFP4, bias: Optional[torch.Tensor] = None,
                         activation: str = "none", residual: Optional[torch.Tensor] = None,
                         rotated_pair: bool = False, dtype: torch.dtype = torch.bfloat16,
                         keep_z: bool = False, stream=None) -> MXLinearForward:
    """y = act(z) + residual with z = A B^T + bias, of two MXFP4 row-layout operands ([M, K] and
    [n, K]; both row-major or both K-tiled, as for mxfp4_gemm, but of any M and n), in one kernel.
    bias [n] has the type `dtype` or float32, residual [M, n] (rows at one distance) the type
    `dtype`, as have y and, with `keep_z`, z."""
    return _forward(a, b, bias, activation, residual, False, rotated_pair, dtype, keep_z, stream)


def mxfp4_gated_forward(a: MXFP4, b: MXFP4, bias: Optional[torch.Tensor] = None,
                        activation: str = "silu", rotated_pair: bool = False,
                        dtype: torch.dtype = torch.bfloat16, keep_z: bool = False,
                        stream=None) -> MXLinearForward:
    """y = act(gate) up with (gate, up) = A B^T + bias: both projections of a gated feed-forward
    layer, the activation and the product in one kernel.  b [2n, K] holds the gate's rows, then
    up's; y is [M, n], and with `keep_z` z is [M, 2n], gate and up side by side."""
    return _forward(a, b, bias, activation, None, True, rotated_pair, dtype, keep_z, stream)


def _backward(dy, z, activation, gated, bias, bias_type, stream) -> ActivationBackward:
    kind = _activation(activation)
    _device_tensor(dy, "dy")
    rows, n, dy_stride = _as_rows(dy, "dy")
    wide = (2 if gated else 1) * n
    z_stride = wide
    if z is None and (gated or kind):
        raise ValueError("z is needed for the derivative")
    if z is not None:
        _device_tensor(z, "z", (dy.dtype,))
        if z.shape != (*dy.shape[:-1], wide) or z.device != dy.device:
            raise ValueError(f"z must have the shape {(*dy.shape[:-1], wide)} and dy's device; got "
                             f"{tuple(z.shape)} on {z.device}")
        z_stride = _as_rows(z, "z")[2]
    if bias_type is None:
        bias_type = dy.dtype
    if bias_type not in (dy.dtype, torch.float32):
        raise ValueError(f"bias_type must be {dy.dtype} or float32; got {bias_type}")
    L = _lib()
    where, raw = _where(stream, dy.device)
    with where:
        dz = torch.empty((*dy.shape[:-1], wide), dtype=dy.dtype, device=dy.device)
        dbias = ws = None
        nbytes = 0
        if bias:
            dbias = torch.empty((wide,), dtype=bias_type, device=dy.device)
            nbytes = L.activation_backward_workspace_bytes(TYPES[dy.dtype], int(gated), rows, n)
            ws = _workspace(nbytes, dy.device) if nbytes else None
        _check("activation_backward", L.activation_backward(
            TYPES[dy.dtype], TYPES[bias_type], kind, int(gated), dy.data_ptr(), dy_stride, _ptr(z),
            z_stride, rows, n, dz.data_ptr(), _ptr(dbias), _ptr(ws), nbytes, raw))
    return ActivationBackward(dz, dbias)


def activation_backward(dy: torch.Tensor, z: Optional[torch.Tensor], activation: str = "none",
                        bias: bool = False, bias_type: Optional[torch.dtype] = None,
                        stream=None) -> ActivationBackward:
    """dz = dy act'(z) of y = act(z), and where `bias` asks for it the sum of dz over the rows (in
    dy's type, or in bias_type: that or float32), taken before dz is rounded.  z (of dy's shape and
    type) may be None for the activation "none"."""
    return _backward(dy, z, activation, False, bias, bias_type, stream)


def gated_activation_backward(dy: torch.Tensor, z: torch.Tensor, activation: str = "silu",
                              bias: bool = False, bias_type: Optional[torch.dtype] = None,
                              stream=None) -> ActivationBackward:
    """The gradient dz of z = (gate, up), side by side in the last dimension, for dy of
    y = act(gate) up; dbias as in activation_backward, over both."""
    return _backward(dy, z, activation, True, bias, bias_type, stream)
