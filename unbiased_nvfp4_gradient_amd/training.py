"""The operators around the quantized linear layer in a training step: layer norm, softmax
cross entropy of a linear head over a large vocabulary, and the global gradient norm with
clipping.  They run in this package's HIP kernels through the C ABI of include/nvfp4_train.h;
this module checks and marshals arguments and adds autograd functions and modules.

    y, mean, rstd = layer_norm_forward(x, weight, bias)
    dx, dweight, dbias = layer_norm_backward(dy, x, mean, rstd, weight, bias=True)
    loss, lse = linear_cross_entropy_forward(h, w, target)
    dh, dw = linear_cross_entropy_backward(dloss, h, w, target, lse)
    norm = clip_grads(grads, max_norm)

Element types are float32, bfloat16 and float16 (the linear head's loss: the last two).  Work is
enqueued on `stream`, by default the current one; tensors used on another stream than their own
are the caller's to order and to keep, as everywhere in torch.

Every call can be captured into a graph, and so can a backward pass through the autograd
functions.  Before one is captured, the graphs of eager passes over the same parameters have to
be gone (losses deleted): torch runs a parameter's accumulation on the stream of the oldest pass
that still lives, and leaving a capture's stream ends the process.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import NamedTuple, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import _check, _check_buffer, lib

EXPORTED = ("layer_norm_forward", "layer_norm_workspace_bytes", "layer_norm_backward",
            "linear_cross_entropy_workspace_bytes", "linear_cross_entropy_forward",
            "linear_cross_entropy_backward", "grad_norm_workspace_bytes", "grad_norm",
            "clip_grads")

TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
REDUCTIONS = {"sum": 0, "mean": 1, "none": 2}

_ready = None


def _lib() -> ctypes.CDLL:
    """The library with this module's entry points declared."""
    global _ready
    if _ready is None:
        h = lib()
        P, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                ctypes.c_size_t)
        h.layer_norm_forward.argtypes = [i32, i32, P, P, P, i64, i64, i64, f32, P, P, P, P]
        h.layer_norm_workspace_bytes.argtypes = [i32, i64, i64]
        h.layer_norm_backward.argtypes = [i32, i32, P, P, P, P, P, i64, i64, i64, i64, P, P, P, P,
                                          sz, P]
        h.linear_cross_entropy_workspace_bytes.argtypes = [i32, i64, i64, i64]
        h.linear_cross_entropy_forward.argtypes = [i32, P, i64, P, i64, P, i64, i64, i64, i64,
                                                   i32, P, P, P, sz, P]
        h.linear_cross_entropy_backward.argtypes = [i32, P, P, i64, P, i64, P, P, i64, i64, i64,
                                                    i64, i32, P, P, P, sz, P]
        h.grad_norm_workspace_bytes.argtypes = [P, i64]
        h.grad_norm.argtypes = [P, P, P, i64, i32, P, P, sz, P]
        h.clip_grads.argtypes = [P, P, P, P, i64, f32, i32, P, P, sz, P]
        for name in EXPORTED:
            getattr(h, name).restype = sz if name.endswith("_bytes") else i32
        _ready = h
    return _ready


class LayerNormForward(NamedTuple):
    y: torch.Tensor
    mean: torch.Tensor              # float32, one per row
    rstd: torch.Tensor              # float32, one per row


class LayerNormBackward(NamedTuple):
    dx: torch.Tensor
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class LinearCrossEntropyForward(NamedTuple):
    loss: torch.Tensor              # float32: [t] for "none", else [1]
    lse: torch.Tensor               # float32 [t]


class LinearCrossEntropyBackward(NamedTuple):
    dh: Optional[torch.Tensor]
    dw: Optional[torch.Tensor]


_SAME = contextlib.nullcontext()


def _where(stream, device):
    """(context in which outputs and workspaces are allocated and the call is made, raw stream):
    those of the stream the call is enqueued on, so that a freed workspace goes only to later
    work on it, with the tensors' device current."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
        return (_SAME if device.index == torch._C._cuda_getDevice() else torch.cuda.device(device),
                raw)
    if stream.device != device:
        raise ValueError(f"stream must be one of the tensors' device, {device}; got one of "
                         f"{stream.device}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _like(x: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of x's shape and type."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _device_tensor(t, name: str, types=tuple(TYPES)):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in types:
        got = f"{t.dtype} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__
        raise ValueError(f"{name} must be a device tensor of "
                         f"{', '.join(str(x)[6:] for x in types)}; got {got}")


def _as_rows(t: torch.Tensor, name: str):
    """(rows, n, row stride) of a tensor whose last dimension is a row: any strides where its
    rows lie at one distance from each other and a row's elements are adjacent."""
    if t.dim() == 0 or t.shape[-1] == 0:
        raise ValueError(f"{name} must have a last dimension of at least one element; got "
                         f"{tuple(t.shape)}")
    n = t.shape[-1]
    if t.is_contiguous():
        return t.numel() // n, n, n
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous; got strides {t.stride()}")
    if t.dim() == 1:
        return 1, n, n
    try:
        flat = t.view(-1, n)
    except RuntimeError:
        raise ValueError(f"{name}'s rows must lie at one distance from each other; got shape "
                         f"{tuple(t.shape)}, strides {t.stride()}") from None
    stride = flat.stride(0) if flat.shape[0] > 1 else n
    if stride < n:
        raise ValueError(f"{name}'s rows overlap (stride {stride} for rows of {n})")
    return flat.shape[0], n, stride


def _check_parameters(x, params, n: int) -> torch.dtype:
    """The common type of the given weight and bias: x's own or float32."""
    found = None
    for name, p in params:
        if p is None:
            continue
        if not isinstance(p, torch.Tensor):
            _device_tensor(p, name)
        kind = p.dtype
        if found is not None and kind is not found:
            raise ValueError("weight and bias must be of one type")
        found = kind
        if kind is not x.dtype and kind is not torch.float32:
            _device_tensor(p, name)
            raise ValueError(f"{name} must be {x.dtype} or float32; got {kind}")
        if p.dim() != 1 or p.numel() != n or p.device != x.device or not p.is_contiguous():
            _check_buffer(p, name, kind, (n,), x.device)
    return x.dtype if found is None else found


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, eps: float = 1e-5,
                       stream=None) -> LayerNormForward:
    """Layer norm over the last dimension of x.  weight and bias have x's type or float32; the
    statistics are float32 in the shape of x's other dimensions."""
    _device_tensor(x, "x")
    rows, n, stride = _as_rows(x, "x")
    p_type = _check_parameters(x, (("weight", weight), ("bias", bias)), n)
    where, raw = _where(stream, x.device)
    with where:
        y = _like(x)
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        _check("layer_norm_forward", _lib().layer_norm_forward(
            TYPES[x.dtype], TYPES[p_type], x.data_ptr(), _ptr(weight), _ptr(bias), rows, n, stride,
            eps, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), raw))
    return LayerNormForward(y, mean, rstd)


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                        bias: bool = False, stream=None, bias_type: Optional[torch.dtype] = None,
                        need_dweight: bool = True) -> LayerNormBackward:
    """Gradients of layer_norm_forward: dx, dweight where there is a weight and `need_dweight`,
    and dbias where `bias` asks for it (in the weight's type; without one in `bias_type`, x's
    by default, or float32)."""
    _device_tensor(x, "x")
    _device_tensor(dy, "dy", (x.dtype,))
    if dy.shape != x.shape or dy.device != x.device:
        raise ValueError(f"dy must have x's shape and device; got {tuple(dy.shape)} on "
                         f"{dy.device} for {tuple(x.shape)} on {x.device}")
    rows, n, x_stride = _as_rows(x, "x")
    _, _, dy_stride = _as_rows(dy, "dy")
    p_type = _check_parameters(x, (("weight", weight),), n)
    if bias_type is not None:
        if bias_type not in ((x.dtype, torch.float32) if weight is None else (p_type,)):
            raise ValueError(f"bias_type must be the weight's type, or without one {x.dtype} or "
                             f"float32; got {bias_type}")
        p_type = bias_type
    for name, s in (("mean", mean), ("rstd", rstd)):
        _check_buffer(s, name, torch.float32, x.shape[:-1], x.device)
    L = _lib()
    where, raw = _where(stream, x.device)
    with where:
        dx = _like(x)
        dweight = dbias = ws = None
        if weight is not None and need_dweight:
            dweight = torch.empty((n,), dtype=p_type, device=x.device)
        if bias:
            dbias = torch.empty((n,), dtype=p_type, device=x.device)
        nbytes = 0
        if dweight is not None or bias:
            nbytes = L.layer_norm_workspace_bytes(TYPES[x.dtype], rows, n)
            ws = _workspace(nbytes, x.device)
        _check("layer_norm_backward", L.layer_norm_backward(
            TYPES[x.dtype], TYPES[p_type], dy.data_ptr(), x.data_ptr(), mean.data_ptr(),
            rstd.data_ptr(), _ptr(weight), rows, n, dy_stride, x_stride, dx.data_ptr(),
            _ptr(dweight), _ptr(dbias), _ptr(ws), nbytes, raw))
    return LayerNormBackward(dx, dweight, dbias)


def _check_loss(h, w, target, reduction):
    """(t, d, v, row strides of h and w) of the loss's arguments."""
    _device_tensor(h, "h", (torch.bfloat16, torch.float16))
    _device_tensor(w, "w", (h.dtype,))
    _device_tensor(target, "target", (torch.int64,))
    if reduction not in REDUCTIONS:
        raise ValueError(f"unknown reduction {reduction!r}; use one of {tuple(REDUCTIONS)}")
    if h.dim() != 2 or w.dim() != 2 or h.shape[1] != w.shape[1]:
        raise ValueError(f"need h [t, d] and w [v, d], got {tuple(h.shape)} and "
                         f"{tuple(w.shape)}")
    if w.shape[0] == 0 or w.shape[1] == 0:
        raise ValueError(f"w must not be empty; got {tuple(w.shape)}")
    if w.device != h.device:
        raise ValueError("h and w must be on one device")
    _check_buffer(target, "target", torch.int64, (h.shape[0],), h.device)
    return h.shape[0], h.shape[1], w.shape[0], _as_rows(h, "h")[2], _as_rows(w, "w")[2]


def linear_cross_entropy_forward(h: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                                 ignore_index: int = -100, reduction: str = "mean",
                                 stream=None) -> LinearCrossEntropyForward:
    """Cross entropy of the logits h w^T (h [t, d], w [v, d], bfloat16 or float16) against
    target [t] (int64), without holding the logits.  Tokens whose target is ignore_index do
    not count: their loss and lse are 0, and the mean is over the others (0 if there are
    none).  Any other target outside [0, v) makes the token's loss NaN."""
    t, d, v, h_stride, w_stride = _check_loss(h, w, target, reduction)
    L = _lib()
    where, raw = _where(stream, h.device)
    with where:
        loss = torch.empty((t if reduction == "none" else 1,), dtype=torch.float32,
                           device=h.device)
        lse = torch.empty((t,), dtype=torch.float32, device=h.device)
        nbytes = L.linear_cross_entropy_workspace_bytes(0, t, d, v)
        ws = _workspace(nbytes, h.device)
        _check("linear_cross_entropy_forward", L.linear_cross_entropy_forward(
            TYPES[h.dtype], h.data_ptr(), h_stride, w.data_ptr(), w_stride, target.data_ptr(), t,
            d, v, ignore_index, REDUCTIONS[reduction], loss.data_ptr(), lse.data_ptr(), ws.data_ptr(),
            nbytes, raw))
    return LinearCrossEntropyForward(loss, lse)


def linear_cross_entropy_backward(dloss: torch.Tensor, h: torch.Tensor, w: torch.Tensor,
                                  target: torch.Tensor, lse: torch.Tensor,
                                  ignore_index: int = -100, reduction: str = "mean",
                                  need_dh: bool = True, need_dw: bool = True,
                                  stream=None) -> LinearCrossEntropyBackward:
    """Gradients of linear_cross_entropy_forward's loss for h and w.  dloss is float32, [t] for
    the reduction "none" and [1] otherwise; lse is the forward pass's."""
    t, d, v, h_stride, w_stride = _check_loss(h, w, target, reduction)
    _check_buffer(dloss, "dloss", torch.float32, (t if reduction == "none" else 1,), h.device)
    _check_buffer(lse, "lse", torch.float32, (t,), h.device)
    L = _lib()
    where, raw = _where(stream, h.device)
    with where:
        dh = torch.empty((t, d), dtype=h.dtype, device=h.device) if need_dh else None
        dw = torch.empty((v, d), dtype=h.dtype, device=h.device) if need_dw else None
        nbytes = L.linear_cross_entropy_workspace_bytes(1, t, d, v)
        ws = _workspace(nbytes, h.device)
        _check("linear_cross_entropy_backward", L.linear_cross_entropy_backward(
            TYPES[h.dtype], dloss.data_ptr(), h.data_ptr(), h_stride, w.data_ptr(), w_stride,
            target.data_ptr(), lse.data_ptr(), t, d, v, ignore_index, REDUCTIONS[reduction],
            _ptr(dh), _ptr(dw), ws.data_ptr(), nbytes, raw))
    return LinearCrossEntropyBackward(dh, dw)


def _tensors_module():
    """The reader of tensor lists."""
    global _tensors
    if _tensors is None:
        try:
            from . import _tensors as module
        except ImportError as e:
            raise RuntimeError("_tensors.so is missing: build it with `python "
                               "-m unbiased_nvfp4_gradient_amd.build`") from e
        _tensors = module
    return _tensors


def _table(tensors: list, name: str):
    """(device index, addresses, sizes, types) of a list of contiguous device tensors, the last
    three as the C ABI's arrays."""
    return _tensors_module().table(tensors, name)


_tensors = None


def _norm_kind(norm_type) -> int:
    if norm_type == 2 or norm_type == math.inf:
        return int(norm_type == math.inf)
    raise ValueError(f"norm_type must be 2 or infinity; got {norm_type!r}")


def _norm_call(grads, norm_type, stream, clip=None):
    kind = _norm_kind(norm_type)
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    index, ptrs, sizes, types = _table(grads, "grads")
    n = len(grads)
    device = grads[0].device
    outs = None
    if clip is not None:
        max_norm, out = clip
        if not max_norm >= 0:
            raise ValueError(f"max_norm must not be negative; got {max_norm}")
        outs = ptrs
        if out is not None:
            out = list(out)
            if len(out) != n:
                raise ValueError(f"out must hold {n} tensors; got {len(out)}")
            o_index, outs, o_sizes, o_types = _table(out, "out")
            if o_index != index or o_types != types or o_sizes != sizes:
                raise ValueError("out must match grads in sizes, types and device")
    L = _lib()
    where, raw = _where(stream, device)
    with where:
        norm = torch.empty((1,), dtype=torch.float32, device=device)
        nbytes = L.grad_norm_workspace_bytes(sizes, n)
        ws = _workspace(nbytes, device)
        if clip is None:
            _check("grad_norm", L.grad_norm(ptrs, sizes, types, n, kind, norm.data_ptr(),
                                            ws.data_ptr(), nbytes, raw))
        else:
            _check("clip_grads", L.clip_grads(ptrs, outs, sizes, types, n, max_norm, kind,
                                              norm.data_ptr(), ws.data_ptr(), nbytes, raw))
            _tensors.written(grads if out is None else out)
    return norm


def grad_norm(grads: Sequence[torch.Tensor], norm_type: float = 2.0,
              stream=None) -> torch.Tensor:
    """The norm over all elements of all tensors together (2, or infinity: the largest
    magnitude), float32 [1].  The tensors may differ in size and type."""
    return _norm_call(grads, norm_type, stream)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, norm_type: float = 2.0,
               out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> torch.Tensor:
    """Scales the tensors by min(1, max_norm / (norm + 1e-6)), in place or into `out` (of the
    same sizes and types), and returns the norm before it, float32 [1].  A NaN norm makes all
    of them NaN; nothing is copied to the host to find out.  Tensors that are written must not
    share memory with each other or with one that is read.  To autograd they are changed in place,
    whatever the factor."""
    return _norm_call(grads, norm_type, stream, (max_norm, out))


class LayerNormFunction(torch.autograd.Function):
    """layer_norm_forward and layer_norm_backward in autograd."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps: float):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, mean, rstd, weight)
        ctx.bias_type = bias.dtype if bias is not None else None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, mean, rstd, weight = ctx.saved_tensors
        _, need_dweight, need_dbias, _ = ctx.needs_input_grad
        g = layer_norm_backward(dy.to(x.dtype).contiguous(), x, mean, rstd, weight,
                                bias=need_dbias, bias_type=ctx.bias_type,
                                need_dweight=need_dweight)
        return g.dx, g.dweight, g.dbias, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over the last dimension of x."""
    return LayerNormFunction.apply(x, weight, bias, eps)


class LinearCrossEntropyFunction(torch.autograd.Function):
    """linear_cross_entropy_forward and _backward in autograd."""

    @staticmethod
    def forward(ctx, h, w, target, ignore_index: int, reduction: str):
        loss, lse = linear_cross_entropy_forward(h, w, target, ignore_index, reduction)
        ctx.save_for_backward(h, w, target, lse)
        ctx.args = (ignore_index, reduction)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        h, w, target, lse = ctx.saved_tensors
        need_dh, need_dw = ctx.needs_input_grad[:2]
        g = linear_cross_entropy_backward(dloss.to(torch.float32).contiguous(), h, w, target, lse,
                                          *ctx.args, need_dh=need_dh, need_dw=need_dw)
        return g.dh, g.dw, None, None, None


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, target: torch.Tensor,
                         ignore_index: int = -100, reduction: str = "mean") -> torch.Tensor:
    """Differentiable linear_cross_entropy_forward: the loss, [t] for "none" and [1] otherwise."""
    return LinearCrossEntropyFunction.apply(h, w, target, ignore_index, reduction)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension with a weight and, by default, a bias."""

    def __init__(self, features: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype=torch.float32):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(features, device=device, dtype=dtype)) \
            if bias else None

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return layer_norm(x, self.weight, self.bias, self.eps)
