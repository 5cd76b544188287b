"""AdamW over many tensors at once, with moments in 32 or 8 bits, through the C ABI of
include/nvfp4_block.h.

    states = [adamw_state(p, bits=8) for p in params]
    norm = grad_norm(grads)
    adamw_step(params, grads, states, step=1, lr=3e-4, norm=norm, max_norm=1.0, seed=1)

or, as an optimizer of torch's kind, `AdamW(model.parameters(), lr=3e-4, bits=8)`.

Moments in 8 bits take a quarter of the memory and of its traffic: blocks of 128 elements below one
power of two each, a code of 8 bits for an element, rounded stochastically from `seed`, the
parameter's place in the list and the step (include/nvfp4_block.h has the format).  AdamW keeps its
updates bounded where a block's gradients differ widely (`bounded` in adamw_step).  A parameter of
16 bits can have a float32 master, which the step updates and rounds to it.
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Sequence

import torch

from . import _check, _check_buffer, lib
from . import training
from .training import TYPES, _where

EXPORTED = ("adamw_step", "adamw_moment_values")

MOMENT_BLOCK = 128


class _CAdamWOptions(ctypes.Structure):
    _fields_ = [(name, ctypes.c_double) for name in ("lr", "beta1", "beta2", "eps",
                                                     "weight_decay")] + \
               [("step", ctypes.c_int64), ("lr_device", ctypes.c_void_p),
                ("step_device", ctypes.c_void_p), ("norm", ctypes.c_void_p),
                ("max_norm", ctypes.c_float), ("bounded", ctypes.c_int32),
                ("seed", ctypes.c_uint64)]


_ready = None


def _lib() -> ctypes.CDLL:
    """The library with this module's entry points declared."""
    global _ready
    if _ready is None:
        h = lib()
        P, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        h.adamw_step.argtypes = [P, i64, ctypes.POINTER(_CAdamWOptions), P]
        h.adamw_moment_values.argtypes = [P, P, i64, i32, P, P]
        for name in EXPORTED:
            getattr(h, name).restype = i32
        _ready = h
    return _ready


class AdamWState(NamedTuple):
    """What AdamW keeps of one parameter of n elements."""
    m: torch.Tensor                              # float32 of n elements; 8 bits: codes uint8
    v: torch.Tensor                              # [blocks, 128], of m and of sqrt(v)
    m_scale: Optional[torch.Tensor] = None       # 8 bits: uint8 [blocks]
    v_scale: Optional[torch.Tensor] = None
    master: Optional[torch.Tensor] = None        # float32 of n elements


def adamw_state(param: torch.Tensor, bits: int = 32, master: bool = False,
                stream=None) -> AdamWState:
    """The state before a parameter's first step: zeros, and with `master` (for parameters of 16
    bits) a float32 copy of it."""
    if not isinstance(param, torch.Tensor) or param.dtype not in TYPES:
        got = param.dtype if isinstance(param, torch.Tensor) else type(param).__name__
        raise ValueError(f"param must be a float32, bfloat16 or float16 tensor; got {got}")
    if bits not in (32, 8):
        raise ValueError(f"bits must be 32 or 8; got {bits}")
    if master and param.dtype is torch.float32:
        raise ValueError("a float32 parameter is its own master")
    where = training._SAME if stream is None else torch.cuda.stream(stream)
    with where, torch.no_grad():
        def zeros(dtype, *shape):
            return torch.zeros(shape, dtype=dtype, device=param.device)
        copy = param.detach().float().contiguous() if master else None
        if bits == 32:
            return AdamWState(zeros(torch.float32, *param.shape), zeros(torch.float32, *param.shape),
                              master=copy)
        blocks = -(-param.numel() // MOMENT_BLOCK)
        return AdamWState(zeros(torch.uint8, blocks, MOMENT_BLOCK),
                          zeros(torch.uint8, blocks, MOMENT_BLOCK), zeros(torch.uint8, blocks),
                          zeros(torch.uint8, blocks), copy)


def _device_number(t, name: str, dtype, device):
    """A number that is read on the device."""
    if t.dtype != dtype or t.device != device or t.numel() != 1:
        raise ValueError(f"{name} must be a number or a {dtype} tensor of one element on {device}; "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _whole(step) -> int:
    number = int(step)
    if number != step or not 1 <= number < 1 << 63:
        raise ValueError(f"step must be a whole number from 1; got {step}")
    return number


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               states: Sequence[AdamWState], step, lr, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 1e-2, norm: Optional[torch.Tensor] = None,
               max_norm: Optional[float] = None, seed: int = 0, stream=None,
               bounded: bool = False) -> None:
    """AdamW step number `step` (from 1) of all parameters, in place.  All tensors are
    contiguous, and a gradient has its parameter's type and size.  With `norm` (float32 [1], of all gradients: grad_norm) the
    gradients are taken times min(1, max_norm / (norm + 1e-6)), and are left as they are.
    `step` and `lr` can be tensors of one element on the device (int64, float32), which a captured
    call reads at each replay.  Tensors that are written must not share memory with any other.

    With `bounded`, as AdamW has it, a second moment in 8 bits that is not 0 keeps a code of at least
    1: training wants it.  Without, its codes are plain stochastic rounding's, and where the gradients
    of 128 neighbours differ by 10^5 and more single updates reach hundreds of lr."""
    params, grads, states = list(params), list(grads), list(states)
    if not params:
        raise ValueError("params must hold at least one tensor")
    if (norm is None) != (max_norm is None):
        raise ValueError("norm and max_norm go together")
    index, table, written = training._tensors_module().adamw(params, grads, states)
    device = params[0].device
    beta1, beta2 = betas
    o = _CAdamWOptions(beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                       seed=int(seed) & (1 << 64) - 1, max_norm=0.0, bounded=int(bool(bounded)))
    if isinstance(step, torch.Tensor) and step.is_cuda:
        o.step_device = _device_number(step, "step", torch.int64, device)
    else:
        o.step = _whole(step)
    if isinstance(lr, torch.Tensor) and lr.is_cuda:
        o.lr_device = _device_number(lr, "lr", torch.float32, device)
    else:
        o.lr = float(lr)
    if norm is not None:
        _check_buffer(norm, "norm", torch.float32, (1,), device)
        if not max_norm >= 0:
            raise ValueError(f"max_norm must not be negative; got {max_norm}")
        o.norm, o.max_norm = norm.data_ptr(), max_norm
    L = _lib()
    where, raw = _where(stream, device)
    with where:
        _check("adamw_step", L.adamw_step(table, len(params), ctypes.byref(o), raw))
    training._tensors_module().written(written)


def moment_values(codes: torch.Tensor, scales: torch.Tensor, second: bool = False,
                  stream=None) -> torch.Tensor:
    """The float32 values [blocks, 128] of an 8-bit moment: m, or with `second` sqrt(v)."""
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dim() != 2:
        raise ValueError("codes must be a 2-D uint8 device tensor")
    blocks = codes.shape[0]
    _check_buffer(codes, "codes", torch.uint8, (blocks, MOMENT_BLOCK), codes.device)
    _check_buffer(scales, "scales", torch.uint8, (blocks,), codes.device)
    L = _lib()
    where, raw = _where(stream, codes.device)
    with where:
        out = torch.empty((blocks, MOMENT_BLOCK), dtype=torch.float32, device=codes.device)
        _check("adamw_moment_values", L.adamw_moment_values(
            codes.data_ptr(), scales.data_ptr(), blocks, int(bool(second)), out.data_ptr(), raw))
    return out


class AdamW(torch.optim.Optimizer):
    """AdamW in one call a step for each group of parameters.  `bits`, `master` and the usual
    numbers can differ from group to group; parameters of float32 have no master.  `step` can take
    the gradients' norm and clip by it on the way (see adamw_step).  A master is taken from its
    parameter at the first step and leads from then on: a parameter that is set to something else
    later needs its state removed (`del optimizer.state[p]`)."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, bits: int = 32, master: bool = False, seed: int = 0):
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                                      bits=bits, master=master, seed=int(seed)))

    def add_param_group(self, group):
        new = {**self.defaults, **group}                # refused before it is one of the groups
        if new["bits"] not in (32, 8):
            raise ValueError(f"bits must be 32 or 8; got {new['bits']}")
        for name in ("lr", "eps", "weight_decay"):
            if not 0 <= new[name] < math.inf:
                raise ValueError(f"{name} must be a number from 0; got {new[name]}")
        if not all(0 <= b < 1 for b in new["betas"]):
            raise ValueError(f"betas must be from 0 to below 1; got {new['betas']}")
        super().add_param_group(group)

    def _state_of(self, p, group) -> dict:
        state = self.state[p]
        if not state:
            new = adamw_state(p, group["bits"], group["master"] and p.dtype is not torch.float32)
            state.update(step=0, **{k: t for k, t in new._asdict().items() if t is not None})
        return state

    @torch.no_grad()
    def step(self, closure=None, *, norm: Optional[torch.Tensor] = None,
             max_norm: Optional[float] = None):
        """One step of every parameter that has a gradient.  It counts on the host, so a graph
        cannot capture it: capture adamw_step with a step on the device instead (and, for moments in 8
        bits, with `bounded`, as here).  With `norm` all of these parameters are on its device."""
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("AdamW.step counts its steps on the host; capture adamw_step with "
                               "`step` as a tensor instead")
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if (norm is None) != (max_norm is None):
            raise ValueError("norm and max_norm go together")
        given = [(group, [p for p in group["params"] if p.grad is not None])
                 for group in self.param_groups]
        if norm is not None:            # before any parameter is stepped
            for device in {p.device for _, params in given for p in params}:
                _check_buffer(norm, "norm", torch.float32, (1,), device)
        calls = 0
        for group, params in given:
            alike = {}                  # parameters that have taken as many steps, on one device
            for p in params:
                state = self._state_of(p, group)
                alike.setdefault((state["step"] + 1, p.device), []).append((p, state))
            for (step, _), members in alike.items():
                adamw_step([p for p, _ in members], [p.grad.contiguous() for p, _ in members],
                           [tuple(s.get(k) for k in AdamWState._fields) for _, s in members],
                           step=step, lr=group["lr"], betas=group["betas"], eps=group["eps"],
                           weight_decay=group["weight_decay"], norm=norm, max_norm=max_norm,
                           seed=group["seed"] + (calls << 32),      # a stream of noise for each call
                           bounded=True)
                calls += 1
                for _, state in members:
                    state["step"] = step
        return loss

    def load_state_dict(self, state_dict):
        """torch would cast every tensor to its parameter's type; the moments and masters keep
        theirs.  Hooks registered before and after loading see and change what they do with torch's."""
        given = []

        def keep(_, loaded):                    # after the other hooks: what is loaded
            given.append(loaded)

        def restore(_):                         # before the other hooks
            loaded, = given
            for saved, group in zip(loaded["param_groups"], self.param_groups):
                for key, p in zip(saved["params"], group["params"]):
                    if key in loaded["state"]:
                        self.state[p] = {
                            k: v.detach().to(p.device, copy=True) if isinstance(v, torch.Tensor)
                            else v for k, v in loaded["state"][key].items()}
        hooks = (self.register_load_state_dict_pre_hook(keep),
                 self.register_load_state_dict_post_hook(restore, prepend=True))
        try:
            super().load_state_dict(state_dict)
        finally:
            for hook in hooks:
                hook.remove()
