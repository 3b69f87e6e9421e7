"""Binding of include/qstate_group_norm.h: the group norm of a mixer's readout
with its activation or gate, channels last, and its gradients.

`qstate_group_norm` and `qstate_group_norm_backward` marshal arguments like the
functions in norm.py; `group_norm` is the differentiable operator on top."""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from ._lib import GroupNormConfigC, check, lib
from .norm import SIGMOID, SILU
from .sequence import (DTYPES, _array, _bytes_on, _call, _note_alive, _on_device, _ptr,
                       _refuse_capture, _refuse_tracing, _stream, _through_autograd, _workspace)

__all__ = ["PLAIN", "GATE", "GATE_FIRST", "ACTIVATE", "GroupNormConfig", "qstate_group_norm",
           "qstate_group_norm_workspace", "qstate_group_norm_backward", "group_norm"]

PLAIN, GATE, GATE_FIRST, ACTIVATE = 0, 1, 2, 3


@dataclass
class GroupNormConfig:
    tokens: int
    groups: int
    width: int  # channels of a group
    dtype: torch.dtype = torch.float32
    act: int = SILU
    mode: int = PLAIN
    center: bool = True
    eps: float = 1e-5
    shared: bool = False  # weight and bias are [width], the same for all groups
    x_stride: int = 0  # elements between two tokens; 0: packed
    gate_stride: int = 0

    def to_c(self) -> GroupNormConfigC:
        if self.dtype not in DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {self.dtype}")
        return GroupNormConfigC(self.tokens, self.groups, self.width, DTYPES[self.dtype], self.act,
                                self.mode, int(self.center), self.eps, int(self.shared), self.x_stride,
                                self.gate_stride)


def _rows(t, name, cfg: GroupNormConfig, stride, device, optional=True):
    """Pointer of [tokens][groups * width] rows, `stride` elements apart."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{name} is missing")
    _on_device(t, name, device)
    row = cfg.groups * cfg.width
    if t.dtype != cfg.dtype or tuple(t.shape) != (cfg.tokens, row):
        raise ValueError(f"{name}: expected {cfg.dtype} {(cfg.tokens, row)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if t.numel() and not ((row == 1 or t.stride(1) == 1)
                          and (cfg.tokens <= 1 or t.stride(0) == (stride or row))):
        raise ValueError(f"{name}: strides {t.stride()} are not {stride or row} elements between "
                         "packed tokens")
    return t.data_ptr()


def _inputs(cfg: GroupNormConfig, x, weight, bias, gate):
    _on_device(x, "x", None)
    dev, f32, C = x.device, torch.float32, cfg.width * (1 if cfg.shared else cfg.groups)
    return (
        _rows(x, "x", cfg, cfg.x_stride, dev, optional=False),
        _array(weight, "weight", f32, C, dev, optional=True),
        _array(bias, "bias", f32, C, dev, optional=True),
        _rows(gate, "gate", cfg, cfg.gate_stride, dev),
    )


def _launch(c, dev, inputs, y, stream):
    check("qstate_group_norm", _call(dev, lib().qstate_group_norm, c, *inputs, y,
                                     _stream(stream, dev)))


def _launch_backward(c, dev, inputs, more, workspace, stream):
    check("qstate_group_norm_backward", _call(dev, lib().qstate_group_norm_backward, c, *inputs,
                                              *more, *workspace, _stream(stream, dev)))


def _workspace_bytes(c: GroupNormConfigC) -> int:
    n = ctypes.c_size_t()
    check("qstate_group_norm_workspace", lib().qstate_group_norm_workspace(c, n))
    return n.value


def _own_workspace(c, wanted, dev, stream=None):
    """A workspace of this call where sums over rows are wanted: the tensor, (pointer, bytes)."""
    if not wanted:
        return None, (None, 0)
    w = _bytes_on(max(_workspace_bytes(c), 1), dev, stream)
    return w, (w.data_ptr(), w.numel())


def qstate_group_norm(cfg: GroupNormConfig, x, weight=None, bias=None, gate=None, y=None,
                      stream=None) -> None:
    """The norm of the groups of x [tokens, groups * width] into `y`."""
    args = _inputs(cfg, x, weight, bias, gate)
    _launch(cfg.to_c(), x.device, args, _rows(y, "y", cfg, 0, x.device, optional=False), stream)


def qstate_group_norm_workspace(cfg: GroupNormConfig) -> int:
    return _workspace_bytes(cfg.to_c())


def qstate_group_norm_backward(cfg: GroupNormConfig, x, weight=None, bias=None, gate=None, dy=None,
                               dx=None, dgate=None, dweight=None, dbias=None, workspace=None,
                               stream=None) -> None:
    """Gradients from `dy`; outputs that are None are not wanted."""
    args = _inputs(cfg, x, weight, bias, gate)
    dev, f32, C = x.device, torch.float32, cfg.width * (1 if cfg.shared else cfg.groups)
    more = [_rows(dy, "dy", cfg, 0, dev, optional=False)]
    more += [_rows(t, n, cfg, 0, dev) for t, n in ((dx, "dx"), (dgate, "dgate"))]
    more += [_array(dweight, "dweight", f32, C, dev, optional=True),
             _array(dbias, "dbias", f32, C, dev, optional=True)]
    c = cfg.to_c()
    if workspace is not None:
        keep, w = None, _workspace(workspace, dev)
    else:
        keep, w = _own_workspace(c, dweight is not None or dbias is not None, dev, stream)
    _launch_backward(c, dev, args, more, w, stream)


def _token_rows(t):
    """([tokens][channels], elements between tokens); a copy only where the channels are not packed or
    the tokens do not lie at one distance."""
    if t is None:
        return None, 0
    C = t.shape[-1]
    try:
        r = t.view(-1, C)
    except RuntimeError:
        r = t.reshape(-1, C)
    if (C > 1 and r.stride(1) != 1) or (r.shape[0] > 1 and r.stride(0) < C):
        r = r.clone(memory_format=torch.contiguous_format)
    return r, 0 if r.shape[0] <= 1 or r.stride(0) == C else r.stride(0)


def _forward(x, weight, bias, gate, groups, mode, center, eps, act, shared):
    """The checked call: y, and what backward needs."""
    (x2, xs), (gate2, gs) = _token_rows(x), _token_rows(gate)
    weight, bias = (None if t is None else t.contiguous() for t in (weight, bias))
    c = GroupNormConfigC(x2.shape[0], groups, x.shape[-1] // groups, DTYPES[x.dtype], act, mode,
                         int(center), eps, int(shared), xs, gs)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    saved = (x2, weight, bias, gate2)
    _launch(c, x.device, [_ptr(t) for t in saved], y.data_ptr(), None)
    return y, c, saved


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, *how):
        y, ctx.cfg, saved = _forward(x, weight, bias, gate, *how)
        _note_alive(ctx, x.device)
        ctx.shape = x.shape
        ctx.save_for_backward(*saved)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        saved = ctx.saved_tensors
        x, weight, bias, gate = saved
        need = ctx.needs_input_grad
        dev = x.device
        _refuse_capture(ctx, dev)
        dy = dy.contiguous()
        dx, dgate = (torch.empty(ctx.shape, dtype=x.dtype, device=dev) if need[i] else None
                     for i in (0, 3))
        sums = [torch.empty_like(t) if need[i] else None for t, i in ((weight, 1), (bias, 2))]
        keep, w = _own_workspace(ctx.cfg, any(t is not None for t in sums), dev)
        _launch_backward(ctx.cfg, dev, [_ptr(t) for t in saved],
                         [_ptr(t) for t in (dy, dx, dgate, *sums)], w, None)
        return dx, *sums, dgate, *(None,) * 6


def group_norm(x, groups: int, *, weight=None, bias=None, gate=None, gate_first: bool = False,
               activate: bool = False, center: bool = True, eps: float = 1e-5, act: int = SILU):
    """The norm of each of `groups` groups of neighbouring channels of x [.., channels], per token:

        u = x * act(gate) with gate_first, else x
        n = (u - mean(u)) * rsqrt(var(u) + eps) * weight + bias       (center)
        n = u * rsqrt(mean(u^2) + eps) * weight + bias                (otherwise)
        y = n * act(gate) with a gate that is not first; act(n) with `activate`, where act(n) is
            n sigmoid(n) (SILU) or sigmoid(n) (SIGMOID); else n

    x and gate have one shape and one dtype (float32, bfloat16, float16), weight and bias are
    float32 [channels], or both [channels / groups], the same for all groups.  FP32 between inputs and outputs.  Differentiable once in every tensor (a
    backward pass is captured into a graph only where no eager graph of the same leaves lives);
    forward-mode derivatives and tracing (make_fx, torch.jit.trace) are refused."""
    _refuse_tracing("group_norm")
    _on_device(x, "x", None)
    if x.dtype not in DTYPES or x.dim() < 1:
        raise ValueError(f"x: one of float32, bfloat16, float16 [.., channels], got {x.dtype} "
                         f"{tuple(x.shape)}")
    C = x.shape[-1]
    if groups < 1 or C % groups or C < 1:
        raise ValueError(f"{C} channels in {groups} groups")
    if act not in (SILU, SIGMOID):
        raise ValueError(f"act: {act}")
    if activate and gate is not None or gate_first and gate is None:
        raise ValueError("activate goes without a gate, gate_first with one")
    if gate is not None:
        _on_device(gate, "gate", x.device)
        if gate.shape != x.shape or gate.dtype != x.dtype:
            raise ValueError(f"gate: expected {x.dtype} {tuple(x.shape)}, got {gate.dtype} "
                             f"{tuple(gate.shape)}")
    given = [t for t in (weight, bias) if t is not None]
    shared = bool(given) and isinstance(given[0], torch.Tensor) and tuple(given[0].shape) == (C // groups,)
    want = (C // groups,) if shared else (C,)
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _on_device(t, name, x.device)
            if tuple(t.shape) != want or t.dtype != torch.float32:
                raise ValueError(f"{name}: expected float32 {want}, got {t.dtype} {tuple(t.shape)}")
    mode = ACTIVATE if activate else PLAIN if gate is None else GATE_FIRST if gate_first else GATE
    how = (groups, mode, center, eps, act, shared)
    if _through_autograd((x, weight, bias, gate)):
        return _GroupNorm.apply(x, weight, bias, gate, *how)
    return _forward(x, weight, bias, gate, *how)[0]
