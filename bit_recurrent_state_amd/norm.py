"""Binding of include/qstate_norm.h: the norms around the mixer block (the
readout's norm with its gate, the residual with its scale, the next block's
norm) and their gradients.

`qstate_norm` and `qstate_norm_backward` marshal arguments like the functions
in qstate.py; `block_norm` is the differentiable operator on top of them."""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from ._lib import NormConfigC, check, lib
from .sequence import (DTYPES, _array, _bytes_on, _call, _note_alive, _on_device, _ptr,
                       _refuse_capture, _refuse_tracing, _stream, _through_autograd, _workspace)

__all__ = ["SILU", "SIGMOID", "NormConfig", "qstate_norm", "qstate_norm_workspace",
           "qstate_norm_backward", "block_norm"]

SILU, SIGMOID = 0, 1


@dataclass
class NormConfig:
    tokens: int
    groups: int
    width: int
    dtype: torch.dtype = torch.float32
    act: int = SILU
    weight_groups: bool = False  # weight is [groups][width]
    eps: float = 1e-6
    x_stride: int = 0  # elements between two tokens; 0: packed
    gate_stride: int = 0
    residual_stride: int = 0

    def to_c(self) -> NormConfigC:
        if self.dtype not in DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {self.dtype}")
        return NormConfigC(self.tokens, self.groups, self.width, DTYPES[self.dtype], self.act,
                           int(self.weight_groups), self.eps, self.x_stride, self.gate_stride,
                           self.residual_stride)


def _rows(t, name, cfg: NormConfig, stride, device, optional=True):
    """Pointer of [tokens][groups][width] rows, tokens `stride` elements apart."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{name} is missing")
    _on_device(t, name, device)
    want = (cfg.tokens, cfg.groups, cfg.width)
    if t.dtype != cfg.dtype or tuple(t.shape) != want:
        raise ValueError(f"{name}: expected {cfg.dtype} {want}, got {t.dtype} {tuple(t.shape)}")
    ok = ((cfg.width == 1 or t.stride(2) == 1)
          and (cfg.groups == 1 or t.stride(1) == cfg.width)
          and (cfg.tokens <= 1 or t.stride(0) == (stride or cfg.groups * cfg.width)))
    if t.numel() and not ok:
        raise ValueError(f"{name}: strides {t.stride()} are not "
                         f"{stride or cfg.groups * cfg.width} elements between tokens with packed "
                         "rows")
    return t.data_ptr()


def _inputs(cfg: NormConfig, x, weight, gate, residual, scale, next_weight):
    _on_device(x, "x", None)
    dev, f32 = x.device, torch.float32
    nw = cfg.width * (cfg.groups if cfg.weight_groups else 1)
    return (
        _rows(x, "x", cfg, cfg.x_stride, dev, optional=False),
        _array(weight, "weight", f32, nw, dev, optional=True),
        _rows(gate, "gate", cfg, cfg.gate_stride, dev),
        _rows(residual, "residual", cfg, cfg.residual_stride, dev),
        _array(scale, "scale", f32, cfg.width, dev, optional=True),
        _array(next_weight, "next_weight", f32, cfg.width, dev, optional=True),
    )


def qstate_norm(cfg: NormConfig, x, weight=None, gate=None, residual=None, scale=None,
                next_weight=None, r=None, h=None, stream=None) -> None:
    """r = residual + scale * act(gate) * rms(x) weight into `r`, rms(r) next_weight into `h`."""
    args = _inputs(cfg, x, weight, gate, residual, scale, next_weight)
    dev = x.device
    out = _rows(r, "r", cfg, 0, dev), _rows(h, "h", cfg, 0, dev)
    _launch(cfg.to_c(), dev, args, out, stream)


def _launch(c, dev, inputs, out, stream):
    check("qstate_norm", _call(dev, lib().qstate_norm, c, *inputs, *out, _stream(stream, dev)))


def _launch_backward(c, dev, inputs, has_h, more, workspace, stream):
    check("qstate_norm_backward", _call(dev, lib().qstate_norm_backward, c, *inputs, has_h, *more,
                                        *workspace, _stream(stream, dev)))


def qstate_norm_workspace(cfg: NormConfig) -> int:
    return _workspace_bytes(cfg.to_c())


def _workspace_bytes(c: NormConfigC) -> int:
    n = ctypes.c_size_t()
    check("qstate_norm_workspace", lib().qstate_norm_workspace(c, n))
    return n.value


def _own_workspace(c, wanted, dev, stream=None):
    """A workspace of this call where sums over rows are wanted: the tensor, (pointer, bytes)."""
    if not wanted:
        return None, (None, 0)
    w = _bytes_on(max(_workspace_bytes(c), 1), dev, stream)
    return w, (w.data_ptr(), w.numel())


def qstate_norm_backward(cfg: NormConfig, x, weight=None, gate=None, residual=None, scale=None,
                         next_weight=None, has_h=False, dr=None, dh=None, dx=None, dgate=None,
                         dresidual=None, dweight=None, dscale=None, dnext_weight=None,
                         workspace=None, stream=None) -> None:
    """Gradients from `dr` and `dh`; outputs that are None are not wanted."""
    args = _inputs(cfg, x, weight, gate, residual, scale, next_weight)
    dev, f32 = x.device, torch.float32
    nw = cfg.width * (cfg.groups if cfg.weight_groups else 1)
    more = [_rows(t, n, cfg, 0, dev) for t, n in
            ((dr, "dr"), (dh, "dh"), (dx, "dx"), (dgate, "dgate"), (dresidual, "dresidual"))]
    more += [_array(dweight, "dweight", f32, nw, dev, optional=True),
             _array(dscale, "dscale", f32, cfg.width, dev, optional=True),
             _array(dnext_weight, "dnext_weight", f32, cfg.width, dev, optional=True)]
    c = cfg.to_c()
    if workspace is not None:
        keep, w = None, _workspace(workspace, dev)
    else:
        keep, w = _own_workspace(c, any(t is not None for t in (dweight, dscale, dnext_weight)),
                                 dev, stream)
    _launch_backward(c, dev, args, int(has_h), more, w, stream)


def _token_rows(t, groups, width):
    """[.., width] as [tokens][groups][width]; a copy only where tokens do not lie at one distance
    with packed rows in them."""
    if t is None:
        return None, 0
    try:
        r = t.view(-1, groups, width)
    except RuntimeError:
        r = t.reshape(-1, groups, width)
    packed = (width == 1 or r.stride(2) == 1) and (groups == 1 or r.stride(1) == width)
    if not packed or (r.shape[0] > 1 and r.stride(0) < groups * width):
        r = r.clone(memory_format=torch.contiguous_format)
    return r, 0 if r.shape[0] <= 1 or r.stride(0) == groups * width else r.stride(0)


def _one_distance(t, width) -> bool:
    if t is None or t.is_contiguous():
        return True
    try:
        t.view(-1, width)
        return True
    except RuntimeError:
        return False


def _forward(x, weight, gate, residual, scale, next_weight, eps, act):
    """The checked call: r, h, and what backward needs."""
    width = x.shape[-1]
    each = weight is not None and weight.dim() == 2
    # [tokens][groups]: a weight per group needs it; else it only says how the rows lie, and they
    # mostly lie at one distance
    groups = 1
    if each or (x.dim() > 2 and x.shape[-2] <= 65535
                and not all(_one_distance(t, width) for t in (x, gate, residual))):
        groups = x.shape[-2]
    (x3, xs), (gate3, gs), (res3, rs) = (_token_rows(t, groups, width) for t in (x, gate, residual))
    weight, scale, next_weight = (None if t is None else t.contiguous()
                                  for t in (weight, scale, next_weight))
    c = NormConfigC(x3.shape[0], groups, width, DTYPES[x.dtype], act, int(each), eps, xs, gs, rs)
    r = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    h = torch.empty_like(r) if next_weight is not None else None
    saved = (x3, weight, gate3, res3, scale, next_weight)
    _launch(c, x.device, [_ptr(t) for t in saved], (r.data_ptr(), _ptr(h)), None)
    return r, h, c, saved


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, gate, residual, scale, next_weight, eps, act):
        r, h, ctx.cfg, saved = _forward(x, weight, gate, residual, scale, next_weight, eps, act)
        _note_alive(ctx, x.device)
        ctx.shape = x.shape
        ctx.save_for_backward(*saved)
        ctx.set_materialize_grads(False)
        return r if h is None else (r, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dh=None):
        if dr is None and dh is None:
            return (None,) * 8
        saved = ctx.saved_tensors
        x, weight, gate, residual, scale, next_weight = saved
        need = ctx.needs_input_grad
        dev = x.device
        _refuse_capture(ctx, dev)
        dr, dh = (None if t is None else t.contiguous() for t in (dr, dh))
        dx, dgate, dres = (torch.empty(ctx.shape, dtype=x.dtype, device=dev) if need[i] else None
                           for i in (0, 2, 3))
        sums = [torch.empty_like(t) if need[i] else None
                for t, i in ((weight, 1), (scale, 4), (next_weight, 5))]
        keep, w = _own_workspace(ctx.cfg, any(t is not None for t in sums), dev)
        _launch_backward(ctx.cfg, dev, [_ptr(t) for t in saved], int(next_weight is not None),
                         [_ptr(t) for t in (dr, dh, dx, dgate, dres, *sums)], w, None)
        return dx, sums[0], dgate, dres, sums[1], sums[2], None, None


def block_norm(x, *, weight=None, gate=None, residual=None, scale=None, next_weight=None,
               eps: float = 1e-6, act: int = SILU):
    """The end of a mixer block in one pass over its rows, over the last dimension of x:

        r = residual + scale * act(gate) * (x * rsqrt(mean(x^2) + eps) * weight)
        h = r * rsqrt(mean(r^2) + eps) * next_weight

    Parts that are None are left out; returns r, or (r, h) with next_weight.  x, gate and residual
    have one shape [.., width] and one dtype (float32, bfloat16, float16); weight is float32
    [width], or [heads, width] for x [.., heads, width]; scale and next_weight float32 [width].
    FP32 between inputs and outputs.  Differentiable once in every tensor (a backward pass is
    captured into a graph only where no eager graph of the same leaves lives); forward-mode
    derivatives and tracing (make_fx, torch.jit.trace) are refused."""
    _refuse_tracing("block_norm")
    _on_device(x, "x", None)
    if x.dtype not in DTYPES or x.dim() < 1:
        raise ValueError(f"x: one of float32, bfloat16, float16 [.., width], got {x.dtype} "
                         f"{tuple(x.shape)}")
    if act not in (SILU, SIGMOID):
        raise ValueError(f"act: {act}")
    for t, name in ((gate, "gate"), (residual, "residual")):
        if t is not None:
            _on_device(t, name, x.device)
            if t.shape != x.shape or t.dtype != x.dtype:
                raise ValueError(f"{name}: expected {x.dtype} {tuple(x.shape)}, got {t.dtype} "
                                 f"{tuple(t.shape)}")
    width = x.shape[-1]
    for t, name in ((weight, "weight"), (scale, "scale"), (next_weight, "next_weight")):
        if t is None:
            continue
        _on_device(t, name, x.device)
        each = name == "weight" and t.dim() == 2
        want = (x.shape[-2] if x.dim() > 1 else -1, width) if each else (width,)
        if tuple(t.shape) != want or t.dtype != torch.float32:
            raise ValueError(f"{name}: expected float32 {want}, got {t.dtype} {tuple(t.shape)}")
    if _through_autograd((x, weight, gate, residual, scale, next_weight)):
        return _BlockNorm.apply(x, weight, gate, residual, scale, next_weight, eps, act)
    r, h = _forward(x, weight, gate, residual, scale, next_weight, eps, act)[:2]
    return r if h is None else (r, h)
