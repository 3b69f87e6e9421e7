"""Binding of include/qstate_linear.h: products with 4-bit weights and group
scales, for the projections around the mixer while a few tokens are decoded.

`qstate_linear*` marshal arguments like the functions in qstate.py; `Weight4`
holds weights laid out once, `linear4` multiplies by them."""

from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from ._lib import LinearConfigC, check, lib
from .sequence import (DTYPES, _array, _call, _on_device, _refuse_tracing, _stream,
                       _through_autograd)

__all__ = ["LinearConfig", "Weight4", "qstate_linear", "qstate_linear_bytes", "qstate_linear_pack",
           "qstate_linear_quantize", "linear4"]

_ROWS = 1 << 19  # of x in a call of the library


@dataclass
class LinearConfig:
    inputs: int
    outputs: int
    group: int = 64
    dtype: torch.dtype = torch.float32
    rows: int = 0
    x_stride: int = 0  # elements between two rows; 0: packed

    def to_c(self) -> LinearConfigC:
        if self.dtype not in DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {self.dtype}")
        return LinearConfigC(self.inputs, self.outputs, self.group, DTYPES[self.dtype], self.rows,
                             self.x_stride)


def qstate_linear_bytes(cfg: LinearConfig):
    """Bytes of the packed codes and of the packed scales."""
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    check("qstate_linear_bytes", lib().qstate_linear_bytes(cfg.to_c(), a, b))
    return a.value, b.value


def _packed(cfg: LinearConfig, packed, scales, device):
    a, b = qstate_linear_bytes(cfg)
    return (_array(packed, "packed", torch.uint8, a, device),
            _array(scales, "scales", torch.float32, b // 4, device))


def qstate_linear_pack(cfg: LinearConfig, codes, group_scales, packed, scales, stream=None) -> None:
    """int8 codes [outputs, inputs] and their scales [outputs, inputs / group] into the layout of
    `qstate_linear`."""
    _on_device(codes, "codes", None)
    dev = codes.device
    out = _packed(cfg, packed, scales, dev)
    check("qstate_linear_pack", _call(
        dev, lib().qstate_linear_pack, cfg.to_c(),
        _array(codes, "codes", torch.int8, cfg.outputs * cfg.inputs, dev),
        _array(group_scales, "group_scales", torch.float32,
               cfg.outputs * (cfg.inputs // cfg.group), dev), *out, _stream(stream, dev)))


def qstate_linear_quantize(cfg: LinearConfig, weights, packed, scales, stream=None) -> None:
    """Weights [outputs, inputs] of cfg's dtype, quantized into the layout of `qstate_linear`."""
    _on_device(weights, "weights", None)
    dev = weights.device
    out = _packed(cfg, packed, scales, dev)
    check("qstate_linear_quantize", _call(
        dev, lib().qstate_linear_quantize, cfg.to_c(),
        _array(weights, "weights", cfg.dtype, cfg.outputs * cfg.inputs, dev), *out,
        _stream(stream, dev)))


def qstate_linear(cfg: LinearConfig, x, packed, scales, bias, y, stream=None) -> None:
    """x [rows, inputs] times the packed weights, and `bias` (or None), into y [rows, outputs]."""
    _on_device(x, "x", None)
    dev = x.device
    if x.dtype != cfg.dtype or tuple(x.shape) != (cfg.rows, cfg.inputs):
        raise ValueError(f"x: expected {cfg.dtype} {(cfg.rows, cfg.inputs)}, got {x.dtype} "
                         f"{tuple(x.shape)}")
    stride = cfg.x_stride or cfg.inputs
    if x.numel() and not ((cfg.inputs == 1 or x.stride(1) == 1)
                          and (cfg.rows <= 1 or x.stride(0) == stride)):
        raise ValueError(f"x: strides {x.stride()} are not {stride} elements between packed rows")
    w = _packed(cfg, packed, scales, dev)
    check("qstate_linear", _call(
        dev, lib().qstate_linear, cfg.to_c(), x.data_ptr(), *w,
        _array(bias, "bias", torch.float32, cfg.outputs, dev, optional=True),
        _array(y, "y", cfg.dtype, cfg.rows * cfg.outputs, dev), _stream(stream, dev)))


class Weight4:
    """Weights [outputs, inputs] in four bits, laid out once for `linear4`: codes -7 .. 7 and a
    float32 scale for each output and `group` (32, 64 or 128) neighbouring inputs."""

    def __init__(self, outputs: int, inputs: int, group: int, device):
        self.outputs, self.inputs, self.group = outputs, inputs, group
        a, b = qstate_linear_bytes(LinearConfig(inputs, outputs, group))
        self.packed = torch.empty(a, dtype=torch.uint8, device=device)
        self.scales = torch.empty(b // 4, dtype=torch.float32, device=device)

    @classmethod
    def quantize(cls, weight, group: int = 64) -> "Weight4":
        """From weights [outputs, inputs] (float32, bfloat16, float16): scale = the group's largest
        magnitude / 7, codes to nearest, as the state is quantized."""
        _refuse_tracing("Weight4")
        _on_device(weight, "weight", None)
        if weight.dim() != 2 or weight.dtype not in DTYPES:
            raise ValueError(f"weight: expected [outputs, inputs] of float32, bfloat16 or float16, "
                             f"got {weight.dtype} {tuple(weight.shape)}")
        w = cls(*weight.shape, group, weight.device)
        qstate_linear_quantize(LinearConfig(w.inputs, w.outputs, group, weight.dtype),
                               weight.detach().contiguous(), w.packed, w.scales)
        return w

    @classmethod
    def from_codes(cls, codes, scales) -> "Weight4":
        """From int8 codes [outputs, inputs], -7 .. 7, and float32 scales [outputs, inputs / group]."""
        _refuse_tracing("Weight4")
        _on_device(codes, "codes", None)
        _on_device(scales, "scales", codes.device)
        if codes.dim() != 2 or codes.dtype != torch.int8 or not codes.numel():
            raise ValueError(f"codes: expected int8 [outputs, inputs], got {codes.dtype} "
                             f"{tuple(codes.shape)}")
        if (scales.dim() != 2 or scales.dtype != torch.float32 or scales.shape[0] != codes.shape[0]
                or not scales.shape[1] or codes.shape[1] % scales.shape[1]):
            raise ValueError(f"scales: expected float32 [{codes.shape[0]}, inputs / group], got "
                             f"{scales.dtype} {tuple(scales.shape)}")
        low, high = (int(t) for t in codes.aminmax())
        if low < -7 or high > 7:
            raise ValueError(f"codes reach from {low} to {high}: -7 .. 7 are held")
        w = cls(*codes.shape, codes.shape[1] // scales.shape[1], codes.device)
        qstate_linear_pack(LinearConfig(w.inputs, w.outputs, w.group), codes.contiguous(),
                           scales.contiguous(), w.packed, w.scales)
        return w

    @classmethod
    def from_nibbles(cls, nibbles, scales) -> "Weight4":
        """From uint8 [outputs, inputs / 2], two's-complement nibbles, the even input in bits 0..3 (as
        the state's INT4 rows), and scales as `from_codes`."""
        _on_device(nibbles, "nibbles", None)
        if nibbles.dim() != 2 or nibbles.dtype != torch.uint8:
            raise ValueError(f"nibbles: expected uint8 [outputs, inputs / 2], got {nibbles.dtype} "
                             f"{tuple(nibbles.shape)}")
        c = torch.stack([nibbles & 15, nibbles >> 4], -1).flatten(-2).to(torch.int8)
        return cls.from_codes(torch.where(c > 7, c - 16, c), scales)


def linear4(x, weight: Weight4, bias=None):
    """x [.., inputs] times weights in four bits, [.., outputs]: x W^T + bias.

    x float32, bfloat16 or float16, bias float32 [outputs]; FP32 sums, rounded once to x's type.
    Meant for few rows: every 16 of them read the weights.  A call takes less time than a bfloat16 product's
    up to about 128 rows with 4096 x 4096 weights, 64 with 12288 x 4096; with 4096 rows it takes five times as
    long.  Not differentiable: inputs that want a gradient are refused, and so is tracing (make_fx,
    torch.jit.trace)."""
    _refuse_tracing("linear4")
    _on_device(x, "x", weight.packed.device)
    if x.dtype not in DTYPES or x.dim() < 1 or x.shape[-1] != weight.inputs:
        raise ValueError(f"x: expected float32, bfloat16 or float16 [.., {weight.inputs}], got "
                         f"{x.dtype} {tuple(x.shape)}")
    if bias is not None:
        _on_device(bias, "bias", x.device)
        if tuple(bias.shape) != (weight.outputs,) or bias.dtype != torch.float32:
            raise ValueError(f"bias: expected float32 {(weight.outputs,)}, got {bias.dtype} "
                             f"{tuple(bias.shape)}")
        bias = bias.contiguous()
    if _through_autograd((x, bias)):
        raise RuntimeError("linear4 is not differentiable: call it under torch.no_grad()")
    r = x.reshape(-1, weight.inputs)
    stride = r.stride(0) if r.shape[0] > 1 else weight.inputs
    if ((weight.inputs > 1 and r.stride(1) != 1) or stride < weight.inputs
            or stride * r.element_size() % 16 or r.data_ptr() % 16):
        r, stride = r.clone(memory_format=torch.contiguous_format), weight.inputs
    dev = x.device
    y = torch.empty(x.shape[:-1] + (weight.outputs,), dtype=x.dtype, device=dev)
    size, start = r.element_size(), 0
    while True:
        rows = min(r.shape[0] - start, _ROWS)
        c = LinearConfigC(weight.inputs, weight.outputs, weight.group, DTYPES[x.dtype], rows, stride)
        check("qstate_linear", _call(
            dev, lib().qstate_linear, c, r.data_ptr() + start * stride * size,
            weight.packed.data_ptr(), weight.scales.data_ptr(),
            None if bias is None else bias.data_ptr(),
            y.data_ptr() + start * weight.outputs * size, _stream(None, dev)))
        start += rows
        if start >= r.shape[0]:
            return y
