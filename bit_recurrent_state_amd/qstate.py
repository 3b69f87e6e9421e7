"""Python binding of the qstate C ABI (include/qstate.h), same names.

Argument marshalling only: torch supplies device memory and the HIP stream,
every step of the path runs in the library's kernels.  Shapes and dtypes are
checked here so that a wrong tensor fails before it reaches the C ABI."""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import (BDR, GDN, GLA, KDA, KEY_AXIS, RTN, SCALAR, SR, VALUE_AXIS, QStateConfig, check,
                   lib)
from .norm import SILU, NormConfig, qstate_norm, qstate_norm_workspace
from .sequence import _array, _on, scan

__all__ = [
    "GDN", "GLA", "SCALAR", "KDA", "RTN", "SR", "BDR", "VALUE_AXIS", "KEY_AXIS", "Config",
    "QState", "ReadoutNorm",
    "qstate_state_bytes", "qstate_create", "qstate_load_fp32", "qstate_step",
    "qstate_readout", "qstate_store_fp32", "qstate_get_step", "qstate_set_step",
    "qstate_destroy", "qstate_bits_by_decay",
]


@dataclass
class Config:
    batch: int
    heads: int
    dk: int
    dv: int
    group: int = 64
    mixer: int = GDN
    rounding: int = RTN
    fp32_state: bool = False
    head_bits: Optional[Sequence[int]] = None
    seed: int = 0
    layer: int = 0
    group_axis: int = VALUE_AXIS
    channel_bits: Optional[Sequence[Sequence[int]]] = None  # [heads][dk/16], overrides head_bits
    window: int = 0  # pure-write window length W (0, 4, 8 or 16)
    window_merge: int = 0  # 0 pure-write window, 1 low-rank bypass (merge every W steps)
    lrb_threshold: float = 0.5  # low-rank bypass: merge |m| >= threshold * group scale

    def to_c(self):
        """(QStateConfig, keep-alive buffers)."""
        keep = []
        ptr = cptr = None
        if self.head_bits is not None:
            hb = (ctypes.c_uint8 * self.heads)(*[int(x) for x in self.head_bits])
            ptr = ctypes.cast(hb, ctypes.POINTER(ctypes.c_uint8))
            keep.append(hb)
        if self.channel_bits is not None:
            flat = np.asarray(self.channel_bits, np.uint8).reshape(-1)
            if flat.size != self.heads * (self.dk // 16):
                raise ValueError("channel_bits: expected [heads][dk/16] widths")
            cb = (ctypes.c_uint8 * flat.size)(*[int(x) for x in flat])
            cptr = ctypes.cast(cb, ctypes.POINTER(ctypes.c_uint8))
            keep.append(cb)
        c = QStateConfig(self.batch, self.heads, self.dk, self.dv, self.group, self.mixer,
                         self.rounding, int(bool(self.fp32_state)), ptr, self.seed, self.layer,
                         self.group_axis, cptr, self.window, self.window_merge,
                         self.lrb_threshold)
        return c, keep

    def bits(self) -> np.ndarray:
        """Widths per head and 16-column block, [heads][dk/16] (32 for an FP32 state)."""
        nb = self.dk // 16
        if self.fp32_state:
            return np.full((self.heads, nb), 32, np.int64)
        if self.channel_bits is not None:
            return np.asarray(self.channel_bits, np.int64).reshape(self.heads, nb)
        if self.head_bits is None:
            return np.full((self.heads, nb), 8, np.int64)
        return np.repeat(np.asarray(self.head_bits, np.int64)[:, None], nb, axis=1)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dev(t: torch.Tensor, name: str, dtype, numel: int):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != numel:
        raise ValueError(f"{name}: expected contiguous {dtype} with {numel} elements, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")
    return ctypes.c_void_p(t.data_ptr())


def qstate_state_bytes(cfg: Config):
    c, _keep = cfg.to_c()
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    check("qstate_state_bytes", lib().qstate_state_bytes(ctypes.byref(c), ctypes.byref(cb),
                                                          ctypes.byref(sb)))
    return cb.value, sb.value


def qstate_create(cfg: Config, codes: torch.Tensor, scales: Optional[torch.Tensor]):
    cb, sb = qstate_state_bytes(cfg)
    if cfg.fp32_state:
        pc = _dev(codes, "state", torch.float32, cb // 4)
        ps = None
    else:
        pc = _dev(codes, "codes", torch.uint8, cb)
        ps = _dev(scales, "scales", torch.float32, sb // 4)
    c, _keep = cfg.to_c()
    h = ctypes.c_void_p()
    check("qstate_create", lib().qstate_create(ctypes.byref(c), pc, ps, ctypes.byref(h)))
    return h


def qstate_load_fp32(h, S: torch.Tensor, cfg: Config, stream=None):
    n = cfg.batch * cfg.heads * cfg.dv * cfg.dk
    check("qstate_load_fp32", lib().qstate_load_fp32(h, _dev(S, "S", torch.float32, n),
                                                      _stream(stream)))


def qstate_step(h, cfg: Config, q, k, v, alpha, beta=None, o=None, stream=None):
    bh = cfg.batch * cfg.heads
    na = bh * cfg.dk if cfg.mixer in (GLA, KDA) else bh
    args = (
        _dev(q, "q", torch.float32, bh * cfg.dk), _dev(k, "k", torch.float32, bh * cfg.dk),
        _dev(v, "v", torch.float32, bh * cfg.dv), _dev(alpha, "alpha", torch.float32, na),
        None if cfg.mixer == GLA else _dev(beta, "beta", torch.float32, bh),
        _dev(o, "o", torch.float32, bh * cfg.dv),
    )
    check("qstate_step", lib().qstate_step(h, *args, _stream(stream)))


def qstate_readout(h, cfg: Config, q, o, stream=None):
    bh = cfg.batch * cfg.heads
    check("qstate_readout", lib().qstate_readout(h, _dev(q, "q", torch.float32, bh * cfg.dk),
                                                  _dev(o, "o", torch.float32, bh * cfg.dv),
                                                  _stream(stream)))


def qstate_store_fp32(h, cfg: Config, S, stream=None):
    n = cfg.batch * cfg.heads * cfg.dv * cfg.dk
    check("qstate_store_fp32", lib().qstate_store_fp32(h, _dev(S, "S", torch.float32, n),
                                                        _stream(stream)))


def qstate_get_step(h) -> int:
    s = ctypes.c_uint64()
    check("qstate_get_step", lib().qstate_get_step(h, ctypes.byref(s)))
    return s.value


def qstate_set_step(h, step: int) -> None:
    check("qstate_set_step", lib().qstate_set_step(h, step))


def qstate_destroy(h) -> None:
    check("qstate_destroy", lib().qstate_destroy(h))


def qstate_bits_by_decay(retention, mode: int, thr_or_frac: float, lo_bits: int = 4,
                         hi_bits: int = 8) -> np.ndarray:
    r = np.ascontiguousarray(retention, dtype=np.float32)
    out = np.zeros(r.size, np.uint8)
    check("qstate_bits_by_decay",
          lib().qstate_bits_by_decay(r.ctypes.data_as(ctypes.c_void_p), r.size, mode,
                                     thr_or_frac, lo_bits, hi_bits,
                                     out.ctypes.data_as(ctypes.c_void_p)))
    return out


@dataclass
class ReadoutNorm:
    """What a layer does with the readout before its output projection:
    o * rsqrt(mean(o^2) + eps) * weight * act(gate), over each head's dv values."""

    weight: Optional[torch.Tensor] = None  # float32 [dv] or [heads, dv]
    gate: Optional[torch.Tensor] = None    # of o's type and shape (or its rows or values in a row)
    eps: float = 1e-6
    act: int = SILU

    def config(self, shape, dtype, device, o_shape=None) -> NormConfig:
        """The configuration for a readout of this shape, its tensors checked.  o_shape: the shape in
        which the caller has it."""
        tokens, heads, dv = shape
        each = self.weight is not None and self.weight.dim() == 2
        if self.weight is not None:
            w = tuple(self.weight.shape)
            if w[-1:] != (dv,) or each and w != (heads, dv):
                raise ValueError(f"weight: expected [{dv}] or [{heads}, {dv}], got {w}")
        if self.gate is not None:
            g = tuple(self.gate.shape)
            if g not in (tuple(shape), (tokens * heads * dv,), tuple(o_shape or shape)):
                raise ValueError(f"gate: expected {tuple(o_shape or shape)}, got {g}")
        cfg = NormConfig(tokens, heads, dv, dtype, self.act, each, self.eps)
        qstate_norm_workspace(cfg)  # the library's checks of it
        _array(self.weight, "weight", torch.float32, dv * (heads if each else 1), device,
               optional=True)
        _array(self.gate, "gate", dtype, tokens * heads * dv, device, optional=True)
        return cfg

    def apply_(self, o: torch.Tensor, stream=None) -> None:
        """In place on o [tokens, heads, dv]."""
        self._run(self.config(o.shape, o.dtype, o.device), o, stream)

    def _run(self, cfg: NormConfig, o: torch.Tensor, stream=None) -> None:
        o = o.view(cfg.tokens, cfg.groups, cfg.width)
        gate = None if self.gate is None else self.gate.view(o.shape)
        qstate_norm(cfg, o, self.weight, gate, r=o, stream=stream)


class QState:
    """A handle plus the torch device buffers it works on (caller-owned memory)."""

    def __init__(self, cfg: Config, device="cuda"):
        self.cfg = cfg
        cb, sb = qstate_state_bytes(cfg)
        if cfg.fp32_state:
            self.codes = torch.zeros(cb // 4, dtype=torch.float32, device=device)
            self.scales = None
        else:
            self.codes = torch.zeros(cb, dtype=torch.uint8, device=device)
            self.scales = torch.zeros(sb // 4, dtype=torch.float32, device=device)
        self.handle = qstate_create(cfg, self.codes, self.scales)

    def load_fp32(self, S, stream=None):
        qstate_load_fp32(self.handle, S, self.cfg, stream)

    def step(self, q, k, v, alpha, beta=None, o=None, stream=None, norm=None):
        """One token for every sequence; with `norm` (a ReadoutNorm), o is the normed and gated
        readout."""
        if norm is not None:  # refused before the state changes
            if o is None:
                raise ValueError("norm: there is no readout without o")
            shape = (self.cfg.batch, self.cfg.heads, self.cfg.dv)
            cfg = norm.config(shape, torch.float32, o.device, o.shape)
        qstate_step(self.handle, self.cfg, q, k, v, alpha, beta, o, stream)
        if norm is not None:
            norm._run(cfg, o, stream)

    def prefill(self, q, k, v, log_alpha, beta=None, offsets=None, norm=None, stream=None):
        """A prompt's or a chunk's tokens at once, for sequences that decode on with `step`: the
        scan from the stored state, whose end is stored back (one quantization event for every
        sequence, those without tokens too: the counter goes up by one, a window starts empty).
        Arguments as `scan`'s, one sequence per batch row, q and k with the handle's heads or a
        divisor of them; returns o, which lies in the memory of the stream of the call."""
        c = self.cfg
        if offsets is not None and offsets.numel() != c.batch + 1:
            raise ValueError(f"offsets: expected {c.batch + 1} elements, got {offsets.numel()}")
        if v.shape[-2:] != (c.heads, c.dv) or q.shape[-1] != c.dk or (
                offsets is None and v.shape[0] != c.batch):
            raise ValueError(f"q {tuple(q.shape)}, v {tuple(v.shape)} do not go with the state "
                             f"[{c.batch}][{c.heads}][{c.dv}][{c.dk}]")
        if norm is not None:
            cfg = norm.config((v[..., 0, 0].numel(), c.heads, c.dv), v.dtype, v.device, v.shape)
        with torch.no_grad(), torch.cuda.device(v.device), _on(stream, v.device):
            S = torch.empty((c.batch, c.heads, c.dv, c.dk), dtype=torch.float32, device=v.device)
            self.store_fp32(S)
            o, S = scan(q, k, v, log_alpha, beta, mixer=c.mixer, initial_state=S, offsets=offsets)
            self.load_fp32(S)
            if norm is not None:
                norm._run(cfg, o)
        return o

    def readout(self, q, o, stream=None):
        qstate_readout(self.handle, self.cfg, q, o, stream)

    def store_fp32(self, S, stream=None):
        qstate_store_fp32(self.handle, self.cfg, S, stream)

    @property
    def step_counter(self) -> int:
        return qstate_get_step(self.handle)

    @step_counter.setter
    def step_counter(self, value: int) -> None:
        qstate_set_step(self.handle, value)

    def close(self):
        if self.handle is not None:
            qstate_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
