"""Python binding of the qstate C ABI (include/qstate.h), same names.

Argument marshalling only: torch supplies device memory and the HIP stream,
every step of the path runs in the library's kernels.  Shapes and dtypes are
checked here so that a wrong tensor fails before it reaches the C ABI."""

from __future__ import annotations

import copy
import ctypes
from contextlib import nullcontext
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import (BDR, GDN, GLA, KDA, KEY_AXIS, RTN, SCALAR, SR, VALUE_AXIS, QStateConfig, check,
                   lib)
from .draft import Draft, _accept, _refuse_gradients, _verify
from .group_norm import (GATE, GATE_FIRST, PLAIN, GroupNormConfig, qstate_group_norm,
                         qstate_group_norm_workspace)
from .linear import Weight4, linear4
from .norm import SILU, NormConfig, qstate_norm, qstate_norm_workspace
from .sequence import _array, _on, _on_device, scan

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
    o * rsqrt(mean(o^2) + eps) * weight * act(gate), over each head's dv values; with `center`, `bias`
    or `gate_first` the forms of `group_norm` over heads (a retention layer's, a Mamba2 block's)."""

    weight: Optional[torch.Tensor] = None  # float32 [dv] or [heads, dv]
    gate: Optional[torch.Tensor] = None    # of o's type and shape (or its rows or values in a row)
    eps: float = 1e-6
    act: int = SILU
    bias: Optional[torch.Tensor] = None    # as weight
    center: bool = False                   # the mean is taken off before the variance
    gate_first: bool = False               # the norm of o * act(gate)

    @property
    def grouped(self) -> bool:
        return self.center or self.gate_first or self.bias is not None

    def config(self, shape, dtype, device, o_shape=None):
        """The configuration for a readout of this shape, its tensors checked.  o_shape: the shape in
        which the caller has it."""
        tokens, heads, dv = shape
        each = any(t is not None and t.dim() == 2 for t in (self.weight, self.bias))
        for t, name in ((self.weight, "weight"), (self.bias, "bias")):
            if t is not None:
                w = tuple(t.shape)
                if w[-1:] != (dv,) or each and w != (heads, dv):
                    raise ValueError(f"{name}: expected [{dv}] or [{heads}, {dv}], got {w}")
        if self.gate is not None:
            g = tuple(self.gate.shape)
            if g not in (tuple(shape), (tokens * heads * dv,), tuple(o_shape or shape)):
                raise ValueError(f"gate: expected {tuple(o_shape or shape)}, got {g}")
        if self.grouped:
            if self.gate_first and self.gate is None:
                raise ValueError("gate_first: there is no gate")
            mode = PLAIN if self.gate is None else GATE_FIRST if self.gate_first else GATE
            cfg = GroupNormConfig(tokens, heads, dv, dtype, self.act, mode, self.center, self.eps,
                                  not each)
            qstate_group_norm_workspace(cfg)  # the library's checks of it
        else:
            cfg = NormConfig(tokens, heads, dv, dtype, self.act, each, self.eps)
            qstate_norm_workspace(cfg)
        n = dv * (heads if each else 1)
        _array(self.weight, "weight", torch.float32, n, device, optional=True)
        _array(self.bias, "bias", torch.float32, n, device, optional=True)
        _array(self.gate, "gate", dtype, tokens * heads * dv, device, optional=True)
        return cfg

    def apply_(self, o: torch.Tensor, stream=None) -> None:
        """In place on o [tokens, heads, dv]."""
        self._run(self.config(o.shape, o.dtype, o.device), o, stream)

    def _run(self, cfg, o: torch.Tensor, stream=None) -> None:
        if self.grouped:
            o = o.view(cfg.tokens, cfg.groups * cfg.width)
            gate = None if self.gate is None else self.gate.view(o.shape)
            qstate_group_norm(cfg, o, self.weight, self.bias, gate, o, stream)
            return
        o = o.view(cfg.tokens, cfg.groups, cfg.width)
        gate = None if self.gate is None else self.gate.view(o.shape)
        qstate_norm(cfg, o, self.weight, gate, r=o, stream=stream)


def _check_projection(project, cfg: Config, device) -> None:
    """A projection of the readout [.., heads, dv], refused before any launch."""
    _refuse_gradients("project", ())
    if not isinstance(project, Weight4):
        raise TypeError(f"project: expected a Weight4, got {type(project).__name__}")
    if project.inputs != cfg.heads * cfg.dv:
        raise ValueError(f"project: {project.inputs} inputs for a readout of {cfg.heads} x {cfg.dv}")
    if project.packed.device != device:
        raise ValueError(f"project is on {project.packed.device}, the state on {device}")


class QState:
    """A handle plus the torch device buffers it works on (caller-owned memory)."""

    def __init__(self, cfg: Config, device="cuda"):
        # the handle's own: the caller may change its configuration for the next handle, and every call's
        # checks go by the sizes of this one's memory
        self.cfg = cfg = copy.deepcopy(cfg)
        self._c, self._keep = cfg.to_c()  # what the calls that take a configuration get
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

    def step(self, q, k, v, alpha, beta=None, o=None, stream=None, norm=None, project=None):
        """One token for every sequence; with `norm` (a ReadoutNorm), o is the normed and gated
        readout; with `project` (a Weight4 of heads * dv inputs), o's projection [N, outputs] is
        returned, in the memory of the stream of the call (`linear4`: beyond about a hundred sequences
        a product with 16-bit weights is the faster one)."""
        if project is not None:
            if o is None:
                raise ValueError("project: there is no readout without o")
            _check_projection(project, self.cfg, self.codes.device)
        if norm is not None:  # refused before the state changes
            if o is None:
                raise ValueError("norm: there is no readout without o")
            shape = (self.cfg.batch, self.cfg.heads, self.cfg.dv)
            cfg = norm.config(shape, torch.float32, o.device, o.shape)
        qstate_step(self.handle, self.cfg, q, k, v, alpha, beta, o, stream)
        if norm is not None:
            norm._run(cfg, o, stream)
        if project is None:
            return None
        with torch.no_grad(), nullcontext() if stream is None else _on(stream, o.device):
            return linear4(o.view(self.cfg.batch, -1), project)

    def prefill(self, q, k, v, log_alpha, beta=None, offsets=None, norm=None, stream=None,
                project=None):
        """A prompt's or a chunk's tokens at once, for sequences that decode on with `step`: the
        scan from the stored state, whose end is stored back (one quantization event for every
        sequence, those without tokens too: the counter goes up by one, a window starts empty).
        Arguments as `scan`'s, one sequence per batch row, q and k with the handle's heads or a
        divisor of them; returns o (with `project`, its projection [.., outputs], by `linear4`, which is
        meant for chunks of up to about a hundred tokens in all), in the memory of the stream of the
        call."""
        c = self.cfg
        if project is not None:
            _check_projection(project, c, self.codes.device)
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
            if project is not None:
                o = linear4(o.flatten(-2), project)
        return o

    def verify(self, q, k, v, log_alpha, beta=None, parents=None, norm=None, stream=None,
               project=None):
        """The readouts of drafted tokens, for every sequence a tree of them over its stored state,
        which stays as it is; returns (o, draft), `draft` for `accept`.

        q, k [N, T, heads_qk, dk], v [N, T, heads, dv], one dtype (float32, bfloat16, float16), T up
        to 64 (32 with dk = 256), heads_qk a divisor of the handle's heads; log_alpha [N, T, heads]
        (GDN, SCALAR) or [N, T, heads, dk] (GLA, KDA) and beta [N, T, heads] (not for GLA) in float32.
        parents [N, T] (int32, on the device): the earlier row of the sequence that a row hangs on, -1
        for the stored state, anything else (-2) where the row is padding; None is a chain.  o, of v's
        shape and dtype, is what `step` would read out behind each node's path, without the
        quantization after every token; zero in rows of no node.  A node that is not finite spoils
        those that hang on it and no other.  With `norm` o is normed and gated as in `step`, with
        `project` its projection [N, T, outputs] is returned; both take rows of no node as rows of
        zeros, which a norm's bias (and gate) makes others.  (The projection is `linear4`'s: beyond about
        a hundred rows N T a product with 16-bit weights is the faster one.)  o and draft lie in the
        memory of the stream of the call.  Not differentiable: inputs that want a gradient are refused, and so are
        forward-mode derivatives and tracing (make_fx, torch.jit.trace).  Not for key-axis groups and
        pair windows."""
        dev = self.codes.device
        if norm is not None:  # refused before any launch
            _refuse_gradients("verify", (norm.weight, norm.gate, norm.bias))
            _on_device(v, "v", dev)
            rows = v.shape[0] * v.shape[1] if v.dim() == 4 else 0
            cfg = norm.config((rows, self.cfg.heads, self.cfg.dv), v.dtype, dev, v.shape)
        if project is not None:
            _check_projection(project, self.cfg, dev)
        with nullcontext() if stream is None else _on(stream, dev):
            o, draft = _verify(self.cfg, self._c, self.codes, self.scales, q, k, v, log_alpha, beta,
                               parents)
            if norm is not None:
                norm._run(cfg, o)
            if project is not None:
                o = linear4(o.flatten(-2), project)
        return o, draft

    def accept(self, draft: Draft, last, stream=None):
        """The path of drafted tokens that ends in row last[n] (int32 [N], on the device) enters the
        stored state of sequence n, in one quantization event: the counter goes up by one.  A sequence
        with last[n] = -1 accepts none and keeps its state bit for bit.  In a captured graph every
        replay is the event of the capture: the counter stays, and SR's random bits repeat.  Not
        differentiable, as `verify`."""
        dev = self.codes.device
        step = self.step_counter
        with nullcontext() if stream is None else _on(stream, dev):
            _accept(self.cfg, self._c, self.codes, self.scales, step, draft, last)
        self.step_counter = step + 1

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
