"""Binding of include/qstate_draft.h: a tree of drafted tokens over the stored
state, and the state's way along the accepted path.

`qstate_verify` and `qstate_accept` marshal arguments like the functions in
qstate.py; `QState.verify` and `QState.accept` are the calls on a handle."""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from ._lib import GLA, KDA, DraftConfigC, check, lib
from .sequence import (DTYPES, _array, _call, _on_device, _ptr, _refuse_tracing, _stream,
                       _through_autograd)

__all__ = ["Draft", "DraftConfig", "qstate_verify", "qstate_accept"]


@dataclass
class DraftConfig:
    tokens: int  # rows of drafted tokens of a sequence
    heads_qk: int
    dtype: torch.dtype = torch.float32
    q_stride: int = 0  # elements between two rows; 0: packed
    k_stride: int = 0
    v_stride: int = 0

    def to_c(self) -> DraftConfigC:
        if self.dtype not in DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {self.dtype}")
        return DraftConfigC(self.tokens, self.heads_qk, DTYPES[self.dtype], 0, self.q_stride,
                            self.k_stride, self.v_stride)


@dataclass
class Draft:
    """What `verify` leaves for `accept`: the drafted tokens' keys, log decays and parents as they were
    given, and their writes.  Their memory must hold until the accept has run."""

    k: torch.Tensor                  # [N, T, heads_qk, dk]
    log_alpha: torch.Tensor          # float32 [N, T, heads] or [N, T, heads, dk]
    parents: Optional[torch.Tensor]  # int32 [N, T]; None: a chain
    writes: torch.Tensor             # float32 [N, T, heads, dv]


def _rows(t, name, dtype, shape, stride, device):
    """Pointer of [N][T][heads][d] rows, `stride` elements apart."""
    _on_device(t, name, device)
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    N, T, heads, d = shape
    row = stride or heads * d
    ok = ((d == 1 or t.stride(3) == 1) and (heads == 1 or t.stride(2) == d)
          and (T == 1 or t.stride(1) == row) and (N == 1 or t.stride(0) == T * row))
    if not ok:
        raise ValueError(f"{name}: strides {t.stride()} are not {row} elements between rows with "
                         "packed heads")
    return t.data_ptr()


def _state(cfg, codes, scales):
    """(QStateConfig, keep-alive buffers, pointers of the stored state, its device)."""
    from .qstate import qstate_state_bytes
    cb, sb = qstate_state_bytes(cfg)
    _on_device(codes, "codes", None)
    dev = codes.device
    if cfg.fp32_state:
        pc, ps = _array(codes, "state", torch.float32, cb // 4, dev), None
    else:
        pc = _array(codes, "codes", torch.uint8, cb, dev)
        ps = _array(scales, "scales", torch.float32, sb // 4, dev)
    c, keep = cfg.to_c()
    return c, keep, (pc, ps), dev


def _gate(cfg, draft):
    lead = (cfg.batch, draft.tokens, cfg.heads)
    return lead + (cfg.dk,) if cfg.mixer in (GLA, KDA) else lead


def _gates(t, name, shape, device):
    _on_device(t, name, device)
    if tuple(t.shape) != shape or t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous float32 {shape}, got {t.dtype} "
                         f"{tuple(t.shape)} contiguous={t.is_contiguous()}")
    return t.data_ptr()


def qstate_verify(cfg, draft: DraftConfig, codes, scales, q, k, v, log_alpha, beta=None,
                  parents=None, o=None, writes=None, stream=None) -> None:
    """Readouts of a tree of drafted tokens into `o`, what they write into `writes` (either may be
    None); cfg as the state's handle was made with."""
    c, _keep, state, dev = _state(cfg, codes, scales)
    N, T, H, dt = cfg.batch, draft.tokens, cfg.heads, draft.dtype
    args = (
        _rows(q, "q", dt, (N, T, draft.heads_qk, cfg.dk), draft.q_stride, dev),
        _rows(k, "k", dt, (N, T, draft.heads_qk, cfg.dk), draft.k_stride, dev),
        _rows(v, "v", dt, (N, T, H, cfg.dv), draft.v_stride, dev),
        _gates(log_alpha, "log_alpha", _gate(cfg, draft), dev),
        None if cfg.mixer == GLA else _gates(beta, "beta", (N, T, H), dev),
        _array(parents, "parents", torch.int32, N * T, dev, optional=True),
        _array(o, "o", dt, N * T * H * cfg.dv, dev, optional=True),
        _array(writes, "writes", torch.float32, N * T * H * cfg.dv, dev, optional=True),
    )
    check("qstate_verify", _call(dev, lib().qstate_verify, ctypes.byref(c), draft.to_c(), *state,
                                 *args, _stream(stream, dev)))


def qstate_accept(cfg, draft: DraftConfig, step: int, codes, scales, k, log_alpha, parents, writes,
                  last, stream=None) -> None:
    """The stored state behind each sequence's last accepted node, in place, as the quantization
    event `step`."""
    c, _keep, state, dev = _state(cfg, codes, scales)
    N, T = cfg.batch, draft.tokens
    args = (
        _rows(k, "k", draft.dtype, (N, T, draft.heads_qk, cfg.dk), draft.k_stride, dev),
        _gates(log_alpha, "log_alpha", _gate(cfg, draft), dev),
        _array(parents, "parents", torch.int32, N * T, dev, optional=True),
        _array(writes, "writes", torch.float32, N * T * cfg.heads * cfg.dv, dev),
        _array(last, "last", torch.int32, N, dev),
    )
    check("qstate_accept", _call(dev, lib().qstate_accept, ctypes.byref(c), draft.to_c(), step,
                                 *state, *args, _stream(stream, dev)))


def _row_stride(t: torch.Tensor) -> int:
    """Elements between the rows [N][T] of t, or -1 where it takes a copy."""
    if t.data_ptr() % 16:
        return -1
    if t.is_contiguous():
        return 0
    N, T, heads, d = t.shape
    if not ((d == 1 or t.stride(3) == 1) and (heads == 1 or t.stride(2) == d)):
        return -1
    row = t.stride(1) if T > 1 else t.stride(0) if N > 1 else heads * d
    if not heads * d <= row <= 1 << 22 or (N > 1 and T > 1 and t.stride(0) != T * row):
        return -1
    return 0 if row == heads * d else row


def _token_rows(t: torch.Tensor):
    """(t, its row stride); a copy only where the heads are not packed, the rows do not lie at one
    distance, or start off a 16-byte boundary."""
    stride = _row_stride(t)
    if stride < 0:
        t, stride = t.detach().clone(memory_format=torch.contiguous_format), 0
    return t, stride


def _aligned(t: torch.Tensor) -> torch.Tensor:
    if not t.is_contiguous():
        t = t.detach().contiguous()
    return t.detach().clone() if t.data_ptr() % 16 else t


def _check_parents(parents, N, T, device):
    if parents is None:
        return None
    _on_device(parents, "parents", device)
    if tuple(parents.shape) != (N, T) or parents.dtype != torch.int32:
        raise ValueError(f"parents: expected int32 {(N, T)}, got {parents.dtype} "
                         f"{tuple(parents.shape)}")
    return parents.contiguous()


def _check_gate(t, name, shape, device):
    _on_device(t, name, device)
    if tuple(t.shape) != shape or t.dtype != torch.float32:
        raise ValueError(f"{name}: expected float32 {shape}, got {t.dtype} {tuple(t.shape)}")
    return _aligned(t)


def _refuse_gradients(name, tensors):
    _refuse_tracing(name)
    if _through_autograd([t for t in tensors if isinstance(t, torch.Tensor)]):
        raise RuntimeError(f"{name} is not differentiable: call it under torch.no_grad()")


def _verify(cfg, c_cfg, codes, scales, q, k, v, log_alpha, beta, parents):
    """The checked call of QState.verify on the current stream, c_cfg and the state its own: o, the
    draft."""
    _refuse_gradients("verify", (q, k, v, log_alpha, beta))
    dev = codes.device
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _on_device(t, name, dev)
    dt = v.dtype
    if dt not in DTYPES or q.dtype != dt or k.dtype != dt:
        raise ValueError(f"q, k, v: one of float32, bfloat16, float16, got {q.dtype}, {k.dtype}, {dt}")
    shape = v.shape
    if v.dim() != 4 or shape[0] != cfg.batch or shape[2] != cfg.heads or shape[3] != cfg.dv:
        raise ValueError(f"v: expected [{cfg.batch}, T, {cfg.heads}, {cfg.dv}], got {tuple(shape)}")
    N, T = shape[:2]
    qk = q.shape
    if q.dim() != 4 or qk != k.shape or qk[:2] != shape[:2] or qk[3] != cfg.dk:
        raise ValueError(f"q {tuple(qk)} and k {tuple(k.shape)} do not go with v {tuple(shape)} and "
                         f"dk = {cfg.dk}")
    (q, qs), (k, ks), (v, vs) = _token_rows(q), _token_rows(k), _token_rows(v)
    gate = (N, T, cfg.heads) + ((cfg.dk,) if cfg.mixer in (GLA, KDA) else ())
    log_alpha = _check_gate(log_alpha, "log_alpha", gate, dev)
    if cfg.mixer == GLA:
        if beta is not None:
            raise ValueError("GLA takes no beta")
    else:
        beta = _check_gate(beta, "beta", (N, T, cfg.heads), dev)
    parents = _check_parents(parents, N, T, dev)
    o = torch.empty(shape, dtype=dt, device=dev)
    writes = torch.empty(shape, dtype=torch.float32, device=dev)
    c = DraftConfigC(T, qk[2], DTYPES[dt], 0, qs, ks, vs)
    check("qstate_verify", _call(dev, lib().qstate_verify, c_cfg, c, codes.data_ptr(), _ptr(scales),
                                 q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(),
                                 _ptr(beta), _ptr(parents), o.data_ptr(), writes.data_ptr(),
                                 _stream(None, dev)))
    return o, Draft(k, log_alpha, parents, writes)


def _accept(cfg, c_cfg, codes, scales, step, draft, last):
    """The checked call of QState.accept on the current stream, c_cfg and the state its own."""
    _refuse_gradients("accept", (draft.k, draft.log_alpha, draft.writes))
    dev = codes.device
    k, writes = draft.k, draft.writes
    for t, name in ((k, "k"), (writes, "writes"), (last, "last")):
        _on_device(t, name, dev)
    if k.dtype not in DTYPES or k.dim() != 4 or k.shape[0] != cfg.batch or k.shape[3] != cfg.dk:
        raise ValueError(f"k: expected [{cfg.batch}, T, heads_qk, {cfg.dk}], got {k.dtype} "
                         f"{tuple(k.shape)}")
    N, T, heads_qk = k.shape[:3]
    k, ks = _token_rows(k)
    gate = (N, T, cfg.heads) + ((cfg.dk,) if cfg.mixer in (GLA, KDA) else ())
    log_alpha = _check_gate(draft.log_alpha, "log_alpha", gate, dev)
    parents = _check_parents(draft.parents, N, T, dev)
    writes = _check_gate(writes, "writes", (N, T, cfg.heads, cfg.dv), dev)
    if tuple(last.shape) != (N,) or last.dtype != torch.int32:
        raise ValueError(f"last: expected int32 {(N,)}, got {last.dtype} {tuple(last.shape)}")
    last = last.contiguous()
    c = DraftConfigC(T, heads_qk, DTYPES[k.dtype], 0, 0, ks, 0)
    check("qstate_accept", _call(dev, lib().qstate_accept, c_cfg, c, step, codes.data_ptr(),
                                 _ptr(scales), k.data_ptr(), log_alpha.data_ptr(), _ptr(parents),
                                 writes.data_ptr(), last.data_ptr(), _stream(None, dev)))
