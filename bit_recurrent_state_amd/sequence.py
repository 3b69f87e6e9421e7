"""Binding of include/qstate_scan.h: the recurrences of qstate_step over whole
sequences, and their gradients.

`qstate_scan` and `qstate_scan_backward` marshal arguments like the functions
in qstate.py; `scan` is the differentiable operator on top of them.  Shapes
and dtypes are checked here so that a wrong tensor fails before it reaches the
C ABI; every product runs in the library's kernels."""

from __future__ import annotations

import ctypes
import threading
import weakref
from dataclasses import dataclass
from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from ._lib import GDN, GLA, KDA, SCALAR, ScanConfigC, check, lib

__all__ = ["ScanConfig", "qstate_scan_workspace", "qstate_scan", "qstate_scan_backward", "scan"]

DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


@dataclass
class ScanConfig:
    batch: int
    heads: int
    dk: int
    dv: int
    tokens: int
    heads_qk: int = 0  # 0: heads
    mixer: int = GDN
    dtype: torch.dtype = torch.float32
    q_stride: int = 0  # elements between two tokens; 0: packed
    k_stride: int = 0
    v_stride: int = 0
    o_stride: int = 0

    def to_c(self) -> ScanConfigC:
        if self.dtype not in DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, got {self.dtype}")
        return ScanConfigC(self.batch, self.heads, self.heads_qk or self.heads, self.dk, self.dv,
                           self.mixer, DTYPES[self.dtype], 0, self.tokens, self.q_stride,
                           self.k_stride, self.v_stride, self.o_stride)

    @property
    def vector_gate(self) -> bool:
        return self.mixer in (GLA, KDA)


def _stream(stream, device) -> int:
    """The handle of `stream`, or of the current stream of the device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on(stream, device):
    """A context with `stream` as the current one (None: as it is)."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _call(device, fn, *args):
    """fn(*args) with the tensors' device as the current one."""
    if torch.cuda.current_device() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _on_device(t, name, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the others on {device}")


def _array(t: Optional[torch.Tensor], name: str, dtype, numel: int, device, optional=False):
    """Pointer of a contiguous array of `numel` elements."""
    if t is None:
        if optional:
            return None
        raise TypeError(f"{name} is missing")
    _on_device(t, name, device)
    if t.dtype != dtype or not t.is_contiguous() or t.numel() != numel:
        raise ValueError(f"{name}: expected contiguous {dtype} with {numel} elements, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()}")
    return t.data_ptr()


def _rows(t: Optional[torch.Tensor], name: str, cfg: ScanConfig, heads: int, width: int,
          stride: int, device, optional=False):
    """Pointer of [tokens][heads][width] rows, `stride` elements apart."""
    if t is None and optional:
        return None
    _on_device(t, name, device)
    want = (cfg.tokens, heads, width)
    if t.dtype != cfg.dtype or tuple(t.shape) != want:
        raise ValueError(f"{name}: expected {cfg.dtype} {want}, got {t.dtype} {tuple(t.shape)}")
    ok = ((width == 1 or t.stride(2) == 1) and (heads == 1 or t.stride(1) == width)
          and (cfg.tokens <= 1 or t.stride(0) == (stride or heads * width)))
    if t.numel() and not ok:
        raise ValueError(f"{name}: strides {t.stride()} are not {stride or heads * width} elements "
                         "between tokens with packed heads")
    return t.data_ptr()


def qstate_scan_workspace(cfg: ScanConfig, backward: bool = False) -> int:
    return _workspace_bytes(cfg.to_c(), backward)


def _workspace_bytes(c: ScanConfigC, backward: bool) -> int:
    n = ctypes.c_size_t()
    check("qstate_scan_workspace", lib().qstate_scan_workspace(c, int(backward), n))
    return n.value


def _launch_scan(c, dev, inputs, o, final_state, workspace, stream):
    check("qstate_scan", _call(dev, lib().qstate_scan, c, *inputs, o, final_state, *workspace,
                               _stream(stream, dev)))


def _launch_backward(c, dev, inputs, more, workspace, stream):
    check("qstate_scan_backward", _call(dev, lib().qstate_scan_backward, c, *inputs, *more,
                                        *workspace, _stream(stream, dev)))


def _bytes_on(n: int, dev, stream) -> torch.Tensor:
    """n bytes that belong to the stream of the call: once freed they are used again only behind
    its kernels, also where it is not the current one."""
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=dev)
    with _on(stream, dev):
        return torch.empty(n, dtype=torch.uint8, device=dev)


def _own_workspace(c, backward, dev, stream=None):
    """A workspace of this call: the tensor, and (pointer, bytes)."""
    w = _bytes_on(_workspace_bytes(c, backward), dev, stream)
    return w, (w.data_ptr(), w.numel())


def _inputs(cfg: ScanConfig, q, k, v, log_alpha, beta, offsets, initial_state):
    _on_device(q, "q", None)
    dev = q.device
    hq = cfg.heads_qk or cfg.heads
    gates = cfg.tokens * cfg.heads
    return (
        _rows(q, "q", cfg, hq, cfg.dk, cfg.q_stride, dev),
        _rows(k, "k", cfg, hq, cfg.dk, cfg.k_stride, dev),
        _rows(v, "v", cfg, cfg.heads, cfg.dv, cfg.v_stride, dev),
        _array(log_alpha, "log_alpha", torch.float32,
               gates * (cfg.dk if cfg.vector_gate else 1), dev),
        None if cfg.mixer == GLA else _array(beta, "beta", torch.float32, gates, dev),
        _array(offsets, "offsets", torch.int64, cfg.batch + 1, dev, optional=True),
        _array(initial_state, "initial_state", torch.float32,
               cfg.batch * cfg.heads * cfg.dv * cfg.dk, dev, optional=True),
    )


def _workspace(workspace, dev):
    _on_device(workspace, "workspace", dev)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor")
    return workspace.data_ptr(), workspace.numel()


def qstate_scan(cfg: ScanConfig, q, k, v, log_alpha, beta=None, offsets=None, initial_state=None,
                o=None, final_state=None, workspace=None, stream=None) -> None:
    """The scan into `o` and `final_state` (either may be None)."""
    args = _inputs(cfg, q, k, v, log_alpha, beta, offsets, initial_state)
    dev = q.device
    po = _rows(o, "o", cfg, cfg.heads, cfg.dv, cfg.o_stride, dev, optional=True)
    ps = _array(final_state, "final_state", torch.float32,
                cfg.batch * cfg.heads * cfg.dv * cfg.dk, dev, optional=True)
    c = cfg.to_c()
    keep, w = (None, _workspace(workspace, dev)) if workspace is not None else \
        _own_workspace(c, False, dev, stream)
    _launch_scan(c, dev, args, po, ps, w, stream)


def qstate_scan_backward(cfg: ScanConfig, q, k, v, log_alpha, beta, offsets, initial_state, d_o,
                         d_final_state, dq, dk, dv, dlog_alpha, dbeta=None, d_initial_state=None,
                         workspace=None, stream=None) -> None:
    """Gradients of the scan's inputs from those of `o` and `final_state`; `d_o` and the gradients are
    packed."""
    args = _inputs(cfg, q, k, v, log_alpha, beta, offsets, initial_state)
    dev = q.device
    hq = cfg.heads_qk or cfg.heads
    state = cfg.batch * cfg.heads * cfg.dv * cfg.dk
    gates = cfg.tokens * cfg.heads
    f32 = torch.float32
    more = (
        _array(d_o, "d_o", cfg.dtype, gates * cfg.dv, dev),
        _array(d_final_state, "d_final_state", f32, state, dev, optional=True),
        _array(dq, "dq", cfg.dtype, cfg.tokens * hq * cfg.dk, dev),
        _array(dk, "dk", cfg.dtype, cfg.tokens * hq * cfg.dk, dev),
        _array(dv, "dv", cfg.dtype, gates * cfg.dv, dev),
        _array(dlog_alpha, "dlog_alpha", f32, gates * (cfg.dk if cfg.vector_gate else 1), dev),
        None if cfg.mixer == GLA else _array(dbeta, "dbeta", f32, gates, dev),
        _array(d_initial_state, "d_initial_state", f32, state, dev, optional=True),
    )
    c = cfg.to_c()
    keep, w = (None, _workspace(workspace, dev)) if workspace is not None else \
        _own_workspace(c, True, dev, stream)
    _launch_backward(c, dev, args, more, w, stream)


def _token_rows(t: torch.Tensor) -> torch.Tensor:
    """[.., heads, d] with any leading dims as [tokens][heads][d]; a copy only where the heads are
    not packed, the tokens do not lie at one distance (or 2^22 elements and more apart), or rows
    start off a 16-byte boundary."""
    heads, d = t.shape[-2:]
    try:
        r = t.view(-1, heads, d)
    except RuntimeError:
        r = t.reshape(-1, heads, d)
    packed = (d == 1 or r.stride(2) == 1) and (heads == 1 or r.stride(1) == d)
    apart = r.shape[0] <= 1 or heads * d <= r.stride(0) <= 1 << 22
    if not (packed and apart) or r.data_ptr() % 16:
        r = r.clone(memory_format=torch.contiguous_format)
    return r


def _row_stride(t: torch.Tensor) -> int:
    n = t.shape[1] * t.shape[2]
    return 0 if t.shape[0] <= 1 or t.stride(0) == n else t.stride(0)


def _aligned(t: torch.Tensor) -> torch.Tensor:
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


def _forward(q, k, v, log_alpha, beta, initial_state, offsets, mixer, batch):
    """The checked call: outputs, and what backward needs."""
    q3, k3, v3 = _token_rows(q), _token_rows(k), _token_rows(v)
    g = _aligned(log_alpha)
    b = None if beta is None else _aligned(beta)
    s0 = None if initial_state is None else _aligned(initial_state)
    tokens, heads, dv = v3.shape
    heads_qk, dk = q3.shape[1:]
    dev = v.device
    c = ScanConfigC(batch, heads, heads_qk, dk, dv, mixer, DTYPES[v.dtype], 0, tokens,
                    _row_stride(q3), _row_stride(k3), _row_stride(v3), 0)
    # rows of no sequence are left alone by the kernels
    new = torch.empty if offsets is None else torch.zeros
    o = new(v.shape, dtype=v.dtype, device=dev)
    final = torch.empty((batch, heads, dv, dk), dtype=torch.float32, device=dev)
    keep, w = _own_workspace(c, False, dev)
    saved = (q3, k3, v3, g, b, s0, offsets)
    _launch_scan(c, dev, [_ptr(t) for t in (q3, k3, v3, g, b, offsets, s0)], o.data_ptr(),
                 final.data_ptr(), w, None)
    return o, final, c, saved


def _refuse_tracing(name: str) -> None:
    """A trace records PyTorch's own operations and not the launches: it would hold this call as
    memory that nothing writes."""
    if torch.jit.is_tracing() or torch._C._get_dispatch_mode(
            torch._C._TorchDispatchModeKey.PROXY) is not None:
        raise RuntimeError(f"{name} cannot be traced (make_fx, torch.jit.trace)")


def _through_autograd(tensors) -> bool:
    """Whether a call needs its autograd function: where a gradient is wanted, and inside forward-mode
    differentiation, which has no rule here and is refused by it."""
    if getattr(forward_ad, "_current_level", 0) >= 0:
        return True
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


_alive = weakref.WeakKeyDictionary()  # differentiable calls whose graph lives: their stream
_alive_lock = threading.Lock()  # a pass may be captured in one thread while another begins one


def _note_alive(ctx, device) -> None:
    with _alive_lock:
        _alive[ctx] = _stream(None, device)


def _leaves(nodes) -> set:
    """The leaves that the graph behind these nodes ends in."""
    seen, todo, found = set(nodes), list(nodes), set()
    while todo:
        try:
            behind = todo.pop().next_functions
        except RuntimeError:  # of a call that is just made, or dropped, in another thread
            continue
        for n, _ in behind:
            if n is None or n in seen:
                continue
            seen.add(n)
            if hasattr(n, "variable"):
                found.add(id(n.variable))
            else:
                todo.append(n)
    return found


def _refuse_capture(ctx, device) -> None:
    """Before a backward pass that is being captured: a leaf belongs to the stream of the graph
    that it was first used in for as long as that lives.  PyTorch would have the capture wait for
    another stream, which breaks it off and can end the process.  Looked for are leaves behind this
    call, passed directly or through other operations (a projection's weight), and behind live calls
    of these operators from other streams; graphs without any of these operators are not known here."""
    if not torch.cuda.is_current_stream_capturing():
        return
    here = _stream(None, device)
    with _alive_lock:
        others = [other for other, stream in _alive.items() if stream != here]
    if others and _leaves([ctx]) & _leaves(others):
        raise RuntimeError("a backward pass cannot be captured while a graph of the same "
                           "leaves from another stream lives: drop the results of that call")


class _Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_alpha, beta, initial_state, offsets, mixer, batch):
        o, final, ctx.cfg, saved = _forward(q, k, v, log_alpha, beta, initial_state, offsets,
                                            mixer, batch)
        _note_alive(ctx, v.device)
        ctx.shapes = q.shape, v.shape
        ctx.save_for_backward(*saved)
        ctx.set_materialize_grads(False)
        return o, final

    @staticmethod
    @once_differentiable
    def backward(ctx, d_o, d_final):
        q, k, v, g, b, s0, offsets = ctx.saved_tensors
        dev = v.device
        _refuse_capture(ctx, dev)
        qk, vo = ctx.shapes
        new = torch.empty if offsets is None else torch.zeros
        d_o = torch.zeros(vo, dtype=v.dtype, device=dev) if d_o is None else _aligned(d_o)
        d_final = None if d_final is None else _aligned(d_final)
        dq, dk = new(qk, dtype=v.dtype, device=dev), new(qk, dtype=v.dtype, device=dev)
        dv = new(vo, dtype=v.dtype, device=dev)
        dg = new(g.shape, dtype=torch.float32, device=dev)
        db = None if b is None else new(b.shape, dtype=torch.float32, device=dev)
        ds = torch.empty_like(s0) if s0 is not None and ctx.needs_input_grad[5] else None
        keep, w = _own_workspace(ctx.cfg, True, dev)
        _launch_backward(ctx.cfg, dev, [_ptr(t) for t in (q, k, v, g, b, offsets, s0)],
                         [_ptr(t) for t in (d_o, d_final, dq, dk, dv, dg, db, ds)], w, None)
        return dq, dk, dv, dg, db, ds, None, None, None


def scan(q, k, v, log_alpha, beta=None, *, mixer: int = GDN, initial_state=None, offsets=None):
    """The recurrence of `qstate_step` over whole sequences; returns (o, final_state).

    q, k [N, T, heads_qk, dk], v [N, T, heads, dv], one dtype (float32, bfloat16, float16); or
    packed sequences [tokens, heads, d] with `offsets` [N + 1] (int64, on the device): sequence n
    is rows offsets[n] .. offsets[n+1] - 1.  Head h of v uses head h // (heads / heads_qk) of q
    and k.  log_alpha [.., heads] (GDN, SCALAR) or [.., heads, dk] (GLA, KDA), the logarithm of
    the decay, at most 0; beta [.., heads] (not for GLA); both float32.  initial_state
    [N, heads, dv, dk] float32 (zeros if None).  o has the shape and dtype of v, zero in rows of
    no sequence; final_state is float32 and can go to `QState.load_fp32` to decode on from there.

    Differentiable once in every input but offsets; backward computes the states again.  A backward
    pass is captured into a graph only where no eager graph of the same leaves lives.  Forward-mode
    derivatives and tracing (make_fx, torch.jit.trace) are refused."""
    _refuse_tracing("scan")
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (log_alpha, "log_alpha")):
        _on_device(t, name, v.device if isinstance(v, torch.Tensor) else None)
    if mixer not in (GDN, GLA, SCALAR, KDA):
        raise ValueError(f"mixer: {mixer}")
    packed = offsets is not None
    if v.dim() != (3 if packed else 4):
        raise ValueError("v: expected [tokens, heads, dv] with offsets, else [N, T, heads, dv], got "
                         f"{tuple(v.shape)}")
    if v.dtype not in DTYPES or q.dtype != v.dtype or k.dtype != v.dtype:
        raise ValueError(f"q, k, v: one of float32, bfloat16, float16, got {q.dtype}, {k.dtype}, "
                         f"{v.dtype}")
    lead, heads, dv = v.shape[:-2], v.shape[-2], v.shape[-1]
    if q.dim() != v.dim() or q.shape != k.shape or q.shape[:-2] != lead:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} do not go with v {tuple(v.shape)}")
    heads_qk, dk = q.shape[-2:]
    if heads_qk < 1 or heads % heads_qk:
        raise ValueError(f"{heads} heads of v over {heads_qk} of q and k")
    gate = tuple(lead) + ((heads, dk) if mixer in (GLA, KDA) else (heads,))
    if tuple(log_alpha.shape) != gate or log_alpha.dtype != torch.float32:
        raise ValueError(f"log_alpha: expected float32 {gate}, got {log_alpha.dtype} "
                         f"{tuple(log_alpha.shape)}")
    if mixer == GLA:
        if beta is not None:
            raise ValueError("GLA takes no beta")
    else:
        _on_device(beta, "beta", v.device)
        if tuple(beta.shape) != tuple(lead) + (heads,) or beta.dtype != torch.float32:
            raise ValueError(f"beta: expected float32 {tuple(lead) + (heads,)}, got {beta.dtype} "
                             f"{tuple(beta.shape)}")
    if packed:
        _on_device(offsets, "offsets", v.device)
        if offsets.dim() != 1 or offsets.numel() < 2 or offsets.dtype != torch.int64:
            raise ValueError("offsets: expected int64 [N + 1]")
        offsets = offsets.contiguous()
        batch = offsets.numel() - 1
    else:
        batch = lead[0]
    if initial_state is not None:
        _on_device(initial_state, "initial_state", v.device)
        if (tuple(initial_state.shape) != (batch, heads, dv, dk)
                or initial_state.dtype != torch.float32):
            raise ValueError(f"initial_state: expected float32 {(batch, heads, dv, dk)}, got "
                             f"{initial_state.dtype} {tuple(initial_state.shape)}")
    if _through_autograd((q, k, v, log_alpha, beta, initial_state)):
        return _Scan.apply(q, k, v, log_alpha, beta, initial_state, offsets, mixer, batch)
    return _forward(q, k, v, log_alpha, beta, initial_state, offsets, mixer, batch)[:2]
