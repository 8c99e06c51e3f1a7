"""Python binding of the transformer block's operators: layer norm and packed causal attention.

Each has a forward and a backward call; the caller keeps what the backward
call needs (its inputs, and the statistics that the forward call returns).
Where torch records gradients (grad mode is on and an input requires grad),
the forward calls take part: y and out carry a graph whose backward pass is
the backward call.  It is differentiable once, and the statistics (mean, rstd,
lse) pass no gradient on: one that arrives there raises.  The backward calls
themselves return plain values.  A given output cannot be recorded, so with
such inputs it is refused, and so is a tensor that requires grad in place of a
number (eps, scale).
A recorded backward pass may be captured in a graph under torch's own rule:
forward and backward in the same capture, and no eager graph of the same
leaves alive (torch ends the process otherwise, whatever the operators).
Every call runs in the HIP library on the current torch stream of the
tensors' device, which need not be the current device; this module checks
the tensors, allocates outputs that are not given, and the workspace, with
torch, and fills descriptors.  There is no fallback: if the library is
missing, `_lib.load` raises.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import AttentionDesc, Heads, LayerNormDesc

_DTYPES = {torch.float32: _lib.MUON_DTYPE_F32, torch.bfloat16: _lib.MUON_DTYPE_BF16}


def _check(t: torch.Tensor, name: str, device: torch.device, dtype=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} is not a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, cols, leading dimension) of a tensor whose leading dimensions step as one."""
    if t.dim() < 1:
        raise ValueError(f"{name} must have at least one dimension")
    cols = t.shape[-1]
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    rows, ld, step = 1, cols, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size != 1:
            if step is None:
                ld = stride
            elif stride != step:
                raise ValueError(f"{name}: the leading dimensions do not step as one (call .contiguous())")
            step = stride * size
        rows *= size
    if rows > 1 and ld < cols:
        raise ValueError(f"{name}: rows overlap (stride {ld} for {cols} columns)")
    return rows, cols, ld if rows > 1 else cols


def _param(p: Optional[torch.Tensor], name: str, cols: int, device, dtype):
    if p is None:
        return dtype, None
    _check(p, name, device, dtype)
    if p.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16")
    if p.shape != (cols,) or not p.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {cols} elements")
    return p.dtype, p.data_ptr()


# The current stream's handle by device index; torch.cuda.current_stream builds an object around it first (1.8 us
# instead of 0.1, of about 10 in a call).
_stream = torch._C._cuda_getCurrentRawStream


class _On:
    """The device guard of a call: nothing when the tensors' device is current already."""

    def __init__(self, device: torch.device):
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


_grad_on = torch.is_grad_enabled


def _recorded(a, b, c) -> bool:
    """Whether torch differentiates with respect to one of these inputs (None, or no tensor: refused later, is none)."""
    if _grad_on():
        for t in (a, b, c):
            if getattr(t, "requires_grad", False):
                return True
    return forward_ad._current_level >= 0 and any(
        isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None for t in (a, b, c))


def _refuse_number(name: str, value) -> None:
    """A tensor in place of a number: refused where torch would differentiate with respect to it."""
    if _recorded(value, None, None):
        raise ValueError(f"{name} is a number, which no gradient reaches (detach it)")


def _refuse_recorded(**given) -> None:
    for name, t in given.items():
        if t is not None:
            raise ValueError(f"{name} cannot be given where gradients are recorded (use torch.no_grad() and the "
                             "backward call, or leave it out)")


def _given(*outputs) -> list:
    """The outputs that the caller gave, checked: torch must not take them for results of something else."""
    outputs = [t for t in outputs if t is not None]
    if _grad_on() and any([t.requires_grad for t in outputs]):
        raise ValueError("a given output requires grad, and writing into it would not be recorded")
    return outputs


# Tells torch that tensors were written, so that a graph that saved one notices.
_written = torch.autograd.graph.increment_version


def _only_values(name: str, *grads) -> None:
    if any(g is not None for g in grads):
        raise RuntimeError(f"{name} pass no gradient on: detach them")


def layer_norm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                       eps: float = 1e-5, out: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Layer norm over the last dimension: (y, mean, rstd), the statistics in float32 and of x's leading shape.

    x: float32 or bfloat16, with a contiguous last dimension and rows of one
    stride.  weight and bias (one dtype, float32 or bfloat16) may be None.
    """
    if isinstance(eps, torch.Tensor):
        _refuse_number("eps", eps)
    if _recorded(x, weight, bias):
        _refuse_recorded(out=out)
        return _LayerNorm.apply(x, weight, bias, eps)
    return _norm_forward(x, weight, bias, eps, out)


def _norm_forward(x, weight, bias, eps, out=None):
    lib = _lib.load()
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x is not a device tensor")
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    rows, cols, ld = _rows(x, "x")
    pt, w = _param(weight, "weight", cols, x.device, None)
    pt, b = _param(bias, "bias", cols, x.device, pt)
    with _On(x.device):
        y, given = x.new_empty(x.shape) if out is None else out, None
        if out is not None:
            _check(y, "out", x.device, x.dtype)
            if y.shape != x.shape:
                raise ValueError("out must have x's shape")
            given = _given(out)
        mean = x.new_empty(x.shape[:-1], dtype=torch.float32)
        rstd = torch.empty_like(mean)
        d = LayerNormDesc(rows, cols, ld, 0 if out is None else _rows(y, "out")[2], 0, 0, _DTYPES[x.dtype],
                          _lib.MUON_DTYPE_F32 if pt is None else _DTYPES[pt], eps, 0)
        _lib.check(lib.muon_layernorm_forward(ctypes.byref(d), x.data_ptr(), w, b, y.data_ptr(), mean.data_ptr(),
                                              rstd.data_ptr(), _stream(x.device.index)))
    if given:
        _written(given)
    return y, mean, rstd


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, *, dx: Optional[torch.Tensor] = None,
                        need_weight: bool = True, need_bias: bool = True
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of `layer_norm_forward`: (dx, dweight, dbias).

    dx has x's dtype; dweight and dbias are float32, and None where not needed.
    mean and rstd are the forward call's.
    """
    return _norm_backward(dy, x, mean, rstd, weight, dx, True, need_weight, need_bias)


def _norm_backward(dy, x, mean, rstd, weight, dx, need_x, need_weight, need_bias):
    lib = _lib.load()
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("x is not a device tensor")
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    dev = x.device
    rows, cols, ld = _rows(x, "x")
    _check(dy, "dy", dev, x.dtype)
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    for name, t in (("mean", mean), ("rstd", rstd)):
        _check(t, name, dev, torch.float32)
        if t.shape != x.shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous and of x's leading shape")
    pt, w = _param(weight, "weight", cols, dev, None)
    given = None
    with _On(dev):
        if dx is not None:
            _check(dx, "dx", dev, x.dtype)
            if dx.shape != x.shape:
                raise ValueError("dx must have x's shape")
            given = _given(dx)
        elif need_x:
            dx = x.new_empty(x.shape)
        d = LayerNormDesc(rows, cols, ld, 0, _rows(dy, "dy")[2], 0 if given is None else _rows(dx, "dx")[2],
                          _DTYPES[x.dtype],
                          _lib.MUON_DTYPE_F32 if pt is None else _DTYPES[pt], 0.0, 0)
        dw = x.new_empty(cols, dtype=torch.float32) if need_weight else None
        db = x.new_empty(cols, dtype=torch.float32) if need_bias else None
        ws, nbytes = None, 0
        if need_weight or need_bias:
            nbytes = lib.muon_layernorm_workspace_size(ctypes.byref(d))
            if nbytes == 0:
                raise _lib.MuonError(_lib.MUON_E_INVAL, _lib.last_error())
            ws = x.new_empty(nbytes, dtype=torch.uint8)
        _lib.check(lib.muon_layernorm_backward(
            ctypes.byref(d), dy.data_ptr(), x.data_ptr(), w, mean.data_ptr(), rstd.data_ptr(),
            None if dx is None else dx.data_ptr(), None if dw is None else dw.data_ptr(),
            None if db is None else db.data_ptr(),
            None if ws is None else ws.data_ptr(), nbytes, _stream(dev.index)))
    if given:
        _written(given)
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = _norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.set_materialize_grads(False)
        ctx.params = [None if p is None else p.dtype for p in (weight, bias)]
        return y, mean, rstd

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dmean, drstd):
        _only_values("layer norm's mean and rstd", dmean, drstd)
        need = ctx.needs_input_grad
        if dy is None or not any(need[:3]):
            return None, None, None, None
        x, weight, mean, rstd = ctx.saved_tensors
        try:
            _rows(dy, "dy")
        except ValueError:  # the gradient of a sum, for example, repeats one value
            dy = dy.contiguous()
        dx, dw, db = _norm_backward(dy, x, mean, rstd, weight, None, need[0], need[1], need[2])
        dw, db = (g if g is None else g.to(dtype) for g, dtype in zip((dw, db), ctx.params))
        return dx, dw, db, None


def _heads(t: torch.Tensor, name: str, device, dtype, shape) -> Heads:
    """The descriptor of a (tokens, heads, head_dim) operand after its checks."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} is not a device tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    token, head, elem = t.stride()
    if elem != 1 and shape[2] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return Heads(t.data_ptr(), token, head)


def _readable(g: torch.Tensor) -> torch.Tensor:
    """A (tokens, heads, head_dim) gradient as the library reads it: itself, or a copy where its strides or its start do
    not suit (the gradient of a sum, for example, repeats one value; one through torch.cat may start anywhere)."""
    token, head, elem = g.stride()
    size = g.element_size()
    if elem != 1 or token > 1 << 24 or head > 1 << 31 or any([n % 16 for n in (token * size, head * size, g.data_ptr())]):
        return g.clone(memory_format=torch.contiguous_format)
    return g


def _attention(q, k, v, cu_seqlens, scale):
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} is not a device tensor")
        if t.dim() != 3:
            raise ValueError(f"{name} must have shape (tokens, heads, head_dim)")
    dtype, dev, qs, ks = q.dtype, q.device, q.shape, k.shape
    if dtype not in _DTYPES:
        raise ValueError("q must be float32 or bfloat16")
    if ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError(f"k has shape {tuple(ks)}, which does not go with q's {tuple(qs)}")
    hq, hk, hv = _heads(q, "q", dev, dtype, qs), _heads(k, "k", dev, dtype, ks), _heads(v, "v", dev, dtype, ks)
    _check(cu_seqlens, "cu_seqlens", dev, torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous vector of at least one offset")
    tokens, heads, dim = qs
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    return AttentionDesc(tokens, cu_seqlens.shape[0] - 1, heads, ks[1], dim, _DTYPES[dtype], scale, 0), hq, hk, hv


def packed_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, *,
                             scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention inside each of the packed sequences: (out, lse).

    q (tokens, q_heads, head_dim), k and v (tokens, kv_heads, head_dim):
    bfloat16 or float32, possibly slices of one projection's output.
    cu_seqlens: device int32 offsets of the sequences, 0 first.  scale: of the
    scores, default 1 / sqrt(head_dim).  lse (q_heads, tokens), float32, is for
    the backward call.  Rows behind the last sequence are zero in results that
    this call allocates and left as they were in those given.
    """
    if isinstance(scale, torch.Tensor):
        _refuse_number("scale", scale)
    if _recorded(q, k, v):
        _refuse_recorded(out=out, lse=lse)
        return _Attention.apply(q, k, v, cu_seqlens, scale)
    return _attention_forward(q, k, v, cu_seqlens, scale, out, lse)


def _attention_forward(q, k, v, cu_seqlens, scale, out=None, lse=None):
    lib = _lib.load()
    d, hq, hk, hv = _attention(q, k, v, cu_seqlens, scale)
    dev, flags, given = q.device, 0, None if out is None and lse is None else (out, lse)
    with _On(dev):
        if out is None:
            out, flags = q.new_empty(q.shape), flags | _lib.ATTENTION_ZERO_OUT
        if lse is None:
            lse = q.new_empty((q.shape[1], q.shape[0]), dtype=torch.float32)
            flags |= _lib.ATTENTION_ZERO_LSE
        ho = _heads(out, "out", dev, q.dtype, q.shape)
        _check_lse(lse, q)
        given = given and _given(*given)
        _lib.check(lib.muon_attention_forward(
            ctypes.byref(d), cu_seqlens.data_ptr(), ctypes.byref(hq), ctypes.byref(hk), ctypes.byref(hv),
            ctypes.byref(ho), lse.data_ptr(), flags, _stream(dev.index)))
    if given:
        _written(given)
    return out, lse


def _check_lse(lse, q):
    _check(lse, "lse", q.device, torch.float32)
    if lse.shape != (q.shape[1], q.shape[0]) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous (q_heads, tokens) tensor")


def packed_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              out: torch.Tensor, lse: torch.Tensor, cu_seqlens: torch.Tensor, *,
                              scale: Optional[float] = None, dq: Optional[torch.Tensor] = None,
                              dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None
                              ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of `packed_attention_forward`: (dq, dk, dv), in the inputs' dtype.

    out and lse are the forward call's, under the same scale.  dq, dk and dv
    may be given, for example as slices of one buffer, and are overwritten.
    Rows behind the last sequence are zero in gradients that this call
    allocates and left as they were in those given.
    """
    lib = _lib.load()
    d, hq, hk, hv = _attention(q, k, v, cu_seqlens, scale)
    dev, flags, given = q.device, 0, (dq, dk, dv)
    _check_lse(lse, q)
    dtype, qs, ks = q.dtype, q.shape, k.shape
    hdo, ho = _heads(dout, "dout", dev, dtype, qs), _heads(out, "out", dev, dtype, qs)
    with _On(dev):
        if dq is None:
            dq, flags = q.new_empty(qs), flags | _lib.ATTENTION_ZERO_DQ
        if dk is None:
            dk, flags = q.new_empty(ks), flags | _lib.ATTENTION_ZERO_DK
        if dv is None:
            dv, flags = q.new_empty(ks), flags | _lib.ATTENTION_ZERO_DV
        gq, gk = _heads(dq, "dq", dev, dtype, qs), _heads(dk, "dk", dev, dtype, ks)
        gv = _heads(dv, "dv", dev, dtype, ks)
        given = _given(*given)
        nbytes = lib.muon_attention_workspace_size(ctypes.byref(d))
        if nbytes == 0:
            raise _lib.MuonError(_lib.MUON_E_INVAL, _lib.last_error())
        ws = q.new_empty(nbytes, dtype=torch.uint8)
        _lib.check(lib.muon_attention_backward(
            ctypes.byref(d), cu_seqlens.data_ptr(), ctypes.byref(hdo), ctypes.byref(hq), ctypes.byref(hk),
            ctypes.byref(hv), ctypes.byref(ho), lse.data_ptr(), ctypes.byref(gq), ctypes.byref(gk), ctypes.byref(gv),
            flags, ws.data_ptr(), nbytes, _stream(dev.index)))
    if given:
        _written(given)
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale):
        out, lse = _attention_forward(q, k, v, cu_seqlens, scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.set_materialize_grads(False)
        ctx.scale = scale
        return out, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dlse):
        _only_values("attention's lse", dlse)
        if dout is None:
            return None, None, None, None, None
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        grads = packed_attention_backward(_readable(dout), q, k, v, out, lse, cu_seqlens, scale=ctx.scale)
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None)
