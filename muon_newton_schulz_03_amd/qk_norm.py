"""Python binding of the norm of queries and keys for each head, with the position rotation in the same pass.

In the manner of `block`: the forward call takes part in torch's autograd where
an input requires grad (differentiable once, no given outputs then), every
call runs in the HIP library on the current torch stream of the tensors'
device, and there is no fallback.  Nothing is kept for the backward call but
the inputs.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import Heads, QkNormDesc, RotationDesc
from .block import (_DTYPES, _check, _given, _heads, _On, _param, _readable, _recorded, _refuse_number, _refuse_recorded,
                    _stream, _written)
from .embedding import _INDEX

_PAIRS = {"halves": _lib.PAIRS_HALVES, "neighbours": _lib.PAIRS_NEIGHBOURS}


class Rotation:
    """Which elements of a head turn with the position, and how fast.

    The first `dim` elements turn in pairs, (i, i + dim / 2) as "halves" or
    (2 i, 2 i + 1) as "neighbours", pair i by position * base ** (-2 i / dim)
    radians, or by position * frequencies[i] where those are given (0 keeps a
    pair as it is, a negative one turns it back).
    """

    def __init__(self, dim: int, base: float = 10000.0, *, frequencies: Optional[Sequence[float]] = None,
                 pairs: str = "halves"):
        if pairs not in _PAIRS:
            raise ValueError(f"pairs must be one of {tuple(_PAIRS)}")
        if dim < 0 or dim % 8:
            raise ValueError("dim must be a multiple of 8")
        if frequencies is None:
            if not base > 0:
                raise ValueError("base must be positive")
            frequencies = [base ** (-2 * i / dim) for i in range(dim // 2)]
        if len(frequencies) != dim // 2:
            raise ValueError(f"{dim} elements need {dim // 2} frequencies, not {len(frequencies)}")
        if any(_recorded(f, None, None) for f in frequencies):
            raise ValueError("base and frequencies are numbers, which no gradient reaches (detach them)")
        self.dim, self.pairs = dim, pairs
        self.frequencies = tuple(float(f) for f in frequencies)
        self._host = (ctypes.c_double * max(1, dim // 2))(*self.frequencies)
        self._desc = RotationDesc(self._host, dim, _PAIRS[pairs])

    def __reduce__(self):  # copied and saved with the model that holds it; the host array is not
        return _rebuilt, (self.dim, self.frequencies, self.pairs)

    def __repr__(self):
        return f"Rotation({self.dim}, frequencies={self.frequencies}, pairs={self.pairs!r})"


def _rebuilt(dim, frequencies, pairs):
    return Rotation(dim, frequencies=frequencies, pairs=pairs)


_DIMS = "{} must have shape (tokens, heads, head_dim)"


def _inputs(q, k, rotation, q_weight, k_weight, cu_seqlens, positions, eps):
    """The descriptor and pointers that both calls share, after their checks."""
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} is not a device tensor")
    dtype, dev, qs, ks = q.dtype, q.device, q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError(_DIMS.format("q" if len(qs) != 3 else "k"))
    if dtype not in _DTYPES:
        raise ValueError("q must be float32 or bfloat16")
    tokens, heads, dim = qs
    if ks[0] != tokens or ks[2] != dim:
        raise ValueError(f"k has shape {tuple(ks)}, which does not go with q's {tuple(qs)}")
    if rotation is None:
        turn = None
    elif isinstance(rotation, Rotation):
        turn = ctypes.byref(rotation._desc)
    else:
        raise ValueError("rotation must be a Rotation or None")
    hq, hk = _heads(q, "q", dev, dtype, qs), _heads(k, "k", dev, dtype, ks)
    pt = wq = wk = cu = pos = None
    seqs, index = 0, _lib.MUON_INDEX_I32
    if q_weight is not None:
        pt, wq = _param(q_weight, "q_weight", dim, dev, None)
    if k_weight is not None:
        pt, wk = _param(k_weight, "k_weight", dim, dev, pt)
    if cu_seqlens is not None:
        _check(cu_seqlens, "cu_seqlens", dev, torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous vector of at least one offset")
        cu, seqs = cu_seqlens.data_ptr(), cu_seqlens.shape[0] - 1
    if positions is not None:
        _check(positions, "positions", dev)
        if positions.dtype not in _INDEX:
            raise ValueError("positions must be int32 or int64")
        if positions.shape != (tokens,) or not positions.is_contiguous():
            raise ValueError("positions must be a contiguous vector of one position per token")
        pos, index = positions.data_ptr(), _INDEX[positions.dtype]
    d = QkNormDesc(tokens, seqs, heads, ks[1], dim, _DTYPES[dtype],
                   _lib.MUON_DTYPE_F32 if pt is None else _DTYPES[pt], index, eps, 0)
    return ctypes.byref(d), turn, cu, pos, hq, hk, wq, wk


def _output(like, given, name):
    """A result in the shape of `like`, and its descriptor: a new one, or the given one after its checks."""
    shape = like.shape
    if given is None:
        new = torch.empty_like(like, memory_format=torch.contiguous_format)  # 1.2 us, like.new_empty(shape) 1.6
        return new, Heads(new.data_ptr(), shape[1] * shape[2], shape[2])
    return given, _heads(given, name, like.device, like.dtype, shape)


def qk_norm_forward(q: torch.Tensor, k: torch.Tensor, rotation: Optional[Rotation] = None, *,
                    q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Root-mean-square norm of each head of q and k, then the rotation by position: (q_out, k_out).

    q (tokens, q_heads, head_dim) and k (tokens, k_heads, head_dim): bfloat16
    or float32, possibly slices of one projection's output.  q_weight and
    k_weight: head_dim elements of one dtype, the same for every head, or None.
    A token's position is positions[token] (device int32 or int64), or without
    them its offset in its sequence of cu_seqlens (device int32 offsets, 0
    first), or without either its number.  Rows behind the last sequence of
    cu_seqlens are zero in results that this call allocates and left as they
    were in those given.
    """
    if isinstance(eps, torch.Tensor):
        _refuse_number("eps", eps)
    if _recorded(q, k, q_weight) or k_weight is not None and _recorded(k_weight, None, None):
        _refuse_recorded(q_out=q_out, k_out=k_out)
        return _QkNorm.apply(q, k, q_weight, k_weight, rotation, cu_seqlens, positions, eps)
    return _forward(q, k, rotation, q_weight, k_weight, cu_seqlens, positions, eps, q_out, k_out)


def _forward(q, k, rotation, q_weight, k_weight, cu_seqlens, positions, eps, q_out=None, k_out=None):
    lib = _lib.load()
    d, turn, cu, pos, hq, hk, wq, wk = _inputs(q, k, rotation, q_weight, k_weight, cu_seqlens, positions, eps)
    given = None if q_out is None and k_out is None else (q_out, k_out)
    flags = (q_out is None) * _lib.QK_ZERO_Q | (k_out is None) * _lib.QK_ZERO_K
    index = q.device.index
    with _On(q.device):
        q_out, oq = _output(q, q_out, "q_out")
        k_out, ok = _output(k, k_out, "k_out")
        given = given and _given(*given)
        _lib.check(lib.muon_qk_norm_forward(d, turn, cu, pos, ctypes.byref(hq), ctypes.byref(hk), wq, wk,
                                            ctypes.byref(oq), ctypes.byref(ok), flags, _stream(index)))
    if given:
        _written(given)
    return q_out, k_out


def qk_norm_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     rotation: Optional[Rotation] = None, *, q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None, eps: float = 1e-6, dq: Optional[torch.Tensor] = None,
                     dk: Optional[torch.Tensor] = None, need_q_weight: Optional[bool] = None,
                     need_k_weight: Optional[bool] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients of `qk_norm_forward` under the same arguments: (dq, dk, dq_weight, dk_weight).

    q and k are the forward call's inputs, dq_out and dk_out the gradients of
    its results.  dq and dk may be given, for example as slices of the
    projection's gradient, and are overwritten.  The weight gradients are
    float32, and None where not needed (by default: where there is no weight).
    Rows behind the last sequence are zero in gradients that this call
    allocates and left as they were in those given.
    """
    lib = _lib.load()
    d, turn, cu, pos, hq, hk, wq, wk = _inputs(q, k, rotation, q_weight, k_weight, cu_seqlens, positions, eps)
    dev, dtype = q.device, q.dtype
    gq, gk = _heads(dq_out, "dq_out", dev, dtype, q.shape), _heads(dk_out, "dk_out", dev, dtype, k.shape)
    given = None if dq is None and dk is None else (dq, dk)
    flags = (dq is None) * _lib.QK_ZERO_Q | (dk is None) * _lib.QK_ZERO_K
    with _On(dev):
        dq, oq = _output(q, dq, "dq")
        dk, ok = _output(k, dk, "dk")
        given = given and _given(*given)
        dwq = dwk = pwq = pwk = ws = None
        nbytes = 0
        if wq is not None if need_q_weight is None else need_q_weight:
            dwq = q.new_empty(q.shape[2], dtype=torch.float32)
            pwq = dwq.data_ptr()
        if wk is not None if need_k_weight is None else need_k_weight:
            dwk = q.new_empty(q.shape[2], dtype=torch.float32)
            pwk = dwk.data_ptr()
        if pwq or pwk:
            nbytes = lib.muon_qk_norm_workspace_size(d)
            if nbytes == 0:
                raise _lib.MuonError(_lib.MUON_E_INVAL, _lib.last_error())
            ws = q.new_empty(nbytes, dtype=torch.uint8)
        _lib.check(lib.muon_qk_norm_backward(
            d, turn, cu, pos, ctypes.byref(gq), ctypes.byref(gk), ctypes.byref(hq), ctypes.byref(hk), wq, wk,
            ctypes.byref(oq), ctypes.byref(ok), pwq, pwk, flags, None if ws is None else ws.data_ptr(), nbytes,
            _stream(dev.index)))
    if given:
        _written(given)
    return dq, dk, dwq, dwk


class _QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, rotation, cu_seqlens, positions, eps):
        q_out, k_out = _forward(q, k, rotation, q_weight, k_weight, cu_seqlens, positions, eps)
        ctx.save_for_backward(q, k, q_weight, k_weight, cu_seqlens, positions)
        ctx.how = rotation, eps
        return q_out, k_out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cu_seqlens, positions = ctx.saved_tensors
        rotation, eps = ctx.how
        need = ctx.needs_input_grad
        dq, dk, dwq, dwk = qk_norm_backward(_readable(dq_out), _readable(dk_out), q, k, rotation, q_weight=q_weight,
                                            k_weight=k_weight, cu_seqlens=cu_seqlens, positions=positions, eps=eps,
                                            need_q_weight=need[2], need_k_weight=need[3])
        dwq, dwk = (g if g is None else g.to(w.dtype) for g, w in ((dwq, q_weight), (dwk, k_weight)))
        return dq if need[0] else None, dk if need[1] else None, dwq, dwk, None, None, None, None
