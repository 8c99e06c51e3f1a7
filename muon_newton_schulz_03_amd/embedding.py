"""Python binding of the embedding: the lookup with scaling, and its gradient by sorted tokens.

In the manner of `block`: the forward call takes part in torch's autograd where
the table requires grad (differentiable once, no given output then), every
call runs in the HIP library on the current torch stream of the tensors'
device, and there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import EmbeddingDesc
from .block import _DTYPES, _check, _given, _On, _recorded, _refuse_recorded, _rows, _stream, _written

_INDEX = {torch.int32: _lib.MUON_INDEX_I32, torch.int64: _lib.MUON_INDEX_I64}


def _check_ids(ids: torch.Tensor) -> None:
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise ValueError("ids is not a device tensor")
    if ids.dtype not in _INDEX:
        raise ValueError("ids must be int32 or int64")
    if not ids.is_contiguous():
        raise ValueError("ids must be contiguous")


def _table(t: torch.Tensor, name: str, device) -> Tuple[int, int, int]:
    _check(t, name, device)
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32 or bfloat16")
    if t.dim() != 2:
        raise ValueError(f"{name} must have shape (vocab, columns)")
    return _rows(t, name)


def _check_scale(scale) -> None:
    if isinstance(scale, torch.Tensor):  # no gradient would reach it, and the call would wait for one on a device
        raise ValueError("scale must be a number, not a tensor (multiply the result by it instead)")


def embedding_forward(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0,
                      dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids], of shape ids.shape + (columns,).

    table (vocab, columns): float32 or bfloat16, with contiguous columns.
    ids: int32 or int64, contiguous; one outside [0, vocab), such as the
    padding of a batch, has a row of zeros and passes no gradient on.  dtype:
    the result's, default the table's (or that of a given out).  scale: a
    number; a tensor is refused, for its gradient would be lost.
    """
    _check_scale(scale)
    if _recorded(table, None, None):
        _refuse_recorded(out=out)
        return _Embedding.apply(table, ids, scale, dtype)
    return _forward(table, ids, scale, dtype, out)


def _forward(table, ids, scale, dtype, out=None):
    lib = _lib.load()
    _check_ids(ids)
    dev = ids.device
    vocab, cols, ld = _table(table, "table", dev)
    if dtype is None:
        dtype = table.dtype if out is None else getattr(out, "dtype", None)
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    shape, given, ld_out = (*ids.shape, cols), None, 0
    with _On(dev):
        if out is None:
            out = table.new_empty(shape, dtype=dtype)
        else:
            _check(out, "out", dev, dtype)
            if out.shape != shape:
                raise ValueError(f"out has shape {tuple(out.shape)}, not {shape}")
            ld_out, given = _rows(out, "out")[2], _given(out)
        d = EmbeddingDesc(ids.numel(), vocab, cols, ld, ld_out, _DTYPES[table.dtype], _DTYPES[dtype],
                          _INDEX[ids.dtype], scale, 0)
        _lib.check(lib.muon_embedding_forward(ctypes.byref(d), ids.data_ptr(), table.data_ptr(), out.data_ptr(),
                                              _stream(dev.index)))
    if given:
        _written(given)
    return out


def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, vocab: int, *, scale: float = 1.0,
                       dtype: torch.dtype = torch.float32, dtable: Optional[torch.Tensor] = None,
                       accumulate: bool = False) -> torch.Tensor:
    """Gradient of `embedding_forward` for its table: dtable (vocab, columns), in `dtype`.

    Sums are float32, rounded once, and reproducible: they depend on the ids
    and values alone.  A given dtable (whose dtype counts then) is overwritten,
    or with accumulate added to, where rows that no id names stay as they are.
    """
    _check_scale(scale)
    lib = _lib.load()
    _check_ids(ids)
    dev = ids.device
    _check(dout, "dout", dev)
    if dout.dtype not in _DTYPES:
        raise ValueError("dout must be float32 or bfloat16")
    if dout.dim() != ids.dim() + 1 or dout.shape[:-1] != ids.shape:
        raise ValueError(f"dout has shape {tuple(dout.shape)}, which does not go with ids of {tuple(ids.shape)}")
    if not vocab > 0:
        raise ValueError("vocab must be positive")
    _, cols, ld_out = _rows(dout, "dout")
    given, ld = None, 0
    with _On(dev):
        if dtable is None:
            if accumulate:
                raise ValueError("accumulate needs a given dtable")
            if dtype not in _DTYPES:
                raise ValueError("dtype must be float32 or bfloat16")
            dtable = dout.new_empty((vocab, cols), dtype=dtype)
        else:
            rows, width, ld = _table(dtable, "dtable", dev)
            if (rows, width) != (vocab, cols):
                raise ValueError(f"dtable has shape {tuple(dtable.shape)}, not {(vocab, cols)}")
            given = _given(dtable)
        d = EmbeddingDesc(ids.numel(), vocab, cols, ld, ld_out, _DTYPES[dtable.dtype], _DTYPES[dout.dtype],
                          _INDEX[ids.dtype], scale, 0)
        nbytes = lib.muon_embedding_workspace_size(ctypes.byref(d))
        if nbytes == 0:
            raise _lib.MuonError(_lib.MUON_E_INVAL, _lib.last_error())
        ws = dout.new_empty(nbytes, dtype=torch.uint8)
        _lib.check(lib.muon_embedding_backward(
            ctypes.byref(d), ids.data_ptr(), dout.data_ptr(), dtable.data_ptr(),
            _lib.EMBEDDING_ACCUMULATE if accumulate else 0, ws.data_ptr(), nbytes, _stream(dev.index)))
    if given:
        _written(given)
    return dtable


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, scale, dtype):
        out = _forward(table, ids, scale, dtype)
        ctx.save_for_backward(ids)
        ctx.set_materialize_grads(False)
        ctx.table = table.shape[0], table.dtype, scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        if dout is None:
            return None, None, None, None
        (ids,) = ctx.saved_tensors
        vocab, dtype, scale = ctx.table
        try:
            _rows(dout, "dout")
        except ValueError:  # the gradient of a sum, for example, repeats one value
            dout = dout.contiguous()
        return embedding_backward(dout, ids, vocab, scale=scale, dtype=dtype), None, None, None
