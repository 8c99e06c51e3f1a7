"""The block operators' C ABI and binding on the host (no GPU): refusals and workspace sizes.

Every call here is rejected by argument checks before any HIP call, or is host-only.
"""
import ctypes
import math
import os

import pytest
import torch

import block_reference as R
from muon_newton_schulz_03_amd import _lib, block
from muon_newton_schulz_03_amd._lib import AttentionDesc, Heads, LayerNormDesc

INVAL, UNSUP, WORK = _lib.MUON_E_INVAL, _lib.MUON_E_UNSUPPORTED, _lib.MUON_E_WORKSPACE
P = 0x10000  # a pointer that no call follows


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from muon_newton_schulz_03_amd.build import build_library
        build_library()
    return _lib.load()


def norm_desc(**kw):
    d = dict(rows=8, cols=64, ld_x=0, ld_y=0, ld_dy=0, ld_dx=0, x_dtype=1, p_dtype=0, eps=1e-5, reserved=0)
    d.update(kw)
    return LayerNormDesc(*d.values())


BAD_NORM = [(dict(rows=-1), INVAL), (dict(rows=(1 << 40) + 1), INVAL), (dict(cols=0), INVAL), (dict(cols=-3), INVAL),
            (dict(cols=(1 << 20) + 1), INVAL), (dict(ld_x=63), INVAL), (dict(ld_y=1), INVAL), (dict(ld_dy=-64), INVAL),
            (dict(ld_dx=(1 << 31) + 1), INVAL), (dict(x_dtype=2), UNSUP), (dict(p_dtype=-1), UNSUP),
            (dict(eps=-1e-9), INVAL), (dict(eps=math.nan), INVAL), (dict(eps=math.inf), INVAL),
            (dict(reserved=1), INVAL)]


@pytest.mark.parametrize("kw,code", BAD_NORM, ids=str)
def test_layer_norm_refuses_descriptors(lib, kw, code):
    d = ctypes.byref(norm_desc(**kw))
    assert lib.muon_layernorm_forward(d, P, P, P, 2 * P, P, P, None) == code
    assert _lib.last_error()
    assert lib.muon_layernorm_workspace_size(d) == 0
    assert lib.muon_layernorm_backward(d, P, P, P, P, P, 2 * P, P, P, P, 1 << 40, None) == code


def test_layer_norm_refuses_pointers(lib):
    d = ctypes.byref(norm_desc())
    fwd, bwd = lib.muon_layernorm_forward, lib.muon_layernorm_backward
    assert fwd(None, P, P, P, 2 * P, P, P, None) == INVAL
    good = [P, P, P, 2 * P, P, P]
    for i, bad in ((0, None), (3, None), (4, None), (5, None), (3, P), (0, P + 1), (1, P + 2), (2, P + 2),
                   (3, 2 * P + 1), (4, P + 2), (5, P + 1)):
        args = list(good)
        args[i] = bad
        assert fwd(d, *args, None) == INVAL, (i, bad)
    need = lib.muon_layernorm_workspace_size(d)
    good = [P, P, P, P, P, 2 * P, P, P, P, need]
    for i, bad, code in ((0, None, INVAL), (1, None, INVAL), (3, None, INVAL), (4, None, INVAL), (5, P, INVAL),
                         (0, P + 1, INVAL), (1, P + 1, INVAL), (2, P + 2, INVAL), (5, 2 * P + 1, INVAL),
                         (6, P + 2, INVAL), (7, P + 2, INVAL), (8, None, WORK), (8, P + 64, WORK), (9, 0, WORK),
                         (9, need // 4, WORK)):
        args = list(good)
        args[i] = bad
        assert bwd(d, *args, None) == code, (i, bad)
    assert bwd(d, P, P, P, P, P, None, None, None, P, need, None) == INVAL  # nothing wanted
    # no rows: nothing is launched, and no pointer is needed
    assert fwd(ctypes.byref(norm_desc(rows=0)), None, None, None, None, None, None, None) == 0


def test_layer_norm_without_rows_needs_nothing(lib):
    """The dx of an empty batch is an empty tensor, whose pointer is NULL: with no sums wanted there is nothing to do."""
    d = ctypes.byref(norm_desc(rows=0))
    assert lib.muon_layernorm_backward(d, *[None] * 9, 0, None) == 0
    assert lib.muon_layernorm_backward(d, *[None] * 6, P, None, None, 0, None) == WORK


@pytest.mark.parametrize("ld,apart", [(0, 2), (0, 128), (0, 7 * 128 + 126), (200, 2), (200, 126), (200, 400),
                                      (200, 400 - 126), (200, 6 * 400 + 274), (200, 7 * 400 + 126)])
def test_layer_norm_refuses_overlapping_rows(lib, ld, apart):
    """8 rows of 64 bf16 elements, an output `apart` bytes before or behind an input of the same leading dimension."""
    d = ctypes.byref(norm_desc(ld_x=ld, ld_y=ld, ld_dy=ld, ld_dx=ld))
    for off in (apart, -apart):
        assert lib.muon_layernorm_forward(d, P, P, P, P + off, P, P, None) == INVAL
        assert "overlap" in _lib.last_error()
        for dy, x in ((P, 8 * P), (8 * P, P)):
            assert lib.muon_layernorm_backward(d, dy, x, P, P, P, P + off, P, P, P, 1 << 40, None) == INVAL
            assert "overlap" in _lib.last_error()


def test_layer_norm_workspace_covers_every_kernel(lib):
    """One row of 2 cols sums for each block: a wave holds a row of up to 2048 elements, and at most 1024 blocks of
    four waves run."""
    for rows in (0, 1, 5, 1023, 1024, 5000, 1 << 33):
        for cols in (1, 64, 1001, 1 << 20):
            need = lib.muon_layernorm_workspace_size(ctypes.byref(norm_desc(rows=rows, cols=cols)))
            blocks = min((rows + 3) // 4 if cols <= 2048 else rows, 1024)
            assert max(blocks * 2 * cols * 4, 1) <= need <= blocks * 2 * cols * 4 + 1024


def attn_desc(**kw):
    d = dict(tokens=100, seqs=2, q_heads=4, kv_heads=2, head_dim=64, dtype=1, scale=0.125, reserved=0)
    d.update(kw)
    return AttentionDesc(*d.values())


def heads(n=4, base=P, dim=64, **kw):
    return Heads(kw.get("data", base), kw.get("token", n * dim), kw.get("head", dim))


BAD_ATTN = [(dict(tokens=-1), INVAL), (dict(tokens=1 << 31), INVAL), (dict(seqs=-1), INVAL),
            (dict(seqs=(1 << 24) + 1), INVAL), (dict(q_heads=0), INVAL), (dict(kv_heads=0), INVAL),
            (dict(kv_heads=3), INVAL), (dict(q_heads=2, kv_heads=4), INVAL), (dict(q_heads=1 << 17), INVAL),
            (dict(head_dim=0), UNSUP), (dict(head_dim=-8), UNSUP), (dict(head_dim=68), UNSUP),
            (dict(head_dim=136), UNSUP), (dict(dtype=2), UNSUP), (dict(scale=0.0), INVAL), (dict(scale=-1.0), INVAL),
            (dict(scale=math.nan), INVAL), (dict(scale=math.inf), INVAL), (dict(scale=2.0 ** -61), INVAL),
            (dict(scale=2.0 ** 61), INVAL), (dict(reserved=7), INVAL),
            (dict(tokens=1 << 30, q_heads=1 << 14, kv_heads=1 << 14), UNSUP)]


def attn_call(lib, d, back, flags=0, cu=P, lse=P, ws=P, ws_bytes=1 << 40, **over):
    h = {n: heads(2 if n in ("k", "v", "dk", "dv") else 4, P * (i + 1)) for i, n in
         enumerate(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))}
    h.update(over)
    r = {n: None if v is None else ctypes.byref(v) for n, v in h.items()}
    if back:
        return lib.muon_attention_backward(ctypes.byref(d), cu, r["dout"], r["q"], r["k"], r["v"], r["out"], lse,
                                           r["dq"], r["dk"], r["dv"], flags, ws, ws_bytes, None)
    return lib.muon_attention_forward(ctypes.byref(d), cu, r["q"], r["k"], r["v"], r["out"], lse, flags, None)


@pytest.mark.parametrize("kw,code", BAD_ATTN, ids=str)
def test_attention_refuses_descriptors(lib, kw, code):
    d = attn_desc(**kw)
    assert attn_call(lib, d, False) == code
    assert attn_call(lib, d, True) == code
    assert _lib.last_error()
    assert lib.muon_attention_workspace_size(ctypes.byref(d)) == 0


@pytest.mark.parametrize("kw", [dict(), dict(dtype=0), dict(dtype=0, head_dim=128), dict(head_dim=128)], ids=str)
def test_attention_refuses_what_one_launch_cannot_hold(lib, kw):
    """A launch has fewer than 2^32 threads: blocks of 256 for 128 query rows, or 512 for 64 (fp32, heads up to 64)."""
    rows, most = (64, (1 << 23) - 1) if kw == dict(dtype=0) else (128, (1 << 24) - 1)
    for heads_, seqs in ((40, 2), (1, 1000), (1, most // 2), (40, 0)):
        slots = most // heads_
        last = min((slots - seqs - 1) * rows + rows - 1, 0x7FFFFF00)
        ok, over = ({**kw, "tokens": t, "seqs": seqs, "q_heads": heads_, "kv_heads": heads_} for t in (last, last + 1))
        assert lib.muon_attention_workspace_size(ctypes.byref(attn_desc(**ok))) > 0
        if last < 0x7FFFFF00:
            d = attn_desc(**over)
            assert attn_call(lib, d, False) == UNSUP and attn_call(lib, d, True) == UNSUP
            assert lib.muon_attention_workspace_size(ctypes.byref(d)) == 0 and "launch" in _lib.last_error()
    d = attn_desc(**{**kw, "seqs": 1 << 24, "q_heads": 1, "kv_heads": 1})
    assert attn_call(lib, d, False) == UNSUP


@pytest.mark.parametrize("back", [False, True])
def test_attention_refuses_operands(lib, back):
    d = attn_desc()
    assert attn_call(lib, d, back, cu=None) == INVAL
    assert attn_call(lib, d, back, cu=P + 2) == INVAL
    assert attn_call(lib, d, back, lse=None) == INVAL
    assert attn_call(lib, d, back, lse=P + 1) == INVAL
    assert attn_call(lib, d, back, flags=8) == INVAL
    names = ("q", "k", "v", "out") + (("dout", "dq", "dk", "dv") if back else ())
    for n in names:
        w = 2 if n in ("k", "v", "dk", "dv") else 4
        for bad, code in ((None, INVAL), (heads(w, data=None), INVAL), (heads(w, data=P + 8), UNSUP),
                          (heads(w, token=w * 64 + 4), UNSUP), (heads(w, head=68), UNSUP),
                          (heads(w, token=-64), INVAL), (heads(w, head=-64), INVAL),
                          (heads(w, token=(1 << 24) + 8), INVAL), (heads(w, head=(1 << 31) + 8), INVAL)):
            assert attn_call(lib, d, back, **{n: bad}) == code, (n, bad)
    for n in (("dq", "dk", "dv") if back else ("out",)):  # rows of an output must not overlap
        w = 2 if n in ("dk", "dv") else 4
        for bad in (heads(w, token=64), heads(w, head=0), heads(w, token=0), heads(w, head=32, token=4096)):
            assert attn_call(lib, d, back, **{n: bad}) == INVAL, n
    if not back:
        for n in ("q", "k", "v"):
            assert attn_call(lib, d, False, out=heads(4, P * (1 + "qkv".index(n)))) == INVAL
        return
    for n in ("q", "dq"):
        assert attn_call(lib, d, True, dk=heads(2, P * (1 if n == "q" else 6))) == INVAL
    need = lib.muon_attention_workspace_size(ctypes.byref(d))
    assert attn_call(lib, d, True, ws=None) == WORK
    assert attn_call(lib, d, True, ws=P + 128) == WORK
    assert attn_call(lib, d, True, ws_bytes=need // 2) == WORK


def test_attention_without_tokens_needs_nothing(lib):
    d = attn_desc(tokens=0, seqs=0)
    assert attn_call(lib, d, False, cu=None, lse=None, q=None, out=None) == 0
    assert attn_call(lib, d, True, cu=None, lse=None, dq=None, ws=None, ws_bytes=0) == 0


def test_attention_workspace_holds_delta(lib):
    for tokens in (1, 1000, 1 << 20):
        for q, kv in ((12, 12), (16, 4), (32, 1)):
            need = lib.muon_attention_workspace_size(ctypes.byref(attn_desc(tokens=tokens, q_heads=q, kv_heads=kv)))
            assert need >= 2 * q * tokens * 4  # delta and lse of every query row
            assert need <= 2 * q * tokens * 4 + q * tokens * 2 * 64 * 4 + 1024  # and at most one partial per query head


def test_binding_refuses_tensors_before_any_call():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        block.layer_norm_forward(x)
    with pytest.raises(ValueError, match="device tensor"):
        block.layer_norm_backward(x, x, x[:, 0], x[:, 0])
    q = torch.zeros(4, 2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        block.packed_attention_forward(q, q, q, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        block.packed_attention_backward(q, q, q, q, q, q, torch.zeros(2, dtype=torch.int32))
    rows = block._rows
    assert rows(torch.zeros(3, 4, 8), "x") == (12, 8, 8)
    assert rows(torch.zeros(6, 20)[:, :8], "x") == (6, 8, 20)
    assert rows(torch.zeros(1, 1, 8), "x") == (1, 8, 8)
    assert rows(torch.zeros(8), "x") == (1, 8, 8)
    assert rows(torch.zeros(0, 8), "x")[:2] == (0, 8)
    for bad in (torch.zeros(8, 3).t(), torch.zeros(3, 5, 8).transpose(0, 1), torch.zeros(1, 8).expand(4, 8),
                torch.tensor(1.0)):
        with pytest.raises(ValueError):
            rows(bad, "x")


def test_binding_refuses_given_outputs_where_gradients_are_recorded():
    """Before anything else: writing into a given tensor would lose the gradients without a word."""
    x, y = torch.zeros(4, 8, requires_grad=True), torch.zeros(4, 8)
    q, cu = torch.zeros(4, 2, 8, requires_grad=True), torch.zeros(2, dtype=torch.int32)
    calls = [lambda: block.layer_norm_forward(x, out=y), lambda: block.layer_norm_forward(y, x[0], out=y),
             lambda: block.packed_attention_forward(q, y, y, cu, out=y),
             lambda: block.packed_attention_forward(y, y, q, cu, lse=y)]
    for call in calls:
        with pytest.raises(ValueError, match="recorded"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            call()


# ------------------------------------------------- the reference's own pins --
def test_reference_gradients_against_differences():
    """The fp64 formulas' gradients equal autograd's, and central differences, on the CPU."""
    torch.manual_seed(0)
    lengths, H, G, D = [5, 0, 1, 9], 4, 2, 8
    T = sum(lengths)
    q, k, v, do = (torch.randn(T, n, D, dtype=torch.float64) for n in (H, G, G, H))
    ref = R.attention(q, k, v, lengths, 0.3, do, dtype=torch.float32)

    def loss(q, k, v):
        return (R.attention(q, k, v, lengths, 0.3)["out"][0] * do).sum()

    for name, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        args = [q, k, v]
        d = torch.randn_like(args[i])
        h = 1e-5
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * d, args[i] + h * d
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - (ref[name][0] * d).sum()) < 1e-8
    x, w, b, dy = torch.randn(6, 10).double(), torch.randn(10).double(), torch.randn(10).double(), torch.randn(6, 10).double()
    for t in (x, w, b):
        t.requires_grad_(True)
    (torch.nn.functional.layer_norm(x, (10,), w, b, 1e-5) * dy).sum().backward()
    for got, t in zip(R.norm_backward(dy, x.detach(), w.detach(), 1e-5), (x, w, b)):
        assert (got - t.grad).abs().max() < 1e-12


def test_reference_check_sees_a_wrong_value():
    """A mistake planted in the reference is outside the bounds (a sequence border one token off, a wrong group)."""
    torch.manual_seed(1)
    q, k, v = (torch.randn(40, n, 16) for n in (4, 2, 2))
    good = R.attention(q, k, v, [17, 23], 0.25, q, dtype=torch.bfloat16)
    for other in (R.attention(q, k, v, [18, 22], 0.25, q), R.attention(q, k.flip(1), v, [17, 23], 0.25, q),
                  R.attention(q, k, v, [17, 23], 0.26, q)):
        for name in ("out", "lse", "dq", "dk", "dv"):
            with pytest.raises(AssertionError):
                R.check(name, other[name][0], *good[name])


# --------------------------------------------------- operands that share memory --
Q = 1 << 20  # apart from P by more than any operand below


def test_layer_norm_refuses_outputs_that_share_memory(lib):
    """Statistics, parameter gradients and the workspace too, and rows of different steps."""
    d = norm_desc()  # 8 rows of 64 bf16: 1024 bytes; fp32 parameters: 256 bytes
    fwd = dict(x=P, weight=P + Q, bias=P + 2 * Q, y=P + 3 * Q, mean=P + 4 * Q, rstd=P + 5 * Q)
    for over in (dict(mean=P + 1020), dict(rstd=P + Q + 252), dict(mean=P + 3 * Q), dict(rstd=P + 4 * Q + 28),
                 dict(y=P + 2 * Q + 254), dict(mean=P + 2 * Q - 28), dict(y=P + 5 * Q - 1022)):
        args = {**fwd, **over}
        assert lib.muon_layernorm_forward(ctypes.byref(d), *args.values(), None) == INVAL, over
        assert "overlap" in _lib.last_error()
    strided = norm_desc(ld_x=128, ld_y=64)
    for y in (P + 128, P - 512, P + 7 * 256 + 126):
        assert lib.muon_layernorm_forward(ctypes.byref(strided), *{**fwd, "y": y}.values(), None) == INVAL
        assert "overlap" in _lib.last_error()
    need = lib.muon_layernorm_workspace_size(ctypes.byref(d))
    bwd = dict(dy=P, x=P + Q, weight=P + 2 * Q, mean=P + 3 * Q, rstd=P + 4 * Q, dx=P + 5 * Q, dw=P + 6 * Q,
               db=P + 7 * Q, ws=P + 8 * Q)
    for over in (dict(dw=P), dict(db=P + Q + 1020), dict(dw=P + 7 * Q + 252), dict(dx=P + 6 * Q), dict(db=P + 3 * Q),
                 dict(dw=P + 4 * Q + 28), dict(ws=P), dict(ws=P + 7 * Q), dict(ws=P + 5 * Q), dict(dx=P + 2 * Q),
                 dict(dx=P + 3 * Q - 1020), dict(ws=P + 4 * Q)):
        args = {**bwd, **over}
        assert lib.muon_layernorm_backward(ctypes.byref(d), *args.values(), need, None) == INVAL, over
        assert "overlap" in _lib.last_error()


def test_layer_norm_refuses_rows_past_any_memory(lib):
    assert lib.muon_layernorm_workspace_size(ctypes.byref(norm_desc(rows=1 << 40, ld_dy=1 << 31))) == 0
    assert "exceed" in _lib.last_error()


# (token stride, head stride, bytes from the first operand's start to the second's) for 100 tokens, 4 heads, 64 bf16
FUSED = 12 * 64  # one buffer of (100, 12, 64)
SHARED = [(FUSED, 64, 3 * 128), (FUSED, 64, -3 * 128), (FUSED, 64, 99 * FUSED * 2 + 3 * 128),
          (FUSED, 64, 9 * 128),  # its last head is the first head of the next token
          (FUSED, 192, 128 - 16), (FUSED, 192, 3 * 128), (64, 6400, 16), (64, 6400, 3 * 12800 + 99 * 128),
          (64, 6400, -12800), (64, 6400, 12800 - 128)]


@pytest.mark.parametrize("token,head,apart", SHARED, ids=str)
def test_attention_refuses_outputs_inside_other_operands(lib, token, head, apart):
    d = attn_desc(kv_heads=4)
    far = {n: heads(4, P + (10 + i) * Q, token=token, head=head) for i, n in
           enumerate(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))}
    far.update(cu=P, lse=P + Q, ws=P + 64 * Q)
    for other in ("q", "k", "v"):
        over = {**far, "out": heads(4, far[other].data + apart, token=token, head=head)}
        assert attn_call(lib, d, False, **over) == INVAL, other
        assert "overlap" in _lib.last_error()
    for mine in ("dq", "dk", "dv"):
        for other in set(("q", "k", "v", "out", "dout", "dq", "dk", "dv")) - {mine}:
            over = {**far, mine: heads(4, far[other].data + apart, token=token, head=head)}
            assert attn_call(lib, d, True, **over) == INVAL, (mine, other)
            assert "overlap" in _lib.last_error()


def test_attention_refuses_outputs_of_other_strides_and_flat_buffers(lib):
    d = attn_desc(kv_heads=4)
    far = {n: heads(4, P + (10 + i) * Q, token=FUSED) for i, n in
           enumerate(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))}
    far.update(cu=P, lse=P + Q, ws=P + 64 * Q)
    q, out, dq = far["q"].data, far["out"].data, far["dq"].data
    for over in (dict(out=heads(4, q + 512, token=256)), dict(out=heads(4, q + 128, token=FUSED, head=128)),
                 dict(lse=q), dict(lse=out + 99 * FUSED * 2), dict(lse=P - 1596), dict(cu=P + Q + 1596),
                 dict(cu=out + 3 * 128), dict(out=heads(4, P - 16, token=FUSED))):
        assert attn_call(lib, d, False, **{**far, **over}) == INVAL, over
        assert "overlap" in _lib.last_error()
    for over in (dict(ws=q + 256), dict(ws=dq), dict(ws=P + Q), dict(dq=heads(4, P - 128, token=FUSED)),
                 dict(dk=heads(4, P + Q, token=FUSED)), dict(dv=heads(4, q + 512, token=256))):
        assert attn_call(lib, d, True, **{**far, **over}) == INVAL, over
        assert "overlap" in _lib.last_error()


# ------------------------------------------------------------ the sources --
def test_every_barrier_before_a_tile_is_overwritten_waits_for_lds_reads():
    """A copy into a tile may only start when every wave's reads of it have returned.  The compiler orders its LDS
    reads before an assembly barrier, not their return, so each such barrier has to wait for them itself."""
    path = os.path.join(os.path.dirname(_lib.LIB_PATH), "csrc", "attention.hip")
    with open(path) as f:
        barriers = [line for line in f if "asm" in line and "s_barrier" in line]
    assert len(barriers) >= 2
    for line in barriers:
        assert "lgkmcnt(0)" in line.split("s_barrier")[0], line
