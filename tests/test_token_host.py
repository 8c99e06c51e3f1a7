"""The embedding's and the query/key norm's C ABI and binding on the host (no GPU): refusals, workspaces, pins.

Every call here is rejected by argument checks before any HIP call, or is host-only.
"""
import copy
import ctypes
import math
import os
import pickle

import pytest
import torch

import block_reference as B
import muon_newton_schulz_03_amd as pkg
import token_reference as R
from muon_newton_schulz_03_amd import _lib
from muon_newton_schulz_03_amd._lib import EmbeddingDesc, Heads, QkNormDesc, RotationDesc

INVAL, UNSUP, WORK = _lib.MUON_E_INVAL, _lib.MUON_E_UNSUPPORTED, _lib.MUON_E_WORKSPACE
P = 0x10000  # a pointer that no call follows
Q = 1 << 20  # apart from P by more than any operand below


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from muon_newton_schulz_03_amd.build import build_library
        build_library()
    return _lib.load()


# ---------------------------------------------------- query and key norms --
def qk_desc(**kw):
    d = dict(tokens=100, seqs=2, q_heads=4, k_heads=2, head_dim=64, dtype=1, p_dtype=0, position_dtype=0, eps=1e-6,
             reserved=0)
    d.update(kw)
    return QkNormDesc(*d.values())


def rotation(dim=64, pairs=0, freqs=None):
    f = freqs if freqs is not None else [0.5] * (dim // 2)
    r = RotationDesc((ctypes.c_double * max(1, len(f)))(*f), dim, pairs)
    return r


def heads(n, at, dim=64, **kw):
    return Heads(kw.get("data", at), kw.get("token", n * dim), kw.get("head", dim))


def qk_call(lib, d, back, rot=None, cu=P, pos=P + Q, qw=P + 2 * Q, kw=P + 3 * Q, dqw=P + 4 * Q, dkw=P + 5 * Q, flags=0,
            ws=P + 6 * Q, ws_bytes=1 << 40, **over):
    h = {n: heads(2 if "k" in n else 4, P + (16 + i) * Q) for i, n in
         enumerate(("q", "k", "yq", "yk", "gq", "gk"))}
    h.update(over)
    r = {n: None if v is None else ctypes.byref(v) for n, v in h.items()}
    ro = None if rot is None else ctypes.byref(rot)
    if back:
        return lib.muon_qk_norm_backward(ctypes.byref(d), ro, cu, pos, r["gq"], r["gk"], r["q"], r["k"], qw, kw, r["yq"],
                                         r["yk"], dqw, dkw, flags, ws, ws_bytes, None)
    return lib.muon_qk_norm_forward(ctypes.byref(d), ro, cu, pos, r["q"], r["k"], qw, kw, r["yq"], r["yk"], flags, None)


BAD_QK = [(dict(tokens=-1), INVAL), (dict(tokens=1 << 31), INVAL), (dict(seqs=-1), INVAL),
          (dict(seqs=(1 << 24) + 1), INVAL), (dict(q_heads=0), INVAL), (dict(k_heads=0), INVAL),
          (dict(q_heads=(1 << 16) + 1), INVAL), (dict(k_heads=1 << 17), INVAL), (dict(head_dim=0), UNSUP),
          (dict(head_dim=68), UNSUP), (dict(head_dim=136), UNSUP), (dict(head_dim=-8), UNSUP), (dict(dtype=2), UNSUP),
          (dict(p_dtype=-1), UNSUP), (dict(position_dtype=2), UNSUP), (dict(eps=-1e-9), INVAL),
          (dict(eps=math.nan), INVAL), (dict(eps=math.inf), INVAL), (dict(reserved=1), INVAL)]


@pytest.mark.parametrize("kw,code", BAD_QK, ids=str)
def test_qk_norm_refuses_descriptors(lib, kw, code):
    d = qk_desc(**kw)
    assert qk_call(lib, d, False) == code and qk_call(lib, d, True) == code
    assert _lib.last_error()
    assert lib.muon_qk_norm_workspace_size(ctypes.byref(d)) == 0
    assert lib.muon_qk_norm_forward(None, *[None] * 9, 0, None) == INVAL


@pytest.mark.parametrize("rot,code", [
    (dict(dim=-8, freqs=[]), UNSUP), (dict(dim=72), UNSUP), (dict(dim=12), UNSUP), (dict(pairs=2), INVAL),
    (dict(pairs=-1), INVAL), (dict(dim=8, freqs=[0, 1, math.nan, 0]), INVAL), (dict(dim=8, freqs=[0, 1, 0, 65]), INVAL),
    (dict(dim=8, freqs=[-math.inf, 1, 0, 0]), INVAL)], ids=str)
def test_qk_norm_refuses_rotations(lib, rot, code):
    for back in (False, True):
        assert qk_call(lib, qk_desc(), back, rot=rotation(**rot)) == code
        assert _lib.last_error()
        null = RotationDesc(None, 8, 0)
        assert qk_call(lib, qk_desc(), back, rot=null) == INVAL


@pytest.mark.parametrize("back", [False, True])
def test_qk_norm_refuses_operands(lib, back):
    d = qk_desc()
    for over, code in ((dict(cu=P + 2), INVAL), (dict(pos=P + 2), INVAL), (dict(qw=P + 2), INVAL), (dict(kw=P + 1), INVAL),
                       (dict(flags=4), INVAL)):
        assert qk_call(lib, d, back, **over) == code, over
    assert qk_call(lib, qk_desc(position_dtype=1), back, pos=P + Q + 4) == INVAL
    for n in ("q", "k", "yq", "yk") + (("gq", "gk") if back else ()):
        w = 2 if "k" in n else 4
        for bad, code in ((None, INVAL), (heads(w, P, data=None), INVAL), (heads(w, P + 8), UNSUP),
                          (heads(w, P, token=w * 64 + 4), UNSUP), (heads(w, P, head=68), UNSUP),
                          (heads(w, P, token=-64), INVAL), (heads(w, P, head=-64), INVAL),
                          (heads(w, P, token=(1 << 24) + 8), INVAL), (heads(w, P, head=(1 << 31) + 8), INVAL)):
            assert qk_call(lib, d, back, **{n: bad}) == code, (n, bad)
    for n in ("yq", "yk"):  # rows of an output must not overlap
        w = 2 if "k" in n else 4
        for bad in (heads(w, P, token=64), heads(w, P, head=0), heads(w, P, token=0), heads(w, P, head=32, token=4096)):
            assert qk_call(lib, d, back, **{n: bad}) == INVAL, n
    if back:
        need = lib.muon_qk_norm_workspace_size(ctypes.byref(d))
        for over, code in ((dict(ws=None), WORK), (dict(ws=P + 128), WORK), (dict(ws_bytes=need // 2), WORK),
                           (dict(dqw=P + 2), INVAL), (dict(dkw=P + 1), INVAL)):
            assert qk_call(lib, d, back, **over) == code, over


@pytest.mark.parametrize("back", [False, True])
def test_qk_norm_refuses_outputs_that_share_memory(lib, back):
    d = qk_desc()
    fused = 8 * 64
    inputs = ("q", "k") + (("gq", "gk") if back else ())
    base = {n: heads(1, P + (16 + i) * Q, token=fused) for i, n in enumerate(("q", "k", "yq", "yk", "gq", "gk"))}
    for mine in ("yq", "yk"):
        for other in inputs + tuple({"yq", "yk"} - {mine}):
            for apart in (0, 128, -128, 99 * fused * 2, 16):
                over = {**base, mine: heads(1, base[other].data + apart, token=fused)}
                assert qk_call(lib, d, back, **over) == INVAL, (mine, other, apart)
                assert "overlap" in _lib.last_error()
        for flat in (P, P + Q, P + 2 * Q, P + 3 * Q) + ((P + 4 * Q, P + 5 * Q, P + 6 * Q) if back else ()):
            assert qk_call(lib, d, back, **{**base, mine: heads(1, flat, token=fused)}) == INVAL, (mine, flat)
    if back:
        for over in (dict(dqw=P + 5 * Q + 252), dict(dkw=P + 2 * Q), dict(dqw=P + 16 * Q), dict(ws=P + 18 * Q),
                     dict(ws=P), dict(dkw=P + Q + 396), dict(ws=P + 20 * Q)):
            assert qk_call(lib, d, True, **{**base, **over}) == INVAL, over
            assert "overlap" in _lib.last_error()


def test_qk_norm_without_tokens_needs_nothing(lib):
    d = qk_desc(tokens=0)
    none = dict(cu=None, pos=None, q=None, k=None, yq=None, yk=None, gq=None, gk=None)
    assert qk_call(lib, d, False, **none) == 0
    assert qk_call(lib, d, True, dqw=None, dkw=None, ws=None, ws_bytes=0, **none) == 0
    assert qk_call(lib, d, True, ws=None, ws_bytes=0, **none) == WORK


def test_qk_norm_workspace(lib):
    for dim in (8, 64, 128):
        need = lib.muon_qk_norm_workspace_size(ctypes.byref(qk_desc(head_dim=dim)))
        assert 2 * 1024 * dim * 4 <= need <= 2 * 1024 * dim * 4 + 512  # a row for each block of both sides


def test_rotation_arguments():
    r = pkg.Rotation(16, 100.0)
    assert r.frequencies == tuple(100.0 ** (-i / 8) for i in range(8)) and r.pairs == "halves"
    assert pkg.Rotation(8, frequencies=torch.zeros(4)).frequencies == (0.0,) * 4
    assert pkg.Rotation(0).frequencies == ()
    for again in (copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert (again.dim, again.frequencies, again.pairs) == (r.dim, r.frequencies, r.pairs)
        assert again._desc.dim == 16 and again._desc.frequencies[1] == r.frequencies[1]
    for bad in (dict(dim=12), dict(dim=-8), dict(dim=8, pairs="both"), dict(dim=8, frequencies=[1.0]),
                dict(dim=8, base=0.0), dict(dim=8, base=-2.0)):
        with pytest.raises(ValueError):
            pkg.Rotation(**bad)


# -------------------------------------------------------------- embedding --
def embed_desc(**kw):
    d = dict(tokens=10, vocab=20, cols=64, ld_table=0, ld_out=0, table_dtype=1, out_dtype=1, id_dtype=1, scale=1.0,
             reserved=0)
    d.update(kw)
    return EmbeddingDesc(*d.values())


def embed_call(lib, d, back, ids=P, a=P + Q, out=P + 2 * Q, flags=0, ws=P + 3 * Q, ws_bytes=1 << 40):
    if back:
        return lib.muon_embedding_backward(ctypes.byref(d), ids, a, out, flags, ws, ws_bytes, None)
    return lib.muon_embedding_forward(ctypes.byref(d), ids, a, out, None)


BAD_EMBED = [(dict(tokens=-1), INVAL), (dict(tokens=(1 << 30) + 1), INVAL), (dict(vocab=0), INVAL),
             (dict(vocab=-5), INVAL), (dict(vocab=1 << 30), INVAL), (dict(cols=0), INVAL), (dict(cols=(1 << 20) + 1), INVAL),
             (dict(ld_table=63), INVAL), (dict(ld_out=-64), INVAL), (dict(ld_out=(1 << 31) + 1), INVAL),
             (dict(table_dtype=2), UNSUP), (dict(out_dtype=-1), UNSUP), (dict(id_dtype=2), UNSUP),
             (dict(scale=math.nan), INVAL), (dict(scale=-math.inf), INVAL), (dict(reserved=3), INVAL)]


@pytest.mark.parametrize("kw,code", BAD_EMBED, ids=str)
def test_embedding_refuses_descriptors(lib, kw, code):
    d = embed_desc(**kw)
    assert embed_call(lib, d, False) == code and embed_call(lib, d, True) == code
    assert _lib.last_error()
    assert lib.muon_embedding_workspace_size(ctypes.byref(d)) == 0
    assert lib.muon_embedding_forward(None, P, P, P, None) == INVAL


def test_embedding_refuses_pointers(lib):
    d = embed_desc()
    for over in (dict(ids=None), dict(a=None), dict(out=None), dict(ids=P + 4), dict(a=P + Q + 1), dict(out=P + 1)):
        assert embed_call(lib, d, False, **over) == INVAL, over
        assert embed_call(lib, d, True, **over) == INVAL, over
    need = lib.muon_embedding_workspace_size(ctypes.byref(d))
    for over, code in ((dict(flags=2), INVAL), (dict(ws=None), WORK), (dict(ws=P + 64), WORK),
                       (dict(ws_bytes=need // 2), WORK)):
        assert embed_call(lib, d, True, **over) == code, over
    assert embed_call(lib, embed_desc(tokens=0), False, ids=None, a=None, out=None) == 0
    assert embed_call(lib, embed_desc(tokens=0), True, ids=None, a=None, out=None, ws=None, flags=1) == 0
    assert embed_call(lib, embed_desc(tokens=0), True, ids=None, a=None, out=None) == INVAL


def test_embedding_refuses_outputs_that_share_memory(lib):
    d = embed_desc()  # 10 ids of 8 bytes, rows of 128 bytes: 20 in the table, 10 out
    for over in (dict(out=P), dict(out=P + 78), dict(out=P - 1278), dict(out=P + Q), dict(out=P + Q + 2558),
                 dict(out=P + Q - 1278)):
        assert embed_call(lib, d, False, **over) == INVAL, over
        assert "overlap" in _lib.last_error()
    for over in (dict(out=P), dict(out=P + Q + 1278), dict(out=P + Q - 2558), dict(ws=P), dict(ws=P + Q),
                 dict(ws=P + 2 * Q), dict(out=P + 3 * Q)):
        assert embed_call(lib, d, True, **over) == INVAL, over
        assert "overlap" in _lib.last_error()


def test_binding_refuses_tensors_before_any_call():
    t, ids = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    q = torch.zeros(4, 2, 8)
    for call in (lambda: pkg.embedding_forward(t, ids), lambda: pkg.embedding_backward(t, ids, 4),
                 lambda: pkg.qk_norm_forward(q, q), lambda: pkg.qk_norm_backward(q, q, q, q)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    g, w = t.clone().requires_grad_(True), torch.zeros(8, requires_grad=True)
    qg = q.clone().requires_grad_(True)
    for call in (lambda: pkg.embedding_forward(g, ids, out=t), lambda: pkg.qk_norm_forward(qg, q, q_out=q),
                 lambda: pkg.qk_norm_forward(q, qg, k_out=q), lambda: pkg.qk_norm_forward(q, q, q_weight=w, k_out=q),
                 lambda: pkg.qk_norm_forward(q, q, k_weight=w, q_out=q)):
        with pytest.raises(ValueError, match="recorded"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
            call()


# ------------------------------------------------- the reference's own pins --
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dim", [0, 8, 16])
def test_reference_gradients_against_differences(pairs, dim):
    """The formulas' gradients equal autograd's and central differences; a turn keeps every head's length."""
    torch.manual_seed(0)
    x, dy = torch.randn(6, 3, 16).double(), torch.randn(6, 3, 16).double()
    w = torch.randn(16).double()
    turns = R.angles([0, 1, 5, -3, 1 << 20, 17], [0.3, 1.0, 0.01, 2.0, 0.7, 0.1, 3.0, 0.2][:dim // 2])
    ref = R.qk_norm(x, w, turns, dim, pairs, 1e-3, dy)

    def loss(x, w):
        return (R.qk_norm(x, w, turns, dim, pairs, 1e-3)["y"][0] * dy).sum()

    xg, wg = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss(xg, wg).backward()
    assert (xg.grad - ref["dx"][0]).abs().max() < 1e-12 and (wg.grad - ref["dw"][0]).abs().max() < 1e-11
    d, h = torch.randn_like(x), 1e-6
    assert abs((loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h) - (ref["dx"][0] * d).sum()) < 1e-6
    y, _ = R.qk_norm(x, None, turns, dim, pairs, 0.0)["y"]
    assert (y.pow(2).mean(2) - 1).abs().max() < 1e-12


def test_reference_turns_depend_on_distance_only():
    """Products of turned queries and keys depend on the difference of their positions."""
    torch.manual_seed(1)
    q, k = torch.randn(1, 1, 16).double(), torch.randn(1, 1, 16).double()
    f = [1.0, 0.3, 0.1, 0.03, 0.01, 0.003, 0.001, 0.0003]
    for pairs in ("halves", "neighbours"):
        def dot(a, b):
            (ca, sa, _), (cb, sb, _) = R.angles([a], f), R.angles([b], f)
            return (R.turn(q, ca, sa, 16, pairs) * R.turn(k, cb, sb, 16, pairs)).sum()
        assert abs(dot(100, 93) - dot(7, 0)) < 1e-12 and abs(dot(100, 93) - dot(7, 1)) > 1e-3


def test_reference_check_sees_a_wrong_value():
    """Mistakes planted in the reference are outside its bounds, in bf16 too."""
    torch.manual_seed(2)
    x, dy, w = torch.randn(30, 2, 16).bfloat16(), torch.randn(30, 2, 16).bfloat16(), torch.randn(16)
    f = [0.9 ** i for i in range(8)]
    pos = list(range(30))
    good = R.qk_norm(x, w, R.angles(pos, f), 16, "halves", 1e-6, dy)
    wrong = [R.qk_norm(x, w, R.angles([p + 1 for p in pos], f), 16, "halves", 1e-6, dy),
             R.qk_norm(x, w, R.angles([-p for p in pos], f), 16, "halves", 1e-6, dy),
             R.qk_norm(x, w, R.angles(pos, f), 16, "neighbours", 1e-6, dy),
             R.qk_norm(x, w, R.angles(pos, f), 16, "halves", 0.1, dy)]
    for other in wrong:
        for name in ("y", "dx", "dw"):
            with pytest.raises(AssertionError):
                B.check(name, other[name][0], *good[name])
    table, ids, do = torch.randn(9, 16), torch.randint(0, 9, (50,)), torch.randn(50, 16)
    good = R.embedding(table, ids, 1.5, torch.bfloat16, do, torch.bfloat16)
    for other in (R.embedding(table, ids.roll(1), 1.5, torch.bfloat16, do, torch.bfloat16),
                  R.embedding(table, ids, 1.52, torch.bfloat16, do, torch.bfloat16)):
        for name in ("out", "dtable"):
            with pytest.raises(AssertionError):
                B.check(name, other[name][0], *good[name])


def test_reference_embedding_against_autograd():
    torch.manual_seed(3)
    table, ids, do = torch.randn(7, 5).double().requires_grad_(True), torch.tensor([3, 3, 0, 6, -1, 7, 3]), torch.randn(7, 5)
    ref = R.embedding(table.detach(), ids, 0.5, torch.float32, do, torch.float32)
    known = (ids >= 0) & (ids < 7)
    out = torch.where(known[:, None], 0.5 * table[ids.clamp(0, 6)], 0.0)
    (out * do).sum().backward()
    assert (out.detach() - ref["out"][0]).abs().max() == 0 and (table.grad - ref["dtable"][0]).abs().max() < 1e-12
