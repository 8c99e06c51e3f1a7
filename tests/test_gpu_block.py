"""Layer norm and packed causal attention on the GPU against their fp64 definitions.

Tolerances are the elementwise bounds of block_reference (derived from the
roundings of the computation); sizes are those at which tiles, vectors and
sequences end badly.
"""
import itertools

import pytest
import torch

import block_reference as R
import muon_newton_schulz_03_amd as lib
from muon_harness import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


# -------------------------------------------------------------- layer norm --
def norm_case(x, w, b, dy, eps=1e-5):
    dev = [None if t is None else t.to(DEV) for t in (x, w, b, dy)]
    y, mean, rstd = lib.layer_norm_forward(dev[0], dev[1], dev[2], eps=eps)
    dx, dw, db = lib.layer_norm_backward(dev[3], dev[0], mean, rstd, dev[1])
    torch.cuda.synchronize()
    ry, rm, rr = R.norm_forward(x, w, b, eps)
    rdx, rdw, rdb = R.norm_backward(dy, x, w, eps)
    bound = R.norm_bounds(dy, x, w, b, eps)
    worst = 0.0
    for name, got, ref in (("y", y, ry), ("mean", mean, rm), ("rstd", rstd, rr), ("dx", dx, rdx), ("dw", dw, rdw),
                           ("db", db, rdb)):
        worst = max(worst, R.check(name, got, ref, bound[name]))
    return worst


NORM_COLS = [1, 7, 8, 64, 100, 513, 768, 1001, 1024, 2048, 2056, 2500, 4096, 4100, 8192, 8200, 20000]


@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("cols", NORM_COLS)
def test_layer_norm(cols, dtype, pdtype):
    rows = 37
    say(f"[gpu] layer norm {rows}x{cols} {dtype} params {pdtype}")
    x = randn((rows, cols), 1, dtype, 2.0) + randn((rows, 1), 2).to(dtype)
    worst = norm_case(x, (1 + randn((cols,), 3, std=0.2)).to(pdtype), randn((cols,), 4, pdtype),
                      randn((rows, cols), 5, dtype))
    say(f"[gpu]   worst error {worst:.3f} of its bound")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 1023, 4099, 9000])
@pytest.mark.parametrize("cols", [64, 768, 2304])
def test_layer_norm_rows(rows, cols):
    x = randn((rows, cols), 11, BF)
    norm_case(x, None, None, randn((rows, cols), 12, BF))


@pytest.mark.parametrize("dtype,rows,cols", [(BF, 9001, 520), (BF, 8203, 1536), (BF, 8195, 770), (F32, 8201, 1024),
                                             (BF, 2561, 4096), (BF, 2051, 6000), (F32, 2053, 2309)])
def test_layer_norm_rows_in_turn(dtype, rows, cols):
    """More rows than the launch holds at once, with parameters: each thread takes several."""
    say(f"[gpu] layer norm {rows}x{cols} {dtype}")
    norm_case(randn((rows, cols), 13, dtype), 1 + randn((cols,), 14, std=0.2), randn((cols,), 15),
              randn((rows, cols), 16, dtype))


def test_layer_norm_between_columns_of_one_buffer():
    """Input and output interleaved row by row: the same bits as in separate buffers, nothing else written."""
    rows, cols = 9000, 128
    buf = randn((rows, 3 * cols), 17, BF).to(DEV)
    x, dy = buf[:, :cols], buf[:, 2 * cols:]
    y, mean, rstd = lib.layer_norm_forward(x.contiguous())
    dx, _, _ = lib.layer_norm_backward(dy.contiguous(), x.contiguous(), mean, rstd)
    keep = buf.clone()
    lib.layer_norm_forward(x, out=buf[:, cols:2 * cols])
    assert torch.equal(buf[:, cols:2 * cols], y)
    lib.layer_norm_backward(dy, x, mean, rstd, dx=buf[:, cols:2 * cols])
    assert torch.equal(buf[:, cols:2 * cols], dx)
    assert torch.equal(buf[:, :cols], keep[:, :cols]) and torch.equal(buf[:, 2 * cols:], keep[:, 2 * cols:])


def test_layer_norm_offset_and_constant_rows():
    """A large common offset must not cancel the variance; a constant row has rstd 1 / sqrt(eps)."""
    x = randn((16, 768), 21) + 1000.0
    x[3] = 7.0
    x[4] = 0.0
    norm_case(x, 1 + randn((768,), 22, std=0.1), randn((768,), 23), randn((16, 768), 24), eps=1e-3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_layer_norm_strided_and_unaligned(dtype):
    """Rows of a wider buffer, starting on and off 16-byte boundaries; (a, b, cols) inputs; outputs given."""
    cols = 768
    for off, ld in ((0, 2304), (1, 1000), (8, 1001)):
        buf = randn((33, ld), 31, dtype)
        x = buf[:, off:off + cols] if off + cols <= ld else buf[:, :cols]
        w, b, dy = randn((cols,), 32), randn((cols,), 33), randn((33, cols), 34, dtype)
        xd = buf.to(DEV)[:, off:off + cols]
        outbuf = torch.full((33, ld), 5.0, dtype=dtype, device=DEV)
        y, mean, rstd = lib.layer_norm_forward(xd, w.to(DEV), b.to(DEV), out=outbuf[:, off:off + cols])
        dxbuf = torch.full((33, ld), 5.0, dtype=dtype, device=DEV)
        dx, dw, db = lib.layer_norm_backward(dy.to(DEV), xd, mean, rstd, w.to(DEV), dx=dxbuf[:, off:off + cols])
        bound = R.norm_bounds(dy, x, w, b, 1e-5)
        R.check("y", y, R.norm_forward(x, w, b, 1e-5)[0], bound["y"])
        for name, got, ref in zip(("dx", "dw", "db"), (dx, dw, db), R.norm_backward(dy, x, w, 1e-5)):
            R.check(name, got, ref, bound[name])
        for o in (outbuf, dxbuf):  # nothing outside the views was written
            assert (o[:, :off] == 5).all() and (o[:, off + cols:] == 5).all()
    x3 = randn((3, 5, cols), 35, dtype)
    y, mean, rstd = lib.layer_norm_forward(x3.to(DEV))
    assert y.shape == x3.shape and mean.shape == (3, 5)
    R.check("y3", y.reshape(15, cols), R.norm_forward(x3.reshape(15, cols), None, None, 1e-5)[0],
            R.norm_bounds(None, x3.reshape(15, cols), None, None, 1e-5)["y"])


def test_layer_norm_optional_gradients_and_no_rows():
    x, dy = randn((9, 96), 41).to(DEV), randn((9, 96), 42).to(DEV)
    _, mean, rstd = lib.layer_norm_forward(x)
    dx, dw, db = lib.layer_norm_backward(dy, x, mean, rstd)
    for nw, nb in itertools.product((False, True), repeat=2):
        dx2, dw2, db2 = lib.layer_norm_backward(dy, x, mean, rstd, need_weight=nw, need_bias=nb)
        assert torch.equal(dx, dx2)
        assert (dw2 is None) == (not nw) and (db2 is None) == (not nb)
        assert dw2 is None or torch.equal(dw, dw2)
        assert db2 is None or torch.equal(db, db2)
    e = torch.empty(0, 96, device=DEV)
    y, m, r = lib.layer_norm_forward(e)
    dx, dw, db = lib.layer_norm_backward(e, e.clone(), m, r)
    assert y.shape == (0, 96) and dx.shape == (0, 96) and (dw == 0).all() and (db == 0).all()


def test_layer_norm_nan_stays_in_its_row():
    x = randn((40, 768), 51, BF)
    x[7, 3] = float("nan")
    x[9, 0] = float("inf")
    y, _, _ = lib.layer_norm_forward(x.to(DEV))
    bad = (~torch.isfinite(y.float())).any(1).cpu()
    assert bad[7] and bad[9] and bad.sum() == 2


def test_layer_norm_offsets_past_32_bits():
    """Rows 2^31 bytes apart: element offsets pass 32 bits."""
    ld, rows, cols = (1 << 30), 5, 768
    buf = torch.empty((rows - 1) * ld + cols, dtype=BF, device=DEV)
    x = torch.as_strided(buf, (rows, cols), (ld, 1))
    src = randn((rows, cols), 61, BF)
    x.copy_(src)
    y, mean, rstd = lib.layer_norm_forward(x)
    dx, _, _ = lib.layer_norm_backward(src.to(DEV), x, mean, rstd)
    bound = R.norm_bounds(src, src, None, None, 1e-5)
    R.check("y", y, R.norm_forward(src, None, None, 1e-5)[0], bound["y"])
    R.check("dx", dx, R.norm_backward(src, src, None, 1e-5)[0], bound["dx"])


# --------------------------------------------------------------- attention --
def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def attention_case(lengths, heads, kv, dim, dtype, seed, scale=None, std=1.0, tail=0, layout="fused"):
    T = sum(lengths) + tail
    qkv = randn((T, heads + 2 * kv, dim), seed, dtype, std)
    dout = randn((T, heads, dim), seed + 1, dtype)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    dev = qkv.to(DEV)
    if tail:
        dev[T - tail:] = float("nan")
    if layout == "fused":
        qd, kd, vd = dev[:, :heads], dev[:, heads:heads + kv], dev[:, heads + kv:]
        dd = dout.to(DEV)
    else:  # heads before tokens in memory
        hm = dev.transpose(0, 1).contiguous().transpose(0, 1)
        qd, kd, vd = hm[:, :heads], hm[:, heads:heads + kv], hm[:, heads + kv:]
        dd = dout.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    if tail:
        dd[T - tail:] = float("nan")
    cu = cu_of(lengths)
    out, lse = lib.packed_attention_forward(qd, kd, vd, cu, scale=scale)
    dq, dk, dv = lib.packed_attention_backward(dd, qd, kd, vd, out, lse, cu, scale=scale)
    torch.cuda.synchronize()
    ref = R.attention(q, k, v, lengths, dim ** -0.5 if scale is None else scale, dout)
    worst = 0.0
    for name, got in (("out", out), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        worst = max(worst, R.check(name, got, *ref[name]))
    return worst


# Sets of a mean of 256 tokens and more, in grids this small, take two groups of waves a block; the others take one.
LENGTHS = [[1], [1, 1, 1], [2, 31, 32, 33], [63, 64, 65], [127, 128, 129], [0, 5, 0, 0, 300, 0], [257, 1, 190, 64],
           [511], [640], [700, 20, 400],
           [256, 3, 509]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_attention_lengths(lengths, dim, dtype):
    say(f"[gpu] attention lengths {lengths} dim {dim} {dtype}")
    worst = attention_case(lengths, 4, 2, dim, dtype, 100)
    say(f"[gpu]   worst error {worst:.3f} of its bound")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 48, 56, 72, 80, 88, 96, 104, 112, 120])
def test_attention_head_sizes(dim, dtype):
    attention_case([70, 130, 9], 3, 1, dim, dtype, 200)


@pytest.mark.parametrize("heads,kv", [(1, 1), (8, 1), (6, 3), (12, 12), (5, 5), (9, 3)])
@pytest.mark.parametrize("layout", ["fused", "heads first"])
def test_attention_heads_and_layouts(heads, kv, layout):
    for dtype in (BF, F32):
        attention_case([150, 77], heads, kv, 64, dtype, 300, layout=layout)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_large_scores(dtype):
    """Scores up to several hundred: the running maximum has to move, and most weights vanish."""
    attention_case([300, 65], 2, 1, 64, dtype, 400, scale=1.0, std=3.0)
    attention_case([300, 65], 2, 1, 64, dtype, 401, scale=1e-4)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_rising_scores(dtype):
    """Keys that grow along the sequence raise the maximum in every tile."""
    n, d = 400, 64
    q = randn((n, 2, d), 410).abs().to(dtype)
    k = (randn((n, 2, d), 411).abs() * torch.linspace(0.01, 4, n)[:, None, None]).to(dtype)
    v, do = randn((n, 2, d), 412, dtype), randn((n, 2, d), 413, dtype)
    for flip in (False, True):
        kk = k.flip(0).contiguous() if flip else k
        qd, kd, vd, dd = (t.to(DEV) for t in (q, kk, v, do))
        cu = cu_of([n])
        out, lse = lib.packed_attention_forward(qd, kd, vd, cu)
        grads = lib.packed_attention_backward(dd, qd, kd, vd, out, lse, cu)
        ref = R.attention(q, kk, v, [n], d ** -0.5, do)
        for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
            R.check(name, got, *ref[name])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_attention_groups_of_waves(dim, dtype):
    """The same tokens under both block shapes: alone (two groups), and with so many empty sequences behind them that
    the grid takes one group.  Rounding differs, the bounds hold for both."""
    lengths = [300, 470]
    T = sum(lengths)
    q, k, v, do = (randn((T, h, dim), 505 + i, dtype) for i, h in enumerate((4, 2, 2, 4)))
    ref = R.attention(q, k, v, lengths, dim ** -0.5, do)
    dev = [t.to(DEV) for t in (q, k, v, do)]
    for extra in (0, 40):
        cu = cu_of(lengths + [0] * extra)
        out, lse = lib.packed_attention_forward(*dev[:3], cu)
        g = lib.packed_attention_backward(dev[3], *dev[:3], out, lse, cu)
        for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
            R.check(name, got, *ref[name])


def test_attention_many_sequences():
    """More sequences than one search step covers, lengths 0 to 9."""
    lengths = [(i * 7) % 10 for i in range(700)]
    attention_case(lengths, 2, 2, 32, F32, 500)
    attention_case([1] * 5000, 1, 1, 8, BF, 501)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tail", [1, 130, 300])
def test_attention_rows_behind_the_last_sequence(tail, dtype):
    """They are not read (NaN there changes nothing), zero in allocated results, untouched in given ones."""
    lengths, H, G, D = [100, 37], 4, 2, 64
    attention_case(lengths, H, G, D, dtype, 600, tail=tail)
    T, n = sum(lengths) + tail, sum(lengths)
    q, k, v, do = (randn((T, h, D), 610 + i, dtype).to(DEV) for i, h in enumerate((H, G, G, H)))
    cu = cu_of(lengths)
    given = dict(out=torch.full((T, H, D), 3.0, dtype=dtype, device=DEV), lse=torch.full((H, T), 3.0, device=DEV))
    out, lse = lib.packed_attention_forward(q, k, v, cu, **given)
    assert (out[n:] == 3).all() and (lse[:, n:] == 3).all()
    g = dict(dq=torch.full((T, H, D), 3.0, dtype=dtype, device=DEV),
             dk=torch.full((T, G, D), 3.0, dtype=dtype, device=DEV),
             dv=torch.full((T, G, D), 3.0, dtype=dtype, device=DEV))
    given_grads = lib.packed_attention_backward(do, q, k, v, out, lse, cu, **g)
    out2, lse2 = lib.packed_attention_forward(q, k, v, cu)
    own_grads = lib.packed_attention_backward(do, q, k, v, out2, lse2, cu)
    assert torch.equal(out[:n], out2[:n]) and torch.equal(lse[:, :n], lse2[:, :n])
    assert (out2[n:] == 0).all() and (lse2[:, n:] == 0).all()
    for a, b in zip(given_grads, own_grads):
        assert torch.equal(a[:n], b[:n]) and (a[n:] == 3).all() and (b[n:] == 0).all()


def test_attention_no_tokens_and_no_sequences():
    e = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    out, lse = lib.packed_attention_forward(e, e, e, cu_of([0, 0]))
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    grads = lib.packed_attention_backward(e, e, e, e, out, lse, cu_of([0, 0]))
    assert all(g.shape == e.shape for g in grads)
    x = randn((200, 4, 64), 1, BF).to(DEV)  # only rows behind "the last sequence"
    out, lse = lib.packed_attention_forward(x, x, x, cu_of([]))
    assert (out == 0).all() and (lse == 0).all()
    grads = lib.packed_attention_backward(x, x, x, x, out, lse, cu_of([]))
    assert all((g == 0).all() for g in grads)


def test_attention_offsets_out_of_range_are_clamped():
    """Offsets that no caller should pass reach no memory outside the operands (guard rows stay as they were)."""
    n, H, D = 150, 2, 64
    for bad in ([0, 400], [0, 100, 50, 150], [-5, 70, 150], [0, 2 ** 31 - 1, 10], [100, 20]):
        bufs = [randn((n + 64, H, D), 700 + i, BF).to(DEV) for i in range(5)]
        keep = [b.clone() for b in bufs]
        q, k, v, o, do = (b[32:32 + n] for b in bufs)
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        lse = torch.zeros(H, n, device=DEV)
        lib.packed_attention_forward(q, k, v, cu, out=o, lse=lse)
        g = torch.full((3, n + 64, H, D), 9.0, dtype=BF, device=DEV)
        lib.packed_attention_backward(do, q, k, v, o, lse, cu, dq=g[0, 32:32 + n], dk=g[1, 32:32 + n],
                                      dv=g[2, 32:32 + n])
        torch.cuda.synchronize()
        assert (g[:, :32] == 9).all() and (g[:, 32 + n:] == 9).all()
        assert torch.equal(bufs[3][:32], keep[3][:32]) and torch.equal(bufs[3][32 + n:], keep[3][32 + n:])


def test_attention_nan_stays_in_its_sequence():
    lengths, D = [70, 90, 60], 64
    T = sum(lengths)
    q, k, v, do = (randn((T, 2, D), 720 + i, BF).to(DEV) for i in range(4))
    cu = cu_of(lengths)
    out0, lse0 = lib.packed_attention_forward(q, k, v, cu)
    g0 = lib.packed_attention_backward(do, q, k, v, out0, lse0, cu)
    for t in (q, k, v, do):
        t[100, 0, 5] = float("nan")
        t[120, 1, 0] = float("inf")
    out, lse = lib.packed_attention_forward(q, k, v, cu)
    g = lib.packed_attention_backward(do, q, k, v, out, lse, cu)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[70:160] = False
    for a, b in zip((out0, *g0), (out, *g)):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(out[100:160, 0].float()).any(1).all()
    assert torch.equal(lse0[:, keep], lse[:, keep])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_broadcast_inputs(dtype):
    """Inputs that repeat one head's or one token's memory (stride 0), or whose rows overlap, are read as they stand."""
    n, D = 90, 64
    k1, v1 = randn((n, 1, D), 730, dtype), randn((n, 1, D), 731, dtype)
    q, do = randn((n, 4, D), 732, dtype), randn((n, 4, D), 733, dtype)
    cu = cu_of([n])
    kd, vd = k1.to(DEV).expand(n, 4, D), v1.to(DEV).expand(n, 4, D)
    out, lse = lib.packed_attention_forward(q.to(DEV), kd, vd, cu)
    g = lib.packed_attention_backward(do.to(DEV), q.to(DEV), kd, vd, out, lse, cu)
    ref = R.attention(q, k1.expand(n, 4, D), v1.expand(n, 4, D), [n], D ** -0.5, do)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
        R.check(name, got, *ref[name])
    one = randn((1, 1, D), 734, dtype)  # the gradient of a sum: one value everywhere
    line = randn((n * 8 + D,), 735, dtype)
    roll = torch.as_strided(line, (n, 1, D), (8, D, 1))
    rolld = torch.as_strided(line.to(DEV), (n, 1, D), (8, D, 1))
    oned = one.to(DEV).expand(n, 4, D)
    out, lse = lib.packed_attention_forward(q.to(DEV), rolld, vd[:, :1], cu)
    g = lib.packed_attention_backward(oned, q.to(DEV), rolld, vd[:, :1], out, lse, cu)
    ref = R.attention(q, roll, v1, [n], D ** -0.5, one.expand(n, 4, D))
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
        R.check(name, got, *ref[name])
    out, lse = lib.packed_attention_forward(rolld.expand(n, 4, D), kd[:, :1], oned[:, :1], cu)
    g = lib.packed_attention_backward(do.to(DEV), rolld.expand(n, 4, D), kd[:, :1], oned[:, :1], out, lse, cu)
    ref = R.attention(roll.expand(n, 4, D), k1, one.expand(n, 1, D), [n], D ** -0.5, do)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
        R.check(name, got, *ref[name])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_scores_of_minus_infinity_weigh_nothing(dtype):
    """Keys whose scores are -inf for every query, from single ones to whole tiles and the sequence's first: the other
    keys' softmax stands; a row that sees no other key is NaN."""
    n, D = 300, 64
    q, k, v = (randn((n, 1, D), 745 + i, dtype) for i in range(3))
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    for dead in ([0], list(range(64)), list(range(64, 128)) + [200], list(range(128))):
        kk = k.clone()
        kk[dead, :, 0] = float("-inf")
        out, lse = lib.packed_attention_forward(q.to(DEV), kk.to(DEV), v.to(DEV), cu_of([n]))
        live = torch.ones(n, dtype=torch.bool)
        live[dead] = False
        s = (q[:, 0].double() @ k[:, 0].double().T) * D ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1) | ~live[None], float("-inf"))
        sees = live.cumsum(0) > 0
        want = torch.softmax(s, 1) @ v[:, 0].double()
        mass = torch.softmax(s, 1) @ v[:, 0].double().abs()
        u = R.unit(dtype)
        # p and the result rounded (bf16), and in fp32 the scores' sums of 64 terms and the sum over at most 300 keys
        bound = u * want.abs() + ((u if dtype == BF else 0) + (64 + 300 + 64) * 2 * R.U32 * 8) * mass
        R.check("out", out[sees.to(DEV), 0], want[sees], bound[sees])
        assert torch.isnan(out[~sees.to(DEV)].float()).all()
        assert (lse[0, ~sees.to(DEV)] == float("-inf")).all() and torch.isfinite(lse[0, sees.to(DEV)]).all()


def test_binding_refuses_what_does_not_go_together():
    x, w = torch.zeros(4, 64, device=DEV, dtype=BF), torch.ones(64, device=DEV)
    y, mean, rstd = lib.layer_norm_forward(x, w)
    bad = [lambda: lib.layer_norm_forward(x.half()), lambda: lib.layer_norm_forward(x, w[:32]),
           lambda: lib.layer_norm_forward(x, w.cpu()), lambda: lib.layer_norm_forward(x, w, w.to(BF)),
           lambda: lib.layer_norm_forward(x, w.half()), lambda: lib.layer_norm_forward(x, w, out=x.float()),
           lambda: lib.layer_norm_forward(x, w, out=x[:2]), lambda: lib.layer_norm_forward(x.t()),
           lambda: lib.layer_norm_forward(x[:1].expand(4, 64)), lambda: lib.layer_norm_forward(x, out=x[:1].expand(4, 64)),
           lambda: lib.layer_norm_backward(x.float(), x, mean, rstd), lambda: lib.layer_norm_backward(x, x, mean[:2], rstd),
           lambda: lib.layer_norm_backward(x, x, mean.to(BF), rstd),
           lambda: lib.layer_norm_backward(x, x, mean, rstd, dx=x[:2])]
    q, k = torch.zeros(10, 4, 64, device=DEV, dtype=BF), torch.zeros(10, 2, 64, device=DEV, dtype=BF)
    cu = cu_of([10])
    out, lse = lib.packed_attention_forward(q, k, k, cu)
    f, b = lib.packed_attention_forward, lib.packed_attention_backward
    bad += [lambda: f(q, k.float(), k, cu), lambda: f(q, k, k[:5], cu), lambda: f(q, k[:5], k[:5], cu),
            lambda: f(q, k, k, cu.long()), lambda: f(q, k, k, cu.cpu()), lambda: f(q, k, k, cu[:0]),
            lambda: f(q, k, k, cu.expand(2, 2)), lambda: f(q.half(), k.half(), k.half(), cu),
            lambda: f(q.transpose(1, 2), k, k, cu), lambda: f(q[0], k[0], k[0], cu), lambda: f(q, k, k, cu, out=q[:5]),
            lambda: f(q, k, k, cu, lse=lse.t()), lambda: f(q, k[..., :32], k[..., :32], cu),
            lambda: f(q.cpu(), k, k, cu), lambda: b(q[:5], q, k, k, out, lse, cu),
            lambda: b(q, q, k, k, out, lse[:2], cu), lambda: b(q, q, k, k, out, lse, cu, dk=q)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was not refused")
    x3, k3 = torch.zeros(10, 3, 64, device=DEV, dtype=BF), torch.zeros(10, 1, 64, device=DEV, dtype=BF)
    errors = [lambda: lib.layer_norm_forward(x, out=x), lambda: lib.layer_norm_backward(x, x.clone(), mean, rstd, dx=x),
              lambda: lib.layer_norm_forward(x, eps=-1.0), lambda: f(x3, k, k, cu), lambda: f(q, k, k, cu, out=q),
              lambda: f(q, k, k, cu, scale=0.0), lambda: f(q[..., :60], k[..., :60], k[..., :60], cu),
              lambda: f(q, k, k, cu, out=k3.expand(10, 4, 64)), lambda: b(q.clone(), q, k, k, out, lse, cu, dq=q),
              lambda: b(q, q.clone(), k, k, out, lse, cu, dk=torch.zeros_like(k), dv=k)]
    buf = torch.zeros(10 * 4 * 64 + 8, device=DEV, dtype=BF)
    errors.append(lambda: f(buf[4:4 + 2560].view(10, 4, 64), k, k, cu))  # not at a multiple of 16 bytes
    for i, call in enumerate(errors):
        with pytest.raises(lib._lib.MuonError):
            call()
            raise AssertionError(f"call {i} was not refused")


def test_attention_offsets_past_32_bits():
    """Tokens 2^25 bytes apart: byte offsets pass 2^32 within one sequence."""
    n, D, step = 200, 64, 1 << 24
    buf = torch.empty((n - 1) * step + 3 * D, dtype=BF, device=DEV)
    qkv = torch.as_strided(buf, (n, 3, D), (step, D, 1))
    src = randn((n, 3, D), 740, BF)
    qkv.copy_(src)
    do = randn((n, 1, D), 741, BF)
    cu = cu_of([n])
    q, k, v = qkv[:, :1], qkv[:, 1:2], qkv[:, 2:]
    out, lse = lib.packed_attention_forward(q, k, v, cu)
    gbuf = torch.empty_like(buf)
    gr = torch.as_strided(gbuf, (n, 3, D), (step, D, 1))
    g = lib.packed_attention_backward(do.to(DEV), q, k, v, out, lse, cu, dq=gr[:, :1], dk=gr[:, 1:2], dv=gr[:, 2:])
    ref = R.attention(src[:, :1], src[:, 1:2], src[:, 2:], [n], D ** -0.5, do)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *g)):
        R.check(name, got, *ref[name])


def test_gradients_against_differences():
    """fp32 gradients against central differences of the kernels' own forward results.

    L = sum(dout * out) in fp64 of fp32 results.  A step h along a unit
    direction changes L by 2 h <grad, dir> up to h^3 terms; the results' own
    roundings (2^-23 of about sqrt(N) values of order 1) over 2 h are the noise.
    """
    n, H, D, h = 96, 2, 32, 2.0 ** -5
    q, k, v, do = (randn((n, H, D), 750 + i).to(DEV) for i in range(4))
    cu = cu_of([40, 56])

    def loss(q, k, v):
        return (lib.packed_attention_forward(q, k, v, cu)[0].double() * do.double()).sum().item()

    out, lse = lib.packed_attention_forward(q, k, v, cu)
    grads = lib.packed_attention_backward(do, q, k, v, out, lse, cu)
    args = [q, k, v]
    for i, g in enumerate(grads):
        d = randn((n, H, D), 760 + i).to(DEV)
        d /= d.norm()
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * d, args[i] + h * d
        diff = (loss(*hi) - loss(*lo)) / (2 * h)
        want = (g.double() * d.double()).sum().item()
        noise = 2.0 ** -22 * (n * H * D) ** 0.5 * 4 / h
        assert abs(diff - want) <= noise + h * h * g.norm().item(), ("qkv"[i], diff, want)
    x, w, b, dy = (randn(s, 770 + i).to(DEV) for i, s in enumerate(((20, 96), (96,), (96,), (20, 96))))
    y, mean, rstd = lib.layer_norm_forward(x, w, b)
    grads = lib.layer_norm_backward(dy, x, mean, rstd, w)
    args = [x, w, b]
    for i, g in enumerate(grads):
        d = randn(tuple(args[i].shape), 780 + i).to(DEV)
        d /= d.norm()
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * d, args[i] + h * d
        diff = sum(s * (lib.layer_norm_forward(*a)[0].double() * dy.double()).sum().item()
                   for s, a in ((1, hi), (-1, lo))) / (2 * h)
        want = (g.double() * d.double()).sum().item()
        noise = 2.0 ** -22 * (20 * 96) ** 0.5 * 8 / h
        assert abs(diff - want) <= noise + h * h * g.norm().item(), ("xwb"[i], diff, want)


# ------------------------------------------------- streams, graphs, together --
def block_tensors(lengths, seed, heads=4, dim=64, dtype=BF):
    T, width = sum(lengths), heads * dim
    t = dict(x=randn((T, width), seed, dtype), w=1 + randn((width,), seed + 1, std=0.1), b=randn((width,), seed + 2),
             wqkv=randn((width, 3 * width), seed + 3, dtype, width ** -0.5),
             wo=randn((width, width), seed + 4, dtype, width ** -0.5), dout=randn((T, width), seed + 5, dtype))
    t = {k: v.to(DEV) for k, v in t.items()}
    t["cu"], t["heads"], t["dim"] = cu_of(lengths), heads, dim
    return t


def block_step(t):
    """norm -> qkv product -> attention -> output product, and back to every gradient."""
    H, D = t["heads"], t["dim"]
    T = t["x"].shape[0]
    y, mean, rstd = lib.layer_norm_forward(t["x"], t["w"], t["b"])
    qkv = (y @ t["wqkv"]).view(T, 3 * H, D)
    q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:]
    o, lse = lib.packed_attention_forward(q, k, v, t["cu"])
    z = o.view(T, H * D) @ t["wo"]
    do = (t["dout"] @ t["wo"].t()).view(T, H, D)
    dwo = o.view(T, H * D).t() @ t["dout"]
    dqkv = torch.empty_like(qkv)
    lib.packed_attention_backward(do, q, k, v, o, lse, t["cu"], dq=dqkv[:, :H], dk=dqkv[:, H:2 * H],
                                  dv=dqkv[:, 2 * H:])
    dqkv = dqkv.view(T, 3 * H * D)
    dwqkv = y.t() @ dqkv
    dx, dw, db = lib.layer_norm_backward(dqkv @ t["wqkv"].t(), t["x"], mean, rstd, t["w"])
    return dict(z=z, dwo=dwo, dwqkv=dwqkv, dx=dx, dw=dw, db=db)


def test_block_run_and_muon_step():
    """The operators as they are used: a block's forward and backward pass in fp32 against fp64 autograd, and its
    matrix gradients into a Muon step."""
    lengths = [70, 1, 129]
    t = block_tensors(lengths, 800, dtype=F32)
    got = block_step(t)
    c = {k: v.double().cpu().requires_grad_(k in ("x", "w", "b", "wqkv", "wo")) for k, v in t.items()
         if isinstance(v, torch.Tensor) and v.is_floating_point()}
    H, D, T = t["heads"], t["dim"], sum(lengths)
    y = torch.nn.functional.layer_norm(c["x"], (H * D,), c["w"], c["b"], 1e-5)
    qkv = (y @ c["wqkv"]).view(T, 3 * H, D).permute(1, 0, 2)
    doc = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
    i = torch.arange(T)
    hidden = (doc[:, None] != doc[None]) | (i[None] > i[:, None])
    s = (qkv[:H] @ qkv[H:2 * H].transpose(1, 2) * D ** -0.5).masked_fill(hidden, float("-inf"))
    o = (torch.softmax(s, 2) @ qkv[2 * H:]).permute(1, 0, 2).reshape(T, H * D)
    z = o @ c["wo"]
    (z * c["dout"]).sum().backward()
    want = dict(z=z.detach(), dwo=c["wo"].grad, dwqkv=c["wqkv"].grad, dx=c["x"].grad, dw=c["w"].grad, db=c["b"].grad)
    for name, w in want.items():
        rel = ((got[name].double().cpu() - w).norm() / w.norm()).item()
        say(f"[gpu] block {name}: rel {rel:.2e}")
        # fp32 throughout: five chained sums of at most 800 terms, each off by at most 800 * 2^-24 = 4.8e-5
        assert rel <= 5 * 800 * 2.0 ** -24, (name, rel)
    W = [t["wqkv"].clone(), t["wo"].clone()]
    M = [torch.zeros_like(w) for w in W]
    step = lib.MuonStep(W, [got["dwqkv"].contiguous(), got["dwo"].contiguous()], M)
    step.step(lr=0.02)
    torch.cuda.synchronize()
    step.close()
    assert all(torch.isfinite(w).all() for w in W) and not torch.equal(W[0], t["wqkv"])


def test_block_is_deterministic_and_graph_replays_match():
    t = block_tensors([200, 33, 64, 301], 820)
    ref = block_step(t)
    again = block_step(t)
    assert all(torch.equal(ref[k], again[k]) for k in ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block_step(t)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = block_step(t)
    second = torch.cuda.CUDAGraph()  # a second graph has workspaces of its own
    with torch.cuda.graph(second):
        res2 = block_step(t)
    for rep in range(4):
        # new data and other sequence lengths in the same buffers
        t["x"].copy_(randn(tuple(t["x"].shape), 830 + rep, BF).to(DEV))
        t["cu"].copy_(cu_of([[200, 33, 64, 301], [0, 598, 0, 0], [1, 2, 3, 592], [149, 150, 149, 150]][rep]))
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        want = block_step(t)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(res[k], want[k]), (rep, k)
            assert torch.equal(res2[k], want[k]), (rep, k)


def test_block_on_two_streams_at_once():
    a, b = block_tensors([300, 212], 840), block_tensors([17] * 40, 850)
    ra, rb = block_step(a), block_step(b)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(3):
        with torch.cuda.stream(sa):
            ga = block_step(a)
        with torch.cuda.stream(sb):
            gb = block_step(b)
        outs.append((ga, gb))
    torch.cuda.synchronize()
    for ga, gb in outs:
        assert all(torch.equal(ga[k], ra[k]) for k in ra)
        assert all(torch.equal(gb[k], rb[k]) for k in rb)


def test_attention_long_packed_sequences():
    """A long pack in bf16 against the fp32 kernels, which the other tests pin: several hundred tiles, every
    sequence start inside a tile, and (grouped heads) a split of a group over blocks."""
    lengths = [5000, 1, 1300, 77, 2000, 640]
    T, D = sum(lengths), 128
    for heads, kv in ((4, 4), (8, 1)):
        q, k, v, do = (randn((T, h, D), 860 + i, BF).to(DEV) for i, h in enumerate((heads, kv, kv, heads)))
        cu = cu_of(lengths)
        out, lse = lib.packed_attention_forward(q, k, v, cu)
        g = lib.packed_attention_backward(do, q, k, v, out, lse, cu)
        f = [t.float() for t in (q, k, v, do)]
        out32, lse32 = lib.packed_attention_forward(*f[:3], cu)
        g32 = lib.packed_attention_backward(f[3], *f[:3], out32, lse32, cu)
        assert (lse - lse32).abs().max().item() <= 1e-4  # both fp32; 5000 terms of at most 2^-24 each, and scores of ~10
        for name, x, y in zip(("out", "dq", "dk", "dv"), (out, *g), (out32, *g32)):
            rel = ((x.float() - y).norm() / y.norm()).item()
            say(f"[gpu] long pack {heads}/{kv} {name}: rel {rel:.2e}")
            # roundings of p or ds, of delta's output, and of the result, each at most 2^-8
            assert rel <= 3 * 2.0 ** -8, (name, rel)
