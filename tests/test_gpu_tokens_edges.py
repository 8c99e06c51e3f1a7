"""The embedding and the query/key norm as they are used: under torch's autograd, on streams, in graphs, together with
the layer norm and the attention, and what their binding refuses."""
import itertools

import pytest
import torch

import block_reference as B
import muon_newton_schulz_03_amd as lib
import token_reference as R
from muon_harness import say
from muon_newton_schulz_03_amd._lib import MuonError

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(DEV)


def randint(lo, hi, shape, seed, dtype=torch.int64):
    return torch.randint(lo, hi, shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def leaf(t):
    return t.detach().clone().requires_grad_(True)


# --------------------------------------------------------------- torch's gradients --
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (F32, BF), (F32, F32)])
def test_embedding_takes_part_in_autograd(dtype, out_dtype):
    table, ids = randn((50, 72), 1, dtype), randint(-1, 51, (4, 33), 2)
    do = randn((4, 33, 72), 3, out_dtype)
    want = lib.embedding_forward(table, ids, scale=1.5, dtype=out_dtype)
    assert not want.requires_grad and want.dtype == out_dtype
    grad = lib.embedding_backward(do, ids, 50, scale=1.5, dtype=dtype)
    t = leaf(table)
    out = lib.embedding_forward(t, ids, scale=1.5, dtype=out_dtype)
    assert torch.equal(out, want)
    out.backward(do)
    assert t.grad.dtype == dtype and torch.equal(t.grad, grad)
    for weight in (torch.ones((), device=DEV, dtype=out_dtype).expand(4, 33, 72), do[:, :1].expand(4, 33, 72),
                   do.transpose(0, 1).contiguous().transpose(0, 1), torch.cat([do[..., :1], do], 2)[..., 1:]):
        t = leaf(table)
        lib.embedding_forward(t, ids, scale=1.5, dtype=out_dtype).backward(weight)
        assert torch.equal(t.grad, lib.embedding_backward(weight.contiguous(), ids, 50, scale=1.5, dtype=dtype))
    t = leaf(table)  # columns of a wider table: the gradient reaches its own columns
    (lib.embedding_forward(t[:, 8:40], ids, dtype=out_dtype) * do[..., 8:40]).sum().backward()
    assert torch.equal(t.grad[:, 8:40], lib.embedding_backward(do[..., 8:40], ids, 50, dtype=dtype))
    assert (t.grad[:, :8] == 0).all() and (t.grad[:, 40:] == 0).all()


@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (BF, BF), (F32, F32)])
def test_qk_norm_takes_part_in_autograd(dtype, pdtype):
    T, H, G, D = 60, 4, 2, 64
    qkv, do = randn((T, H + 2 * G, D), 10, dtype), randn((T, H + G, D), 11, dtype)
    w = [(1 + randn((D,), 12 + i, std=0.2)).to(pdtype) for i in (0, 1)]
    rot, cu = lib.Rotation(D), cu_of([40, 15])
    cut = lambda t: (t[:, :H], t[:, H:H + G])  # noqa: E731
    names = dict(cu_seqlens=cu, eps=1e-5)
    q0, k0 = lib.qk_norm_forward(*cut(qkv), rot, q_weight=w[0], k_weight=w[1], **names)
    assert not q0.requires_grad
    want = lib.qk_norm_backward(*cut(do), *cut(qkv), rot, q_weight=w[0], k_weight=w[1], **names)
    for wanted in itertools.product((0, 1), repeat=4):
        if not any(wanted):
            continue
        args = [t.detach().clone().requires_grad_(bool(n)) for t, n in zip((*cut(qkv), *w), wanted)]
        q, k = lib.qk_norm_forward(args[0], args[1], rot, q_weight=args[2], k_weight=args[3], **names)
        assert torch.equal(q, q0) and torch.equal(k, k0)
        torch.autograd.backward([q, k], list(cut(do)))
        for t, g, n in zip(args, want, wanted):
            assert (t.grad is None) if not n else (t.grad.dtype == t.dtype and torch.equal(t.grad, g.to(t.dtype)))
    p = leaf(qkv)  # slices of one projection; only the keys' result is used
    _, k = lib.qk_norm_forward(*cut(p), rot, **names)
    k.backward(do[:, H:])
    zero = torch.zeros_like(do[:, :H])
    dq, dk, _, _ = lib.qk_norm_backward(zero, do[:, H:], *cut(qkv), rot, **names)
    assert torch.equal(p.grad, torch.cat([dq, dk, torch.zeros_like(qkv[:, H + G:])], 1))
    for weight in (torch.ones((), device=DEV, dtype=dtype).expand(T, H, D), do[:, :1].expand(T, H, D),
                   torch.cat([do[..., :1], do], 2)[:, :H, 1:]):
        p = leaf(qkv)
        lib.qk_norm_forward(*cut(p), rot, **names)[0].backward(weight)
        dq = lib.qk_norm_backward(weight.contiguous(), torch.zeros_like(k0), *cut(qkv), rot, **names)[0]
        assert torch.equal(p.grad[:, :H], dq)
    x = leaf(qkv[:, :H])  # one tensor as queries and keys, one weight for both: the gradients add up
    v = leaf(w[0])
    a, b = lib.qk_norm_forward(x, x, rot, q_weight=v, k_weight=v, **names)
    torch.autograd.backward([a, b], [do[:, :H], do[:, 2:]])
    da, db, dwa, dwb = lib.qk_norm_backward(do[:, :H], do[:, 2:], x.detach(), x.detach(), rot, q_weight=w[0],
                                            k_weight=w[0], **names)
    assert torch.equal(x.grad, da + db) and torch.equal(v.grad, dwa.to(pdtype) + dwb.to(pdtype))


def test_gradients_that_would_be_lost_are_refused():
    table, ids = leaf(randn((20, 64), 20)), randint(0, 20, (30,), 21)
    q, k, w = leaf(randn((30, 2, 32), 22)), leaf(randn((30, 2, 32), 23)), leaf(randn((32,), 24))
    out = lib.embedding_forward(table, ids)
    a, b = lib.qk_norm_forward(q, k, q_weight=w)
    for z, t in ((out, table), (a, q), (a, w), (b, k)):  # differentiable once
        g, = torch.autograd.grad(z.square().sum(), t, create_graph=True, retain_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
    buf, qb = torch.zeros(30, 64, device=DEV), torch.zeros(30, 2, 32, device=DEV)
    td, qd, kd = table.detach(), q.detach(), k.detach()
    for call in (lambda: lib.embedding_forward(table, ids, out=buf), lambda: lib.qk_norm_forward(q, kd, q_out=qb),
                 lambda: lib.qk_norm_forward(qd, k, q_out=qb), lambda: lib.qk_norm_forward(qd, kd, k_weight=w, k_out=qb)):
        with pytest.raises(ValueError, match="recorded"):
            call()
    for call in (lambda: lib.embedding_forward(td, ids, out=out * 1),
                 lambda: lib.embedding_backward(buf, ids, 20, dtable=table),
                 lambda: lib.qk_norm_forward(qd, kd, k_out=a * 1),
                 lambda: lib.qk_norm_backward(qb, qb.clone(), qd, kd, dq=q * 1),
                 lambda: lib.qk_norm_backward(qb, qb.clone(), qd, kd, dk=k * 1)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            lib.embedding_forward(torch.autograd.forward_ad.make_dual(td, td.clone()), ids)
        with pytest.raises((RuntimeError, NotImplementedError)):
            lib.qk_norm_forward(torch.autograd.forward_ad.make_dual(qd, qb), kd)


def test_a_graph_that_saved_a_given_output_notices_that_it_was_written():
    table, ids = randn((20, 64), 30), randint(0, 20, (30,), 31)
    q, k = randn((30, 2, 32), 32), randn((30, 2, 32), 33)
    writes = [((30, 64), lambda t: lib.embedding_forward(table, ids, out=t)),
              ((20, 64), lambda t: lib.embedding_backward(table.new_zeros(30, 64), ids, 20, dtable=t)),
              ((20, 64), lambda t: lib.embedding_backward(table.new_zeros(30, 64), ids, 20, dtable=t, accumulate=True)),
              ((30, 2, 32), lambda t: lib.qk_norm_forward(q, k, q_out=t)),
              ((30, 2, 32), lambda t: lib.qk_norm_forward(q, k, k_out=t)),
              ((30, 2, 32), lambda t: lib.qk_norm_backward(q.clone(), k.clone(), q, k, dq=t)),
              ((30, 2, 32), lambda t: lib.qk_norm_backward(q.clone(), k.clone(), q, k, dk=t))]
    for i, (shape, write) in enumerate(writes):
        p, saved = torch.ones(shape, device=DEV, requires_grad=True), torch.ones(shape, device=DEV)
        loss = (p * saved).sum()
        write(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
            raise AssertionError(f"write {i} went unnoticed")


# -------------------------------------------------------------------- refusals --
def test_binding_refuses_what_does_not_go_together():
    table, ids, out = randn((20, 64), 40), randint(0, 20, (30,), 41), torch.zeros(30, 64, device=DEV)
    bad = [lambda: lib.embedding_forward(table, ids.float()), lambda: lib.embedding_forward(table, ids.to(torch.int16)),
           lambda: lib.embedding_forward(table, ids.repeat(2)[::2]), lambda: lib.embedding_forward(table, ids.cpu()),
           lambda: lib.embedding_forward(table.half(), ids), lambda: lib.embedding_forward(table[0], ids),
           lambda: lib.embedding_forward(table.t(), ids), lambda: lib.embedding_forward(table, ids, dtype=torch.half),
           lambda: lib.embedding_forward(table, ids, out=out[:29]), lambda: lib.embedding_forward(table, ids, out=3),
           lambda: lib.embedding_forward(table, ids, out=out, dtype=BF), lambda: lib.embedding_forward("table", ids),
           lambda: lib.embedding_forward(table, ids, out=out.t()),
           lambda: lib.embedding_backward(out, ids, 20, accumulate=True),
           lambda: lib.embedding_backward(out[:29], ids, 20), lambda: lib.embedding_backward(out.half(), ids, 20),
           lambda: lib.embedding_backward(out, ids, 20, dtable=table[:19]),
           lambda: lib.embedding_backward(out, ids, 20, dtype=torch.half), lambda: lib.embedding_backward(out, ids, 0),
           lambda: lib.embedding_backward(out, ids, -1), lambda: lib.embedding_backward(out[:1].expand(30, 64), ids, 20),
           lambda: lib.embedding_backward(out, ids.view(5, 6), 20)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was taken")
    with pytest.raises(MuonError, match="scale"):
        lib.embedding_forward(table, ids, scale=float("nan"))
    big = torch.zeros(60, 64, device=DEV)
    with pytest.raises(MuonError, match="overlap"):  # the table's rows are written while others read them
        lib.embedding_forward(big[:20], ids, out=big[15:45])
    with pytest.raises(MuonError, match="overlap"):
        lib.embedding_backward(big[:30], ids, 20, dtable=big[20:40])
    with pytest.raises(MuonError, match="overlap"):
        lib.embedding_forward(table[:, :2], ids, out=ids.view(torch.float32).view(30, 2))
    q, k, w = randn((30, 4, 64), 42), randn((30, 2, 64), 43), randn((64,), 44)
    rot, pos = lib.Rotation(64), torch.arange(30, device=DEV)
    bad = [lambda: lib.qk_norm_forward(q, k[:29]), lambda: lib.qk_norm_forward(q, k[..., :32]),
           lambda: lib.qk_norm_forward(q, k.to(BF)), lambda: lib.qk_norm_forward(q.half(), k.half()),
           lambda: lib.qk_norm_forward(q[0], k), lambda: lib.qk_norm_forward(q, k.cpu()),
           lambda: lib.qk_norm_forward(q, k, 64), lambda: lib.qk_norm_forward(q, k, q_weight=w[:32]),
           lambda: lib.qk_norm_forward(q, k, q_weight=w, k_weight=w.to(BF)),
           lambda: lib.qk_norm_forward(q, k, k_weight=w.half()), lambda: lib.qk_norm_forward(q, k, positions=pos[:29]),
           lambda: lib.qk_norm_forward(q, k, positions=pos.float()),
           lambda: lib.qk_norm_forward(q, k, positions=pos.repeat(2)[::2]),
           lambda: lib.qk_norm_forward(q, k, cu_seqlens=pos), lambda: lib.qk_norm_forward(q, k, cu_seqlens=cu_of([30])[None]),
           lambda: lib.qk_norm_forward(q, k, q_out=k), lambda: lib.qk_norm_forward(q, k, k_out=k.to(BF)),
           lambda: lib.qk_norm_forward(q.transpose(1, 2), k.transpose(1, 2)),
           lambda: lib.qk_norm_backward(q[:, :2], k, q, k), lambda: lib.qk_norm_backward(q, k.to(BF), q, k),
           lambda: lib.qk_norm_backward(q, k, q, k, dq=k)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was taken")
    for call, match in ((lambda: lib.qk_norm_forward(q, k, rot, q_out=q), "overlap"),
                        (lambda: lib.qk_norm_forward(q[..., :60], k[..., :60]), "multiple of 8"),
                        (lambda: lib.qk_norm_forward(q[..., :32], k[..., :32], rot), "rotation"),
                        (lambda: lib.qk_norm_forward(q, k, eps=-1.0), "eps"),
                        (lambda: lib.qk_norm_forward(q[..., 2:58], k[..., 2:58]), "16 bytes"),
                        (lambda: lib.qk_norm_forward(q, k, lib.Rotation(8, frequencies=[1, 2, 3, 65.0])), "frequency"),
                        (lambda: lib.qk_norm_backward(q, k, q, k, dq=torch.zeros(1, 4, 64, device=DEV).expand(30, 4, 64)),
                         "overlap")):
        with pytest.raises(MuonError, match=match):
            call()


# -------------------------------------------------------------- together, streams, graphs --
def model(seed, lengths, dtype=F32):
    """A token table, a layer norm, one attention with normalised and rotated queries and keys (four and two heads of
    32), an output matrix."""
    T, V, C, H, G, D = sum(lengths), 90, 128, 4, 2, 32
    t = dict(table=randn((V, C), seed, dtype), w=1 + randn((C,), seed + 1, std=0.1), b=randn((C,), seed + 2, std=0.1),
             wqkv=randn((C, (H + 2 * G) * D), seed + 3, dtype, C ** -0.5), qw=1 + randn((D,), seed + 4, std=0.2),
             kw=1 + randn((D,), seed + 5, std=0.2), wo=randn((H * D, C), seed + 6, dtype, C ** -0.5),
             dout=randn((T, C), seed + 7, dtype))
    t["ids"], t["cu"] = randint(-1, V, (T,), seed + 8), cu_of(lengths)
    return t, (H, G, D)


NAMES = ("table", "w", "b", "wqkv", "qw", "kw", "wo")
SCALE = 11.0


def model_step(t, dims):
    """Forward and back with the operators' own calls: the gradients in NAMES' order."""
    H, G, D = dims
    T, rot = t["ids"].shape[0], lib.Rotation(D)
    x = lib.embedding_forward(t["table"], t["ids"], scale=SCALE)
    y, mean, rstd = lib.layer_norm_forward(x, t["w"], t["b"])
    qkv = (y @ t["wqkv"]).view(T, H + 2 * G, D)
    q, k, v = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
    how = dict(q_weight=t["qw"], k_weight=t["kw"], cu_seqlens=t["cu"])
    qn, kn = lib.qk_norm_forward(q, k, rot, **how)
    o, lse = lib.packed_attention_forward(qn, kn, v, t["cu"])
    do = (t["dout"] @ t["wo"].t()).view(T, H, D)
    dqkv = torch.empty_like(qkv)
    dqn, dkn, _ = lib.packed_attention_backward(do, qn, kn, v, o, lse, t["cu"], dv=dqkv[:, H + G:])
    _, _, dqw, dkw = lib.qk_norm_backward(dqn, dkn, q, k, rot, dq=dqkv[:, :H], dk=dqkv[:, H:H + G], **how)
    dqkv = dqkv.view(T, -1)
    dx, dw, db = lib.layer_norm_backward(dqkv @ t["wqkv"].t(), x, mean, rstd, t["w"])
    dtable = lib.embedding_backward(dx, t["ids"], t["table"].shape[0], scale=SCALE, dtype=t["table"].dtype)
    return dtable, dw, db, y.t() @ dqkv, dqw, dkw, o.view(T, H * D).t() @ t["dout"]


def model_loss(p, t, dims):
    """The same forward pass as torch records it."""
    H, G, D = dims
    T = t["ids"].shape[0]
    x = lib.embedding_forward(p["table"], t["ids"], scale=SCALE)
    y, _, _ = lib.layer_norm_forward(x, p["w"], p["b"])
    qkv = (y @ p["wqkv"]).view(T, H + 2 * G, D)
    qn, kn = lib.qk_norm_forward(qkv[:, :H], qkv[:, H:H + G], lib.Rotation(D), q_weight=p["qw"], k_weight=p["kw"],
                                 cu_seqlens=t["cu"])
    o, _ = lib.packed_attention_forward(qn, kn, qkv[:, H + G:], t["cu"])
    return (o.reshape(T, H * D) @ p["wo"] * t["dout"]).sum()


def model_truth(t, dims, lengths):
    """Its gradients by fp64 autograd on the CPU."""
    H, G, D = dims
    T = sum(lengths)
    c = {n: t[n].double().cpu().requires_grad_(True) for n in NAMES}
    ids = t["ids"].cpu()
    known = (ids >= 0) & (ids < t["table"].shape[0])
    x = torch.where(known[:, None], SCALE * c["table"][ids.clamp(min=0)], 0.0)
    y = torch.nn.functional.layer_norm(x, x.shape[1:], c["w"], c["b"], 1e-5)
    qkv = (y @ c["wqkv"]).view(T, H + 2 * G, D)
    turns = R.angles(R.positions_of(T, lengths), lib.Rotation(D).frequencies)

    def normed(z, w):
        z = z / torch.sqrt(z.square().mean(2, keepdim=True) + 1e-6) * w
        return R.turn(z, turns[0], turns[1], D, "halves")

    q, k, v = normed(qkv[:, :H], c["qw"]), normed(qkv[:, H:H + G], c["kw"]), qkv[:, H + G:]
    q, k, v = (z.repeat_interleave(H // z.shape[1], 1).permute(1, 0, 2) for z in (q, k, v))
    doc = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
    i = torch.arange(T)
    hidden = (doc[:, None] != doc[None]) | (i[None] > i[:, None])
    s = (q @ k.transpose(1, 2) * D ** -0.5).masked_fill(hidden, float("-inf"))
    o = (torch.softmax(s, 2) @ v).permute(1, 0, 2).reshape(T, H * D)
    return torch.autograd.grad((o @ c["wo"] * t["dout"].double().cpu()).sum(), [c[n] for n in NAMES])


def test_operators_together_against_autograd():
    """ids -> rows -> norm -> projection -> normalised, rotated queries and keys -> attention, and back, in fp32."""
    lengths = [70, 1, 129]
    t, dims = model(50, lengths)
    got, want = model_step(t, dims), model_truth(t, dims, lengths)
    p = {n: leaf(t[n]) for n in NAMES}
    recorded = torch.autograd.grad(model_loss(p, t, dims), [p[n] for n in NAMES])
    for name, a, r, w in zip(NAMES, got, recorded, want):
        rel = ((a.double().cpu() - w).norm() / w.norm()).item()
        say(f"[gpu] together d{name}: rel {rel:.2e}")
        # fp32 throughout: seven chained sums of at most 256 terms (tokens, columns), each off by at most 264 * 2^-24
        # of its terms' magnitude, which cancellation (the norms' backward passes) leaves within 4 of the result's
        assert rel <= 4 * 7 * 264 * 2.0 ** -24, (name, rel)
        # under autograd the same calls, but v's gradient is copied into the projection's
        rel = ((r.double().cpu() - w).norm() / w.norm()).item()
        assert rel <= 4 * 7 * 264 * 2.0 ** -24, (name, rel)


def test_operators_on_two_streams_at_once():
    sets = [model(60, [300, 212], BF), model(70, [17] * 40, BF)]
    want = [model_step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(model_step(*s))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2])), i


@pytest.mark.parametrize("T", [200, 5000, 20000])
def test_operators_in_a_graph(T):
    """Captured and replayed with new ids, rows and sequences, beside eager work; one case for each way to sort."""
    def lengths_of(rep):
        return [[T], [T - 3, 0, 3], [1, 2, T // 2, T - T // 2 - 3], [0, T]][rep % 4]

    t, dims = model(80, [T // 4, T - T // 4, 0, 0], BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        model_step(t, dims)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = model_step(t, dims)
    with torch.cuda.graph(second):  # a second graph has workspaces of its own
        res2 = model_step(t, dims)
    for rep in range(4):
        t["ids"].copy_(randint(-1, 90 if rep else 5, (T,), 90 + rep))
        t["table"].copy_(randn(tuple(t["table"].shape), 95 + rep, BF))
        lengths = lengths_of(rep)
        t["cu"].copy_(cu_of(lengths + [0] * (4 - len(lengths))))
        graph.replay()
        second.replay()
        torch.cuda.synchronize()
        want = model_step(t, dims)
        torch.cuda.synchronize()
        for n, a, b, w in zip(NAMES, res, res2, want):
            assert torch.equal(a, w) and torch.equal(b, w), (rep, n)


def test_recorded_backward_in_a_graph():
    t, dims = model(100, [70, 1, 129])
    p = {n: leaf(t[n]) for n in NAMES}  # leaves that no eager graph holds
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(model_loss(p, t, dims), [p[n] for n in NAMES])
    for rep in range(3):
        t["ids"].copy_(randint(-1, 91, (200,), 110 + rep))
        graph.replay()
        torch.cuda.synchronize()
        q = {n: leaf(t[n]) for n in NAMES}
        want = torch.autograd.grad(model_loss(q, t, dims), [q[n] for n in NAMES])
        for n, a, b in zip(NAMES, grads, want):
            assert torch.equal(a, b), (rep, n)


def test_results_do_not_depend_on_what_runs_beside():
    """The same bits from call to call, weight gradients among them."""
    q, k = randn((5000, 12, 64), 120, BF), randn((5000, 4, 64), 121, BF)
    w, rot = randn((64,), 122), lib.Rotation(64)
    first = lib.qk_norm_backward(q * 0.5, k * 0.5, q, k, rot, q_weight=w, k_weight=w)
    side = torch.cuda.Stream()
    x = randn((2048, 2048), 123)
    for _ in range(3):
        with torch.cuda.stream(side):
            x = x @ x * 1e-3
        again = lib.qk_norm_backward(q * 0.5, k * 0.5, q, k, rot, q_weight=w, k_weight=w)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    torch.cuda.synchronize()


def test_gradients_against_differences():
    """Directional differences of the operators' own forward calls, in fp32."""
    q, k, g = randn((40, 2, 32), 130), randn((40, 1, 32), 131), randn((40, 3, 32), 132)
    w, rot, cu = 1 + randn((32,), 133, std=0.2), lib.Rotation(32), cu_of([25, 15])

    def loss(q, k, w):
        a, b = lib.qk_norm_forward(q, k, rot, q_weight=w, k_weight=w, cu_seqlens=cu)
        return (a.double() * g[:, :2]).sum().item() + (b.double() * g[:, 2:]).sum().item()

    dq, dk, dqw, dkw = lib.qk_norm_backward(g[:, :2].contiguous(), g[:, 2:].contiguous(), q, k, rot, q_weight=w,
                                            k_weight=w, cu_seqlens=cu)
    for i, grad in ((0, dq), (1, dk), (2, dqw + dkw)):
        args, h = [q, k, w], 2.0 ** -6
        d = randn(tuple(args[i].shape), 140 + i)
        lo, hi = list(args), list(args)
        lo[i], hi[i] = args[i] - h * d, args[i] + h * d
        diff, want = (loss(*hi) - loss(*lo)) / (2 * h), (grad.double() * d).sum().item()
        # fp32 values of y: each off by 40 u32, divided by 2 h; the differences' own error: h^2 / 6 of third derivatives,
        # below 60 |g d| a head for rows of unit scale
        mass = g.abs().sum().item()
        assert abs(diff - want) <= 40 * 2.0 ** -24 * mass / h + 60 * h * h / 6 * mass, (i, diff, want)
    table, ids, go = randn((9, 16), 150), randint(0, 9, (50,), 151), randn((50, 16), 152)
    d = randn((9, 16), 153)
    dt = lib.embedding_backward(go, ids, 9, scale=0.5)
    diff = ((lib.embedding_forward(table + d, ids, scale=0.5).double() -
             lib.embedding_forward(table, ids, scale=0.5).double()) * go).sum().item()
    assert abs(diff - (dt.double() * d).sum().item()) <= 64 * 2.0 ** -24 * (go.abs().sum().item() * 4)  # linear
