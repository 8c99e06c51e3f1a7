"""Calls of the block's operators at the edges of what their contract allows, on the GPU.

Values are held against the fp64 definitions within block_reference's bounds.
"""
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


def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def run_attention(q, k, v, do, cu):
    dev = [t.to(DEV) for t in (q, k, v, do)]
    out, lse = lib.packed_attention_forward(*dev[:3], cu)
    grads = lib.packed_attention_backward(dev[3], *dev[:3], out, lse, cu)
    torch.cuda.synchronize()
    return dict(zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)))


# ---------------------------------------------- what a mask hides, no one sees --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("extra", [0, 40])  # 40 empty sequences behind: one group of waves a block instead of two
def test_attention_later_tokens_never_reach_earlier_ones(dim, dtype, extra):
    """NaN and infinities in a token's operands reach what its own scores reach, by the formulas, and nothing else:
    no earlier token's out and dq (k, v), no later token's dk and dv (q, dout), no other row (q, dout)."""
    n, H, G = 330, 4, 2
    q, k, v, do = (randn((n, h, dim), 900 + i, dtype) for i, h in enumerate((H, G, G, H)))
    ref = R.attention(q, k, v, [n], dim ** -0.5, do)
    cu = cu_of([n] + [0] * extra)

    def clean(name, got, rows, heads):
        rows = torch.tensor(list(rows), dtype=torch.long)
        for h in heads:
            at = (h, rows) if name == "lse" else (rows, h)
            R.check(f"{name} head {h}", got[name].cpu()[at], *(t[at] for t in ref[name]))

    everything, mine = range(n), [0, 1]  # query heads 0 and 1 read key/value head 0
    for t, bad in ((1, float("nan")), (40, float("inf")), (62, float("nan")), (127, float("-inf")),
                   (130, float("nan")), (255, float("inf")), (n - 1, float("nan"))):
        say(f"[gpu] poisoned token {t} dim {dim} {dtype} extra {extra}: {bad}")
        before, after, others = range(t), range(t + 1, n), [i for i in range(n) if i != t]
        x = v.clone()
        x[t, 0, dim - 3] = bad
        got = run_attention(q, k, x, do, cu)
        clean("lse", got, everything, range(H))
        clean("dv", got, everything, range(G))
        for name in ("out", "dq"):
            clean(name, got, before, mine)
            clean(name, got, everything, [2, 3])
        clean("dk", got, everything, [1])
        assert not torch.isfinite(got["out"][t:, :2, dim - 3].float()).any()
        x = k.clone()
        x[t, 0, 5] = bad
        got = run_attention(q, x, v, do, cu)
        for name in ("out", "dq", "lse"):
            clean(name, got, before, mine)
            clean(name, got, everything, [2, 3])
        x = q.clone()
        x[t, 0, 5] = bad
        got = run_attention(x, k, v, do, cu)
        for name in ("out", "dq", "lse"):
            clean(name, got, others, [0])
            clean(name, got, everything, [1, 2, 3])
        for name in ("dk", "dv"):
            clean(name, got, after, [0])
            clean(name, got, everything, [1])
        x = do.clone()
        x[t, 1, 2] = bad
        got = run_attention(q, k, v, x, cu)
        clean("dq", got, others, [1])
        clean("dq", got, everything, [0, 2, 3])
        for name in ("dk", "dv"):
            clean(name, got, after, [0])
            clean(name, got, everything, [1])
        assert not torch.isfinite(got["dv"][:t + 1, 0, 2].float()).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
@pytest.mark.parametrize("n,H,G,extra", [(33, 2, 1, 0), (65, 2, 2, 0), (300, 4, 2, 0), (300, 4, 2, 40), (1100, 8, 2, 0)])
def test_attention_gradients_of_keys_with_scores_of_minus_infinity(n, H, G, extra, dim, dtype):
    """Such keys have weight 0: their dk and dv are zero, whatever the sequence's length, and all other gradients those
    of keys whose weights vanish (the reference's have scores below -120, and so weights below 1e-50)."""
    q, k, v, do = (randn((n, h, dim), 940 + i, dtype) for i, h in enumerate((H, G, G, H)))
    q[:, :, 0] = q[:, :, 0].abs() + 0.5
    dead = [1, 2, 30, n - 2] + list(range(40, min(n - 3, 200)))
    far = k.clone()
    far[dead, :, 0] = -2.0 ** 12
    k[dead, :, 0] = float("-inf")
    got = run_attention(q, k, v, do, cu_of([n] + [0] * extra))
    ref = R.attention(q, far, v, [n], dim ** -0.5, do, dtype)
    for name in ("dk", "dv"):
        assert (got[name][dead] == 0).all(), name
    for name, x in got.items():
        if name == "dq":  # -inf times a weight of 0: the formula has NaN in this place
            R.check(name, x[..., 1:], *(t[..., 1:] for t in ref[name]))
        else:
            R.check(name, x, *ref[name])


# ------------------------------------------------ operands of one buffer that share nothing --
@pytest.mark.parametrize("layout", ["tokens, heads", "heads, tokens", "tokens, heads, operands"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_operands_between_each_others_rows(layout, dtype):
    """Inputs and outputs of one buffer: the same bits as in buffers of their own, and nothing else is written."""
    n, H, D = 150, 2, 64
    names = ("q", "k", "v", "dout", "out", "dq", "dk", "dv")
    cu = cu_of([100, 50])
    if layout == "tokens, heads":
        buf = randn((n, 8 * H, D), 950, dtype).to(DEV)
        view = {x: buf[:, i * H:(i + 1) * H] for i, x in enumerate(names)}
    elif layout == "heads, tokens":
        buf = randn((8 * H, n, D), 950, dtype).to(DEV)
        view = {x: buf[i * H:(i + 1) * H].transpose(0, 1) for i, x in enumerate(names)}
    else:
        buf = randn((n, H, 8, D), 950, dtype).to(DEV)
        view = {x: buf[:, :, i] for i, x in enumerate(names)}
    q, k, v, do = (view[x].contiguous() for x in names[:4])
    out, lse = lib.packed_attention_forward(q, k, v, cu)
    want = dict(zip(names[5:], lib.packed_attention_backward(do, q, k, v, out, lse, cu)), out=out, q=q, k=k, v=v,
                dout=do)
    _, lse2 = lib.packed_attention_forward(view["q"], view["k"], view["v"], cu, out=view["out"])
    lib.packed_attention_backward(view["dout"], view["q"], view["k"], view["v"], view["out"], lse2, cu,
                                  dq=view["dq"], dk=view["dk"], dv=view["dv"])
    assert torch.equal(lse, lse2)
    for x in names:
        assert torch.equal(view[x], want[x]), x


def test_binding_refuses_outputs_that_share_memory():
    n, H, D = 20, 2, 64
    buf = torch.zeros(n, 4 * H, D, device=DEV, dtype=BF)
    q, k, v = buf[:, :H], buf[:, H:2 * H], buf[:, 2 * H:3 * H]
    cu = cu_of([n])
    out, lse = lib.packed_attention_forward(q, k, v, cu)
    x = torch.zeros(16, 64, device=DEV)
    y, mean, rstd = lib.layer_norm_forward(x)
    calls = [lambda: lib.packed_attention_forward(q, k, v, cu, out=buf[:, 1:1 + H]),
             lambda: lib.packed_attention_forward(q, k, v, cu, out=buf.view(-1)[8:8 + n * H * D].view(n, H, D)),
             lambda: lib.packed_attention_backward(out, q, k, v, out, lse, cu, dk=buf[:, 3 * H - 1:4 * H - 1]),
             lambda: lib.packed_attention_backward(out, q, k, v, out, lse, cu, dq=buf[:, 3 * H:], dv=buf[:, 3 * H:]),
             lambda: lib.layer_norm_forward(x[:8], out=x[1:9]),
             lambda: lib.layer_norm_forward(x[:8, :32], out=x.view(-1)[:256].view(8, 32)),
             lambda: lib.layer_norm_backward(y[:8], x[:8], mean[:8], rstd[:8], dx=y[7:15])]
    for i, call in enumerate(calls):
        with pytest.raises(lib._lib.MuonError, match="overlap"):
            call()
            raise AssertionError(f"call {i} was not refused")


# ------------------------------------------------------------ the largest launches --
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_most_sequences_of_one_launch(dtype):
    """As many sequences as the launch's 2^32 threads allow, nearly all of them empty."""
    n, D = 100, 32
    seqs = (1 << 24) - 2 if dtype == BF else (1 << 23) - 2 - n // 64
    q, k, v, do = (randn((n, 1, D), 960 + i, dtype) for i in range(4))
    cu = torch.zeros(seqs + 1, dtype=torch.int32, device=DEV)
    cu[seqs // 2:] = 40
    cu[-1] = n
    dev = [t.to(DEV) for t in (q, k, v, do)]
    out, lse = lib.packed_attention_forward(*dev[:3], cu)
    grads = lib.packed_attention_backward(dev[3], *dev[:3], out, lse, cu)
    ref = R.attention(q, k, v, [40, 60], D ** -0.5, do)
    for name, got in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *grads)):
        R.check(name, got, *ref[name])
    with pytest.raises(lib._lib.MuonError, match="launch"):
        lib.packed_attention_forward(*dev[:3], torch.zeros(seqs + 2, dtype=torch.int32, device=DEV))


# ---------------------------------------------------------------------- no rows --
@pytest.mark.parametrize("need_weight", [False, True])
@pytest.mark.parametrize("need_bias", [False, True])
def test_layer_norm_gradients_of_an_empty_batch(need_weight, need_bias):
    for shape in ((0, 96), (3, 0, 96)):
        x = torch.empty(shape, device=DEV, dtype=BF)
        y, mean, rstd = lib.layer_norm_forward(x)
        dx, dw, db = lib.layer_norm_backward(y, x, mean, rstd, need_weight=need_weight, need_bias=need_bias)
        assert dx.shape == shape and dx.dtype == BF
        for g, need in ((dw, need_weight), (db, need_bias)):
            assert (g is not None and g.shape == (96,) and (g == 0).all()) if need else g is None


# --------------------------------------------------------------- torch's gradients --
def leaves(*tensors):
    return [t.detach().clone().requires_grad_(True) for t in tensors]


@pytest.mark.parametrize("dtype,pdtype", [(BF, F32), (BF, BF), (F32, F32)])
def test_layer_norm_takes_part_in_autograd(dtype, pdtype):
    x, dy = randn((3, 7, 96), 970, dtype).to(DEV), randn((3, 7, 96), 971, dtype).to(DEV)
    w, b = (1 + randn((96,), 972, std=0.2)).to(pdtype).to(DEV), randn((96,), 973, pdtype).to(DEV)
    y0, mean, rstd = lib.layer_norm_forward(x, w, b)
    assert not y0.requires_grad
    want = lib.layer_norm_backward(dy, x, mean, rstd, w)
    for wanted in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
        args = [t.clone().requires_grad_(bool(n)) for t, n in zip((x, w, b), wanted)]
        y, _, _ = lib.layer_norm_forward(*args)
        assert torch.equal(y, y0)
        y.backward(dy)
        for t, g, n in zip(args, want, wanted):
            assert (t.grad is None) if not n else (t.grad.dtype == t.dtype and torch.equal(t.grad, g.to(t.dtype)))
    xl, = leaves(x)  # without parameters; the gradient of a sum repeats one value; a gradient of other strides
    y, mean, rstd = lib.layer_norm_forward(xl)
    y.sum().backward()
    assert torch.equal(xl.grad, lib.layer_norm_backward(torch.ones_like(x), x, mean, rstd)[0])
    xl, = leaves(x)
    lib.layer_norm_forward(xl, w, b)[0].transpose(0, 2).backward(dy.transpose(0, 2))
    assert torch.equal(xl.grad, want[0])
    with torch.no_grad():
        y, _, _ = lib.layer_norm_forward(xl, w, b)
    assert not y.requires_grad and torch.equal(y, y0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_takes_part_in_autograd(dtype):
    T, H, G, D = 150, 4, 2, 64
    cu = cu_of([100, 45])
    qkv, do = randn((T, H + 2 * G, D), 980, dtype).to(DEV), randn((T, H, D), 981, dtype).to(DEV)
    cut = lambda t: (t[:, :H], t[:, H:H + G], t[:, H + G:])  # noqa: E731
    out0, lse0 = lib.packed_attention_forward(*cut(qkv), cu)
    want = lib.packed_attention_backward(do, *cut(qkv), out0, lse0, cu)
    leaf, = leaves(qkv)  # slices of one projection
    out, lse = lib.packed_attention_forward(*cut(leaf), cu)
    assert torch.equal(out, out0) and torch.equal(lse, lse0)
    out.backward(do)
    assert torch.equal(leaf.grad, torch.cat(want, 1))
    for wanted in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)):
        args = [t.clone().requires_grad_(bool(n)) for t, n in zip(cut(qkv), wanted)]
        lib.packed_attention_forward(*args, cu)[0].backward(do)
        for t, g, n in zip(args, want, wanted):
            assert (t.grad is None) if not n else torch.equal(t.grad, g)
    for weight in (torch.ones((), device=DEV, dtype=dtype).expand(T, H, D), do.transpose(0, 1).contiguous().transpose(0, 1),
                   torch.cat([do[..., :1], do], 2)[..., 1:], do[:, :1].expand(T, H, D)):
        leaf, = leaves(qkv)
        lib.packed_attention_forward(*cut(leaf), cu)[0].backward(weight)
        g = lib.packed_attention_backward(weight.contiguous(), *cut(qkv), out0, lse0, cu)
        assert torch.equal(leaf.grad, torch.cat(g, 1))
    k1, v1 = leaves(qkv[:, H:H + 1], qkv[:, H + 1:H + 2])  # one head's memory for all: its gradient is their sum
    out, _ = lib.packed_attention_forward(qkv[:, :H], k1.expand(T, H, D), v1.expand(T, H, D), cu)
    out.backward(do)
    ref = R.attention(qkv[:145, :H].cpu(), k1.detach()[:145].cpu(), v1.detach()[:145].cpu(), [100, 45], D ** -0.5,
                      do[:145].cpu())
    for g, name in ((k1.grad, "dk"), (v1.grad, "dv")):
        value, bound = ref[name]
        # four heads' results, each rounded, and torch's sum of them in this type
        loose = 8 * R.unit(dtype) * (value.abs() + R.attention(
            qkv[:145, :H].abs().cpu(), k1.detach()[:145].abs().cpu(), v1.detach()[:145].abs().cpu(), [100, 45],
            D ** -0.5, do[:145].abs().cpu())["dv"][0].abs().amax())
        R.check(name, g[:145], value, bound + loose)


def test_gradients_that_would_be_lost_are_refused():
    x, w = leaves(randn((6, 64), 990).to(DEV), randn((64,), 991).to(DEV))
    q, k, v = leaves(*(randn((20, 2, 32), 992 + i).to(DEV) for i in range(3)))
    cu = cu_of([20])
    y, mean, rstd = lib.layer_norm_forward(x, w)
    out, lse = lib.packed_attention_forward(q, k, v, cu)
    for loss in (mean.sum() + y.sum(), rstd.sum(), lse.square().sum(), out.sum() + lse.sum()):
        with pytest.raises(RuntimeError, match="pass no gradient on"):
            torch.autograd.grad(loss, [x, w, q, k, v], retain_graph=True, allow_unused=True)
    for z, t in ((y, x), (out, q)):  # differentiable once
        g, = torch.autograd.grad(z.square().sum(), t, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
    buf = torch.zeros(6, 64, device=DEV)
    with pytest.raises(ValueError, match="recorded"):
        lib.layer_norm_forward(x, w, out=buf)
    with pytest.raises(ValueError, match="recorded"):
        lib.packed_attention_forward(q, k, v, cu, lse=torch.zeros(2, 20, device=DEV))
    xd, qd, kd, vd = (t.detach() for t in (x, q, k, v))
    st = lib.layer_norm_forward(xd)[1:]
    o, l = lib.packed_attention_forward(qd, kd, vd, cu)
    for call in (lambda: lib.layer_norm_forward(xd, out=x), lambda: lib.layer_norm_backward(buf, xd, *st, dx=x * 1),
                 lambda: lib.packed_attention_forward(qd, kd, vd, cu, out=q * 1),
                 lambda: lib.packed_attention_backward(o, qd, kd, vd, o, l, cu, dk=k * 1)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            lib.layer_norm_forward(torch.autograd.forward_ad.make_dual(xd, buf))
        with pytest.raises((RuntimeError, NotImplementedError)):
            lib.packed_attention_forward(torch.autograd.forward_ad.make_dual(qd, kd), kd, vd, cu)
    with pytest.raises(RuntimeError):
        torch.vmap(lambda t: lib.layer_norm_forward(t)[0])(xd.view(2, 3, 64))
    with pytest.raises(RuntimeError):
        torch.func.grad(lambda t: lib.layer_norm_forward(t)[0].sum())(xd)


def test_a_graph_that_saved_a_given_output_notices_that_it_was_written():
    x = randn((6, 64), 995).to(DEV)
    q = randn((20, 2, 32), 996).to(DEV)
    cu = cu_of([20])
    y, mean, rstd = lib.layer_norm_forward(x)
    out, lse = lib.packed_attention_forward(q, q, q, cu)
    writes = [((6, 64), lambda t: lib.layer_norm_forward(x, out=t)),
              ((6, 64), lambda t: lib.layer_norm_backward(y, x, mean, rstd, dx=t)),
              ((20, 2, 32), lambda t: lib.packed_attention_forward(q, q, q, cu, out=t)),
              ((2, 20), lambda t: lib.packed_attention_forward(q, q, q, cu, lse=t)),
              ((20, 2, 32), lambda t: lib.packed_attention_backward(out, q, q, q, out, lse, cu, dq=t)),
              ((20, 2, 32), lambda t: lib.packed_attention_backward(out, q, q, q, out, lse, cu, dk=t)),
              ((20, 2, 32), lambda t: lib.packed_attention_backward(out, q, q, q, out, lse, cu, dv=t))]
    for i, (shape, write) in enumerate(writes):
        leaf, saved = torch.ones(shape, device=DEV, requires_grad=True), torch.ones(shape, device=DEV)
        loss = (leaf * saved).sum()
        write(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
            raise AssertionError(f"write {i} went unnoticed")
    with torch.inference_mode():
        given = torch.empty_like(x)
        assert torch.equal(lib.layer_norm_forward(x, out=given)[0], y)


def block_loss(t, p):
    """A block's forward pass on recorded tensors, as a model calls the operators."""
    H, D, T = 4, 64, t["x"].shape[0]
    y, _, _ = lib.layer_norm_forward(p["x"], p["w"], p["b"])
    qkv = (y @ p["wqkv"]).view(T, 3 * H, D)
    o, _ = lib.packed_attention_forward(qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:], t["cu"])
    return (o.reshape(T, H * D) @ p["wo"] * t["dout"]).sum()


def block_data(lengths, seed):
    T, width = sum(lengths), 256
    t = dict(x=randn((T, width), seed), w=1 + randn((width,), seed + 1, std=0.1), b=randn((width,), seed + 2),
             wqkv=randn((width, 3 * width), seed + 3, std=width ** -0.5), wo=randn((width, width), seed + 4, std=width ** -0.5),
             dout=randn((T, width), seed + 5))
    return {k: v.to(DEV) for k, v in t.items()}


def test_block_under_autograd_on_streams_and_in_a_graph():
    """A block recorded by torch against fp64 autograd, the same on another stream, and captured forward and backward."""
    lengths, names = [70, 1, 129], ("x", "w", "b", "wqkv", "wo")
    t = block_data(lengths, 1000)
    t["cu"] = cu_of(lengths)
    p = {n: leaves(t[n])[0] for n in names}
    block_loss(t, p).backward()
    got = {n: p[n].grad.clone() for n in names}
    c = {n: t[n].double().cpu().requires_grad_(n in names) for n in (*names, "dout")}
    T, H, D = sum(lengths), 4, 64
    y = torch.nn.functional.layer_norm(c["x"], (H * D,), c["w"], c["b"], 1e-5)
    qkv = (y @ c["wqkv"]).view(T, 3 * H, D).permute(1, 0, 2)
    doc = torch.repeat_interleave(torch.arange(len(lengths)), torch.tensor(lengths))
    i = torch.arange(T)
    hidden = (doc[:, None] != doc[None]) | (i[None] > i[:, None])
    s = (qkv[:H] @ qkv[H:2 * H].transpose(1, 2) * D ** -0.5).masked_fill(hidden, float("-inf"))
    o = (torch.softmax(s, 2) @ qkv[2 * H:]).permute(1, 0, 2).reshape(T, H * D)
    (o @ c["wo"] * c["dout"]).sum().backward()
    for n in names:
        rel = ((got[n].double().cpu() - c[n].grad).norm() / c[n].grad.norm()).item()
        say(f"[gpu] block under autograd d{n}: rel {rel:.2e}")
        assert rel <= 5 * 800 * 2.0 ** -24, (n, rel)  # five chained fp32 sums of at most 800 terms
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p2 = {n: leaves(t[n])[0] for n in names}
        block_loss(t, p2).backward()
    side.synchronize()
    for n in names:
        assert torch.equal(p2[n].grad, got[n]), n
    del p2
    p3 = {n: leaves(t[n])[0] for n in names}  # leaves that no eager graph holds
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(block_loss(t, p3), [p3[n] for n in names])
    for rep in range(3):
        with torch.no_grad():
            p3["x"].copy_(randn(tuple(t["x"].shape), 1010 + rep).to(DEV))
        t["cu"].copy_(cu_of([[70, 1, 129], [200, 0, 0], [64, 64, 72]][rep]))
        graph.replay()
        torch.cuda.synchronize()
        q = {n: leaves(p3[n])[0] for n in names}
        want = torch.autograd.grad(block_loss(t, q), [q[n] for n in names])
        for n, a, b in zip(names, grads, want):
            assert torch.equal(a, b), (rep, n)


# ------------------------------------------------------- groups split over blocks --
def splits_of(T, seqs, H, G, D, dtype):
    """The parts that a group's query heads are split into, from the workspace: two rows' words, and the parts."""
    d = lib._lib.AttentionDesc(T, seqs, H, G, D, int(dtype == BF), 1.0, 0)
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    rest = lib._lib.load().muon_attention_workspace_size(d) - 2 * up(H * T * 4) - 256
    return max(1, rest // (T * G * 2 * D * 4))


def check_attention(lengths, H, G, D, dtype, seed, tail=0):
    T, n = sum(lengths) + tail, sum(lengths)
    q, k, v, do = (randn((T, h, D), seed + i, dtype) for i, h in enumerate((H, G, G, H)))
    dev = [t.to(DEV) for t in (q, k, v, do)]
    for t in dev:
        t[n:] = float("nan")  # never read
    got = run_attention(*dev, cu_of(lengths))
    ref = R.attention(q, k, v, lengths, D ** -0.5, do)
    for name, x in got.items():
        R.check(name, x, *ref[name])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G", [(8, 2), (6, 3), (9, 3)])
@pytest.mark.parametrize("D", [32, 64, 80, 128])
def test_attention_split_groups(H, G, D, dtype):
    """Partial dK and dV of several key/value heads, summed by a launch of their own."""
    for lengths, tail in (([1100], 0), ([1300], 77)):
        splits = splits_of(sum(lengths) + tail, 1, H, G, D, dtype)
        say(f"[gpu] split groups {lengths} tail {tail} heads {H}/{G} dim {D} {dtype}: {splits} parts")
        assert splits == H // G
        check_attention(lengths, H, G, D, dtype, 1100, tail)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_split_groups_of_many_heads(dtype):
    """Splits in grids that take one group of waves a block (bf16), of two sequences, and of groups in parts of
    several heads."""
    for lengths, H, G, parts in (([400, 650], 192, 48, 4), ([900], 64, 16, 4), ([700, 500], 256, 32, 4)):
        splits = splits_of(sum(lengths), len(lengths), H, G, 32, dtype)
        say(f"[gpu] split groups {lengths} heads {H}/{G} {dtype}: {splits} parts")
        assert splits == parts
        check_attention(lengths, H, G, 32, dtype, 1200)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_split_groups_see_no_masked_nan(D, dtype):
    n, H, G, t = 1100, 8, 2, 601
    assert splits_of(n, 1, H, G, D, dtype) == 4
    q, k, v, do = (randn((n, h, D), 1300 + i, dtype) for i, h in enumerate((H, G, G, H)))
    ref = R.attention(q, k, v, [n], D ** -0.5, do)
    q[t, 5, 3], do[t, 6, 7] = float("nan"), float("inf")  # heads of key/value head 1
    got = run_attention(q, k, v, do, cu_of([n]))
    for name in ("dk", "dv"):
        x = got[name].cpu()
        R.check(name, x[:, :1], *(r[:, :1] for r in ref[name]))
        R.check(name, x[t + 1:, 1], *(r[t + 1:, 1] for r in ref[name]))
    assert not torch.isfinite(got["dv"][:t + 1, 1, 7].float()).any()


# -------------------------------------------------------------- searches for a tile --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("seqs", [63, 64, 65, 128, 129, 192, 193, 255, 256, 257, 300])
def test_attention_sequence_counts(seqs, dtype):
    """Around every step of the searches for a block's tile: short sequences, empty ones, and some of several tiles."""
    lengths = [129 + i * 53 % 272 if i % 29 == 3 else i * 37 % 41 for i in range(seqs)]
    check_attention(lengths, 2, 1, 32, dtype, 1400, tail=seqs % 3 * 70)
    check_attention(lengths[::-1], 2, 2, 32, dtype, 1410, tail=0)


def test_binding_refuses_outputs_that_are_no_tensors():
    x, q, cu = torch.zeros(4, 64, device=DEV), torch.zeros(8, 2, 64, device=DEV), cu_of([8])
    y, mean, rstd = lib.layer_norm_forward(x)
    out, lse = lib.packed_attention_forward(q, q, q, cu)
    for bad in ("out", 3.0, [1]):
        for call in (lambda: lib.layer_norm_forward(x, out=bad), lambda: lib.layer_norm_backward(y, x, mean, rstd, dx=bad),
                     lambda: lib.layer_norm_forward(x, bad), lambda: lib.layer_norm_forward(bad),
                     lambda: lib.packed_attention_forward(q, q, q, cu, out=bad),
                     lambda: lib.packed_attention_forward(q, q, q, cu, lse=bad),
                     lambda: lib.packed_attention_forward(q, bad, q, cu),
                     lambda: lib.packed_attention_backward(out, q, q, q, out, lse, cu, dk=bad)):
            with pytest.raises(ValueError, match="not a device tensor"):
                call()


def test_attention_pack_of_65536_tokens():
    """The tokens of a long training pack, two sequences of them beside a short one, with a split group: each kilotoken
    of every result against fp64, which is taken in strips on the GPU."""
    lengths, H, D = [40000, 37, 25499], 2, 64
    T = sum(lengths)
    assert T == 65536 and splits_of(T, 3, H, 1, D, BF) == 2
    q, k, v, do = (randn((T, h, D), 1500 + i, BF).to(DEV) for i, h in enumerate((H, 1, 1, H)))
    cu = cu_of(lengths)
    got = run_attention(q, k, v, do, cu)
    want = {n: torch.zeros(got[n].shape, dtype=torch.float64, device=DEV) for n in got}
    a = 0
    for n in lengths:
        kk, vv = k[a:a + n, 0].double(), v[a:a + n, 0].double()
        for h in range(H):
            for r in range(0, n, 2500):
                z = min(n, r + 2500)
                qq, dd = q[a + r:a + z, h].double(), do[a + r:a + z, h].double()
                s = (qq @ kk[:z].t().contiguous()) * D ** -0.5
                s.masked_fill_(torch.ones_like(s, dtype=torch.bool).triu_(r + 1), float("-inf"))
                lse = torch.logsumexp(s, 1)
                p = torch.exp_(s.sub_(lse[:, None]))
                out = p @ vv[:z]
                ds = (dd @ vv[:z].t().contiguous()).sub_((dd * out).sum(1, keepdim=True)).mul_(p).mul_(D ** -0.5)
                want["lse"][h, a + r:a + z] = lse
                want["out"][a + r:a + z, h] = out
                want["dq"][a + r:a + z, h] = ds @ kk[:z]
                want["dk"][a:a + z, 0] += ds.t().contiguous() @ qq
                want["dv"][a:a + z, 0] += p.t().contiguous() @ dd
        a += n
    # lse: fp32 scores of about 10 and sums of 40000 terms, 16 at a time
    assert (got["lse"].double() - want["lse"]).abs().max().item() <= 1e-4
    for name in ("out", "dq", "dk", "dv"):
        for r in range(0, T, 1024):
            x, y = got[name][r:r + 1024].double(), want[name][r:r + 1024]
            rel = ((x - y).norm() / y.norm()).item()
            # roundings of p or ds, of delta's output, and of the result, each at most 2^-8
            assert rel <= 3 * 2.0 ** -8, (name, r, rel)
