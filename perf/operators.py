"""Workloads of the transformer block's operators: layer norm and packed causal attention, each forward
and as a training step (forward, then backward), in their plain form and through the library.

``prepare(case, seed)`` makes the inputs on the GPU, ``run(state)`` is one pass: with ``own`` false in
elementary torch operations held in 32 bits, with ``own`` true through ``muon_newton_schulz_03_amd``.
``exact`` evaluates the definitions in 64 bits, ``work`` counts the bytes and operations a pass cannot do
without.  The shapes follow the GPT-2-small block whose hidden matrices the Muon step trains (width 768,
12 heads of 64) and generic wider ones with grouped heads of 128.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_EPS = 1e-5


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one short document through one norm: launch latency
        dict(name="norm_fwd_short", op="norm", train=False, rows=64, cols=768, dtype="bf16", params="f32", bias=True),
        # the norm of a 65,536-token pack at width 768
        dict(name="norm_fwd_pack", op="norm", train=False, rows=65536, cols=768, dtype="bf16", params="f32", bias=True),
        # the same norm in a training step
        dict(name="norm_train_pack", op="norm", train=True, rows=65536, cols=768, dtype="bf16", params="f32",
             bias=True),
        # an odd width (no row but the first is aligned to a vector) in 32 bits
        dict(name="norm_train_odd", op="norm", train=True, rows=4099, cols=1001, dtype="f32", params="f32", bias=True),
        # a wide model's norm, weights in bf16, no bias
        dict(name="norm_train_wide", op="norm", train=True, rows=8192, cols=4096, dtype="bf16", params="bf16",
             bias=False),
        # one short document: launch latency
        dict(name="attn_fwd_short", op="attn", train=False, tokens=128, seqs=1, pack=1, heads=12, kv_heads=12, dim=64,
             dtype="bf16"),
        # ragged documents packed into one training sequence, 12 heads of 64
        dict(name="attn_fwd_pack", op="attn", train=False, tokens=16384, seqs=24, pack=2, heads=12, kv_heads=12,
             dim=64, dtype="bf16"),
        # one long prompt with grouped heads of 128
        dict(name="attn_fwd_long", op="attn", train=False, tokens=16384, seqs=1, pack=3, heads=16, kv_heads=4, dim=128,
             dtype="bf16"),
        # the training step of the packed documents
        dict(name="attn_train_pack", op="attn", train=True, tokens=16384, seqs=24, pack=2, heads=12, kv_heads=12,
             dim=64, dtype="bf16"),
        # the training step of one long sequence with grouped heads of 128
        dict(name="attn_train_long", op="attn", train=True, tokens=8192, seqs=1, pack=4, heads=16, kv_heads=4, dim=128,
             dtype="bf16"),
        # few tokens in very short and single-token documents, shared heads, a head size between the usual ones
        dict(name="attn_train_odd", op="attn", train=True, tokens=1023, seqs=37, pack=5, heads=6, kv_heads=2, dim=80,
             dtype="bf16"),
        # the 32-bit path, as used to check a training run
        dict(name="attn_train_f32", op="attn", train=True, tokens=2048, seqs=5, pack=6, heads=12, kv_heads=12, dim=64,
             dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    train = rng.random() < 0.6
    if rng.random() < 0.45:
        cols = _log_int(rng, 32, 8192)
        if rng.random() < 0.6:
            cols = -(-cols // 8) * 8
        rows = _log_int(rng, 1, max(1, min(65536, (1 << 25) // cols)))
        return dict(op="norm", train=train, rows=rows, cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    params=rng.choice(["f32", "bf16"]), bias=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads, group = rng.choice([(1, 8), (2, 3), (2, 4), (4, 1), (4, 4), (12, 1), (8, 2), (16, 1)])
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128])
    tokens = _log_int(rng, 1, 2048 if dtype == "f32" else 8192)
    return dict(op="attn", train=train, tokens=tokens, seqs=_log_int(rng, 1, min(64, tokens)),
                pack=rng.randrange(1 << 30), heads=kv_heads * group, kv_heads=kv_heads, dim=dim, dtype=dtype)


def _lengths(case):
    """The documents' lengths: ragged over a factor of 64, at least one token each, and summing to the tokens."""
    n, total = case["seqs"], case["tokens"]
    rng = random.Random(case["pack"])
    share = [math.exp(rng.uniform(0.0, math.log(64.0))) for _ in range(n)]
    part, cuts, at = sum(share), [0], 0.0
    for s in share:
        at += s / part * (total - n)
        cuts.append(int(round(at)))
    cuts[-1] = total - n
    return [b - a + 1 for a, b in zip(cuts, cuts[1:])]


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    st = dict(case)
    if case["op"] == "norm":
        r, c, pt = case["rows"], case["cols"], _DTYPES[case["params"]]
        # a residual stream: tokens of different scale, a common offset in each feature
        st["x"] = (randn(r, c) * torch.exp(0.5 * randn(r, 1)) + 0.5 * randn(1, c)).to(dt)
        st["weight"] = (1.0 + 0.2 * randn(c)).to(pt)
        st["bias"] = (0.1 * randn(c)).to(pt) if case["bias"] else None
        if case["train"]:
            st["dy"] = randn(r, c).to(dt)
        return st
    t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    # the output of one projection: query heads, then key heads, then value heads
    st["qkv"] = randn(t, h + 2 * g, d).to(dt)
    cu = [0]
    for n in _lengths(case):
        cu.append(cu[-1] + n)
    st["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["train"]:
        st["dout"] = randn(t, h, d).to(dt)
    return st


# ------------------------------------------------------------ plain forms --
def _norm_plain(st):
    x = st["x"].float()
    w = st["weight"].float()
    mean = x.mean(dim=1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt(xc.square().mean(dim=1, keepdim=True) + _EPS)
    xh = xc * rstd
    y = xh * w
    if st["bias"] is not None:
        y = y + st["bias"].float()
    out = dict(y=y.to(st["x"].dtype), mean=mean.squeeze(1), rstd=rstd.squeeze(1))
    if st["train"]:
        dy = st["dy"].float()
        gw = dy * w
        dx = rstd * (gw - gw.mean(dim=1, keepdim=True) - xh * (gw * xh).mean(dim=1, keepdim=True))
        out["dx"] = dx.to(st["x"].dtype)
        out["dweight"] = (dy * xh).sum(dim=0)
        if st["bias"] is not None:
            out["dbias"] = dy.sum(dim=0)
    return out


def _attn_plain(st):
    qkv, h, g, d = st["qkv"], st["heads"], st["kv_heads"], st["dim"]
    t, grp, scale = qkv.shape[0], h // g, 1.0 / math.sqrt(d)
    f = qkv.float()
    q = f[:, :h].reshape(t, g, grp, d).permute(1, 2, 0, 3).reshape(g, grp * t, d)  # one product per shared head
    k = f[:, h:h + g].permute(1, 0, 2).contiguous()
    v = f[:, h + g:].permute(1, 0, 2).contiguous()
    pos = torch.arange(t, device=qkv.device, dtype=torch.int32)
    doc = torch.bucketize(pos, st["cu_seqlens"][1:], right=True)
    hidden = (doc[:, None] != doc[None, :]) | (pos[None, :] > pos[:, None])
    s = torch.matmul(q, k.transpose(1, 2).contiguous()).view(g, grp, t, t).mul_(scale)
    s.masked_fill_(hidden, float("-inf"))
    top = s.amax(dim=3, keepdim=True)
    p = s.sub_(top).exp_()
    norm = p.sum(dim=3, keepdim=True)
    p.div_(norm)
    o = torch.matmul(p.view(g, grp * t, t), v)
    lse = (top + torch.log(norm)).reshape(h, t)

    def rows(z):  # (g, grp * t, d) -> (t, h, d)
        return z.view(g, grp, t, d).permute(2, 0, 1, 3).reshape(t, h, d)

    out = dict(out=rows(o).to(qkv.dtype), lse=lse)
    if st["train"]:
        do = st["dout"].float().reshape(t, g, grp, d).permute(1, 2, 0, 3).reshape(g, grp * t, d)
        p = p.view(g, grp * t, t)
        dv = torch.matmul(p.transpose(1, 2), do)
        ds = torch.matmul(do, v.transpose(1, 2).contiguous())
        ds.sub_((do * o).sum(dim=2, keepdim=True)).mul_(p).mul_(scale)
        dq = rows(torch.matmul(ds, k))
        dk = torch.matmul(ds.transpose(1, 2), q)
        out["dqkv"] = torch.cat([dq, dk.permute(1, 0, 2), dv.permute(1, 0, 2)], dim=1).to(qkv.dtype)
    return out


# ---------------------------------------------------------- library calls --
def _norm_own(st):
    import muon_newton_schulz_03_amd as lib

    y, mean, rstd = lib.layer_norm_forward(st["x"], st["weight"], st["bias"], eps=_EPS)
    out = dict(y=y, mean=mean, rstd=rstd)
    if st["train"]:
        dx, dw, db = lib.layer_norm_backward(st["dy"], st["x"], mean, rstd, st["weight"],
                                             need_bias=st["bias"] is not None)
        out["dx"], out["dweight"] = dx, dw
        if db is not None:
            out["dbias"] = db
    return out


def _attn_own(st):
    import muon_newton_schulz_03_amd as lib

    qkv, h, g = st["qkv"], st["heads"], st["kv_heads"]
    q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    o, lse = lib.packed_attention_forward(q, k, v, st["cu_seqlens"])
    out = dict(out=o, lse=lse)
    if st["train"]:
        dqkv = torch.empty_like(qkv)
        lib.packed_attention_backward(st["dout"], q, k, v, o, lse, st["cu_seqlens"], dq=dqkv[:, :h],
                                      dk=dqkv[:, h:h + g], dv=dqkv[:, h + g:])
        out["dqkv"] = dqkv
    return out


def run(state):
    if state["op"] == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    return _attn_own(state) if own else _attn_plain(state)


# ------------------------------------------------------------ cost, truth --
def work(case):
    b = _BYTES[case["dtype"]]
    if case["op"] == "norm":
        r, c, pb = case["rows"], case["cols"], _BYTES[case["params"]]
        n = r * c
        params = c * pb * (2 if case["bias"] else 1)
        if not case["train"]:
            return {"bytes": 2 * n * b + params + 8 * r, "flops": 7 * n}
        return {"bytes": 4 * n * b + params + 8 * r + 4 * c * (2 if case["bias"] else 1), "flops": 20 * n}
    t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
    qkv, o = t * (h + 2 * g) * d * b, t * h * d * b
    if not case["train"]:
        return {"bytes": qkv + o + 4 * h * t, "flops": 4 * d * h * pairs}
    # products: scores, output; scores and dP again, and the gradients of Q, K and V
    return {"bytes": 2 * qkv + 2 * o + 4 * h * t, "flops": 14 * d * h * pairs}


def _norm_exact(st):
    x, dy = st["x"].double(), st["dy"].double() if st["train"] else None
    n = x.shape[1]
    mean = x.sum(1) / n
    var = (x * x).sum(1) / n - mean * mean
    rstd = (var + _EPS).pow(-0.5)
    xh = (x - mean[:, None]) * rstd[:, None]
    w = st["weight"].double()
    shift = 0.0 if st["bias"] is None else st["bias"].double()
    out = dict(y=torch.addcmul(torch.zeros_like(xh) + shift, xh, w), mean=mean, rstd=rstd)
    if dy is not None:
        e = dy * w
        c1 = e.sum(1, keepdim=True) / n
        c2 = (e * xh).sum(1, keepdim=True) / n
        out["dx"] = (e - c1 - c2 * xh) * rstd[:, None]
        out["dweight"] = (dy * xh).sum(0)
        if st["bias"] is not None:
            out["dbias"] = dy.sum(0)
    return out


def _attn_exact(st):
    """Document by document and head by head, over strips of query rows."""
    qkv = st["qkv"].double()
    h, g, d = st["heads"], st["kv_heads"], st["dim"]
    t, scale = qkv.shape[0], d ** -0.5
    o = torch.zeros(t, h, d, dtype=torch.float64, device=qkv.device)
    lse = torch.zeros(h, t, dtype=torch.float64, device=qkv.device)
    grad = torch.zeros_like(qkv)
    do = st["dout"].double() if st["train"] else None
    lo = 0
    for n in _lengths(st):
        seq = slice(lo, lo + n)
        for i in range(h):
            q, k, v = qkv[seq, i], qkv[seq, h + i * g // h], qkv[seq, h + g + i * g // h]
            for a in range(0, n, 2048):
                z = min(n, a + 2048)
                s = (q[a:z] @ k[:z].T) * scale
                s += torch.full_like(s, float("-inf")).triu(a + 1)
                strip = torch.logsumexp(s, dim=1)
                p = torch.exp(s - strip[:, None])
                lse[i, lo + a:lo + z] = strip
                o[lo + a:lo + z, i] = p @ v[:z]
                if do is None:
                    continue
                gi = do[lo + a:lo + z, i]
                dp = gi @ v[:z].T
                ds = p * (dp - (dp * p).sum(1, keepdim=True)) * scale
                grad[lo + a:lo + z, i] = ds @ k[:z]
                grad[lo:lo + z, h + i * g // h] += ds.T @ q[a:z]
                grad[lo:lo + z, h + g + i * g // h] += p.T @ gi
        lo += n
    out = dict(out=o, lse=lse)
    if do is not None:
        out["dqkv"] = grad
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return _norm_exact(st) if case["op"] == "norm" else _attn_exact(st)
