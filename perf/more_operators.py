"""Workloads of the operators between the token ids and the block's attention: the embedding lookup with its
gradient, and the norm of queries and keys with the position rotation, each forward and as a training step
(forward, then backward), in their plain form and through the library.

``prepare(case, seed)`` makes the inputs on the GPU, ``run(state)`` is one pass: with ``own`` false in
elementary torch operations held in 32 bits (angles in 64), with ``own`` true through
``muon_newton_schulz_03_amd``.  ``exact`` evaluates the definitions in 64 bits, ``work`` counts the bytes and
operations a pass cannot do without.  The shapes follow the GPT-2-small block whose hidden matrices the Muon
step trains (width 768, 12 heads of 64, a vocabulary of 50257 or padded to 50304) and generic wider ones.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_INDEX = {"i32": torch.int32, "i64": torch.int64}
_EPS = 1e-6
_BASE = 10000.0


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one short document through the token table: launch latency
        dict(name="embed_fwd_short", op="embed", train=False, tokens=64, vocab=50304, cols=768, ids="i64", freq="words",
             pad=0.0, table="bf16", dtype="bf16", scale=1.0),
        # a 65,536-token pack through the token table
        dict(name="embed_fwd_pack", op="embed", train=False, tokens=65536, vocab=50304, cols=768, ids="i64",
             freq="words", pad=0.0, table="bf16", dtype="bf16", scale=27.7),
        # a training step on few tokens: what it writes is nearly all zeros
        dict(name="embed_train_short", op="embed", train=True, tokens=500, vocab=50304, cols=768, ids="i64",
             freq="words", pad=0.0, table="bf16", dtype="bf16", scale=1.0),
        # the training step of the pack
        dict(name="embed_train_pack", op="embed", train=True, tokens=65536, vocab=50304, cols=768, ids="i64",
             freq="words", pad=0.0, table="bf16", dtype="bf16", scale=27.7),
        # a table of hashed token pairs, larger and hit evenly; 32-bit weights under bf16 activations
        dict(name="embed_train_hash", op="embed", train=True, tokens=32768, vocab=251520, cols=128, ids="i32",
             freq="even", pad=0.0, table="f32", dtype="bf16", scale=0.25),
        # an odd width and vocabulary in 32 bits, a tenth of the batch padding
        dict(name="embed_train_odd", op="embed", train=True, tokens=4099, vocab=50257, cols=1001, ids="i32",
             freq="words", pad=0.1, table="f32", dtype="f32", scale=1.0),
        # one new token for each of 64 running sequences, at positions of their own: launch latency
        dict(name="qk_fwd_step", op="qk", train=False, tokens=64, seqs=0, pack=1, heads=12, kv_heads=12, dim=64,
             rotary=64, pairs="halves", weights=None, dtype="bf16"),
        # a 65,536-token pack of ragged documents
        dict(name="qk_fwd_pack", op="qk", train=False, tokens=65536, seqs=90, pack=2, heads=12, kv_heads=12, dim=64,
             rotary=64, pairs="halves", weights=None, dtype="bf16"),
        # the training step of a smaller pack
        dict(name="qk_train_pack", op="qk", train=True, tokens=16384, seqs=24, pack=3, heads=12, kv_heads=12, dim=64,
             rotary=64, pairs="halves", weights=None, dtype="bf16"),
        # the training step of one long sequence, grouped heads of 128 with learned weights
        dict(name="qk_train_long", op="qk", train=True, tokens=16384, seqs=1, pack=4, heads=32, kv_heads=8, dim=128,
             rotary=128, pairs="halves", weights="bf16", dtype="bf16"),
        # few tokens in very short documents, a head size between the usual ones, rotated in part, neighbouring pairs
        dict(name="qk_train_odd", op="qk", train=True, tokens=1023, seqs=37, pack=5, heads=6, kv_heads=2, dim=80,
             rotary=32, pairs="neighbours", weights="f32", dtype="bf16"),
        # the 32-bit path, as used to check a training run
        dict(name="qk_train_f32", op="qk", train=True, tokens=2048, seqs=5, pack=6, heads=12, kv_heads=12, dim=64,
             rotary=64, pairs="halves", weights="f32", dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    train = rng.random() < 0.6
    if rng.random() < 0.5:
        cols = _log_int(rng, 16, 4096)
        if rng.random() < 0.6:
            cols = -(-cols // 8) * 8
        table = rng.choice(["bf16", "bf16", "f32"])
        return dict(op="embed", train=train, tokens=_log_int(rng, 1, max(1, min(65536, (1 << 24) // cols))),
                    vocab=_log_int(rng, 64, min(262144, (1 << 25) // cols)), cols=cols, ids=rng.choice(["i32", "i64"]),
                    freq=rng.choice(["words", "words", "even"]), pad=rng.choice([0.0, 0.0, 0.2]), table=table,
                    dtype=rng.choice(["bf16", table]), scale=rng.choice([1.0, 0.25, round(math.sqrt(cols), 1)]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads, group = rng.choice([(1, 8), (2, 3), (2, 4), (4, 1), (4, 4), (12, 1), (8, 2), (16, 1), (8, 4)])
    dim = rng.choice([32, 64, 64, 80, 96, 128, 128])
    heads = kv_heads * group
    tokens = _log_int(rng, 1, min(32768, (1 << 24) // ((heads + kv_heads) * dim)))
    return dict(op="qk", train=train, tokens=tokens, seqs=rng.choice([0, _log_int(rng, 1, min(64, tokens))]),
                pack=rng.randrange(1 << 30), heads=heads, kv_heads=kv_heads, dim=dim,
                rotary=rng.choice([dim, dim, dim // 2, 16]), pairs=rng.choice(["halves", "halves", "neighbours"]),
                weights=rng.choice([None, "f32", "bf16"]), dtype=dtype)


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


def _frequency(case):
    """How often each rank of the vocabulary comes up: as words do (Zipf's law), or evenly."""
    v = case["vocab"]
    p = 1.0 / (np.arange(v) + 2.7) if case["freq"] == "words" else np.ones(v)
    return p / p.sum()


def _padding(case):
    return int(case["tokens"] * case["pad"])


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    st = dict(case)
    t = case["tokens"]
    if case["op"] == "embed":
        v, c = case["vocab"], case["cols"]
        st["weight"] = (randn(v, c) * (1.0 if case["scale"] < 1.0 else 0.02)).to(_DTYPES[case["table"]])
        upto = torch.tensor(np.cumsum(_frequency(case)), device="cuda")
        rank = torch.searchsorted(upto, torch.rand(t, generator=gen, device="cuda", dtype=torch.float64))
        names = torch.randperm(v, generator=gen, device="cuda")  # frequent words lie all over the table
        ids = names[rank.clamp_(max=v - 1)]
        if _padding(case):
            ids[t - _padding(case):] = -1  # the padding of a batch
        st["tokens_in"] = ids.to(_INDEX[case["ids"]])
        if case["train"]:
            st["dout"] = randn(t, c).to(dt)
        return st
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    # the output of one projection: query heads, then key heads, then value heads; tokens of different scale
    st["qkv"] = (randn(t, h + 2 * g, d) * torch.exp(0.5 * randn(t, 1, 1))).to(dt)
    st["cu_seqlens"] = st["positions"] = None
    if case["seqs"]:
        cu = [0]
        for n in _lengths(case):
            cu.append(cu[-1] + n)
        st["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    else:
        st["positions"] = torch.randint(0, 131072, (t,), generator=gen, device="cuda")
    pt = None if case["weights"] is None else _DTYPES[case["weights"]]
    st["q_weight"], st["k_weight"] = (None if pt is None else (1.0 + 0.2 * randn(d)).to(pt) for _ in range(2))
    if case["train"]:
        st["dq_out"], st["dk_out"] = randn(t, h, d).to(dt), randn(t, g, d).to(dt)
    if own:
        import muon_newton_schulz_03_amd as lib

        st["rotation"] = lib.Rotation(case["rotary"], _BASE, pairs=case["pairs"])
    return st


# ------------------------------------------------------------ plain forms --
def _embed_plain(st):
    w, ids, s = st["weight"], st["tokens_in"].long(), st["scale"]
    known = ((ids >= 0) & (ids < st["vocab"]))[:, None]
    at = ids.clamp(0, st["vocab"] - 1)
    out = dict(out=torch.where(known, w[at].float() * s, 0.0).to(_DTYPES[st["dtype"]]))
    if st["train"]:
        g = torch.where(known, st["dout"].float(), 0.0)
        dtable = torch.zeros(w.shape, dtype=torch.float32, device=w.device).index_add_(0, at, g)
        out["dtable"] = (dtable * s).to(w.dtype)
    return out


def _angles(st):
    t, n = st["tokens"], st["rotary"] // 2
    dev = st["qkv"].device
    if st["positions"] is not None:
        pos = st["positions"].double()
    else:
        at = torch.arange(t, device=dev, dtype=torch.int32)
        doc = torch.bucketize(at, st["cu_seqlens"][1:], right=True)
        pos = (at - st["cu_seqlens"][doc]).double()
    freq = _BASE ** (-torch.arange(n, device=dev, dtype=torch.float64) / n)
    ang = pos[:, None] * freq
    return torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]


def _split(z, st):
    """The two members of each pair, and what is not rotated."""
    r = st["rotary"]
    if st["pairs"] == "halves":
        return z[..., :r // 2], z[..., r // 2:r], z[..., r:]
    return z[..., 0:r:2], z[..., 1:r:2], z[..., r:]


def _merge(a, b, rest, st):
    if st["pairs"] == "halves":
        return torch.cat([a, b, rest], dim=-1)
    return torch.cat([torch.stack([a, b], dim=-1).flatten(-2), rest], dim=-1)


def _qk_plain(st):
    h, g = st["heads"], st["kv_heads"]
    cos, sin = _angles(st)
    out = {}
    for n, lo, hi in (("q", 0, h), ("k", h, h + g)):
        x = st["qkv"][:, lo:hi].float()
        w = None if st["weights"] is None else st[n + "_weight"].float()
        r = 1.0 / torch.sqrt(x.square().mean(dim=2, keepdim=True) + _EPS)
        xh = x * r
        a, b, rest = _split(xh if w is None else xh * w, st)
        out[n] = _merge(a * cos - b * sin, b * cos + a * sin, rest, st).to(st["qkv"].dtype)
        if st["train"]:
            a, b, rest = _split(st[f"d{n}_out"].float(), st)
            dz = _merge(a * cos + b * sin, b * cos - a * sin, rest, st)
            gz = dz if w is None else dz * w
            out["d" + n] = (r * (gz - xh * (gz * xh).mean(dim=2, keepdim=True))).to(st["qkv"].dtype)
            if w is not None:
                out[f"d{n}_weight"] = (dz * xh).sum(dim=(0, 1))
    return out


# ---------------------------------------------------------- library calls --
def _embed_own(st):
    import muon_newton_schulz_03_amd as lib

    out = dict(out=lib.embedding_forward(st["weight"], st["tokens_in"], scale=st["scale"],
                                         dtype=_DTYPES[st["dtype"]]))
    if st["train"]:
        out["dtable"] = lib.embedding_backward(st["dout"], st["tokens_in"], st["vocab"], scale=st["scale"],
                                               dtype=st["weight"].dtype)
    return out


def _qk_own(st):
    import muon_newton_schulz_03_amd as lib

    h, g = st["heads"], st["kv_heads"]
    q, k = st["qkv"][:, :h], st["qkv"][:, h:h + g]
    how = dict(q_weight=st["q_weight"], k_weight=st["k_weight"], cu_seqlens=st["cu_seqlens"],
               positions=st["positions"], eps=_EPS)
    qo, ko = lib.qk_norm_forward(q, k, st["rotation"], **how)
    out = dict(q=qo, k=ko)
    if st["train"]:
        dqkv = torch.empty_like(st["qkv"])  # the gradient of the projection, whose last part is the attention's dv
        dq, dk, dqw, dkw = lib.qk_norm_backward(st["dq_out"], st["dk_out"], q, k, st["rotation"], dq=dqkv[:, :h],
                                                dk=dqkv[:, h:h + g], **how)
        out["dq"], out["dk"] = dq, dk
        if st["weights"] is not None:
            out["dq_weight"], out["dk_weight"] = dqw, dkw
    return out


def run(state):
    if state["op"] == "embed":
        return _embed_own(state) if own else _embed_plain(state)
    return _qk_own(state) if own else _qk_plain(state)


# ------------------------------------------------------------ cost, truth --
def work(case):
    b, t = _BYTES[case["dtype"]], case["tokens"]
    if case["op"] == "embed":
        c, tb, n = case["cols"], _BYTES[case["table"]], t - _padding(case)
        rows = float(np.sum(-np.expm1(n * np.log1p(-np.minimum(_frequency(case), 1.0 - 1e-12)))))  # read, on average
        ids = t * (8 if case["ids"] == "i64" else 4)
        if not case["train"]:
            return {"bytes": int(ids + rows * c * tb + t * c * b), "flops": n * c}
        return {"bytes": int(ids + rows * c * tb + t * c * b + n * c * b + case["vocab"] * c * tb), "flops": 3 * n * c}
    n = t * (case["heads"] + case["kv_heads"]) * case["dim"]
    place = (case["seqs"] + 1) * 4 if case["seqs"] else 8 * t
    params = 0 if case["weights"] is None else 2 * case["dim"] * _BYTES[case["weights"]]
    if not case["train"]:
        return {"bytes": 2 * n * b + place + params, "flops": 8 * n}
    return {"bytes": 4 * n * b + place + params + (8 * case["dim"] if params else 0), "flops": 24 * n}


def _embed_exact(st):
    ids = st["tokens_in"].long()
    keep = (ids >= 0) & (ids < st["vocab"])
    out = torch.zeros(st["tokens"], st["cols"], dtype=torch.float64, device=ids.device)
    out[keep] = st["scale"] * st["weight"][ids[keep]].double()
    res = dict(out=out)
    if st["train"]:
        grad = torch.zeros(st["vocab"], st["cols"], dtype=torch.float64, device=ids.device)
        grad.index_put_((ids[keep],), st["scale"] * st["dout"][keep].double(), accumulate=True)
        res["dtable"] = grad
    return res


def _qk_exact(st):
    """Pairs as complex numbers; the gradients by differentiating the definition."""
    h, g, n = st["heads"], st["kv_heads"], st["rotary"] // 2
    dev, train = st["qkv"].device, st["train"]
    if st["positions"] is not None:
        pos = st["positions"].double()
    else:
        pos = torch.cat([torch.arange(m, device=dev) for m in _lengths(st)]).double()
    freq = torch.exp(torch.arange(n, device=dev, dtype=torch.float64) * (-math.log(_BASE) / n))
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=dev), torch.outer(pos, freq))[:, None]
    res = {}
    for name, part in (("q", slice(0, h)), ("k", slice(h, h + g))):
        x = st["qkv"][:, part].double().requires_grad_(train)
        w = st[name + "_weight"]
        w = (torch.ones(st["dim"], device=dev) if w is None else w).double().requires_grad_(train)
        z = x * (x.pow(2).sum(2, keepdim=True) / st["dim"] + _EPS).pow(-0.5) * w
        front = z[..., :2 * n]
        if st["pairs"] == "halves":
            y = torch.complex(front[..., :n], front[..., n:]) * turn
            y = torch.cat([y.real, y.imag, z[..., 2 * n:]], dim=2)
        else:
            y = torch.complex(front[..., ::2], front[..., 1::2]) * turn
            y = torch.cat([torch.view_as_real(y).reshape(front.shape), z[..., 2 * n:]], dim=2)
        res[name] = y.detach()
        if train:
            dx, dw = torch.autograd.grad(y, (x, w), st[f"d{name}_out"].double())
            res["d" + name] = dx
            if st["weights"] is not None:
                res[f"d{name}_weight"] = dw
    return res


def exact(case, seed):
    st = prepare(case, seed)
    return _embed_exact(st) if case["op"] == "embed" else _qk_exact(st)
