"""fp64 definitions of layer norm and packed causal attention, with gradients and error bounds (CPU).

The bounds follow the arithmetic: an operand rounded to a type of relative
half step u is off by at most u of its value, and an fp32 sum of n terms by at
most (n + 8) 2^-24 of the sum of their magnitudes.  `u` is 2^-8 for bf16 and
2^-24 for fp32.
"""
import math

import torch

U32 = 2.0 ** -24


def unit(dtype):
    return torch.finfo(dtype).eps / 2


# -------------------------------------------------------------- layer norm --
def norm_forward(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    y = (x - mean) * rstd
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return y, mean.squeeze(-1), rstd.squeeze(-1)


def norm_backward(dy, x, w, eps):
    x, dy = x.double(), dy.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mean) * rstd
    g = dy if w is None else dy * w.double()
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def norm_bounds(dy, x, w, b, eps):
    """Elementwise bounds on the errors of y, mean, rstd, dx, dw and db for 2-D inputs.

    The mean is off by e_m <= (n + 2) u32 mean|x|.  That shifts every centred
    value (which its own subtraction rounds too), so xh is off by e_h <=
    rstd (e_m + 2 u32 |x - mean|) + |xh| e_r, where e_r, rstd's relative error,
    is half the variance's, (n + 8) u32 + (e_m rstd)^2, plus 4 u32.
    """
    u = unit(x.dtype)
    x = x.double()
    n, r = x.shape[-1], x.shape[0]
    y, mean, rstd = norm_forward(x, w, b, eps)
    mean, rstd = mean[:, None], rstd[:, None]
    xh = (x - mean) * rstd
    e_m = (n + 2) * U32 * x.abs().mean(-1, keepdim=True)
    e_r = ((n + 8) * U32 + (e_m * rstd) ** 2) / 2 + 4 * U32
    e_h = rstd * (e_m + 2 * U32 * (x - mean).abs()) + xh.abs() * e_r
    wa = torch.ones_like(x[:1]) if w is None else w.double().abs()[None]
    out = dict(mean=e_m.squeeze(1) + 2 * U32 * mean.abs().squeeze(1), rstd=(rstd * e_r).squeeze(1),
               y=u * y.abs() + 1.01 * (e_h * wa + 4 * U32 * (xh.abs() * wa + y.abs())))
    if dy is not None:
        dy = dy.double()
        g = dy.abs() * wa
        dx, dw, _ = norm_backward(dy, x, w, eps)
        c1, c2 = g.mean(-1, keepdim=True), (g * xh.abs()).mean(-1, keepdim=True)
        e_c1 = (n + 8) * U32 * c1
        e_c2 = (n + 8) * U32 * c2 + (g * e_h).mean(-1, keepdim=True)
        mass = g + c1 + xh.abs() * c2
        out["dx"] = u * dx.abs() + 1.01 * rstd * (e_c1 + xh.abs() * e_c2 + e_h * c2 + (8 * U32 + e_r) * mass)
        out["dw"] = (r + 8) * U32 * (dy * xh).abs().sum(0) + 1.01 * (dy.abs() * e_h).sum(0)
        out["db"] = (r + 8) * U32 * dy.abs().sum(0)
    return out


# --------------------------------------------------------------- attention --
def attention(q, k, v, lengths, scale, dout=None, dtype=None):
    """Outputs and gradients by the definition, and bounds on the errors of a computation with operands of `dtype`.

    q (T, H, D), k and v (T, G, D).  Returns {name: (value, bound)} for out,
    lse and, with dout, dq, dk, dv; rows behind the last sequence are zero.
    With u = unit(dtype), for bf16: p is rounded once for each product (u p),
    ds once (u |ds|), every result once, and delta comes from the rounded
    output.  In fp32 terms: a score is off by at most e_s, and p by the
    relative e_p = e_s + lse's error + exp2's; sums of n terms add (n + 8) u32.
    """
    dtype = dtype or q.dtype
    u = unit(dtype)
    low = u if dtype != torch.float32 else 0.0  # rounding of p and ds
    q, k, v = q.double(), k.double(), v.double()
    T, H, D = q.shape
    G = k.shape[1]
    z = lambda n: torch.zeros(T, n, D, dtype=torch.float64)  # noqa: E731
    out, e_out, lse, e_lse = z(H), z(H), torch.zeros(H, T, dtype=torch.float64), torch.zeros(H, T, dtype=torch.float64)
    dq, e_dq, dk, e_dk, dv, e_dv = z(H), z(H), z(G), z(G), z(G), z(G)
    at = 0
    for n in lengths:
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        acc = (n + 8) * U32
        for h in range(H):
            g = h // (H // G)
            qh, kh, vh = q[r, h], k[r, g], v[r, g]
            s = (qh @ kh.T) * scale
            s = s.masked_fill(hidden, -math.inf)
            l = torch.logsumexp(s, 1)
            p = torch.exp(s - l[:, None])
            o = p @ vh
            out[r, h], lse[h, r] = o, l
            # scores: D products in fp32, one scaling, one subtraction, the running maximum within 8 of the largest
            smass = ((qh.abs() @ kh.abs().T) * scale).masked_fill(hidden, 0.0).amax(1, keepdim=True)
            e_s = (D + 8) * U32 * smass
            e_l = e_s + (n + 16) * U32 + 8 * U32 * (l.abs()[:, None] + smass)
            e_p = 1.01 * (e_s + e_l + 8 * U32 * (l.abs()[:, None] + smass) + 8 * U32)
            e_lse[h, r] = e_l.squeeze(1)
            mass = p @ vh.abs()
            eo = u * o.abs() + 1.01 * (low + e_p + acc) * mass
            e_out[r, h] = eo
            if dout is None:
                continue
            do = dout[r, h].double()
            dp = (do @ vh.T).masked_fill(hidden, 0.0)
            delta = (do * o).sum(1, keepdim=True)
            ds = p * (dp - delta)
            e_delta = (do.abs() * eo).sum(1, keepdim=True) + (D + 8) * U32 * (do.abs() * o.abs()).sum(1, keepdim=True)
            e_dp = ((D + 8) * U32 * (do.abs() @ vh.abs().T)).masked_fill(hidden, 0.0)
            # dK's ds has delta corrected by the ds' own sum (zero by definition), and so has dQ's in the first 128 rows
            e_base = low * ds.abs() + (e_p + 4 * U32) * p * (dp.abs() + delta.abs()) + p * e_dp
            e_sum = (acc + e_p) * (p * (dp.abs() + delta.abs())).sum(1, keepdim=True) + (p * e_dp).sum(1, keepdim=True)
            e_fixed = 1.01 * (e_base + p * (torch.minimum(e_sum, e_delta) if low else e_delta))
            e_ds = 1.01 * (e_base + p * e_delta)
            e_ds[:128] = e_fixed[:128]
            dq[r, h] = ds @ kh * scale
            e_dq[r, h] = scale * (1.01 * e_ds @ kh.abs() + acc * (ds.abs() @ kh.abs()))
            dk[r, g] += ds.T @ qh * scale
            e_dk[r, g] += scale * (1.01 * e_fixed.T @ qh.abs() + (H // G) * acc * (ds.abs().T @ qh.abs()))
            dv[r, g] += p.T @ do
            e_dv[r, g] += 1.01 * (low + e_p.amax() + (H // G) * acc) * (p.T @ do.abs())
    res = dict(out=(out, e_out), lse=(lse, e_lse))
    if dout is not None:
        for name, val, e in (("dq", dq, e_dq), ("dk", dk, e_dk), ("dv", dv, e_dv)):
            res[name] = (val, e + u * val.abs() + 4 * U32 * val.abs())
    return res


def check(name, got, value, bound):
    """Every element within its bound; returns the largest error over bound."""
    got = got.double().cpu()
    assert got.shape == value.shape, f"{name}: shape {tuple(got.shape)} != {tuple(value.shape)}"
    if got.numel() == 0:
        return 0.0
    assert torch.isfinite(got).all(), f"{name}: not finite"
    tiny = 1e-30  # results that are exactly zero
    ratio = ((got - value).abs() / (bound + tiny)).max().item()
    assert ratio <= 1.0, f"{name}: error {ratio:.3g} times its bound"
    return ratio
