"""fp64 definitions of the query/key norm with rotation and of the embedding, with gradients and error bounds (CPU).

The bounds follow the arithmetic, as in block_reference: an operand rounded to
a type of relative half step u is off by at most u of its value, an fp32 sum
of n terms by at most (n + 8) 2^-24 of the sum of their magnitudes.
"""
import numpy as np
import torch

from block_reference import U32, unit

# cos and sin in fp32: the reduced angle is off by 3 roundings of at most pi/4 (2.4 u32), the series' value by its own
# last roundings (2 u32), the remainder is below 0.1 u32.
E_TRIG = 6 * U32


def positions_of(tokens, lengths=None, positions=None):
    if positions is not None:
        return positions.tolist()
    if lengths is None:
        return list(range(tokens))
    out = [i for n in lengths for i in range(n)]
    return out + [0] * (tokens - len(out))


def angles(pos, freqs):
    """cos and sin, and a bound on the angles' errors: (T, 1, dim / 2) twice, and (T, 1, 1).

    The kernels hold f / 2 pi as a fraction of 2^64: the frequency's own division (half a step of a 64-bit mantissa,
    and the constant's) and the fraction's rounding put it off by at most 2^-63 |f / 2 pi| + 2^-65 turns, the
    reference by 2^-63 |f / 2 pi| and another 2^-64 of the product.  The position multiplies that: 2^-30 radians up
    to position 2^32, far below the roundings of cos and sin, but 2^-17 at 2^44.
    """
    tau = np.longdouble("6.283185307179586476925286766559")
    turns = np.array(pos, dtype=np.longdouble)[:, None] * (np.array(freqs, dtype=np.longdouble) / tau)[None]
    ang = ((turns - np.rint(turns)) * tau).astype(np.float64)
    off = 2.0 ** -65 + 2.5 * 2.0 ** -63 * max([abs(f) / 6.28 for f in freqs], default=0.0)
    e = torch.tensor([abs(p) * off * 6.29 for p in pos], dtype=torch.float64).reshape(-1, 1, 1)
    return torch.from_numpy(np.cos(ang))[:, None], torch.from_numpy(np.sin(ang))[:, None], e


def turn(z, cos, sin, dim, pairs):
    """R z, pair by pair; z (T, H, D), cos and sin (T, 1, dim / 2)."""
    ia = torch.arange(dim // 2) * (2 if pairs == "neighbours" else 1)
    ib = ia + (1 if pairs == "neighbours" else dim // 2)
    out = z.clone()
    out[..., ia] = z[..., ia] * cos - z[..., ib] * sin
    out[..., ib] = z[..., ib] * cos + z[..., ia] * sin
    return out


def qk_norm(x, w, turns, dim, pairs, eps, dy=None):
    """One side: {name: (value, bound)} for y and, with dy, dx and dw.  x (T, H, D), turns: `angles`."""
    u = unit(x.dtype)
    cos, sin, e_ang = turns
    x = x.double()
    n = x.shape[2]
    wd = torch.ones(n, dtype=torch.float64) if w is None else w.double()
    r = 1 / torch.sqrt((x * x).mean(2, keepdim=True) + eps)
    z = x * r * wd
    y = turn(z, cos, sin, dim, pairs)
    one, zero = torch.ones_like(cos), torch.zeros_like(sin)

    def pair_mass(t):  # |a| + |b| of the element's pair, |t| where nothing turns
        t = t.abs()
        return t.clone() if dim == 0 else turn(t, one, zero, dim, pairs) + _other(t, dim, pairs)

    e_r = ((n + 8) / 2 + 4) * U32
    res = dict(y=(y, u * y.abs() + 1.01 * pair_mass(z) * (e_r + E_TRIG + e_ang + 5 * U32)))
    if dy is None:
        return res
    dy = dy.double()
    dz = turn(dy, cos, -sin, dim, pairs)
    e_z = pair_mass(dy) * (E_TRIG + e_ang + 3 * U32)
    g, e_g = dz * wd, (e_z + U32 * dz.abs()) * wd.abs()
    c = (g * x).sum(2, keepdim=True) * r * r / n
    dx = r * (g - x * c)
    e_sum = (e_g * x.abs()).sum(2, keepdim=True) + (n + 8) * U32 * (g * x).abs().sum(2, keepdim=True)
    e_c = r * r / n * e_sum + c.abs() * (2 * e_r + 6 * U32)
    mass = g.abs() + (x * c).abs()
    res["dx"] = dx, u * dx.abs() + 1.01 * r * (e_g + x.abs() * e_c + (e_r + 4 * U32) * mass)
    t = dz * x * r
    terms = x.shape[0] * x.shape[1]
    res["dw"] = (t.sum((0, 1)), 1.01 * (e_z * x.abs() * r + (e_r + 3 * U32) * t.abs()).sum((0, 1)) +
                 (terms + 8) * U32 * t.abs().sum((0, 1)))
    return res


def _other(t, dim, pairs):
    """Each element's partner in its pair, 0 for elements that do not turn."""
    out = torch.zeros_like(t)
    ia = torch.arange(dim // 2) * (2 if pairs == "neighbours" else 1)
    ib = ia + (1 if pairs == "neighbours" else dim // 2)
    out[..., ia], out[..., ib] = t[..., ib], t[..., ia]
    return out


def embedding(table, ids, scale, dtype, dout=None, grad_dtype=None, old=None):
    """{name: (value, bound)} for out and, with dout, dtable (added to `old` where given)."""
    scale = float(np.float32(scale))
    flat = ids.reshape(-1).long()
    known = (flat >= 0) & (flat < table.shape[0])
    out = torch.zeros(flat.numel(), table.shape[1], dtype=torch.float64)
    out[known] = table.double()[flat[known]] * scale
    res = dict(out=(out.reshape(*ids.shape, -1), (unit(dtype) + 1.01 * U32) * out.abs().reshape(*ids.shape, -1)))
    if dout is not None:
        g = dout.double().reshape(flat.numel(), -1)[known]
        at = flat[known]
        total = torch.zeros(table.shape, dtype=torch.float64).index_add_(0, at, g) * scale
        mass = torch.zeros(table.shape, dtype=torch.float64).index_add_(0, at, g.abs()) * abs(scale)
        count = torch.bincount(at, minlength=table.shape[0]).double()[:, None]
        bound = (count + 8) * U32 * mass
        if old is not None:
            total = total + old.double()
            bound = bound + 1.01 * U32 * total.abs()
            bound[count[:, 0] == 0] = 0.0  # left as they were
        bound = bound + torch.where(count > 0, unit(grad_dtype), 0.0) * 1.01 * total.abs()
        res["dtable"] = (total, bound)
    return res
