"""What the tests of long sums compare with: integers, whose fp32 sums are exact in every order, and bounds by the
depth of a sum (CPU).

A bound of (terms + 8) 2^-24 holds for every order of a sum, but with 10^5 terms it is as large as the sum itself.
"""
import torch

import token_reference as R
from block_reference import U32


def small_integers(shape, seed, dtype, top=8):
    """Integers from -top to top without 0, which every type holds: a term that is lost or added twice shows."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(1, top + 1, shape, generator=g)
    return torch.where(torch.rand(shape, generator=g) < 0.5, -n, n).to(dtype)


def embedding_sums(ids, dout, vocab, old=None):
    """Sums of dout's integer rows by id, in int64 (added to `old`); what fp32 makes of them is the same below 2^24."""
    flat, rows = ids.reshape(-1).long(), dout.reshape(-1, dout.shape[-1]).long()
    known = (flat >= 0) & (flat < vocab)
    total = torch.zeros(vocab, rows.shape[1], dtype=torch.int64) if old is None else old.long()
    total = total.index_add(0, flat[known], rows[known])
    mass = torch.zeros_like(total).index_add_(0, flat[known], rows[known].abs())
    assert int(mass.max()) < 1 << 24
    return total


# A pass over many tokens has 4096 waves, each with `at_once` = 64 / (lanes a head) heads of one or several tokens at a
# time, and a weight's gradient is summed over a lane's terms, a wave's heads (at most 5 exchanges), a block's 4 waves,
# and 1024 blocks: 32 in turn, then 32 such sums.
def dw_depth(tokens, heads, dim, vec):
    at_once = 64 // ((64 if dim <= 64 else 128) // vec)
    serial, wide = 0, 1
    while wide <= at_once:
        groups = -(-tokens // (at_once // wide))
        serial = max(serial, -(-groups // 4096) * -(-heads // wide))
        wide *= 2
    return serial + 5 + 4 + 32 + 32


def dw_bound(x, w, turns, dim, pairs, eps, dy, depth):
    """The weight gradient of one side (fp64) and its bound where no term goes through more than `depth` additions."""
    value, bound = R.qk_norm(x, w, turns, dim, pairs, eps, dy)["dw"]
    xd, dyd = x.double(), dy.double()
    cos, sin, _ = turns
    r = 1 / torch.sqrt((xd * xd).mean(2, keepdim=True) + eps)
    mass = (R.turn(dyd, cos, -sin, dim, pairs) * xd * r).abs().sum((0, 1))
    return value, bound - (x.shape[0] * x.shape[1] + 8) * U32 * mass + 1.01 * depth * U32 * mass


# Sizes at which a wave takes several groups of tokens, some of them without a whole number of them.
DW_CASES = [(70001, 2, 1, 32), (33000, 1, 4, 128), (40003, 3, 2, 64)]


def dw_inputs(tokens, heads, dim, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(tokens, heads, dim, generator=g) * torch.exp(0.5 * torch.randn(tokens, 1, 1, generator=g))).to(dtype)
    return x, torch.randn(tokens, heads, dim, generator=g).to(dtype)


# Runs of one id: tokens, how many entries of lower ids come first (so that it starts inside a chunk), how many follow.
RUNS = [(70000, 0, 0), (70000, 1, 0), (70000, 31, 1), (70000, 33, 500), (70000, 127, 2), (70000, 300, 34007)]


def run_ids(tokens, before, behind, seed):
    """Ids 0 to 2 before the run (of id 5) and 9 to 40 behind it, in random order."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.cat([torch.arange(before) % 3, torch.full((tokens - before - behind,), 5), 9 + torch.arange(behind) % 32])
    return ids[torch.randperm(tokens, generator=g)]
