"""The cosines and sines of the query/key norm's rotation against angles in exact arithmetic."""
import math
from fractions import Fraction

import pytest
import torch

import muon_newton_schulz_03_amd as lib
from muon_harness import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def exact_angles(positions, frequencies):
    """cos and sin (T, F) of position times frequency, whose turns are held to 2^-180."""
    one = 1 << 180
    turns = [round(Fraction(f) / (2 * PI) * one) for f in frequencies]
    frac = torch.tensor([[((p * t + one // 2) % one - one // 2) / one for t in turns] for p in positions],
                        dtype=torch.float64)
    return torch.cos(frac * (2 * math.pi)), torch.sin(frac * (2 * math.pi))


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("frequencies", [[1.0, 0.1, 0.01, 0.001], [64.0, -63.9, 31.4159, -0.5],
                                         [math.pi / 4, math.pi / 4 * (1 - 2e-9), -math.pi / 2, 1e-9]])
def test_cosines_and_sines_are_off_by_what_is_stated(pairs, frequencies):
    """2^-31 turns, times 2^-32 of the position where that is beyond 2^32, and 2^-23.

    A head whose mean square is 1 and whose pairs are (1, 0) comes out as the cosines and sines themselves.
    """
    g = torch.Generator().manual_seed(7)
    near = torch.arange(-2000, 2001)
    far = torch.randint(-(1 << 32), (1 << 32) + 1, (4000,), generator=g)
    farther = torch.randint(-(1 << 45), 1 << 45, (500,), generator=g)
    pos = torch.cat([near, far, farther, torch.tensor([1 << 32, -(1 << 32), (1 << 31) - 1, -(1 << 31)])])
    ia = torch.arange(4) * (2 if pairs == "neighbours" else 1)
    ib = ia + (1 if pairs == "neighbours" else 4)
    head = torch.zeros(16)
    head[ia], head[8:11] = 1.0, 2.0  # four squares of 1 and three of 4
    q = head.repeat(len(pos), 1, 1).to(DEV)
    out, _ = lib.qk_norm_forward(q, q, lib.Rotation(8, frequencies=frequencies, pairs=pairs), positions=pos.to(DEV), eps=0.0)
    out = out[:, 0].double().cpu()
    assert torch.equal(out[:, 8:], head[8:].double().expand(len(pos), 8))
    cos, sin = exact_angles(pos.tolist(), frequencies)
    turns = 2.0 ** -31 * torch.clamp(pos.abs().double() * 2.0 ** -32, min=1.0)
    bound = 2.0 ** -23 + 2 * math.pi * turns[:, None]
    worst = max(((out[:, ia] - cos).abs() / bound).max().item(), ((out[:, ib] - sin).abs() / bound).max().item())
    say(f"[gpu] cosines and sines, {pairs}, {frequencies}: worst error {worst:.3f} of its bound")
    assert worst <= 1.0
