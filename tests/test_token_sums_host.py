"""What the tests of long sums compare with sees one lost piece of them (no GPU)."""
import pytest
import torch

import block_reference as B
import token_reference as R
import token_sums as S


@pytest.mark.parametrize("case", range(len(S.DW_CASES)))
def test_weight_gradient_bound_sees_a_lost_tile(case):
    """Zeros, and a sum without one wave's group of tokens (two at least), are outside the bound."""
    T, H, _, D = S.DW_CASES[case]
    f = [0.9 ** i for i in range(D // 2)]
    turns = R.angles(range(T), f)
    x, dy = S.dw_inputs(T, H, D, torch.bfloat16, 10 + case)
    depth = S.dw_depth(T, H, D, 8)
    assert depth < 150
    value, bound = S.dw_bound(x, None, turns, D, "halves", 1e-6, dy, depth)
    B.check("dw", value, value, bound)
    at = T // 3
    lost = dy.clone()
    lost[at:at + 2] = 0
    for wrong in (torch.zeros_like(value), S.dw_bound(x, None, turns, D, "halves", 1e-6, lost, depth)[0]):
        with pytest.raises(AssertionError):
            B.check("dw", wrong, value, bound)


def test_sums_of_integers_see_a_lost_or_doubled_token():
    for T, before, behind in S.RUNS:
        ids, dout = S.run_ids(T, before, behind, 3), S.small_integers((T, 4), 4, torch.bfloat16)
        assert ids.shape == (T,) and int((ids == 5).sum()) == T - before - behind and int((ids < 5).sum()) == before
        want = S.embedding_sums(ids, dout, 41)
        assert torch.equal(want.float().long(), want)  # fp32 holds it
        token = int((ids == 5).nonzero()[77])
        for n in (0, 2):
            wrong = dout.clone()
            wrong[token] *= n
            assert (S.embedding_sums(ids, wrong, 41) != want).any(1).nonzero().tolist() == [[5]]
    old = S.small_integers((41, 4), 5, torch.float32)
    assert torch.equal(S.embedding_sums(ids, dout, 41, old), want + old.long())
    assert torch.equal(S.embedding_sums(torch.tensor([-1, 41, 1]), dout[:3], 41)[1], dout[2].long())
