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


def test_crowded_ids_fall_where_they_are_meant_to():
    from test_gpu_token_gradients import CROWDED, crowded

    lanes_seen = set()
    for cols, dtype, lanes in CROWDED:
        vectors = -(-cols // (8 if dtype == torch.bfloat16 else 4))
        most = 64
        while most > 8 and -(-vectors // most) * most * 8 > vectors * 9:
            most //= 2
        assert lanes == most, (cols, dtype, most)
        lanes_seen.add(lanes)
        for vocab in (5000, 50257):
            for size in (2, 4):
                rows = min(65536 // (cols * size), vocab // 512, 1024)
                for tokens in (511, 512, 513):
                    ids = crowded(tokens, vocab, rows, tokens)
                    assert len(ids) == tokens
                    n = torch.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab)
                    block = n[3 * rows:4 * rows]
                    assert block[0] >= 40 and block[-1] >= 200 and (block > 8).sum() >= 3 and (block[1:3] > 0).all()
                    assert n[vocab - 1] >= 9 and vocab % rows and n[vocab // rows * rows] >= (17 if vocab % rows > 1 else 9)
    assert lanes_seen == {8, 16, 32, 64}
