"""Gradients of the operators around the attention, at starts, sizes and sums of many terms that the other tests leave
out."""
import pytest
import torch

import block_reference as B
import muon_newton_schulz_03_amd as lib
import token_reference as R
import token_sums as S
from muon_harness import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def randn(shape, seed, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


# --------------------------------------------------------------- where a gradient starts --
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off", [1, 2, 7])
def test_recorded_gradients_may_start_anywhere(dtype, off):
    """A contiguous gradient that starts between two multiples of 16 bytes, as one that comes through torch.cat."""
    T, H, G, D = 21, 4, 2, 32
    q, k, v = randn((T, H, D), 1, dtype), randn((T, G, D), 2, dtype), randn((T, G, D), 3, dtype)
    cu, rot = torch.tensor([0, 15, 21], dtype=torch.int32, device=DEV), lib.Rotation(D)
    flat = randn((off + T * (H + G) * D,), 4, dtype)
    dq = flat[off:off + T * H * D].view(T, H, D)
    dk = flat[off + T * H * D:].view(T, G, D)
    assert dq.is_contiguous() and dk.is_contiguous()
    qn, kn = lib.qk_norm_forward(q, k, rot, cu_seqlens=cu)
    want = lib.qk_norm_backward(dq.clone(), dk.clone(), q, k, rot, cu_seqlens=cu)[:2]
    a, b = (t.clone().requires_grad_(True) for t in (q, k))
    torch.autograd.backward(lib.qk_norm_forward(a, b, rot, cu_seqlens=cu), [dq, dk])
    assert torch.equal(a.grad, want[0]) and torch.equal(b.grad, want[1])
    a, b = (t.clone().requires_grad_(True) for t in (q, k))
    y, z = lib.qk_norm_forward(a, b, rot, cu_seqlens=cu)
    (torch.cat([flat[:off], y.flatten(), z.flatten()]) * flat).sum().backward()
    assert torch.equal(a.grad, want[0]) and torch.equal(b.grad, want[1])
    out, lse = lib.packed_attention_forward(qn, kn, v, cu)
    want = lib.packed_attention_backward(dq.clone(), qn, kn, v, out, lse, cu)
    leaves = [t.clone().requires_grad_(True) for t in (qn, kn, v)]
    lib.packed_attention_forward(*leaves, cu)[0].backward(dq)
    assert all(torch.equal(t.grad, w) for t, w in zip(leaves, want))


# --------------------------------------------------------------- sums of many terms --
@pytest.mark.parametrize("cols,dtype,tokens", [(64, BF, 70000), (128, BF, 140000), (256, BF, 70000), (512, BF, 70000),
                                               (505, BF, 70000), (33, BF, 70000), (40, F32, 270000), (9, F32, 70000),
                                               (128, F32, 70000), (256, F32, 40000)])
def test_embedding_sums_of_integers_are_exact(cols, dtype, tokens):
    """Every lane layout, 4 and 8 entries a group, streamed or not: no token of a run over many chunks is lost or added
    twice, whatever the chunk in which it starts or ends."""
    dout = S.small_integers((tokens, cols), 20, dtype)
    dev = dout.to(DEV)
    for i, (_, before, behind) in enumerate(S.RUNS):
        say(f"[gpu] embedding sums {tokens}x{cols} {dtype}: {before} entries before the run, {behind} behind it")
        ids = S.run_ids(tokens, before, behind, 30 + i)
        want = S.embedding_sums(ids, dout, 41)
        for index in (torch.int32, torch.int64):
            got = lib.embedding_backward(dev, ids.to(index).to(DEV), 41, scale=0.5)
            assert torch.equal(got.cpu(), want.float() * 0.5)
        low = lib.embedding_backward(dev, ids.to(DEV), 41, dtype=BF, scale=-2.0)
        assert torch.equal(low.cpu(), (want.float() * -2.0).to(BF))  # the exact sum, rounded once
        old = S.small_integers((41, cols), 40 + i, F32)
        got = old.to(DEV)
        lib.embedding_backward(dev, ids.to(DEV), 41, dtable=got, accumulate=True)
        assert torch.equal(got.cpu(), S.embedding_sums(ids, dout, 41, old).float())


@pytest.mark.parametrize("tokens", [600, 3000, 8192, 8193, 20000])
def test_embedding_sums_of_integers_over_many_rows(tokens):
    """Runs of every length at once, in one block's sort and in several blocks'."""
    g = torch.Generator().manual_seed(50)
    for cols, dtype in ((24, BF), (136, BF), (768, BF), (20, F32), (1001, F32)):
        say(f"[gpu] embedding sums of rows {tokens}x{cols} {dtype}")
        ids = (torch.rand(tokens, generator=g) ** 6 * 4000).long() - 1  # -1 is padding
        dout = S.small_integers((tokens, cols), 51, dtype)
        dev = dout.to(DEV)
        dev[ids.to(DEV) < 0] = float("nan")
        want = S.embedding_sums(ids, dout, 4000)
        assert torch.equal(lib.embedding_backward(dev, ids.to(DEV), 4000).cpu(), want.float())


@pytest.mark.parametrize("tokens,heads,kv_heads,dim", S.DW_CASES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_gradients_of_integers_are_exact(tokens, heads, kv_heads, dim, dtype):
    """Heads of ones and minus ones have r = 1, so with integer gradients and no turn every sum is exact."""
    x = S.small_integers((tokens, heads + kv_heads, dim), 60, dtype, top=1)
    dy = S.small_integers(x.shape, 61, dtype)
    dev, ddy = x.to(DEV), dy.to(DEV)
    still = [None] + [lib.Rotation(dim, frequencies=[0.0] * (dim // 2), pairs=p) for p in ("halves", "neighbours")]
    for used in (tokens, tokens - 1, tokens // 2 + 1):
        cu = None if used == tokens else torch.tensor([0, used // 3, used], dtype=torch.int32, device=DEV)
        terms = (x[:used].long() * dy[:used].long())
        want = terms[:, :heads].sum((0, 1)).float(), terms[:, heads:].sum((0, 1)).float()
        for rotation in still:
            got = lib.qk_norm_backward(ddy[:, :heads], ddy[:, heads:], dev[:, :heads], dev[:, heads:], rotation,
                                       cu_seqlens=cu, eps=0.0, need_q_weight=True, need_k_weight=True)[2:]
            assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1]), (used, rotation)


@pytest.mark.parametrize("case", range(len(S.DW_CASES)))
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weight_gradients_within_their_depth(case, dtype):
    """Turned heads of every scale: as far off as the additions that a term goes through, not as their number."""
    T, H, G, D = S.DW_CASES[case]
    f = [0.9 ** i for i in range(D // 2)]
    turns, rot = R.angles(range(T), f), lib.Rotation(D, frequencies=f)
    (q, gq), (k, gk) = S.dw_inputs(T, H, D, dtype, 10 + case), S.dw_inputs(T, G, D, dtype, 70 + case)
    got = lib.qk_norm_backward(gq.to(DEV), gk.to(DEV), q.to(DEV), k.to(DEV), rot, need_q_weight=True,
                               need_k_weight=True)[2:]
    for name, dw, x, dy in (("dq_weight", got[0], q, gq), ("dk_weight", got[1], k, gk)):
        depth = S.dw_depth(T, x.shape[1], D, 8 if dtype == BF else 4)
        worst = B.check(name, dw, *S.dw_bound(x, None, turns, D, "halves", 1e-6, dy, depth))
        say(f"[gpu] {name} {T}x{x.shape[1]}x{D} {dtype}: depth {depth}, worst error {worst:.3f} of its bound")


# --------------------------------------------------------------- few tokens, rows of many --
def crowded(tokens, vocab, rows, seed):
    """Ids of which many fall on neighbouring rows: with `rows` rows a block, 40, 1, 8, 9 and 200 on the first three, a
    middle and the last row of one block, 17 and 9 on the first and last row of the table's last, partial block (9 where
    that is one row)."""
    at, end = 3 * rows, (vocab - 1) // rows * rows
    assert rows >= 5 and end > at + rows and vocab - end < rows
    counts = {at: 40, at + 1: 1, at + 2: 8, at + rows // 2 + 1: 9, at + rows - 1: 200, end: 17, vocab - 1: 9}
    ids = torch.cat([torch.full((n,), v) for v, n in counts.items()])
    g = torch.Generator().manual_seed(seed)
    rest = torch.randint(-2, vocab + 2, (tokens - len(ids),), generator=g)  # some outside the table
    return torch.cat([ids, rest])[torch.randperm(tokens, generator=g)]


# columns and dtype of the gradient, and the lanes of a row that go with them; 64 KiB of the table a block, but at least
# 512 blocks
CROWDED = [(64, BF, 8), (72, BF, 8), (33, BF, 8), (128, BF, 16), (256, BF, 32), (768, BF, 32), (505, BF, 64), (512, BF, 64),
           (32, F32, 8), (61, F32, 16), (128, F32, 32), (768, F32, 64), (1001, F32, 64)]


@pytest.mark.parametrize("cols,dtype,lanes", CROWDED)
@pytest.mark.parametrize("vocab", [5000, 50257])
def test_embedding_gradient_of_few_tokens_on_neighbouring_rows(cols, dtype, lanes, vocab):
    """Rows of more than 8 tokens, several in a block and beside rows of fewer, and both sides of the rule: 512 tokens
    go in one launch, 513 are sorted."""
    say(f"[gpu] crowded rows {vocab}x{cols} {dtype}, {lanes} lanes")
    for table in (BF, F32):
        size = 2 if table == BF else 4
        rows = min(65536 // (cols * size), vocab // 512, 1024)
        for tokens in (511, 512, 513):
            ids = crowded(tokens, vocab, rows, tokens)
            dout = S.small_integers((tokens, cols), 80, dtype)
            known = (ids >= 0) & (ids < vocab)
            at, back = torch.unique(ids[known], return_inverse=True)
            total = torch.zeros(len(at), cols, dtype=torch.int64).index_add_(0, back, dout[known].long())
            dev, ddev = ids.to(DEV), dout.to(DEV)
            ddev[~known.to(DEV)] = float("nan")  # not read
            want = torch.zeros(vocab, cols, dtype=table, device=DEV)
            want[at.to(DEV)] = total.float().to(table).to(DEV)
            assert torch.equal(lib.embedding_backward(ddev, dev, vocab, dtype=table), want), (table, tokens)
            wide = torch.full((vocab, cols + 3), 5.0, dtype=table, device=DEV)  # rows of a wider table
            lib.embedding_backward(ddev, dev.int(), vocab, dtable=wide[:, 1:1 + cols])
            assert torch.equal(wide[:, 1:1 + cols], want), (table, tokens)
            assert (wide[:, 0] == 5).all() and (wide[:, 1 + cols:] == 5).all()
            old = S.small_integers((vocab, cols), 81, table).to(DEV)
            want = old.clone()
            want[at.to(DEV)] = (total.float() * 0.5 + old[at.to(DEV)].cpu().float()).to(table).to(DEV)
            lib.embedding_backward(ddev, dev, vocab, scale=0.5, dtable=old, accumulate=True)
            assert torch.equal(old, want), (table, tokens)


@pytest.mark.parametrize("cols,dtype,lanes", CROWDED[::2])
def test_embedding_gradient_of_few_tokens_against_fp64(cols, dtype, lanes):
    for table, tokens in ((BF, 512), (F32, 512), (F32, 513)):
        size = 2 if table == BF else 4
        ids = crowded(tokens, 5000, min(65536 // (cols * size), 9, 1024), 90)
        dout, weight, old = randn((tokens, cols), 91, dtype), randn((5000, cols), 92, table), randn((5000, cols), 93, table)
        for given in (None, old):
            ref = R.embedding(weight.cpu(), ids, 0.7, dtype, dout.cpu(), table, None if given is None else given.cpu())
            got = lib.embedding_backward(dout, ids.to(DEV), 5000, scale=0.7, dtype=table,
                                         dtable=None if given is None else given.clone(), accumulate=given is not None)
            say(f"[gpu] crowded rows {tokens} tokens x{cols} {dtype} into {table}: worst error "
                f"{B.check('dtable', got, *ref['dtable']):.3f} of its bound")
