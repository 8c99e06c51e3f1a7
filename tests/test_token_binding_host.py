"""Arguments of the block operators' binding that are looked at before any tensor (no GPU)."""
import pytest
import torch

import muon_newton_schulz_03_amd as pkg


@pytest.mark.parametrize("grad", [False, True])
def test_a_tensor_is_no_scale_of_the_embedding(grad):
    """Its gradient would be lost, and the call would wait for one on a device."""
    table, ids, dout = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8)
    scale = torch.tensor(1.5, requires_grad=grad)
    for s in (scale, scale * 2, scale.reshape(1), torch.nn.Parameter(torch.ones(()), grad)):
        for call in (lambda: pkg.embedding_forward(table, ids, scale=s),
                     lambda: pkg.embedding_forward(table.clone().requires_grad_(True), ids, scale=s),
                     lambda: pkg.embedding_backward(dout, ids, 4, scale=s)):
            with pytest.raises(ValueError, match="scale must be a number"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="scale must be a number"):
                call()
    for s in (1.5, 2, True, scale.detach().numpy().item()):  # numbers go on to the tensors' checks
        with pytest.raises(ValueError, match="device tensor"):
            pkg.embedding_forward(table, ids, scale=s)
        with pytest.raises(ValueError, match="device tensor"):
            pkg.embedding_backward(dout, ids, 4, scale=s)


def test_gradients_of_numbers_are_not_lost():
    """A tensor that records gradients, where the operators take a number, is refused; a plain one counts as its value."""
    q, x, cu = torch.zeros(4, 2, 8), torch.zeros(4, 8), torch.zeros(2, dtype=torch.int32)
    g = torch.full((), 0.5, requires_grad=True)
    for name, call in (("eps", lambda t: pkg.qk_norm_forward(q, q, eps=t)),
                       ("eps", lambda t: pkg.layer_norm_forward(x, eps=t)),
                       ("scale", lambda t: pkg.packed_attention_forward(q, q, q, cu, scale=t))):
        for t in (g, g * 2, torch.nn.Parameter(torch.ones(()))):
            with pytest.raises(ValueError, match=f"{name} is a number"):
                call(t)
            with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
                call(t)
        for t in (0.5, g.detach()):
            with pytest.raises(ValueError, match="device tensor"):
                call(t)
        with torch.autograd.forward_ad.dual_level(), pytest.raises(ValueError, match=f"{name} is a number"):
            call(torch.autograd.forward_ad.make_dual(g.detach(), torch.ones(())))


def test_gradients_of_frequencies_are_not_lost():
    f = torch.tensor([1.0, 0.5, 0.25, 0.125], requires_grad=True)
    for bad in (dict(frequencies=f), dict(frequencies=list(f)), dict(frequencies=[1.0, 0.5, 0.25, f[3]]),
                dict(base=torch.tensor(100.0, requires_grad=True))):
        with pytest.raises(ValueError, match="frequencies are numbers"):
            pkg.Rotation(8, **bad)
        with torch.no_grad():
            pkg.Rotation(8, **bad)
    want = tuple(f.tolist())
    assert pkg.Rotation(8, frequencies=f.detach()).frequencies == want
    assert pkg.Rotation(8, frequencies=want).frequencies == want
    assert pkg.Rotation(0, base=torch.tensor(100.0, requires_grad=True)).frequencies == ()


def test_gradients_are_read_as_they_are_or_copied():
    """What the attention's and the query/key norm's backward pass reads starts, and steps, at multiples of 16 bytes."""
    from muon_newton_schulz_03_amd.block import _readable

    def fits(t):
        return t.stride(2) == 1 and not any(n * t.element_size() % 16 for n in t.stride()[:2]) and t.data_ptr() % 16 == 0

    for dtype in (torch.float32, torch.bfloat16):
        flat = torch.arange(8 + 5 * 3 * 8).to(dtype)
        flat = flat[(-flat.data_ptr() // flat.element_size()) % 8:]  # at a multiple of 16 bytes
        whole, wide = flat[:120].view(5, 3, 8), torch.ones(5, 3, 24, dtype=dtype)
        for t in (whole, wide[..., 8:16], whole.transpose(0, 1).contiguous().transpose(0, 1), whole[:, :1].expand(5, 3, 8),
                  whole[:1].expand(5, 3, 8), whole[:0]):
            assert _readable(t) is t
        for t in (flat[1:121].view(5, 3, 8), wide[..., 1:9], torch.ones((), dtype=dtype).expand(5, 3, 8),
                  whole.transpose(1, 2).contiguous().transpose(1, 2), flat[3:11].view(1, 1, 8),
                  torch.ones(5, 3, 9, dtype=dtype)[..., :8]):
            got = _readable(t)
            assert torch.equal(got, t) and got.is_contiguous() and fits(got) and got.data_ptr() != t.data_ptr()
    assert flat[1:121].view(5, 3, 8).is_contiguous()  # and yet does not start there
