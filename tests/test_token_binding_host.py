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
