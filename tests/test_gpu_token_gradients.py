"""Gradients of the operators around the attention, at starts, sizes and sums of many terms that the other tests leave
out."""
import pytest
import torch

import muon_newton_schulz_03_amd as lib

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
