"""The autograd wrappers: gradients that are slices of other tensors' memory."""
import pytest
import torch

import gated_delta_rule_bwd_gb300 as gdn

gpu = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rand(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def attention(dtype):
    q, k, v = (rand(i, 1, 37, h, 24, dtype=dtype) for i, h in enumerate((4, 2, 2)))
    return gdn.attention, (q, k, v)


def layer_norm(dtype):
    return gdn.layer_norm, (rand(0, 37, 64, dtype=dtype), rand(1, 64), rand(2, 64))


def mixer(dtype):
    q, k, v = (rand(i, 1, 37, 2, 24, dtype=dtype) * 0.3 for i in range(3))
    g, beta = -rand(3, 1, 37, 2).abs(), rand(4, 1, 37, 2).sigmoid()
    return (lambda *x: gdn.gated_delta_rule(*x, chunk=16)[0]), (q, k, v, g, beta)


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("make", [attention, layer_norm, mixer])
def test_gradient_between_boundaries(make, dtype):
    """The backward of a concatenation hands on a slice of its own gradient, which
    is contiguous and starts on no 16-byte boundary here: as good as a copy."""
    f, x = make(dtype)
    x = [t.requires_grad_() for t in x]
    do = rand(9, f(*x).numel() + 3, dtype=dtype)
    want = torch.autograd.grad((f(*x).flatten() * do[3:]).sum(), x)
    got = torch.autograd.grad((torch.cat([do[:3], f(*x).flatten()]) * do).sum(), x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert gdn.device_status() == 0


@gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_layer_norm_input_between_boundaries(dtype):
    x, w = rand(0, 1 + 5 * 64, dtype=dtype), rand(1, 64)
    assert torch.equal(gdn.layer_norm(x[1:].view(5, 64), w), gdn.layer_norm(x[1:].clone().view(5, 64), w))


@gpu
@pytest.mark.parametrize("make", [attention, layer_norm])
def test_second_derivatives_are_refused(make):
    """The gradients have no gradient of their own: a loss that holds one raises
    instead of going on without its share."""
    f, x = make(F32)
    x = [t.requires_grad_() for t in x]
    first, *_ = torch.autograd.grad(f(*x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        (first.square().sum() + x[0].sum()).backward()
