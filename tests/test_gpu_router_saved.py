"""Logits that lie in a larger buffer, such as a dispatch's workspace: the
backward pass uses them as they were in the forward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    from combine_route_mask_amd import router, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return router


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E", [33, 600])
def test_logits_in_a_workspace(R, E, renormalize):
    g = torch.Generator().manual_seed(E)
    space = torch.randn((20, E), generator=g).cuda()
    gw = torch.randn((7, 3), generator=g).cuda()
    part = space[5:12].requires_grad_()
    r = R.route_top_k(part, 3, renormalize=renormalize)
    want = R.route_top_k_backward(part.detach().clone(), r.ids, gw, renormalize=renormalize)
    space.data.copy_(torch.randn((20, E), generator=g))  # as a kernel writes: unseen by autograd
    got, = torch.autograd.grad(r.weights, part, gw)
    assert torch.equal(got, want)
    # what autograd sees is refused as ever
    whole = torch.randn((7, E), generator=g).cuda().requires_grad_()
    moved = whole * 1
    r = R.route_top_k(moved, 3, renormalize=renormalize)
    moved.detach().zero_()
    with pytest.raises(RuntimeError, match="inplace"):
        r.weights.sum().backward()
