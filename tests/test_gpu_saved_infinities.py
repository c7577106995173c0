"""What the gated product saves in fp16 beside an infinity: the scale of eight
follows their largest finite element, and the others keep their 11 bits."""
import pytest
import torch

from tests import ffn_util as U

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from combine_route_mask_amd import ffn, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return ffn


def test_neighbours_of_an_infinity(F):
    """Products of one element with weights of very different size: 2^100 times 2^100 passes fp32's largest number."""
    I, K = 16, 8
    w = torch.zeros(2 * I, K)
    w[:, 0] = 2.0 ** -80
    w[1, 0] = 1.25 * 2.0 ** -81
    w[3, 0], w[I + 9, 0] = 2.0 ** 100, -2.0 ** 100  # one infinity of either sign, in a block of the gate and one of up
    w[5, 0], w[I + 15, 0] = 129 * 2.0 ** -90, 0
    x = torch.zeros(3, K)
    x[:, 0] = torch.tensor([2.0 ** 100, 129 * 2.0 ** 93, 2.0 ** 60])  # past fp16's largest number, and near its least
    got = F.gated_product(x.bfloat16().cuda(), w.bfloat16().cuda(), checkpoint="bf16")
    values = U.half_values(got[1], got[2])
    want = x.double() @ w.double().t()
    want[want.abs() >= 2.0 ** 128] = want[want.abs() >= 2.0 ** 128].sign() * float("inf")
    assert int(want.isinf().sum()) == 6
    # each finite product is a number of 15 bits at most, within 2^-13 of its eight's largest: fp16 holds 11 of them
    fine = want.isfinite()
    assert torch.equal(values[~fine], want[~fine])
    assert bool(((values - want)[fine].abs() <= 2.0 ** -11 * want[fine].abs()).all())


def test_blocks_without_a_finite_number(F):
    """Eight infinities and NaN: they come back as they are, next to a block of zeros."""
    w = torch.zeros(16, 8)
    w[:8, 0], w[8:, 1] = 2.0 ** 100, 1.0
    x = torch.zeros(2, 8)
    x[0, 0], x[1, 0] = 2.0 ** 100, float("nan")
    _, pre, scales = F.gated_product(x.bfloat16().cuda(), w.bfloat16().cuda(), checkpoint="bf16")
    got = U.half_values(pre, scales)
    assert bool(got[0, :8].isposinf().all()) and not bool(got[0, 8:].any()) and bool(got[1].isnan().all())
