"""The product with 4-bit weights against 64-bit references: every code and
scale, one row, ragged and empty experts, odd channel counts, gated."""
import numpy as np
import pytest
import torch

from tests import ffn_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def F():
    from combine_route_mask_amd import ffn, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return ffn


def _weights(rng, E, N, K, low=120, high=130):
    many = (E,) if E else ()
    codes = torch.from_numpy(rng.integers(0, 256, (*many, N, K // 2), dtype=np.uint8))
    scales = torch.from_numpy(rng.integers(low, high, (*many, N, K // 32), dtype=np.uint8))
    return codes, scales.view(torch.float8_e8m0fnu)


SHAPES = [(1, 0, 1, 32, ""), (1, 0, 4096, 4096, ""), (8, 32, 64, 96, "single rows"), (3, 5, 18, 160, "ragged"),
          (17, 2, 34, 224, "one"), (100, 7, 50, 512, "ragged"), (16, 1, 130, 1056, "even"), (33, 0, 258, 992, ""),
          (50, 3, 32, 64, "none"), (300, 4, 100, 288, "ragged"), (2, 0, 20, 7168, ""), (5, 4096, 16, 32, "ragged"),
          (65, 2, 1024, 128, "one"), (4, 3, 4098, 2080, "ragged"), (130, 1, 72, 64, "even")]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,E,N,K,kind", SHAPES)
def test_product(F, M, E, N, K, kind, dtype, gated):
    if gated:
        N += N % 2
    log(f"4-bit {M}x{N}x{K} over {E} {kind} {dtype} gated={gated}")
    rng = np.random.default_rng(M + N + K)
    o = U.ragged(rng, M, E, kind) if E else None
    x = U.bf16(rng, M, K)
    codes, scales = _weights(rng, E, N, K)
    ref, bound, held = U.product(x, U.mxfp4_values(codes, scales), o)
    if gated:
        ref, bound = U.gated(ref, bound)
    x[~held] = float("nan")
    off = None if o is None else torch.from_numpy(o).cuda()
    out = torch.full(ref.shape, 7.0, dtype=dtype, device="cuda")
    got = F.expert_matmul_mxfp4(x.cuda(), codes.cuda(), scales.cuda(), offsets=off, gated=gated, out=out)
    U.close(got.cpu()[held], ref[held], U.rounded(bound, ref, dtype)[held], "4-bit product")
    assert bool((got.cpu()[~held] == 7).all()), "a row outside the experts' ranges was written"


def test_every_code_and_scale(F):
    """Unit rows read the weights themselves: all codes at all scales, exactly where bf16 holds them."""
    K = 32
    codes = torch.arange(256, dtype=torch.uint8).view(16, 16)
    x = torch.eye(K).bfloat16().cuda()
    for b in (2, 60, 127, 200, 251, 255):
        scales = torch.full((16, 1), b, dtype=torch.uint8).view(torch.float8_e8m0fnu)
        got = F.expert_matmul_mxfp4(x, codes.cuda(), scales.cuda(), dtype=F32).cpu().double().t()
        want = U.mxfp4_values(codes, scales)
        if b == 255:
            assert bool(got.isnan().all())
        else:
            assert torch.equal(got, want), b


def test_rows_of_one_expert_do_not_meet(F):
    """A NaN row leaves its neighbours alone, and so do rows of zeros."""
    rng = np.random.default_rng(0)
    codes, scales = _weights(rng, 0, 40, 64)
    x = U.bf16(rng, 20, 64)
    want = F.expert_matmul_mxfp4(x.cuda(), codes.cuda(), scales.cuda()).cpu()
    x[3], x[19] = float("nan"), 0
    got = F.expert_matmul_mxfp4(x.cuda(), codes.cuda(), scales.cuda()).cpu()
    keep = [i for i in range(20) if i not in (3, 19)]
    assert torch.equal(got[keep], want[keep])
    assert bool(got[3].isnan().all() and (got[19] == 0).all())
