"""The int8 product over experts against exact integer sums: ragged and empty
experts, one row, odd channel counts, every k tail, rows outside the experts'
ranges left alone, the extreme codes at the longest k."""
import numpy as np
import pytest
import torch

from tests import expert_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def X():
    from combine_route_mask_amd import experts, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return experts


def _inputs(rng, M, E, N, K):
    x = torch.from_numpy(rng.integers(-128, 128, size=(M, K), dtype=np.int8))
    w = torch.from_numpy(rng.integers(-128, 128, size=(E, N, K), dtype=np.int8))
    sx = torch.from_numpy(rng.uniform(0.001, 2, size=M).astype(np.float32))
    sw = torch.from_numpy(rng.uniform(0.001, 2, size=(E, N)).astype(np.float32))
    return x, w, sx, sw


def _reference(x, w, sx, sw, offsets):
    """Integer sums in float64 (exact below 2^53), rows without an expert NaN."""
    y = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64)
    xd = x.double().cuda()
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            acc = (xd[a:b] @ w[e].double().cuda().t().contiguous()).cpu()
            y[a:b] = acc * sx[a:b].double()[:, None] * sw[e].double()
    return y


def _check(got, ref, dtype, fill):
    # fp32: the sum's conversion, the scales' product and the product round once each
    held = ~ref.isnan()
    bound = torch.where(held, (U.unit(dtype) + 3.01 * U.U32 * (1 + U.unit(dtype))) * ref.abs(), 0.0)
    assert bool((got.cpu()[~held] == fill).all()), "a row outside the experts' ranges was written"
    U.check_close(got.cpu()[held], ref[held], bound[held], "product")


def _ragged(rng, M, E, kind):
    if kind == "even":
        counts = np.full(E, M // E)
    elif kind == "one":
        counts = np.zeros(E, int)
        counts[E // 2] = M
    elif kind == "single rows":
        counts = (np.arange(E) < M).astype(int)
    else:
        counts = np.bincount(rng.integers(0, max(1, E - 1), size=max(0, M - 2)), minlength=E)  # two rows left over
        counts[rng.random(E) < 0.2] = 0
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


CASES = [
    (1, 1, 1, 16, "even"), (1, 4, 17, 48, "one"), (3, 2, 64, 64, "ragged"), (64, 32, 4096, 7168, "ragged"),
    (8, 8, 256, 7168, "single rows"), (100, 300, 33, 80, "ragged"), (257, 5, 130, 144, "ragged"),
    (500, 3, 2055, 2064, "ragged"), (1023, 1, 2055, 2064, "even"), (700, 4, 512, 4096, "one"),
    (2048, 8, 512, 1024, "even"), (2300, 8, 515, 1040, "ragged"), (5000, 2, 258, 16, "ragged"),
    (5000, 7, 300, 112, "ragged"), (4096, 16, 1024, 512, "ragged"), (1500, 4096, 8, 32, "ragged"),
    (16, 1, 1024, 131056, "even"), (520, 1, 264, 16384, "even"), (2048, 8, 2055, 1040, "ragged"),
    (2100, 4, 16400, 4112, "ragged"), (600, 40, 700, 1040, "ragged"), (3100, 12, 4400, 1552, "ragged"),
    (2600, 20, 1290, 4224, "ragged"),
    # several tiles a workgroup, more experts than a wave has lanes
    (9000, 100, 1500, 272, "ragged"), (5100, 17, 3400, 1040, "ragged"), (4900, 16, 3401, 1136, "ragged"), (300, 70, 1000, 4112, "ragged"), (14000, 70, 1100, 1040, "ragged"),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,E,N,K,kind", CASES)
def test_expert_product(X, M, E, N, K, kind, dtype):
    log(f"product M{M} E{E} N{N} K{K} {kind} {dtype}")
    rng = np.random.default_rng(M + E + N + K)
    x, w, sx, sw = _inputs(rng, M, E, N, K)
    offsets = _ragged(rng, M, E, kind)
    ref = _reference(x, w, sx, sw, offsets)
    out = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
    got = X.expert_matmul(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), offsets=torch.from_numpy(offsets).cuda(), out=out)
    _check(got, ref, dtype, 3.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(1, 7, 32), (1, 4096, 7168), (17, 64, 4096), (129, 129, 128), (300, 1000, 2064),
                                   (2049, 513, 1040)])
def test_dense_product(X, M, N, K, dtype):
    log(f"dense M{M} N{N} K{K} {dtype}")
    rng = np.random.default_rng(M + N + K)
    x, w, sx, sw = _inputs(rng, M, 1, N, K)
    ref = _reference(x, w, sx, sw, [0, M])
    _check(X.expert_matmul(x.cuda(), sx.cuda(), w[0].cuda(), sw[0].cuda(), dtype=dtype), ref, dtype, 0)


@pytest.mark.parametrize("M", [3, 300])
def test_extreme_codes(X, M):
    """-128 everywhere at the longest k: 2^31 - 2^18, still an int32."""
    K, N = 131056, 20
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = torch.ones(max(M, N), device="cuda")
    y = X.expert_matmul(x, one[:M], w, one[:N], dtype=F32)
    assert bool((y[:, 0] == 16384.0 * K).all()) and bool((y[:, 1] == float(np.float32(-16256 * K))).all())


def test_most_rows(X):
    """As many rows as a call takes: the last ones and the first have their products."""
    M, K = 2 ** 31 - 1, 16
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GiB of free device memory")
    log(f"product M{M} N1 K{K}")
    x = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    sx = torch.ones(M, device="cuda")
    w = torch.arange(1, K + 1, dtype=torch.int8, device="cuda").view(1, K)
    for at in (slice(0, 300), slice(M - 300, M)):
        x[at] = torch.arange(300, device="cuda").remainder(120).to(torch.int8)[:, None]
    want = torch.arange(300, device="cuda").remainder(120).float() * (K * (K + 1) // 2)
    for offsets in (None, torch.tensor([0, M], dtype=torch.int32, device="cuda")):
        y = torch.full((M, 1), 3.0, device="cuda")
        X.expert_matmul(x, sx, w if offsets is None else w[None], sx[:1] if offsets is None else sx[None, :1],
                        offsets=offsets, out=y)
        assert torch.equal(y[:300, 0], want) and torch.equal(y[-300:, 0], want)
        assert not bool(y[300:-300].any())
        del y


def test_offsets_beyond_the_rows(X):
    """Offsets past the rows are taken as their number, descending ones as empty: nothing is written out of range."""
    rng = np.random.default_rng(5)
    x, w, sx, sw = _inputs(rng, 40, 3, 24, 64)
    room = torch.full((60, 24), 3.0, device="cuda")
    off = torch.tensor([-7, 10, 1000, 2], dtype=torch.int32, device="cuda")
    X.expert_matmul(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), offsets=off, out=room[:40])
    ref = _reference(x, w, sx, sw, [0, 10, 40, 40])
    _check(room[:40], ref, F32, 3.0)
    assert bool((room[40:] == 3).all())


def test_row_scales_carry_nan(X):
    """A row whose scale is NaN (it held a NaN before it was quantised) is NaN throughout, its neighbours are not."""
    x, w, sx, sw = _inputs(np.random.default_rng(6), 20, 1, 40, 64)
    sx[7] = float("nan")
    x[7] = 0
    y = X.expert_matmul(x.cuda(), sx.cuda(), w[0].cuda(), sw[0].cuda()).cpu()
    assert bool(y[7].isnan().all()) and int(y.isnan().sum()) == 40


def test_most_channels(X):
    """As many channels as a call takes: the first and the last have their products, and nothing is written behind them."""
    M, N, K = 2, 2 ** 31 - 1, 16
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free device memory")
    log(f"product M{M} N{N} K{K}")
    x = torch.arange(1, K + 1, dtype=torch.int8, device="cuda").repeat(M, 1)
    x[1] *= -1
    sx = torch.ones(M, device="cuda")
    sw = torch.ones(N, device="cuda")
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    ramp = torch.arange(300, device="cuda").remainder(120)
    for at in (slice(0, 300), slice(N - 300, N)):
        w[at] = ramp.to(torch.int8)[:, None]
    want = (ramp.float() * (K * (K + 1) // 2)).to(BF)
    for offsets in (None, torch.tensor([0, M], dtype=torch.int32, device="cuda")):
        room = torch.full((M * N + 64,), 3.0, dtype=BF, device="cuda")
        y = room[:M * N].view(M, N)
        X.expert_matmul(x, sx, w if offsets is None else w[None], sw if offsets is None else sw[None],
                        offsets=offsets, out=y)
        for m, sign in enumerate((1, -1)):
            assert torch.equal(y[m, :300], sign * want) and torch.equal(y[m, -300:], sign * want)
            assert not bool(y[m, 300:-300].any())
        assert bool((room[M * N:] == 3).all())
        del room, y


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(5, 24, 64), (130, 40, 1040)])
def test_scales_of_extreme_rows(X, M, N, K, dtype):
    """Rows of any magnitude that fp32 holds: the scales' own product may be below fp32 (rows of about 2^-130) or past
    it (2^125 by channels of 2^4) where the result is not, and a sum of zero stays zero beside it."""
    rng = np.random.default_rng(M)
    x, w, sx, sw = _inputs(rng, M, 1, N, K)
    sw = sw * 2.0 ** -10
    exponent = torch.tensor([-135.0, -126.0, -118.0, 95.0, 0.0])[torch.arange(M) % 5]
    sx = sx.double().mul(torch.exp2(exponent.double())).float()
    w[0, 7] = 0          # sums of zero, with scales whose product with the rows' is past fp32
    sw[0, 7] = 2.0 ** 100
    ref = _reference(x, w, sx, sw, [0, M])
    assert bool((ref[:, 7] == 0).all()) and float(ref.abs().max()) < 2.0 ** 127
    got = X.expert_matmul(x.cuda(), sx.cuda(), w[0].cuda(), sw[0].cuda(), dtype=dtype)
    # three roundings and the last one's; among the smallest numbers the last fp32 one is off by up to half of
    # 2^-149 and the one to bf16 by up to half of 2^-133
    bound = ((U.unit(dtype) + 3.01 * U.U32 * (1 + U.unit(dtype))) * ref.abs() + 2.0 ** -150 +
             (2.0 ** -134 if dtype == BF else 0.0))
    U.check_close(got, ref, bound, "scaled product")
