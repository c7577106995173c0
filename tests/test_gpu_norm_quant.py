"""add_rms_norm and silu_mul_quantize against 64-bit references: every
format and row shape, blocks and rows of zeros, NaN and infinities, tiny and
large rows, in-place residuals, rows behind the last valid one left alone."""
import numpy as np
import pytest
import torch

from tests import expert_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# y relative to its exact value: the squares' sum over at most 32 terms a
# thread, 6 lane steps and 16 waves, halved by the root, division, root,
# reciprocal, two products and the rounding of s: fewer than 40 roundings
Y_REL = 40 * U.U32


@pytest.fixture(scope="module")
def X():
    from combine_route_mask_amd import experts, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return experts


def _reference(x, residual, weight, eps):
    s = x.double().cpu() + (residual.double().cpu() if residual is not None else 0)
    return s, s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * weight.double().cpu()


def _check_blocks(codes, scales, y, fmt, rel):
    """e4m3 codes times their block scale within half a step of y."""
    n = 32 if fmt == "mxfp8" else 128
    M, H = y.shape
    b = y.view(M, H // n, n)
    top = b.abs().amax(2)
    got = codes.cpu().float().double().view(M, H // n, n)
    if fmt == "mxfp8":
        e = scales.view(torch.uint8).cpu().double() - 127
        s = torch.exp2(e)
        # the smallest power of two that keeps the block within 448, decided
        # on values known to `rel`
        assert bool((top * (1 - rel) <= 448 * s).all()), "a block passes 448"
        assert bool(((top * (1 + rel) > 224 * s) | (e == -127)).all()), "a smaller scale would do"
    else:
        s = scales.double().cpu()
        assert bool(((s - top / 448).abs() <= (rel + 2 * U.U32) * top / 448 + 2.0 ** -149).all()), "scales"
    v = b.abs() / s.clamp(min=2.0 ** -140)[:, :, None]
    # half a step: 2^-4 of a normal value, 2^-10 of the scale below 2^-6;
    # deepseek_fp8 divides by its scale through two more roundings
    step = torch.maximum(v * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) * (1 + 2.0 ** -20) + v * (rel + 3 * U.U32)
    U.check_close((got * s[:, :, None]).view(M, H), y, (step * s[:, :, None]).view(M, H) + 2.0 ** -149, fmt)


# rows, hidden
SHAPES = [(1, 7168), (1, 128), (3, 256), (5, 512), (33, 640), (7, 1152), (4, 2048), (9, 2176), (6, 4096), (5, 8192),
          (3, 8320), (2, 16384), (2, 32768), (1025, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", ["int8", "mxfp8", "deepseek_fp8"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_add_rms_norm(X, M, H, fmt, dtype):
    log(f"norm M{M} H{H} {fmt} {dtype}")
    rng = np.random.default_rng(M + H)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x, res = draw(M, H).to(dtype), (4 * draw(M, H)).to(dtype)
    w = (1 + 0.2 * draw(H)).to(dtype)
    if M > 2:
        x[1], res[1] = x[1] * 2.0 ** -40, res[1] * 2.0 ** -40   # eps dominates
        x[2], res[2] = x[2] * 2.0 ** 40, res[2] * 2.0 ** 40
    w[-128:] = 0  # a block of zeros
    s, y = _reference(x, res, w, 1e-5)
    n = X.add_rms_norm(x.cuda(), res.cuda(), w.cuda(), 1e-5, format=fmt)
    U.check_close(n.residual, s, (U.unit(dtype) + U.U32) * s.abs() * 1.001, "residual")
    if fmt == "int8":
        U.check_int8(n.rows, n.scales, y, Y_REL, "int8")
        return
    _check_blocks(n.rows, n.scales, y, fmt, Y_REL)
    last = n.scales.view(torch.uint8).cpu().view(M, -1)[:, -4:]
    assert not bool(last.any()) and not bool(n.rows[:, -128:].float().any()), "a block of zeros"


@pytest.mark.parametrize("fmt,H", [("int8", 16), ("int8", 48), ("int8", 2064), ("mxfp8", 32), ("mxfp8", 96),
                                   ("mxfp8", 7200)])
@pytest.mark.parametrize("residual", [True, False])
def test_add_rms_norm_odd_sizes(X, fmt, H, residual):
    log(f"norm H{H} {fmt} residual={residual}")
    rng = np.random.default_rng(H)
    x = torch.from_numpy(rng.standard_normal((11, H)).astype(np.float32)).to(BF)
    res = x.flip(0).contiguous() if residual else None
    w = torch.from_numpy(rng.uniform(0.5, 2, H).astype(np.float32)).to(BF)
    s, y = _reference(x, res, w, 0.0)
    gx = x.cuda()
    n = X.add_rms_norm(gx, res.cuda() if residual else None, w.cuda(), 0.0, format=fmt)
    if fmt == "int8":
        U.check_int8(n.rows, n.scales, y, Y_REL, "int8")
    else:
        _check_blocks(n.rows, n.scales, y, fmt, Y_REL)
    assert residual or n.residual is gx


@pytest.mark.parametrize("fmt", ["int8", "mxfp8", "deepseek_fp8"])
def test_add_rms_norm_in_place_and_special_rows(X, fmt):
    H = 1024
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((8, H)).astype(np.float32)).to(BF).cuda()
    res = x.flip(1).contiguous()
    w = torch.ones(H, dtype=BF, device="cuda")
    want = X.add_rms_norm(x, res, w, format=fmt)
    into = res.clone()
    got = X.add_rms_norm(x, into, w, format=fmt, residual_out=into)
    assert got.residual is into
    for a, b in zip(want, got):
        assert np.array_equal(U.bits(a), U.bits(b))
    into = x.clone()
    got = X.add_rms_norm(into, res, w, format=fmt, residual_out=into)
    assert np.array_equal(U.bits(want.residual), U.bits(into)) and np.array_equal(U.bits(want.rows), U.bits(got.rows))
    x[1, 5], x[3, 7], x[4, 9] = float("nan"), float("inf"), float("-inf")
    x[5], res[5] = 0, 0
    x[6], res[6] = 3e38, 3e38  # squares past fp32
    bad = [1, 3, 4, 6]
    n = X.add_rms_norm(x, res, w, format=fmt)
    if fmt == "mxfp8":
        s = n.scales.view(torch.uint8)
        assert bool((s[bad] == 255).all()) and not bool((s[[0, 2, 7]] == 255).any()) and not bool(s[5].any())
    else:
        assert bool(n.scales[bad].isnan().all()) and bool(n.scales[[0, 2, 5, 7]].isfinite().all())
    codes = n.rows.view(torch.uint8)
    assert bool((codes[bad] == (0 if fmt == "int8" else 0x7F)).all()) and not bool(codes[5].any())
    for r in (0, 2, 7):  # their neighbours are what they were
        assert np.array_equal(U.bits(want.rows[r]), U.bits(n.rows[r]))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,I", [(1, 16), (3, 48), (5, 512), (9, 1040), (4, 2048), (3, 4112), (2, 8192), (2, 16400),
                                 (1, 32768), (700, 64)])
def test_silu_mul_quantize(X, M, I, dtype):
    log(f"silu M{M} I{I} {dtype}")
    rng = np.random.default_rng(I)
    x = torch.from_numpy((3 * rng.standard_normal((M, 2 * I))).astype(np.float32)).to(dtype)
    g, u = x.double().chunk(2, 1)
    ref = g / (1 + torch.exp(-g)) * u
    # exp of x takes |x| roundings of its argument and 4 of its own, the rest 4
    rel = (float(g.abs().max()) * 2 + 10) * U.U32
    q = X.silu_mul_quantize(x.cuda())
    U.check_int8(q.rows, q.scales, ref, rel, "silu")


def test_silu_rows_and_special_values(X):
    x = torch.randn(20, 64, device="cuda")
    x[2, 3] = float("nan")
    x[3, 40] = float("inf")
    x[4] = 0
    x[5, :32] = -200.0  # the activation vanishes
    want = X.silu_mul_quantize(x)
    offsets = torch.tensor([0, 3, 9, 11], dtype=torch.int32, device="cuda")
    out = torch.full((20, 32), 9, dtype=torch.int8, device="cuda")
    scales = torch.full((20,), 9.0, device="cuda")
    got = X.silu_mul_quantize(x, offsets=offsets, out=out, out_scales=scales)
    assert np.array_equal(U.bits(got.rows[:11]), U.bits(want.rows[:11])), "rows"
    assert np.array_equal(U.bits(got.scales[:11]), U.bits(want.scales[:11])), "scales"
    assert bool((got.rows[11:] == 9).all()) and bool((got.scales[11:] == 9).all()), "rows behind the last"
    assert bool(want.scales[2:4].isnan().all()) and not bool(want.rows[2:4].any())
    assert float(want.scales[4]) == 0.0 and not bool(want.rows[4].any())
    assert float(want.scales[5]) < 1e-80 or float(want.scales[5]) == 0.0
    # a count past the rows is taken as their number
    offsets[3] = 1000
    got = X.silu_mul_quantize(x, offsets=offsets)
    assert np.array_equal(U.bits(got.rows), U.bits(want.rows))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", ["int8", "mxfp8", "deepseek_fp8"])
def test_scales_and_codes_are_the_definitions(X, fmt, dtype):
    """Rows of 1 and -1 have the norm 1, so that y is the weight with their signs: the scales are the quotients of
    the largest magnitudes, correctly rounded, and the codes those of the values by the format's rule, exactly."""
    log(f"norm definitions {fmt} {dtype}")
    H, M = 4096, 5
    rng = np.random.default_rng(17)
    w = torch.from_numpy((rng.standard_normal(H) * np.exp2(rng.integers(-60, 60, size=H // 128).repeat(128))).astype(
        np.float32)).to(dtype)
    x = torch.from_numpy(rng.choice(np.float32([-1, 1]), size=(M, H))).to(dtype)
    n = X.add_rms_norm(x.cuda(), None, w.cuda(), 0.0, format=fmt)
    y = (x.float() * w.float()).view(M, -1, {"int8": H, "mxfp8": 32, "deepseek_fp8": 128}[fmt])
    top = y.abs().amax(2, keepdim=True)
    codes, scales = n.rows.cpu().float().view(y.shape), n.scales.cpu().view(top.shape)
    if fmt == "int8":
        assert torch.equal(scales, top / 127)
        q = 127 * y.double() / top.double()
        assert bool(((codes - q).abs() <= 0.5 + 2.0 ** -15).all())
    elif fmt == "mxfp8":
        e = torch.ceil(torch.log2(top.double() / 448))  # none of the largest magnitudes is 448 times a power of two
        assert torch.equal(scales.view(torch.uint8).double(), e + 127)
        assert torch.equal(codes, (y.double() / torch.exp2(e)).float().to(torch.float8_e4m3fn).float())
    else:
        assert torch.equal(scales, top / 448)
        # y * (448 / amax), each rounded to fp32 (torch takes `448 / top` as a reciprocal times 448, rounded twice)
        assert torch.equal(codes, (y * (torch.full_like(top, 448.0) / top)).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", ["int8", "mxfp8", "deepseek_fp8"])
@pytest.mark.parametrize("M,H", [(1, 128), (1025, 128), (4099, 256), (700, 1152), (300, 4224)])
def test_add_rms_norm_of_many_rows(X, M, H, fmt, dtype):
    """Every row and block against the 64-bit reference, no block of zeros."""
    log(f"norm of many rows M{M} H{H} {fmt} {dtype}")
    rng = np.random.default_rng(M * H)
    draw = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))  # noqa: E731
    x, res, w = draw(M, H).to(dtype), (4 * draw(M, H)).to(dtype), (1 + 0.2 * draw(H)).to(dtype)
    s, y = _reference(x, res, w, 1e-5)
    n = X.add_rms_norm(x.cuda(), res.cuda(), w.cuda(), 1e-5, format=fmt)
    U.check_close(n.residual, s, (U.unit(dtype) + U.U32) * s.abs() * 1.001, "residual")
    if fmt == "int8":
        U.check_int8(n.rows, n.scales, y, Y_REL, "int8")
        assert bool((n.scales > 0).all())
        # the largest value of a row has the code 127 or -127
        assert bool((n.rows.abs().amax(1) == 127).all())
    else:
        _check_blocks(n.rows, n.scales, y, fmt, Y_REL)


def test_codes_of_zero_rows_are_zeros(X):
    """Where the scale is 0 the codes are: rows of zeros, and a weight of zeros."""
    x = torch.randn(70, 128, device="cuda")
    x[::3] = 0
    n = X.add_rms_norm(x, None, torch.ones(128, device="cuda"), format="int8")
    assert torch.equal(n.scales == 0, (x == 0).all(1)) and not bool(n.rows[::3].any()) and bool(n.rows[1::3].any())
    q = X.silu_mul_quantize(x)
    assert torch.equal(q.scales == 0, (x == 0).all(1)) and not bool(q.rows[::3].any()) and bool(q.rows[1::3].any())
    for fmt in ("int8", "mxfp8", "deepseek_fp8"):
        n = X.add_rms_norm(x, None, torch.zeros(128, device="cuda"), format=fmt)
        assert not bool(n.rows.float().any()) and not bool(n.scales.view(torch.uint8).any())


@pytest.mark.parametrize("H", [128, 1024, 4096])
def test_more_rows_than_workgroups(X, H):
    """A workgroup's second row is what it is in a call of its own (2^20 workgroups at most; 64, 128 and 256 threads)."""
    M, half = (1 << 20) + 77, 1 << 19
    log(f"rows past the grid M{M} H{H}")
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    x = torch.randn((M, H), generator=g, device="cuda", dtype=BF)
    w = torch.randn(H, generator=g, device="cuda", dtype=BF)
    parts = [slice(0, half), slice(half, 2 * half), slice(2 * half, M)]
    for fmt in ("int8", "mxfp8", "deepseek_fp8"):
        n = X.add_rms_norm(x, x, w, format=fmt)
        for p in parts:
            m = X.add_rms_norm(x[p], x[p], w, format=fmt)
            assert torch.equal(n.rows[p].view(torch.uint8), m.rows.view(torch.uint8)), fmt
            assert torch.equal(n.scales[p].view(torch.uint8), m.scales.view(torch.uint8)), fmt
            assert torch.equal(n.residual[p], m.residual), fmt
        del n, m
    a = X.silu_mul_quantize(x)
    for p in parts:
        b = X.silu_mul_quantize(x[p])
        assert torch.equal(a.rows[p], b.rows) and torch.equal(a.scales[p], b.scales)
