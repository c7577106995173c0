"""The gated feed-forward block of experts, its gradients and its 8-bit
checkpoints against 64-bit references: ragged and empty experts, one row, odd
widths, rows outside the experts' ranges, each order of the weights' axes."""
import numpy as np
import pytest
import torch

from tests import ffn_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from combine_route_mask_amd import ffn, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return ffn


# rows, experts (0: dense), first width, second width, kind of offsets
SHAPES = [
    (1, 1, 8, 8, "even"), (1, 0, 64, 32, ""), (3, 5, 16, 24, "single rows"), (33, 4, 72, 40, "ragged"),
    (64, 2, 64, 64, "one"), (65, 3, 96, 160, "ragged"), (129, 7, 264, 136, "ragged"), (200, 0, 136, 520, ""),
    (300, 64, 200, 72, "ragged"), (50, 3, 32, 32, "none"), (700, 3, 328, 776, "ragged"), (1500, 2, 520, 264, "one"),
    (2100, 0, 776, 392, ""), (1025, 130, 64, 96, "ragged"), (40, 4096, 32, 64, "ragged"), (4000, 6, 512, 1024, "ragged"),
]


def _offsets(rng, M, E, kind):
    o = U.ragged(rng, M, E, kind) if E else None
    return o, None if o is None else torch.from_numpy(o).cuda()


def _weight(rng, E, N, K):
    return U.bf16(rng, *((E, N, K) if E else (N, K)), size=K ** -0.5)


def _rest(out, held, fill, what):
    assert bool((out.cpu()[~held] == fill).all()), f"{what}: a row outside the experts' ranges was written"


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,E,N,K,kind", SHAPES)
def test_product(F, M, E, N, K, kind, transposed):
    log(f"product {M}x{N}x{K} over {E} {kind} transposed={transposed}")
    rng = np.random.default_rng(M + N)
    o, off = _offsets(rng, M, E, kind)
    x, w = U.bf16(rng, M, K), _weight(rng, E, N, K)
    if transposed:
        w = w.transpose(-1, -2).contiguous()
    ref, bound, held = U.product(x, w, o, transposed)
    if o is not None:
        x[~held] = float("nan")  # rows without an expert reach nothing
    out = torch.full((M, N), 7.0, dtype=BF, device="cuda")
    got = F.expert_product(x.cuda(), w.cuda(), offsets=off, transposed=transposed, out=out)
    assert got is out
    U.close(got.cpu()[held], ref[held], U.rounded(bound, ref)[held], "product")
    _rest(got, held, 7.0, "product")


@pytest.mark.parametrize("checkpoint", [None, "bf16", "mxfp8"])
@pytest.mark.parametrize("M,E,I,K,kind", SHAPES)
def test_gated_product(F, M, E, I, K, kind, checkpoint):
    if checkpoint == "mxfp8":
        I = (I + 31) // 32 * 32
    log(f"gated {M}x{I}x{K} over {E} {kind} {checkpoint}")
    rng = np.random.default_rng(M + I)
    o, off = _offsets(rng, M, E, kind)
    x, w = U.bf16(rng, M, K), _weight(rng, E, 2 * I, K) * 2
    pre, poff, held = U.product(x, w, o)
    ref, bound = U.gated(pre, poff)
    out = torch.full((M, I), 7.0, dtype=BF, device="cuda")
    got, kept, scales = F.gated_product(x.cuda(), w.cuda(), offsets=off, checkpoint=checkpoint, out=out)
    U.close(got.cpu()[held], ref[held], U.rounded(bound, ref)[held], "gated")
    _rest(got, held, 7.0, "gated")
    if checkpoint is None:
        assert kept is None and scales is None
    elif checkpoint == "bf16":
        assert kept.dtype == torch.float16 and scales.shape == (M, 2 * I // 8)
        if bool(held.any()):
            U.close(U.half_values(kept, scales)[held], pre[held], U.half_step(pre[held], poff[held]), "pre")
    elif bool(held.any()):
        p, q = pre[held], poff[held]
        exponent = scales.cpu()[held].view(torch.uint8).double() - 127
        blocks = p.view(p.shape[0], -1, 32)
        near = q.view(blocks.shape)
        lo, hi = (blocks.abs() - near).amax(2).clamp(min=0), (blocks.abs() + near).amax(2)
        assert bool((U.mx_scale(lo) <= exponent).all() and (exponent <= U.mx_scale(hi)).all()), "scales"
        step = torch.maximum(2.0 ** -4 * blocks.abs(), torch.exp2(exponent - 10)[:, :, None]).view(p.shape)
        U.close(U.mx_values(kept.cpu()[held], scales.cpu()[held]), p, step + q * (1 + 2.0 ** -4), "MXFP8 pre")


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
@pytest.mark.parametrize("M,E,I,N,kind", SHAPES)
def test_gated_product_backward(F, M, E, I, N, kind, checkpoint):
    if checkpoint == "mxfp8":
        I = (I + 31) // 32 * 32
    log(f"gated backward {M}x{I}x{N} over {E} {kind} {checkpoint}")
    rng = np.random.default_rng(M + I + 1)
    o, off = _offsets(rng, M, E, kind)
    dy, w = U.bf16(rng, M, N), _weight(rng, E, N, I)
    pre = U.bf16(rng, M, 2 * I, size=3.0)
    d, doff, held = U.product(dy, w, o, transposed=True)
    if checkpoint == "mxfp8":
        given, scales = F.checkpoint_rows(pre.cuda())
        pre = U.mx_values(given, scales)
    else:
        given = pre.half().cuda()
        scales = torch.from_numpy(rng.integers(124, 130, (M, 2 * I // 8), dtype=np.uint8)).view(torch.float8_e8m0fnu).cuda()
        pre = U.half_values(given, scales)
    ref, bound, rows, rbound = U.gated_backward(d, doff, pre.double())
    got, again = F.gated_product_backward(dy.cuda(), w.cuda(), given, scales, offsets=off)
    U.close(got.cpu()[held], ref[held], U.rounded(bound, ref)[held], "grad_pre")
    U.close(again.cpu()[held], rows[held], U.rounded(rbound, rows)[held], "activation")
    alone, none = F.gated_product_backward(dy.cuda(), w.cuda(), given, scales, offsets=off, need_rows=False)
    assert none is None and torch.equal(alone.cpu()[held], got.cpu()[held])


@pytest.mark.parametrize("M,E,N,K,kind", SHAPES)
def test_weight_grad(F, M, E, N, K, kind):
    log(f"weight grad {M}x{N}x{K} over {E} {kind}")
    rng = np.random.default_rng(M + K + 2)
    o, off = _offsets(rng, M, E, kind)
    dy, x = U.bf16(rng, M, N), U.bf16(rng, M, K)
    ref, bound = U.outer(dy, x, o, max(E, 1))
    if o is not None:
        dy[o[-1]:], x[o[-1]:] = float("nan"), float("nan")
    got = F.product_weight_grad(dy.cuda(), x.cuda(), offsets=off)
    U.close(got.cpu().view(ref.shape), ref, U.rounded(bound, ref), "grad_w")


def test_saved_products_of_extremes(F):
    """Large, small and unequal products keep 11 bits beside their largest; what is no finite number stays so."""
    w = torch.eye(16, dtype=BF).repeat(2, 1)  # gate = up = x
    x = torch.ones(6, 16, dtype=BF)
    x[0], x[1], x[2, 3], x[3, 9] = 2.0 ** 127, 2.0 ** -126, float("inf"), float("nan")
    x[4, :8] = torch.tensor([1, 2.0 ** -8, 2.0 ** -13, 0, -3, 100, -2.0 ** -9, 7], dtype=BF)
    x[5] = 0
    _, pre, scales = F.gated_product(x.cuda(), w.cuda(), checkpoint="bf16")
    got = U.half_values(pre, scales)[:, :16]
    want = x.double() @ w[:16].double().t()  # 0 times an infinity or NaN is NaN in the other channels
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    fine = want.isfinite()
    assert torch.equal(got[fine], want[fine])  # each is a bf16 number within 2^-14 of its eight's largest


def _pieces(F, x, w1, w2, off, checkpoint, dy):
    """The block and its gradients from its parts."""
    rows, pre, scales = F.gated_product(x, w1, offsets=off, checkpoint=checkpoint)
    y = F.expert_product(rows, w2, offsets=off, out=torch.zeros_like(x))
    kept = x if checkpoint == "bf16" else F.restore_rows(*F.checkpoint_rows(x))
    grad_pre, again = F.gated_product_backward(dy, w2, pre, scales, offsets=off)
    dx = F.expert_product(grad_pre, w1, offsets=off, transposed=True, out=torch.zeros_like(x))
    return y, dx, F.product_weight_grad(grad_pre, kept, offsets=off), F.product_weight_grad(dy, again, offsets=off)


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
@pytest.mark.parametrize("M,E,H,I,kind", [(1, 1, 32, 32, "even"), (300, 5, 160, 96, "ragged"), (130, 0, 96, 352, ""),
                                          (50, 3, 32, 64, "none"), (900, 2, 512, 288, "one")])
def test_block(F, M, E, H, I, kind, checkpoint):
    """Autograd's block and the explicit calls are the parts' results, rows outside the experts' ranges zeros."""
    log(f"block {M}x{H}x{I} over {E} {kind} {checkpoint}")
    rng = np.random.default_rng(M)
    o, off = _offsets(rng, M, E, kind)
    x, dy = U.bf16(rng, M, H).cuda(), U.bf16(rng, M, H).cuda()
    w1, w2 = _weight(rng, E, 2 * I, H).cuda(), _weight(rng, E, H, I).cuda()
    want = _pieces(F, x, w1, w2, off, checkpoint, dy)
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    y = F.expert_ffn(*leaves, offsets=off, checkpoint=checkpoint)
    got = (y.detach(), *torch.autograd.grad(y, leaves, dy))
    for g, w, name in zip(got, want, ("y", "grad_x", "grad_w1", "grad_w2")):
        assert torch.equal(g, w), name
    y2, saved = F.expert_ffn_forward(x, w1, w2, offsets=off, checkpoint=checkpoint)
    assert torch.equal(y2, want[0])
    for needs in ((True, False, False), (False, True, False), (False, False, True)):
        grads = F.expert_ffn_backward(dy, saved, w1, w2, offsets=off, needs=needs)
        for g, w, need in zip(grads, want[1:], needs):
            assert torch.equal(g, w) if need else g is None
    last = M if o is None else int(o[-1])
    plain = F.expert_ffn(x, w1, w2, offsets=off, checkpoint=checkpoint)
    assert torch.equal(plain[:last], want[0][:last])


def test_formula_against_differences():
    """The gradient's formula, in 64 bits, against central differences of the block's."""
    rng = np.random.default_rng(3)
    M, H, I = 3, 4, 2
    x, w1, w2, dy = (torch.from_numpy(rng.standard_normal(s)) for s in ((M, H), (2 * I, H), (H, I), (M, H)))

    def loss(x, w1, w2):
        pre = x @ w1.t()
        return float(((U.silu(pre[:, :I]) * pre[:, I:]) @ w2.t() * dy).sum())

    grad_pre, _, rows, _ = U.gated_backward(dy @ w2, torch.zeros(M, I), x @ w1.t())
    grads = (grad_pre @ w1, grad_pre.t() @ x, dy.t() @ rows)
    for i, (t, g) in enumerate(zip((x, w1, w2), grads)):
        for at in np.ndindex(*t.shape):
            args = [[a.clone() for a in (x, w1, w2)] for _ in range(2)]
            h = 1e-5
            args[0][i][at] += h
            args[1][i][at] -= h
            # the third derivative times h^2 / 6 and 2^-52 |loss| / h are below 1e-8
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * h) - float(g[at])) < 1e-7


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("M,H", [(1, 32), (3, 96), (1000, 160), (7, 7168), (70000, 32)])
def test_checkpoint_rows(F, M, H, dtype):
    log(f"checkpoint {M}x{H} {dtype}")
    rng = np.random.default_rng(H)
    x = torch.from_numpy((rng.standard_normal((M, H)) * 2.0 ** rng.integers(-40, 40, (M, 1))).astype(np.float32)).to(dtype)
    x[0, :32] = 0
    if H > 64:
        x[0, 32:64] = torch.linspace(-448, 448, 32).to(dtype)  # a block on the border of its scale
    c = F.checkpoint_rows(x.cuda())
    exponent = U.mx_scale(x.double().abs().view(M, -1, 32).amax(2))
    want = U.mx_round(x, exponent)
    assert torch.equal(c.scales.cpu().view(torch.uint8).double(), exponent + 127)
    assert torch.equal(U.mx_values(c.rows, c.scales), want)
    for t in (BF, torch.float32):
        assert torch.equal(F.restore_rows(c.rows, c.scales, dtype=t).cpu().double(), want)


def test_checkpoint_of_extremes(F):
    """Blocks with a NaN or an infinity are NaN, their neighbours are not; the largest and smallest numbers."""
    x = torch.ones(4, 64)
    x[0, 3], x[1, 40], x[2, :32], x[3, :32] = float("nan"), float("-inf"), torch.finfo(torch.float32).max, 2.0 ** -120
    c = F.checkpoint_rows(x.cuda())
    back = F.restore_rows(c.rows, c.scales, dtype=torch.float32).cpu()
    nan = torch.zeros(4, 64, dtype=torch.bool)
    nan[0, :32] = nan[1, 32:] = True
    assert torch.equal(back.isnan(), nan)
    assert bool((back[0, 32:] == 1).all() and (back[1, :32] == 1).all() and (back[3, :32] == 2.0 ** -120).all())
    # the largest fp32 number is 2^128 less a step: e4m3 rounds it to 256 * 2^120
    assert bool(torch.isinf(back[2, :32]).all())
    every = torch.arange(256, dtype=torch.uint8).view(8, 32)
    scales = torch.tensor([0, 1, 100, 127, 150, 254, 255, 127], dtype=torch.uint8).view(8, 1)
    got = F.restore_rows(every.view(torch.float8_e4m3fn).cuda(), scales.view(torch.float8_e8m0fnu).cuda(),
                         dtype=torch.float32).cpu()
    want = U.mx_values(every.view(torch.float8_e4m3fn), scales).float()
    want[6] = float("nan")
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
