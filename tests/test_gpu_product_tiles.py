"""The products over experts at sizes that choose each tile there is, of each
height, against 64-bit references: the 256-wide tiles of all bf16 products with
several steps, and the 4-bit product's stages of 16 rows with scales as words
and byte by byte.  ``test_product_shapes.py`` holds these sizes against the
rules that choose."""
import numpy as np
import pytest
import torch

from tests import ffn_util as U
from tests.gpu_util import log
from tests.test_gpu_ffn_layer import _normal, _product_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# rows an expert, channels, depth: row tiles of 64, 128, 192, 256 and 320 rows in the first
BF16_TILES = [((300, 290, 310, 255, 192, 128, 60, 1, 640, 500, 311, 277, 0), 4128, 544), ((600,) * 6, 2080, 1056),
              ((250,) * 16, 2080, 1056)]
BEFORE, BEHIND = 3, 5  # rows outside the experts'

# rows, experts, channels, depth, kind of offsets; channels beyond a multiple of 64 and of 4, experts of more than 16 rows
FOUR_BIT_TILES = [(40, 8, 2106, 1280, "ragged"), (40, 8, 2106, 1184, "ragged"), (30, 30, 700, 96, "single rows"),
                  (16, 0, 16390, 384, ""), (100, 16, 2106, 1280, "ragged"), (100, 16, 2106, 1184, "ragged"),
                  (150, 10, 4098, 160, "one"), (64, 64, 1030, 256, "ragged")]


@pytest.fixture(scope="module")
def F():
    from combine_route_mask_amd import ffn, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return ffn


def _offsets(counts):
    o = (np.concatenate([[0], np.cumsum(counts)]) + BEFORE).astype(np.int32)
    rows = int(o[-1]) + BEHIND
    held = (torch.arange(rows) >= BEFORE) & (torch.arange(rows) < int(o[-1]))
    return o, torch.from_numpy(o).cuda(), rows, held


def _outside(t, held):
    """NaN in the rows outside the experts': they reach nothing."""
    t[~held.cuda()] = float("nan")
    return t


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts,n,k", BF16_TILES)
def test_product(F, counts, n, k, transposed):
    log(f"product of {len(counts)} experts {n}x{k} transposed={transposed}")
    o, off, rows, held = _offsets(counts)
    x = _normal(1, rows, k)
    w = _normal(2, len(counts), *((k, n) if transposed else (n, k)), size=k ** -0.5)
    ref, bound, _ = _product_gpu(x, w, o, transposed)
    out = torch.full((rows, n), 7.0, dtype=BF, device="cuda")
    F.expert_product(_outside(x, held), w, offsets=off, transposed=transposed, out=out)
    U.close(out[held.cuda()], ref[held], U.rounded(bound, ref)[held], "product")
    assert bool((out.cpu()[~held] == 7).all())


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
@pytest.mark.parametrize("counts,n,k", BF16_TILES)
def test_gated_product(F, counts, n, k, checkpoint):
    """`n` channels, gate and up."""
    I = n // 2 // 32 * 32
    log(f"gated of {len(counts)} experts {I}x{k} {checkpoint}")
    o, off, rows, held = _offsets(counts)
    x, w = _normal(1, rows, k), _normal(2, len(counts), 2 * I, k, size=2 * k ** -0.5)
    pre, poff, _ = _product_gpu(x, w, o, False)
    ref, bound = U.gated(pre, poff)
    got, kept, scales = F.gated_product(_outside(x, held), w, offsets=off, checkpoint=checkpoint)
    U.close(got[held.cuda()], ref[held], U.rounded(bound, ref)[held], "gated")
    pre, poff = pre[held], poff[held]
    kept, scales = kept.cpu()[held], scales.view(torch.uint8).cpu()[held]
    if checkpoint == "bf16":
        U.close(U.half_values(kept, scales), pre, U.half_step(pre, poff), "pre")
    else:
        exponent = scales.double() - 127
        step = torch.maximum(2.0 ** -4 * pre.abs(), torch.exp2(exponent - 10).repeat_interleave(32, dim=1))
        U.close(U.mx_values(kept, scales), pre, step + poff * (1 + 2.0 ** -4), "MXFP8 pre")


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
@pytest.mark.parametrize("counts,n,k", BF16_TILES)
def test_gated_product_backward(F, counts, n, k, checkpoint):
    """`n` channels of the activation, through weights [k, n]."""
    log(f"gated backward of {len(counts)} experts {n}x{k} {checkpoint}")
    o, off, rows, held = _offsets(counts)
    dy, w = _normal(1, rows, k), _normal(2, len(counts), k, n, size=k ** -0.5)
    pre = _normal(3, rows, 2 * n, size=3.0)
    if checkpoint == "mxfp8":
        given, scales = F.checkpoint_rows(pre)
        values = U.mx_values(given, scales)
    else:
        given = pre.half()
        g = torch.Generator(device="cuda")
        g.manual_seed(4)
        scales = torch.randint(124, 130, (rows, 2 * n // 8), generator=g, device="cuda",
                               dtype=torch.uint8).view(torch.float8_e8m0fnu)
        values = U.half_values(given, scales)
    d, doff, _ = _product_gpu(dy, w, o, True)
    ref, bound, act, abound = U.gated_backward(d, doff, values)
    got, again = F.gated_product_backward(_outside(dy, held), w, given, scales, offsets=off)
    U.close(got[held.cuda()], ref[held], U.rounded(bound, ref)[held], "grad_pre")
    U.close(again[held.cuda()], act[held], U.rounded(abound, act)[held], "activation")
    alone, none = F.gated_product_backward(dy, w, given, scales, offsets=off, need_rows=False)
    assert none is None and torch.equal(alone[held.cuda()], got[held.cuda()])


@pytest.mark.parametrize("counts,n,k", BF16_TILES)
def test_weight_grad(F, counts, n, k):
    """Rows before the first expert's and behind the last one's are NaN: no sum has them."""
    log(f"weight grad of {len(counts)} experts {n}x{k}")
    o, off, rows, held = _offsets(counts)
    dy, x = _outside(_normal(1, rows, n), held), _outside(_normal(2, rows, k), held)
    got = F.product_weight_grad(dy, x, offsets=off)
    for e, (a, b) in enumerate(zip(o, o[1:])):
        ref = dy[a:b].double().t() @ x[a:b].double()
        mag = dy[a:b].double().abs().t() @ x[a:b].double().abs()
        U.close(got[e], ref.cpu(), U.rounded(int(b - a) * 2 * U.U32 * mag, ref).cpu(), "grad_w")


def test_block_zeros_its_rest(F):
    """The block and its gradient at these tiles: rows outside the experts' are zeros, the others the parts'."""
    counts, n, k = BF16_TILES[1]
    o, off, rows, held = _offsets(counts)
    H, I = n, k
    x, dy = _outside(_normal(1, rows, H), held), _outside(_normal(2, rows, H), held)
    w1, w2 = _normal(3, len(counts), 2 * I, H, size=H ** -0.5), _normal(4, len(counts), H, I, size=I ** -0.5)
    y, saved = F.expert_ffn_forward(x, w1, w2, offsets=off)
    gx, _, _ = F.expert_ffn_backward(dy, saved, w1, w2, offsets=off, needs=(True, False, False))
    act = F.gated_product(x, w1, offsets=off)[0]
    want = F.expert_product(act, w2, offsets=off, out=torch.zeros_like(x))
    assert torch.equal(y, want) and bool(y[held.cuda()].isfinite().all())
    assert not bool(gx[~held.cuda()].any()) and bool(gx[held.cuda()].isfinite().all())


def _four_bit(rng, M, E, N, K, kind, scales_at):
    o = U.ragged(rng, M, E, kind) if E else None
    many = (E,) if E else ()
    codes = torch.from_numpy(rng.integers(0, 256, (*many, N, K // 2), dtype=np.uint8))
    count = int(np.prod((*many, N, K // 32)))
    # scales that begin `scales_at` bytes behind an aligned address
    space = torch.from_numpy(rng.integers(120, 130, count + 16, dtype=np.uint8)).cuda()
    scales = space[scales_at:scales_at + count].view(*many, N, K // 32)
    return o, U.bf16(rng, M, K), codes, scales.view(torch.float8_e8m0fnu)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scales_at", [0, 1])
@pytest.mark.parametrize("M,E,N,K,kind", FOUR_BIT_TILES)
def test_four_bit_product(F, M, E, N, K, kind, scales_at, dtype, gated):
    log(f"4-bit {M}x{N}x{K} over {E} {kind} {dtype} gated={gated} scales at {scales_at}")
    rng = np.random.default_rng(M + N + K)
    o, x, codes, scales = _four_bit(rng, M, E, N, K, kind, scales_at)
    w = U.mxfp4_values(codes, scales.cpu()).cuda()
    bounds = np.array([0, M]) if o is None else o
    # w is exact in bf16
    ref, bound, held = _product_gpu(x.cuda(), (w if E else w[None]).bfloat16(), bounds, False)
    if gated:
        ref, bound = U.gated(ref, bound)
    x[~held] = float("nan")
    off = None if o is None else torch.from_numpy(o).cuda()
    out = torch.full(ref.shape, 7.0, dtype=dtype, device="cuda")
    got = F.expert_matmul_mxfp4(x.cuda(), codes.cuda(), scales, offsets=off, gated=gated, out=out)
    U.close(got.cpu()[held], ref[held], U.rounded(bound, ref, dtype)[held], "4-bit product")
    assert bool((got.cpu()[~held] == 7).all())
