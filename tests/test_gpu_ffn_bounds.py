"""The products over experts touch their own rows only, whatever the offsets
hold: every buffer lies between rows of a pattern that must stay, inputs outside
the experts' rows are NaN, and the entry points are called with outputs that the
binding would allocate itself."""
import numpy as np
import pytest
import torch

from tests import ffn_util as U
from tests.gpu_util import log
from tests.test_ffn_refusals import _pack
from tests.test_gpu_ffn_layer import _normal

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
GUARD = 64  # rows before and behind a buffer


@pytest.fixture(scope="module")
def L():
    from combine_route_mask_amd import ffn, moe_ep, router
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()

    class Modules:
        F, R, m = ffn, router, moe_ep
    return Modules


class Guarded:
    """An output of `rows` rows between guards, all of a pattern."""

    def __init__(self, rows, width, dtype):
        item = torch.empty((), dtype=dtype).element_size()
        self.space = torch.full((rows + 2 * GUARD, width * item), 0x5A, dtype=torch.uint8, device="cuda")
        self.bytes = self.space[GUARD:GUARD + rows]
        self.t = self.bytes.view(dtype)

    def ptr(self):
        return self.bytes.data_ptr()

    def check(self, held, what):
        """`held`: the rows that may have been written."""
        s = self.space.cpu()
        s[GUARD:GUARD + self.bytes.shape[0]][held] = 0x5A
        assert bool((s == 0x5A).all()), f"{what}: written outside its rows"


def _surrounded(t):
    """The same rows between rows of NaN."""
    wide = torch.full((t.shape[0] + 2 * GUARD, t.shape[1]), float("nan"), dtype=t.dtype, device="cuda")
    wide[GUARD:GUARD + t.shape[0]] = t
    return wide[GUARD:GUARD + t.shape[0]]


# entries of the offsets -> the experts' rows as they are documented (None: they do not ascend, only the bounds hold)
def _offsets(M, kind):
    third = M // 3
    return {"below and past": ([-7, third, 2 * third, 2 ** 31 - 1], [0, third, 2 * third, M]),
            "first and last rows outside": ([5, third, third, M - 7], [5, third, third, M - 7]),
            "past the rows": ([2 ** 31 - 1] * 4, [M] * 4), "below": ([-2 ** 31, -5, -1, 0], [0] * 4),
            "not ascending": ([third, 10, M - 5, 20], None),
            "falling": ([M, 2 * third, third, 0], None)}[kind]


@pytest.mark.parametrize("kind", ["below and past", "first and last rows outside", "past the rows", "below",
                                  "not ascending", "falling"])
@pytest.mark.parametrize("M,H,I", [(40, 64, 32), (700, 328, 264), (2000, 2064, 2080)])
def test_rows_outside_stay(L, M, H, I, kind):
    log(f"bounds {M}x{H}x{I} {kind}")
    F, lib, E = L.F, L.m.lib, 3
    entries, meant = _offsets(M, kind)
    off = torch.tensor(entries, dtype=torch.int32, device="cuda")
    held = torch.zeros(M, dtype=torch.bool)
    if meant:
        held[meant[0]:meant[3]] = True
        good = torch.tensor(meant, dtype=torch.int32, device="cuda")
    else:  # every row that some expert's clamped range holds
        for a, b in zip(entries, entries[1:]):
            held[min(max(a, 0), M):min(max(b, a, 0), M)] = True
    on = held.cuda()
    x, dy = _normal(1, M, H), _normal(2, M, H)
    x[~on], dy[~on] = float("nan"), float("nan")
    xg, dyg = _surrounded(x), _surrounded(dy)
    w1, w2 = _normal(3, E, 2 * I, H, size=H ** -0.5), _normal(4, E, H, I, size=I ** -0.5)

    def call(name, **args):
        lib_call = getattr(lib, name)
        assert lib_call(_pack(F, L.R, name, dict(args, num_rows=M, num_experts=E)), None) == 0, name
        torch.cuda.synchronize()

    def same(got, want, what):
        assert meant is None or torch.equal(got[on], want[on]), what

    def pointers(**tensors):
        return {n: t.data_ptr() for n, t in tensors.items()}

    torch.cuda.synchronize()
    every = torch.ones(M, dtype=torch.bool)
    # the products, along and across, and with zeros in the other rows
    for transposed, a, w, n, k in ((0, xg, w1, 2 * I, H), (1, xg, _normal(5, E, H, I, size=H ** -0.5), I, H)):
        for rest in (0, 1):
            out = Guarded(M, n, BF)
            call("moe_ep_expert_product", **pointers(x=a, w=w, offsets=off), out=out.ptr(), n=n, k=k,
                 transposed=transposed, zero_rest=rest)
            out.check(every if rest else held, "product")
            if meant:
                same(out.t, F.expert_product(x, w, offsets=good, transposed=bool(transposed)), "product")
                assert rest == 0 or not bool(out.t[~on].any())
    # the gated product with what it saves, and the gradient through it
    for save, dtype, block, checkpoint in ((1, torch.float16, 8, "bf16"), (2, torch.uint8, 32, "mxfp8")):
        if I % block:
            continue
        out, pre, scales = Guarded(M, I, BF), Guarded(M, 2 * I, dtype), Guarded(M, 2 * I // block, torch.uint8)
        call("moe_ep_gated_product", **pointers(x=xg, w=w1, offsets=off), out=out.ptr(), pre=pre.ptr(),
             pre_scales=scales.ptr(), inter_size=I, k=H, save=save)
        for g, what in ((out, "gated"), (pre, "pre"), (scales, "pre's scales")):
            g.check(held, what)
        if meant:
            want = F.gated_product(x, w1, offsets=good, checkpoint=checkpoint)
            for g, v in zip((out.bytes, pre.bytes, scales.bytes), want):
                same(g, v.view(torch.uint8), "gated")
        grad, again = Guarded(M, 2 * I, BF), Guarded(M, I, BF)
        call("moe_ep_gated_product_backward", **pointers(grad_out=dyg, w=w2, offsets=off), pre=pre.ptr(),
             pre_scales=scales.ptr(), grad_pre=grad.ptr(), out=again.ptr(), inter_size=I, n=H, save=save)
        grad.check(held, "grad_pre")
        again.check(held, "activation")
        if meant:
            want = F.gated_product_backward(dy, w2, want[1], want[2], offsets=good)
            for g, v in zip((grad.t, again.t), want):
                same(g, v, "gated backward")
                assert bool(g[on].isfinite().all())
    # the weights' gradient: all of it is written, and nothing else
    gw = Guarded(E * H, I, BF)
    a = _surrounded(_normal(6, M, I).masked_fill(~on[:, None], float("nan")))
    call("moe_ep_product_weight_grad", **pointers(grad_out=dyg, x=a, offsets=off), grad_w=gw.ptr(), n=H, k=I)
    gw.check(torch.ones(E * H, dtype=torch.bool), "grad_w")
    if meant:
        assert torch.equal(gw.t.view(E, H, I), F.product_weight_grad(dy, a, offsets=good))
        assert bool(gw.t.isfinite().all())
    # 4-bit weights
    if H % 32 == 0:
        codes = torch.randint(0, 256, (E, 2 * I, H // 2), dtype=torch.uint8, device="cuda")
        sc = torch.full((E, 2 * I, H // 32), 120, dtype=torch.uint8, device="cuda")
        for gated in (0, 1):
            out = Guarded(M, I if gated else 2 * I, BF)
            call("moe_ep_four_bit_product", **pointers(x=xg, w=codes, w_scales=sc, offsets=off), out=out.ptr(), n=2 * I,
                 k=H, gated=gated, out_type=0)
            out.check(held, "4-bit product")
            if meant:
                same(out.t, F.expert_matmul_mxfp4(x, codes, sc.view(torch.float8_e8m0fnu), offsets=good,
                                                  gated=bool(gated)), "4-bit product")


@pytest.mark.parametrize("M,N", [(64, 544), (300, 4128)])
def test_four_bit_rows_outside_stay(L, M, N):
    """The 4-bit product's stages of 16 and 64 rows."""
    F, lib, E, K = L.F, L.m.lib, 30, 192
    rng = np.random.default_rng(M)
    counts = np.bincount(rng.integers(0, E, M - 12), minlength=E)
    o = np.concatenate([[0], np.cumsum(counts)]) + 5
    off = torch.from_numpy(o.astype(np.int32)).cuda()
    held = (torch.arange(M) >= 5) & (torch.arange(M) < int(o[-1]))
    x = _surrounded(_normal(1, M, K).masked_fill(~held.cuda()[:, None], float("nan")))
    codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    sc = torch.full((E, N, K // 32), 120, dtype=torch.uint8, device="cuda")
    w = U.mxfp4_values(codes.cpu(), sc.cpu())
    ref, bound, _ = U.product(x.cpu(), w, o)
    torch.cuda.synchronize()
    for gated in (0, 1):
        out = Guarded(M, N // 2 if gated else N, BF)
        assert lib.moe_ep_four_bit_product(_pack(F, L.R, "moe_ep_four_bit_product", dict(
            x=x.data_ptr(), w=codes.data_ptr(), w_scales=sc.data_ptr(), offsets=off.data_ptr(), out=out.ptr(),
            num_rows=M, num_experts=E, n=N, k=K, gated=gated, out_type=0)), None) == 0
        torch.cuda.synchronize()
        out.check(held, "4-bit product")
        y, b = U.gated(ref, bound) if gated else (ref, bound)
        U.close(out.t[held.cuda()], y[held], U.rounded(b, y)[held], "4-bit product")
