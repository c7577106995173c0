"""The router, the sort, the gated feed-forward block and the unsort together:
with all gradients, between a dispatch and its combine, with 4-bit weights,
captured into graphs, on other streams and from several threads; the largest
tiles, long buffers and refusals."""
import threading

import numpy as np
import pytest
import torch

from tests import ffn_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def M():
    from combine_route_mask_amd import experts, ffn, moe_ep, router
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()

    class Modules:
        X, F, R, m = experts, ffn, router, moe_ep
    return Modules


def _normal(seed, *shape, size=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=BF) * size


def _weights(seed, E, H, I):
    return _normal(seed, E, 2 * I, H, size=H ** -0.5), _normal(seed + 1, E, H, I, size=I ** -0.5)


def _same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8)) for x, y in zip(a, b))


# ----------------------------------------------------------------------------
# the chain
# ----------------------------------------------------------------------------

def _block_reference(x, w1, w2, o):
    """(y, bound) of the block in 64 bits: the activation is rounded to bf16 once."""
    I = w2.shape[2]
    pre, off = U.product(x, w1, o)[:2]
    act, off = U.gated(pre, off)
    off = U.rounded(off, act)
    y, _, held = U.product(act, w2, o)
    spread, _, _ = U.product(off, w2.double().abs(), o)
    mag, _, _ = U.product(act.abs() + off, w2.double().abs(), o)
    return y, U.rounded(spread + I * 2 * U.U32 * mag, y), held


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 64, 32), (37, 8, 3, 96, 64), (260, 16, 4, 128, 96)])
def test_layer_with_gradients(M, T, E, k, H, I, renormalize, checkpoint):
    """The layer by autograd is its parts' results bit for bit, and the output lies within the parts' roundings of the
    64-bit one; an expert without tokens has no gradient, a masked one is not chosen."""
    log(f"layer T{T} E{E} k{k} {renormalize} {checkpoint}")
    X, F, R = M.X, M.F, M.R
    x, (w1, w2), go = _normal(1, T, H), _weights(2, E, H, I), _normal(3, T, H)
    logits = _normal(4, T, E).float() * 2
    logits[:, 1] = float("-inf")
    leaves = [t.clone().requires_grad_() for t in (x, logits, w1, w2)]
    r = R.route_top_k(leaves[1], k, renormalize=renormalize)
    s = X.expert_sort(r.ids[None], leaves[0][None], E)
    y = F.expert_ffn(s.rows, leaves[2], leaves[3], offsets=s.offsets, checkpoint=checkpoint)
    out = X.expert_unsort(s.position, y, r.weights[None])[0]
    got = torch.autograd.grad(out, leaves, go)

    r1 = R.route_top_k(logits, k, renormalize=renormalize)
    s1 = X.expert_sort(r1.ids[None], x[None], E)
    last = int(s1.offsets[-1])
    assert int(s1.counts[1]) == 0 and int(s1.counts.sum()) == last
    rows = torch.where(torch.arange(T * k, device="cuda")[:, None] < last, s1.rows, 0)
    y1, saved = F.expert_ffn_forward(rows, w1, w2, offsets=s1.offsets, checkpoint=checkpoint)
    assert torch.equal(out, X.expert_unsort(s1.position, y1, r1.weights[None])[0])
    gy, gw = X.expert_unsort_backward(s1.position, go[None], y1, r1.weights[None])
    gx, gw1, gw2 = F.expert_ffn_backward(gy, saved, w1, w2, offsets=s1.offsets)
    want = (X.expert_sort_backward(s1.position, gx)[0],
            R.route_top_k_backward(logits, r1.ids, gw[0], renormalize=renormalize), gw1, gw2)
    for g, v, name in zip(got, want, ("x", "logits", "w1", "w2")):
        assert torch.equal(g, v), name
    assert not bool(gw1[1].any() or gw2[1].any() or got[1][:, 1].any())

    o = s1.offsets.cpu().numpy()
    ref, off, _ = _block_reference(rows.cpu(), w1.cpu(), w2.cpu(), o)
    p, w = s1.position[0].cpu().long(), r1.weights.cpu().double()
    total, bound = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        here = (p[:, j] >= 0).nonzero()[:, 0]
        at, wj = p[here, j], w[here, j][:, None]
        total[here] += wj * ref[at]
        bound[here] += wj * off[at] + (k + 1) * 2 * U.U32 * wj * (ref[at].abs() + off[at])
    U.close(out.detach(), total, U.rounded(bound, total), "layer")


@pytest.mark.parametrize("P,T,E,k,H,I,fmt", [(4, 13, 16, 4, 256, 96, "bf16"), (2, 200, 8, 2, 512, 64, "bf16"),
                                             (4, 40, 8, 3, 128, 64, "mxfp8")])
def test_between_dispatch_and_combine(M, P, T, E, k, H, I, fmt):
    """Routed by the router, dispatched (an MXFP8 payload is restored behind the sort), through the block and
    combined: what the same tokens give without an exchange, to the combine's one more rounding."""
    log(f"exchange P{P} T{T} E{E} k{k} {fmt}")
    X, F, R = M.X, M.F, M.R
    x, (w1, w2) = _normal(1, P, T, H), _weights(2, E, H, I)
    r = R.route_top_k(_normal(3, P, T, E), k)
    ex = M.m.MoeEpExchange(P, E, k, T, H, dispatch_format=fmt)
    n = [T - i for i in range(P)]
    if fmt == "mxfp8":
        c = F.checkpoint_rows(x.view(P * T, H))
        recv = ex.dispatch(c.rows.view(P, T, H), r.ids, r.weights, scales=c.scales.view(P, T, H // 32), num_tokens=n)
        x = F.restore_rows(c.rows, c.scales).view(P, T, H)
    else:
        recv = ex.dispatch(x, r.ids, r.weights, num_tokens=n)
    s = ex.expert_sort(recv)
    rows = F.restore_rows(s.rows, s.scales) if fmt == "mxfp8" else s.rows
    y = F.expert_ffn(rows, w1, w2, offsets=s.offsets)
    eo = torch.full((P, P * T, H), float("nan"), dtype=BF, device="cuda")
    X.expert_unsort(s.position, y, recv["weights"], out=eo, keep_empty=True)
    got = ex.combine(eo)
    held = torch.arange(T, device="cuda")[None] < torch.tensor(n, device="cuda")[:, None]
    one = torch.where(held[:, :, None], r.ids, E)
    s1 = X.expert_sort(one.view(1, P * T, k), x.reshape(1, P * T, H), E)
    m = int(s1.offsets[-1])
    assert torch.equal(s.offsets, s1.offsets) and torch.equal(rows[:m], s1.rows[:m])
    y1 = F.expert_ffn(s1.rows, w1, w2, offsets=s1.offsets)
    assert torch.equal(y[:m], y1[:m])
    p, w = s1.position.view(P * T, k).cpu().long(), r.weights.view(P * T, k).cpu().double()
    ref = torch.zeros(P * T, H, dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for j in range(k):
        here = (p[:, j] >= 0).nonzero()[:, 0]
        t = y1.cpu().double()[p[here, j]] * w[here, j][:, None]
        ref[here] += t
        mag[here] += t.abs()
    sel = held.view(-1).cpu()
    # each rank's sum rounds to bf16 once, their sum once more
    U.close(got.view(P * T, H)[sel.cuda()], ref[sel], ((2 * U.UBF + (k + P + 2) * U.U32) * mag * 1.01)[sel], "combined")
    ex.destroy()


def test_four_bit_layer(M):
    """Two 4-bit products, the first one gated, make the block of the dequantised weights."""
    X, F = M.X, M.F
    E, T, k, H, I = 8, 5, 2, 256, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    make = lambda N, K: (torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8),  # noqa: E731
                         torch.randint(120, 125, (E, N, K // 32), generator=g, device="cuda",
                                       dtype=torch.uint8).view(torch.float8_e8m0fnu))
    (c1, s1), (c2, s2) = make(2 * I, H), make(H, I)
    ids = torch.randint(0, E, (1, T, k), generator=g, device="cuda", dtype=torch.int32)
    s = X.expert_sort(ids, _normal(2, 1, T, H), E)
    a = F.expert_matmul_mxfp4(s.rows, c1, s1, offsets=s.offsets, gated=True)
    y = F.expert_matmul_mxfp4(a, c2, s2, offsets=s.offsets, dtype=torch.float32)
    w1, w2 = (U.mxfp4_values(c.cpu(), sc.cpu()).bfloat16() for c, sc in ((c1, s1), (c2, s2)))
    assert torch.equal(w1.double(), U.mxfp4_values(c1.cpu(), s1.cpu()))  # bf16 holds them
    o = s.offsets.cpu().numpy()
    pre, off, held = U.product(s.rows.cpu(), w1, o)
    act, off = U.gated(pre, off)
    U.close(a, act, U.rounded(off, act), "gated")
    ref, bound, _ = U.product(a.cpu(), w2, o)
    U.close(y, ref, U.rounded(bound, ref, torch.float32), "4-bit")
    out = X.expert_unsort(s.position, y)
    assert out.shape == (1, T, H) and bool(out.isfinite().all())


# ----------------------------------------------------------------------------
# graphs, streams, threads
# ----------------------------------------------------------------------------

def _state(seed, T=70, E=6, k=3, H=128, I=96):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 100)
    codes = torch.randint(0, 256, (E, 2 * I, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 126, (E, 2 * I, H // 32), generator=g, device="cuda", dtype=torch.uint8)
    return {"x": _normal(seed, T, H), "logits": _normal(seed + 1, T, E).float(), "go": _normal(seed + 2, T, H),
            "w1": _weights(seed + 3, E, H, I)[0], "w2": _weights(seed + 3, E, H, I)[1], "codes": codes, "scales": scales}


def _layer(M, st, stream=None, k=3):
    """Every operator once, on the given stream; all its results."""
    X, F, R, kw = M.X, M.F, M.R, {"stream": stream}
    E = st["logits"].shape[1]
    r = R.route_top_k(st["logits"], k, **kw)
    s = X.expert_sort(r.ids[None], st["x"][None], E, **kw)
    results = [r.ids, r.weights, s.position]
    for checkpoint in ("bf16", "mxfp8"):
        y, saved = F.expert_ffn_forward(s.rows, st["w1"], st["w2"], offsets=s.offsets, checkpoint=checkpoint, **kw)
        out = X.expert_unsort(s.position, y, r.weights[None], **kw)
        gy, gw = X.expert_unsort_backward(s.position, st["go"][None], y, r.weights[None], **kw)
        gx, gw1, gw2 = F.expert_ffn_backward(gy, saved, st["w1"], st["w2"], offsets=s.offsets, **kw)
        gl = R.route_top_k_backward(st["logits"], r.ids, gw[0], **kw)
        results += [out, gx, gw1, gw2, gl]
    results.append(F.expert_matmul_mxfp4(s.rows, st["codes"], st["scales"].view(torch.float8_e8m0fnu), offsets=s.offsets,
                                         gated=True, **kw))
    results.append(F.expert_ffn(s.rows, st["w1"], st["w2"], offsets=s.offsets, **kw))
    return results


@pytest.mark.parametrize("T", [1, 70, 900])
def test_layer_replays_from_captured_graphs(M, T):
    """Two graphs of the whole layer, forward and backward, replayed in turn with new inputs in place and eager work
    between."""
    log(f"graphs T{T}")
    fresh = [_state(10 * i, T=T) for i in range(6)]
    eager = [_layer(M, st) for st in fresh]
    held = [{n: v.clone() for n, v in fresh[i].items()} for i in range(2)]
    graphs, outs = [], []
    for st in held:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(M, st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_layer(M, st))
        graphs.append(g)
    for turn in range(3):
        for i in range(2):
            for n, v in held[i].items():
                v.copy_(fresh[2 * turn + i][n])
        for g in graphs:
            g.replay()
        other = _layer(M, fresh[5 - turn])
        torch.cuda.synchronize()
        assert _same(other, eager[5 - turn]), f"eager call {turn}"
        for i in range(2):
            assert _same(outs[i], eager[2 * turn + i]), f"graph {i}, replay {turn}"
    del graphs


def test_layer_on_other_streams(M):
    sts = [_state(seed, T=300) for seed in (1, 20, 40)]
    want = [_layer(M, st) for st in sts]
    torch.cuda.synchronize()
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    for _ in range(3):
        got = [_layer(M, sts[0], stream=a), _layer(M, sts[1], stream=b.cuda_stream)]
        with torch.cuda.stream(c):
            got.append(_layer(M, sts[2]))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert _same(g, w)


def test_calls_from_several_threads(M):
    sts = [_state(7 * i, T=20 + 60 * i) for i in range(4)]
    want = [_layer(M, st) for st in sts]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            for _ in range(10):
                if not _same(_layer(M, sts[i]), want[i]):
                    wrong.append(i)
                try:
                    M.R.route_top_k(sts[i]["logits"], 65 + i)
                except M.m.MoeEpArgError as e:
                    if str(65 + i) not in str(e):
                        wrong.append(str(e))
        except Exception as e:  # a thread's failure is the test's
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_gradients_at_any_address(M):
    """Gradients that autograd hands over expanded, or from between 16 bytes."""
    F = M.F
    x, (w1, w2) = _normal(1, 20, 64), _weights(2, 1, 64, 32)
    off = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    y, saved = F.expert_ffn_forward(x, w1, w2, offsets=off)
    want = F.expert_ffn_backward(torch.ones_like(y), saved, w1, w2, offsets=off)
    for loss in (lambda y: y.sum(), lambda y: (torch.cat([y.new_ones(3), y.view(-1)])[3:]).sum()):
        leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
        assert _same(torch.autograd.grad(loss(F.expert_ffn(*leaves, offsets=off)), leaves), want)
    # a frozen weight gets none, and the others' stay
    leaves = [x.clone().requires_grad_(), w1, w2.clone().requires_grad_()]
    got = torch.autograd.grad(F.expert_ffn(*leaves, offsets=off).sum(), (leaves[0], leaves[2]))
    assert _same(got, (want[0], want[2]))
    # what was saved and then written is not used in silence
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    moved = leaves[0] * 1
    y = F.expert_ffn(moved, leaves[1], leaves[2], offsets=off)
    moved.detach().zero_()
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


# ----------------------------------------------------------------------------
# sizes
# ----------------------------------------------------------------------------

# rows an expert, first width, second width: those that take the largest tiles, of each height
LARGE = [((1000, 0, 1100, 900), 4096, 1024), ((320, 640, 70, 200, 330, 257, 513, 1), 4096, 1536), ((2048,), 4112, 1032),
         ((600,) * 6, 2064, 776)]


@pytest.mark.parametrize("counts,N,K", LARGE)
def test_large_tiles(M, counts, N, K):
    log(f"large tiles {counts} {N}x{K}")
    F = M.F
    rows = sum(counts) + 5
    o = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    off, E = torch.from_numpy(o).cuda(), len(counts)
    x, dy, w = _normal(1, rows, K), _normal(2, rows, N), _normal(3, E, N, K, size=K ** -0.5)
    held = torch.arange(rows) < int(o[-1])
    for transposed in (False, True):
        a, b = (dy, w) if transposed else (x, w)
        ref, bound, _ = _product_gpu(a, b, o, transposed)
        got = F.expert_product(a, b, offsets=off, transposed=transposed)
        U.close(got[held.cuda()], ref[held], U.rounded(bound, ref)[held], "product")
    pre, poff, _ = _product_gpu(x, w, o, False)
    ref, bound = U.gated(pre, poff)
    for checkpoint in ("bf16", "mxfp8") if N % 64 == 0 else ("bf16",):
        got, kept, scales = F.gated_product(x, w, offsets=off, checkpoint=checkpoint)
        U.close(got[held.cuda()], ref[held], U.rounded(bound, ref)[held], "gated")
        if checkpoint == "bf16":
            U.close(U.half_values(kept, scales)[held], pre[held], U.half_step(pre[held], poff[held]), "pre")
        else:
            v = U.mx_values(kept, scales)
            exponent = scales.cpu().view(torch.uint8).double() - 127
            step = torch.maximum(2.0 ** -4 * pre.abs(),
                                 torch.exp2(exponent - 10).repeat_interleave(32, dim=1))
            U.close(v[held], pre[held], (step + poff * (1 + 2.0 ** -4))[held], "MXFP8 pre")
        # through the second product's weights [E, K, I] and the activation
        I = N // 2
        w2, go = _normal(5, E, K, I, size=I ** -0.5), _normal(6, rows, K)
        d, doff, _ = _product_gpu(go, w2, o, True)
        values = (U.half_values if checkpoint == "bf16" else U.mx_values)(kept, scales)
        gref, gbound, act, abound = U.gated_backward(d, doff, values)
        gp, again = F.gated_product_backward(go, w2, kept, scales, offsets=off)
        U.close(gp[held.cuda()], gref[held], U.rounded(gbound, gref)[held], "grad_pre")
        U.close(again[held.cuda()], act[held], U.rounded(abound, act)[held], "activation")
    dd, xd = dy.double(), x.double()
    got = F.product_weight_grad(dy, x, offsets=off)
    for e in range(E):
        a, b = int(o[e]), int(o[e + 1])
        ref = dd[a:b].t() @ xd[a:b]
        mag = dd[a:b].abs().t() @ xd[a:b].abs()
        U.close(got[e], ref.cpu(), U.rounded((b - a) * 2 * U.U32 * mag, ref).cpu(), "grad_w")


def _product_gpu(x, w, o, transposed):
    """U.product's, computed on the GPU in float64 (torch's products)."""
    M_, K = x.shape
    N = w.shape[2] if transposed else w.shape[1]
    y, mag = (torch.zeros(M_, N, dtype=torch.float64, device="cuda") for _ in range(2))
    held = torch.zeros(M_, dtype=torch.bool)
    for e, a, b in U.by_expert(o, M_):
        v = w[e].double() if transposed else w[e].double().t().contiguous()
        y[a:b], mag[a:b] = x[a:b].double() @ v, x[a:b].double().abs() @ v.abs()
        held[a:b] = True
    return y.cpu(), (K * 2 * U.U32 * mag).cpu(), held


def test_offsets_past_32_bits(M):
    """More than 2^32 bytes of rows, weights, logits and gradients: the last ones are right."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free device memory")
    F, R = M.F, M.R
    rows, K, N = 70007, 32768, 64
    x, w = _normal(1, rows, K), _normal(2, N, K, size=K ** -0.5)
    y = F.expert_product(x, w)
    ref, bound, _ = _product_gpu(x[-40:], w[None], np.array([0, 40]), False)
    U.close(y[-40:], ref, U.rounded(bound, ref), "last rows")
    # as the transposed product's output, and as the gradients' rows
    z = F.expert_product(y, w, transposed=True)
    ref, bound, _ = _product_gpu(y[-40:], w[None], np.array([0, 40]), True)
    U.close(z[-40:], ref, U.rounded(bound, ref), "last rows, transposed")
    off = torch.tensor([0, rows - 30, rows], dtype=torch.int32, device="cuda")
    g = F.product_weight_grad(y, x, offsets=off)
    ref = y[-30:].double().t() @ x[-30:].double()
    mag = y[-30:].double().abs().t() @ x[-30:].double().abs()
    U.close(g[1], ref.cpu(), U.rounded(30 * 2 * U.U32 * mag, ref).cpu(), "last expert's gradient")
    c = F.checkpoint_rows(x)
    few = F.checkpoint_rows(x[-40:].contiguous())
    assert _same((c.rows[-40:], c.scales[-40:]), few)
    assert torch.equal(F.restore_rows(c.rows, c.scales)[-40:], F.restore_rows(*few))
    del x, z, c, y, g
    E = 130
    w = _normal(3, E, 4096, 4096, size=2.0 ** -6)
    x = _normal(4, 12, 4096)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = 12
    got = F.expert_product(x, w, offsets=off)
    ref, bound, _ = _product_gpu(x, w[-1:], np.array([0, 12]), False)
    U.close(got, ref, U.rounded(bound, ref), "last expert")
    del w
    codes = torch.randint(0, 256, (E, 8192, 4160), dtype=torch.uint8, device="cuda")
    scales = torch.randint(110, 120, (E, 8192, 260), dtype=torch.uint8, device="cuda")
    x = _normal(5, 12, 8320)
    for gated in (False, True):
        got = F.expert_matmul_mxfp4(x, codes, scales.view(torch.float8_e8m0fnu), offsets=off, gated=gated, dtype=torch.float32)
        ref, bound, _ = U.product(x.cpu(), U.mxfp4_values(codes[-1].cpu(), scales[-1].cpu().view(torch.float8_e8m0fnu)), [0, 12])
        if gated:
            ref, bound = U.gated(ref, bound)
        U.close(got, ref, U.rounded(bound, ref, torch.float32), "last expert's 4-bit weights")
    del codes, scales
    T = 1100003
    logits = torch.randn((T, 1024), device="cuda")
    assert logits.numel() * 4 > 1 << 32
    r = R.route_top_k(logits, 3, renormalize=False)
    few = R.route_top_k(logits[-50:].contiguous(), 3, renormalize=False)
    assert _same((r.ids[-50:], r.weights[-50:]), few)
    gw = torch.randn((T, 3), device="cuda")
    d = R.route_top_k_backward(logits, r.ids, gw, renormalize=False)
    assert torch.equal(d[-50:], R.route_top_k_backward(logits[-50:].contiguous(), few.ids, gw[-50:].contiguous(), renormalize=False))


def test_offsets_out_of_range(M):
    """Entries below 0 and past the rows are taken as the ends: nothing else is read or written."""
    F = M.F
    x, w = _normal(1, 40, 64), _normal(2, 3, 32, 64)
    dy = _normal(3, 40, 32)
    bad = torch.tensor([-7, 10, 30, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 10, 30, 40], dtype=torch.int32, device="cuda")
    assert torch.equal(F.expert_product(x, w, offsets=bad), F.expert_product(x, w, offsets=good))
    assert torch.equal(F.product_weight_grad(dy, x, offsets=bad), F.product_weight_grad(dy, x, offsets=good))
    codes = torch.randint(0, 256, (3, 32, 32), dtype=torch.uint8, device="cuda")
    scales = torch.full((3, 32, 2), 120, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    assert torch.equal(F.expert_matmul_mxfp4(x, codes, scales, offsets=bad), F.expert_matmul_mxfp4(x, codes, scales, offsets=good))


def test_rows_outside_the_experts(M):
    """Under autograd rows before the first and behind the last expert's are zeros, in the result and the gradient."""
    F = M.F
    x, (w1, w2) = _normal(1, 50, 64), _weights(2, 2, 64, 32)
    off = torch.tensor([7, 20, 41], dtype=torch.int32, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    y = F.expert_ffn(*leaves, offsets=off)
    gx, = torch.autograd.grad(y.sum(), leaves[:1])
    for t in (y.detach(), gx):
        assert not bool(t[:7].any() or t[41:].any()) and bool(t[7:41].any(dim=1).all())
    # rows that lie in a larger buffer are kept as they were in the forward pass
    space = torch.cat([x, x])
    part = space[:50].requires_grad_()
    y = F.expert_ffn(part, leaves[1], leaves[2], offsets=off)
    space.data.fill_(7.0)  # as a kernel writes: unseen by autograd
    want = F.expert_ffn(x.clone().requires_grad_(), leaves[1], leaves[2], offsets=off)
    assert _same(torch.autograd.grad(y.sum(), leaves[1:]), torch.autograd.grad(want.sum(), leaves[1:]))


def test_empty_calls(M):
    F, R = M.F, M.R
    (w1, w2), off = _weights(1, 2, 64, 32), torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    assert F.expert_ffn(x, w1, w2, offsets=off).shape == (0, 64)
    leaves = [t.clone().requires_grad_() for t in (x, w1, w2)]
    y = F.expert_ffn(*leaves, offsets=off, checkpoint="mxfp8")
    for g, t in zip(torch.autograd.grad(y, leaves, torch.empty_like(y)), leaves):
        assert g.shape == t.shape and not bool(g.any())
    assert F.checkpoint_rows(x).rows.shape == (0, 64)
    r = R.route_top_k(torch.empty((0, 8), device="cuda"), 2)
    assert r.ids.shape == (0, 2)
    assert R.route_top_k_backward(torch.empty((0, 8), device="cuda"), r.ids, r.weights).shape == (0, 8)


def test_binding_refusals(M):
    F, R, refused = M.F, M.R, M.m.MoeEpArgError
    x, (w1, w2) = _normal(1, 6, 64), _weights(2, 2, 64, 32)
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    codes = torch.zeros((2, 8, 32), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((2, 8, 2), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
    y, saved = F.expert_ffn_forward(x, w1, w2, offsets=off)
    for call in (lambda: F.expert_ffn(x, w1, w2), lambda: F.expert_ffn(x, w1[0], w2[0], offsets=off),
                 lambda: F.expert_ffn(x.float(), w1, w2, offsets=off), lambda: F.expert_ffn(x, w1, w2[:1], offsets=off),
                 lambda: F.expert_ffn(x, w2, w1, offsets=off), lambda: F.expert_ffn(x, w1, w2, offsets=off.long()),
                 lambda: F.expert_ffn(x, w1, w2, offsets=off[:2]), lambda: F.expert_ffn(x.t(), w1, w2, offsets=off),
                 lambda: F.expert_ffn(x, w1, w2, offsets=off, checkpoint="int8"),
                 lambda: F.expert_ffn(x, w1, w2, offsets=off, out=torch.empty((6, 32), dtype=BF, device="cuda")),
                 lambda: F.expert_ffn_forward(x, w1[:, :48].contiguous(), w2[:, :, :24].contiguous(), offsets=off,
                                              checkpoint="mxfp8"),
                 lambda: F.expert_product(x[:, :60].contiguous(), w1[:, :, :60].contiguous(), offsets=off),
                 lambda: F.expert_product(x.view(-1)[8:8 + 4 * 64].view(4, 64)[:, :32], w1, offsets=off),
                 lambda: F.expert_product(x.view(-1)[4:4 + 4 * 64].view(4, 64), w1, offsets=off),
                 lambda: F.gated_product(x, w1[:, :31].contiguous(), offsets=off),
                 lambda: F.gated_product_backward(x, w2, saved.pre[:5], saved.pre_scales, offsets=off),
                 lambda: F.gated_product_backward(x, w2, saved.pre.to(BF), saved.pre_scales, offsets=off),
                 lambda: F.gated_product_backward(x, w2, saved.pre, scales, offsets=off),
                 lambda: F.product_weight_grad(x, y[:5], offsets=off), lambda: F.product_weight_grad(x, y, offsets=off[:1]),
                 lambda: F.expert_ffn_backward(y, saved._replace(x=x[:, :32].contiguous()), w1, w2, offsets=off),
                 lambda: F.checkpoint_rows(x[:, :48].contiguous()), lambda: F.checkpoint_rows(x.half()),
                 lambda: F.restore_rows(codes[0], scales[0]),
                 lambda: F.expert_matmul_mxfp4(x, codes[:, :, :16].contiguous(), scales, offsets=off),
                 lambda: F.expert_matmul_mxfp4(x, codes, scales[:, :, :1].contiguous(), offsets=off),
                 lambda: F.expert_matmul_mxfp4(x, codes[:, :7].contiguous(), scales[:, :7].contiguous(), offsets=off, gated=True),
                 lambda: F.expert_matmul_mxfp4(x, codes, scales, offsets=off, dtype=torch.float16),
                 lambda: R.route_top_k(x, 65), lambda: R.route_top_k(x, 0), lambda: R.route_top_k(x.half(), 2),
                 lambda: R.route_top_k(x.t(), 2), lambda: R.route_top_k(x, 2, scale=float("nan")),
                 lambda: R.route_top_k(x, 2, ids=torch.empty((6, 3), dtype=torch.int32, device="cuda")),
                 lambda: R.route_top_k_backward(x, off[:2].view(1, 2), torch.zeros((1, 2), device="cuda"))):
        with pytest.raises(refused):
            call()
