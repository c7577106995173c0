"""The expert layer as it is used: between a dispatch and its combine, into
the next layer's payload; captured into HIP graphs; on other streams; and
with buffers past 32-bit offsets."""
import numpy as np
import pytest
import torch

import workloads as W
from tests import expert_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def X():
    from combine_route_mask_amd import experts, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    yield experts
    torch.cuda.empty_cache()


def _codes(rng, *shape):
    return torch.from_numpy(rng.integers(-127, 128, size=shape, dtype=np.int8)).cuda()


def _scales(rng, *shape):
    return torch.from_numpy(rng.uniform(0.5, 1.5, size=shape).astype(np.float32)).cuda() / 2000


def _weights(rng, E, H, I):
    return _codes(rng, E, 2 * I, H), _scales(rng, E, 2 * I), _codes(rng, E, H, I), _scales(rng, E, H)


def _experts(X, s, w, out=None):
    """Both products and the activation of sorted int8 rows."""
    h = X.expert_matmul(s.rows, s.scales, w[0], w[1], offsets=s.offsets)
    a = X.silu_mul_quantize(h, offsets=s.offsets)
    return X.expert_matmul(a.rows, a.scales, w[2], w[3], offsets=s.offsets, out=out), h, a


@pytest.mark.parametrize("P,T,E,k,H,I,mask", [(4, 13, 16, 4, 256, 96, None), (8, 40, 32, 3, 512, 64, 0b10111011),
                                              (2, 300, 8, 2, 1024, 272, None), (1, 9, 4, 4, 7168, 48, None)])
def test_layer_between_dispatch_and_combine(X, P, T, E, k, H, I, mask):
    from combine_route_mask_amd.moe_ep import MoeEpExchange
    log(f"layer P{P} T{T} E{E} k{k} H{H} I{I} mask {mask}")
    rng = np.random.default_rng(P + T)
    w = W.Workload("layer", P=P, T=T, H=H, E=E, k=k, n_lo=max(1, T // 2), n_hi=T, seed=P)
    R = W.draw_routing(w, 7)
    ids, wts = torch.from_numpy(R.ids).cuda(), torch.from_numpy(R.weights).cuda()
    ids[0, 0, 0] = E + 3  # an id of no expert
    x = torch.randn((P, T, H), device="cuda", dtype=BF)
    weights = _weights(rng, E, H, I)
    ex = MoeEpExchange(P, E, k, T, H)
    recv = ex.dispatch(x, ids, wts, num_tokens=R.counts.tolist(), active_rank_mask=mask)
    s = ex.expert_sort(recv, quantize=True)
    live = [r for r in range(P) if mask is None or mask >> r & 1]
    assert s.rows.shape[0] == k * sum(int(R.counts[r]) for r in live) == ex.most_pairs
    y, h, a = _experts(X, s, weights)
    eo = torch.full((P, P * T, H), float("nan"), dtype=BF, device="cuda")
    X.expert_unsort(s.position, y, recv["weights"], out=eo, keep_empty=True)
    got = ex.combine(eo)

    # the same tokens with every expert on one rank, without an exchange
    held = torch.zeros((P, T), dtype=torch.bool, device="cuda")
    for r in live:
        held[r, :int(R.counts[r])] = True
    one = torch.where(held[:, :, None], ids, E)
    for r in range(P):
        if r not in live:  # nothing bound for a masked-off rank arrives
            one = torch.where((one >= r * (E // P)) & (one < (r + 1) * (E // P)), E, one)
    s1 = X.expert_sort(one.view(1, P * T, k), x.view(1, P * T, H), E, quantize=True)
    m = int(s1.offsets[-1])
    if mask is None:
        # the live ranks' regions of an unmasked step hold the same pairs in the same order
        assert torch.equal(s.counts, s1.counts) and torch.equal(s.offsets, s1.offsets)
        assert torch.equal(s.rows[:m], s1.rows[:m]) and torch.equal(s.scales[:m], s1.scales[:m])
    y1, _, _ = _experts(X, s1, weights)
    if mask is None:
        assert np.array_equal(U.bits(y[:m]), U.bits(y1[:m])), "expert outputs"
    # each rank's sum rounds to bf16 once, their sum once more
    ref, mag = U.unsort_reference(s1.position.cpu(), torch.where(torch.arange(len(y1), device="cuda")[:, None] < m, y1, 0),
                                  wts.view(1, P * T, k))
    bound = (2 * U.UBF + (k + P + 2) * U.U32) * mag * 1.01
    sel = held.view(1, -1).cpu()
    U.check_close(got.view(1, P * T, H)[sel.cuda()], ref[sel], bound[sel], "combined layer")

    # stage by stage from what the stage before gave
    hd = h[:m].double().cpu()
    g, u = hd.chunk(2, 1)
    act = g / (1 + torch.exp(-g)) * u
    U.check_int8(a.rows[:m], a.scales[:m], act, (float(g.abs().max()) * 2 + 10) * U.U32, "activation")

    # the next layer's MXFP8 payload from the combined rows
    norm_w = torch.ones(H, dtype=BF, device="cuda")
    n = X.add_rms_norm(got.view(P * T, H), x.view(P * T, H), norm_w, format="mxfp8")
    ex8 = MoeEpExchange(P, E, k, T, H, dispatch_format="mxfp8")
    recv8 = ex8.dispatch(n.rows.view(P, T, H), ids, wts, scales=n.scales.view(P, T, H // 32),
                         num_tokens=R.counts.tolist())
    s8 = ex8.expert_sort(recv8)
    r, q, j = (s8.position >= 0).nonzero(as_tuple=True)
    at = s8.position[r, q, j].long()
    assert torch.equal(s8.rows[at], n.rows.view(torch.uint8).view(P * T, H)[q])
    assert torch.equal(s8.scales[at], n.scales.view(torch.uint8).view(P * T, H // 32)[q])
    with pytest.raises(ValueError):
        ex8.expert_sort(recv8, quantize=True)
    ex.destroy()
    ex8.destroy()


@pytest.mark.parametrize("P,T,E,k", [(4, 9, 16, 4), (4, 130, 16, 4), (8, 700, 32, 2), (4, 2200, 16, 4), (64, 5, 64, 2)])
def test_masked_ranks_hold_no_pairs(X, P, T, E, k):
    """A dispatch leaves a masked-off rank's region as the step before left
    it (at first: whatever the workspace held): its ids are no pairs, at every
    size class of the sort, and take no place from the live ranks' ones."""
    from combine_route_mask_amd.moe_ep import MoeEpArgError, MoeEpExchange
    H = 64
    log(f"masked ranks P{P} T{T} E{E} k{k}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    ids = torch.rand((P, T, E), generator=g, device="cuda").argsort(2)[:, :, :k].to(torch.int32)
    wts = torch.rand((P, T, k), generator=g, device="cuda")
    x = torch.randn((P, T, H), generator=g, device="cuda", dtype=BF)
    ex = MoeEpExchange(P, E, k, T, H)
    ex.workspace.zero_()  # zeros: ids of expert 0, on rank 0
    for mask in (0b0110, None, 0b1101 | (0xF0 if P == 8 else 0)):
        recv = ex.dispatch(x, ids, wts, num_tokens=[T] * P, active_rank_mask=mask)
        live = [r for r in range(P) if mask is None or mask >> r & 1]
        want = recv["ids"].clone()
        for r in range(P):
            if r not in live:
                want[r] = E
        for quantize in (False, True):
            s = ex.expert_sort(recv, quantize=quantize)
            ref = X.expert_sort(want, recv["payload"].view(BF).contiguous(), E // P, capacity=ex.most_pairs,
                                quantize=quantize)
            m = int(ref.offsets[-1])
            assert torch.equal(s.counts, ref.counts) and torch.equal(s.offsets, ref.offsets), mask
            assert torch.equal(s.position, ref.position) and torch.equal(s.rows[:m], ref.rows[:m]), mask
            if mask is None:
                assert m == P * T * k
    with pytest.raises(MoeEpArgError):
        X.expert_sort(want, x.view(P, T, H).repeat(1, P, 1), E // P, active_rank_mask=1 << P)
    ex.destroy()
    odd = MoeEpExchange(P, E, k, T, H, invalid_expert_id=0)
    recv = odd.dispatch(x, ids, wts, num_tokens=[T] * P)
    with pytest.raises(MoeEpArgError):  # empty slots would be pairs
        odd.expert_sort(recv)
    odd.destroy()


def _state(rng, seed, R=2, S=70, k=3, epr=4, H=256, I=96):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = torch.from_numpy(U.draw_ids(np.random.default_rng(seed), R, S, k, epr)).cuda()
    return {"ids": ids, "rows": torch.randn((R, S, H), generator=g, device="cuda", dtype=BF),
            "w": torch.rand((R, S, k), generator=g, device="cuda"),
            "x": torch.randn((33, H), generator=g, device="cuda", dtype=BF)}


def _layer(X, st, weights, stream=None):
    """Every operator once, on the given stream; all its results."""
    s = X.expert_sort(st["ids"], st["rows"], 4, quantize=True, stream=stream)
    c = X.expert_sort(st["ids"], st["rows"], 4, stream=stream)
    h = X.expert_matmul(s.rows, s.scales, weights[0], weights[1], offsets=s.offsets, stream=stream)
    a = X.silu_mul_quantize(h, offsets=s.offsets, stream=stream)
    y = X.expert_matmul(a.rows, a.scales, weights[2], weights[3], offsets=s.offsets, stream=stream)
    out = X.expert_unsort(s.position, y, st["w"], stream=stream)
    gr, gw = X.expert_unsort_backward(s.position, st["rows"], y, st["w"], stream=stream)
    gx = X.expert_sort_backward(s.position, gr, stream=stream)
    n = X.add_rms_norm(st["x"], st["x"], weights[4], format="deepseek_fp8", stream=stream)
    z = X.add_rms_norm(st["x"], None, weights[4], format="int8", stream=stream)
    d = X.expert_matmul(z.rows, z.scales, weights[0][0], weights[1][0], stream=stream)
    return [s.position, s.offsets, s.counts, c.position, out, gw, gx, n.rows, n.scales, n.residual, z.rows, z.scales, d]


def _same(a, b):
    return all(np.array_equal(U.bits(x), U.bits(y)) for x, y in zip(a, b))


@pytest.mark.parametrize("S", [70, 700, 3000])
def test_layer_replays_from_captured_graphs(X, S):
    """Two graphs of the whole layer, captured and replayed in turn with new
    inputs in place and eager work between: each replay is the eager result
    (the graphs' workspaces are their own)."""
    log(f"layer graphs S{S}")
    rng = np.random.default_rng(3)
    weights = _weights(rng, 8, 256, 96) + (torch.ones(256, dtype=BF, device="cuda"),)
    fresh = [_state(rng, seed, S=S) for seed in range(6)]
    eager = [_layer(X, st, weights) for st in fresh]
    held = [{k: v.clone() for k, v in fresh[i].items()} for i in range(2)]
    graphs, outs = [], []
    for st in held:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(X, st, weights)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_layer(X, st, weights))
        graphs.append(g)
    for turn in range(3):
        for i in range(2):
            for k, v in held[i].items():
                v.copy_(fresh[2 * turn + i][k])
        for g in graphs:
            g.replay()
        other = _layer(X, fresh[5 - turn], weights)
        torch.cuda.synchronize()
        assert _same(other, eager[5 - turn]), f"eager call {turn}"
        for i in range(2):
            assert _same(outs[i], eager[2 * turn + i]), f"graph {i}, replay {turn}"
    del graphs


def test_layer_on_other_streams(X):
    """The stream argument (an object or a raw handle), two streams at a time
    with buffers of their own, and the current stream of a with-block."""
    rng = np.random.default_rng(4)
    weights = _weights(rng, 8, 256, 96) + (torch.ones(256, dtype=BF, device="cuda"),)
    sts = [_state(rng, seed, S=600) for seed in (1, 2, 3)]
    want = [_layer(X, st, weights) for st in sts]
    torch.cuda.synchronize()
    a, b, c = (torch.cuda.Stream() for _ in range(3))
    for _ in range(3):
        got = [_layer(X, sts[0], weights, stream=a), _layer(X, sts[1], weights, stream=b.cuda_stream)]
        with torch.cuda.stream(c):
            got.append(_layer(X, sts[2], weights))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert _same(g, w)


def test_calls_from_several_threads(X):
    """Threads that launch on the same stream at the same time: a call's
    workspace is its own until its launches are out, and messages are a
    thread's own."""
    import threading
    from combine_route_mask_amd.moe_ep import MoeEpArgError
    sizes = [(1, 3000, 4, 40), (4, 500, 3, 8), (1, 2900, 3, 70), (2, 40, 8, 16)]
    states = []
    for i, (R, S, k, epr) in enumerate(sizes):
        ids = U.draw_ids(np.random.default_rng(i), R, S, k, epr)
        rows = torch.randn((R, S, 64), device="cuda", dtype=BF)
        states.append((torch.from_numpy(ids).cuda(), rows, epr, X.expert_sort(torch.from_numpy(ids).cuda(), rows, epr)))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        ids, rows, epr, want = states[i]
        try:
            for _ in range(40):
                got = X.expert_sort(ids, rows, epr)
                m = int(got.offsets[-1])
                if not (torch.equal(got.position, want.position) and torch.equal(got.rows[:m], want.rows[:m])
                        and torch.equal(got.offsets, want.offsets) and torch.equal(got.counts, want.counts)):
                    wrong.append(sizes[i])
                try:
                    X.expert_sort(ids, rows, 4097 + i)
                except MoeEpArgError as e:
                    if str(4097 + i) not in str(e):
                        wrong.append(str(e))
        except Exception as e:  # a thread's failure is the test's
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


def test_an_earlier_error_is_not_this_calls(X):
    """An error that a runtime call of this thread left behind (a device that does not exist) fails no launch."""
    import ctypes
    import re
    path = re.search(r"\S*libamdhip64\S*", open("/proc/self/maps").read()).group(0)
    hip = ctypes.CDLL(path)
    st = _state(None, 5, S=700)
    want = X.expert_sort(st["ids"], st["rows"], 4)
    torch.cuda.synchronize()
    assert hip.hipSetDevice(1 << 20) != 0
    got = X.expert_sort(st["ids"], st["rows"], 4)
    assert torch.equal(got.position, want.position)


def test_gradients_on_a_captured_stream(X):
    """Autograd through the sort and the unsort while a captured graph of the
    same operators' gradients, made of their functional forms, is replayed."""
    st = _state(None, 9, S=200)
    ids, w = st["ids"], st["w"]
    x = st["rows"].clone()
    go = torch.randn_like(x)

    def functional():
        s = X.expert_sort(ids, x, 4)
        gr, gw = X.expert_unsort_backward(s.position, go, s.rows, w)
        return X.expert_sort_backward(s.position, gr), gw

    def by_autograd():
        xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
        s = X.expert_sort(ids, xl, 4)
        y = X.expert_unsort(s.position, s.rows, wl)
        return torch.autograd.grad(y, (xl, wl), go)

    want = functional()
    auto = by_autograd()
    assert _same(want, auto)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = functional()
    for i in range(3):
        x.mul_(-1)
        go.mul_(0.5)
        eager = by_autograd()
        g.replay()
        torch.cuda.synchronize()
        assert _same(got, eager), f"replay {i}"
    del g


def test_saved_tensors_are_the_forward_ones(X):
    """Weights in a workspace that the next step overwrites keep the values
    of their forward in its gradient; a buffer that an operator writes in place
    is no longer the one that autograd saved, and backward says so."""
    st = _state(None, 11, S=40)
    ids, x, w = st["ids"], st["rows"], st["w"]
    space = torch.zeros((2, 4096), device="cuda")
    plane = space[:, :40 * 3].view(2, 40, 3)
    plane.copy_(w)
    go = torch.randn_like(x)
    for own_grad in (False, True):
        xl = x.clone().requires_grad_()
        wl = plane.detach().requires_grad_(own_grad)
        s = X.expert_sort(ids, xl, 4)
        y = X.expert_unsort(s.position, s.rows, wl)
        kept = space.clone()
        space.data.fill_(7.0)  # as a kernel writes: unseen by autograd
        got = torch.autograd.grad(y, (xl, wl) if own_grad else (xl,), go)
        space.data.copy_(kept)
        gr, gw = X.expert_unsort_backward(s.position, go, s.rows.detach(), w)
        want = (X.expert_sort_backward(s.position, gr), gw)
        assert _same(got, want[:len(got)])
    rows = X.expert_sort(ids, x, 4)
    wl = w.clone().requires_grad_()
    y = X.expert_unsort(rows.position, rows.rows, wl)
    X.expert_sort(ids, go, 4, out=rows.rows)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward(go)


def test_offsets_past_32_bits(X):
    """More than 2^32 bytes of sorted rows, expert weights, tokens and norm rows: the last ones are right."""
    free = torch.cuda.mem_get_info()[0]
    if free < 80 << 30:
        pytest.skip("needs 80 GiB of free device memory")
    S, k, H, E = 40003, 8, 7168, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(0, E, (1, S, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((1, S, H), generator=g, device="cuda", dtype=BF)
    s = X.expert_sort(ids, x, E)
    order = torch.argsort(ids.view(-1), stable=True)
    assert s.rows.numel() * 2 > 1 << 32
    for lo in (0, S * k // 2, S * k - 5000):
        assert torch.equal(s.rows[lo:lo + 5000], x[0][order[lo:lo + 5000] // k])
    assert torch.equal(s.position.view(-1)[order], torch.arange(S * k, device="cuda", dtype=torch.int32))
    w = torch.full((1, S, k), 0.125, device="cuda")  # eight equal rows, exact weights
    assert torch.equal(X.expert_unsort(s.position, s.rows, w), x)
    gr, gw = X.expert_unsort_backward(s.position, x, s.rows, w)
    assert torch.equal(gr[-3000:], (x[0][order[-3000:] // k].float() * 0.125).to(BF))
    del s, gr, gw
    q = X.expert_sort(ids, x, E, quantize=True)
    assert torch.equal(q.rows[-3000:].float() * q.scales[-3000:, None],
                       (lambda t: t.rows.float() * t.scales[:, None])(
                           X.expert_sort(torch.zeros((1, 3000, 1), dtype=torch.int32, device="cuda"),
                                         x[:, order[-3000:] // k].contiguous(), 1, quantize=True)))
    del q, x, order
    # 5 GB of weights: the last expert's
    wts = torch.randint(-127, 128, (40, 8200, 16384), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.randint(-127, 128, (700, 16384), generator=g, device="cuda", dtype=torch.int8)
    sw = torch.rand((40, 8200), generator=g, device="cuda")
    sx = torch.rand(700, generator=g, device="cuda")
    for first in (690, 0):  # ten rows, and all of them
        off = torch.zeros(41, dtype=torch.int32, device="cuda")
        off[40] = 700
        off[39] = first
        off[38] = first
        off[1:38] = first
        got = X.expert_matmul(xs, sx, wts, sw, offsets=off, dtype=F32)[first:]
        ref = (xs[first:].double() @ wts[39].double().t().contiguous()).cpu() * sx[first:].double().cpu()[:, None] * sw[39].double().cpu()
        U.check_close(got, ref, 3.01 * U.U32 * ref.abs(), "last expert")
    del wts
    xs = torch.randint(-127, 128, (270011, 16384), generator=g, device="cuda", dtype=torch.int8)
    sx = torch.rand(270011, generator=g, device="cuda")
    wd = torch.randint(-127, 128, (72, 16384), generator=g, device="cuda", dtype=torch.int8)
    got = X.expert_matmul(xs, sx, wd, sw[0, :72].contiguous(), dtype=F32)[-100:]
    ref = (xs[-100:].double() @ wd.double().t().contiguous()).cpu() * sx[-100:].double().cpu()[:, None] * sw[0, :72].double().cpu()
    U.check_close(got, ref, 3.01 * U.U32 * ref.abs(), "last rows")
    del xs
    x = torch.randn((310007, 7168), generator=g, device="cuda", dtype=BF)
    n = X.add_rms_norm(x, None, torch.ones(7168, dtype=BF, device="cuda"), format="mxfp8")
    m = X.add_rms_norm(x[-50:].contiguous(), None, torch.ones(7168, dtype=BF, device="cuda"), format="mxfp8")
    assert torch.equal(n.rows[-50:].view(torch.uint8), m.rows.view(torch.uint8))
    assert torch.equal(n.scales[-50:].view(torch.uint8), m.scales.view(torch.uint8))
    a = X.silu_mul_quantize(x)
    b = X.silu_mul_quantize(x[-50:].contiguous())
    assert torch.equal(a.rows[-50:], b.rows) and torch.equal(a.scales[-50:], b.scales)


def test_binding_refusals(X):
    """Shapes, types, strides and gradients that the binding refuses on GPU tensors."""
    ids = torch.zeros((2, 4, 2), dtype=torch.int32, device="cuda")
    rows = torch.zeros((2, 4, 16), dtype=BF, device="cuda")
    pos = torch.zeros((2, 4, 2), dtype=torch.int32, device="cuda")
    flat = torch.zeros((16, 16), dtype=BF, device="cuda")
    w = torch.zeros((2, 4, 2), device="cuda")
    q, s = torch.zeros((8, 16), dtype=torch.int8, device="cuda"), torch.zeros(8, device="cuda")
    ew, es = torch.zeros((3, 8, 16), dtype=torch.int8, device="cuda"), torch.zeros((3, 8), device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    wt = torch.ones(16, dtype=BF, device="cuda")
    leaf = flat.clone().requires_grad_()
    bad = [
        lambda: X.expert_sort(ids.long(), rows, 4), lambda: X.expert_sort(ids[0], rows, 4),
        lambda: X.expert_sort(ids, rows[:1], 4), lambda: X.expert_sort(ids, rows.transpose(1, 2), 4),
        lambda: X.expert_sort(ids, rows, 0), lambda: X.expert_sort(ids, rows, 4, capacity=-1),
        lambda: X.expert_sort(ids, rows, 4, scales=torch.zeros((2, 3, 4), device="cuda")),
        lambda: X.expert_sort(ids, rows, 4, out=flat.float()), lambda: X.expert_sort(ids, rows, 4, out=flat[:3]),
        lambda: X.expert_sort(ids, rows.half(), 4, quantize=True),
        lambda: X.expert_sort(ids, rows, 4, quantize=True, scales=w),
        lambda: X.expert_sort(ids, rows[:, :, :4], 4), lambda: X.expert_sort(ids, rows[:, :, :7].contiguous(), 4),
        lambda: X.expert_sort(ids, rows.clone().requires_grad_(), 4, quantize=True),
        lambda: X.expert_sort(ids, rows.clone().requires_grad_(), 4, out=flat),
        lambda: X.expert_sort(ids, rows.clone().requires_grad_(), 4, stream=torch.cuda.Stream()),
        lambda: X.expert_unsort(pos, leaf, stream=torch.cuda.Stream()),
        lambda: X.expert_unsort(pos, flat.half()), lambda: X.expert_unsort(pos[0], flat),
        lambda: X.expert_unsort(pos.long(), flat), lambda: X.expert_unsort(pos, flat, w.double()),
        lambda: X.expert_unsort(pos, flat, w[:, :, :1]), lambda: X.expert_unsort(pos, flat, out=rows.float()),
        lambda: X.expert_unsort(pos, flat, keep_empty=True), lambda: X.expert_unsort(pos, flat.t()),
        lambda: X.expert_unsort(pos, leaf, out=rows), lambda: X.expert_unsort(pos, flat[:, :4].contiguous()),
        lambda: X.expert_unsort_backward(pos, rows), lambda: X.expert_unsort_backward(pos, rows, flat.float()),
        lambda: X.expert_unsort_backward(pos, rows, None, w, grad_rows=flat),
        lambda: X.expert_unsort_backward(pos, rows[:1], flat),
        lambda: X.expert_matmul(q, s, ew, es), lambda: X.expert_matmul(q, s, ew, es, offsets=off[:3]),
        lambda: X.expert_matmul(q, s, ew[0], es[0], offsets=off), lambda: X.expert_matmul(q, s, ew[:, :, :8], es, offsets=off),
        lambda: X.expert_matmul(q, s[:4], ew, es, offsets=off), lambda: X.expert_matmul(q.float(), s, ew, es, offsets=off),
        lambda: X.expert_matmul(q, s, ew, es, offsets=off, dtype=torch.float16),
        lambda: X.expert_matmul(q, s.clone().requires_grad_(), ew, es, offsets=off),
        lambda: X.expert_matmul(q[:, :8].contiguous(), s, ew[0, :, :8].contiguous(), es[0]),
        lambda: X.silu_mul_quantize(flat.half()), lambda: X.silu_mul_quantize(flat[:, :15].contiguous()),
        lambda: X.silu_mul_quantize(flat), lambda: X.silu_mul_quantize(leaf),
        lambda: X.silu_mul_quantize(flat.repeat(1, 2), offsets=off.long()),
        lambda: X.add_rms_norm(flat, flat, wt, format="mxfp8"), lambda: X.add_rms_norm(flat, flat, wt.float(), format="int8"),
        lambda: X.add_rms_norm(flat, flat[:3], wt, format="int8"), lambda: X.add_rms_norm(flat, None, wt, -1.0, format="int8"),
        lambda: X.add_rms_norm(leaf, None, wt, format="int8"),
        lambda: X.add_rms_norm(flat, None, wt, format="int8", out=flat),
        lambda: X.add_rms_norm(flat, None, wt, format="int8", residual_out=flat.float()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with torch.no_grad():
        X.silu_mul_quantize(flat.repeat(1, 2).requires_grad_())


def test_sizes_past_the_argument_blocks(X):
    """Numbers that an argument block cannot hold are refused by name."""
    from combine_route_mask_amd.moe_ep import MoeEpArgError
    ids = torch.zeros((1, 4, 2), dtype=torch.int32, device="cuda")
    rows = torch.zeros((1, 4, 16), dtype=BF, device="cuda")
    for call in (lambda: X.expert_sort(ids, rows, 4, capacity=2.5, out=None),
                 lambda: X.expert_sort(ids, rows, 4, active_rank_mask=-1),
                 lambda: X.expert_sort(ids, rows, 4, scales=torch.zeros((1, 4, 2), device="cuda", requires_grad=True)),
                 lambda: X.expert_sort_workspace_bytes(1 - (1 << 32), 4, 2, 4),
                 lambda: X.expert_matmul(torch.zeros((0, 1 << 33), dtype=torch.int8, device="cuda"),
                                         torch.zeros(0, device="cuda"),
                                         torch.zeros((0, 1 << 33), dtype=torch.int8, device="cuda"),
                                         torch.zeros(0, device="cuda"))):
        with pytest.raises((MoeEpArgError, TypeError)):
            call()


def test_empty_calls(X):
    """No row, no slot, no capacity: nothing to do, and the offsets say so."""
    ids, rows = torch.zeros((2, 0, 3), dtype=torch.int32, device="cuda"), torch.zeros((2, 0, 32), dtype=BF, device="cuda")
    s = X.expert_sort(ids, rows, 5, quantize=True)
    assert s.rows.shape == (0, 32) and s.offsets.tolist() == [0] * 11 and s.counts.tolist() == [0] * 10
    w1, s1, w2, s2 = _weights(np.random.default_rng(0), 10, 32, 16)
    y, _, a = _experts(X, s, (w1, s1, w2, s2))
    assert y.shape == (0, 32) and a.rows.shape == (0, 16)
    assert X.expert_unsort(s.position, y).shape == (2, 0, 32)
    gr, gw = X.expert_unsort_backward(s.position, rows, y)
    assert gr.shape == (0, 32) and gw.shape == (2, 0, 3)
    n = X.add_rms_norm(y, None, torch.ones(32, dtype=BF, device="cuda"), format="mxfp8")
    assert n.rows.shape == (0, 32) and n.scales.shape == (0, 1)
    # slots, but none of their experts here
    ids = torch.full((2, 5, 3), 10, dtype=torch.int32, device="cuda")
    rows = torch.ones((2, 5, 32), dtype=BF, device="cuda")
    s = X.expert_sort(ids, rows, 5, capacity=4)
    assert s.offsets.tolist() == [0] * 11 and bool((s.position == -1).all())
    assert not bool(X.expert_unsort(s.position, s.rows).any())
    gr, gw = X.expert_unsort_backward(s.position, rows, s.rows)
    assert not bool(gr.any()) and not bool(gw.any())


def test_gradients_at_any_address(X):
    """Gradients that begin between 16-byte boundaries (parts of one flat buffer) or repeat one number are the same
    gradients."""
    st = _state(None, 13, S=60)
    ids, w = st["ids"], st["w"]
    x = st["rows"]
    for dtype in (BF, F32):
        xl, wl = x.to(dtype).requires_grad_(), w.clone().requires_grad_()
        s = X.expert_sort(ids, xl, 4)
        y = X.expert_unsort(s.position, s.rows, wl)
        go, gs = torch.randn_like(y), torch.randn_like(s.rows)
        for shift in (1, 3):
            odd = []
            for g in (go, gs):
                flat = torch.empty(g.numel() + shift, dtype=dtype, device="cuda")
                odd.append(flat[shift:].view(g.shape))
                odd[-1].copy_(g)
                assert odd[-1].data_ptr() % 16 and odd[-1].is_contiguous()
            want = torch.autograd.grad((y, s.rows), (xl, wl), (go, gs), retain_graph=True)
            got = torch.autograd.grad((y, s.rows), (xl, wl), tuple(odd), retain_graph=True)
            assert _same(got, want)
            # each operator's own
            assert _same(torch.autograd.grad(s.rows, xl, odd[1], retain_graph=True),
                         torch.autograd.grad(s.rows, xl, gs, retain_graph=True))
        got = torch.autograd.grad(y.sum(), (xl, wl), retain_graph=True)
        assert _same(got, torch.autograd.grad(y, (xl, wl), torch.ones_like(y)))


def test_the_default_streams_raw_handle(X):
    """stream=0 is the default stream (the handle of torch's current stream at first): a call waits for the inputs
    that it is still making, and work there waits for the call."""
    rng = np.random.default_rng(6)
    weights = _weights(rng, 8, 256, 96) + (torch.ones(256, dtype=BF, device="cuda"),)
    assert torch.cuda.current_stream().cuda_stream == 0
    a, b = _state(rng, 21, S=600), _state(rng, 22, S=600)
    want = [_layer(X, st, weights) for st in (a, b)]
    held = {k: v.clone() for k, v in a.items()}
    for turn in range(4):
        torch.cuda._sleep(10_000_000)
        for k, v in held.items():
            v.copy_((a, b)[turn & 1][k])
        got = [t.clone() for t in _layer(X, held, weights, stream=torch.cuda.current_stream().cuda_stream)]
        torch.cuda.synchronize()
        assert _same(got, want[turn & 1]), turn
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the argument, not the current stream, says where
        out = X.expert_sort(held["ids"], held["rows"], 4, stream=0)
    assert torch.equal(out.position, X.expert_sort(held["ids"], held["rows"], 4).position)
    on = X._On(held["rows"].device, 0)
    with torch.cuda.stream(side):
        with on:
            assert torch.cuda.current_stream().cuda_stream == 0
        assert torch.cuda.current_stream().cuda_stream == side.cuda_stream
