"""Expert sort, unsort and their gradients against 64-bit references: the
order and every moved byte exactly, sums within their roundings; one-token,
odd and ragged shapes on both the one-launch and the tiled path, ids out of
range, duplicate ids, slots and whole ranks without a row, capacities below
the pairs, planes whose ranks lie apart."""
import numpy as np
import pytest
import torch

from tests import expert_util as U
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module")
def X():
    from combine_route_mask_amd import experts, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return experts


def _plane(rng, shape, dtype, apart):
    """A random plane [R, S, row] on the GPU; `apart`: ranks 256 bytes further apart than they need."""
    R, S, n = shape
    if dtype == U8:
        t = torch.from_numpy(rng.integers(0, 256, size=shape, dtype=np.uint8))
    else:
        t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)
    t = t.cuda()
    if not apart:
        return t
    gap = 256 // t.element_size()
    room = torch.zeros(R * (S * n + gap), dtype=dtype, device="cuda")
    v = room.as_strided((R, S, n), (S * n + gap, n, 1))
    v.copy_(t)
    return v


# R, S, k, experts a rank, row, dtype, scale row bytes, capacity (None: all; a share of the pairs)
SORTS = [
    (1, 1, 8, 256, 7168, BF, 0, None),      # one token
    (1, 1, 1, 1, 8, BF, 0, None),
    (1, 0, 8, 64, 64, BF, 0, None),         # no slot at all
    (3, 0, 2, 300, 64, BF, 0, None),
    (1, 255, 8, 64, 136, BF, 0, None),      # the last sizes of one launch
    (1, 256, 8, 64, 136, BF, 0, None),
    (1, 257, 8, 64, 136, BF, 0, None),      # the first tiled ones
    (8, 16, 4, 32, 72, F32, 0, None),
    (64, 4, 8, 4, 8, BF, 0, None),
    (64, 33, 3, 5, 16, BF, 0, None),
    (1, 32, 64, 128, 24, BF, 0, None),      # top_k 64 in one launch
    (2, 600, 64, 70, 16, BF, 0, None),      # and tiled
    (1, 37, 8, 1024, 8, BF, 0, None),
    (1, 37, 8, 1025, 8, BF, 0, None),       # too many experts for one launch
    (1, 700, 5, 4096, 8, BF, 0, None),      # the most experts
    (64, 70, 8, 64, 8, BF, 0, None),
    (1, 20011, 1, 3, 8, BF, 0, None),       # several tiles of one-id slots
    (4, 3001, 2, 7, 40, BF, 0, None),
    (8, 128, 8, 32, 3584, U8, 448, None),   # payload formats with scale rows
    (8, 40, 8, 32, 7168, U8, 224, None),
    (2, 33, 3, 8, 16, U8, 7, None),         # a scale row of odd bytes
    (2, 700, 3, 8, 16, U8, 20, None),
    (2, 33, 3, 8, 16, U8, 4099, None),      # longer than a pass of the workgroup
    (1, 61, 8, 16, 48, BF, 0, 0.5),         # rows dropped past the capacity
    (2, 900, 4, 16, 48, BF, 0, 0.37),
    (1, 61, 8, 16, 48, BF, 0, 0.0),
    (1, 900, 4, 16, 48, BF, 0, 0.0),
    (2, 0, 2, 2000, 64, BF, 0, None),       # no slot, experts of a table
    (3, 3000, 3, 1300, 8, BF, 0, 0.9),      # several experts a thread, ranks before
    (1, 132000, 8, 200, 8, BF, 0, None),    # an expert's tiles take two passes of its scan
]


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("case", SORTS, ids=lambda c: "R%d S%d k%d e%d row%d %s scale%d cap%s" % (
    c[0], c[1], c[2], c[3], c[4], str(c[5])[6:], c[6], c[7]))
def test_sort_is_exact(X, case, apart):
    R, S, k, epr, n, dtype, srow, share = case
    log(f"sort {case} apart={apart}")
    rng = np.random.default_rng(abs(hash((R, S, k, epr, n))) % 2 ** 32)
    ids = U.draw_ids(rng, R, S, k, epr)
    if S > 2:
        ids[0, 1] = ids[0, 0, 0]  # one expert several times
    capacity = None if share is None else int(share * R * S * k)
    position, offsets, counts, kept = U.sort_reference(ids, epr, R * S * k if capacity is None else capacity)
    rows = _plane(rng, (R, S, n), dtype, apart)
    scales = _plane(rng, (R, S, srow), U8, apart) if srow else None
    gid = torch.from_numpy(ids).cuda()
    if apart:
        room = torch.zeros((R, S * k + 64), dtype=torch.int32, device="cuda")
        v = room[:, :S * k].unflatten(1, (S, k)) if S else room[:, :0].view(R, 0, k)
        v.copy_(gid)
        gid = v
    cap = R * S * k if capacity is None else capacity
    out = torch.full((cap, n), 77, dtype=dtype, device="cuda")
    os_ = torch.full((cap, srow), 77, dtype=U8, device="cuda") if srow else None
    s = X.expert_sort(gid, rows, epr, scales=scales, capacity=capacity, out=out, out_scales=os_)
    torch.cuda.synchronize()
    assert np.array_equal(s.position.cpu().numpy(), position)
    assert np.array_equal(s.offsets.cpu().numpy(), offsets)
    assert np.array_equal(s.counts.cpu().numpy(), counts)
    m = len(kept)
    for got, plane in ((s.rows, rows), (s.scales, scales)):
        if got is None:
            continue
        r, q = np.array([p[0] for p in kept], int), np.array([p[1] for p in kept], int)
        want = plane.cpu()[r, q]
        assert np.array_equal(U.bits(got[:m]), U.bits(want)), "moved rows differ"
        assert bool((got[m:] == 77).all()), "a row behind the last pair was written"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,S,k,epr,n", [(1, 1, 8, 64, 7168), (1, 3, 2, 4, 16), (8, 16, 4, 8, 8208), (1, 300, 8, 32, 144),
                                         (4, 1000, 2, 4, 48), (1, 400, 8, 16, 16400), (1, 2, 3, 4, 33024)])
def test_quantized_sort(X, R, S, k, epr, n, dtype):
    log(f"quantized sort R{R} S{S} k{k} e{epr} n{n} {dtype}")
    rng = np.random.default_rng(n + S)
    ids = U.draw_ids(rng, R, S, k, epr)
    rows = _plane(rng, (R, S, n), dtype, False) * torch.from_numpy(
        np.exp2(rng.integers(-90, 60, size=(R, S, 1))).astype(np.float32)).cuda().to(dtype)
    special = {}
    if S > 2:
        rows[0, 0] = 0
        rows[0, 1, 3] = float("nan")
        rows[0, 2, n - 1] = float("-inf")
        ids[0, :3, 0] = [0, 1 % epr, 0]
        special = {(0, 1), (0, 2)}
    position, _, _, kept = U.sort_reference(ids, epr, R * S * k)
    s = X.expert_sort(torch.from_numpy(ids).cuda(), rows, epr, quantize=True)
    torch.cuda.synchronize()
    assert np.array_equal(s.position.cpu().numpy(), position)
    m = len(kept)
    r, q = np.array([p[0] for p in kept], int), np.array([p[1] for p in kept], int)
    want = rows.cpu()[r, q].double()
    odd = np.array([p in special for p in kept], bool)
    U.check_int8(s.rows[:m].cpu()[~odd], s.scales[:m].cpu()[~odd], want[~odd], 0.0, "int8 rows")
    assert bool(s.scales[:m].cpu()[odd].isnan().all()) and int(s.rows[:m].cpu()[odd].abs().sum()) == 0
    if special:
        zero = position[0, 0, 0]
        assert float(s.scales[zero]) == 0.0 and int(s.rows[zero].abs().sum()) == 0


# R, S, k, rows H, num_rows beyond the largest place
UNSORTS = [(1, 1, 8, 7168), (1, 1, 1, 8), (8, 16, 4, 136), (1, 1000, 8, 72), (64, 70, 8, 16), (2, 9, 64, 1032),
           (1, 33, 3, 16392), (16, 64, 2, 8)]


def test_unsort_rounds_every_bf16_back_to_itself(X):
    """One row a slot without weights: every finite bf16 value, subnormals
    among them, comes back (-0 as the sum +0 + -0 = +0), NaN and infinities
    as themselves."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF).view(1, 8, 8192).cuda()
    p = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8, 1)
    got = X.expert_unsort(p, v[0])
    nan = v.isnan()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[~nan].view(torch.int16), (v[~nan] + 0.0).view(torch.int16))
    # halves between neighbours round to even: 2^-9 (1 + m / 128) twice of its half step
    x = torch.tensor([1 + 2 * i / 256 + (2 ** -9 if i % 2 else -2 ** -9) for i in range(8)], dtype=F32)
    rows = torch.stack([x, torch.full((8,), 2.0 ** -9)]).cuda()
    p = torch.tensor([[[0, 1]]], dtype=torch.int32, device="cuda")
    assert torch.equal(X.expert_unsort(p, rows).cpu()[0, 0], x + 2.0 ** -9)
    half = torch.tensor([[1.0 + i / 128 for i in range(8)], [2.0 ** -8] * 8], dtype=BF).cuda()
    ref = (half[0].double() + half[1].double()).cpu()
    even = torch.where((torch.arange(8) % 2) == 0, half[0].double().cpu(), ref + 2.0 ** -8)
    assert torch.equal(X.expert_unsort(p, half).double().cpu()[0, 0], even)


def _positions(rng, R, S, k, full=False):
    """Places of a random share of the pairs, in random order, and the number of rows (more than the places)."""
    here = np.ones((R, S, k), bool) if full else rng.random((R, S, k)) < 0.6
    if not full:
        here[rng.random((R, S)) < 0.3] = False
    n = int(here.sum())
    position = np.full((R, S, k), -1, np.int32)
    position[here] = rng.permutation(n + 3)[:n]
    return position, n + 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("R,S,k,H", UNSORTS)
def test_unsort(X, R, S, k, H, weighted, dtype):
    log(f"unsort R{R} S{S} k{k} H{H} {weighted} {dtype}")
    rng = np.random.default_rng(H + S + k)
    position, M = _positions(rng, R, S, k)
    rows = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(dtype)
    named = np.zeros(M, bool)
    named[position[position >= 0]] = True
    rows[~torch.from_numpy(named)] = float("nan")  # never read
    position[0, 0, 0] = M + 5 if position[0, 0, 0] < 0 else position[0, 0, 0]  # outside: adds nothing
    w = _plane(rng, (R, S, k), F32, R > 1) if weighted else None
    ref, mag = U.unsort_reference(position, rows, w)
    # k terms, each step of the fp32 chain rounds once
    slack = (k + 1) * U.U32 * mag * 1.001
    bound = slack + U.unit(dtype) * (ref.abs() + slack) + 2.0 ** -133
    gp, gr = torch.from_numpy(position).cuda(), rows.cuda()
    U.check_close(X.expert_unsort(gp, gr, w), ref, bound, "unsort")
    # into planes that lie apart, empty slots left alone
    room = torch.full((R, S * H + 64), 7.0, dtype=dtype, device="cuda")
    out = room[:, :S * H].unflatten(1, (S, H))
    got = X.expert_unsort(gp, gr, w, out=out, keep_empty=True)
    empty = torch.from_numpy(((position < 0) | (position >= M)).all(2))
    assert bool((got.cpu()[empty] == 7).all()) and bool((room[:, S * H:] == 7).all())
    ref[empty] = 7
    U.check_close(got, ref, bound, "unsort into planes")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("R,S,k,H", UNSORTS)
def test_unsort_backward(X, R, S, k, H, weighted, dtype):
    log(f"unsort backward R{R} S{S} k{k} H{H} {weighted} {dtype}")
    rng = np.random.default_rng(H + S + k + 1)
    position, M = _positions(rng, R, S, k)
    here = position >= 0
    rows = torch.from_numpy(rng.standard_normal((M, H)).astype(np.float32)).to(dtype)
    go = _plane(rng, (R, S, H), dtype, R > 1)
    w = _plane(rng, (R, S, k), F32, R > 1) if weighted else None
    gr0 = torch.full((M, H), 5.0, dtype=dtype, device="cuda")
    gr, gw = X.expert_unsort_backward(torch.from_numpy(position).cuda(), go, rows.cuda(), w, grad_rows=gr0)
    r, q, j = here.nonzero()
    at = torch.from_numpy(position[here]).long()
    g = go.cpu().double()[r, q]
    ref_rows = torch.full((M, H), 5.0, dtype=torch.float64)  # rows that no pair names stay
    ref_rows[at] = g * (w.cpu().double()[r, q, j][:, None] if weighted else 1.0)
    U.check_close(gr, ref_rows, (U.unit(dtype) + 2 * U.U32) * ref_rows.abs() + 2.0 ** -133, "grad_rows")
    ref_w, mag = torch.zeros(R, S, k, dtype=torch.float64), torch.zeros(R, S, k, dtype=torch.float64)
    ref_w[r, q, j] = (rows.double()[at] * g).sum(1)
    mag[r, q, j] = (rows.double()[at] * g).abs().sum(1)
    # a sum of H products, whatever its order, with at most H + 16 roundings
    U.check_close(gw, ref_w, (H + 16) * U.U32 * mag * 1.001, "grad_weights")
    only, none = X.expert_unsort_backward(torch.from_numpy(position).cuda(), go, None, w, need_weights=False,
                                          grad_rows=torch.full_like(gr0, 5.0))
    assert none is None and torch.equal(only, gr)
    none, only = X.expert_unsort_backward(torch.from_numpy(position).cuda(), go, rows.cuda(), w, need_rows=False)
    assert none is None and torch.equal(only, gw)


@pytest.mark.parametrize("R,S,k,epr,H", [(1, 5, 3, 4, 24), (4, 30, 4, 8, 40), (1, 700, 4, 16, 16)])
def test_gradients_against_differences(X, R, S, k, epr, H):
    """The loss sum(g * unsort(2 * sort(x), w)) is linear in x and in w; on
    small whole numbers in fp32 every sum is exact, so its differences equal
    the gradient exactly."""
    rng = np.random.default_rng(S)
    ids = torch.from_numpy(U.draw_ids(rng, R, S, k, epr)).cuda()
    whole = lambda *shape: torch.from_numpy(rng.integers(-4, 5, size=shape).astype(np.float32)).cuda()  # noqa: E731
    x, w, g = whole(R, S, H), whole(R, S, k), whole(R, S, H)

    def loss(x, w):
        s = X.expert_sort(ids, x, epr)
        return (g * X.expert_unsort(s.position, 2 * s.rows, w)).double().sum()

    x.requires_grad_(), w.requires_grad_()
    gx, gw = torch.autograd.grad(loss(x, w), (x, w))
    with torch.no_grad():
        for _ in range(4):
            d, e = whole(R, S, H), whole(R, S, k)
            assert float((loss(x + d, w) - loss(x - d, w)) / 2) == float((gx.double() * d).sum())
            assert float((loss(x, w + e) - loss(x, w - e)) / 2) == float((gw.double() * e).sum())
    # the formula's: the gradient of the sort is the unweighted way back
    s = X.expert_sort(ids, x.detach(), epr)
    back = X.expert_unsort_backward(s.position, g, torch.zeros_like(s.rows), w.detach())[0]
    m = int(s.offsets[-1])
    back[m:] = 0
    ref, _ = U.unsort_reference(s.position.cpu(), 2 * back, None)
    assert torch.equal(gx.cpu().double(), ref)


def test_gradient_with_dropped_rows(X):
    """Pairs past the capacity carry no gradient; rows behind the last are zeros."""
    ids = torch.tensor([[[0, 1], [1, 0], [1, 9]]], dtype=torch.int32, device="cuda")
    x = torch.arange(1.0, 49, device="cuda").view(1, 3, 16).requires_grad_()
    s = X.expert_sort(ids, x, 2, capacity=3)
    assert s.position.tolist() == [[[0, 2], [-1, 1], [-1, -1]]]
    assert s.offsets.tolist() == [0, 2, 3] and s.counts.tolist() == [2, 3]
    s.rows.sum().backward()
    assert x.grad[0, :, 0].tolist() == [2.0, 1.0, 0.0]
    s = X.expert_sort(ids, x, 2, capacity=8)
    assert bool((s.rows[5:] == 0).all())
    w = torch.ones((1, 3, 2), device="cuda", requires_grad=True)
    y = X.expert_unsort(s.position, s.rows.detach(), w)
    y.sum().backward()
    assert w.grad[0, 2].tolist() == [float(x.detach()[0, 2].sum()), 0.0]


def test_most_pairs(X):
    """2^31 - 8 pairs, the most that a call takes: id j % 4 for every slot's pair j, so that every place is known."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of free device memory")
    S, k, E, H = 2 ** 28 - 1, 8, 4, 8
    log(f"sort S{S} k{k}")
    ids = (torch.arange(k, device="cuda", dtype=torch.int32) % E).expand(1, S, k).contiguous()
    rows = torch.arange(S, device="cuda", dtype=torch.int32).remainder_(251).to(BF)[None, :, None].expand(1, S, H).contiguous()
    s = X.expert_sort(ids, rows, E)
    del ids
    assert s.counts.tolist() == [2 * S] * E and s.offsets.tolist() == [2 * S * e for e in range(E + 1)]
    q = torch.arange(S, device="cuda", dtype=torch.int32)
    for j in range(k):
        assert torch.equal(s.position[0, :, j], 2 * S * (j % E) + 2 * q + j // E)
    for e in range(E):
        for b in range(2):
            assert torch.equal(s.rows.view(E, S, 2, H)[e, :, b], rows[0])
    out = X.expert_unsort(s.position, s.rows)
    assert torch.equal(out, rows * 8)
    gr, gw = X.expert_unsort_backward(s.position, rows, s.rows, grad_rows=s.rows, need_weights=False)
    for e in range(E):
        assert torch.equal(gr.view(E, S, 2, H)[e, :, 1], rows[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [16, 1056])
def test_more_slots_than_workgroups(X, H, dtype):
    """A workgroup's second slot is what it is in a call of its own (2^22 workgroups at most), in the quantising
    sort, the weighted way back and both gradients; small whole numbers make every sum exact."""
    S, E = (1 << 22) + 77, 3
    log(f"slots past the grid S{S} H{H} {dtype}")
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GiB of free device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    ids = torch.randint(0, E, (1, S, 1), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randint(-8, 9, (1, S, H), generator=g, device="cuda", dtype=torch.int8).to(dtype)
    s = X.expert_sort(ids, x, E, quantize=True)
    p = s.position[0, :, 0].long()
    assert torch.equal(p[torch.argsort(ids.view(-1), stable=True)], torch.arange(S, device="cuda"))
    for part in (slice(0, S // 2), slice(S // 2, S)):
        t = X.expert_sort(ids[:, part].contiguous(), x[:, part].contiguous(), E, quantize=True)
        q = t.position[0, :, 0].long()
        assert torch.equal(s.scales[p[part]], t.scales[q])
        assert torch.equal(s.rows[p[part]], t.rows[q])
        del t, q
    position = s.position
    del s
    w = torch.exp2(torch.randint(-2, 3, (1, S, 1), generator=g, device="cuda").float())
    rows = torch.empty_like(x[0])
    rows[p] = x[0]
    out = X.expert_unsort(position, rows, w)
    assert torch.equal(out, (x.float() * w).to(dtype))
    go = out.mul_(2)  # some other whole or binary fractions
    gr, gw = X.expert_unsort_backward(position, go, rows, w)
    assert torch.equal(gw[0, :, 0], (x[0].float() * go[0].float()).sum(1))
    assert torch.equal(gr[p], (w[0] * go[0].float()).to(dtype))
