"""The router and its gradient against 64-bit references: ties, masked
experts, rows that the mask leaves nothing, infinities and NaN, every count of
experts and places."""
import numpy as np
import pytest
import torch

from tests.ffn_util import U32
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def R():
    from combine_route_mask_amd import router, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return router


def _chosen(row, k):
    """Experts of a row: largest first, equal ones by index, none at -infinity or NaN."""
    held = [i for i in range(len(row)) if row[i] > -np.inf]
    held.sort(key=lambda i: (-row[i], i))
    return held[:k] + [len(row)] * (k - len(held[:k]))


def reference(logits, k, renormalize, scale):
    """(ids, weights, softmax [T, E]) in float64."""
    x = logits.double().numpy()
    T, E = x.shape
    ids = np.array([_chosen(r, k) for r in x], dtype=np.int64).reshape(T, k)
    p = np.zeros((T, E))
    for t in range(T):
        among = [i for i in ids[t] if i < E] if renormalize else range(E)
        if len(among) and ids[t, 0] < E:
            v = x[t, list(among)]
            with np.errstate(invalid="ignore"):
                e = np.exp(v - x[t, ids[t, 0]])
            p[t, list(among)] = e / e.sum()
    w = np.concatenate([p, np.zeros((T, 1))], 1)[np.arange(T)[:, None], ids] * scale
    return ids, w, p


def _logits(rng, T, E, dtype, kind):
    x = rng.standard_normal((T, E)) * 2
    if kind == "ties":
        x = np.round(x)
        x[rng.random((T, E)) < 0.2] = -0.0
    if kind == "masked":
        x[rng.random((T, E)) < 0.5] = -np.inf
        x[:, 0] = -np.inf
        x[0] = -np.inf  # a row that the mask leaves nothing
    if kind == "lowest":
        x[rng.random((T, E)) < 0.7] = float(torch.finfo(dtype).min)
        x[0] = float(torch.finfo(dtype).min)
    return torch.from_numpy(x).to(dtype)


def _error(logits, E):
    """Relative error of a weight: the argument's rounding (its size times 2^-24), expf, E additions, a quotient and a
    product."""
    x = logits.double()
    top = x.where(x > -np.inf, torch.full_like(x, -1e4)).amax(1, keepdim=True)
    far = (top - x).where(x > -np.inf, torch.zeros_like(x)).clamp(max=104.0)
    return ((far + E + 16) * 2 * U32).numpy()


SHAPES = [(1, 1, 1), (1, 256, 8), (5, 4, 4), (3, 7, 2), (64, 64, 64), (33, 65, 6), (100, 130, 8), (17, 512, 16),
          (9, 1000, 3), (4, 4096, 64), (1025, 32, 4), (3000, 8, 2), (2, 257, 1),
          (5, 200, 40), (7, 500, 17), (18, 260, 16), (16, 256, 16), (31, 16, 16), (6, 17, 17),
          (2051, 130, 8), (2049, 300, 16)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "lowest"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_route_and_gradient(R, T, E, k, kind, dtype, renormalize):
    log(f"route {T}x{E} top {k} {kind} {dtype} {renormalize}")
    rng = np.random.default_rng(T * E + k)
    logits = _logits(rng, T, E, dtype, kind)
    scale = 2.5 if renormalize else 1.0
    ids, w, p = reference(logits, k, renormalize, scale)
    r = R.route_top_k(logits.cuda(), k, renormalize=renormalize, scale=scale)
    assert r.ids.dtype == torch.int32 and np.array_equal(r.ids.cpu().numpy(), ids)
    rel = np.concatenate([_error(logits, E), np.zeros((T, 1))], 1)[np.arange(T)[:, None], ids]
    assert (np.abs(r.weights.cpu().double().numpy() - w) <= rel * np.abs(w) + 2.0 ** -126).all()

    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    got = R.route_top_k_backward(logits.cuda(), r.ids, g.cuda(), renormalize=renormalize, scale=scale).cpu()
    spread = np.zeros((T, E + 1))
    np.put_along_axis(spread, ids, g.double().numpy(), 1)
    pj = np.concatenate([p, np.zeros((T, 1))], 1)[np.arange(T)[:, None], ids]
    mean = (pj * g.double().numpy()).sum(1, keepdims=True)
    size = np.abs(g.double().numpy()).max(1, keepdims=True)
    want = scale * p * (spread[:, :E] - mean)
    err = scale * p * (np.abs(spread[:, :E]) + size) * (2 * _error(logits, E).max(1, keepdims=True) + (k + 8) * 2 * U32)
    err = err + (2.0 ** -8 if dtype == BF else U32) * (np.abs(want) + err) + 2.0 ** -126
    assert got.dtype == dtype
    assert (np.abs(got.double().numpy() - want) <= err).all()


def test_infinities_and_nan(R):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[1.0, nan, 2.0, 0.0], [inf, 1.0, inf, 0.0], [nan] * 4, [-inf, -inf, 5.0, -inf],
                      [3e38, -3e38, 0.0, 1.0]]).cuda()
    for renormalize in (True, False):
        r = R.route_top_k(x, 2, renormalize=renormalize)
        assert r.ids.tolist() == [[2, 0], [0, 2], [4, 4], [2, 4], [0, 3]]
        w = r.weights.cpu()
        assert bool(w[0].isnan().all() and w[1].isnan().all())
        assert w[2].tolist() == [0, 0] and w[3].tolist() == [1, 0] and w[4].tolist() == [1, 0]
        g = R.route_top_k_backward(x, r.ids, torch.ones_like(r.weights), renormalize=renormalize).cpu()
        assert g[2].tolist() == [0] * 4 or bool(g[2].isnan().all())
        assert g[3].tolist() == [0] * 4 and g[4].tolist() == [0] * 4


def test_autograd(R):
    """autograd gives the explicit call's gradient, for leading axes and expanded gradients too."""
    torch.manual_seed(5)
    x = torch.randn(2, 7, 33, device="cuda", requires_grad=True)
    r = R.route_top_k(x, 3, renormalize=False, scale=2.0)
    assert r.ids.shape == r.weights.shape == (2, 7, 3) and not r.ids.requires_grad
    g, = torch.autograd.grad(r.weights.sum(), x)
    want = R.route_top_k_backward(x.detach(), r.ids, torch.ones_like(r.weights).detach(), renormalize=False, scale=2.0)
    assert torch.equal(g, want)
    # against differences of the definition in 64 bits
    t = x.detach().cpu().double().view(14, 33)
    ids = r.ids.cpu().view(14, 3).long()
    h = 1e-6
    for i in (0, 5, 32):
        up, down = t.clone(), t.clone()
        up[:, i] += h
        down[:, i] -= h
        d = (2 * up.softmax(1).gather(1, ids).sum(1) - 2 * down.softmax(1).gather(1, ids).sum(1)) / (2 * h)
        # differences to 1e-8, the gradient to 64 roundings of numbers up to 2
        assert bool(((g.cpu().double().view(14, 33)[:, i] - d).abs() < 1e-8 + 64 * 2 * U32).all())


def test_rows_at_any_address(R):
    """Logits that begin between 16 bytes, and given outputs."""
    x = torch.randn(5, 9, device="cuda")
    ids, w = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(4, 2, device="cuda")
    r = R.route_top_k(x[1:], 2, ids=ids, weights=w)
    assert r.ids is ids and r.weights is w
    want = R.route_top_k(x[1:].clone(), 2)
    assert torch.equal(ids, want.ids) and torch.equal(w, want.weights)
    b = x.bfloat16()
    assert torch.equal(R.route_top_k(b[1:], 2).ids, R.route_top_k(b[1:].clone(), 2).ids)
    out = torch.empty(5, 9, device="cuda")[1:]
    R.route_top_k_backward(x[1:], ids, w, out=out)
    assert torch.equal(out, R.route_top_k_backward(x[1:].clone(), ids, w))


def test_ids_out_of_range_have_no_part(R):
    x = torch.randn(3, 6, device="cuda")
    g = torch.randn(3, 3, device="cuda")
    ids = torch.tensor([[0, -1, 3], [6, 2, 2 ** 31 - 1], [-2 ** 31, 7, 6]], dtype=torch.int32, device="cuda")
    got = R.route_top_k_backward(x, ids, g).cpu()
    p = x[0, [0, 3]].softmax(0).cpu()
    gg = g[0, [0, 2]].cpu()
    want = p * (gg - (p * gg).sum())
    assert bool(((got[0, [0, 3]] - want).abs() < 1e-5).all())  # a few roundings of numbers of size 1
    assert bool((got[0, [1, 2, 4, 5]] == 0).all() and (got[1:] == 0).all())
