"""NaN and infinite logits in the router's gradient, in each of its kernels: a
NaN that was not chosen has no part in a gradient over the chosen experts, and
makes all of one over all experts NaN."""
import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")

# tokens, experts, places: 16 lanes a token, 64 lanes, and logits in LDS
PATHS = [(8, 8, 2), (8, 20, 3), (2200, 100, 2), (2200, 400, 4), (8, 100, 2), (8, 400, 4), (8, 64, 20), (8, 600, 2),
         (8, 2000, 20)]


@pytest.fixture(scope="module")
def R():
    from combine_route_mask_amd import router, moe_ep
    assert torch.cuda.is_available() and moe_ep.moe_ep_is_supported()
    return router


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", PATHS)
def test_gradient_of_rows_with_nan(R, T, E, k, dtype):
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn((T, E), generator=g)
    gw = torch.randn((T, k), generator=g)
    x[0, E // 2] = NAN          # not chosen
    x[1, E // 3] = x[1, 0] = INF  # chosen
    x[2] = NAN                  # nothing to choose
    x[3] = -INF
    x[4, 1:] = -INF             # one expert
    x[T - 1, E - 1] = NAN
    x = x.to(dtype)
    for renormalize in (True, False):
        r = R.route_top_k(x.cuda(), k, renormalize=renormalize)
        w, ids = r.weights.cpu(), r.ids.cpu().long()
        assert bool(w[[0, 1, T - 1]].isnan().all()) and w[2].tolist() == w[3].tolist() == [0] * k
        assert w[4].tolist() == [1] + [0] * (k - 1)
        d = R.route_top_k_backward(x.cuda(), r.ids, gw.cuda(), renormalize=renormalize).cpu()
        assert not bool(d[3].any() or d[4].any())
        if not renormalize:
            assert bool(d[[0, 1, 2, T - 1]].isnan().all())
        else:
            assert not bool(d[2].any())
            chosen = torch.zeros(E, dtype=torch.bool)
            chosen[ids[1]] = True
            assert bool(d[1][chosen].isnan().all()) and not bool(d[1][~chosen].any())
            for t in (0, T - 1):  # the softmax over the chosen, as without the NaN
                p = x[t, ids[t]].double().softmax(0)
                gt = gw[t].double()
                want = torch.zeros(E, dtype=torch.float64)
                want[ids[t]] = p * (gt - (p * gt).sum())
                # p is off by 32 + k roundings, the difference and the products by three, of numbers up to 2 max |g|
                err = (2 * 2.0 ** -24 * (40 + 2 * k) * 2 * float(gt.abs().max()))
                unit = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
                assert bool(((d[t].double() - want).abs() <= err + unit * (want.abs() + err)).all())
        rest = torch.ones(T, dtype=torch.bool)
        rest[[0, 1, 2, T - 1]] = False
        assert bool(d[rest].isfinite().all()), "a NaN reached another token"
