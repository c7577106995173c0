"""Forward-mode tangents are refused, not dropped: a dual tensor asks for no
gradient and has a readable address, so nothing but a look at it would tell."""
import pytest
import torch
from torch.autograd import forward_ad

from combine_route_mask_amd import experts as X, ffn as F, moe_ep as m, router as R
from tests.test_ffn_refusals import _calls

BF = torch.bfloat16


def _dual(t):
    return forward_ad.make_dual(t.clone(), torch.ones_like(t))


def _expert_calls(dual):
    ids = torch.zeros((1, 2, 2), dtype=torch.int32)
    rows, flat, w, wt = torch.zeros(1, 2, 16), torch.zeros(2, 16), torch.zeros(1, 2, 2), torch.zeros(16)
    q, s = torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)
    return {
        "sort rows": lambda: X.expert_sort(ids, dual(rows), 4),
        "sort scales": lambda: X.expert_sort(ids, rows, 4, scales=dual(torch.zeros(1, 2, 4))),
        "sort backward": lambda: X.expert_sort_backward(ids, dual(flat)),
        "unsort rows": lambda: X.expert_unsort(ids, dual(flat)),
        "unsort weights": lambda: X.expert_unsort(ids, flat, dual(w)),
        "unsort backward": lambda: X.expert_unsort_backward(ids, dual(rows), flat, w),
        "int8 scales": lambda: X.expert_matmul(q, dual(s), q, s),
        "silu": lambda: X.silu_mul_quantize(dual(torch.zeros(2, 32))),
        "norm": lambda: X.add_rms_norm(dual(flat), None, wt, format="int8"),
        "norm residual": lambda: X.add_rms_norm(flat, dual(flat), wt, format="int8"),
    }


def _layer_calls(dual):
    x, w1, w2 = torch.zeros(2, 32, dtype=BF), torch.zeros(64, 32, dtype=BF), torch.zeros(32, 32, dtype=BF)
    calls = {n: c for n, c in _calls(F, R, dual).items() if n not in ("restore_rows", "expert_ffn", "route_top_k")}
    calls.update({
        "ffn x": lambda: F.expert_ffn(dual(x), w1, w2), "ffn w1": lambda: F.expert_ffn(x, dual(w1), w2),
        "ffn w2": lambda: F.expert_ffn(x, w1, dual(w2)), "route": lambda: R.route_top_k(dual(torch.zeros(2, 4)), 2),
        "product weight": lambda: F.expert_product(x, dual(w2)), "gated weight": lambda: F.gated_product(x, dual(w1)),
    })
    return calls


@pytest.mark.parametrize("calls", [_expert_calls, _layer_calls])
def test_tangents_are_refused(calls):
    with forward_ad.dual_level():
        for name, call in calls(_dual).items():
            with pytest.raises(m.MoeEpArgError, match="forward-mode"):
                call()
            with torch.no_grad(), pytest.raises(m.MoeEpArgError, match="forward-mode"):  # no_grad leaves tangents on
                call()


def test_tangents_of_leaves_are_refused():
    """Next to a reverse gradient too."""
    with forward_ad.dual_level():
        with pytest.raises(m.MoeEpArgError, match="forward-mode"):
            R.route_top_k(_dual(torch.zeros(2, 4).requires_grad_()), 2)
        with pytest.raises(m.MoeEpArgError, match="forward-mode"):
            F.expert_ffn(_dual(torch.zeros(2, 32, dtype=BF)).requires_grad_(), torch.zeros(64, 32, dtype=BF),
                         torch.zeros(32, 32, dtype=BF))


@pytest.mark.parametrize("calls", [_expert_calls, _layer_calls])
def test_plain_tensors_within_a_dual_level(calls):
    """Tensors without a tangent meet the other checks."""
    with forward_ad.dual_level():
        for call in calls(lambda t: t).values():
            with pytest.raises(m.MoeEpArgError, match="GPU tensor"):
                call()
