"""The router and the trainable expert layer refuse bad calls before any
launch, through the C ABI (argument blocks with made-up addresses; nothing is
launched) and in the binding (CPU tensors, shapes, types)."""
import pytest
import torch

from tests.test_experts_refusals import _fields


@pytest.fixture(scope="module")
def F():
    from combine_route_mask_amd import ffn
    return ffn


@pytest.fixture(scope="module")
def R():
    from combine_route_mask_amd import router
    return router


@pytest.fixture(scope="module")
def m():
    from combine_route_mask_amd import moe_ep
    return moe_ep


BLOCKS = {"moe_ep_route_args": "_ROUTE", "moe_ep_route_grad_args": "_ROUTE_GRAD", "moe_ep_checkpoint_args": "_CHECKPOINT",
          "moe_ep_product_args": "_PRODUCT", "moe_ep_gated_args": "_GATED", "moe_ep_gated_grad_args": "_GATED_GRAD",
          "moe_ep_weight_grad_args": "_WEIGHT_GRAD", "moe_ep_four_bit_args": "_FOUR_BIT"}


def _block(F, R, struct):
    return getattr(R if "route" in struct else F, BLOCKS[struct])


@pytest.mark.parametrize("struct", BLOCKS)
def test_argument_blocks_match_the_header(F, R, struct):
    assert "@" + "".join(k for _, k in _fields(struct)) == _block(F, R, struct).format


A = 1 << 20  # an aligned address that nothing reads
GOOD = {
    "moe_ep_route_top_k": ("moe_ep_route_args", dict(
        logits=A, ids=A, weights=A, tokens=4, num_experts=16, top_k=2, renormalize=1, row_type=1, scale=1.0, reserved=0)),
    "moe_ep_route_top_k_backward": ("moe_ep_route_grad_args", dict(
        logits=A, ids=A, grad_weights=A, grad_logits=A, tokens=4, num_experts=16, top_k=2, renormalize=1, row_type=1,
        scale=1.0, reserved=0)),
    "moe_ep_checkpoint_rows": ("moe_ep_checkpoint_args", dict(
        rows=A, codes=A, scales=A, num_rows=4, hidden_size=64, row_type=0)),
    "moe_ep_restore_rows": ("moe_ep_checkpoint_args", dict(
        rows=A, codes=A, scales=A, num_rows=4, hidden_size=64, row_type=0)),
    "moe_ep_expert_product": ("moe_ep_product_args", dict(
        x=A, w=A, offsets=A, out=A, num_rows=10, num_experts=4, n=32, k=64, transposed=0, zero_rest=0, reserved=0)),
    "moe_ep_gated_product": ("moe_ep_gated_args", dict(
        x=A, w=A, offsets=A, out=A, pre=A, pre_scales=A, num_rows=10, num_experts=4, inter_size=32, k=64, save=2)),
    "moe_ep_gated_product_backward": ("moe_ep_gated_grad_args", dict(
        grad_out=A, w=A, offsets=A, pre=A, pre_scales=A, grad_pre=A, out=A, num_rows=10, num_experts=4, inter_size=32, n=64,
        save=2)),
    "moe_ep_product_weight_grad": ("moe_ep_weight_grad_args", dict(
        grad_out=A, x=A, offsets=A, grad_w=A, num_rows=10, num_experts=4, n=32, k=64, reserved=0)),
    "moe_ep_four_bit_product": ("moe_ep_four_bit_args", dict(
        x=A, w=A, w_scales=A, offsets=A, out=A, num_rows=10, num_experts=4, n=32, k=64, gated=0, out_type=0, reserved=0)),
}

ARG, UNSUP, CAP = -1, -2, -4
PRODUCTS = ("moe_ep_expert_product", "moe_ep_gated_product", "moe_ep_gated_product_backward", "moe_ep_product_weight_grad",
            "moe_ep_four_bit_product")
BAD = [(name, change, code) for name in PRODUCTS for change, code in (
    (dict(num_experts=0), ARG), (dict(num_experts=4097), ARG), (dict(offsets=0), ARG), (dict(offsets=A + 2), ARG),
    (dict(num_rows=-1), CAP), (dict(num_rows=1 << 31), CAP))]
BAD += [(name, change, code) for name in ("moe_ep_route_top_k", "moe_ep_route_top_k_backward") for change, code in (
    (dict(num_experts=0), ARG), (dict(num_experts=4097), ARG), (dict(top_k=0), ARG), (dict(top_k=17), ARG),
    (dict(top_k=65, num_experts=100), ARG), (dict(renormalize=2), ARG), (dict(row_type=2), UNSUP), (dict(reserved=1), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(tokens=-1), CAP), (dict(tokens=1 << 31), CAP),
    (dict(logits=0), ARG), (dict(logits=A + 2), ARG), (dict(ids=0), ARG), (dict(ids=A + 2), ARG))]
BAD += [(name, change, code) for name in ("moe_ep_checkpoint_rows", "moe_ep_restore_rows") for change, code in (
    (dict(hidden_size=0), ARG), (dict(hidden_size=48), ARG), (dict(hidden_size=(1 << 20) + 32), ARG),
    (dict(row_type=2), UNSUP), (dict(num_rows=-1), CAP), (dict(num_rows=1 << 31), CAP), (dict(rows=0), ARG),
    (dict(rows=A + 8), ARG), (dict(codes=A + 8), ARG), (dict(scales=0), ARG))]
BAD += [
    ("moe_ep_route_top_k", dict(weights=0), ARG), ("moe_ep_route_top_k_backward", dict(grad_weights=A + 1), ARG),
    ("moe_ep_route_top_k_backward", dict(grad_logits=0), ARG),
    ("moe_ep_expert_product", dict(n=0), ARG), ("moe_ep_expert_product", dict(n=12), ARG),
    ("moe_ep_expert_product", dict(k=4), ARG), ("moe_ep_expert_product", dict(k=131080), ARG),
    ("moe_ep_expert_product", dict(transposed=2), ARG), ("moe_ep_expert_product", dict(zero_rest=2), ARG),
    ("moe_ep_expert_product", dict(reserved=1), ARG), ("moe_ep_expert_product", dict(x=0), ARG),
    ("moe_ep_expert_product", dict(w=A + 8), ARG), ("moe_ep_expert_product", dict(out=A + 2), ARG),
    ("moe_ep_gated_product", dict(inter_size=65544), ARG), ("moe_ep_gated_product", dict(inter_size=12), ARG),
    ("moe_ep_gated_product", dict(inter_size=40), ARG), ("moe_ep_gated_product", dict(k=20), ARG),
    ("moe_ep_gated_product", dict(save=3), UNSUP), ("moe_ep_gated_product", dict(pre=0), ARG),
    ("moe_ep_gated_product", dict(pre_scales=0), ARG), ("moe_ep_gated_product", dict(save=1, pre=A + 8), ARG),
    ("moe_ep_gated_product", dict(save=1, pre_scales=0), ARG),
    ("moe_ep_gated_product", dict(out=0), ARG),
    ("moe_ep_gated_product_backward", dict(save=0), UNSUP), ("moe_ep_gated_product_backward", dict(save=7), UNSUP),
    ("moe_ep_gated_product_backward", dict(inter_size=40), ARG), ("moe_ep_gated_product_backward", dict(n=12), ARG),
    ("moe_ep_gated_product_backward", dict(grad_pre=0), ARG), ("moe_ep_gated_product_backward", dict(out=A + 8), ARG),
    ("moe_ep_gated_product_backward", dict(pre_scales=0), ARG),
    ("moe_ep_product_weight_grad", dict(n=12), ARG), ("moe_ep_product_weight_grad", dict(k=0), ARG),
    ("moe_ep_product_weight_grad", dict(grad_w=0), ARG), ("moe_ep_product_weight_grad", dict(x=A + 8), ARG),
    ("moe_ep_product_weight_grad", dict(reserved=1), ARG),
    ("moe_ep_four_bit_product", dict(n=0), ARG), ("moe_ep_four_bit_product", dict(n=1 << 30), ARG),
    ("moe_ep_four_bit_product", dict(n=33, gated=1), ARG), ("moe_ep_four_bit_product", dict(gated=2), ARG),
    ("moe_ep_four_bit_product", dict(k=16), ARG), ("moe_ep_four_bit_product", dict(k=48), ARG),
    ("moe_ep_four_bit_product", dict(k=131104), ARG), ("moe_ep_four_bit_product", dict(out_type=2), UNSUP),
    ("moe_ep_four_bit_product", dict(x=0), ARG), ("moe_ep_four_bit_product", dict(w=A + 8), ARG),
    ("moe_ep_four_bit_product", dict(w_scales=0), ARG), ("moe_ep_four_bit_product", dict(out=A + 1), ARG),
    ("moe_ep_four_bit_product", dict(reserved=1), ARG),
]


def _pack(F, R, name, change):
    struct, good = GOOD[name]
    values = dict(good, **change)
    fields = _fields(struct)
    assert set(values) == {n for n, _ in fields}
    return _block(F, R, struct).pack(*(values[n] for n, _ in fields))


@pytest.mark.parametrize("name,change,code", BAD, ids=lambda v: str(v))
def test_refused_blocks(F, R, m, name, change, code):
    assert getattr(m.lib, name)(_pack(F, R, name, change), None) == code
    assert m.lib.moe_ep_last_error().decode() != ""


@pytest.mark.parametrize("name", GOOD)
def test_no_block(m, name):
    assert getattr(m.lib, name)(None, None) == ARG


@pytest.mark.parametrize("name", [n for n in GOOD if n != "moe_ep_product_weight_grad"])
def test_nothing_to_do_needs_no_gpu(F, R, m, name):
    """Calls over no row or token return at once (a weights' gradient is then zeros, which a launch writes)."""
    rows = "tokens" if "route" in name else "num_rows"
    assert getattr(m.lib, name)(_pack(F, R, name, {rows: 0}), None) == 0


BF = torch.bfloat16


def _calls(F, R, make=lambda t: t):
    """Every public call with CPU tensors; `make` may change the differentiable ones."""
    x, w1, w2 = torch.zeros(2, 32, dtype=BF), torch.zeros(64, 32, dtype=BF), torch.zeros(32, 32, dtype=BF)
    q, s = torch.zeros(2, 32, dtype=torch.float8_e4m3fn), torch.zeros(2, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    codes, scales = torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    ids, w = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    saved = F.FfnCheckpoint(x, None, torch.zeros(2, 64, dtype=torch.float16),
                            torch.zeros(2, 8, dtype=torch.uint8).view(torch.float8_e8m0fnu))
    return {
        "checkpoint_rows": lambda: F.checkpoint_rows(make(x)), "restore_rows": lambda: F.restore_rows(q, s),
        "expert_product": lambda: F.expert_product(make(x), w2),
        "gated_product": lambda: F.gated_product(make(x), w1),
        "gated_product_backward": lambda: F.gated_product_backward(make(x), w2, saved.pre, saved.pre_scales),
        "product_weight_grad": lambda: F.product_weight_grad(make(x), x),
        "expert_matmul_mxfp4": lambda: F.expert_matmul_mxfp4(make(x), codes, scales),
        "expert_ffn": lambda: F.expert_ffn(x, w1, w2),
        "expert_ffn_forward": lambda: F.expert_ffn_forward(make(x), w1, w2),
        "expert_ffn_backward": lambda: F.expert_ffn_backward(make(x), saved, w1, w2),
        "route_top_k": lambda: R.route_top_k(torch.zeros(2, 4), 2),
        "route_top_k_backward": lambda: R.route_top_k_backward(make(torch.zeros(2, 4)), ids, w),
    }


def test_cpu_tensors_are_refused(F, R, m):
    for call in _calls(F, R).values():
        with pytest.raises(m.MoeEpArgError, match="GPU tensor"):
            call()


def test_gradients_are_not_dropped_in_silence(F, R, m):
    for name, call in _calls(F, R, lambda t: t.clone().requires_grad_()).items():
        if name in ("restore_rows", "expert_ffn", "route_top_k"):
            continue  # they have a gradient, or nothing to derive
        with pytest.raises(m.MoeEpArgError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(m.MoeEpArgError, match="GPU tensor"):
            call()


def test_differentiable_calls_refuse_what_has_no_gradient(F, R, m):
    x = torch.zeros(2, 32, dtype=BF, requires_grad=True)
    w1, w2 = torch.zeros(64, 32, dtype=BF), torch.zeros(32, 32, dtype=BF)
    with pytest.raises(m.MoeEpArgError, match="new tensor"):
        F.expert_ffn(x, w1, w2, out=torch.zeros(2, 32, dtype=BF))
    logits = torch.zeros(2, 4, requires_grad=True)
    with pytest.raises(m.MoeEpArgError, match="new tensors"):
        R.route_top_k(logits, 2, ids=torch.zeros(2, 2, dtype=torch.int32))
    follows = torch.zeros(2, 32, dtype=BF, requires_grad=True) * 1
    for call in (lambda: F.expert_product(x.detach(), w2, out=follows), lambda: F.expert_ffn(x.detach(), w1, w2, out=follows),
                 lambda: R.route_top_k(logits.detach(), 2, weights=torch.zeros(2, 2, requires_grad=True) * 1)):
        with pytest.raises(m.MoeEpArgError, match="no gradient"):
            call()


def test_result_type_and_output_agree(F, m):
    q, s = torch.zeros(2, 32, dtype=torch.float8_e4m3fn), torch.zeros(2, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(m.MoeEpArgError, match="dtype"):
        F.restore_rows(q, s, dtype=BF, out=torch.zeros(2, 32))
    with pytest.raises(m.MoeEpArgError, match="dtype"):
        F.expert_matmul_mxfp4(torch.zeros(2, 32, dtype=BF), q, s, dtype=BF, out=torch.zeros(2, 2))
