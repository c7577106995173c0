"""The expert layer refuses bad calls before any launch, through the C ABI
(argument blocks with made-up addresses; nothing is launched) and in the
binding (CPU tensors, shapes, types)."""
import os
import re

import pytest
import torch

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def X():
    from combine_route_mask_amd import experts
    return experts


@pytest.fixture(scope="module")
def m():
    from combine_route_mask_amd import moe_ep
    return moe_ep


def _fields(struct):
    """(name, kind) of a struct's members, from the header's text."""
    hdr = open(os.path.join(ROOT, "include", "moe_ep.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (struct, struct), hdr, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    out = []
    for decl in body.split(";"):
        if decl.strip():
            kind = "P" if "*" in decl else {"int64_t": "q", "uint64_t": "Q", "int32_t": "i", "float": "f"}[decl.split()[0]]
            out.append((re.findall(r"\w+", decl)[-1], kind))
    return out


BLOCKS = {"moe_ep_sort_args": "_SORT", "moe_ep_unsort_args": "_UNSORT", "moe_ep_unsort_grad_args": "_UNSORT_GRAD",
          "moe_ep_matmul_args": "_MATMUL", "moe_ep_silu_args": "_SILU", "moe_ep_norm_args": "_NORM"}


@pytest.mark.parametrize("struct", BLOCKS)
def test_argument_blocks_match_the_header(X, struct):
    assert "@" + "".join(k for _, k in _fields(struct)) == getattr(X, BLOCKS[struct]).format


A = 1 << 20  # an aligned address that nothing reads
GOOD = {
    "moe_ep_expert_sort": ("moe_ep_sort_args", dict(
        ids=A, ids_rank_stride=512, rows=A, rows_rank_stride=4096, row_bytes=128, scales=0, scales_rank_stride=0,
        scale_row_bytes=0, out_rows=A, out_scales=0, position=A, offsets=A, counts=A, workspace=A,
        workspace_bytes=1 << 16, capacity=100, ranks=2, slots=32, top_k=4, experts_per_rank=8, quantize=0,
        row_type=0, masked_ranks=2)),
    "moe_ep_expert_unsort": ("moe_ep_unsort_args", dict(
        position=A, rows=A, weights=A, weights_rank_stride=512, out=A, out_rank_stride=4096, num_rows=100, ranks=2,
        slots=32, top_k=4, hidden_size=64, row_type=0, keep_empty=0)),
    "moe_ep_expert_unsort_backward": ("moe_ep_unsort_grad_args", dict(
        position=A, grad_out=A, grad_out_rank_stride=4096, rows=A, weights=A, weights_rank_stride=512, grad_rows=A,
        grad_weights=A, num_rows=100, ranks=2, slots=32, top_k=4, hidden_size=64, row_type=0, reserved=0)),
    "moe_ep_expert_matmul": ("moe_ep_matmul_args", dict(
        x=A, x_scales=A, w=A, w_scales=A, offsets=A, out=A, num_rows=10, num_experts=4, n=32, k=64, out_type=0)),
    "moe_ep_silu_mul_quantize": ("moe_ep_silu_args", dict(
        x=A, num_valid=A, out=A, out_scales=A, num_rows=10, inter_size=32, row_type=0)),
    "moe_ep_add_rms_norm": ("moe_ep_norm_args", dict(
        x=A, residual=A, weight=A, residual_out=A, out=A, scales=A, num_rows=10, hidden_size=128, row_type=0,
        format=1, eps=1e-6)),
}

ARG, UNSUP, CAP = -1, -2, -4
BAD = [
    ("moe_ep_expert_sort", dict(ranks=0), ARG), ("moe_ep_expert_sort", dict(ranks=65), ARG),
    ("moe_ep_expert_sort", dict(slots=-1), ARG), ("moe_ep_expert_sort", dict(top_k=0), ARG),
    ("moe_ep_expert_sort", dict(top_k=65), ARG), ("moe_ep_expert_sort", dict(experts_per_rank=0), ARG),
    ("moe_ep_expert_sort", dict(experts_per_rank=2049), ARG),
    ("moe_ep_expert_sort", dict(masked_ranks=4), ARG), ("moe_ep_expert_sort", dict(slots=1 << 30), CAP), ("moe_ep_expert_sort", dict(capacity=-1), CAP),
    ("moe_ep_expert_sort", dict(capacity=1 << 31), CAP), ("moe_ep_expert_sort", dict(row_bytes=0), ARG),
    ("moe_ep_expert_sort", dict(row_bytes=24), ARG), ("moe_ep_expert_sort", dict(row_bytes=(1 << 24) + 16), ARG),
    ("moe_ep_expert_sort", dict(ids=0), ARG), ("moe_ep_expert_sort", dict(ids=A + 2), ARG),
    ("moe_ep_expert_sort", dict(ids_rank_stride=508), ARG), ("moe_ep_expert_sort", dict(rows=A + 8), ARG),
    ("moe_ep_expert_sort", dict(rows_rank_stride=4080), ARG), ("moe_ep_expert_sort", dict(rows_rank_stride=-4096), ARG),
    ("moe_ep_expert_sort", dict(rows_rank_stride=4104), ARG), ("moe_ep_expert_sort", dict(scale_row_bytes=8), ARG),
    ("moe_ep_expert_sort", dict(scale_row_bytes=-8), ARG),
    ("moe_ep_expert_sort", dict(scale_row_bytes=8, scales=A, scales_rank_stride=256), ARG),  # no out_scales
    ("moe_ep_expert_sort", dict(scale_row_bytes=8, scales=A, scales_rank_stride=200, out_scales=A), ARG),
    ("moe_ep_expert_sort", dict(out_rows=0), ARG), ("moe_ep_expert_sort", dict(out_rows=A + 4), ARG),
    ("moe_ep_expert_sort", dict(position=0), ARG), ("moe_ep_expert_sort", dict(offsets=0), ARG),
    ("moe_ep_expert_sort", dict(counts=A + 1), ARG), ("moe_ep_expert_sort", dict(quantize=2), ARG),
    ("moe_ep_expert_sort", dict(quantize=1), ARG),  # no out_scales
    ("moe_ep_expert_sort", dict(quantize=1, out_scales=A, row_type=2), UNSUP),
    ("moe_ep_expert_sort", dict(quantize=1, out_scales=A, row_bytes=112, rows_rank_stride=4096), ARG),
    ("moe_ep_expert_sort", dict(slots=1000, ids_rank_stride=1 << 20, rows_rank_stride=1 << 20, workspace=0), ARG),
    ("moe_ep_expert_sort", dict(slots=1000, ids_rank_stride=1 << 20, rows_rank_stride=1 << 20, workspace_bytes=8), CAP),
    ("moe_ep_expert_unsort", dict(ranks=0), ARG), ("moe_ep_expert_unsort", dict(top_k=65), ARG),
    ("moe_ep_expert_unsort", dict(hidden_size=4), ARG), ("moe_ep_expert_unsort", dict(hidden_size=0), ARG),
    ("moe_ep_expert_unsort", dict(row_type=7), UNSUP), ("moe_ep_expert_unsort", dict(keep_empty=2), ARG),
    ("moe_ep_expert_unsort", dict(position=0), ARG), ("moe_ep_expert_unsort", dict(rows=0), ARG),
    ("moe_ep_expert_unsort", dict(weights=A + 2), ARG), ("moe_ep_expert_unsort", dict(weights_rank_stride=0), ARG),
    ("moe_ep_expert_unsort", dict(out=0), ARG), ("moe_ep_expert_unsort", dict(out_rank_stride=4080), ARG),
    ("moe_ep_expert_unsort", dict(num_rows=1 << 31), CAP), ("moe_ep_expert_unsort", dict(num_rows=-1), CAP),
    ("moe_ep_expert_unsort_backward", dict(grad_out=0), ARG), ("moe_ep_expert_unsort_backward", dict(rows=0), ARG),
    ("moe_ep_expert_unsort_backward", dict(grad_rows=A + 8), ARG),
    ("moe_ep_expert_unsort_backward", dict(grad_weights=A + 2), ARG),
    ("moe_ep_expert_unsort_backward", dict(reserved=1), ARG), ("moe_ep_expert_unsort_backward", dict(row_type=3), UNSUP),
    ("moe_ep_expert_unsort_backward", dict(position=A + 2), ARG),
    ("moe_ep_expert_matmul", dict(num_experts=0), ARG), ("moe_ep_expert_matmul", dict(num_experts=4097), ARG),
    ("moe_ep_expert_matmul", dict(offsets=0), ARG), ("moe_ep_expert_matmul", dict(offsets=A + 2), ARG),
    ("moe_ep_expert_matmul", dict(n=0), ARG), ("moe_ep_expert_matmul", dict(k=8), ARG),
    ("moe_ep_expert_matmul", dict(k=72), ARG), ("moe_ep_expert_matmul", dict(k=131072), ARG),
    ("moe_ep_expert_matmul", dict(out_type=2), UNSUP), ("moe_ep_expert_matmul", dict(x=A + 8), ARG),
    ("moe_ep_expert_matmul", dict(w=0), ARG), ("moe_ep_expert_matmul", dict(x_scales=0), ARG),
    ("moe_ep_expert_matmul", dict(out=A + 1), ARG), ("moe_ep_expert_matmul", dict(num_rows=-1), CAP),
    ("moe_ep_silu_mul_quantize", dict(inter_size=24), ARG), ("moe_ep_silu_mul_quantize", dict(inter_size=32784), ARG),
    ("moe_ep_silu_mul_quantize", dict(x=0), ARG), ("moe_ep_silu_mul_quantize", dict(out_scales=0), ARG),
    ("moe_ep_silu_mul_quantize", dict(row_type=2), UNSUP), ("moe_ep_silu_mul_quantize", dict(num_valid=A + 2), ARG),
    ("moe_ep_add_rms_norm", dict(format=3), UNSUP), ("moe_ep_add_rms_norm", dict(hidden_size=48), ARG),
    ("moe_ep_add_rms_norm", dict(format=2, hidden_size=192), ARG),
    ("moe_ep_add_rms_norm", dict(format=0, hidden_size=8), ARG),
    ("moe_ep_add_rms_norm", dict(hidden_size=32768 + 32), ARG), ("moe_ep_add_rms_norm", dict(eps=-1.0), ARG),
    ("moe_ep_add_rms_norm", dict(eps=float("nan")), ARG), ("moe_ep_add_rms_norm", dict(eps=float("inf")), ARG),
    ("moe_ep_add_rms_norm", dict(weight=0), ARG), ("moe_ep_add_rms_norm", dict(residual=A + 2), ARG),
    ("moe_ep_add_rms_norm", dict(scales=0), ARG), ("moe_ep_add_rms_norm", dict(format=2, scales=A + 2), ARG),
    ("moe_ep_add_rms_norm", dict(row_type=-1), UNSUP), ("moe_ep_add_rms_norm", dict(out=A + 8), ARG),
]


@pytest.mark.parametrize("name,change,code", BAD, ids=lambda v: str(v))
def test_refused_blocks(X, m, name, change, code):
    struct, good = GOOD[name]
    values = dict(good, **change)
    fields = _fields(struct)
    assert set(values) == {n for n, _ in fields}
    block = getattr(X, BLOCKS[struct]).pack(*(values[n] for n, _ in fields))
    assert getattr(m.lib, name)(block, None) == code
    assert m.lib.moe_ep_last_error().decode() != ""


@pytest.mark.parametrize("name", GOOD)
def test_no_block(m, name):
    assert getattr(m.lib, name)(None, None) == ARG


def test_nothing_to_do_needs_no_gpu(X, m):
    """Calls over no slot or row return at once."""
    for name, change in (("moe_ep_expert_unsort", dict(slots=0)), ("moe_ep_expert_unsort_backward", dict(slots=0)),
                         ("moe_ep_expert_unsort_backward", dict(grad_rows=0, grad_weights=0)),
                         ("moe_ep_expert_matmul", dict(num_rows=0)), ("moe_ep_silu_mul_quantize", dict(num_rows=0)),
                         ("moe_ep_add_rms_norm", dict(num_rows=0))):
        struct, good = GOOD[name]
        values = dict(good, **change)
        block = getattr(X, BLOCKS[struct]).pack(*(values[n] for n, _ in _fields(struct)))
        assert getattr(m.lib, name)(block, None) == 0


def test_sort_workspace(X, m):
    assert X.expert_sort_workspace_bytes(1, 256, 8, 64) == 0          # one launch
    assert X.expert_sort_workspace_bytes(1, 257, 8, 64) == 4 * (1 + 257 * 8)  # one workgroup a rank
    assert X.expert_sort_workspace_bytes(8, 1024, 8, 32) == 4 * (8 + 8 * 1024 * 8)
    assert X.expert_sort_workspace_bytes(1, 1025, 8, 64) == 4 * 64 * 9        # tiles of 128 slots
    assert X.expert_sort_workspace_bytes(1, 257, 8, 513) == 4 * 513 * 3
    assert X.expert_sort_workspace_bytes(64, 32768, 8, 4) == 4 * 256 * 256
    for bad in ((0, 1, 1, 1), (1, -1, 1, 1), (1, 1, 65, 1), (1, 1, 1, 4097), (1, 1, 1, 1 << 32), (64, 1 << 30, 8, 4)):
        with pytest.raises(m.MoeEpArgError):
            X.expert_sort_workspace_bytes(*bad)


def test_cpu_tensors_are_refused(X, m):
    ids, rows = torch.zeros((1, 2, 2), dtype=torch.int32), torch.zeros((1, 2, 16), dtype=torch.bfloat16)
    q, s = torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)
    for call in (lambda: X.expert_sort(ids, rows, 4), lambda: X.expert_unsort(ids, rows[0]),
                 lambda: X.expert_sort_backward(ids, rows[0]),
                 lambda: X.expert_unsort_backward(ids, rows, rows[0]), lambda: X.expert_matmul(q, s, q, s),
                 lambda: X.silu_mul_quantize(rows[0]), lambda: X.add_rms_norm(rows[0], rows[0], rows[0, 0]),
                 lambda: X.add_rms_norm(rows[0], None, rows[0, 0], format="fp4")):
        with pytest.raises(m.MoeEpArgError):
            call()


def test_gradients_are_not_dropped_in_silence(X, m):
    """Scale rows have no gradient, next to differentiable rows either; neither have the gradients' own calls."""
    ids = torch.zeros((1, 2, 2), dtype=torch.int32)
    rows = torch.zeros((1, 2, 16), requires_grad=True)
    scales = torch.zeros((1, 2, 4), requires_grad=True)
    flat, w = torch.zeros((2, 16), requires_grad=True), torch.zeros((1, 2, 2), requires_grad=True)
    plain, plain_w = flat.detach(), w.detach()
    for call in (lambda: X.expert_sort(ids, rows, 4, scales=scales),
                 lambda: X.expert_sort(ids, rows.detach(), 4, scales=scales),
                 lambda: X.expert_sort_backward(ids, flat),
                 lambda: X.expert_unsort_backward(ids, rows, plain, plain_w),
                 lambda: X.expert_unsort_backward(ids, rows.detach(), flat, plain_w),
                 lambda: X.expert_unsort_backward(ids, rows.detach(), plain, w)):
        with pytest.raises(m.MoeEpArgError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(m.MoeEpArgError, match="GPU tensor"):
            call()


def test_product_type_and_output_agree(X, m):
    """A result type that is not the given output's is refused."""
    q, s = torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)
    for given, dtype in ((torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float16)):
        with pytest.raises(m.MoeEpArgError, match="dtype"):
            X.expert_matmul(q, s, q, s, out=torch.zeros((2, 2), dtype=given), dtype=dtype)
    for dtype in (None, torch.float32):
        with pytest.raises(m.MoeEpArgError, match="GPU tensor"):
            X.expert_matmul(q, s, q, s, out=torch.zeros((2, 2)), dtype=dtype)


def test_outputs_with_a_gradient_are_refused(X, m):
    """Written in place, an output that autograd follows would keep the history of what it no longer holds."""
    ids = torch.zeros((1, 2, 2), dtype=torch.int32)
    rows, flat = torch.zeros((1, 2, 16)), torch.zeros((2, 16))
    q, s = torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)
    wt = torch.zeros(16)
    grad = lambda *shape: (torch.zeros(shape, requires_grad=True) * 1)  # noqa: E731
    for call in (lambda: X.expert_sort(ids, rows, 4, out=grad(4, 16)),
                 lambda: X.expert_sort(ids, rows, 4, quantize=True, out_scales=grad(4)),
                 lambda: X.expert_sort_backward(ids, flat, out=grad(1, 2, 16)),
                 lambda: X.expert_unsort(ids, flat, out=grad(1, 2, 16)),
                 lambda: X.expert_unsort_backward(ids, rows, flat, grad_rows=grad(2, 16)),
                 lambda: X.expert_matmul(q, s, q, s, out=grad(2, 2)),
                 lambda: X.silu_mul_quantize(torch.zeros((2, 32)), out_scales=grad(2)),
                 lambda: X.add_rms_norm(flat, None, wt, format="int8", out_scales=grad(2)),
                 lambda: X.add_rms_norm(flat, flat, wt, format="int8", residual_out=grad(2, 16))):
        with pytest.raises(m.MoeEpArgError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(m.MoeEpArgError, match="GPU tensor"):
            call()
