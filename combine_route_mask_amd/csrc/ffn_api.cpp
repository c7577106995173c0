// Host side of the trainable expert layer's entry points in moe_ep.h: every
// check runs before the first launch, so a call either launches all its
// kernels or none.  No exception leaves an entry point.
#include <climits>
#include <cmath>

#include "api_checks.h"
#include "ffn_internal.h"

using namespace moe_ep;

namespace {

constexpr int32_t kMaxWidth = 131072; // elements of a row of a product

bool width(int32_t n) { return n >= 8 && n % 8 == 0 && n <= kMaxWidth; }

// What every product over experts asks of its rows and offsets.
int check_rows(int64_t num_rows, int32_t num_experts, const int32_t *offsets)
{
    if (num_experts < 1 || num_experts > MOE_EP_MAX_SORT_EXPERTS)
        return bad("num_experts must be in [1, 4096]");
    if (!offsets && num_experts != 1)
        return bad("a product over several experts needs offsets");
    if (!aligned(offsets, 4))
        return bad("offsets must be a 4-byte aligned device pointer");
    if (num_rows < 0 || num_rows > INT32_MAX)
        return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
    return MOE_EP_OK;
}

int check_route(int64_t tokens, int32_t num_experts, int32_t top_k, int32_t renormalize, int32_t row_type, float scale,
                int32_t reserved)
{
    if (num_experts < 1 || num_experts > MOE_EP_MAX_ROUTED_EXPERTS)
        return bad("num_experts must be in [1, 4096]");
    if (top_k < 1 || top_k > MOE_EP_MAX_TOP_K || top_k > num_experts)
        return bad("top_k must be in [1, 64] and at most num_experts");
    if (renormalize != 0 && renormalize != 1)
        return bad("renormalize must be 0 or 1");
    if (!item_bytes(row_type))
        return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
    if (!std::isfinite(scale))
        return bad("scale must be finite");
    if (reserved != 0)
        return bad("reserved must be 0");
    if (tokens < 0 || tokens > INT32_MAX)
        return fail(MOE_EP_ERR_CAPACITY, "tokens must be in [0, 2^31 - 1]");
    return MOE_EP_OK;
}

// What a gated block keeps of its first product; `needed`: of an input.
int check_saved(int32_t save, int32_t inter_size, const void *pre, const void *pre_scales, bool needed)
{
    if (save != MOE_EP_SAVE_HALF && save != MOE_EP_SAVE_MXFP8 && (needed || save != MOE_EP_SAVE_NONE))
        return fail(MOE_EP_ERR_UNSUPPORTED, "unknown save");
    if (save == MOE_EP_SAVE_MXFP8 && inter_size % 32)
        return bad("an MXFP8 checkpoint needs an inter_size that is a multiple of 32");
    if (save != MOE_EP_SAVE_NONE && !good(pre, 16))
        return bad("pre must be a 16-byte aligned device pointer");
    if (save != MOE_EP_SAVE_NONE && !pre_scales)
        return bad("pre_scales is NULL");
    return MOE_EP_OK;
}

int check_checkpoint(const moe_ep_checkpoint_args &a)
{
    if (!item_bytes(a.row_type))
        return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
    if (a.hidden_size < 32 || a.hidden_size % 32 || a.hidden_size > 1 << 20)
        return bad("hidden_size must be a multiple of 32 in [32, 2^20]");
    if (a.num_rows < 0 || a.num_rows > INT32_MAX)
        return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
    if (a.num_rows && (!good(a.rows, 16) || !good(a.codes, 16) || !a.scales))
        return bad("rows and codes must be 16-byte aligned device pointers, scales a device pointer");
    return MOE_EP_OK;
}

} // namespace

extern "C" {

int moe_ep_route_top_k(const moe_ep_route_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_route_args &a = *args;
        if (int rc = check_route(a.tokens, a.num_experts, a.top_k, a.renormalize, a.row_type, a.scale, a.reserved))
            return rc;
        if (a.tokens == 0)
            return ok();
        if (!good(a.logits, (uintptr_t)item_bytes(a.row_type)) || !good(a.ids, 4) || !good(a.weights, 4))
            return bad("logits, ids and weights must be aligned device pointers");
        return launched("route_top_k", [&] { return launch_route_top_k(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_route_top_k_backward(const moe_ep_route_grad_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_route_grad_args &a = *args;
        if (int rc = check_route(a.tokens, a.num_experts, a.top_k, a.renormalize, a.row_type, a.scale, a.reserved))
            return rc;
        if (a.tokens == 0)
            return ok();
        const uintptr_t item = (uintptr_t)item_bytes(a.row_type);
        if (!good(a.logits, item) || !good(a.ids, 4) || !good(a.grad_weights, 4) || !good(a.grad_logits, item))
            return bad("logits, ids, grad_weights and grad_logits must be aligned device pointers");
        return launched("route_top_k backward",
                        [&] { return launch_route_top_k_backward(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_checkpoint_rows(const moe_ep_checkpoint_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        if (int rc = check_checkpoint(*args))
            return rc;
        if (args->num_rows == 0)
            return ok();
        return launched("checkpoint_rows", [&] { return launch_checkpoint_rows(*args, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_restore_rows(const moe_ep_checkpoint_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        if (int rc = check_checkpoint(*args))
            return rc;
        if (args->num_rows == 0)
            return ok();
        return launched("restore_rows", [&] { return launch_restore_rows(*args, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_expert_product(const moe_ep_product_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_product_args &a = *args;
        if (int rc = check_rows(a.num_rows, a.num_experts, a.offsets))
            return rc;
        if (!width(a.n) || !width(a.k))
            return bad("n and k must be multiples of 8 in [8, 131072]");
        if ((a.transposed != 0 && a.transposed != 1) || (a.zero_rest != 0 && a.zero_rest != 1) || a.reserved != 0)
            return bad("transposed and zero_rest must be 0 or 1, reserved 0");
        if (a.num_rows == 0)
            return ok();
        if (!good(a.x, 16) || !good(a.w, 16) || !good(a.out, 16))
            return bad("x, w and out must be 16-byte aligned device pointers");
        return launched("expert product", [&] { return launch_expert_product(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_gated_product(const moe_ep_gated_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_gated_args &a = *args;
        if (int rc = check_rows(a.num_rows, a.num_experts, a.offsets))
            return rc;
        if (!width(a.inter_size) || a.inter_size > kMaxWidth / 2 || !width(a.k))
            return bad("inter_size and k must be multiples of 8, at most 65536 and 131072");
        if (a.num_rows == 0)
            return ok();
        if (int rc = check_saved(a.save, a.inter_size, a.pre, a.pre_scales, false))
            return rc;
        if (!good(a.x, 16) || !good(a.w, 16) || !good(a.out, 16))
            return bad("x, w and out must be 16-byte aligned device pointers");
        return launched("gated product", [&] { return launch_gated_product(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_gated_product_backward(const moe_ep_gated_grad_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_gated_grad_args &a = *args;
        if (int rc = check_rows(a.num_rows, a.num_experts, a.offsets))
            return rc;
        if (!width(a.inter_size) || a.inter_size > kMaxWidth / 2 || !width(a.n))
            return bad("inter_size and n must be multiples of 8, at most 65536 and 131072");
        if (a.num_rows == 0)
            return ok();
        if (int rc = check_saved(a.save, a.inter_size, a.pre, a.pre_scales, true))
            return rc;
        if (!good(a.grad_out, 16) || !good(a.w, 16) || !good(a.grad_pre, 16) || !aligned(a.out, 16))
            return bad("grad_out, w, grad_pre and out must be 16-byte aligned device pointers");
        return launched("gated product backward",
                        [&] { return launch_gated_product_backward(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_product_weight_grad(const moe_ep_weight_grad_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_weight_grad_args &a = *args;
        if (int rc = check_rows(a.num_rows, a.num_experts, a.offsets))
            return rc;
        if (!width(a.n) || !width(a.k))
            return bad("n and k must be multiples of 8 in [8, 131072]");
        if (a.reserved != 0)
            return bad("reserved must be 0");
        if (!good(a.grad_w, 16) || (a.num_rows && (!good(a.grad_out, 16) || !good(a.x, 16))))
            return bad("grad_out, x and grad_w must be 16-byte aligned device pointers");
        return launched("product weight grad",
                        [&] { return launch_product_weight_grad(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_four_bit_product(const moe_ep_four_bit_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_four_bit_args &a = *args;
        if (int rc = check_rows(a.num_rows, a.num_experts, a.offsets))
            return rc;
        if (a.gated != 0 && a.gated != 1)
            return bad("gated must be 0 or 1");
        if (a.n < 1 || a.n >= 1 << 30 || (a.gated && a.n % 2))
            return bad("n must be in [1, 2^30), even for a gated product");
        if (a.k < 32 || a.k % 32 || a.k > kMaxWidth)
            return bad("k must be a multiple of 32 in [32, 131072]");
        if (!item_bytes(a.out_type))
            return fail(MOE_EP_ERR_UNSUPPORTED, "unknown out_type");
        if (a.reserved != 0)
            return bad("reserved must be 0");
        if (a.num_rows == 0)
            return ok();
        if (!good(a.x, 16) || !good(a.w, 16) || !a.w_scales)
            return bad("x and w must be 16-byte aligned device pointers, w_scales a device pointer");
        if (!good(a.out, (uintptr_t)item_bytes(a.out_type)))
            return bad("out must be an aligned device pointer");
        return launched("four-bit product", [&] { return launch_four_bit_product(a, static_cast<hipStream_t>(stream)); });
    });
}

} // extern "C"
