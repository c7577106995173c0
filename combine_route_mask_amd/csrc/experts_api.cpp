// Host side of the expert layer's entry points in moe_ep.h: every check runs
// before the first launch, so a call either launches all its kernels or none.
// No exception leaves an entry point.
#include <climits>
#include <cmath>
#include <string>

#include "experts_internal.h"

using namespace moe_ep;

namespace {

constexpr int64_t kMaxRowBytes = 1 << 24;

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int bad(const char *msg) { return fail(MOE_EP_ERR_INVALID_ARG, msg); }

// A required device pointer: present and aligned.
bool good(const void *p, uintptr_t a) { return p && aligned(p, a); }

template <typename F>
int guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return MOE_EP_ERR_HIP; // no memory for a message
    }
}

// Launches; an error that an earlier call of the thread left behind is not
// this call's.
template <typename F>
int launched(const char *what, F launch)
{
    (void)hipGetLastError();
    const hipError_t e = launch();
    if (e == hipErrorInvalidConfiguration) // the launchers' own limit
        return fail(MOE_EP_ERR_CAPACITY, std::string(what) + " needs more workgroups than a launch holds");
    if (e != hipSuccess)
        return fail(MOE_EP_ERR_HIP, std::string(what) + " launch failed: " + hipGetErrorString(e));
    return ok();
}

// Bytes of one element, 0 for an unknown type.
int64_t item_bytes(int32_t row_type)
{
    return row_type == MOE_EP_BF16_ROWS ? 2 : row_type == MOE_EP_FP32_ROWS ? 4 : 0;
}

int check_slots(int32_t ranks, int32_t slots, int32_t top_k)
{
    if (ranks < 1 || ranks > MOE_EP_MAX_RANKS)
        return bad("ranks must be in [1, 64]");
    if (slots < 0)
        return bad("slots may not be negative");
    if (top_k < 1 || top_k > MOE_EP_MAX_TOP_K)
        return bad("top_k must be in [1, 64]");
    if ((int64_t)ranks * slots * top_k > INT32_MAX)
        return fail(MOE_EP_ERR_CAPACITY, "ranks * slots * top_k exceeds 2^31 - 1 pairs");
    return MOE_EP_OK;
}

int check_sort_shape(int32_t ranks, int32_t slots, int32_t top_k, int32_t experts_per_rank)
{
    if (int rc = check_slots(ranks, slots, top_k))
        return rc;
    if (experts_per_rank < 1 || (int64_t)ranks * experts_per_rank > MOE_EP_MAX_SORT_EXPERTS)
        return bad("ranks * experts_per_rank must be in [1, 4096]");
    return MOE_EP_OK;
}

int64_t sort_workspace(int32_t ranks, int32_t slots, int32_t top_k, int32_t epr)
{
    if (sort_is_direct(ranks, slots, top_k, ranks * epr))
        return 0;
    // a total for each rank and a place for each pair
    if (sort_is_planned(slots, top_k, epr))
        return 4 * ((int64_t)ranks + (int64_t)ranks * slots * top_k);
    // one count for each (expert, tile of its rank)
    return 4 * (int64_t)ranks * epr * sort_tiles(slots, top_k);
}

// A plane [R][S][row] whose ranks lie rank_stride bytes apart.
bool good_plane(const void *p, int64_t stride, int32_t ranks, int32_t slots, int64_t row, uintptr_t a)
{
    if (ranks == 0 || slots == 0)
        return true;
    return good(p, a) && (ranks == 1 || (stride >= 0 && stride % (int64_t)a == 0 && stride >= slots * row));
}

} // namespace

extern "C" {

int64_t moe_ep_expert_sort_workspace_bytes(int32_t ranks, int32_t slots, int32_t top_k,
                                           int32_t experts_per_rank)
{
    int64_t n = -1;
    guarded([&] {
        if (int rc = check_sort_shape(ranks, slots, top_k, experts_per_rank))
            return rc;
        n = sort_workspace(ranks, slots, top_k, experts_per_rank);
        return ok();
    });
    return n;
}

int moe_ep_expert_sort(const moe_ep_sort_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_sort_args &a = *args;
        if (int rc = check_sort_shape(a.ranks, a.slots, a.top_k, a.experts_per_rank))
            return rc;
        if (a.ranks < 64 && a.masked_ranks >> a.ranks)
            return bad("masked_ranks has bits set at or above ranks");
        if (a.capacity < 0 || a.capacity > INT32_MAX)
            return fail(MOE_EP_ERR_CAPACITY, "capacity must be in [0, 2^31 - 1]");
        if (a.quantize != 0 && a.quantize != 1)
            return bad("quantize must be 0 or 1");
        if (a.row_bytes < 16 || a.row_bytes % 16 || a.row_bytes > kMaxRowBytes)
            return bad("row_bytes must be a multiple of 16 in [16, 2^24]");
        if (a.quantize) {
            const int64_t item = item_bytes(a.row_type);
            if (!item)
                return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
            if (a.row_bytes % (16 * item))
                return bad("a quantised row must be a multiple of 16 elements");
            if (a.scales || a.scale_row_bytes)
                return bad("quantised rows take no scale rows");
        }
        if (a.scale_row_bytes < 0 || a.scale_row_bytes > kMaxRowBytes)
            return bad("scale_row_bytes must be in [0, 2^24]");
        if (!good_plane(a.ids, a.ids_rank_stride, a.ranks, a.slots, 4ll * a.top_k, 4))
            return bad("ids must be a 4-byte aligned device pointer with rank strides of whole planes");
        if (!good_plane(a.rows, a.rows_rank_stride, a.ranks, a.slots, a.row_bytes, 16))
            return bad("rows must be a 16-byte aligned device pointer with rank strides of whole planes");
        if (a.scale_row_bytes &&
            !good_plane(a.scales, a.scales_rank_stride, a.ranks, a.slots, a.scale_row_bytes, 1))
            return bad("scales must be a device pointer with rank strides of whole planes");
        if (!good(a.offsets, 4) || !good(a.counts, 4))
            return bad("offsets and counts must be 4-byte aligned device pointers");
        if (a.slots && !good(a.position, 4))
            return bad("position must be a 4-byte aligned device pointer");
        if (a.capacity && !good(a.out_rows, 16))
            return bad("out_rows must be a 16-byte aligned device pointer");
        if (a.capacity && a.quantize && !good(a.out_scales, 4))
            return bad("out_scales must be a 4-byte aligned device pointer");
        if (a.capacity && a.scale_row_bytes && !a.out_scales)
            return bad("out_scales is NULL");
        const int64_t need = sort_workspace(a.ranks, a.slots, a.top_k, a.experts_per_rank);
        if (need && !good(a.workspace, 16))
            return bad("workspace must be a 16-byte aligned device pointer");
        if (a.workspace_bytes < need)
            return fail(MOE_EP_ERR_CAPACITY, "workspace is below moe_ep_expert_sort_workspace_bytes()");
        return launched("expert sort", [&] { return launch_expert_sort(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_expert_unsort(const moe_ep_unsort_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_unsort_args &a = *args;
        if (int rc = check_slots(a.ranks, a.slots, a.top_k))
            return rc;
        const int64_t item = item_bytes(a.row_type);
        if (!item)
            return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
        if (a.hidden_size < 1 || (a.hidden_size * item) % 16 || a.hidden_size * item > kMaxRowBytes)
            return bad("a row must be a multiple of 16 bytes in [16, 2^24]");
        if (a.num_rows < 0 || a.num_rows > INT32_MAX)
            return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
        if (a.keep_empty != 0 && a.keep_empty != 1)
            return bad("keep_empty must be 0 or 1");
        if (a.slots == 0)
            return ok();
        if (!good(a.position, 4))
            return bad("position must be a 4-byte aligned device pointer");
        if (a.num_rows && !good(a.rows, 16))
            return bad("rows must be a 16-byte aligned device pointer");
        if (a.weights && !good_plane(a.weights, a.weights_rank_stride, a.ranks, a.slots, 4ll * a.top_k, 4))
            return bad("weights must be 4-byte aligned with rank strides of whole planes");
        if (!good_plane(a.out, a.out_rank_stride, a.ranks, a.slots, a.hidden_size * item, 16))
            return bad("out must be a 16-byte aligned device pointer with rank strides of whole planes");
        return launched("expert unsort", [&] { return launch_expert_unsort(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_expert_unsort_backward(const moe_ep_unsort_grad_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_unsort_grad_args &a = *args;
        if (int rc = check_slots(a.ranks, a.slots, a.top_k))
            return rc;
        const int64_t item = item_bytes(a.row_type);
        if (!item)
            return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
        if (a.hidden_size < 1 || (a.hidden_size * item) % 16 || a.hidden_size * item > kMaxRowBytes)
            return bad("a row must be a multiple of 16 bytes in [16, 2^24]");
        if (a.num_rows < 0 || a.num_rows > INT32_MAX)
            return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
        if (a.reserved != 0)
            return bad("reserved must be 0");
        if (a.slots == 0 || (!a.grad_rows && !a.grad_weights))
            return ok();
        if (!good(a.position, 4))
            return bad("position must be a 4-byte aligned device pointer");
        if (!good_plane(a.grad_out, a.grad_out_rank_stride, a.ranks, a.slots, a.hidden_size * item, 16))
            return bad("grad_out must be a 16-byte aligned device pointer with rank strides of whole planes");
        if (a.grad_weights && a.num_rows && !good(a.rows, 16))
            return bad("grad_weights needs rows, a 16-byte aligned device pointer");
        if (a.weights && !good_plane(a.weights, a.weights_rank_stride, a.ranks, a.slots, 4ll * a.top_k, 4))
            return bad("weights must be 4-byte aligned with rank strides of whole planes");
        if (!aligned(a.grad_rows, 16) || !aligned(a.grad_weights, 4))
            return bad("grad_rows must be 16-byte, grad_weights 4-byte aligned");
        return launched("expert unsort backward",
                        [&] { return launch_expert_unsort_backward(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_expert_matmul(const moe_ep_matmul_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_matmul_args &a = *args;
        if (a.num_experts < 1 || a.num_experts > MOE_EP_MAX_SORT_EXPERTS)
            return bad("num_experts must be in [1, 4096]");
        if (!a.offsets && a.num_experts != 1)
            return bad("a product over several experts needs offsets");
        if (a.num_rows < 0 || a.num_rows > INT32_MAX)
            return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
        if (a.n < 1)
            return bad("n must be >= 1");
        if (a.k < 16 || a.k % 16 || a.k > 131056)
            return bad("k must be a multiple of 16 in [16, 131056]");
        if (!item_bytes(a.out_type))
            return fail(MOE_EP_ERR_UNSUPPORTED, "unknown out_type");
        if (a.num_rows == 0)
            return ok();
        if (!good(a.x, 16) || !good(a.w, 16))
            return bad("x and w must be 16-byte aligned device pointers");
        if (!good(a.x_scales, 4) || !good(a.w_scales, 4) || (a.offsets && !aligned(a.offsets, 4)))
            return bad("x_scales, w_scales and offsets must be 4-byte aligned device pointers");
        if (!good(a.out, (uintptr_t)item_bytes(a.out_type)))
            return bad("out must be an aligned device pointer");
        return launched("expert matmul", [&] { return launch_expert_matmul(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_silu_mul_quantize(const moe_ep_silu_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_silu_args &a = *args;
        if (!item_bytes(a.row_type))
            return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
        if (a.inter_size < 16 || a.inter_size % 16 || a.inter_size > 32768)
            return bad("inter_size must be a multiple of 16 in [16, 32768]");
        if (a.num_rows < 0 || a.num_rows > INT32_MAX)
            return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
        if (a.num_rows == 0)
            return ok();
        if (!good(a.x, 16) || !good(a.out, 16))
            return bad("x and out must be 16-byte aligned device pointers");
        if (!good(a.out_scales, 4) || (a.num_valid && !aligned(a.num_valid, 4)))
            return bad("out_scales and num_valid must be 4-byte aligned device pointers");
        return launched("silu_mul_quantize", [&] { return launch_silu_mul_quantize(a, static_cast<hipStream_t>(stream)); });
    });
}

int moe_ep_add_rms_norm(const moe_ep_norm_args *args, void *stream)
{
    return guarded([&]() -> int {
        if (!args)
            return bad("args is NULL");
        const moe_ep_norm_args &a = *args;
        if (!item_bytes(a.row_type))
            return fail(MOE_EP_ERR_UNSUPPORTED, "unknown row_type");
        int block;
        switch (a.format) {
        case MOE_EP_NORM_INT8: block = 16; break;
        case MOE_EP_NORM_MXFP8: block = 32; break;
        case MOE_EP_NORM_DEEPSEEK_FP8: block = 128; break;
        default: return fail(MOE_EP_ERR_UNSUPPORTED, "unknown format");
        }
        if (a.hidden_size < block || a.hidden_size % block || a.hidden_size > 32768)
            return bad("hidden_size must be a multiple of the format's block (int8 16, MXFP8 32, "
                       "DeepSeekFp8 128), at most 32768");
        if (!(a.eps >= 0.0f) || std::isinf(a.eps))
            return bad("eps must be finite and >= 0");
        if (a.num_rows < 0 || a.num_rows > INT32_MAX)
            return fail(MOE_EP_ERR_CAPACITY, "num_rows must be in [0, 2^31 - 1]");
        if (a.num_rows == 0)
            return ok();
        if (!good(a.x, 16) || !aligned(a.residual, 16) || !good(a.weight, 16) || !aligned(a.residual_out, 16))
            return bad("x, residual, weight and residual_out must be 16-byte aligned device pointers");
        if (!good(a.out, 16))
            return bad("out must be a 16-byte aligned device pointer");
        if (!good(a.scales, a.format == MOE_EP_NORM_MXFP8 ? 1 : 4))
            return bad("scales must be an aligned device pointer");
        return launched("add_rms_norm", [&] { return launch_add_rms_norm(a, static_cast<hipStream_t>(stream)); });
    });
}

} // extern "C"
