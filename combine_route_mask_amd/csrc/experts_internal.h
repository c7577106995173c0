// Shared by the host entry points and the gfx950 kernels of the expert
// layer: the launchers, each taking an argument block that the entry point
// has checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_ep.h"

namespace moe_ep {

// A sort's ids are cut into tiles of this many pairs (whole slots).
constexpr int kSortTilePairs = 1024;
// Largest sort whose every workgroup ranks its slot against all pairs itself.
constexpr int64_t kSortDirectPairs = 2048;
constexpr int kSortDirectExperts = 1024;

__host__ __device__ inline int sort_tile_slots(int top_k)
{
    return kSortTilePairs / top_k; // top_k <= 64
}

inline int64_t sort_tiles(int64_t slots, int top_k)
{
    const int64_t ts = sort_tile_slots(top_k);
    return slots ? (slots + ts - 1) / ts : 1; // an empty one still writes counts and offsets
}

inline bool sort_is_direct(int ranks, int64_t slots, int top_k, int experts)
{
    return (int64_t)ranks * slots * top_k <= kSortDirectPairs && experts <= kSortDirectExperts;
}

// Sorts whose ranks' pairs fit one workgroup each (sort_plan_kernel).
constexpr int kSortPlanPairs = 8192;
constexpr int kSortPlanExperts = 512;

inline bool sort_is_planned(int64_t slots, int top_k, int experts_per_rank)
{
    return slots > 0 && slots * top_k <= kSortPlanPairs && experts_per_rank <= kSortPlanExperts;
}

hipError_t launch_expert_sort(const moe_ep_sort_args &a, hipStream_t s);
hipError_t launch_expert_unsort(const moe_ep_unsort_args &a, hipStream_t s);
hipError_t launch_expert_unsort_backward(const moe_ep_unsort_grad_args &a, hipStream_t s);
hipError_t launch_expert_matmul(const moe_ep_matmul_args &a, hipStream_t s);
hipError_t launch_silu_mul_quantize(const moe_ep_silu_args &a, hipStream_t s);
hipError_t launch_add_rms_norm(const moe_ep_norm_args &a, hipStream_t s);

} // namespace moe_ep
