// The launchers of the trainable expert layer, each taking an argument block
// that the entry point has checked.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_ep.h"

namespace moe_ep {

hipError_t launch_route_top_k(const moe_ep_route_args &a, hipStream_t s);
hipError_t launch_route_top_k_backward(const moe_ep_route_grad_args &a, hipStream_t s);
hipError_t launch_checkpoint_rows(const moe_ep_checkpoint_args &a, hipStream_t s);
hipError_t launch_restore_rows(const moe_ep_checkpoint_args &a, hipStream_t s);
hipError_t launch_expert_product(const moe_ep_product_args &a, hipStream_t s);
hipError_t launch_gated_product(const moe_ep_gated_args &a, hipStream_t s);
hipError_t launch_gated_product_backward(const moe_ep_gated_grad_args &a, hipStream_t s);
hipError_t launch_product_weight_grad(const moe_ep_weight_grad_args &a, hipStream_t s);
hipError_t launch_four_bit_product(const moe_ep_four_bit_args &a, hipStream_t s);

} // namespace moe_ep
