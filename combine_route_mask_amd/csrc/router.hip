// gfx950 kernels of the router: the largest logits of each token with their
// softmax weights, and the gradient of the weights for the logits.  One wave a
// token, its logits in LDS.
#include "ffn_internal.h"
#include "rows.h"

namespace moe_ep {
namespace {

template <typename T>
__device__ __forceinline__ float logit(const void *base, int64_t i)
{
    if (RowType<T>::kBytes == 2)
        return bf16_to_f32(static_cast<const uint16_t *>(base)[i]);
    return static_cast<const float *>(base)[i];
}

template <typename T>
__device__ __forceinline__ void store_logit(void *base, int64_t i, float x)
{
    if (RowType<T>::kBytes == 2)
        static_cast<uint16_t *>(base)[i] = (uint16_t)f32_to_bf16_rne(x);
    else
        static_cast<float *>(base)[i] = x;
}

__device__ __forceinline__ float nan_value() { return __uint_as_float(0x7FC00000u); }

template <typename T>
__global__ __launch_bounds__(64) void route_kernel(moe_ep_route_args a)
{
    extern __shared__ float row[];
    const int E = a.num_experts, lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        bool nan = false;
        for (int i = lane; i < E; i += 64) {
            const float x = logit<T>(a.logits, t * E + i);
            nan |= x != x;
            row[i] = x;
        }
        nan = __any(nan);
        __syncthreads();
        float value = -INFINITY, top = 0.0f; // of the place that is this lane's
        int id = E;
        float last = INFINITY;
        int last_id = -1;
        for (int j = 0; j < a.top_k; ++j) {
            // the largest behind (last, last_id)
            float best = -INFINITY;
            int at = E;
            for (int i = lane; i < E; i += 64) {
                const float x = row[i];
                if ((x < last || (x == last && i > last_id)) && x > best) {
                    best = x;
                    at = i;
                }
            }
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const float ob = __shfl_xor(best, m);
                const int oa = __shfl_xor(at, m);
                if (ob > best || (ob == best && oa < at)) {
                    best = ob;
                    at = oa;
                }
            }
            if (at == E)
                break;
            if (j == 0)
                top = best;
            if (lane == j) {
                value = best;
                id = at;
            }
            last = best;
            last_id = at;
        }
        const float e = id < E ? expf(value - top) : 0.0f;
        float total = e;
        if (!a.renormalize) {
            total = 0.0f;
            for (int i = lane; i < E; i += 64)
                total += expf(row[i] - top);
        }
        total = wave_sum(total);
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = id;
            a.weights[t * a.top_k + lane] = id == E ? 0.0f : nan ? nan_value() : a.scale * (e / total);
        }
        __syncthreads();
    }
}

template <typename T>
__global__ __launch_bounds__(64) void route_backward_kernel(moe_ep_route_grad_args a)
{
    extern __shared__ float place[]; // g of each expert, and behind them whether it has a place
    const int E = a.num_experts, lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        int id = E;
        float g = 0.0f;
        if (lane < a.top_k) {
            id = a.ids[t * a.top_k + lane];
            g = a.grad_weights[t * a.top_k + lane];
        }
        const bool held = id >= 0 && id < E;
        const float mine = held ? logit<T>(a.logits, t * E + id) : -INFINITY;
        float top = mine;
        if (!a.renormalize)
            for (int i = lane; i < E; i += 64)
                top = fmaxf(top, logit<T>(a.logits, t * E + i));
#pragma unroll
        for (int m = 1; m < 64; m <<= 1)
            top = fmaxf(top, __shfl_xor(top, m));
        if (top == -INFINITY)
            top = 0.0f;
        const float e = held ? expf(mine - top) : 0.0f;
        float total = e;
        if (!a.renormalize) {
            total = 0.0f;
            for (int i = lane; i < E; i += 64)
                total += expf(logit<T>(a.logits, t * E + i) - top);
        }
        total = wave_sum(total);
        const float by = total != 0.0f ? 1.0f / total : 0.0f;
        const float mean = wave_sum(held ? e * by * g : 0.0f);
        for (int i = lane; i < E; i += 64)
            place[i] = 0.0f;
        __syncthreads();
        if (held)
            place[id] = a.renormalize ? a.scale * (e * by) * (g - mean) : g;
        __syncthreads();
        for (int i = lane; i < E; i += 64) {
            float d = place[i];
            if (!a.renormalize)
                d = a.scale * (expf(logit<T>(a.logits, t * E + i) - top) * by) * (d - mean);
            store_logit<T>(a.grad_logits, t * E + i, d);
        }
        __syncthreads();
    }
}

inline dim3 tokens_grid(int64_t tokens)
{
    const int64_t cap = 1 << 20;
    return dim3((unsigned)(tokens < cap ? tokens : cap));
}

} // namespace

hipError_t launch_route_top_k(const moe_ep_route_args &a, hipStream_t s)
{
    if (a.row_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL(route_kernel<Bf16>, tokens_grid(a.tokens), dim3(64), 4 * a.num_experts, s, a);
    else
        hipLaunchKernelGGL(route_kernel<Fp32>, tokens_grid(a.tokens), dim3(64), 4 * a.num_experts, s, a);
    return hipGetLastError();
}

hipError_t launch_route_top_k_backward(const moe_ep_route_grad_args &a, hipStream_t s)
{
    if (a.row_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL(route_backward_kernel<Bf16>, tokens_grid(a.tokens), dim3(64), 4 * a.num_experts, s, a);
    else
        hipLaunchKernelGGL(route_backward_kernel<Fp32>, tokens_grid(a.tokens), dim3(64), 4 * a.num_experts, s, a);
    return hipGetLastError();
}

} // namespace moe_ep
