// gfx950 kernels of the 8-bit activation checkpoints: rows to MXFP8 codes and
// scales, and back.  Every byte passes once; HBM bounds them.
#include "ffn_internal.h"
#include "rows.h"

namespace moe_ep {
namespace {

constexpr int kThreads = 256;

// Eight elements a thread, four threads a block of 32.
template <typename T>
__global__ __launch_bounds__(kThreads) void checkpoint_kernel(moe_ep_checkpoint_args a, int64_t units)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < units; i += (int64_t)gridDim.x * kThreads) {
        float f[8];
        load_elements<T, 8>(static_cast<const uint8_t *>(a.rows) + i * 8 * RowType<T>::kBytes, f);
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max(top, magnitude(f[e]));
        top = max4(top); // units are whole blocks: the four lanes run together
        uint8_t scale;
        const u32x2 codes = mx_codes(f, top, scale);
        __builtin_nontemporal_store(codes, reinterpret_cast<u32x2 *>(a.codes + 8 * i));
        if ((threadIdx.x & 3) == 0)
            a.scales[i >> 2] = scale;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void restore_kernel(moe_ep_checkpoint_args a, int64_t units)
{
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < units; i += (int64_t)gridDim.x * kThreads) {
        float f[8];
        mx_values(load8_nt(a.codes + 8 * i), e8m0_value(a.scales[i >> 2]), f);
        uint8_t *out = static_cast<uint8_t *>(a.rows) + i * 8 * RowType<T>::kBytes;
        constexpr int N = RowType<T>::kPer;
#pragma unroll
        for (int v = 0; v < 8 / N; ++v)
            store16_nt(out + 16 * v, RowType<T>::pack(f + v * N));
    }
}

inline dim3 units_grid(int64_t units)
{
    const int64_t n = (units + kThreads - 1) / kThreads, cap = 1 << 20;
    return dim3((unsigned)(n < cap ? n : cap));
}

} // namespace

hipError_t launch_checkpoint_rows(const moe_ep_checkpoint_args &a, hipStream_t s)
{
    const int64_t units = a.num_rows * (a.hidden_size / 8);
    if (a.row_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL(checkpoint_kernel<Bf16>, units_grid(units), dim3(kThreads), 0, s, a, units);
    else
        hipLaunchKernelGGL(checkpoint_kernel<Fp32>, units_grid(units), dim3(kThreads), 0, s, a, units);
    return hipGetLastError();
}

hipError_t launch_restore_rows(const moe_ep_checkpoint_args &a, hipStream_t s)
{
    const int64_t units = a.num_rows * (a.hidden_size / 8);
    if (a.row_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL(restore_kernel<Bf16>, units_grid(units), dim3(kThreads), 0, s, a, units);
    else
        hipLaunchKernelGGL(restore_kernel<Fp32>, units_grid(units), dim3(kThreads), 0, s, a, units);
    return hipGetLastError();
}

} // namespace moe_ep
