// gfx950 kernel of the product of bf16 rows with 4-bit weights (e2m1 codes, an
// e8m0 scale for 32): codes become bf16 by the hardware's scaled conversion
// (exact), products and sums run on the matrix cores in fp32.
#include "ffn_internal.h"
#include "rows.h"
#include "tiles.h"

namespace moe_ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bf16x8 four_bit_values(uint32_t codes, float scale)
{
    bf16x8 v = {};
#if defined(__HIP_DEVICE_COMPILE__)
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    v = bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#endif
    return v;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

template <typename T>
__device__ __forceinline__ void store_value(void *out, int64_t i, float x)
{
    if (RowType<T>::kBytes == 2)
        static_cast<uint16_t *>(out)[i] = (uint16_t)f32_to_bf16_rne(x);
    else
        static_cast<float *>(out)[i] = x;
}

// A wave takes 16 channels (gated: 16 gate and their up channels) of one
// expert and all its rows, 16 at a time, 128 of k a step: a lane holds the
// codes of 32 consecutive k of a channel, one scale.
template <typename T, bool GATED>
__global__ __launch_bounds__(64) void four_bit_kernel(moe_ep_four_bit_args a, int ntiles)
{
    const int e = (int)(blockIdx.x / (unsigned)ntiles), tile = (int)(blockIdx.x % (unsigned)ntiles);
    int lo, hi;
    expert_rows(a, e, lo, hi);
    constexpr int F = GATED ? 2 : 1;
    const int lane = threadIdx.x, l16 = lane & 15, l4 = lane >> 4, N = a.n / F;
    const int channel = min(tile * 16 + l16, N - 1);
    for (int64_t m0 = lo; m0 < hi; m0 += 16) {
        const int64_t row = min(m0 + l16, (int64_t)hi - 1);
        f32x4 acc[F] = {};
        for (int k = 32 * l4; k - 32 * l4 < a.k; k += 128) {
            const bool in = k < a.k;
            bf16x8 x[4] = {};
            u32x4 q[F] = {};
            float scale[F];
#pragma unroll
            for (int f = 0; f < F; ++f)
                scale[f] = 1.0f;
            if (in) {
                const bf16x8 *xp = reinterpret_cast<const bf16x8 *>(static_cast<const uint16_t *>(a.x) + row * a.k + k);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = xp[j];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const int64_t w = (int64_t)e * a.n + f * N + channel;
                    q[f] = *reinterpret_cast<const u32x4 *>(a.w + (w * a.k + k) / 2);
                    scale[f] = e8m0_value(a.w_scales[(w * a.k + k) / 32]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(four_bit_values(q[f][j], scale[f]), x[j], acc[f], 0, 0, 0);
        }
        if (m0 + l16 < hi)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = tile * 16 + 4 * l4 + i;
                if (n < N)
                    store_value<T>(a.out, (m0 + l16) * N + n, GATED ? silu(acc[0][i]) * acc[F - 1][i] : acc[0][i]);
            }
    }
}

template <typename T>
hipError_t four_bit_launch(const moe_ep_four_bit_args &a, hipStream_t s)
{
    const int ntiles = channel_tiles(a.gated ? a.n / 2 : a.n, 16);
    const int64_t grid = (int64_t)ntiles * a.num_experts;
    if (grid > INT32_MAX)
        return hipErrorInvalidConfiguration;
    if (a.gated)
        hipLaunchKernelGGL((four_bit_kernel<T, true>), dim3((unsigned)grid), dim3(64), 0, s, a, ntiles);
    else
        hipLaunchKernelGGL((four_bit_kernel<T, false>), dim3((unsigned)grid), dim3(64), 0, s, a, ntiles);
    return hipGetLastError();
}

} // namespace

hipError_t launch_four_bit_product(const moe_ep_four_bit_args &a, hipStream_t s)
{
    return a.out_type == MOE_EP_BF16_ROWS ? four_bit_launch<Bf16>(a, s) : four_bit_launch<Fp32>(a, s);
}

} // namespace moe_ep
