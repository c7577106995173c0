// gfx950 kernels of the expert layer's row-wise operators with an 8-bit
// output: the root-mean-square norm with the residual's addition, and the
// gated activation.  One workgroup holds a whole row in registers between
// the reduction and the codes, so every input is read once and HBM bounds
// large calls; one launch, whose latency bounds small ones.
#include "experts_internal.h"
#include "rows.h"

namespace moe_ep {
namespace {

constexpr int kUnit = 8; // elements of a thread's vector

template <typename T>
__device__ __forceinline__ void load_unit(const void *base, int64_t i, float *f)
{
    load_elements<T, kUnit>(static_cast<const uint8_t *>(base) + i * kUnit * RowType<T>::kBytes, f);
}

template <typename T>
__device__ __forceinline__ void store_unit(void *base, int64_t i, const float *f)
{
    constexpr int N = RowType<T>::kPer;
#pragma unroll
    for (int v = 0; v < kUnit / N; ++v)
        store16_nt(static_cast<uint8_t *>(base) + i * kUnit * RowType<T>::kBytes + 16 * v, RowType<T>::pack(f + v * N));
}

__device__ __forceinline__ void store_codes(void *base, int64_t i, u32x2 codes)
{
    __builtin_nontemporal_store(codes, reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(base) + i * kUnit));
}

// Sum / largest magnitude over the workgroup, in an order the shape fixes.
template <int BS>
__device__ __forceinline__ float block_sum(float x, float *red)
{
    x = wave_sum(x);
    if (BS > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < BS / 64; ++w)
            x += red[w];
    }
    return x;
}

template <int BS>
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t *red)
{
    x = wave_max(x);
    if (BS > 64) {
        if ((threadIdx.x & 63) == 0)
            red[threadIdx.x >> 6] = x;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < BS / 64; ++w)
            x = max(x, red[w]);
    }
    return x;
}

__device__ __forceinline__ u32x2 int8_codes(const Int8Row &rule, const float *f)
{
    return u32x2{rule.codes4(f), rule.codes4(f + 4)};
}

// Rows r, r + grid, ...: thread t holds the 8-element units t, t + BS, ...
template <typename T, int FMT, int BS, int VPT>
__global__ __launch_bounds__(BS) void add_rms_norm_kernel(moe_ep_norm_args a)
{
    __shared__ float sums[BS / 64];
    __shared__ uint32_t tops[BS / 64];
    const int H = a.hidden_size, units = H / kUnit;
    constexpr int NV = kUnit / RowType<T>::kPer;
    u32x4 weight[VPT][NV]; // read once, before the rows
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            weight[u][v] = u32x4{0, 0, 0, 0};
            if ((int)threadIdx.x + u * BS < units)
                weight[u][v] = reinterpret_cast<const u32x4 *>(a.weight)[(threadIdx.x + u * BS) * NV + v];
        }
    for (int64_t row = blockIdx.x; row < a.num_rows; row += gridDim.x) {
        const int64_t first = row * units;
        float f[VPT][kUnit];
        float square = 0.0f;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = threadIdx.x + u * BS;
#pragma unroll
            for (int e = 0; e < kUnit; ++e)
                f[u][e] = 0.0f;
            if (i < units) {
                load_unit<T>(a.x, first + i, f[u]);
                if (a.residual) {
                    float g[kUnit];
                    load_unit<T>(a.residual, first + i, g);
#pragma unroll
                    for (int e = 0; e < kUnit; ++e)
                        f[u][e] += g[e];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = threadIdx.x + u * BS;
#pragma unroll
            for (int e = 0; e < kUnit; ++e)
                square = fmaf(f[u][e], f[u][e], square);
            if (i < units && a.residual_out)
                store_unit<T>(a.residual_out, first + i, f[u]);
        }
        // a row with a NaN, an infinity or squares past fp32 has no norm: its
        // codes and scales are NaN throughout
        const float mean = block_sum<BS>(square, sums) / (float)H;
        const float r = mean < __uint_as_float(kInfinity) ? 1.0f / sqrtf(mean + a.eps) : __uint_as_float(0x7FC00000u);
        uint32_t top[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = threadIdx.x + u * BS;
            float w[kUnit];
#pragma unroll
            for (int v = 0; v < NV; ++v)
                RowType<T>::unpack(weight[u][v], w + v * RowType<T>::kPer);
            top[u] = 0;
#pragma unroll
            for (int e = 0; e < kUnit; ++e) {
                f[u][e] = (f[u][e] * r) * w[e];
                if (i < units)
                    top[u] = max(top[u], magnitude(f[u][e]));
            }
        }
        if (FMT == MOE_EP_NORM_INT8) {
            uint32_t t = 0;
#pragma unroll
            for (int u = 0; u < VPT; ++u)
                t = max(t, top[u]);
            const Int8Row rule(block_max<BS>(t, tops));
#pragma unroll
            for (int u = 0; u < VPT; ++u)
                if (threadIdx.x + u * BS < units)
                    store_codes(a.out, first + threadIdx.x + u * BS, int8_codes(rule, f[u]));
            if (threadIdx.x == 0)
                static_cast<float *>(a.scales)[row] = rule.scale;
        } else {
            constexpr int kLog = FMT == MOE_EP_NORM_MXFP8 ? 2 : 4; // lanes of a block
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                const int i = threadIdx.x + u * BS;
                const uint32_t t = FMT == MOE_EP_NORM_MXFP8 ? max4(top[u]) : max16(top[u]);
                if (i >= units)
                    continue;
                const bool head = (threadIdx.x & ((1 << kLog) - 1)) == 0;
                u32x2 codes;
                if (FMT == MOE_EP_NORM_MXFP8) {
                    const int e = mx_exponent(t);
                    codes = e4m3_codes(f[u], 1.0f, __uint_as_float((uint32_t)(127 - e) << 23));
                    if (t >= kInfinity)
                        codes = kNanCodes;
                    if (head)
                        static_cast<uint8_t *>(a.scales)[(first + i) >> kLog] =
                            t >= kInfinity ? 0xFF : (uint8_t)(e + 127);
                } else {
                    const float m = __uint_as_float(t);
                    const float up = m < 0x1p-100f ? 0x1p+64f : 1.0f;
                    codes = e4m3_codes(f[u], up, t == 0 ? 0.0f : 448.0f / (m * up));
                    if (t >= kInfinity)
                        codes = kNanCodes;
                    if (head)
                        static_cast<float *>(a.scales)[(first + i) >> kLog] =
                            t >= kInfinity ? __uint_as_float(0x7FC00000u) : m / 448.0f;
                }
                store_codes(a.out, first + i, codes);
            }
        }
        if (BS > 64)
            __syncthreads(); // before the next row's sums
    }
}

template <typename T, int BS, int VPT>
__global__ __launch_bounds__(BS) void silu_mul_quantize_kernel(moe_ep_silu_args a)
{
    __shared__ uint32_t tops[BS / 64];
    const int units = a.inter_size / kUnit;
    const int64_t rows = a.num_valid ? min((int64_t)*a.num_valid, a.num_rows) : a.num_rows;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        float f[VPT][kUnit], g[VPT][kUnit];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
            const int i = threadIdx.x + u * BS;
            if (i < units) {
                load_unit<T>(a.x, row * 2 * units + i, f[u]);
                load_unit<T>(a.x, row * 2 * units + units + i, g[u]);
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < VPT; ++u)
            if (threadIdx.x + u * BS < units)
#pragma unroll
                for (int e = 0; e < kUnit; ++e) {
                    // x / (1 + exp(-x)); exp overflows to infinity far below 0, where the limit is -0
                    f[u][e] = f[u][e] / (1.0f + __expf(-f[u][e])) * g[u][e];
                    top = max(top, magnitude(f[u][e]));
                }
        const Int8Row rule(block_max<BS>(top, tops));
#pragma unroll
        for (int u = 0; u < VPT; ++u)
            if (threadIdx.x + u * BS < units)
                store_codes(a.out, row * units + threadIdx.x + u * BS, int8_codes(rule, f[u]));
        if (threadIdx.x == 0)
            a.out_scales[row] = rule.scale;
        if (BS > 64)
            __syncthreads(); // before the next row's maxima
    }
}

inline dim3 rows_grid(int64_t rows)
{
    const int64_t cap = 1 << 20;
    return dim3((unsigned)(rows < cap ? rows : cap));
}

template <typename T, int FMT, int BS, int VPT>
hipError_t norm_launch(const moe_ep_norm_args &a, hipStream_t s)
{
    hipLaunchKernelGGL((add_rms_norm_kernel<T, FMT, BS, VPT>), rows_grid(a.num_rows), dim3(BS), 0, s, a);
    return hipGetLastError();
}

// Two units a thread keep more waves on a row than four: 32768 rows of 7168
// bf16 to DeepSeekFp8 take 266 us (6.2 TB/s) with 512 threads of two units, 277
// with 256 of four, 325 with 128 of seven, 296 with 1024 of one; to int8 262 /
// 273 / 318 / 301, to MXFP8 266.  A call of one row takes 8 us in every shape.
// One workgroup a row: 2048 workgroups that loop over the rows take 285 us for
// each format.
template <typename T, int FMT>
hipError_t norm_shape(const moe_ep_norm_args &a, hipStream_t s)
{
    const int units = a.hidden_size / kUnit;
    if (units <= 64)
        return norm_launch<T, FMT, 64, 1>(a, s);
    if (units <= 128)
        return norm_launch<T, FMT, 128, 1>(a, s);
    if (units <= 256)
        return norm_launch<T, FMT, 256, 1>(a, s);
    if (units <= 512)
        return norm_launch<T, FMT, 256, 2>(a, s);
    if (units <= 1024)
        return norm_launch<T, FMT, 512, 2>(a, s);
    if (units <= 2048)
        return norm_launch<T, FMT, 512, 4>(a, s);
    return norm_launch<T, FMT, 1024, 4>(a, s);
}

template <typename T>
hipError_t norm_format(const moe_ep_norm_args &a, hipStream_t s)
{
    if (a.format == MOE_EP_NORM_INT8)
        return norm_shape<T, MOE_EP_NORM_INT8>(a, s);
    if (a.format == MOE_EP_NORM_MXFP8)
        return norm_shape<T, MOE_EP_NORM_MXFP8>(a, s);
    return norm_shape<T, MOE_EP_NORM_DEEPSEEK_FP8>(a, s);
}

template <typename T, int BS, int VPT>
hipError_t silu_launch(const moe_ep_silu_args &a, hipStream_t s)
{
    hipLaunchKernelGGL((silu_mul_quantize_kernel<T, BS, VPT>), rows_grid(a.num_rows), dim3(BS), 0, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t silu_shape(const moe_ep_silu_args &a, hipStream_t s)
{
    const int units = a.inter_size / kUnit;
    if (units <= 64)
        return silu_launch<T, 64, 1>(a, s);
    if (units <= 128)
        return silu_launch<T, 128, 1>(a, s);
    if (units <= 256)
        return silu_launch<T, 256, 1>(a, s);
    if (units <= 512)
        return silu_launch<T, 256, 2>(a, s);
    if (units <= 1024)
        return silu_launch<T, 512, 2>(a, s);
    if (units <= 2048)
        return silu_launch<T, 512, 4>(a, s);
    return silu_launch<T, 1024, 4>(a, s);
}

} // namespace

hipError_t launch_add_rms_norm(const moe_ep_norm_args &a, hipStream_t s)
{
    return a.row_type == MOE_EP_BF16_ROWS ? norm_format<Bf16>(a, s) : norm_format<Fp32>(a, s);
}

hipError_t launch_silu_mul_quantize(const moe_ep_silu_args &a, hipStream_t s)
{
    return a.row_type == MOE_EP_BF16_ROWS ? silu_shape<Bf16>(a, s) : silu_shape<Fp32>(a, s);
}

} // namespace moe_ep
