// gfx950 kernels of the bf16 products over experts: rows times weights in
// either order of the weights' axes, with the gated block's epilogues, and the
// weights' gradient.  Products on the matrix cores, sums in fp32.
//
// v_mfma_f32_16x16x32_bf16: lane l holds 8 elements of row l % 16 at
// k = 8 * (l / 16) of either matrix; of the result, element i is left row
// 4 * (l / 16) + i and right row l % 16.  The left matrix is the channels',
// the right one the rows'.
#include "ffn_internal.h"
#include "rows.h"
#include "tiles.h"

namespace moe_ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Epilogue { kStore, kGated, kGatedBackward };

struct Job {
    const uint16_t *x, *w;
    const int32_t *offsets;
    uint16_t *out;      // product, activation
    void *pre;          // what the gated block saves or reads
    uint8_t *pre_scales;
    uint16_t *grad_pre;
    int64_t num_rows;
    int num_experts, n, k, save;
};

constexpr int kEdge = 64, kDepth = 32, kPitch = kDepth + 8;

// [kEdge] rows of 32 elements into LDS: of rows that lie one after another
// (ACROSS = false: element (i, k) at i * stride + k) or k after k (true).
template <bool ACROSS, typename ROW>
__device__ __forceinline__ void stage(uint16_t (*to)[kPitch], const uint16_t *from, int64_t stride, int k, int depth,
                                      ROW row)
{
    const int t = threadIdx.x;
    u32x4 v = {};
    if (!ACROSS) {
        const int i = t / 4, c = t % 4 * 8;
        const int64_t r = row(i);
        if (r >= 0 && k + c < depth)
            v = *reinterpret_cast<const u32x4 *>(from + r * stride + k + c);
        *reinterpret_cast<u32x4 *>(&to[i][c]) = v;
    } else {
        const int i = t / 8, c = t % 8 * 8;
        const int64_t r = row(c);
        if (k + i < depth && r >= 0)
            v = *reinterpret_cast<const u32x4 *>(from + (k + i) * stride + r);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            to[c + e][i] = (uint16_t)(v[e / 2] >> (e % 2 * 16));
    }
}

__device__ __forceinline__ void multiply(uint16_t (*a)[kPitch], uint16_t (*b)[kPitch], f32x4 (*acc)[2])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, l4 = lane >> 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bf16x8 u = *reinterpret_cast<const bf16x8 *>(&a[(wave & 1) * 32 + i * 16 + l16][8 * l4]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const bf16x8 v = *reinterpret_cast<const bf16x8 *>(&b[(wave >> 1) * 32 + j * 16 + l16][8 * l4]);
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, v, acc[i][j], 0, 0, 0);
        }
    }
}

// The tile's sums, row m of the right matrix at [m].
__device__ __forceinline__ void put(float (*tile)[kEdge + 4], f32x4 (*acc)[2])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, l4 = lane >> 4;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<f32x4 *>(&tile[(wave >> 1) * 32 + j * 16 + l16][(wave & 1) * 32 + i * 16 + 4 * l4]) = acc[i][j];
}

__device__ __forceinline__ void store8(uint16_t *to, const float *f)
{
    *reinterpret_cast<u32x4 *>(to) = RowType<Bf16>::pack(f);
}

template <int EPI, bool ACROSS>
__global__ __launch_bounds__(256) void product_kernel(Job a, int ntiles)
{
    __shared__ __align__(16) uint16_t aw[kEdge][kPitch], bx[kEdge][kPitch];
    __shared__ __align__(16) float sums[kEdge][kEdge + 4];
    constexpr int WIDE = EPI == kGated ? kEdge / 2 : kEdge; // channels of the output in a tile
    const int N = EPI == kGated ? a.n / 2 : a.n;
    const TileFinder<kEdge, kEdge> find(a, ntiles);
    for (int slot = (int)(blockIdx.x >> 3);; slot += (int)(gridDim.x >> 3)) {
        const Tile t = find.tile(a, slot);
        if (t.expert < 0)
            return;
        const int n0 = t.n * WIDE;
        f32x4 acc[2][2] = {};
        const uint16_t *w = a.w + (int64_t)t.expert * a.n * a.k;
        for (int k = 0; k < a.k; k += kDepth) {
            __syncthreads();
            stage<ACROSS>(aw, w, ACROSS ? a.n : a.k, k, a.k, [&](int i) -> int64_t {
                const int n = n0 + i % WIDE;
                return n < N ? n + i / WIDE * N : -1;
            });
            stage<false>(bx, a.x, a.k, k, a.k, [&](int i) { return t.first + i < t.last ? t.first + i : -1; });
            __syncthreads();
            multiply(aw, bx, acc);
        }
        put(sums, acc);
        __syncthreads();
        const int m = threadIdx.x / 4;
        const int64_t row = t.first + m;
        for (int c = threadIdx.x % 4 * 8; c < WIDE; c += 32) {
            const int n = n0 + c;
            const bool in = row < t.last && n < N;
            const float *f = &sums[m][c];
            if (EPI == kStore) {
                if (in)
                    store8(a.out + row * N + n, f);
            } else if (EPI == kGated) {
                const float *g = f + WIDE;
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = f[i] / (1.0f + __expf(-f[i])) * g[i];
                if (in)
                    store8(a.out + row * N + n, y);
                if (a.save == MOE_EP_SAVE_BF16 && in) {
                    store8(static_cast<uint16_t *>(a.pre) + row * a.n + n, f);
                    store8(static_cast<uint16_t *>(a.pre) + row * a.n + N + n, g);
                } else if (a.save == MOE_EP_SAVE_MXFP8) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float *p = h ? g : f;
                        uint32_t top = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            top = max(top, magnitude(p[i]));
                        top = max4(top);
                        uint8_t scale;
                        const u32x2 codes = mx_codes(p, top, scale);
                        const int64_t at = row * a.n + h * N + n;
                        if (in) {
                            *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.pre) + at) = codes;
                            if (threadIdx.x % 4 == 0)
                                a.pre_scales[at / 32] = scale;
                        }
                    }
                }
            } else if (in) {
                float g[8], u[8], y[8], dg[8], du[8];
                const int64_t at = row * 2 * N + n;
                if (a.save == MOE_EP_SAVE_BF16) {
                    load_elements<Bf16, 8>(reinterpret_cast<const uint8_t *>(static_cast<uint16_t *>(a.pre) + at), g);
                    load_elements<Bf16, 8>(reinterpret_cast<const uint8_t *>(static_cast<uint16_t *>(a.pre) + at + N), u);
                } else {
                    const uint8_t *p = static_cast<uint8_t *>(a.pre);
                    mx_values(load8_nt(p + at), e8m0_value(a.pre_scales[at / 32]), g);
                    mx_values(load8_nt(p + at + N), e8m0_value(a.pre_scales[(at + N) / 32]), u);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = 1.0f / (1.0f + __expf(-g[i]));
                    y[i] = g[i] * s * u[i];
                    du[i] = f[i] * g[i] * s;
                    dg[i] = f[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
                }
                store8(a.grad_pre + at, dg);
                store8(a.grad_pre + at + N, du);
                if (a.out)
                    store8(a.out + row * N + n, y);
            }
        }
        __syncthreads();
    }
}

// Rows from the last expert's last on become zeros.
__global__ __launch_bounds__(256) void zero_rest_kernel(Job a)
{
    const int64_t last = a.offsets ? min(max((int64_t)a.offsets[a.num_experts], (int64_t)0), a.num_rows) : a.num_rows;
    const int64_t units = a.num_rows * (a.n / 8);
    for (int64_t i = last * (a.n / 8) + (int64_t)blockIdx.x * 256 + threadIdx.x; i < units; i += (int64_t)gridDim.x * 256)
        reinterpret_cast<u32x4 *>(a.out)[i] = u32x4{0, 0, 0, 0};
}

__global__ __launch_bounds__(256) void weight_grad_kernel(moe_ep_weight_grad_args a, int ntiles, int ktiles)
{
    __shared__ __align__(16) uint16_t ax[kEdge][kPitch], bg[kEdge][kPitch];
    __shared__ __align__(16) float sums[kEdge][kEdge + 4];
    const int e = (int)(blockIdx.x / (unsigned)(ntiles * ktiles)), in = (int)(blockIdx.x % (unsigned)(ntiles * ktiles));
    const int n0 = in / ktiles * kEdge, k0 = in % ktiles * kEdge;
    int lo, hi;
    expert_rows(a, e, lo, hi);
    f32x4 acc[2][2] = {};
    for (int m = lo; m < hi; m += kDepth) {
        __syncthreads();
        stage<true>(ax, static_cast<const uint16_t *>(a.x), a.k, m, hi,
                    [&](int i) -> int64_t { return k0 + i < a.k ? k0 + i : -1; });
        stage<true>(bg, static_cast<const uint16_t *>(a.grad_out), a.n, m, hi,
                    [&](int i) -> int64_t { return n0 + i < a.n ? n0 + i : -1; });
        __syncthreads();
        multiply(ax, bg, acc);
    }
    put(sums, acc);
    __syncthreads();
    const int n = n0 + threadIdx.x / 4;
    for (int c = threadIdx.x % 4 * 8; c < kEdge; c += 32)
        if (n < a.n && k0 + c < a.k)
            store8(static_cast<uint16_t *>(a.grad_w) + ((int64_t)e * a.n + n) * a.k + k0 + c, &sums[threadIdx.x / 4][c]);
}

template <int EPI, bool ACROSS>
hipError_t product_launch(const Job &a, int wide, hipStream_t s)
{
    const int64_t ntiles = channel_tiles(EPI == kGated ? a.n / 2 : a.n, wide);
    const int64_t tiles = most_tiles(a, kEdge) * ntiles;
    if (tiles > INT32_MAX - 4096)
        return hipErrorInvalidConfiguration;
    const int64_t run = (tiles + 7) / 8, resident = 32 * 4;
    hipLaunchKernelGGL((product_kernel<EPI, ACROSS>), dim3((unsigned)(8 * (run < resident ? run : resident))), dim3(256), 0,
                       s, a, (int)ntiles);
    return hipGetLastError();
}

} // namespace

hipError_t launch_expert_product(const moe_ep_product_args &a, hipStream_t s)
{
    Job j = {};
    j.x = static_cast<const uint16_t *>(a.x);
    j.w = static_cast<const uint16_t *>(a.w);
    j.offsets = a.offsets;
    j.out = static_cast<uint16_t *>(a.out);
    j.num_rows = a.num_rows;
    j.num_experts = a.num_experts;
    j.n = a.n;
    j.k = a.k;
    const hipError_t e = a.transposed ? product_launch<kStore, true>(j, kEdge, s) : product_launch<kStore, false>(j, kEdge, s);
    if (e != hipSuccess || !a.zero_rest || !a.offsets)
        return e;
    hipLaunchKernelGGL(zero_rest_kernel, dim3(256), dim3(256), 0, s, j);
    return hipGetLastError();
}

hipError_t launch_gated_product(const moe_ep_gated_args &a, hipStream_t s)
{
    Job j = {};
    j.x = static_cast<const uint16_t *>(a.x);
    j.w = static_cast<const uint16_t *>(a.w);
    j.offsets = a.offsets;
    j.out = static_cast<uint16_t *>(a.out);
    j.pre = a.pre;
    j.pre_scales = a.pre_scales;
    j.num_rows = a.num_rows;
    j.num_experts = a.num_experts;
    j.n = 2 * a.inter_size;
    j.k = a.k;
    j.save = a.save;
    return product_launch<kGated, false>(j, kEdge / 2, s);
}

hipError_t launch_gated_product_backward(const moe_ep_gated_grad_args &a, hipStream_t s)
{
    Job j = {};
    j.x = static_cast<const uint16_t *>(a.grad_out);
    j.w = static_cast<const uint16_t *>(a.w);
    j.offsets = a.offsets;
    j.out = static_cast<uint16_t *>(a.out);
    j.pre = const_cast<void *>(a.pre);
    j.pre_scales = const_cast<uint8_t *>(a.pre_scales);
    j.grad_pre = static_cast<uint16_t *>(a.grad_pre);
    j.num_rows = a.num_rows;
    j.num_experts = a.num_experts;
    j.n = a.inter_size;
    j.k = a.n;
    j.save = a.save;
    return product_launch<kGatedBackward, true>(j, kEdge, s);
}

hipError_t launch_product_weight_grad(const moe_ep_weight_grad_args &a, hipStream_t s)
{
    const int ntiles = channel_tiles(a.n, kEdge), ktiles = channel_tiles(a.k, kEdge);
    const int64_t grid = (int64_t)a.num_experts * ntiles * ktiles;
    if (grid > INT32_MAX)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(weight_grad_kernel, dim3((unsigned)grid), dim3(256), 0, s, a, ntiles, ktiles);
    return hipGetLastError();
}

} // namespace moe_ep
