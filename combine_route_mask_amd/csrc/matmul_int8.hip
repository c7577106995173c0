// gfx950 kernels of the int8 product over experts: int32 sums on the matrix
// cores (exact, so neither the order of the sum nor its split changes a
// result), scaled by token and channel in fp32 and rounded once.
//
// MFMA operands: the weights are the left matrix (16 channels n) and the
// tokens the right one (16 rows m), so a lane ends with four consecutive
// channels of one token.  v_mfma_i32_16x16x64_i8: lane l holds 16 bytes of
// row l % 16 at k = 16 * (l / 16) of either matrix; of the result, element i
// is channel 4 * (l / 16) + i of token l % 16.
#include "experts_internal.h"
#include "rows.h"

namespace moe_ep {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct Tile {
    int expert;
    int64_t first, last; // rows of the tile: first <= m < last
};

// The tile number `index` of all experts' row tiles of BM rows, found by
// each wave from the offsets; expert -1 when there are fewer tiles.
template <int BM>
__device__ __forceinline__ Tile find_tile(const moe_ep_matmul_args &a, int64_t index)
{
    Tile t = {-1, 0, 0};
    if (!a.offsets) {
        if (index * BM < a.num_rows) {
            t.expert = 0;
            t.first = index * BM;
            t.last = min(a.num_rows, t.first + BM);
        }
        return t;
    }
    const int lane = threadIdx.x & 63;
    const int M = (int)a.num_rows;
    int before = 0; // tiles of the experts so far
    for (int e0 = 0; e0 < a.num_experts; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.num_experts) {
            lo = min(max(a.offsets[e], 0), M);
            hi = min(max(a.offsets[e + 1], lo), M);
        }
        const int n = (hi - lo + BM - 1) / BM;
        int sum = n;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int y = __shfl_up(sum, m);
            sum += lane >= m ? y : 0;
        }
        const int start = before + sum - n;
        const uint64_t hit = __ballot(index >= start && index < start + n);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int s = __builtin_amdgcn_readlane(start, l);
            t.expert = e0 + l;
            t.first = (int64_t)__builtin_amdgcn_readlane(lo, l) + (index - s) * BM;
            t.last = min((int64_t)__builtin_amdgcn_readlane(hi, l), t.first + BM);
            return t;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return t;
}

// At most this many row tiles, whatever the offsets: each expert with rows
// has at most one that is not full.
inline int64_t most_tiles(const moe_ep_matmul_args &a, int64_t bm)
{
    const int64_t full = a.num_rows / bm;
    return a.offsets ? full + (a.num_rows < a.num_experts ? a.num_rows : a.num_experts)
                     : (a.num_rows + bm - 1) / bm;
}

// Four consecutive channels of token m, scaled and rounded.
template <typename T>
__device__ __forceinline__ void store_channels(const moe_ep_matmul_args &a, int64_t m, int n, const i32x4 &sum,
                                               float sx, const float *sw)
{
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = (float)sum[i] * (sx * sw[i]);
    const int64_t at = m * a.n + n;
    if (RowType<T>::kBytes == 2) {
        uint16_t *out = static_cast<uint16_t *>(a.out) + at;
        if (n + 4 <= a.n && (a.n & 3) == 0 && ((uintptr_t)a.out & 7) == 0) {
            *reinterpret_cast<u32x2 *>(out) = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.n)
                out[i] = (uint16_t)f32_to_bf16_rne(f[i]);
    } else {
        float *out = static_cast<float *>(a.out) + at;
        if (n + 4 <= a.n && (a.n & 3) == 0 && ((uintptr_t)a.out & 15) == 0) {
            *reinterpret_cast<u32x4 *>(out) = RowType<Fp32>::pack(f);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < a.n)
                out[i] = f[i];
    }
}

__device__ __forceinline__ void channel_scales(const moe_ep_matmul_args &a, int e, int n, float *sw)
{
    const float *s = a.w_scales + (int64_t)e * a.n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sw[i] = n + i < a.n ? s[n + i] : 0.0f;
}

constexpr int kSkinnyWaves = 4;

// Few rows an expert: the weights stream from HBM once and bound the call.
// A workgroup takes 16 * NT channels of one expert and 16 * MT rows; its
// waves take a quarter of k each, straight from memory into the MFMA's
// registers, and add their int32 sums in LDS.
template <typename T, int NT, int MT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void matmul_skinny_kernel(moe_ep_matmul_args a, uint32_t ntiles)
{
    constexpr int W = kSkinnyWaves, U = 4;
    __shared__ i32x4 part[W - 1][NT * MT][64];
    const Tile t = find_tile<16 * MT>(a, blockIdx.x / ntiles);
    if (t.expert < 0)
        return;
    const int n0 = (int)(blockIdx.x % ntiles) * 16 * NT;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, k16 = (lane >> 4) * 16;
    const int8_t *wp[NT], *xp[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) // channels past the last read the last's weights and are not stored
        wp[i] = a.w + ((int64_t)t.expert * a.n + min(n0 + 16 * i + l16, a.n - 1)) * a.k + k16;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xp[i] = a.x + min(t.first + 16 * i + l16, t.last - 1) * a.k + k16;
    i32x4 acc[NT][MT] = {};
    const int steps = (a.k + 63) / 64, share = (steps + W - 1) / W;
    const int lo = wave * share, hi = min(steps, lo + share);
    for (int s0 = lo; s0 < hi; s0 += U) {
        i32x4 wv[U][NT], xv[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (s0 + u) * 64;
            const bool in = s0 + u < hi && k + k16 < a.k; // zeros past the end add nothing
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                wv[u][i] = i32x4{0, 0, 0, 0};
                if (in)
                    wv[u][i] = __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(wp[i] + k));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                xv[u][i] = i32x4{0, 0, 0, 0};
                if (in)
                    xv[u][i] = *reinterpret_cast<const i32x4 *>(xp[i] + k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u][i], xv[u][j], acc[i][j], 0, 0, 0);
    }
    if (wave) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < MT; ++j)
                part[wave - 1][i * MT + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave)
        return;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        const int64_t m = t.first + 16 * j + l16;
        const bool stored = m < t.last;
        const float sx = stored ? a.x_scales[m] : 0.0f;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int n = n0 + 16 * i + (lane >> 4) * 4;
            float sw[4];
            channel_scales(a, t.expert, n, sw);
            i32x4 sum = acc[i][j];
#pragma unroll
            for (int w = 0; w < W - 1; ++w)
                sum += part[w][i * MT + j][lane];
            if (stored)
                store_channels<T>(a, m, n, sum, sx, sw);
        }
    }
}

template <int NT, int MT>
hipError_t skinny_launch(const moe_ep_matmul_args &a, hipStream_t s)
{
    const int64_t ntiles = (a.n + 16 * NT - 1) / (16 * NT), items = most_tiles(a, 16 * MT) * ntiles;
    if (items > (1 << 23))
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)items), block(kSkinnyWaves * 64);
    if (a.out_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL((matmul_skinny_kernel<Bf16, NT, MT>), grid, block, 0, s, a, (uint32_t)ntiles);
    else
        hipLaunchKernelGGL((matmul_skinny_kernel<Fp32, NT, MT>), grid, block, 0, s, a, (uint32_t)ntiles);
    return hipGetLastError();
}

} // namespace

hipError_t launch_expert_matmul(const moe_ep_matmul_args &a, hipStream_t s)
{
    return skinny_launch<4, 2>(a, s);
}

} // namespace moe_ep
