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
    int expert;          // -1: no such tile
    int64_t first, last; // rows of the tile: first <= m < last
    int n;               // channel tile
};

__device__ __forceinline__ int prefix_sum(int x, int lane)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int y = __shfl_up(x, m);
        x += lane >= m ? y : 0;
    }
    return x;
}

// Rows [lo, hi) of expert e, within the num_rows there are.
__device__ __forceinline__ void expert_rows(const moe_ep_matmul_args &a, int e, int &lo, int &hi)
{
    lo = hi = 0;
    if (e < a.num_experts) {
        lo = min(max(a.offsets[e], 0), (int)a.num_rows);
        hi = min(max(a.offsets[e + 1], lo), (int)a.num_rows);
    }
}

// The workgroup's tile: BM rows of one expert and one of its `ntiles`
// channel tiles, found by each wave from the offsets (the host does not know
// them).  Tiles are numbered by expert, channel tile, row tile, so that
// neighbours share their weights, and each of the eight XCDs (workgroup
// number modulo 8) takes a run of them, so that the sharing is in one L2.
template <int BM>
__device__ __forceinline__ Tile find_tile(const moe_ep_matmul_args &a, int ntiles)
{
    Tile t = {-1, 0, 0, 0};
    const int lane = threadIdx.x & 63;
    if (!a.offsets) {
        const int tiles = (int)((a.num_rows + BM - 1) / BM), total = tiles * ntiles, per = (total + 7) / 8;
        const int at = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
        if ((int)(blockIdx.x >> 3) < per && at < total) {
            t.expert = 0;
            t.n = at / tiles;
            t.first = (int64_t)(at % tiles) * BM;
            t.last = min(a.num_rows, t.first + BM);
        }
        return t;
    }
    // lane l sums the experts l * share ..; then the lane that holds the
    // tile is looked into, one expert a lane
    const int share = (a.num_experts + 63) / 64;
    int lo = 0, hi = 0, n = 0;
    for (int i = 0; i < share; ++i) {
        expert_rows(a, lane * share + i, lo, hi);
        n += (hi - lo + BM - 1) / BM;
    }
    int sum = prefix_sum(n, lane);
    const int total = __builtin_amdgcn_readlane(sum, 63) * ntiles, per = (total + 7) / 8;
    const int at = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= per || at >= total)
        return t;
    int start = (sum - n) * ntiles;
    uint64_t hit = __ballot(at >= start && at < start + n * ntiles);
    if (!hit) // offsets that do not ascend: no tile, and nothing out of range
        return t;
    int l = __builtin_ctzll(hit), base = 0;
    if (share > 1) {
        start = __builtin_amdgcn_readlane(start, l);
        base = l * share;
        lo = hi = 0;
        if (lane < share)
            expert_rows(a, base + lane, lo, hi);
        n = (hi - lo + BM - 1) / BM;
        start += (prefix_sum(n, lane) - n) * ntiles;
        hit = __ballot(at >= start && at < start + n * ntiles);
        if (!hit)
            return t;
        l = __builtin_ctzll(hit);
    }
    const int tiles = __builtin_amdgcn_readlane(n, l), here = at - __builtin_amdgcn_readlane(start, l);
    t.n = here / tiles;
    if (t.n >= ntiles)
        return t;
    t.expert = base + l;
    t.first = (int64_t)__builtin_amdgcn_readlane(lo, l) + (int64_t)(here % tiles) * BM;
    t.last = min((int64_t)__builtin_amdgcn_readlane(hi, l), t.first + BM);
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

// One workgroup a tile, in eight runs of the same length; false when there
// are more than a grid of 32-bit thread numbers holds.
inline bool tile_grid(int64_t tiles, int threads, dim3 &grid)
{
    tiles = (tiles + 7) / 8 * 8;
    grid = dim3((unsigned)tiles);
    return tiles * threads <= INT32_MAX;
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
__global__ __launch_bounds__(kSkinnyWaves * 64) void matmul_skinny_kernel(moe_ep_matmul_args a, int ntiles)
{
    constexpr int W = kSkinnyWaves, U = 4;
    __shared__ i32x4 part[W - 1][NT * MT][64];
    const Tile t = find_tile<16 * MT>(a, ntiles);
    if (t.expert < 0)
        return;
    const int n0 = t.n * 16 * NT;
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
    const int64_t ntiles = (a.n + 16 * NT - 1) / (16 * NT);
    dim3 grid;
    if (!tile_grid(most_tiles(a, 16 * MT) * ntiles, kSkinnyWaves * 64, grid))
        return hipErrorInvalidValue;
    const dim3 block(kSkinnyWaves * 64);
    if (a.out_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL((matmul_skinny_kernel<Bf16, NT, MT>), grid, block, 0, s, a, (int)ntiles);
    else
        hipLaunchKernelGGL((matmul_skinny_kernel<Fp32, NT, MT>), grid, block, 0, s, a, (int)ntiles);
    return hipGetLastError();
}

// Many rows an expert: the matrix cores bound the call.  A workgroup of four
// waves takes 256 channels and 128 rows, 128 bytes of k at a time: the next
// 48 KB travel to registers while the MFMAs work on the 48 KB in LDS.  A wave
// holds 128 x 64 of the result (128 registers), so it reads 24 KB of LDS for
// 64 MFMAs; two workgroups share a CU, and one multiplies while the other
// turns its LDS over.
//
// LDS rows are 128 bytes, all on the same banks: chunk c of row r lies at
// place c ^ (r & 7), so that 8 rows' reads of one chunk cover all banks.
constexpr int kTileN = 256, kTileM = 128, kTileK = 128, kTileThreads = 256;

template <typename T>
__global__ __launch_bounds__(kTileThreads, 2) void matmul_tile_kernel(moe_ep_matmul_args a, int ntiles)
{
    constexpr int LN = kTileN / 32, LM = kTileM / 32; // 16-byte loads of a thread
    constexpr int WN = 8, WM = 4;                     // 16 x 16 results of a wave
    __shared__ __align__(16) uint8_t lds[(kTileN + kTileM) * kTileK];
    const Tile t = find_tile<kTileM>(a, ntiles);
    if (t.expert < 0)
        return;
    const int n0 = t.n * kTileN;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int chunk = tid & 7, row = tid >> 3;

    // channels and rows past the last read the last's and are not stored
    const int8_t *wp = a.w + ((int64_t)t.expert * a.n + n0) * a.k;
    const int8_t *xp = a.x + t.first * a.k;
    const int nlast = min(kTileN, a.n - n0) - 1, mlast = (int)(t.last - t.first) - 1;
    uint32_t wo[LN], xo[LM];
#pragma unroll
    for (int i = 0; i < LN; ++i)
        wo[i] = (uint32_t)min(row + 32 * i, nlast) * (uint32_t)a.k + chunk * 16;
#pragma unroll
    for (int i = 0; i < LM; ++i)
        xo[i] = (uint32_t)min(row + 32 * i, mlast) * (uint32_t)a.k + chunk * 16;
    uint8_t *put = lds + row * kTileK + ((chunk ^ (row & 7)) * 16);

    i32x4 wv[LN], xv[LM];
    auto load = [&](int k) {
        const bool in = k + chunk * 16 < a.k; // zeros past the end add nothing
#pragma unroll
        for (int i = 0; i < LN; ++i) {
            wv[i] = i32x4{0, 0, 0, 0};
            if (in)
                wv[i] = *reinterpret_cast<const i32x4 *>(wp + k + wo[i]);
        }
#pragma unroll
        for (int i = 0; i < LM; ++i) {
            xv[i] = i32x4{0, 0, 0, 0};
            if (in)
                xv[i] = *reinterpret_cast<const i32x4 *>(xp + k + xo[i]);
        }
    };
    const int wn = (wave & 1) * 128, wm = (wave >> 1) * 64, l16 = lane & 15, l4 = lane >> 4;
    i32x4 acc[WN][WM] = {};
    load(0);
    for (int k = 0; k < a.k; k += kTileK) {
        __syncthreads(); // the last step's reads are over
#pragma unroll
        for (int i = 0; i < LN; ++i)
            *reinterpret_cast<i32x4 *>(put + i * 32 * kTileK) = wv[i];
#pragma unroll
        for (int i = 0; i < LM; ++i)
            *reinterpret_cast<i32x4 *>(put + (kTileN + i * 32) * kTileK) = xv[i];
        __syncthreads();
        if (k + kTileK < a.k)
            load(k + kTileK);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = ((h * 4 + l4) ^ (l16 & 7)) * 16 + l16 * kTileK;
            i32x4 xf[WM];
#pragma unroll
            for (int j = 0; j < WM; ++j)
                xf[j] = *reinterpret_cast<const i32x4 *>(lds + (kTileN + wm + 16 * j) * kTileK + at);
#pragma unroll
            for (int i = 0; i < WN; ++i) {
                const i32x4 wf = *reinterpret_cast<const i32x4 *>(lds + (wn + 16 * i) * kTileK + at);
#pragma unroll
                for (int j = 0; j < WM; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, xf[j], acc[i][j], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < WM; ++j) {
        const int64_t m = t.first + wm + 16 * j + l16;
        if (m < t.last) {
            const float sx = a.x_scales[m];
#pragma unroll
            for (int i = 0; i < WN; ++i) {
                const int n = n0 + wn + 16 * i + l4 * 4;
                float sw[4];
                channel_scales(a, t.expert, n, sw);
                store_channels<T>(a, m, n, acc[i][j], sx, sw);
            }
        }
    }
}

hipError_t tile_launch(const moe_ep_matmul_args &a, hipStream_t s)
{
    const int64_t ntiles = (a.n + kTileN - 1) / kTileN;
    dim3 grid;
    if (!tile_grid(most_tiles(a, kTileM) * ntiles, kTileThreads, grid))
        return hipErrorInvalidValue;
    if (a.out_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL((matmul_tile_kernel<Bf16>), grid, dim3(kTileThreads), 0, s, a, (int)ntiles);
    else
        hipLaunchKernelGGL((matmul_tile_kernel<Fp32>), grid, dim3(kTileThreads), 0, s, a, (int)ntiles);
    return hipGetLastError();
}

} // namespace

hipError_t launch_expert_matmul(const moe_ep_matmul_args &a, hipStream_t s)
{
    const int64_t average = a.num_rows / a.num_experts;
    return average >= 48 ? tile_launch(a, s) : skinny_launch<4, 2>(a, s);
}

} // namespace moe_ep
