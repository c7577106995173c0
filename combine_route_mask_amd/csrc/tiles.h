// Shared by the products over experts: how a workgroup finds its tiles from the
// offsets on the device, loads from memory straight into LDS, and the waits
// that go with them.  `A` is an argument block with offsets, num_experts and
// num_rows.
#pragma once

#include "rows.h"

namespace moe_ep {

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
template <typename A>
__device__ __forceinline__ void expert_rows(const A &a, int e, int &lo, int &hi)
{
    if (!a.offsets) {
        lo = 0;
        hi = e == 0 ? (int)a.num_rows : 0;
        return;
    }
    lo = hi = 0;
    if (e < a.num_experts) {
        lo = min(max(a.offsets[e], 0), (int)a.num_rows);
        hi = min(max(a.offsets[e + 1], lo), (int)a.num_rows);
    }
}

// Tiles of up to bm rows for rows [lo, hi); hi - lo + bm may pass 2^31.
__device__ __forceinline__ int row_tiles(int lo, int hi, int bm)
{
    return (int)(((uint32_t)(hi - lo) + (uint32_t)bm - 1) / (uint32_t)bm);
}

// Tiles of bn of the n channels; n + bn may pass 2^31.
__host__ __device__ __forceinline__ int channel_tiles(int n, int bn)
{
    return (int)(((uint32_t)n + (uint32_t)bn - 1) / (uint32_t)bn);
}

constexpr int kBand = 4;
constexpr int kUnit = 64; // tiles begin this many rows apart, or a multiple

// Finds a workgroup's tiles: up to BM rows of one expert and one of its
// `ntiles` channel tiles, by each wave from the offsets (the host does not
// know them).  Tiles are numbered by expert, band of kBand row tiles, channel
// tile, row tile, and each of the eight XCDs (workgroup number modulo 8) takes
// a run of them: the tiles that run at a time on its 32 CUs are 4 x 8, which
// read the least through its L2 (8192 x 8192 x 8192: 429 us; bands of 6 423, of
// 8 441, columns of all row tiles 462).  An expert's row tiles are of even
// height.  Of the tallest tiles BM and OTHERS the finder takes what the CUs are
// done with first: a tile takes about as long as `edge` rows and its own.
template <int BM, int... OTHERS>
struct TileFinder {
    static constexpr int kHeights[] = {BM, OTHERS...};
    int lane, ntiles, share, per, total, first, bm;
    int lo, hi, n, start; // of the lane's experts

    // lane l sums the experts l * share ..; a tile's lane is then looked
    // into, one expert a lane
    template <typename A>
    __device__ __forceinline__ TileFinder(const A &a, int ntiles_, float edge) : ntiles(ntiles_)
    {
        lane = threadIdx.x & 63;
        share = (a.num_experts + 63) / 64;
        constexpr int H = 1 + sizeof...(OTHERS);
        int count[H] = {};
        float rows = 0.0f;
        for (int i = 0; i < share; ++i) {
            expert_rows(a, lane * share + i, lo, hi);
#pragma unroll
            for (int h = 0; h < H; ++h)
                count[h] += row_tiles(lo, hi, kHeights[h]);
            rows += (float)(hi - lo);
        }
        n = count[0];
        int sum = prefix_sum(n, lane);
        bm = BM;
        if (H > 1) {
            rows = wave_sum(rows);
            float best = time_of(__builtin_amdgcn_readlane(sum, 63), rows, edge);
#pragma unroll
            for (int h = 1; h < H; ++h) {
                const int other = prefix_sum(count[h], lane);
                const float time = time_of(__builtin_amdgcn_readlane(other, 63), rows, edge);
                if (time < best) {
                    best = time;
                    bm = kHeights[h];
                    n = count[h];
                    sum = other;
                }
            }
        }
        total = __builtin_amdgcn_readlane(sum, 63) * ntiles;
        per = (total + 7) / 8;
        first = (int)(blockIdx.x & 7) * per;
        start = (sum - n) * ntiles;
    }

    // Rounds of 256 CUs times a tile.
    __device__ __forceinline__ float time_of(int tiles, float rows, float edge) const
    {
        return tiles ? (float)((tiles * ntiles + 255) / 256) * (edge + rows / (float)tiles) : 0.0f;
    }

    template <typename A>
    __device__ __forceinline__ Tile tile(const A &a, int slot) const
    {
        Tile t = {-1, 0, 0, 0};
        const int at = first + slot;
        if (slot >= per || at >= total)
            return t;
        uint64_t hit = __ballot(at >= start && at < start + n * ntiles);
        if (!hit) // offsets that do not ascend: no tile, and nothing out of range
            return t;
        int l = __builtin_ctzll(hit), base = 0;
        int elo = lo, ehi = hi, en = n, estart = start;
        if (share > 1) {
            estart = __builtin_amdgcn_readlane(start, l);
            base = l * share;
            elo = ehi = 0;
            if (lane < share)
                expert_rows(a, base + lane, elo, ehi);
            en = row_tiles(elo, ehi, bm);
            estart += (prefix_sum(en, lane) - en) * ntiles;
            hit = __ballot(at >= estart && at < estart + en * ntiles);
            if (!hit)
                return t;
            l = __builtin_ctzll(hit);
        }
        const int tiles = __builtin_amdgcn_readlane(en, l), here = at - __builtin_amdgcn_readlane(estart, l);
        const int band = here / (kBand * ntiles), height = min(kBand, tiles - band * kBand);
        const int in = here - band * kBand * ntiles;
        if (height < 1)
            return t;
        t.n = in / height;
        if (t.n >= ntiles)
            return t;
        t.expert = base + l;
        const int begin = __builtin_amdgcn_readlane(elo, l), end = __builtin_amdgcn_readlane(ehi, l);
        const int units = (int)(((int64_t)end - begin + kUnit - 1) / kUnit), each = units / tiles, more = units % tiles;
        // row tiles of each + 1 units, `more` of them, then of each; a workgroup's
        // next tile is of another height than its last
        const int within = in % height, row = band * kBand + (within + (unsigned)(at - within) / 32) % height;
        t.first = begin + (int64_t)(row * each + min(row, more)) * kUnit;
        t.last = min((int64_t)end, t.first + (each + (row < more)) * kUnit);
        return t;
    }
};

// At most this many row tiles, whatever the offsets: each expert with rows
// has at most one that is not full.
template <typename A>
inline int64_t most_tiles(const A &a, int64_t bm)
{
    const int64_t full = a.num_rows / bm;
    return a.offsets ? full + (a.num_rows < a.num_experts ? a.num_rows : a.num_experts)
                     : (a.num_rows + bm - 1) / bm;
}

// 16 bytes a lane from base + offset + k into LDS: lane l's to `to` + 16 l.
// (The buffer form: a global load into LDS makes every later LDS wait wait
// for all reads.)  An offset from kPastEnd on is beyond the buffer: zeros.
constexpr uint32_t kPastEnd = 0x80000000u;

__device__ __forceinline__ void load_lds(const int8_t *base, uint32_t offset, int k, uint8_t *to)
{
#if defined(__HIP_DEVICE_COMPILE__) // the host compiler does not know the resource type
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, 0x7FFFFFFF, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 16, offset, k, 0, 0);
#endif
}

// Waits until at most N of the wave's loads are on their way and all its LDS
// reads are back, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

} // namespace moe_ep
