// gfx950 kernels of the expert sort (rows to expert order), its way back
// with weights, and the gradients.  All of them move rows and do little
// else, so HBM bounds the large ones and the launches the small ones.
//
// The order is a stable counting sort by expert id: place(p) = number of
// counted pairs with a smaller id, plus those with the same id before p.
// Every place is an integer sum, so no atomic's order reaches a result.
#include "experts_internal.h"
#include "rows.h"

namespace moe_ep {
namespace {

// Local expert of id on rank r, or -1 (unsigned compare covers both ends; a
// masked-off rank has no expert).
__device__ __forceinline__ int local_expert(const moe_ep_sort_args &a, int32_t id, int r)
{
    const uint32_t epr = (uint32_t)a.experts_per_rank, e = (uint32_t)id - (uint32_t)r * epr;
    return e < (a.masked_ranks >> r & 1 ? 0u : epr) ? (int)e : -1;
}

__device__ __forceinline__ const int32_t *rank_ids(const moe_ep_sort_args &a, int r)
{
    return reinterpret_cast<const int32_t *>(reinterpret_cast<const uint8_t *>(a.ids) +
                                             (int64_t)r * a.ids_rank_stride);
}

// ---------------------------------------------------------------------------
// Rows of one slot to their places.  `pos` holds in lane base + j the place
// of pair j (or -1); every wave of the workgroup holds the same.
// ---------------------------------------------------------------------------

// Copies n bytes to each of the slot's places, in words of type W.
template <typename W, int BS>
__device__ __forceinline__ void copy_small(const uint8_t *src, uint8_t *dst, int64_t n, int pos, int base,
                                           uint64_t pairs)
{
    for (int64_t i = threadIdx.x; i < n / (int64_t)sizeof(W); i += BS) {
        const W v = reinterpret_cast<const W *>(src)[i];
        for (uint64_t m = pairs; m; m &= m - 1) {
            const int64_t p = __builtin_amdgcn_readlane(pos, base + __builtin_ctzll(m));
            reinterpret_cast<W *>(dst + p * n)[i] = v;
        }
    }
}

template <int BS>
__device__ __forceinline__ void copy_scale_row(const moe_ep_sort_args &a, int r, int q, int pos, int base,
                                               uint64_t pairs)
{
    const int64_t n = a.scale_row_bytes;
    const uint8_t *src = static_cast<const uint8_t *>(a.scales) + (int64_t)r * a.scales_rank_stride + q * n;
    uint8_t *dst = static_cast<uint8_t *>(a.out_scales);
    const uint64_t align = (uint64_t)(uintptr_t)a.scales | (uint64_t)a.scales_rank_stride | (uint64_t)n |
                           (uint64_t)(uintptr_t)dst;
    if ((align & 15) == 0)
        copy_small<u32x4, BS>(src, dst, n, pos, base, pairs);
    else if ((align & 3) == 0)
        copy_small<uint32_t, BS>(src, dst, n, pos, base, pairs);
    else
        copy_small<uint8_t, BS>(src, dst, n, pos, base, pairs);
}

// Largest magnitude over the workgroup; `red` holds a word for each wave.
template <int BS>
__device__ __forceinline__ uint32_t block_max(uint32_t top, uint32_t *red)
{
    top = wave_max(top);
    __syncthreads(); // the last use of red is over
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < BS / 64; ++w)
        top = max(top, red[w]);
    return top;
}

// One slot's row as int8 codes to its places, by the whole workgroup.  A
// thread keeps its first two 16-element units in registers between the
// maximum and the codes, so a row of up to 32 * BS elements is read once;
// the rest of a longer one is read again from the cache.  (A wave to a row
// needs no barrier, but its lanes then take four times the codes in turn:
// 8 ranks of 2048 slots, rows of 4096, 42 us against 27.)
template <typename T, int BS>
__device__ __forceinline__ void quantize_slot(const moe_ep_sort_args &a, const uint8_t *row, int pos, int base,
                                              uint64_t pairs, uint32_t *red)
{
    constexpr int kHeld = 2, B = 16 * RowType<T>::kBytes;
    const int n = (int)(a.row_bytes / RowType<T>::kBytes), units = n / 16;
    float f[kHeld][16], g[16];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kHeld; ++u) {
        const int i = threadIdx.x + u * BS;
        if (i < units) {
            load_elements<T, 16>(row + (int64_t)i * B, f[u]);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                top = max(top, magnitude(f[u][e]));
        }
    }
    for (int i = threadIdx.x + kHeld * BS; i < units; i += BS) {
        load_elements<T, 16>(row + (int64_t)i * B, g);
#pragma unroll
        for (int e = 0; e < 16; ++e)
            top = max(top, magnitude(g[e]));
    }
    const Int8Row rule(block_max<BS>(top, red));
    const auto store = [&](int i, const float *x) {
        const u32x4 codes = rule.codes16(x);
        for (uint64_t m = pairs; m; m &= m - 1)
            *reinterpret_cast<u32x4 *>(
                static_cast<uint8_t *>(a.out_rows) +
                (int64_t)__builtin_amdgcn_readlane(pos, base + __builtin_ctzll(m)) * n + 16 * i) = codes;
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
        if ((int)threadIdx.x + u * BS < units)
            store(threadIdx.x + u * BS, f[u]);
    for (int i = threadIdx.x + kHeld * BS; i < units; i += BS) {
        load_elements<T, 16>(row + (int64_t)i * B, g);
        store(i, g);
    }
    if (threadIdx.x == 0)
        for (uint64_t m = pairs; m; m &= m - 1)
            static_cast<float *>(a.out_scales)[__builtin_amdgcn_readlane(pos, base + __builtin_ctzll(m))] = rule.scale;
}

// The k bits of a slot's pairs in a wave's ballot.
__device__ __forceinline__ uint64_t slot_pairs(uint64_t ballot, int i, int k)
{
    const uint64_t all = k == 64 ? ~0ull : (1ull << k) - 1;
    return (ballot >> (i * k)) & all;
}

// ---------------------------------------------------------------------------
// Small sorts: one launch.  Each workgroup places its slot's k pairs by
// counting over all pairs (at most 2048, eight a thread), which takes less
// than a second launch would; the last workgroup writes counts and offsets.
// ---------------------------------------------------------------------------

constexpr int kDirectBlock = 256;

template <typename T, bool QUANT>
__global__ __launch_bounds__(kDirectBlock) void sort_direct_kernel(moe_ep_sort_args a, int nchunk)
{
    constexpr int BS = kDirectBlock;
    const int S = a.slots, k = a.top_k, epr = a.experts_per_rank, per_rank = S * k;
    const int npairs = a.ranks * per_rank, nslots = a.ranks * S, lane = threadIdx.x & 63;
    __shared__ int32_t lds[kSortDirectExperts];
    __shared__ uint32_t red[BS / 64];

    if ((int)blockIdx.x == nslots * nchunk) { // counts and offsets
        const int E = a.ranks * epr;
        for (int e = threadIdx.x; e < E; e += BS)
            lds[e] = 0;
        __syncthreads();
        for (int p = threadIdx.x; p < npairs; p += BS) {
            const int r = p / per_rank;
            const int e = local_expert(a, rank_ids(a, r)[p - r * per_rank], r);
            if (e >= 0)
                atomicAdd(&lds[r * epr + e], 1);
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            const int per = (E + 63) / 64, lo = min(E, lane * per), hi = min(E, lo + per);
            int sum = 0;
            for (int e = lo; e < hi; ++e)
                sum += lds[e];
            int before = sum;
            for (int m = 1; m < 64; m <<= 1) {
                const int y = __shfl_up(before, m);
                before += lane >= m ? y : 0;
            }
            before -= sum;
            for (int e = lo; e < hi; ++e) {
                a.counts[e] = lds[e];
                a.offsets[e] = (int32_t)min((int64_t)before, a.capacity);
                before += lds[e];
            }
            if (lane == 63)
                a.offsets[E] = (int32_t)min((int64_t)before, a.capacity);
        }
        return;
    }
    const int slot = blockIdx.x / nchunk, c = blockIdx.x % nchunk;
    const int r = slot / S, q = slot % S;
    const uint8_t *row = static_cast<const uint8_t *>(a.rows) + (int64_t)r * a.rows_rank_stride + q * a.row_bytes;
    // the row's loads go out before the places are known
    const int64_t at = ((int64_t)c * BS + threadIdx.x) * 16;
    u32x4 v = {0, 0, 0, 0};
    if (!QUANT && at < a.row_bytes)
        v = load16_nt(row + at);

    const int mine = slot * k; // first pair of the slot
    int key = -1;              // lane j: global expert of pair j
    if (lane < k) {
        const int e = local_expert(a, rank_ids(a, r)[q * k + lane], r);
        key = e < 0 ? -1 : r * epr + e;
    }
    if (threadIdx.x < 64)
        lds[threadIdx.x] = 0;
    __syncthreads();
    const uint64_t counted = __ballot(key >= 0);
    int before = 0; // lane j: pairs ahead of pair j among this wave's
    if (counted) {
        for (int p0 = 0; p0 < npairs; p0 += BS) {
            const int p = p0 + threadIdx.x;
            int other = 0x7FFFFFFF;
            if (p < npairs) {
                const int rp = p / per_rank;
                const int e = local_expert(a, rank_ids(a, rp)[p - rp * per_rank], rp);
                other = e < 0 ? other : rp * epr + e;
            }
            for (uint64_t m = counted; m; m &= m - 1) {
                const int j = __builtin_ctzll(m);
                const int kj = __builtin_amdgcn_readlane(key, j);
                const int n = __popcll(__ballot(other < kj || (other == kj && p < mine + j)));
                before += lane == j ? n : 0;
            }
        }
        if (lane < k)
            atomicAdd(&lds[lane], before);
    }
    __syncthreads();
    int pos = key >= 0 ? lds[lane] : -1;
    pos = pos < a.capacity ? pos : -1;
    if (c == 0 && (int)threadIdx.x < k)
        a.position[(int64_t)mine + lane] = pos;
    const uint64_t pairs = __ballot(pos >= 0);
    if (!pairs)
        return;
    if (QUANT) {
        quantize_slot<T, BS>(a, row, pos, 0, pairs, red);
        return;
    }
    if (at < a.row_bytes) {
        uint8_t *out = static_cast<uint8_t *>(a.out_rows) + at;
        for (uint64_t m = pairs; m; m &= m - 1)
            *reinterpret_cast<u32x4 *>(out + (int64_t)__builtin_amdgcn_readlane(pos, __builtin_ctzll(m)) * a.row_bytes) = v;
    }
    if (c == 0 && a.scale_row_bytes)
        copy_scale_row<BS>(a, r, q, pos, 0, pairs);
}

// ---------------------------------------------------------------------------
// Large sorts: counts by tile, a scan for each expert, places by tile, then
// the rows.
// ---------------------------------------------------------------------------

constexpr int kTileBlock = 256;

// ws[(r * epr + e) * tiles + t]: pairs of expert e in tile t of rank r.
__global__ __launch_bounds__(kTileBlock) void sort_count_kernel(moe_ep_sort_args a, int tiles)
{
    extern __shared__ int32_t hist[];
    const int r = blockIdx.x / tiles, t = blockIdx.x % tiles, epr = a.experts_per_rank;
    for (int e = threadIdx.x; e < epr; e += kTileBlock)
        hist[e] = 0;
    __syncthreads();
    const int per = sort_tile_slots(a.top_k) * a.top_k;
    const int64_t lo = (int64_t)t * per, hi = min(lo + per, (int64_t)a.slots * a.top_k);
    const int32_t *ids = rank_ids(a, r);
    for (int64_t p = lo + threadIdx.x; p < hi; p += kTileBlock) {
        const int e = local_expert(a, ids[p], r);
        if (e >= 0)
            atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    int32_t *ws = static_cast<int32_t *>(a.workspace);
    for (int e = threadIdx.x; e < epr; e += kTileBlock)
        ws[((int64_t)r * epr + e) * tiles + t] = hist[e];
}

// Inclusive prefix over the workgroup's threads; `sums` holds a word for each
// wave, `total` is all threads' sum.
template <int BS>
__device__ __forceinline__ int block_prefix(int x, int32_t *sums, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int y = __shfl_up(x, m);
        x += lane >= m ? y : 0;
    }
    __syncthreads(); // the last use of sums is over
    if (lane == 63)
        sums[wave] = x;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < BS / 64; ++w) {
        if (w == wave)
            x += total;
        total += sums[w];
    }
    return x;
}

// Each expert's tiles: exclusive prefix in place, and its pairs.  A workgroup
// an expert (one workgroup for the whole table took 300 us of a sort of
// 524288 pairs over 256 experts).
__global__ __launch_bounds__(kTileBlock) void sort_scan_kernel(moe_ep_sort_args a, int tiles)
{
    constexpr int PER = 4;
    __shared__ int32_t sums[kTileBlock / 64];
    int32_t *row = static_cast<int32_t *>(a.workspace) + (int64_t)blockIdx.x * tiles;
    int carry = 0;
    for (int base = 0; base < tiles; base += kTileBlock * PER) {
        const int first = base + threadIdx.x * PER;
        int v[PER], sum = 0, total;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            v[i] = first + i < tiles ? row[first + i] : 0;
            sum += v[i];
        }
        int before = carry + block_prefix<kTileBlock>(sum, sums, total) - sum;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (first + i < tiles)
                row[first + i] = before;
            before += v[i];
        }
        carry += total;
    }
    if (threadIdx.x == 0)
        a.counts[blockIdx.x] = carry;
}

// Places of a wave's 64 pairs, lane by lane (local experts e, -1 for none):
// lanes with the same expert find each other by ballots over the bits of its
// number, and the first of them takes all their places from next[e].
__device__ __forceinline__ int place_pairs(int e, int bits, int lane, int32_t *next)
{
    uint64_t peers = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t m = __ballot((e >> b) & 1);
        peers &= ((e >> b) & 1) ? m : ~m;
    }
    int place = -1;
    if (e >= 0) {
        const int leader = __builtin_ctzll(peers);
        int start = 0;
        if (lane == leader)
            start = atomicAdd(&next[e], __popcll(peers));
        start = __shfl(start, leader);
        place = start + __popcll(peers & ((1ull << lane) - 1));
    }
    return place;
}

// Places of a tile's pairs: each wave takes a quarter of the tile in order.
// A rank's first tile writes its offsets.
__global__ __launch_bounds__(kTileBlock) void sort_place_kernel(moe_ep_sort_args a, int tiles, int bits)
{
    extern __shared__ int32_t next[]; // [waves][epr], at least a word for each wave
    constexpr int kWaves = kTileBlock / 64, IT = kSortTilePairs / kTileBlock;
    const int r = blockIdx.x / tiles, t = blockIdx.x % tiles, epr = a.experts_per_rank;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = sort_tile_slots(a.top_k) * a.top_k;
    const int64_t lo = (int64_t)t * per, hi = min(lo + per, (int64_t)a.slots * a.top_k);
    const int64_t first = lo + wave * (IT * 64);
    const int32_t *ids = rank_ids(a, r);
    int e[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int64_t p = first + i * 64 + lane;
        e[i] = p < hi ? local_expert(a, ids[p], r) : -1;
    }
    // thread x takes the experts x * share ..: `start` is the first one's
    // first place, behind the pairs of all experts before
    const int32_t *counts = a.counts + r * epr;
    const int share = (epr + kTileBlock - 1) / kTileBlock;
    const int elo = min(epr, (int)threadIdx.x * share), ehi = min(epr, elo + share);
    int own = 0, earlier = 0, start, total;
    for (int x = elo; x < ehi; ++x)
        own += counts[x];
    for (int x = threadIdx.x; x < r * epr; x += kTileBlock)
        earlier += a.counts[x];
    block_prefix<kTileBlock>(earlier, next, total);
    start = total - own;
    start += block_prefix<kTileBlock>(own, next, total);
    __syncthreads();
    for (int x = threadIdx.x; x < kWaves * epr; x += kTileBlock)
        next[x] = 0;
    __syncthreads();
    int32_t *mine = next + wave * epr;
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (e[i] >= 0)
            atomicAdd(&mine[e[i]], 1);
    __syncthreads();
    const int32_t *ws = static_cast<const int32_t *>(a.workspace);
    for (int x = elo; x < ehi; ++x) {
        if (t == 0)
            a.offsets[r * epr + x] = (int32_t)min((int64_t)start, a.capacity);
        int before = start + ws[((int64_t)r * epr + x) * tiles + t];
        for (int w = 0; w < kWaves; ++w) {
            const int c = next[w * epr + x];
            next[w * epr + x] = before;
            before += c;
        }
        start += counts[x];
        if (t == 0 && r == a.ranks - 1 && x == epr - 1)
            a.offsets[a.ranks * epr] = (int32_t)min((int64_t)start, a.capacity);
    }
    __syncthreads();
    int32_t *position = a.position + (int64_t)r * a.slots * a.top_k;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int place = place_pairs(e[i], bits, lane, mine);
        const int64_t p = first + i * 64 + lane;
        if (p < hi)
            position[p] = place < a.capacity ? place : -1;
    }
}

// ---------------------------------------------------------------------------
// Sorts in between: each rank's pairs fit one workgroup's registers, so one
// launch counts, scans and places them within the rank (the gather adds the
// pairs of the ranks before).  A workgroup counts all of its rank's pairs and
// places 2048 of them.  With the gather's launch, 8 ranks of 1024 slots, top_k
// 8, take 9.0 us, where one workgroup a rank takes 11.5 and the three launches
// for large sorts 13.1; for twice the pairs 12.4 against 14.3, but with room
// for them 9.5 at 1024 slots, and 64 ranks then take 35 us against 29.
// ---------------------------------------------------------------------------

constexpr int kPlanBlock = 1024;
constexpr int kPlanWaves = kPlanBlock / 64;
constexpr int kPlanPart = 2048; // pairs that a workgroup places

// ws: totals [ranks], then places within the rank [ranks][slots * k].
__global__ __launch_bounds__(kPlanBlock) void sort_plan_kernel(moe_ep_sort_args a, int parts, int bits)
{
    constexpr int IT = kPlanPart / kPlanBlock, OTHERS = kSortPlanPairs / kPlanBlock;
    extern __shared__ int32_t next[]; // [waves][epr], [2][epr] of the parts before and behind, [waves] sums
    const int r = blockIdx.x / parts, part = blockIdx.x % parts, epr = a.experts_per_rank, pairs = a.slots * a.top_k;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int32_t *others = next + kPlanWaves * epr, *sums = others + 2 * epr, *mine = next + wave * epr;
    const int32_t *ids = rank_ids(a, r);
    const int lo = part * kPlanPart, first = lo + wave * (IT * 64);
    int e[IT]; // wave w takes the part's pairs from w * 64 IT on, 64 at a time
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int p = first + i * 64 + lane;
        e[i] = p < pairs ? local_expert(a, ids[p], r) : -1;
    }
    int other[OTHERS];
    if (parts > 1) {
#pragma unroll
        for (int i = 0; i < OTHERS; ++i) {
            const int p = i * kPlanBlock + threadIdx.x;
            other[i] = p < pairs && p / kPlanPart != part ? local_expert(a, ids[p], r) : -1;
        }
    }
    for (int x = threadIdx.x; x < (kPlanWaves + 2) * epr; x += kPlanBlock)
        next[x] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if (e[i] >= 0)
            atomicAdd(&mine[e[i]], 1);
    if (parts > 1) {
#pragma unroll
        for (int i = 0; i < OTHERS; ++i)
            if (other[i] >= 0)
                atomicAdd(&others[(i * kPlanBlock < lo ? 0 : epr) + other[i]], 1);
    }
    __syncthreads();
    // thread x: the pairs of expert x in each wave's share and the other
    // parts, then those of the experts before
    int count = 0, ahead = 0;
    if ((int)threadIdx.x < epr) {
        ahead = others[threadIdx.x];
        count = ahead + others[epr + threadIdx.x];
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w)
            count += next[w * epr + threadIdx.x];
    }
    int before = count;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int y = __shfl_up(before, m);
        before += lane >= m ? y : 0;
    }
    if (lane == 63)
        sums[wave] = before;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        if (w == wave)
            before += total;
        total += sums[w];
    }
    before += ahead - count;
    int32_t *ws = static_cast<int32_t *>(a.workspace);
    if (part == 0 && threadIdx.x == 0)
        ws[r] = total;
    if ((int)threadIdx.x < epr) {
        if (part == 0)
            a.counts[r * epr + threadIdx.x] = count;
        for (int w = 0; w < kPlanWaves; ++w) {
            const int c = next[w * epr + threadIdx.x];
            next[w * epr + threadIdx.x] = before;
            before += c;
        }
    }
    __syncthreads();
    int32_t *places = ws + a.ranks + (int64_t)r * pairs;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int place = place_pairs(e[i], bits, lane, mine);
        const int p = first + i * 64 + lane;
        if (p < pairs)
            places[p] = place;
    }
}

constexpr int kGatherBlock = 256;
constexpr int kGatherVectors = 2;
constexpr int kShortBlock = 128; // for quantised rows of up to 32 elements a thread

// Offsets from the counts, by one workgroup.
template <int BS>
__device__ __forceinline__ void write_offsets(const moe_ep_sort_args &a)
{
    __shared__ int32_t sums[BS / 64];
    const int E = a.ranks * a.experts_per_rank, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (E + BS - 1) / BS, lo = min(E, (int)threadIdx.x * per), hi = min(E, lo + per);
    int sum = 0;
    for (int e = lo; e < hi; ++e)
        sum += a.counts[e];
    int before = sum;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int y = __shfl_up(before, m);
        before += lane >= m ? y : 0;
    }
    if (lane == 63)
        sums[wave] = before;
    __syncthreads();
    for (int w = 0; w < wave; ++w)
        before += sums[w];
    before -= sum;
    for (int e = lo; e < hi; ++e) {
        a.offsets[e] = (int32_t)min((int64_t)before, a.capacity);
        before += a.counts[e];
        if (e == E - 1)
            a.offsets[E] = (int32_t)min((int64_t)before, a.capacity);
    }
}

// Rows to their places: item (group of g slots, chunk of the row; a quantised
// row is one chunk).  PLANNED: the places are the plan's, within the rank; the
// first chunk writes them out, and the workgroup behind the last item the
// offsets.
template <typename T, bool QUANT, bool PLANNED, int BS>
__global__ __launch_bounds__(BS) void sort_gather_kernel(moe_ep_sort_args a, int g, uint32_t nchunk,
                                                                   uint32_t items)
{
    constexpr int VPT = kGatherVectors;
    __shared__ uint32_t red[BS / 64];
    const int64_t nslots = (int64_t)a.ranks * a.slots;
    const int k = a.top_k, lane = threadIdx.x & 63;
    if (PLANNED && blockIdx.x == gridDim.x - 1) {
        write_offsets<BS>(a);
        return;
    }
    const uint32_t step = PLANNED ? gridDim.x - 1 : gridDim.x;
    const int32_t *plan = static_cast<const int32_t *>(a.workspace);
    const int own = PLANNED && lane < a.ranks ? plan[lane] : 0; // lane x: pairs of rank x
    for (uint32_t item = blockIdx.x; item < items; item += step) {
        const int64_t s0 = (int64_t)(item / nchunk) * g;
        const int c = (int)(item % nchunk), ns = (int)min((int64_t)g, nslots - s0);
        int pos = -1;
        if (lane < ns * k)
            pos = PLANNED ? plan[a.ranks + s0 * k + lane] : a.position[s0 * k + lane];
        if (PLANNED) {
            // the pairs of the ranks before the first slot's, and of those
            // that begin within the group
            const int r0 = (int)((uint32_t)s0 / (uint32_t)a.slots);
            const int r = (int)(((uint32_t)s0 + (uint32_t)lane / (uint32_t)k) / (uint32_t)a.slots);
            int before = wave_add(lane < r0 ? own : 0);
            const int r1 = (int)((uint32_t)(s0 + ns - 1) / (uint32_t)a.slots);
            for (int x = r0; x < r1; ++x)
                before += r > x ? __builtin_amdgcn_readlane(own, x) : 0;
            pos = pos >= 0 ? pos + before : -1;
            pos = pos < a.capacity ? pos : -1;
            if ((int)threadIdx.x < ns * k && c == 0)
                a.position[s0 * k + lane] = pos;
        }
        const uint64_t ballot = __ballot(pos >= 0);
        for (int i = 0; i < ns; ++i) {
            const uint64_t pairs = slot_pairs(ballot, i, k);
            if (!pairs)
                continue;
            const uint32_t slot = (uint32_t)(s0 + i);
            const int r = (int)(slot / (uint32_t)a.slots), q = (int)(slot % (uint32_t)a.slots);
            const uint8_t *row =
                static_cast<const uint8_t *>(a.rows) + (int64_t)r * a.rows_rank_stride + (int64_t)q * a.row_bytes;
            if (QUANT) {
                quantize_slot<T, BS>(a, row, pos, i * k, pairs, red);
                continue;
            }
            u32x4 v[VPT];
            int64_t at[VPT];
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                at[u] = (((int64_t)c * VPT + u) * BS + threadIdx.x) * 16;
                if (at[u] < a.row_bytes)
                    v[u] = load16_nt(row + at[u]);
            }
            for (uint64_t m = pairs; m; m &= m - 1) {
                uint8_t *out = static_cast<uint8_t *>(a.out_rows) +
                               (int64_t)__builtin_amdgcn_readlane(pos, i * k + __builtin_ctzll(m)) * a.row_bytes;
#pragma unroll
                for (int u = 0; u < VPT; ++u)
                    if (at[u] < a.row_bytes)
                        store16_nt(out + at[u], v[u]);
            }
            if (c == 0 && a.scale_row_bytes)
                copy_scale_row<BS>(a, r, q, pos, i * k, pairs);
        }
    }
}

// ---------------------------------------------------------------------------
// Back: sum of a slot's rows, weighted or not.
// ---------------------------------------------------------------------------

constexpr int kUnsortBlock = 128;

// Item (group of g slots, chunk of 128 * VPT vectors): VPT output vectors a
// lane, G rows of a slot in flight.
template <typename T, bool WEIGHTS, int VPT, int G>
__global__ __launch_bounds__(kUnsortBlock) void unsort_kernel(moe_ep_unsort_args a, int g, uint32_t nchunk,
                                                              uint32_t items)
{
    constexpr int BS = kUnsortBlock, N = RowType<T>::kPer;
    const int64_t nslots = (int64_t)a.ranks * a.slots, row_bytes = (int64_t)a.hidden_size * RowType<T>::kBytes;
    const int k = a.top_k, lane = threadIdx.x & 63;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t s0 = (int64_t)(item / nchunk) * g;
        const int ns = (int)min((int64_t)g, nslots - s0);
        const int64_t at = ((int64_t)(item % nchunk) * BS * VPT + threadIdx.x) * 16;
        int pos = -1;
        float w = 1.0f;
        if (lane < ns * k) {
            pos = a.position[s0 * k + lane];
            if (WEIGHTS) {
                const uint32_t slot = (uint32_t)s0 + (uint32_t)lane / (uint32_t)k, S = (uint32_t)a.slots;
                w = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.weights) +
                                                    (int64_t)(slot / S) * a.weights_rank_stride)[(int64_t)(slot % S) * k + lane % k];
            }
        }
        const uint64_t ballot = __ballot(pos >= 0 && pos < a.num_rows);
        const uint8_t *rows = static_cast<const uint8_t *>(a.rows) + at;
        for (int i = 0; i < ns; ++i) {
            uint64_t pairs = slot_pairs(ballot, i, k);
            if (!pairs && a.keep_empty)
                continue;
            float acc[VPT][N];
#pragma unroll
            for (int x = 0; x < VPT; ++x)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    acc[x][e] = 0.0f;
            while (pairs) {
                u32x4 v[G][VPT];
                float wj[G];
                uint64_t m = pairs;
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    if (m) {
                        const int j = i * k + __builtin_ctzll(m);
                        m &= m - 1;
                        wj[u] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
                        const int64_t row = (int64_t)__builtin_amdgcn_readlane(pos, j) * row_bytes;
#pragma unroll
                        for (int x = 0; x < VPT; ++x)
                            if (at + x * BS * 16 < row_bytes)
                                v[u][x] = load16_nt(rows + row + x * BS * 16);
                    }
                }
#pragma unroll
                for (int u = 0; u < G; ++u) {
                    if (pairs) {
                        pairs &= pairs - 1;
#pragma unroll
                        for (int x = 0; x < VPT; ++x) {
                            float f[N];
                            RowType<T>::unpack(v[u][x], f);
#pragma unroll
                            for (int e = 0; e < N; ++e)
                                acc[x][e] = WEIGHTS ? fmaf(wj[u], f[e], acc[x][e]) : acc[x][e] + f[e];
                        }
                    }
                }
            }
            const uint32_t slot = (uint32_t)(s0 + i), S = (uint32_t)a.slots;
            uint8_t *out = static_cast<uint8_t *>(a.out) + (int64_t)(slot / S) * a.out_rank_stride +
                           (int64_t)(slot % S) * row_bytes + at;
#pragma unroll
            for (int x = 0; x < VPT; ++x)
                if (at + x * BS * 16 < row_bytes)
                    store16_nt(out + x * BS * 16, RowType<T>::pack(acc[x]));
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient of the weighted way back.
// ---------------------------------------------------------------------------

// One workgroup for a group of g slots.  The slot's grad_out row is held in
// registers (BS * VPT vectors at a time) while each of its k rows passes once:
// read for the dot product, one row ahead, and written scaled.  The k dot
// products are summed over lanes, then waves, in an order that the shape
// fixes.
template <typename T, int BS, int VPT>
__global__ __launch_bounds__(BS) void unsort_grad_kernel(moe_ep_unsort_grad_args a, int g, uint32_t items)
{
    constexpr int N = RowType<T>::kPer, kWaves = BS / 64;
    __shared__ float dots[kWaves][64];
    const int64_t nslots = (int64_t)a.ranks * a.slots, row_bytes = (int64_t)a.hidden_size * RowType<T>::kBytes;
    const int k = a.top_k, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int64_t s0 = (int64_t)item * g;
        const int ns = (int)min((int64_t)g, nslots - s0);
        int pos = -1;
        float w = 1.0f;
        if (lane < ns * k) {
            pos = a.position[s0 * k + lane];
            if (a.weights) {
                const uint32_t slot = (uint32_t)s0 + (uint32_t)lane / (uint32_t)k, S = (uint32_t)a.slots;
                w = reinterpret_cast<const float *>(reinterpret_cast<const uint8_t *>(a.weights) +
                                                    (int64_t)(slot / S) * a.weights_rank_stride)[(int64_t)(slot % S) * k + lane % k];
            }
        }
        const uint64_t ballot = __ballot(pos >= 0 && pos < a.num_rows);
        dots[wave][lane] = 0.0f;
        for (int i = 0; i < ns; ++i) {
            const uint64_t pairs = slot_pairs(ballot, i, k);
            if (!pairs)
                continue;
            const uint32_t slot = (uint32_t)(s0 + i), S = (uint32_t)a.slots;
            const uint8_t *go = static_cast<const uint8_t *>(a.grad_out) +
                                (int64_t)(slot / S) * a.grad_out_rank_stride + (int64_t)(slot % S) * row_bytes;
            for (int64_t base = 0; base < row_bytes; base += BS * VPT * 16) {
                const int64_t at = base + threadIdx.x * 16;
                const auto load = [&](const uint8_t *row, u32x4 *v) {
#pragma unroll
                    for (int u = 0; u < VPT; ++u) {
                        v[u] = u32x4{0, 0, 0, 0};
                        if (at + u * BS * 16 < row_bytes)
                            v[u] = load16_nt(row + at + u * BS * 16);
                    }
                };
                const auto place = [&](uint64_t m) {
                    return (int64_t)__builtin_amdgcn_readlane(pos, i * k + __builtin_ctzll(m)) * row_bytes;
                };
                u32x4 v[VPT], ahead[VPT];
                float f[VPT][N];
                load(go, v);
                if (a.grad_weights)
                    load(static_cast<const uint8_t *>(a.rows) + place(pairs), ahead);
#pragma unroll
                for (int u = 0; u < VPT; ++u)
                    RowType<T>::unpack(v[u], f[u]);
                for (uint64_t m = pairs; m; m &= m - 1) {
                    const int j = i * k + __builtin_ctzll(m);
                    if (a.grad_weights) {
#pragma unroll
                        for (int u = 0; u < VPT; ++u)
                            v[u] = ahead[u];
                        if (m & (m - 1))
                            load(static_cast<const uint8_t *>(a.rows) + place(m & (m - 1)), ahead);
                    }
                    if (a.grad_rows) {
                        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
                        uint8_t *to = static_cast<uint8_t *>(a.grad_rows) + place(m) + at;
#pragma unroll
                        for (int u = 0; u < VPT; ++u)
                            if (at + u * BS * 16 < row_bytes) {
                                float y[N];
#pragma unroll
                                for (int e = 0; e < N; ++e)
                                    y[e] = wj * f[u][e];
                                store16_nt(to + u * BS * 16, RowType<T>::pack(y));
                            }
                    }
                    if (a.grad_weights) {
                        float dot = 0.0f;
#pragma unroll
                        for (int u = 0; u < VPT; ++u) {
                            float x[N];
                            RowType<T>::unpack(v[u], x);
#pragma unroll
                            for (int e = 0; e < N; ++e)
                                dot = fmaf(x[e], f[u][e], dot);
                        }
                        dot = wave_sum(dot);
                        if (lane == j)
                            dots[wave][j] += dot;
                    }
                }
            }
        }
        if (a.grad_weights) {
            __syncthreads();
            if ((int)threadIdx.x < ns * k) {
                float sum = 0.0f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v)
                    sum += dots[v][lane];
                a.grad_weights[s0 * k + lane] = sum;
            }
            __syncthreads(); // before the next item clears the sums
        }
    }
}

// Slots of one workgroup: several where most slots hold no row (the receive
// regions of many ranks), so that the launch is not mostly empty
// workgroups; a wave's 64 lanes hold their places.
inline int slots_per_group(int64_t nslots, int64_t nrows, int k)
{
    int g = 1;
    while (g * 2 * k <= 64 && g * nrows < nslots)
        g *= 2;
    return g;
}

// Workgroups of a launch over `items`: one each, up to a number whose
// threads a 32-bit grid still counts.
inline dim3 grid_of(int64_t items)
{
    const int64_t cap = 1 << 22;
    return dim3((unsigned)(items < cap ? items : cap));
}

} // namespace

hipError_t launch_expert_sort(const moe_ep_sort_args &a, hipStream_t s)
{
    const int64_t nslots = (int64_t)a.ranks * a.slots, nvec = a.row_bytes / 16;
    const int E = a.ranks * a.experts_per_rank;
    if (sort_is_direct(a.ranks, a.slots, a.top_k, E)) {
        const int nchunk = a.quantize ? 1 : (int)((nvec + kDirectBlock - 1) / kDirectBlock);
        const dim3 grid((unsigned)(nslots * nchunk + 1));
        if (!a.quantize)
            hipLaunchKernelGGL((sort_direct_kernel<Bf16, false>), grid, dim3(kDirectBlock), 0, s, a, nchunk);
        else if (a.row_type == MOE_EP_BF16_ROWS)
            hipLaunchKernelGGL((sort_direct_kernel<Bf16, true>), grid, dim3(kDirectBlock), 0, s, a, nchunk);
        else
            hipLaunchKernelGGL((sort_direct_kernel<Fp32, true>), grid, dim3(kDirectBlock), 0, s, a, nchunk);
        return hipGetLastError();
    }
    const int g = slots_per_group(nslots, a.capacity, a.top_k);
    const int64_t groups = (nslots + g - 1) / g;
    const uint32_t nchunk =
        a.quantize ? 1 : (uint32_t)((nvec + kGatherBlock * kGatherVectors - 1) / (kGatherBlock * kGatherVectors));
    const int64_t items = groups * nchunk;
    if (items > INT32_MAX)
        return hipErrorInvalidConfiguration;
    const int epr = a.experts_per_rank;
    int bits = 0;
    while ((1 << bits) < epr)
        ++bits;
    const bool planned = sort_is_planned(a.slots, a.top_k, epr);
    if (planned) {
        const int parts = (a.slots * a.top_k + kPlanPart - 1) / kPlanPart;
        const size_t lds = (size_t)((kPlanWaves + 2) * epr + kPlanWaves) * 4;
        hipLaunchKernelGGL(sort_plan_kernel, dim3(a.ranks * parts), dim3(kPlanBlock), lds, s, a, parts, bits);
        if (hipError_t e = hipGetLastError())
            return e;
    } else {
        const int tiles = (int)sort_tiles(a.slots, a.top_k);
        hipLaunchKernelGGL(sort_count_kernel, dim3(a.ranks * tiles), dim3(kTileBlock), epr * 4, s, a, tiles);
        if (hipError_t e = hipGetLastError())
            return e;
        hipLaunchKernelGGL(sort_scan_kernel, dim3(E), dim3(kTileBlock), 0, s, a, tiles);
        if (hipError_t e = hipGetLastError())
            return e;
        hipLaunchKernelGGL(sort_place_kernel, dim3(a.ranks * tiles), dim3(kTileBlock), (kTileBlock / 64) * epr * 4, s,
                           a, tiles, bits);
        if (hipError_t e = hipGetLastError())
            return e;
        if (!a.capacity || !a.slots)
            return hipSuccess;
    }
    dim3 grid = grid_of(items);
    grid.x += planned;
    // More rows in flight for smaller workgroups: 8 ranks of 2048 slots, top_k
    // 4, rows of 4096: 27.7 us with the plan, 31.0 with 256 threads; 8 of 4096
    // slots, rows of 1024: 28.5 / 35.4 (one rank, 4096 slots that are all full,
    // top_k 8, rows of 4096: 44 / 43).
    const bool shorter = a.quantize && a.row_bytes / (a.row_type == MOE_EP_BF16_ROWS ? 2 : 4) <= 32 * kShortBlock;
    const dim3 block(shorter ? kShortBlock : kGatherBlock);
#define MOE_EP_GATHER(T, QUANT, PLANNED)                                                                              \
    if (QUANT && shorter)                                                                                             \
        hipLaunchKernelGGL((sort_gather_kernel<T, QUANT, PLANNED, QUANT ? kShortBlock : kGatherBlock>), grid, block,  \
                           0, s, a, g, nchunk, (uint32_t)items);                                                      \
    else                                                                                                              \
        hipLaunchKernelGGL((sort_gather_kernel<T, QUANT, PLANNED, kGatherBlock>), grid, block, 0, s, a, g, nchunk,    \
                           (uint32_t)items)
    const bool bf16 = a.row_type == MOE_EP_BF16_ROWS;
    if (planned) {
        if (!a.quantize) {
            MOE_EP_GATHER(Bf16, false, true);
        } else if (bf16) {
            MOE_EP_GATHER(Bf16, true, true);
        } else {
            MOE_EP_GATHER(Fp32, true, true);
        }
    } else {
        if (!a.quantize) {
            MOE_EP_GATHER(Bf16, false, false);
        } else if (bf16) {
            MOE_EP_GATHER(Bf16, true, false);
        } else {
            MOE_EP_GATHER(Fp32, true, false);
        }
    }
#undef MOE_EP_GATHER
    return hipGetLastError();
}

namespace {

template <typename T, bool WEIGHTS, int VPT, int G>
hipError_t unsort_launch(const moe_ep_unsort_args &a, hipStream_t s, int g)
{
    const int64_t nslots = (int64_t)a.ranks * a.slots, nvec = (int64_t)a.hidden_size * RowType<T>::kBytes / 16;
    const uint32_t nchunk = (uint32_t)((nvec + kUnsortBlock * VPT - 1) / (kUnsortBlock * VPT));
    const int64_t items = (nslots + g - 1) / g * nchunk;
    if (items > INT32_MAX)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((unsort_kernel<T, WEIGHTS, VPT, G>), grid_of(items), dim3(kUnsortBlock), 0, s, a, g, nchunk,
                       (uint32_t)items);
    return hipGetLastError();
}

// Slots with several rows have enough loads in flight with one vector a
// lane; where most have none or one (regions of many ranks), four.
template <typename T, bool WEIGHTS>
hipError_t unsort_shape(const moe_ep_unsort_args &a, hipStream_t s)
{
    const int64_t nslots = (int64_t)a.ranks * a.slots;
    const int g = slots_per_group(nslots, a.num_rows, a.top_k);
    return a.num_rows <= nslots ? unsort_launch<T, WEIGHTS, 4, 2>(a, s, g) : unsort_launch<T, WEIGHTS, 1, 8>(a, s, g);
}

} // namespace

hipError_t launch_expert_unsort(const moe_ep_unsort_args &a, hipStream_t s)
{
    if (a.row_type == MOE_EP_BF16_ROWS)
        return a.weights ? unsort_shape<Bf16, true>(a, s) : unsort_shape<Bf16, false>(a, s);
    return a.weights ? unsort_shape<Fp32, true>(a, s) : unsort_shape<Fp32, false>(a, s);
}

hipError_t launch_expert_unsort_backward(const moe_ep_unsort_grad_args &a, hipStream_t s)
{
    const int64_t nslots = (int64_t)a.ranks * a.slots;
    const int g = slots_per_group(nslots, a.num_rows, a.top_k);
    const int64_t items = (nslots + g - 1) / g;
    const dim3 grid = grid_of(items);
    // 4095 slots of 8 rows of 7168 bf16 take 199-210 us in every shape from
    // 64 threads of 8 vectors to 1024 of one (5.0 TB/s, half of it writes: a
    // device copy's rate); rows of 512 vectors and fewer gain by smaller
    // workgroups (4096 slots of 2 rows of 2048: 18.8 us against 24.8).
    const bool shorter = (int64_t)a.hidden_size * (a.row_type == MOE_EP_BF16_ROWS ? 2 : 4) <= 512 * 16;
    const dim3 block(shorter ? 128 : 256);
    if (a.row_type == MOE_EP_BF16_ROWS) {
        if (shorter)
            hipLaunchKernelGGL((unsort_grad_kernel<Bf16, 128, 4>), grid, block, 0, s, a, g, (uint32_t)items);
        else
            hipLaunchKernelGGL((unsort_grad_kernel<Bf16, 256, 4>), grid, block, 0, s, a, g, (uint32_t)items);
    } else {
        if (shorter)
            hipLaunchKernelGGL((unsort_grad_kernel<Fp32, 128, 4>), grid, block, 0, s, a, g, (uint32_t)items);
        else
            hipLaunchKernelGGL((unsort_grad_kernel<Fp32, 256, 4>), grid, block, 0, s, a, g, (uint32_t)items);
    }
    return hipGetLastError();
}

} // namespace moe_ep
