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
typedef u32x4 AnyAligned __attribute__((aligned(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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
// height.  Of BM and TALL the finder takes what the CUs are done with first:
// a tile takes about as long as 76 rows and its own.
template <int BM, int TALL>
struct TileFinder {
    int lane, ntiles, share, per, total, first, bm;
    int lo, hi, n, start; // of the lane's experts

    // lane l sums the experts l * share ..; a tile's lane is then looked
    // into, one expert a lane
    __device__ __forceinline__ TileFinder(const moe_ep_matmul_args &a, int ntiles_) : ntiles(ntiles_)
    {
        lane = threadIdx.x & 63;
        share = (a.num_experts + 63) / 64;
        n = 0;
        int tall = 0;
        float rows = 0.0f;
        for (int i = 0; i < share; ++i) {
            expert_rows(a, lane * share + i, lo, hi);
            n += row_tiles(lo, hi, BM);
            tall += row_tiles(lo, hi, TALL);
            rows += (float)(hi - lo);
        }
        int sum = prefix_sum(n, lane);
        bm = BM;
        if (TALL != BM) {
            const int sum_tall = prefix_sum(tall, lane);
            rows = wave_sum(rows);
            if (time_of(__builtin_amdgcn_readlane(sum_tall, 63), rows) < time_of(__builtin_amdgcn_readlane(sum, 63), rows)) {
                bm = TALL;
                n = tall;
                sum = sum_tall;
            }
        }
        total = __builtin_amdgcn_readlane(sum, 63) * ntiles;
        per = (total + 7) / 8;
        first = (int)(blockIdx.x & 7) * per;
        start = (sum - n) * ntiles;
    }

    // Rounds of 256 CUs times a tile.
    __device__ __forceinline__ float time_of(int tiles, float rows) const
    {
        return tiles ? (float)((tiles * ntiles + 255) / 256) * (76.0f + rows / (float)tiles) : 0.0f;
    }

    __device__ __forceinline__ Tile tile(const moe_ep_matmul_args &a, int slot) const
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
        const int row = band * kBand + in % height; // row tiles of each + 1 units, `more` of them, then of each
        t.first = begin + (int64_t)(row * each + min(row, more)) * kUnit;
        t.last = min((int64_t)end, t.first + (each + (row < more)) * kUnit);
        return t;
    }
};

// At most this many row tiles, whatever the offsets: each expert with rows
// has at most one that is not full.
inline int64_t most_tiles(const moe_ep_matmul_args &a, int64_t bm)
{
    const int64_t full = a.num_rows / bm;
    return a.offsets ? full + (a.num_rows < a.num_experts ? a.num_rows : a.num_experts)
                     : (a.num_rows + bm - 1) / bm;
}

template <typename T>
__device__ __forceinline__ void store_element(void *p, float y)
{
    if (RowType<T>::kBytes == 2)
        *static_cast<uint16_t *>(p) = (uint16_t)f32_to_bf16_rne(y);
    else
        *static_cast<float *>(p) = y;
}

// A workgroup takes BN channels and BM rows, 128 bytes of k at a time,
// through STAGES of LDS: the next stages' rows go from memory straight into
// LDS while this one's are multiplied.  NW x MW waves, each FN x FM results of
// 16 x 16.
constexpr int kTileK = 128;

template <int NW_, int MW_, int FN_, int FM_, int STAGES_>
struct TileShape {
    static constexpr int NW = NW_, MW = MW_, FN = FN_, FM = FM_, STAGES = STAGES_, W = NW * MW;
    static constexpr int BN = NW * FN * 16, BM = MW * FM * 16, THREADS = 64 * W;
    static constexpr int LN = BN / (8 * W), LM = BM / (8 * W); // loads of a thread and stage; a wave's covers 8 rows
    static constexpr int BYTES = (BN + BM) * kTileK;
};

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

// 4 bytes a lane, as above.
__device__ __forceinline__ void load_lds_word(const float *base, uint32_t offset, uint8_t *to)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(base), 0, 0x7FFFFFFF, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 4, offset, 0, 0, 0);
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

// A tile's operands: where a thread's rows start, and where the wave's first
// fragments lie in a stage.
template <typename S>
struct Operands {
    const int8_t *wp, *xp;
    uint32_t wo[S::LN], xo[S::LM];
    int wave;
    uint32_t wat[2], xat[2];
    int steps, start; // steps of k, and the first of them
    uint32_t end;     // kPastEnd where the lane's chunk of the last step is past k
};

template <typename S>
struct Fragments {
    i32x4 x[2][S::FM], w[2 * S::FN];
};

template <typename S>
__device__ __forceinline__ void read_x(const uint8_t *stage, const Operands<S> &o, Fragments<S> &f, int h, int j)
{
    f.x[h][j] = *reinterpret_cast<const i32x4 *>(stage + o.xat[h] + 16 * j * kTileK);
}

template <typename S>
__device__ __forceinline__ void read_w(const uint8_t *stage, const Operands<S> &o, Fragments<S> &f, int i)
{
    f.w[i] = *reinterpret_cast<const i32x4 *>(stage + o.wat[i / S::FN] + 16 * (i % S::FN) * kTileK);
}

template <typename S>
__device__ __forceinline__ void load_part(uint8_t *stage, const Operands<S> &o, int i, int k, uint32_t past)
{
    if (i < S::LN)
        load_lds(o.wp, o.wo[i] | past, k, stage + (i * S::W + o.wave) * 1024);
    else
        load_lds(o.xp, o.xo[i - S::LN] | past, k, stage + S::BN * kTileK + ((i - S::LN) * S::W + o.wave) * 1024);
}

constexpr int kAhead = 2; // weight fragments are read this many products before they are used

// The products of stage `cur`, groups of FM.  The first kAhead fragments are
// in registers already; the last groups run behind the barrier and read the
// first of `next`, so that neither LDS nor the barrier leaves the matrix
// cores idle for long.  Behind it `cur`, which no wave reads again, takes the
// loads for STAGES steps on: they have at least a whole step to arrive.
// wait_barrier() orders them behind the reads before it, and waits for the loads
// that the reads behind it need.
template <typename S, typename ACC>
__device__ __forceinline__ void tile_step(uint8_t *cur, const uint8_t *next, int k, uint32_t past, const Operands<S> &o,
                                          Fragments<S> &f, ACC &acc, Fragments<S> &g)
{
    constexpr int G = 2 * S::FN, L = S::LN + S::LM, FIRST = S::FN - S::FM - kAhead + 1;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        if (i + kAhead < G)
            read_w<S>(cur, o, f, i + kAhead);
#pragma unroll
        for (int j = 0; j < S::FM; ++j) // the second half's rows, spread before its first product
            if (i == (FIRST + j > 0 ? FIRST + j : 0))
                read_x<S>(cur, o, f, 1, j);
        if (i == G - kAhead)
            wait_barrier<(S::STAGES - 2) * L>(); // this stage is read, the next one has arrived
        __builtin_amdgcn_sched_barrier(0);
        if (i >= G - kAhead) {
            read_w<S>(next, o, g, i - (G - kAhead));
#pragma unroll
            for (int j = 0; j < S::FM; ++j)
                if (j % kAhead == i - (G - kAhead))
                    read_x<S>(next, o, g, 0, j);
#pragma unroll
            for (int u = 0; u < L; ++u)
                if (u * kAhead / L == i - (G - kAhead))
                    load_part<S>(cur, o, u, k, past);
        }
#pragma unroll
        for (int j = 0; j < S::FM; ++j)
            acc[i % S::FN][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.w[i], f.x[i / S::FN][j], acc[i % S::FN][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
    // the fragments read ahead
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        f.w[i] = g.w[i];
#pragma unroll
    for (int j = 0; j < S::FM; ++j)
        f.x[0][j] = g.x[0][j];
}

template <typename T, typename S>
__device__ __forceinline__ Operands<S> find_operands(const moe_ep_matmul_args &a, const Tile &t)
{
    constexpr int FN = S::FN, FM = S::FM;
    const int n0 = t.n * S::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    Operands<S> o;
    o.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    o.wp = a.w + ((int64_t)t.expert * a.n + n0) * a.k;
    o.xp = a.x + t.first * a.k;
    // LDS rows are 128 bytes, all on the same banks: chunk c of row r lies at
    // place c ^ (r & 7), so that 8 rows' reads of one chunk cover all banks.
    // Within a wave's 16 FN channels LDS row 16 i + r holds channel
    // 16 V (i / V) + 4 V (r / 4) + 4 (i % V) + r % 4: V fragments then give a
    // lane the channels of one 16-byte store, and the four lanes of a row
    // store 64 bytes in a row.  Channels and rows past the last read the
    // last's and are not stored.
    constexpr int V = RowType<T>::kPer / 4; // results of 4 channels in a 16-byte store
    static_assert(FN % V == 0);
    const int sub = lane / 8;
    const uint32_t chunk = (uint32_t)((lane % 8) ^ sub) * 16;
    const int nlast = min(S::BN, a.n - n0) - 1, mlast = (int)(t.last - t.first) - 1;
#pragma unroll
    for (int i = 0; i < S::LN; ++i) {
        const int row = (i * S::W + o.wave) * 8 + sub, r = row & 15;
        const int n = (row / (16 * V)) * (16 * V) + 4 * V * (r >> 2) + 4 * (row / 16 % V) + (r & 3);
        o.wo[i] = (uint32_t)min(n, nlast) * (uint32_t)a.k + chunk;
    }
#pragma unroll
    for (int i = 0; i < S::LM; ++i)
        o.xo[i] = (uint32_t)min((i * S::W + o.wave) * 8 + sub, mlast) * (uint32_t)a.k + chunk;
    const int wn = (o.wave % S::NW) * FN * 16, wm = (o.wave / S::NW) * FM * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t place = (uint32_t)(((h * 4 + l4) ^ (l16 & 7)) * 16 + l16 * kTileK);
        o.wat[h] = place + wn * kTileK;
        o.xat[h] = place + (S::BN + wm) * kTileK;
    }
    o.steps = (a.k + kTileK - 1) / kTileK;
    // of the last step, a lane's chunk past the end of k is zeros
    o.end = (o.steps - 1) * kTileK + chunk < (uint32_t)a.k ? 0 : kPastEnd;
    // k starts elsewhere in each channel tile and goes round: rows a power of
    // two apart would otherwise have all workgroups read the same few memory
    // channels at a time (64 rows, 32 experts, N = K = 4096: 106 us all from
    // k = 0, 79 us)
    o.start = (int)(((uint32_t)t.expert * (uint32_t)channel_tiles(a.n, S::BN) + (uint32_t)t.n) % (uint32_t)o.steps);
    return o;
}

// The loads of a tile's scales (channels, then rows; 64 of them to a wave)
// and first stages.
template <typename T, typename S>
__device__ __forceinline__ void load_first(const moe_ep_matmul_args &a, const Tile &t, uint8_t *lds, uint8_t *scales)
{
    const Operands<S> o = find_operands<T, S>(a, t);
    constexpr int NPIECES = S::BN / 64, PIECES = NPIECES + (S::BM + 63) / 64;
    static_assert(S::BN % 64 == 0);
    const int lane = threadIdx.x & 63, n0 = t.n * S::BN;
#pragma unroll
    for (int c = 0; c < PIECES; c += S::W) {
        const int piece = c + o.wave;
        if (piece < NPIECES)
            load_lds_word(a.w_scales + (int64_t)t.expert * a.n + n0, 4 * min(64 * piece + lane, a.n - n0 - 1),
                          scales + 256 * piece);
        else if (piece < PIECES)
            load_lds_word(a.x_scales + t.first, 4 * min(64 * (piece - NPIECES) + lane, (int)(t.last - t.first) - 1),
                          scales + 256 * piece);
    }
#pragma unroll
    for (int st = 0; st < S::STAGES; ++st) {
        const int at = (o.start + st) % o.steps;
#pragma unroll
        for (int i = 0; i < S::LN + S::LM; ++i)
            load_part<S>(lds + st * S::BYTES, o, i, at * kTileK, at == o.steps - 1 ? o.end : 0);
    }
}

// Tile t, whose scales and first stages are on their way.  `ahead` sends off
// the next tile's once this one's LDS is free: they pass while the results are
// scaled and stored.
template <typename T, typename S, typename AHEAD>
__device__ __forceinline__ void multiply_tile(const moe_ep_matmul_args &a, const Tile &t, uint8_t *lds,
                                              const uint8_t *scales, AHEAD ahead)
{
    constexpr int FN = S::FN, FM = S::FM;
    constexpr int V = RowType<T>::kPer / 4;
    const Operands<S> o = find_operands<T, S>(a, t);
    const int steps = o.steps, n0 = t.n * S::BN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
    const int wn = (o.wave % S::NW) * FN * 16, wm = (o.wave / S::NW) * FM * 16;
    i32x4 acc[FN][FM] = {};
    Fragments<S> f, g;
    uint8_t *cur = lds, *next = lds + S::BYTES;
    wait_barrier<(S::STAGES - 1) * (S::LN + S::LM)>();
#pragma unroll
    for (int j = 0; j < FM; ++j)
        read_x<S>(cur, o, f, 0, j);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        read_w<S>(cur, o, f, i);
    int at = (o.start + S::STAGES) % steps;
    // the loads behind the last step are not read, nor do they reach memory
    for (int i = 0; i < steps; ++i) {
        const uint32_t past = i >= steps - S::STAGES ? kPastEnd : at == steps - 1 ? o.end : 0;
        tile_step<S>(cur, next, at * kTileK, past, o, f, acc, g);
        at = at + 1 == steps ? 0 : at + 1;
        cur = next;
        next = next == lds + (S::STAGES - 1) * S::BYTES ? lds : next + S::BYTES;
    }
    wait_barrier<0>(); // all waves are done with LDS, and nothing is on its way there
    const int wl = wn + 4 * V * l4, nw = n0 + wl; // the lane's first channel
    f32x4 sw[FN];
    float sx[FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
        sw[i] = *reinterpret_cast<const f32x4 *>(scales + 4 * (wl + 16 * V * (i / V) + 4 * (i % V)));
#pragma unroll
    for (int j = 0; j < FM; ++j)
        sx[j] = *reinterpret_cast<const float *>(scales + 4 * (S::BN + wm + 16 * j + l16));
    ahead();
    // The sum meets its channel's scale first: the scales' own product may lie
    // outside fp32 (rows of any magnitude) where the result does not.
    // Rows of any n start at any element: 16-byte stores need no more than an
    // element's alignment.
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int64_t m = t.first + wm + 16 * j + l16;
        if (m >= t.last)
            continue;
        uint8_t *out = static_cast<uint8_t *>(a.out) + (m * a.n + nw) * RowType<T>::kBytes;
#pragma unroll
        for (int i = 0; i < FN; i += V) {
            const int n = nw + 16 * i;
            float y[4 * V];
#pragma unroll
            for (int e = 0; e < 4 * V; ++e)
                y[e] = ((float)acc[i + e / 4][j][e % 4] * sw[i + e / 4][e % 4]) * sx[j];
            if (a.n - n >= 4 * V) { // the last channels' n + 4 V may pass 2^31
                *reinterpret_cast<AnyAligned *>(out + 16 * i * RowType<T>::kBytes) = RowType<T>::pack(y);
            } else {
#pragma unroll
                for (int e = 0; e < 4 * V; ++e)
                    if (e < a.n - n)
                        store_element<T>(out + (16 * i + e) * RowType<T>::kBytes, y[e]);
            }
        }
    }
}

// The tile's rows choose among the shapes, smallest first: the last rows of
// an expert do not pay for rows that are not there.
template <typename S, typename... MORE, typename F>
__device__ __forceinline__ void with_shape(const Tile &t, F f)
{
    if constexpr (sizeof...(MORE) == 0) {
        f(S{});
    } else {
        if (t.last - t.first <= S::BM)
            f(S{});
        else
            with_shape<MORE...>(t, f);
    }
}

constexpr int largest(int x) { return x; }

template <typename... MORE>
constexpr int largest(int x, MORE... more)
{
    return x > largest(more...) ? x : largest(more...);
}

// Bytes of a tile's scales.
template <typename S, typename... MORE>
constexpr int tile_scales()
{
    return 256 * largest(S::BN / 64 + (S::BM + 63) / 64, (MORE::BN / 64 + (MORE::BM + 63) / 64)...);
}

// A workgroup takes the tiles `slot`, slot + (workgroups of the XCD), ... of
// its XCD's run.
template <typename T, typename S, typename... MORE>
__global__ __launch_bounds__(S::THREADS, 2) void matmul_tile_kernel(moe_ep_matmul_args a, int ntiles)
{
    __shared__ __align__(16) uint8_t lds[largest(S::STAGES * S::BYTES, (MORE::STAGES * MORE::BYTES)...)];
    // this tile's and the next one's
    __shared__ __align__(16) uint8_t scales[2][tile_scales<S, MORE...>()];
    constexpr int TALL = largest(S::BM, MORE::BM...), BM = TALL > 256 ? 256 : TALL;
    const TileFinder<BM, TALL> find(a, ntiles);
    int slot = (int)(blockIdx.x >> 3);
    Tile t = find.tile(a, slot);
    if (t.expert < 0)
        return;
    with_shape<S, MORE...>(t, [&](auto shape) { load_first<T, decltype(shape)>(a, t, lds, scales[0]); });
    for (int turn = 0; t.expert >= 0; turn ^= 1) {
        slot += (int)(gridDim.x >> 3);
        const Tile next = find.tile(a, slot);
        with_shape<S, MORE...>(t, [&](auto shape) {
            multiply_tile<T, decltype(shape)>(a, t, lds, scales[turn], [&] {
                if (next.expert >= 0)
                    with_shape<S, MORE...>(next, [&](auto ahead) {
                        load_first<T, decltype(ahead)>(a, next, lds, scales[turn ^ 1]);
                    });
            });
        });
        t = next;
    }
}

// As many workgroups as the LDS of 256 CUs holds, at most one a tile, in
// eight runs of the same length.
template <typename S, typename... MORE>
hipError_t tile_launch(const moe_ep_matmul_args &a, hipStream_t s)
{
    constexpr int kLds = largest(S::STAGES * S::BYTES, (MORE::STAGES * MORE::BYTES)...) + 2 * tile_scales<S, MORE...>();
    const int64_t ntiles = channel_tiles(a.n, S::BN);
    constexpr int TALL = largest(S::BM, MORE::BM...);
    const int64_t tiles = most_tiles(a, TALL > 256 ? 256 : TALL) * ntiles;
    if (tiles > INT32_MAX - 4096) // they are numbered in 32 bits, a run's last number and a step behind it too
        return hipErrorInvalidConfiguration;
    const int64_t run = (tiles + 7) / 8, resident = 32 * (160 * 1024 / kLds);
    const dim3 grid((unsigned)(8 * (run < resident ? run : resident))), block(S::THREADS);
    if (a.out_type == MOE_EP_BF16_ROWS)
        hipLaunchKernelGGL((matmul_tile_kernel<Bf16, S, MORE...>), grid, block, 0, s, a, (int)ntiles);
    else
        hipLaunchKernelGGL((matmul_tile_kernel<Fp32, S, MORE...>), grid, block, 0, s, a, (int)ntiles);
    return hipGetLastError();
}

} // namespace

// The shape follows from the average rows of an expert (of num_rows, which a
// caller's capacity may exceed) and from how many tiles there are for 256 CUs.
// Times in us, E experts of N x K, ragged rows:
//  - 256 channels x up to 256 or 320 rows, eight waves, one workgroup a CU:
//    the fewest bytes for its products; wins over 128 x 128 from about 112
//    rows on where there are tiles for the CUs.  E 32, 4096 x 4096: 96 rows
//    122 / 112, 112 rows 130 / 144, 256 rows 167 / 215, 512 rows 280 / 360,
//    1024 rows 532 / 644; E 32, 4096 x 1024: 256 rows 53 / 58, 512 rows
//    104 / 127; E 1, 7168 x 7168, 1024 rows (112 tiles) 78 / 57.  Not for
//    k below 1024: E 32, 2048 x 512, 192 rows 21 / 19, 512 rows 37 / 35.
//    With tiles of up to 256 rows only, an expert somewhat above that takes
//    two: E 32, 4096 x 4096, 256 rows 167 / 215, 512 rows 280 / 297.  The
//    320-row shape takes all 256 registers and spills 5 or 6 of them (24 or 28
//    bytes of scratch a lane); without it the kernel has 220 and spills none;
//  - up to 128 x 128, four waves, two workgroups a CU; for at most 32 rows an
//    expert its 64-row shape with three stages in place of two: E 32,
//    4096 x 4096, 1 row 66 / 76, but 64 rows 114 / 105;
//  - up to 64 x 64, four waves, three workgroups a CU, three stages, or four
//    for up to 32 rows: where 128 x 128 has not 200 tiles (E 1, 7168 x 7168,
//    256 rows 25 / 40, 1 row 13 / 33), and for a few rows against long
//    weights, where only the bytes in flight count (E 8, 4096 x 7168, 1 row
//    27 / 28; 64 rows over E 32, 4096 x 7168: 133 / 141).
hipError_t launch_expert_matmul(const moe_ep_matmul_args &a, hipStream_t s)
{
    using T64 = TileShape<2, 2, 2, 2, 3>;
    using T64Few = TileShape<2, 2, 2, 1, 4>;
    using T128 = TileShape<2, 2, 4, 4, 2>;
    const int64_t average = (a.num_rows + a.num_experts - 1) / a.num_experts;
    const auto tiles = [&](int64_t size) {
        return a.num_experts * ((average + size - 1) / size) * ((a.n + size - 1) / size);
    };
    if (tiles(128) < 200 || (average <= 8 && a.k >= 4096))
        return tile_launch<T64Few, T64>(a, s);
    if (average <= 32)
        return tile_launch<TileShape<2, 2, 4, 2, 3>, T128>(a, s);
    if (average >= 112 && tiles(256) >= 200 && a.k >= 1024)
        return tile_launch<TileShape<4, 2, 4, 2, 2>, TileShape<4, 2, 4, 4, 2>, TileShape<2, 4, 8, 3, 2>,
                           TileShape<2, 4, 8, 4, 2>, TileShape<2, 4, 8, 5, 2>>(a, s);
    return tile_launch<TileShape<2, 2, 4, 2, 2>, T128>(a, s);
}

} // namespace moe_ep
