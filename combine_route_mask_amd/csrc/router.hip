// gfx950 kernels of the router: the largest logits of each token with their
// softmax weights, and the gradient of the weights for the logits.  Up to 512
// experts 16 lanes (more than 16 places, or few tokens: 64) hold a token's logits
// in registers; beyond, a wave holds them in LDS.
//
// Large calls (a sort of each lane's, then a round for each place: 32768 tokens
// of 256 experts, 8 places, fp32 12.1 us, bf16 8.5; the bytes alone would take 5.8
// and 3.0): vector instructions issue in two thirds of the cycles in fp32, three
// quarters in bf16; the rest are waits that too few waves cover, since the fp32
// lists (34.8 KB of LDS for 16 logits a lane, 67.6 for 32) and registers leave a
// SIMD four waves, two with 32 logits a lane (half of the cycles issue there).
// The gradient takes 9.7 us, and about 9 its bytes, whole lines for 8 of 256 logits
// a token among them.
// The launch bounds small calls.  Beyond 512 experts every place reads the row
// again from LDS: 4096 tokens of 1024 experts, fp32, 8 places 31 us (gradient 6.5),
// of 4096 experts 182 (17).
#include <type_traits>

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

// ------------------------------------------------------------ a few logits a lane

typedef u32x4 Words4 __attribute__((aligned(4)));
typedef u32x2 Words2 __attribute__((aligned(2)));

// V consecutive logits from i on, those from E on as `other`.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const void *base, int64_t row, int i, int E, float other, float (&x)[V])
{
    if (V % 4 == 0 && i + V <= E) {
        const uint8_t *p = static_cast<const uint8_t *>(base) + (row + i) * RowType<T>::kBytes;
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            if (RowType<T>::kBytes == 2) {
                const u32x2 w = *reinterpret_cast<const Words2 *>(p + 2 * v);
                unpack_bf16x2(w[0], x[v % V], x[(v + 1) % V]);
                unpack_bf16x2(w[1], x[(v + 2) % V], x[(v + 3) % V]);
            } else {
                const u32x4 w = *reinterpret_cast<const Words4 *>(p + 4 * v);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[(v + e) % V] = __uint_as_float(w[e]);
            }
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        x[v] = i + v < E ? logit<T>(base, row + i + v) : other;
}

template <typename T, int V>
__device__ __forceinline__ void store_logits(void *base, int64_t row, int i, int E, const float (&x)[V])
{
    if (V % 4 == 0 && i + V <= E) {
        uint8_t *p = static_cast<uint8_t *>(base) + (row + i) * RowType<T>::kBytes;
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            const float f[8] = {x[v % V], x[(v + 1) % V], x[(v + 2) % V], x[(v + 3) % V], 0.0f, 0.0f, 0.0f, 0.0f};
            const u32x4 w = RowType<T>::pack(f);
            if (RowType<T>::kBytes == 2)
                *reinterpret_cast<Words2 *>(p + 2 * v) = u32x2{w[0], w[1]};
            else
                *reinterpret_cast<Words4 *>(p + 4 * v) = w;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (i + v < E)
            store_logit<T>(base, row + i + v, x[v]);
}

// Logit v of a lane where LANES lanes share a token's: fours in turn.
template <int LANES, int V>
__device__ __forceinline__ int spread(int lane, int v)
{
    return V < 4 ? lane : 4 * (v / 4 * LANES + lane) + v % 4;
}

template <typename T, int LANES, int V>
__device__ __forceinline__ void load_spread(const void *base, int64_t row, int lane, int E, float other, float (&x)[V])
{
    static_assert(V == 1 || V % 4 == 0);
    constexpr int N = V < 4 ? 1 : 4;
#pragma unroll
    for (int v = 0; v < V; v += N) {
        float f[N];
        load_logits<T, N>(base, row, spread<LANES, V>(lane, v), E, other, f);
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[v + i] = f[i];
    }
}

template <typename T, int LANES, int V>
__device__ __forceinline__ void store_spread(void *base, int64_t row, int lane, int E, const float (&x)[V])
{
    constexpr int N = V < 4 ? 1 : 4;
#pragma unroll
    for (int v = 0; v < V; v += N) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] = x[v + i];
        store_logits<T, N>(base, row, spread<LANES, V>(lane, v), E, f);
    }
}

// A wave's accesses of LDS before are done before those behind.
__device__ __forceinline__ void wave_order()
{
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#endif
}

// Smallest value of each 16 consecutive lanes, in all of them.
__device__ __forceinline__ uint32_t min16(uint32_t x)
{
    x = min(x, dpp<kDppXor1>(x));
    x = min(x, dpp<kDppXor2>(x));
    x = min(x, dpp<kDppMirror8>(x));
    return min(x, dpp<kDppMirror16>(x));
}

// Over the LANES (16 or 64) lanes of a token, in all of them.  Of a wave: rows of
// 16 hand theirs to the next, and the last lane has it; no LDS, whose latency
// each round would wait for.
template <int LANES>
__device__ __forceinline__ uint32_t token_max(uint32_t x)
{
    x = max16(x);
    if (LANES == 64) {
        constexpr int kBroadcast15 = 0x142, kBroadcast31 = 0x143;
        x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kBroadcast15, 0xA, 0xF, false));
        x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, kBroadcast31, 0xC, 0xF, false));
        x = (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
    }
    return x;
}

template <int LANES>
__device__ __forceinline__ float token_sum(float x)
{
    if (LANES == 64)
        return wave_sum(x);
    x += dpp<kDppXor1>(x);
    x += dpp<kDppXor2>(x);
    x += dpp<kDppMirror8>(x);
    return x + dpp<kDppMirror16>(x);
}

// A logit as a number that orders like it, 0 where it is never chosen.
__device__ __forceinline__ uint32_t order_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f); // -0 is 0
    return x > -INFINITY ? u ^ ((uint32_t)((int)u >> 31) | 0x80000000u) : 0;
}

__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// More than 16 places, or few tokens: each lane sorts its V logits once
// (neighbours change places only where the later one is larger, so that equal
// ones keep their order); in a round the lanes' first ones compete, the lowest
// lane wins of equal ones and moves up.  Lane j keeps place j.
template <typename T, int V>
__global__ __launch_bounds__(256) void route_lanes_kernel(moe_ep_route_args a)
{
    constexpr int LANES = 64, PER = 256 / LANES;
    const int E = a.num_experts, lane = threadIdx.x % LANES;
    for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < a.tokens; t0 += (int64_t)gridDim.x * PER) {
        const int64_t mine = t0 + threadIdx.x / LANES, t = min(mine, a.tokens - 1); // lanes without a token do the last's again
        float x[V];
        load_logits<T, V>(a.logits, t * E, lane * V, E, -INFINITY, x);
        uint32_t key[V], bad = 0;
        int id[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = order_of(x[v]);
            id[v] = lane * V + v;
            bad |= x[v] != x[v];
        }
#pragma unroll
        for (int pass = 0; pass < V; ++pass)
#pragma unroll
            for (int v = pass % 2; v + 1 < V; v += 2) {
                const bool turn = key[v + 1] > key[v];
                const uint32_t k = key[v];
                const int i = id[v];
                key[v] = turn ? key[v + 1] : k;
                id[v] = turn ? id[v + 1] : i;
                key[v + 1] = turn ? k : key[v + 1];
                id[v + 1] = turn ? i : id[v + 1];
            }
        uint32_t top = 0, kept = 0;
        int place = E;
        for (int j = 0; j < a.top_k; ++j) {
            const uint32_t best = token_max<LANES>(key[0]);
            const uint64_t ties = __ballot(key[0] == best);
            const int winner = __builtin_ctzll(ties);
            const int chosen = __builtin_amdgcn_readlane(id[0], winner);
            if (j == 0)
                top = best;
            if (lane == j) {
                kept = best;
                place = best ? chosen : E;
            }
            // bit by bit: selects of neighbours would become selects of their places
            const uint32_t pop = lane == winner ? 0xFFFFFFFFu : 0;
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) {
                key[v] = (key[v + 1] & pop) | (key[v] & ~pop);
                id[v] = (int)(((uint32_t)id[v + 1] & pop) | ((uint32_t)id[v] & ~pop));
            }
            key[V - 1] &= ~pop;
        }
        const float peak = value_of(top);
        const float e = kept ? expf(value_of(kept) - peak) : 0.0f;
        float total = e;
        if (!a.renormalize) {
            total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                total += expf(x[v] - peak);
        }
        total = token_sum<LANES>(total);
        const bool nan = token_max<LANES>(bad) != 0;
        if (lane < a.top_k && mine < a.tokens) {
            a.ids[t * a.top_k + lane] = place;
            a.weights[t * a.top_k + lane] = place == E ? 0.0f : nan ? nan_value() : a.scale * (e / total);
        }
    }
}

// A logit and its expert as one number, so that the larger one wins: of equal
// logits the lower expert's.  0 where it is never chosen.  fp32: a double in
// [1, 2) with the logit's order in the first 32 bits of its fraction, of which
// one instruction takes the larger; across lanes 32 bits at a time, the order
// and then the expert, cost less.  (32768 tokens of 256 experts: 12.0 us;
// doubles across lanes too 12.2, pairs of words in the sort too 14.2.)
template <typename T>
struct Ranked {
    double w;
    struct Head {
        uint32_t order, id;
        __device__ __forceinline__ bool any() const { return order != 0; }
        __device__ __forceinline__ bool operator==(const Head &o) const { return order == o.order && id == o.id; }
        __device__ __forceinline__ Head best() const
        {
            const uint32_t k = max16(order);
            return {k, min16(order == k ? id : 0xFFFFFFFFu)};
        }
        __device__ __forceinline__ int expert() const { return (int)id; }
        __device__ __forceinline__ float value() const { return value_of(order); }
    };
    static __device__ __forceinline__ Ranked of(float x, int id)
    {
        const uint32_t k = order_of(x);
        const uint64_t u = (uint64_t)(0x3FF00000u | k >> 12) << 32 | (k << 20 | (0xFFFFFu - (uint32_t)id));
        return {k ? __builtin_bit_cast(double, u) : 0.0};
    }
    __device__ __forceinline__ Head head() const
    {
        const uint64_t u = __builtin_bit_cast(uint64_t, w);
        return {(uint32_t)(u >> 20), 0xFFFFFu - ((uint32_t)u & 0xFFFFFu)};
    }
    __device__ __forceinline__ Ranked larger(const Ranked &o) const
    {
        double y; // the builtin would first turn signalling NaNs into quiet ones
        asm("v_max_f64 %0, %1, %2" : "=v"(y) : "v"(w), "v"(o.w));
        return {y};
    }
    __device__ __forceinline__ Ranked smaller(const Ranked &o) const
    {
        double y;
        asm("v_min_f64 %0, %1, %2" : "=v"(y) : "v"(w), "v"(o.w));
        return {y};
    }
};

template <>
struct Ranked<Bf16> { // order and expert, 16 bits each
    uint32_t w;
    struct Head {
        uint32_t w;
        __device__ __forceinline__ bool any() const { return w != 0; }
        __device__ __forceinline__ bool operator==(const Head &o) const { return w == o.w; }
        __device__ __forceinline__ Head best() const { return {max16(w)}; }
        __device__ __forceinline__ int expert() const { return (int)(0xFFFFu - (w & 0xFFFFu)); }
        __device__ __forceinline__ float value() const { return __uint_as_float(__float_as_uint(value_of(w)) & 0xFFFF0000u); }
    };
    static __device__ __forceinline__ Ranked of(float x, int id)
    {
        const uint32_t k = order_of(x) & 0xFFFF0000u; // not 0 for a number
        return {k ? k | (0xFFFFu - (uint32_t)id) : 0};
    }
    __device__ __forceinline__ Head head() const { return {w}; }
    __device__ __forceinline__ Ranked larger(const Ranked &o) const { return {max(w, o.w)}; }
    __device__ __forceinline__ Ranked smaller(const Ranked &o) const { return {min(w, o.w)}; }
};

// Batcher's network, largest first.
template <int V, typename R>
__device__ __forceinline__ void sort_down(R (&r)[V])
{
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int i = 0; i + k < V; ++i)
                if (i >= k % p && (i - k % p) / k % 2 == 0 && i / (2 * p) == (i + k) / (2 * p)) {
                    const R a = r[i], b = r[i + k];
                    r[i] = a.larger(b);
                    r[i + k] = a.smaller(b);
                }
}

// Sixteen lanes a token, four tokens a wave.  A lane sorts its logits once and
// keeps them in LDS, in its own column; in a round the lanes' first ones
// compete, and the winner's lane reads its next.  Lane j keeps place j.  (A lane
// of 64 with four or eight logits, sorted and moved up in registers, as for
// more places: 32768 tokens of 256 experts 17.6 us against 12.1, bf16 17.3
// against 8.5; 16384 of 384 bf16 16.0 / 9.2; only one place of 384 is faster so,
// 8.7 / 11.7.)
template <typename T, int V>
__global__ __launch_bounds__(256) void route_sorted_kernel(moe_ep_route_args a)
{
    typedef Ranked<T> R;
    __shared__ typename R::Head list[V + 1][256];
    const int E = a.num_experts, lane = threadIdx.x & 15;
    for (int64_t t0 = (int64_t)blockIdx.x * 16; t0 < a.tokens; t0 += (int64_t)gridDim.x * 16) {
        const int64_t mine = t0 + threadIdx.x / 16, t = min(mine, a.tokens - 1); // lanes without a token do the last's again
        float x[V];
        load_spread<T, 16, V>(a.logits, t * E, lane, E, -INFINITY, x);
        R r[V];
        uint32_t bad = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            r[v] = R::of(x[v], spread<16, V>(lane, v));
            bad |= x[v] != x[v];
        }
        sort_down<V>(r);
#pragma unroll
        for (int v = 0; v < V; ++v)
            list[v][threadIdx.x] = r[v].head();
        list[V][threadIdx.x] = {}; // never chosen
        auto head = r[0].head();
        decltype(head) top = {}, kept = {};
        int at = 0;
        for (int j = 0; j < a.top_k; ++j) {
            const auto best = head.best();
            if (j == 0)
                top = best;
            if (lane == j)
                kept = best;
            at += head.any() && head == best; // no further than the last
            head = list[at][threadIdx.x];
        }
        const int place = kept.any() ? kept.expert() : E;
        const float peak = top.value();
        const float e = kept.any() ? expf(kept.value() - peak) : 0.0f;
        float total = e;
        if (!a.renormalize) {
            total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v)
                total += expf(x[v] - peak);
        }
        total = token_sum<16>(total);
        const bool nan = token_max<16>(bad) != 0;
        if (lane < a.top_k && mine < a.tokens) {
            a.ids[t * a.top_k + lane] = place;
            a.weights[t * a.top_k + lane] = place == E ? 0.0f : nan ? nan_value() : a.scale * (e / total);
        }
    }
}

// Over the chosen experts the others' logits are not read (half of the bytes), so
// a NaN among them does not reach the gradient.
// The chosen experts' places go through LDS, a wave's own part of it.  (32768
// tokens of 256 experts, 8 places: 9.7 us, a wave a token 12.9; over all experts
// 14.5, with the places compared in registers 18.5.)
template <typename T, int LANES, int V>
__global__ __launch_bounds__(256) void route_lanes_backward_kernel(moe_ep_route_grad_args a)
{
    constexpr int PER = 256 / LANES;
    __shared__ __align__(16) float places[256 * V];
    const int E = a.num_experts, lane = threadIdx.x % LANES;
    float *place = places + threadIdx.x / LANES * (LANES * V);
    for (int64_t t0 = (int64_t)blockIdx.x * PER; t0 < a.tokens; t0 += (int64_t)gridDim.x * PER) {
        const int64_t mine = t0 + threadIdx.x / LANES, t = min(mine, a.tokens - 1);
        int id = E;
        float g = 0.0f;
        if (lane < a.top_k) {
            id = a.ids[t * a.top_k + lane];
            g = a.grad_weights[t * a.top_k + lane];
        }
        const bool held = id >= 0 && id < E;
        const float chosen = held ? logit<T>(a.logits, t * E + id) : -INFINITY;
        float x[V];
        float top = chosen;
        if (!a.renormalize) {
            load_spread<T, LANES, V>(a.logits, t * E, lane, E, -INFINITY, x);
#pragma unroll
            for (int v = 0; v < V; ++v)
                top = fmaxf(top, x[v]);
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            place[spread<LANES, V>(lane, v)] = 0.0f;
        const uint32_t peak_key = token_max<LANES>(order_of(top));
        const float peak = peak_key ? value_of(peak_key) : 0.0f;
        const float e = held ? expf(chosen - peak) : 0.0f;
        float total = e;
        if (!a.renormalize) {
            total = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                x[v] = expf(x[v] - peak);
                total += x[v];
            }
        }
        total = token_sum<LANES>(total);
        const float by = total != 0.0f ? 1.0f / total : 0.0f;
        const float mean = token_sum<LANES>(held ? e * by * g : 0.0f);
        // what an expert's place gives: the gradient, or its part of it
        wave_order();
        if (held)
            place[id] = a.renormalize ? a.scale * (e * by) * (g - mean) : g;
        wave_order();
        float d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            d[v] = place[spread<LANES, V>(lane, v)];
            if (!a.renormalize)
                d[v] = a.scale * (x[v] * by) * (d[v] - mean);
        }
        if (mine < a.tokens)
            store_spread<T, LANES, V>(a.grad_logits, t * E, lane, E, d);
        wave_order();
    }
}

// ------------------------------------------------------------ logits in LDS

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

// Calls f(lanes, logits a lane) for the kernels in registers, or returns false.
// A few tokens of many experts leave SIMDs without a wave: 64 lanes a token then
// (in a graph, 64 lanes / 16, 256 experts fp32: one token 2.8 / 3.8 us, 2048
// 3.5 / 4.1, 4096 4.3 / 4.1, 8192 6.2 / 4.8; 384 bf16: 3.4 / 4.7, 4.8 / 5.1, 6.5 /
// 5.1, 9.8 / 6.1; 64 fp32: 2.3 / 2.4, 2.9 / 2.7, 3.4 / 2.8, 4.6 / 2.9).
template <typename F>
bool with_lanes(int64_t tokens, int experts, int top_k, F f)
{
    using std::integral_constant;
    if (experts <= 512 && top_k <= 16 && (experts <= 64 || tokens > 2048)) {
        if (experts <= 16)
            f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
        else if (experts <= 64)
            f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
        else if (experts <= 256)
            f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
        else
            f(integral_constant<int, 16>{}, integral_constant<int, 32>{});
    } else if (experts <= 64) {
        f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    } else if (experts <= 256) {
        f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
    } else if (experts <= 512) {
        f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    } else {
        return false;
    }
    return true;
}

template <typename T>
hipError_t route_launch(const moe_ep_route_args &a, hipStream_t s)
{
    if (!with_lanes(a.tokens, a.num_experts, a.top_k, [&](auto lanes, auto logits) {
            constexpr int L = decltype(lanes)::value, V = decltype(logits)::value;
            const dim3 grid = tokens_grid((a.tokens + 256 / L - 1) / (256 / L));
            if constexpr (L == 16)
                hipLaunchKernelGGL((route_sorted_kernel<T, V>), grid, dim3(256), 0, s, a);
            else
                hipLaunchKernelGGL((route_lanes_kernel<T, V>), grid, dim3(256), 0, s, a);
        }))
        hipLaunchKernelGGL(route_kernel<T>, tokens_grid(a.tokens), dim3(64), 4 * a.num_experts, s, a);
    return hipGetLastError();
}

template <typename T>
hipError_t route_backward_launch(const moe_ep_route_grad_args &a, hipStream_t s)
{
    if (!with_lanes(a.tokens, a.num_experts, a.top_k, [&](auto lanes, auto logits) {
            constexpr int L = decltype(lanes)::value, V = decltype(logits)::value;
            hipLaunchKernelGGL((route_lanes_backward_kernel<T, L, V>), tokens_grid((a.tokens + 256 / L - 1) / (256 / L)),
                               dim3(256), 0, s, a);
        }))
        hipLaunchKernelGGL(route_backward_kernel<T>, tokens_grid(a.tokens), dim3(64), 4 * a.num_experts, s, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_route_top_k(const moe_ep_route_args &a, hipStream_t s)
{
    return a.row_type == MOE_EP_BF16_ROWS ? route_launch<Bf16>(a, s) : route_launch<Fp32>(a, s);
}

hipError_t launch_route_top_k_backward(const moe_ep_route_grad_args &a, hipStream_t s)
{
    return a.row_type == MOE_EP_BF16_ROWS ? route_backward_launch<Bf16>(a, s) : route_backward_launch<Fp32>(a, s);
}

} // namespace moe_ep
