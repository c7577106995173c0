// gfx950 kernels of the bf16 products over experts: rows times weights in
// either order of the weights' axes, with the gated block's epilogues, and the
// weights' gradient.  Products on the matrix cores, sums in fp32.
//
// v_mfma_f32_16x16x32_bf16: lane l holds 8 elements of row l % 16 at
// k = 8 * (l / 16) of either matrix; of the result, element i is left row
// 4 * (l / 16) + i and right row l % 16.  The left matrix is the channels',
// the right one the rows' (of the weights' gradient: x's columns and
// grad_out's columns, summed over the rows).
//
// All of them are one loop over tiles whose operands lie in memory either
// along k (an operand's row after another, k next to k) or across it (a k
// after another).  An operand across k goes into LDS as it lies and is turned
// by the transposing LDS read.
//
// The matrix cores bound large calls: 8192^3 takes 772 us along k, 784 across
// (rows times weights) and 786 (weights' gradient) back to back, 1.4 PFLOP/s.
// That is 1.5 M cycles, the cores busy for 1.05 M of them, with no LDS bank
// conflict; the clock follows the load (1.9 GHz at 772 us; counted and traced
// launches of 790 to 980 us ran at 1.5 to 1.9).
// Ragged experts lose a fifth of that to whole tiles of 256 CUs, the weights'
// gradient of few rows to its stores; memory bounds a few rows an expert (5.9
// TB/s of weights). Two workgroups a CU of 256 x 128 tiles, 32 of k a stage in
// three of them, overlap one's stores with the other's products, but take 926
// to 1080 us for 8192^3 and no less for the gradient of 32 experts of 512 rows.
//
// The 256-wide products need more than the 256 registers of a lane at a tile's
// beginning and end: by the compiler's report 52 (gated), 92 and 104 (along and
// across) and 264 bytes (gated backward) of a lane go to memory there, none in
// the loop over k.  The other shapes and the weights' gradient have none.
//
// Results are rounded to bf16 once, from the fp32 sums: they are the next
// product's operand, which has to be bf16 for the matrix cores (fp32 runs at a
// sixteenth of the rate), and half the bytes.  Between a layer's operators that
// makes five such roundings (activation, y, the first product's gradient, the
// activation again, the rows' gradient): the layer's outputs are 0.0033 off the
// 64-bit ones (norm of the difference over the norm), where one rounding of the
// outputs alone leaves 0.0017.
#include "ffn_internal.h"
#include "product_shapes.h"
#include "rows.h"
#include "tiles.h"

namespace moe_ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum Epilogue { kStore, kGated, kGatedBackward };

struct Job {
    const uint8_t *x, *w; // bf16
    const int32_t *offsets;
    uint16_t *out;        // product, activation
    void *pre;            // what the gated block saves or reads
    uint8_t *pre_scales;
    uint16_t *grad_pre;
    int64_t num_rows;
    int num_experts, n, k, save;
    bool zero_rest;
};

// A workgroup takes BN channels and BM rows, 64 elements of k at a time,
// through STAGES of LDS: the next stages go from memory straight into LDS
// while this one is multiplied.  NW x MW waves, each FN x FM results of
// 16 x 16.
constexpr int kDepth = 64, kDepthBytes = 2 * kDepth;

template <int NW_, int MW_, int FN_, int FM_, int STAGES_>
struct TileShape {
    static constexpr int NW = NW_, MW = MW_, FN = FN_, FM = FM_, STAGES = STAGES_, W = NW * MW;
    static constexpr int BN = NW * FN * 16, BM = MW * FM * 16, THREADS = 64 * W;
    static constexpr int LN = BN / (8 * W), LM = BM / (8 * W); // loads of a thread and stage, 1024 bytes a wave
    static constexpr int BYTES = (BN + BM) * kDepthBytes;
    static_assert(BN % (8 * W) == 0 && BM % (8 * W) == 0 && (FN & (FN - 1)) == 0);
};

// Where a tile's operand of EDGE rows lies in memory, for this thread's L loads
// of a stage, and in LDS, for its fragments.
//
// Along k: an LDS row is 128 bytes of k of one operand row, all on the same
// banks: chunk c (16 bytes) of row r lies at place c ^ (r & 7), so that 8 rows'
// reads of one chunk cover all banks.
//
// Across k: an LDS row is one k of all EDGE operand rows.  A transposing read
// takes, for 16 operand rows (32 bytes), four consecutive k in each 16 lanes;
// unit u (32 bytes) of row r lies at place u ^ turn(r), so that the rows of a
// read lie on different banks.
//
// HALF (along): LDS rows go by turns of HALF rows to two parts of the operand,
// `second` bytes apart.
template <bool ACROSS, int EDGE, int L, int W, int HALF = 0>
struct Operand {
    static_assert(HALF % 8 == 0);
    static constexpr int kPitch = 2 * EDGE; // bytes of an LDS row across k
    const uint8_t *base;
    uint32_t offset[L];
    uint32_t stride;  // bytes of a memory row
    int64_t second;
    uint32_t end;     // along: kPastEnd where the lane's chunk of the last step is past the end of k
    int depth;        // across: elements of k
    uint32_t at[2];   // along: the first fragment's place of either half of a step; across: at[0]

    static __device__ __forceinline__ int turn(int k)
    {
        static_assert(!ACROSS || EDGE % 64 == 0);
        if constexpr (EDGE % 128 == 0)
            return (k & 3) | ((k >> 3) & 1) << 2;
        else // two rows of k are 256 bytes
            return ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
    }

    // `first`: of the operand's row 0 at k = 0.  `rows` of them there are, and
    // `map(r)` is the row that LDS row (or column) r holds; rows past the last
    // read another one's, and their results are not stored.  `fragment`: the
    // wave's first one.
    template <typename MAP>
    __device__ __forceinline__ void find(const uint8_t *first, uint32_t stride_, int k, int wave, int fragment, MAP map)
    {
        const int lane = threadIdx.x & 63, l16 = lane & 15, l4 = lane >> 4;
        base = first;
        stride = stride_;
        depth = k;
        end = 0;
        if constexpr (!ACROSS) {
            const int sub = lane / 8;
            const uint32_t chunk = (uint32_t)((lane % 8) ^ sub) * 16;
#pragma unroll
            for (int i = 0; i < L; ++i)
                offset[i] = (uint32_t)map((i * W + wave) * 8 + sub) * stride + chunk;
            const int steps = (k + kDepth - 1) / kDepth;
            end = (steps - 1) * kDepthBytes + chunk < (uint32_t)(2 * k) ? 0 : kPastEnd;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                at[h] = (uint32_t)(((h * 4 + l4) ^ (l16 & 7)) * 16 + (16 * fragment + l16) * kDepthBytes);
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int byte = (i * W + wave) * 1024 + lane * 16, row = byte / kPitch;
                const int chunk = (byte % kPitch / 16) ^ (2 * turn(row));
                offset[i] = (uint32_t)row * stride + 16 * (uint32_t)map(chunk);
            }
            const int row = 8 * l4 + l16 / 4;
            at[0] = (uint32_t)(row * kPitch + l16 % 4 * 8 + (fragment ^ turn(row)) * 32);
            at[1] = 0;
        }
    }

    // Load i of step `step` (of `steps`; later ones bring nothing).
    __device__ __forceinline__ void load(uint8_t *part, int wave, int i, int step, int steps, bool past) const
    {
#if defined(__HIP_DEVICE_COMPILE__) // the host compiler does not know the resource type
        uint8_t *to = part + (i * W + wave) * 1024;
        int64_t ahead = ACROSS ? (int64_t)step * kDepth * stride : (int64_t)step * kDepthBytes;
        if constexpr (HALF > 0)
            ahead += (i * W + wave) * 8 / HALF % 2 ? second : 0;
        // rows of k past the end are beyond the buffer: zeros
        const int left = ACROSS ? min(depth - step * kDepth, kDepth) * (int)stride : 0x7FFFFFFF;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base + ahead), 0,
                                                                              past ? 0 : left, 0x00027000);
        const uint32_t tail = !ACROSS && step == steps - 1 ? end : 0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 16, offset[i] | tail, 0,
                                                 0, 0);
#endif
    }

    // Across: at[0] as something new in each step, so that the fragments'
    // places, which differ in the bits of their unit, are made anew and take no
    // registers.
    __device__ __forceinline__ uint32_t place() const
    {
        uint32_t x = at[0];
        if constexpr (ACROSS)
            asm volatile("" : "+v"(x));
        return x;
    }

    // Fragment i of the wave, half h of the step.  Nothing writes the stage
    // within a read, and __restrict__ says so: without it each transposing read
    // is made to wait for all loads on their way to LDS, wherever to.
    // wait_barrier() orders reads and loads.
    __device__ __forceinline__ bf16x8 read(const uint8_t *__restrict__ part, uint32_t place, int h, int i) const
    {
        bf16x8 v = {};
        if constexpr (!ACROSS) {
            v = *reinterpret_cast<const bf16x8 *>(part + at[h] + 16 * i * kDepthBytes);
        } else {
#if defined(__HIP_DEVICE_COMPILE__)
            typedef __attribute__((address_space(3))) s16x4 *lds;
            const uint8_t *p = part + (place ^ 32 * i) + h * 32 * kPitch;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)p);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(p + 4 * kPitch));
            v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
#endif
        }
        return v;
    }
};

// A tile's operands: weights, or x's columns, and rows, or grad_out's columns.
template <typename S, bool ACROSS_A, bool ACROSS_B, int HALF = 0>
struct Operands {
    Operand<ACROSS_A, S::BN, S::LN, S::W, HALF> a;
    Operand<ACROSS_B, S::BM, S::LM, S::W> b;
    int wave, steps, start; // steps of k, and the first of them

    __device__ __forceinline__ void load_part(uint8_t *stage, int i, int step, bool past) const
    {
        if (i < S::LN)
            a.load(stage, wave, i, step, steps, past);
        else
            b.load(stage + S::BN * kDepthBytes, wave, i - S::LN, step, steps, past);
    }

    __device__ __forceinline__ void load_first(uint8_t *lds) const
    {
#pragma unroll
        for (int st = 0; st < S::STAGES; ++st)
#pragma unroll
            for (int i = 0; i < S::LN + S::LM; ++i)
                load_part(lds + st * S::BYTES, i, (start + st) % steps, st >= steps);
    }
};

template <typename S>
struct Fragments {
    bf16x8 b[2][S::FM], a[2 * S::FN];
};

constexpr int kAhead = 2; // left fragments are read this many products before they are used

// The products of stage `cur`, groups of FM.  The first kAhead fragments are
// in registers already; the last groups run behind the barrier and read the
// first of `next`, so that neither LDS nor the barrier leaves the matrix
// cores idle for long.  Behind it `cur`, which no wave reads again, takes the
// loads for STAGES steps on: they have at least a whole step to arrive.
// wait_barrier() orders them behind the reads before it, and waits for the loads
// that the reads behind it need.
template <typename S, typename O>
__device__ __forceinline__ void tile_step(uint8_t *cur, const uint8_t *next, int step, bool past, const O &o,
                                          Fragments<S> &f, f32x4 (&acc)[S::FN][S::FM], Fragments<S> &g)
{
    constexpr int G = 2 * S::FN, L = S::LN + S::LM, FIRST = S::FN - S::FM - kAhead + 1, B = S::BN * kDepthBytes;
    const uint32_t pa = o.a.place(), pb = o.b.place();
#pragma unroll
    for (int i = 0; i < G; ++i) {
        if (i + kAhead < G)
            f.a[i + kAhead] = o.a.read(cur, pa, (i + kAhead) / S::FN, (i + kAhead) % S::FN);
#pragma unroll
        for (int j = 0; j < S::FM; ++j) // the second half's rows, spread before its first product
            if (i == (FIRST + j > 0 ? FIRST + j : 0))
                f.b[1][j] = o.b.read(cur + B, pb, 1, j);
        if (i == G - kAhead)
            wait_barrier<(S::STAGES - 2) * L>(); // this stage is read, the next one has arrived
        __builtin_amdgcn_sched_barrier(0);
        if (i >= G - kAhead) {
            g.a[i - (G - kAhead)] = o.a.read(next, pa, (i - (G - kAhead)) / S::FN, (i - (G - kAhead)) % S::FN);
#pragma unroll
            for (int j = 0; j < S::FM; ++j)
                if (j % kAhead == i - (G - kAhead))
                    g.b[0][j] = o.b.read(next + B, pb, 0, j);
#pragma unroll
            for (int u = 0; u < L; ++u)
                if (u * kAhead / L == i - (G - kAhead))
                    o.load_part(cur, u, step, past);
        }
#pragma unroll
        for (int j = 0; j < S::FM; ++j)
            acc[i % S::FN][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[i], f.b[i / S::FN][j], acc[i % S::FN][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
    // the fragments read ahead
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        f.a[i] = g.a[i];
#pragma unroll
    for (int j = 0; j < S::FM; ++j)
        f.b[0][j] = g.b[0][j];
}

// The sums of a tile whose first stages are on their way.  Behind it all waves
// are done with LDS, and nothing is on its way there.
template <typename S, typename O>
__device__ __forceinline__ void multiply(const O &o, uint8_t *lds, f32x4 (&acc)[S::FN][S::FM])
{
    Fragments<S> f, g;
    uint8_t *cur = lds, *next = lds + S::BYTES;
    wait_barrier<(S::STAGES - 1) * (S::LN + S::LM)>();
#pragma unroll
    for (int j = 0; j < S::FM; ++j)
        f.b[0][j] = o.b.read(cur + S::BN * kDepthBytes, o.b.at[0], 0, j);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        f.a[i] = o.a.read(cur, o.a.at[0], i / S::FN, i % S::FN);
    int at = (o.start + S::STAGES) % o.steps;
    // the loads behind the last step are not read, nor do they reach memory
    for (int i = 0; i < o.steps; ++i) {
        tile_step<S>(cur, next, at, i >= o.steps - S::STAGES, o, f, acc, g);
        at = at + 1 == o.steps ? 0 : at + 1;
        cur = next;
        next = next == lds + (S::STAGES - 1) * S::BYTES ? lds : next + S::BYTES;
    }
    wait_barrier<0>();
}

// Two neighbouring fragments' sums of a row as eight consecutive channels: a
// lane holds channels 4 (l / 16) .. + 3 of either fragment, and exchanges four
// with a lane of the next or the last 16.  They begin at channel eighth(lane)
// of the 32.
__device__ __forceinline__ void eight(const f32x4 &a, const f32x4 &b, float *f)
{
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[e]), __float_as_uint(b[e]), false, false);
        f[e] = __uint_as_float(s[0]);
        f[4 + e] = __uint_as_float(s[1]);
    }
#endif
}

__device__ __forceinline__ int eighth(int lane) { return (lane >> 4 & 1) * 16 + (lane >> 5) * 8; }

// Two such pairs of fragments, 32 channels apart, as whole lines of memory: p
// becomes the first eight rows' 64 channels, the lanes l % 16 >= 8 holding the
// second pair's, and q the last eight rows'.
__device__ __forceinline__ void whole_lines(float *p, float *q)
{
    constexpr int kRotate8 = 0x128; // within 16 lanes
    const bool low = (threadIdx.x & 8) == 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float other = dpp<kRotate8>(low ? q[e] : p[e]);
        p[e] = low ? p[e] : other;
        q[e] = low ? other : q[e];
    }
}

// Row and channel (of the wave's) of a lane's eight number i of j.
template <bool LINES>
__device__ __forceinline__ void eight_place(int i, int j, int &row, int &channel)
{
    const int lane = threadIdx.x & 63;
    row = 16 * j + (LINES ? i % 2 * 8 + (lane & 7) : lane & 15);
    channel = (LINES ? i / 2 * 64 + (lane & 8) * 4 : 32 * i) + eighth(lane);
}

// The sums of fragments [from, from + F) of j as calls f(row, channel, eight
// values).  LINES: F is a multiple of 4, and a store of all lanes' values fills
// whole lines.
template <int F, bool LINES, typename ACC, typename FN>
__device__ __forceinline__ void each_eight(ACC &acc, int from, int j, FN f)
{
    const int lane = threadIdx.x & 63;
    float p[8], q[8];
    if constexpr (!LINES) {
#pragma unroll
        for (int i = 0; i < F; i += 2) {
            eight(acc[from + i][j], acc[from + i + 1][j], p);
            f(16 * j + (lane & 15), 16 * i + eighth(lane), p);
        }
    } else {
#pragma unroll
        for (int i = 0; i < F; i += 4) {
            eight(acc[from + i][j], acc[from + i + 1][j], p);
            eight(acc[from + i + 2][j], acc[from + i + 3][j], q);
            whole_lines(p, q);
            const int channel = 16 * i + (lane & 8) * 4 + eighth(lane);
            f(16 * j + (lane & 7), channel, p);
            f(16 * j + 8 + (lane & 7), channel, q);
        }
    }
}

__device__ __forceinline__ void store8(uint16_t *to, const float *f)
{
    *reinterpret_cast<u32x4 *>(to) = RowType<Bf16>::pack(f);
}

// Past the caches: the results of all workgroups of a round come at a time, and
// whole lines leave L2 to the operands (gradient of 32 experts' weights of
// 2048 x 4096: 366 -> 308 us; the gated backward of 8191 rows 174 -> 164 us; the
// gated product, whose results the next product reads, is slower so, 249 -> 255
// us).
__device__ __forceinline__ void store8_nt(uint16_t *to, const float *f)
{
    store16_nt(to, RowType<Bf16>::pack(f));
}

// Eight channels `at` of the first product's row as the backward pass reads
// them: fp16 over a power of two of their own, or MXFP8, whose blocks of 32 the
// four lanes of a row hold.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void save8(const Job &a, int64_t at, const float *f, bool in)
{
    uint32_t top = 0;
    if (a.save == MOE_EP_SAVE_HALF) {
        // of the finite ones: an infinity or NaN stays what it is at any scale
#pragma unroll
        for (int i = 0; i < 8; ++i)
            top = max(top, magnitude(f[i]) < kInfinity ? magnitude(f[i]) : 0);
        const uint32_t b = min(max(top >> 23, 1u), 253u);
        const float by = __uint_as_float((254 - b) << 23);
        f16x8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (_Float16)(f[i] * by);
        if (in) {
            *reinterpret_cast<f16x8 *>(static_cast<uint16_t *>(a.pre) + at) = v;
            a.pre_scales[at / 8] = (uint8_t)b;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, magnitude(f[i]));
    top = max_of_rows(top);
    uint8_t scale;
    const u32x2 codes = mx_codes(f, top, scale);
    if (!in)
        return;
    *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.pre) + at) = codes;
    if (at % 32 == 0)
        a.pre_scales[at / 32] = scale;
}

// Eight gate and eight up values of the first product as they were saved.
struct Saved {
    u32x4 gate, up;            // MXFP8: the first two words
    uint32_t gate_scale, up_scale;
    __device__ __forceinline__ void load(const Job &a, int64_t at, int I)
    {
        if (a.save == MOE_EP_SAVE_HALF) {
            gate = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.pre) + at);
            up = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.pre) + at + I);
            gate_scale = a.pre_scales[at / 8];
            up_scale = a.pre_scales[(at + I) / 8];
        } else {
            const uint8_t *p = static_cast<const uint8_t *>(a.pre) + at;
            const u32x2 g = *reinterpret_cast<const u32x2 *>(p), u = *reinterpret_cast<const u32x2 *>(p + I);
            gate = u32x4{g[0], g[1], 0, 0};
            up = u32x4{u[0], u[1], 0, 0};
            gate_scale = a.pre_scales[at / 32];
            up_scale = a.pre_scales[(at + I) / 32];
        }
    }
    __device__ __forceinline__ void values(const Job &a, float *g, float *u) const
    {
        const float gs = e8m0_value(gate_scale), us = e8m0_value(up_scale);
        if (a.save == MOE_EP_SAVE_HALF) {
            const f16x8 gv = __builtin_bit_cast(f16x8, gate), uv = __builtin_bit_cast(f16x8, up);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                g[i] = (float)gv[i] * gs;
                u[i] = (float)uv[i] * us;
            }
        } else {
            mx_values(u32x2{gate[0], gate[1]}, gs, g);
            mx_values(u32x2{up[0], up[1]}, us, u);
        }
    }
};

// ------------------------------------------------------------ rows times weights

// A gated wave's first fragments are gate channels, the others the same
// channels of up.
template <int EPI, bool ACROSS, typename S>
using ProductOperands = Operands<S, ACROSS, false, EPI == kGated ? 8 * S::FN : 0>;

template <int EPI, bool ACROSS, typename S>
__device__ __forceinline__ ProductOperands<EPI, ACROSS, S> find_operands(const Job &a, const Tile &t)
{
    ProductOperands<EPI, ACROSS, S> o;
    o.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint8_t *w = a.w + (int64_t)t.expert * a.n * a.k * 2;
    const int wn = o.wave % S::NW, wm = o.wave / S::NW;
    if constexpr (EPI == kGated) {
        constexpr int HALF = S::FN * 8;
        const int I = a.n / 2, n0 = t.n * (S::BN / 2), last = I - n0 - 1;
        o.a.find(w + (int64_t)n0 * a.k * 2, 2 * a.k, a.k, o.wave, wn * S::FN,
                 [&](int r) { return min(r / (2 * HALF) * HALF + r % HALF, last); });
        o.a.second = (int64_t)I * a.k * 2;
    } else {
        const int n0 = t.n * S::BN, last = a.n - n0 - 1;
        if constexpr (ACROSS)
            o.a.find(w + 2 * n0, 2 * a.n, a.k, o.wave, wn * S::FN, [&](int c) { return min(c, last / 8); });
        else
            o.a.find(w + (int64_t)n0 * a.k * 2, 2 * a.k, a.k, o.wave, wn * S::FN, [&](int r) { return min(r, last); });
    }
    const int last = (int)(t.last - t.first) - 1;
    o.b.find(a.x + t.first * a.k * 2, 2 * a.k, a.k, o.wave, wm * S::FM, [&](int r) { return min(r, last); });
    o.steps = (a.k + kDepth - 1) / kDepth;
    // k starts elsewhere in each channel tile and goes round: rows a power of
    // two apart would otherwise have all workgroups read the same few memory
    // channels at a time
    o.start = (int)(((uint32_t)t.expert * (uint32_t)channel_tiles(a.n, S::BN) + (uint32_t)t.n) % (uint32_t)o.steps);
    return o;
}

template <int EPI, bool ACROSS, typename S, typename AHEAD>
__device__ __forceinline__ void multiply_tile(const Job &a, const Tile &t, uint8_t *lds, AHEAD ahead)
{
    const auto o = find_operands<EPI, ACROSS, S>(a, t);
    f32x4 acc[S::FN][S::FM] = {};
    multiply<S>(o, lds, acc);
    ahead();
    constexpr int F = EPI == kGated ? S::FN / 2 : S::FN; // fragments of channels of the output
    const int N = EPI == kGated ? a.n / 2 : a.n, n0 = (t.n * S::NW + o.wave % S::NW) * F * 16;
    const int64_t m0 = t.first + o.wave / S::NW * S::FM * 16;
    [[maybe_unused]] Saved saved[F / 2];
    [[maybe_unused]] const auto load_saved = [&](int i, int j) {
        int row, channel;
        eight_place<F % 4 == 0>(i, j, row, channel);
        // of rows and channels past the last, the last ones'
        saved[i].load(a, min(m0 + row, t.last - 1) * 2 * N + min(n0 + channel, N - 8), N);
    };
    if constexpr (EPI == kGatedBackward) {
#pragma unroll
        for (int i = 0; i < F / 2; ++i)
            load_saved(i, 0);
    }
#pragma unroll
    for (int j = 0; j < S::FM; ++j) {
        if constexpr (EPI == kGated) {
            // gate and up come one after the other
            float gate[F][8];
            int at = 0;
            each_eight<F, false>(acc, 0, j, [&](int, int, const float *f) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    gate[at][e] = f[e];
                ++at;
            });
            at = 0;
            each_eight<F, false>(acc, F, j, [&](int row, int channel, const float *u) {
                const int64_t m = m0 + row;
                const int n = n0 + channel;
                const float *g = gate[at++];
                const bool in = m < t.last && n < N;
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    y[e] = g[e] / (1.0f + __expf(-g[e])) * u[e];
                if (in)
                    store8(a.out + m * N + n, y);
                if (a.save != MOE_EP_SAVE_NONE) {
                    save8(a, m * 2 * N + n, g, in);
                    save8(a, m * 2 * N + N + n, u, in);
                }
            });
        } else if constexpr (EPI == kStore) {
            each_eight<F, F % 4 == 0>(acc, 0, j, [&](int row, int channel, const float *f) {
                const int64_t m = m0 + row;
                const int n = n0 + channel;
                if (m < t.last && n < N)
                    store8_nt(a.out + m * N + n, f);
            });
        } else {
            int at = 0;
            each_eight<F, F % 4 == 0>(acc, 0, j, [&](int row, int channel, const float *f) {
                const int64_t m = m0 + row;
                const int n = n0 + channel, i = at++;
                float g[8], u[8], y[8], dg[8], du[8];
                saved[i].values(a, g, u);
                if (j + 1 < S::FM) // on its way while the others are stored
                    load_saved(i, j + 1);
                if (m >= t.last || n >= N)
                    return;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float s = 1.0f / (1.0f + __expf(-g[e]));
                    y[e] = g[e] * s * u[e];
                    du[e] = f[e] * g[e] * s;
                    dg[e] = f[e] * u[e] * s * (1.0f + g[e] * (1.0f - s));
                }
                store8_nt(a.grad_pre + m * 2 * N + n, dg);
                store8_nt(a.grad_pre + m * 2 * N + N + n, du);
                if (a.out)
                    store8_nt(a.out + m * N + n, y);
            });
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

// The heights that the finder may take: with more than two shapes each of them
// but the smallest, else the tallest.
template <typename S, typename... MORE>
struct Heights {
    using Finder = TileFinder<largest(S::BM, MORE::BM...)>;
    static constexpr int kLeast = largest(S::BM, MORE::BM...);
};

template <typename S, typename A, typename B, typename... MORE>
struct Heights<S, A, B, MORE...> {
    using Finder = TileFinder<A::BM, B::BM, MORE::BM...>;
    static constexpr int kLeast = A::BM;
};

template <typename... S>
using Finder = typename Heights<S...>::Finder;

// A tile's beginning and end take as long as about this many of its rows (one
// round of 4096^3, 103 us, is as long as a quarter of the four rounds of 8192 x
// 8192 x 4096).  Heights of up to 320 rows against 256 only: 8191 rows over 8
// experts, gated backward 178 us against 261, forward 279 against 314.
constexpr float kEdgeRows = 24.0f;

// Rows before the first expert's first and from the last one's last on become
// zeros, a part of them by each workgroup.
__device__ __forceinline__ void zero_rest(const Job &a)
{
    const int64_t first = min(max((int64_t)a.offsets[0], (int64_t)0), a.num_rows);
    const int64_t last = min(max((int64_t)a.offsets[a.num_experts], first), a.num_rows);
    const int64_t units = a.n / 8, held = (last - first) * units, rest = a.num_rows * units - held;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < rest; i += (int64_t)gridDim.x * blockDim.x)
        reinterpret_cast<u32x4 *>(a.out)[i < first * units ? i : i + held] = u32x4{0, 0, 0, 0};
}

// A workgroup takes the tiles `slot`, slot + (workgroups of the XCD), ... of
// its XCD's run, and sends off the next one's first stages before it stores.
template <int EPI, bool ACROSS, typename S, typename... MORE>
__global__ __launch_bounds__(S::THREADS, 2) void product_kernel(Job a, int ntiles)
{
    __shared__ __align__(256) uint8_t lds[largest(S::STAGES * S::BYTES, (MORE::STAGES * MORE::BYTES)...)];
    if (EPI == kStore && a.zero_rest)
        zero_rest(a);
    const Finder<S, MORE...> find(a, ntiles, kEdgeRows);
    int slot = (int)(blockIdx.x >> 3);
    Tile t = find.tile(a, slot);
    if (t.expert < 0)
        return;
    with_shape<S, MORE...>(t, [&](auto shape) { find_operands<EPI, ACROSS, decltype(shape)>(a, t).load_first(lds); });
    while (t.expert >= 0) {
        slot += (int)(gridDim.x >> 3);
        const Tile next = find.tile(a, slot);
        with_shape<S, MORE...>(t, [&](auto shape) {
            multiply_tile<EPI, ACROSS, decltype(shape)>(a, t, lds, [&] {
                if (next.expert >= 0)
                    with_shape<S, MORE...>(next, [&](auto after) {
                        find_operands<EPI, ACROSS, decltype(after)>(a, next).load_first(lds);
                    });
            });
        });
        t = next;
    }
}

// As many workgroups as the LDS of 256 CUs holds, at most one a tile, in
// eight runs of the same length.
template <int EPI, bool ACROSS, typename S, typename... MORE>
hipError_t product_launch(const Job &a, hipStream_t s)
{
    constexpr int kLds = largest(S::STAGES * S::BYTES, (MORE::STAGES * MORE::BYTES)...);
    const int64_t ntiles = channel_tiles(a.n, S::BN);
    const int64_t tiles = most_tiles(a, Heights<S, MORE...>::kLeast) * ntiles;
    if (tiles > INT32_MAX - 4096) // they are numbered in 32 bits, a run's last number and a step behind it too
        return hipErrorInvalidConfiguration;
    const int64_t run = (tiles + 7) / 8, resident = 32 * (160 * 1024 / kLds);
    hipLaunchKernelGGL((product_kernel<EPI, ACROSS, S, MORE...>), dim3((unsigned)(8 * (run < resident ? run : resident))),
                       dim3(S::THREADS), 0, s, a, (int)ntiles);
    return hipGetLastError();
}

template <int EPI, bool ACROSS>
hipError_t product_shape(const Job &a, hipStream_t s)
{
    switch (product_shape_of(a.num_rows, a.num_experts, a.n, a.k)) {
    case kTile64:
        if constexpr (EPI == kGated) // a wave needs two fragments of either half
            return product_launch<EPI, ACROSS, TileShape<1, 2, 4, 1, 4>, TileShape<1, 2, 4, 2, 3>>(a, s);
        else
            return product_launch<EPI, ACROSS, TileShape<2, 2, 2, 1, 4>, TileShape<2, 2, 2, 2, 3>>(a, s);
    case kTile128x64:
        return product_launch<EPI, ACROSS, TileShape<2, 2, 4, 1, 4>, TileShape<2, 2, 4, 2, 3>>(a, s);
    case kTile128:
        return product_launch<EPI, ACROSS, TileShape<2, 2, 4, 2, 2>, TileShape<2, 2, 4, 4, 2>>(a, s);
    default:
        return product_launch<EPI, ACROSS, TileShape<4, 2, 4, 2, 2>, TileShape<4, 2, 4, 4, 2>, TileShape<2, 4, 8, 3, 2>,
                              TileShape<2, 4, 8, 4, 2>, TileShape<2, 4, 8, 5, 2>>(a, s);
    }
}

// ------------------------------------------------------------ the weights' gradient

struct GradTile {
    int expert, n, k; // expert -1: no such tile
};

// Each XCD (workgroup number modulo 8) takes an eighth of every expert's
// tiles, which are numbered by band of kBand n tiles, k tile, n tile: the tiles
// that run at a time on its 32 CUs read the least through its L2.
struct GradFinder {
    int experts, ntiles, ktiles, share;

    __device__ __forceinline__ GradTile tile(int slot) const
    {
        GradTile t = {-1, 0, 0};
        const int e = slot / share, at = (int)(blockIdx.x & 7) * share + slot % share;
        if (e >= experts || at >= ntiles * ktiles)
            return t;
        const int band = at / (kBand * ktiles), height = min(kBand, ntiles - band * kBand), in = at - band * kBand * ktiles;
        t.expert = e;
        t.n = band * kBand + in % height;
        t.k = in / height;
        return t;
    }
};

template <typename S>
__device__ __forceinline__ Operands<S, true, true> find_operands(const moe_ep_weight_grad_args &a, const GradTile &t)
{
    Operands<S, true, true> o;
    o.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int lo, hi;
    expert_rows(a, t.expert, lo, hi);
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    const int k0 = t.k * S::BN, n0 = t.n * S::BM;
    o.a.find(static_cast<const uint8_t *>(a.x) + ((int64_t)lo * a.k + k0) * 2, 2 * a.k, hi - lo, o.wave,
             o.wave % S::NW * S::FN, [&](int c) { return min(c, (a.k - k0) / 8 - 1); });
    o.b.find(static_cast<const uint8_t *>(a.grad_out) + ((int64_t)lo * a.n + n0) * 2, 2 * a.n, hi - lo, o.wave,
             o.wave / S::NW * S::FM, [&](int c) { return min(c, (a.n - n0) / 8 - 1); });
    o.steps = (int)(((int64_t)hi - lo + kDepth - 1) / kDepth);
    o.start = 0;
    return o;
}

template <typename S>
__global__ __launch_bounds__(S::THREADS, 2) void weight_grad_kernel(moe_ep_weight_grad_args a, GradFinder find)
{
    __shared__ __align__(256) uint8_t lds[S::STAGES * S::BYTES];
    // the next tile of the XCD's that there is, from `slot` on
    const int slots = find.experts * find.share;
    const auto seek = [&](int &slot) {
        GradTile t = {-1, 0, 0};
        for (; slot < slots && t.expert < 0; slot += (int)(gridDim.x >> 3))
            t = find.tile(slot);
        return t;
    };
    int slot = (int)(blockIdx.x >> 3);
    GradTile t = seek(slot);
    if (t.expert < 0)
        return;
    auto o = find_operands<S>(a, t);
    if (o.steps)
        o.load_first(lds);
    while (t.expert >= 0) {
        f32x4 acc[S::FN][S::FM] = {};
        if (o.steps)
            multiply<S>(o, lds, acc);
        const GradTile next = seek(slot);
        if (next.expert >= 0) {
            o = find_operands<S>(a, next);
            if (o.steps)
                o.load_first(lds);
        }
        const int k0 = (t.k * S::NW + o.wave % S::NW) * S::FN * 16, n0 = (t.n * S::MW + o.wave / S::NW) * S::FM * 16;
        uint16_t *out = static_cast<uint16_t *>(a.grad_w) + (int64_t)t.expert * a.n * a.k;
#pragma unroll
        for (int j = 0; j < S::FM; ++j)
            each_eight<S::FN, S::FN % 4 == 0>(acc, 0, j, [&](int row, int channel, const float *f) {
                const int n = n0 + row, k = k0 + channel;
                if (n < a.n && k < a.k)
                    store8_nt(out + (int64_t)n * a.k + k, f);
            });
        t = next;
    }
}

template <typename S>
hipError_t weight_grad_launch(const moe_ep_weight_grad_args &a, hipStream_t s)
{
    GradFinder find = {a.num_experts, channel_tiles(a.n, S::BM), channel_tiles(a.k, S::BN), 0};
    const int64_t tiles = (int64_t)find.ntiles * find.ktiles, share = (tiles + 7) / 8;
    if (share * a.num_experts > INT32_MAX / 8 - 4096)
        return hipErrorInvalidConfiguration;
    find.share = (int)share;
    const int64_t run = share * a.num_experts, resident = 32 * (160 * 1024 / (S::STAGES * S::BYTES));
    hipLaunchKernelGGL(weight_grad_kernel<S>, dim3((unsigned)(8 * (run < resident ? run : resident))), dim3(S::THREADS), 0, s,
                       a, find);
    return hipGetLastError();
}

} // namespace

hipError_t launch_expert_product(const moe_ep_product_args &a, hipStream_t s)
{
    Job j = {};
    j.x = static_cast<const uint8_t *>(a.x);
    j.w = static_cast<const uint8_t *>(a.w);
    j.offsets = a.offsets;
    j.out = static_cast<uint16_t *>(a.out);
    j.num_rows = a.num_rows;
    j.num_experts = a.num_experts;
    j.n = a.n;
    j.k = a.k;
    j.zero_rest = a.zero_rest && a.offsets;
    return a.transposed ? product_shape<kStore, true>(j, s) : product_shape<kStore, false>(j, s);
}

hipError_t launch_gated_product(const moe_ep_gated_args &a, hipStream_t s)
{
    Job j = {};
    j.x = static_cast<const uint8_t *>(a.x);
    j.w = static_cast<const uint8_t *>(a.w);
    j.offsets = a.offsets;
    j.out = static_cast<uint16_t *>(a.out);
    j.pre = a.pre;
    j.pre_scales = a.pre_scales;
    j.num_rows = a.num_rows;
    j.num_experts = a.num_experts;
    j.n = 2 * a.inter_size;
    j.k = a.k;
    j.save = a.save;
    return product_shape<kGated, false>(j, s);
}

hipError_t launch_gated_product_backward(const moe_ep_gated_grad_args &a, hipStream_t s)
{
    Job j = {};
    j.x = static_cast<const uint8_t *>(a.grad_out);
    j.w = static_cast<const uint8_t *>(a.w);
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
    return product_shape<kGatedBackward, true>(j, s);
}

hipError_t launch_product_weight_grad(const moe_ep_weight_grad_args &a, hipStream_t s)
{
    switch (weight_grad_shape_of(a.num_rows, a.num_experts, a.n, a.k)) {
    case kTile64: return weight_grad_launch<TileShape<2, 2, 2, 2, 3>>(a, s);
    case kTile128x64: return weight_grad_launch<TileShape<2, 2, 4, 2, 3>>(a, s);
    case kTile128: return weight_grad_launch<TileShape<2, 2, 4, 4, 2>>(a, s);
    default: return weight_grad_launch<TileShape<2, 4, 8, 4, 2>>(a, s);
    }
}

} // namespace moe_ep
