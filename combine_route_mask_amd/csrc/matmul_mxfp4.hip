// gfx950 kernels of the product of bf16 rows with 4-bit weights (e2m1 codes, an
// e8m0 scale for 32), for a few rows an expert: the weights pass once for every
// 16 (64) rows, and HBM bounds it.  Codes become bf16 by the hardware's scaled
// conversion (exact), products and sums run on the matrix cores in fp32.
//
// v_mfma_f32_16x16x32_bf16: lane l holds 8 elements of row l % 16 at
// k = 8 * (l / 16); k may be in any order as long as both matrices agree.
#include <algorithm>

#include "ffn_internal.h"
#include "product_shapes.h"
#include "rows.h"
#include "tiles.h"

namespace moe_ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kChunk = 256, kWaves = 4; // k of a step, and the waves that share it

typedef u32x2 AnyAligned2 __attribute__((aligned(2)));
typedef f32x4 AnyAligned4 __attribute__((aligned(4)));

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

// Four results of a row, n and on.
template <typename T>
__device__ __forceinline__ void store4(void *out, int64_t row, int n, int N, f32x4 y)
{
    uint8_t *p = static_cast<uint8_t *>(out) + (row * N + n) * RowType<T>::kBytes;
    if (RowType<T>::kBytes == 2) {
        const float f[8] = {y[0], y[1], y[2], y[3], 0.0f, 0.0f, 0.0f, 0.0f};
        const u32x4 v = RowType<Bf16>::pack(f);
        if (N % 4 == 0) {
            *reinterpret_cast<AnyAligned2 *>(p) = u32x2{v[0], v[1]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < N)
                    reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(v[i / 2] >> (i % 2 * 16));
        }
    } else if (N % 4 == 0) {
        *reinterpret_cast<AnyAligned4 *>(p) = y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N)
                reinterpret_cast<float *>(p)[i] = y[i];
    }
}

__device__ __forceinline__ float gate_up(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// ------------------------------------------------------------ many channels

// A workgroup takes 64 channels of one expert (gated: 32 and the same of up) and
// ROWS of its rows at a time, 256 of k a stage through LDS: 128 bytes of each
// channel's codes, its 8 scales, 512 bytes of each row.  The four waves share a
// stage's k (64 each) and join their sums in the end, in their order; a lane
// takes k = 16 (l / 16) .. + 15 of its wave's.  Lanes that read neighbouring
// 16 bytes make one access of L1, which is why codes go through LDS: straight
// into registers (a lane a channel) 128 rows over 32 experts of 4096 x 7168
// take 154 us, L1 busy with 62 accesses a load.
template <int ROWS_, int STAGES_>
struct Stage {
    static constexpr int ROWS = ROWS_, STAGES = STAGES_, FM = ROWS / 16;
    static constexpr int CODES = 64 * 128, X = ROWS * 512, SCALES = 64 * 8; // bytes
    static constexpr int BYTES = CODES + X + 2 * SCALES; // two waves' loads of scales go nowhere
    static constexpr int LX = X / (1024 * kWaves), L = 2 + LX + 1; // a wave's loads of x, and of all
    static constexpr int PITCH = 64 + 4; // floats of a row of sums
    static constexpr int LDS = STAGES * BYTES > 4 * kWaves * ROWS * PITCH ? STAGES * BYTES : 4 * kWaves * ROWS * PITCH;
};

__device__ __forceinline__ void load_part(const uint8_t *base, uint32_t offset, uint8_t *to)
{
#if defined(__HIP_DEVICE_COMPILE__) // the host compiler does not know the resource type
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, 0x7FFFFFFF, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 16, offset, 0, 0, 0);
#endif
}

__device__ __forceinline__ void load_word(const uint8_t *base, uint32_t offset, uint8_t *to)
{
#if defined(__HIP_DEVICE_COMPILE__)
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, 0x7FFFFFFF, 0x00027000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void *)to, 4, offset, 0, 0, 0);
#endif
}

// WORDS: a row's scales are whole aligned words and go through LDS with the stage,
// else their bytes are read one by one where they are used, and the wait for them
// is a wait for every stage on its way: 128 rows over 32 experts of 4096 x 7200
// take 155 us against 106 of 4096 x 7168, of 5760 x 2880 80 against 55 of 5760 x
// 2816 (3.3 to 3.6 against 4.8 to 5.0 TB/s).
template <typename T, bool GATED, bool WORDS, typename S>
__global__ __launch_bounds__(64 * kWaves) void four_bit_kernel(moe_ep_four_bit_args a, int ntiles)
{
    __shared__ __align__(256) uint8_t lds[S::LDS];
    const int e = (int)(blockIdx.x / (unsigned)ntiles), tile = (int)(blockIdx.x % (unsigned)ntiles);
    int lo, hi;
    expert_rows(a, e, lo, hi);
    constexpr int HALF = GATED ? 32 : 64; // channels of the output
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, l4 = lane >> 4;
    const int K = a.k, N = GATED ? a.n / 2 : a.n, n0 = tile * HALF, last = N - n0 - 1, steps = (K + kChunk - 1) / kChunk;
    const int64_t channel = (int64_t)e * a.n + n0;
    const uint8_t *w = a.w + channel * (K / 2), *sc = a.w_scales + channel * (K / 32);
    const int64_t up = (int64_t)N * (K / 2), up_sc = (int64_t)N * (K / 32); // GATED: LDS rows from 32 on
    // codes: 8 rows a load; chunk c (16 bytes) of row r lies at place c ^ (r & 7).
    // Channels past the last read the last's.
    uint32_t code_at[2], code_end;
    {
        const int sub = lane / 8;
        const uint32_t chunk = (uint32_t)((lane % 8) ^ sub) * 16;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            code_at[i] = (uint32_t)min(((i * kWaves + wave) * 8 + sub) % HALF, last) * (uint32_t)(K / 2) + chunk;
        code_end = (steps - 1) * 128 + chunk < (uint32_t)(K / 2) ? 0 : kPastEnd;
    }
    // scales: waves 0 and 1, a row's two words in two lanes
    const int word = lane & 1;
    const uint32_t scale_at = (uint32_t)min((32 * (wave & 1) + lane / 2) % HALF, last) * (uint32_t)(K / 32) + 4 * word;
    const uint32_t scale_end = (steps - 1) * 8 + 4 * word < K / 32 ? 0 : kPastEnd;
    for (int64_t m0 = lo + (int64_t)blockIdx.y * S::ROWS; m0 < hi; m0 += (int64_t)gridDim.y * S::ROWS) {
        const uint8_t *x = static_cast<const uint8_t *>(a.x) + m0 * K * 2;
        const int rows = (int)min((int64_t)S::ROWS, hi - m0);
        const auto load = [&](uint8_t *stage, int step) { // steps past the last bring zeros
            const uint32_t past = step >= steps ? kPastEnd : 0, tail = step == steps - 1 ? 1 : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                load_part(w + (int64_t)step * 128 + (GATED && (i * kWaves + wave) * 8 >= HALF ? up : 0),
                          code_at[i] | past | (tail ? code_end : 0), stage + (i * kWaves + wave) * 1024);
#pragma unroll
            for (int i = 0; i < S::LX; ++i) { // two rows a load, chunk c of row r at place c ^ (r & 15); zeros past the last
                const int row = (i * kWaves + wave) * 2 + lane / 32;
                const uint32_t chunk = (uint32_t)((lane % 32) ^ (row & 15));
                const bool out = row >= rows || (tail && (uint32_t)step * 512 + 16 * chunk >= (uint32_t)(2 * K));
                load_part(x + (int64_t)step * 512, ((uint32_t)row * (uint32_t)(2 * K) + 16 * chunk) | past | (out ? kPastEnd : 0),
                          stage + S::CODES + (i * kWaves + wave) * 1024);
            }
            if (WORDS)
                load_word(sc + (int64_t)step * 8 + (GATED && (wave & 1) ? up_sc : 0), scale_at | past | (tail ? scale_end : 0),
                          stage + S::CODES + S::X + (wave / 2) * S::SCALES + (wave & 1) * 256);
        };
        f32x4 acc[4][S::FM] = {};
        const auto multiply = [&](const uint8_t *stage, int step) {
            const int block = 2 * wave + l4 / 2, chunk = 2 * wave + l4 / 2; // the lane's of the stage's 8
            const bool in = step * kChunk + block * 32 < K;
            bf16x8 v[2][S::FM];
#pragma unroll
            for (int j = 0; j < S::FM; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    v[p][j] = *reinterpret_cast<const bf16x8 *>(
                        stage + S::CODES + (16 * j + l16) * 512 + ((8 * wave + 2 * l4 + p) ^ l16) * 16);
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int r = 16 * f + l16;
                const u32x2 codes = *reinterpret_cast<const u32x2 *>(stage + r * 128 + (chunk ^ (r & 7)) * 16 + l4 % 2 * 8);
                uint32_t b;
                if (WORDS)
                    b = stage[S::CODES + S::X + r * 8 + block];
                else
                    b = sc[(int64_t)min(r % HALF, last) * (K / 32) + (GATED && f >= 2 ? up_sc : 0) + min(step * 8 + block, K / 32 - 1)];
                const float scale = e8m0_value(in ? b : 127); // past the end of k the codes are zeros
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const bf16x8 u = four_bit_values(codes[p], scale);
#pragma unroll
                    for (int j = 0; j < S::FM; ++j)
                        acc[f][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, v[p][j], acc[f][j], 0, 0, 0);
                }
            }
        };
        uint8_t *cur = lds, *free = lds + (S::STAGES - 1) * S::BYTES;
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i)
            load(lds + i * S::BYTES, i);
        for (int i = 0; i < steps; ++i) {
            // this stage has arrived, and no wave reads the last one's place any more
            wait_barrier<(S::STAGES - 2) * (S::L - (WORDS ? 0 : 1))>();
            load(free, i + S::STAGES - 1);
            multiply(cur, i);
            free = cur;
            cur = cur == lds + (S::STAGES - 1) * S::BYTES ? lds : cur + S::BYTES;
        }
        wait_barrier<0>(); // nothing is on its way to LDS, and no wave reads it
        float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int j = 0; j < S::FM; ++j)
                *reinterpret_cast<f32x4 *>(sums + (wave * S::ROWS + 16 * j + l16) * S::PITCH + 16 * f + 4 * l4) = acc[f][j];
        __syncthreads();
        for (int i = threadIdx.x; i < S::ROWS * (HALF / 4); i += 64 * kWaves) {
            const int row = i / (HALF / 4), n = i % (HALF / 4) * 4;
            f32x4 y = {}, u = {};
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                const float *p = sums + (v * S::ROWS + row) * S::PITCH + n;
                y += *reinterpret_cast<const f32x4 *>(p);
                if (GATED)
                    u += *reinterpret_cast<const f32x4 *>(p + 32);
            }
            if (GATED)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    y[c] = gate_up(y[c], u[c]);
            if (row < rows && n0 + n < N)
                store4<T>(a.out, m0 + row, n0 + n, N, y);
        }
        __syncthreads(); // before the next rows' stages
    }
}

// ------------------------------------------------------------ few channels

// A workgroup takes 16 channels (gated: and the same of up) and all its rows, 16
// at a time: where there are not 64 channels for each CU.  Codes go straight
// into registers, a wave's next step is on its way while it multiplies one;
// lane l takes k = 64 (l / 16) .. + 63 of 256.
template <int F>
struct Chunk {
    u32x4 codes[F][2];
    uint32_t scales[F]; // of the lane's two blocks
    bf16x8 x[8];
};

template <typename T, bool GATED>
__global__ __launch_bounds__(64 * kWaves) void four_bit_few_kernel(moe_ep_four_bit_args a, int ntiles)
{
    constexpr int F = GATED ? 2 : 1;
    __shared__ f32x4 sums[kWaves][F][64];
    const int e = (int)(blockIdx.x / (unsigned)ntiles), tile = (int)(blockIdx.x % (unsigned)ntiles);
    int lo, hi;
    expert_rows(a, e, lo, hi);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, l4 = lane >> 4;
    const int K = a.k, N = GATED ? a.n / 2 : a.n, chunks = (K + kChunk - 1) / kChunk, each = (chunks + kWaves - 1) / kWaves;
    const int begin = wave * each, end = min(begin + each, chunks);
    // channels past the last read the last's
    const uint8_t *codes[F], *scales[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int64_t channel = (int64_t)e * a.n + min(tile * 16 + l16, N - 1) + f * N;
        codes[f] = a.w + channel * (K / 2);
        scales[f] = a.w_scales + channel * (K / 32);
    }
    for (int64_t m0 = lo + (int64_t)blockIdx.y * 16; m0 < hi; m0 += (int64_t)gridDim.y * 16) {
        // rows past the last read the last
        const uint16_t *row = static_cast<const uint16_t *>(a.x) + min(m0 + l16, (int64_t)hi - 1) * K;
        const auto load = [&](Chunk<F> &c, int i) {
            // the lane's two blocks of 32, those past the end of k the last one
            const int k = i * kChunk + 64 * l4, k0 = min(k, K - 32), k1 = min(k + 32, K - 32);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                c.codes[f][0] = *reinterpret_cast<const u32x4 *>(codes[f] + k0 / 2);
                c.codes[f][1] = *reinterpret_cast<const u32x4 *>(codes[f] + k1 / 2);
                c.scales[f] = (uint32_t)scales[f][k0 / 32] | (uint32_t)scales[f][k1 / 32] << 8;
            }
#pragma unroll
            for (int p = 0; p < 8; ++p)
                c.x[p] = *reinterpret_cast<const bf16x8 *>(row + (p < 4 ? k0 : k1) + p % 4 * 8);
        };
        f32x4 acc[F] = {};
        const auto multiply = [&](const Chunk<F> &c, int i) {
            const int k = i * kChunk + 64 * l4;
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                const bool in = k + p / 4 * 32 < K; // past the end of k: zeros, whatever was read
                const bf16x8 x = in ? c.x[p] : bf16x8{};
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    const float scale = e8m0_value(in ? c.scales[f] >> (p / 4 * 8) & 255 : 127);
                    acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        four_bit_values(in ? c.codes[f][p / 4][p % 4] : 0, scale), x, acc[f], 0, 0, 0);
                }
            }
        };
        Chunk<F> one, two;
        if (begin < end)
            load(one, begin);
        for (int i = begin; i < end; i += 2) {
            if (i + 1 < end)
                load(two, i + 1);
            multiply(one, i);
            if (i + 2 < end)
                load(one, i + 2);
            if (i + 1 < end)
                multiply(two, i + 1);
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
            sums[wave][f][lane] = acc[f];
        __syncthreads();
        if (wave == 0) {
            f32x4 y[2] = {};
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int v = 0; v < kWaves; ++v)
                    y[f] += sums[v][f][lane];
            if (GATED)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    y[0][c] = gate_up(y[0][c], y[1][c]);
            const int n = tile * 16 + 4 * l4;
            if (m0 + l16 < hi && n < N)
                store4<T>(a.out, m0 + l16, n, N, y[0]);
        }
        __syncthreads(); // before the next rows' sums
    }
}

// Rows of an expert go to several workgroups where there are few channels.
inline dim3 four_bit_grid(const moe_ep_four_bit_args &a, int64_t tiles, int rows)
{
    const int64_t most = (a.num_rows + rows - 1) / rows, busy = std::min<int64_t>(a.num_rows, a.num_experts);
    const int64_t wanted = 1024 / std::max<int64_t>(1, tiles / a.num_experts * busy) + 1;
    return dim3((unsigned)tiles, (unsigned)std::min(std::min(most, wanted), (int64_t)64));
}

template <typename T, bool GATED, typename S>
hipError_t four_bit_launch(const moe_ep_four_bit_args &a, hipStream_t s)
{
    const int ntiles = channel_tiles(GATED ? a.n / 2 : a.n, GATED ? 32 : 64);
    const int64_t tiles = (int64_t)ntiles * a.num_experts;
    if (tiles > INT32_MAX)
        return hipErrorInvalidConfiguration;
    const dim3 grid = four_bit_grid(a, tiles, S::ROWS), block(64 * kWaves);
    if (a.k % 128 == 0 && ((uintptr_t)a.w_scales & 3) == 0)
        hipLaunchKernelGGL((four_bit_kernel<T, GATED, true, S>), grid, block, 0, s, a, ntiles);
    else
        hipLaunchKernelGGL((four_bit_kernel<T, GATED, false, S>), grid, block, 0, s, a, ntiles);
    return hipGetLastError();
}

template <typename T, bool GATED>
hipError_t four_bit_shape(const moe_ep_four_bit_args &a, hipStream_t s)
{
    switch (four_bit_shape_of(a.num_rows, a.num_experts, a.n)) {
    case kRows64: return four_bit_launch<T, GATED, Stage<64, 3>>(a, s);
    case kRows16Stages3: return four_bit_launch<T, GATED, Stage<16, 3>>(a, s);
    case kRows16Stages4: return four_bit_launch<T, GATED, Stage<16, 4>>(a, s);
    case kFew: break;
    }
    const int ntiles = channel_tiles(GATED ? a.n / 2 : a.n, 16);
    const int64_t tiles = (int64_t)ntiles * a.num_experts;
    if (tiles > INT32_MAX)
        return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((four_bit_few_kernel<T, GATED>), four_bit_grid(a, tiles, 16), dim3(64 * kWaves), 0, s, a, ntiles);
    return hipGetLastError();
}

} // namespace

hipError_t launch_four_bit_product(const moe_ep_four_bit_args &a, hipStream_t s)
{
    if (a.gated)
        return a.out_type == MOE_EP_BF16_ROWS ? four_bit_shape<Bf16, true>(a, s) : four_bit_shape<Fp32, true>(a, s);
    return a.out_type == MOE_EP_BF16_ROWS ? four_bit_shape<Bf16, false>(a, s) : four_bit_shape<Fp32, false>(a, s);
}

} // namespace moe_ep
