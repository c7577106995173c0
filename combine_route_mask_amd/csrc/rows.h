// Row elements of the expert layer's kernels: 16-byte vectors of bf16 or
// fp32 to floats and back, wave and workgroup reductions, and the int8 row
// scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "formats.h"
#include "memory_ops.h"

namespace moe_ep {

struct Bf16 {};
struct Fp32 {};

template <typename T>
struct RowType;

template <>
struct RowType<Bf16> {
    static constexpr int kPer = 8;   // elements of a 16-byte vector
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ void unpack(u32x4 v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            unpack_bf16x2(v[i], f[2 * i], f[2 * i + 1]);
    }
    static __device__ __forceinline__ u32x4 pack(const float *f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        return v;
    }
};

template <>
struct RowType<Fp32> {
    static constexpr int kPer = 4;
    static constexpr int kBytes = 4;
    static __device__ __forceinline__ void unpack(u32x4 v, float *f)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = __uint_as_float(v[i]);
    }
    static __device__ __forceinline__ u32x4 pack(const float *f)
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __float_as_uint(f[i]);
        return v;
    }
};

// N elements (a multiple of kPer) from / to a 16-byte aligned address.
template <typename T, int N>
__device__ __forceinline__ void load_elements(const uint8_t *p, float *f)
{
    u32x4 v[N / RowType<T>::kPer];
#pragma unroll
    for (int i = 0; i < N / RowType<T>::kPer; ++i)
        v[i] = load16_nt(p + 16 * i);
#pragma unroll
    for (int i = 0; i < N / RowType<T>::kPer; ++i)
        RowType<T>::unpack(v[i], f + i * RowType<T>::kPer);
}

__device__ __forceinline__ void store16_nt(void *p, u32x4 v)
{
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}

// The value of another lane of the same 16, without LDS: CTRL is a DPP
// control (the lane with the lowest bit, or the second, turned over; the
// mirror image within 8, or 16, lanes).
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float x)
{
    return __uint_as_float(dpp<CTRL>(__float_as_uint(x)));
}

// Largest value of each 4 or 16 consecutive lanes, in all of them.
__device__ __forceinline__ uint32_t max4(uint32_t x)
{
    x = max(x, dpp<kDppXor1>(x));
    return max(x, dpp<kDppXor2>(x));
}

__device__ __forceinline__ uint32_t max16(uint32_t x)
{
    x = max4(x);
    x = max(x, dpp<kDppMirror8>(x));
    return max(x, dpp<kDppMirror16>(x));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = max16(x);
    x = max(x, (uint32_t)__shfl_xor((int)x, 16));
    return max(x, (uint32_t)__shfl_xor((int)x, 32));
}

// Sum over the wave, the same in every lane (each step adds the same two
// numbers on both sides).
__device__ __forceinline__ float wave_sum(float x)
{
    x += dpp<kDppXor1>(x);
    x += dpp<kDppXor2>(x);
    x += dpp<kDppMirror8>(x);
    x += dpp<kDppMirror16>(x);
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

// Magnitude of x as an ordered integer: infinities and NaN are the largest.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

constexpr uint32_t kInfinity = 0x7F800000u;

// The int8 rule of a row whose largest magnitude is `top`: scale = top / 127,
// code = x / scale to nearest even, taken as the correctly rounded quotient
// 127 x / top.  Ties are common (bf16 rows are ratios of 8-bit integers) and
// this form keeps them exact, where a product with 127 / top would fall to
// either side.  A huge row is brought down by a power of two first, so that
// 127 x stays finite.
struct Int8Row {
    float scale, by, top;
    __device__ __forceinline__ explicit Int8Row(uint32_t bits)
    {
        top = __uint_as_float(bits);
        if (bits == 0 || bits >= kInfinity) {
            scale = bits ? __uint_as_float(0x7FC00000u) : 0.0f;
            by = 0.0f;
            top = 1.0f;
        } else {
            scale = top / 127.0f;
            by = top > 0x1p+100f ? 127.0f * 0x1p-20f : 127.0f;
            top = top > 0x1p+100f ? top * 0x1p-20f : top;
        }
    }
    // NaN * 0 and infinity * 0 convert to 0.
    __device__ __forceinline__ int code(float x) const
    {
        const float c = rintf((x * by) / top);
        return c == c ? (int)c : 0;
    }
    __device__ __forceinline__ uint32_t codes4(const float *f) const
    {
        return (uint32_t)(code(f[0]) & 0xFF) | ((uint32_t)(code(f[1]) & 0xFF) << 8) |
               ((uint32_t)(code(f[2]) & 0xFF) << 16) | ((uint32_t)(code(f[3]) & 0xFF) << 24);
    }
    __device__ __forceinline__ u32x4 codes16(const float *f) const
    {
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = codes4(f + 4 * i);
        return v;
    }
};

} // namespace moe_ep
