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
    // gfx950 rounds two floats to bf16 (to nearest even) in one instruction;
    // NaN stays NaN.
    static __device__ __forceinline__ u32x4 pack(const float *f)
    {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 two = {f[2 * i], f[2 * i + 1]};
            v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2));
        }
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

// Largest value of the four lanes l % 16, + 16, + 32, + 48, in all of them, without LDS.
__device__ __forceinline__ uint32_t max_of_rows(uint32_t x)
{
#if defined(__HIP_DEVICE_COMPILE__) // the host compiler does not know the exchanges
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(s[0], s[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(t[0], t[1]);
#endif
    return x;
}

__device__ __forceinline__ int wave_add(int x)
{
    x += (int)dpp<kDppXor1>((uint32_t)x);
    x += (int)dpp<kDppXor2>((uint32_t)x);
    x += (int)dpp<kDppMirror8>((uint32_t)x);
    x += (int)dpp<kDppMirror16>((uint32_t)x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
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
// code = x / scale = 127 x / top to nearest even.  Ties are common (bf16 rows
// are ratios of 8-bit integers), so the quotient has to be right on them: a
// product with 1 / top is brought to the correctly rounded quotient by the
// remainder, which the fma gives exactly (a quotient that fp32 holds, such as
// a tie, comes out as it is).  Rows of extreme magnitude are brought near 1 by
// a power of two first, so that 127 x and 1 / top stay normal.
struct Int8Row {
    float scale, by, top, inv;
    bool finite;
    __device__ __forceinline__ explicit Int8Row(uint32_t bits)
    {
        top = __uint_as_float(bits);
        finite = bits < kInfinity;
        scale = finite ? top / 127.0f : __uint_as_float(0x7FC00000u);
        const float up = top > 0x1p+60f ? 0x1p-100f : top < 0x1p-60f ? 0x1p+100f : 1.0f;
        by = 127.0f * up;
        top = bits ? top * up : 1.0f;
        inv = 1.0f / top;
    }
    // 127 x / top plus 1.5 * 2^23: the sum's low byte is the code.
    __device__ __forceinline__ uint32_t code(float x) const
    {
        const float t = x * by, c = t * inv;
        return __float_as_uint(fmaf(fmaf(-c, top, t), inv, c) + 12582912.0f);
    }
    __device__ __forceinline__ uint32_t codes4(const float *f) const
    {
        const uint32_t lo = __builtin_amdgcn_perm(code(f[1]), code(f[0]), 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(code(f[3]), code(f[2]), 0x04000C0Cu);
        return finite ? lo | hi : 0;
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

// e4m3 codes of f * by, round to nearest even; every product is within 448
// times 1 + 2^-22, which rounds to 448.
__device__ __forceinline__ u32x2 e4m3_codes(const float *f, float up, float by)
{
    u32x2 v;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int p = __builtin_amdgcn_cvt_pk_fp8_f32((f[4 * h] * up) * by, (f[4 * h + 1] * up) * by, 0, false);
        p = __builtin_amdgcn_cvt_pk_fp8_f32((f[4 * h + 2] * up) * by, (f[4 * h + 3] * up) * by, p, true);
        v[h] = (uint32_t)p;
    }
    return v;
}

constexpr u32x2 kNanCodes = {0x7F7F7F7Fu, 0x7F7F7F7Fu};

// Exponent of an MXFP8 block's scale for the bits of its largest magnitude:
// 448 = 1.75 * 2^8, so 1.m * 2^E needs 2^(E - 8), or 2^(E - 7) when 1.m > 1.75.
__device__ __forceinline__ int mx_exponent(uint32_t top)
{
    const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return (top >> 23) == 0 || e < -127 ? -127 : e;
}

// The MXFP8 codes of 8 elements whose block's largest magnitude is `top`, and
// the block's scale byte.  A block with a NaN or an infinity is NaN.
__device__ __forceinline__ u32x2 mx_codes(const float *f, uint32_t top, uint8_t &scale)
{
    const int e = mx_exponent(top);
    scale = top >= kInfinity ? 0xFF : (uint8_t)(e + 127);
    return top >= kInfinity ? kNanCodes : e4m3_codes(f, 1.0f, __uint_as_float((uint32_t)(127 - e) << 23));
}

// 2^(b - 127) of an e8m0 byte; NaN for 255.
__device__ __forceinline__ float e8m0_value(uint32_t b)
{
    const uint32_t bits = max(b << 23, 0x00400000u); // 2^-127 is subnormal
    return __uint_as_float(b == 255 ? 0x7FC00000u : bits);
}

// 8 e4m3 codes times a scale.
__device__ __forceinline__ void mx_values(u32x2 codes, float scale, float *f)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[h], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[h], true);
        f[4 * h] = a[0] * scale;
        f[4 * h + 1] = a[1] * scale;
        f[4 * h + 2] = b[0] * scale;
        f[4 * h + 3] = b[1] * scale;
    }
}

} // namespace moe_ep
