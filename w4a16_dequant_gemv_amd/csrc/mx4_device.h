// mx4_device.h -- MXFP4 on the device: types, the quantization of a block and the
// matrix instructions that take codes and scales as they are (mxfp4.h).
#pragma once

#include "mxfp4.h"
#include "q4_device.h"

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// x's elements as they lie in memory, and to binary32 and back.
template <int TYPE>
struct Mx4Type;
template <>
struct Mx4Type<MX4_F16> {
    typedef uint16_t T;
    static __device__ __forceinline__ float load(T v) { return half_bits_to_float(v); }
    static __device__ __forceinline__ T store(float v) { return bitcast<uint16_t>((_Float16)v); }
};
template <>
struct Mx4Type<MX4_BF16> {
    typedef uint16_t T;
    static __device__ __forceinline__ float load(T v) { return bitcast<float>((uint32_t)v << 16); }
    static __device__ __forceinline__ T store(float v) { return bitcast<uint16_t>((__bf16)v); }
};
template <>
struct Mx4Type<MX4_F32> {
    typedef float T;
    static __device__ __forceinline__ float load(T v) { return v; }
    static __device__ __forceinline__ T store(float v) { return v; }
};

// Eight consecutive elements.
template <int TYPE>
__device__ __forceinline__ void mx4_load8(const typename Mx4Type<TYPE>::T *p, float v[8])
{
    if constexpr (TYPE == MX4_F32) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[i + 4] = b[i];
        }
    } else {
        const u32x4 raw = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Mx4Type<TYPE>::load((uint16_t)(raw[i >> 1] >> (16 * (i & 1))));
    }
}

// The scale's byte of a block whose largest |x| has these bits.  An exponent field f is
// floor(log2) + 127 (0 for subnormal numbers, which are below the smallest scale anyway);
// infinities and NaN have the largest bits of all.
__device__ __forceinline__ int mx4_scale(uint32_t top) { return top >= 0x7F800000u ? 255 : max((int)(top >> 23) - 2, 0); }

// Eight values over 2^(s - 127) as codes.  The power of two comes first and apart: the
// conversion's own scale operand has no value below 2^-126.
__device__ __forceinline__ uint32_t mx4_codes8(const float v[8], int s)
{
    const int e = 127 - s;
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(v[0], e), ldexpf(v[1], e), 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(v[2], e), ldexpf(v[3], e), 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(v[4], e), ldexpf(v[5], e), 1.0f, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, ldexpf(v[6], e), ldexpf(v[7], e), 1.0f, 3);
}

// The largest |x|'s bits of eight values.
__device__ __forceinline__ uint32_t mx4_top8(const float v[8])
{
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, bitcast<uint32_t>(v[i]) & 0x7FFFFFFFu);
    return t;
}

// 16 rows x 16 columns += 128 products each.  Lane l has 32 elements (one block) of row
// l % 16 of A and of column l % 16 of B, blocks in any order that is the same for both,
// and that block's scale in byte OA (OB) of sa (sb); it gets rows 4 (l / 16) .. + 3 of
// column l % 16.
template <int OA, int OB>
__device__ __forceinline__ f32x4 mx4_mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb)
{
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, OA, (int)sa, OB, (int)sb);
}

// 32 rows x 32 columns += 64 products each: lane l has a block of row l % 32 and of column
// l % 32, and gets rows 8 (i / 4) + 4 (l / 32) + i % 4 of column l % 32.
template <int OA, int OB>
__device__ __forceinline__ f32x16 mx4_mfma32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb)
{
    const i32x8 x = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    const i32x8 y = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, OA, (int)sa, OB, (int)sb);
}
