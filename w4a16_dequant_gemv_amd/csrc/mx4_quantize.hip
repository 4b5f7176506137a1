// mx4_quantize.hip -- MXFP4 quantization and the way back (mxfp4.h).
//
// Both are bound by HBM: 2 (fp16) or 4 bytes an element on one side, 17/32 on the other.
// Four lanes have a block, eight elements each: a wave's loads and code stores are
// contiguous, and the block's maximum takes two exchanges between neighbours.  28672 x 8192
// fp32 to codes 221 us (4.8 TB/s; a large copy reaches 4.9) and back 212, 2047 x 11008 bf16 rows
// 22016 apart 10.8 and 11.1, 64 x 8192 fp16 2.4 and 2.5 (a launch).
#include "mx4_device.h"
#include "q4_launch.h"

namespace {

constexpr int kThreads = 256;

template <int TYPE>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(const typename Mx4Type<TYPE>::T *__restrict__ x,
                                                                uint32_t per_row, int64_t rows, int64_t stride,
                                                                uint32_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;                  // eight elements: at most 2^31 of them
    const uint32_t at = i / per_row, c = i - at * per_row;
    const int64_t row = at;
    if (row >= rows) return;
    float v[8];
    mx4_load8<TYPE>(x + row * stride + c * 8, v);
    uint32_t top = mx4_top8(v);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const int s = mx4_scale(top);
    codes[i] = mx4_codes8(v, s);
    const uint32_t b = c / 4, blocks = per_row / 4;
    if (c % 4 == 0) {
        uint8_t *to = scales + ((int64_t)(b / 8) * rows + row) * 8;
        to[b % 8] = (uint8_t)s;
        if (b + 1 == blocks)
            for (uint32_t j = blocks % 8; j && j < 8; ++j) to[j] = 0;
    }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                                  const uint8_t *__restrict__ scales, uint32_t per_row,
                                                                  int64_t rows, typename Mx4Type<TYPE>::T *__restrict__ out)
{
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t at = i / per_row, c = i - at * per_row;
    const int64_t row = at;
    if (row >= rows) return;
    const uint32_t w = codes[i];
    const int s = scales[((int64_t)(c / 32) * rows + row) * 8 + c / 4 % 8];
    float v[8];
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1]; v[4] = d[0]; v[5] = d[1]; v[6] = e[0]; v[7] = e[1];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s == 255 ? __builtin_nanf("") : ldexpf(v[j], s - 127);
    if constexpr (TYPE == MX4_F32) {
        f32x4 *to = reinterpret_cast<f32x4 *>(out + (int64_t)i * 8);
        to[0] = f32x4{v[0], v[1], v[2], v[3]};
        to[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        u32x4 p;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            p[j] = (uint32_t)Mx4Type<TYPE>::store(v[2 * j]) | (uint32_t)Mx4Type<TYPE>::store(v[2 * j + 1]) << 16;
        *reinterpret_cast<u32x4 *>(out + (int64_t)i * 8) = p;
    }
}

unsigned groups(int64_t rows, int64_t k) { return (unsigned)((rows * (k / 8) + kThreads - 1) / kThreads); }

}  // namespace

hipError_t mx4_launch_quantize(const void *x, int type, int64_t rows, int64_t k, int64_t stride, uint8_t *codes,
                               uint8_t *scales, hipStream_t stream)
{
    const unsigned n = groups(rows, k);
    uint32_t *c = reinterpret_cast<uint32_t *>(codes);
    const uint32_t per = (uint32_t)(k / 8);
    if (type == MX4_F16)
        mx4_quantize_kernel<MX4_F16><<<n, kThreads, 0, stream>>>((const uint16_t *)x, per, rows, stride, c, scales);
    else if (type == MX4_BF16)
        mx4_quantize_kernel<MX4_BF16><<<n, kThreads, 0, stream>>>((const uint16_t *)x, per, rows, stride, c, scales);
    else
        mx4_quantize_kernel<MX4_F32><<<n, kThreads, 0, stream>>>((const float *)x, per, rows, stride, c, scales);
    return hipGetLastError();
}

hipError_t mx4_launch_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t k, int type,
                                 void *out, hipStream_t stream)
{
    const unsigned n = groups(rows, k);
    const uint32_t *c = reinterpret_cast<const uint32_t *>(codes);
    const uint32_t per = (uint32_t)(k / 8);
    if (type == MX4_F16)
        mx4_dequantize_kernel<MX4_F16><<<n, kThreads, 0, stream>>>(c, scales, per, rows, (uint16_t *)out);
    else if (type == MX4_BF16)
        mx4_dequantize_kernel<MX4_BF16><<<n, kThreads, 0, stream>>>(c, scales, per, rows, (uint16_t *)out);
    else
        mx4_dequantize_kernel<MX4_F32><<<n, kThreads, 0, stream>>>(c, scales, per, rows, (float *)out);
    return hipGetLastError();
}
