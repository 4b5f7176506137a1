// mx4_matmul.hip -- products of MXFP4 operands on the matrix cores (mxfp4.h).
#include "mx4_device.h"
#include "q4_launch.h"

namespace {

// Few rows of x: a workgroup has 16 rows of W and 16 MT of x, its NW waves take steps of
// 256 elements in turn and are summed at the end.  W goes from memory to operand registers.
template <int TYPE, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void mx4_rows_kernel(const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xs,
                                                           const uint8_t *__restrict__ wc, const uint8_t *__restrict__ ws,
                                                           int m, int n_out, int k, uint16_t *__restrict__ y)
{
    __shared__ f32x4 part[NW][MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * MT;
    const int steps = (k + 255) / 256, blocks = k / 32;
    const int64_t pitch = k / 2;
    const int wr = min(n0 + r, n_out - 1);
    const u32x4 zero = {0u, 0u, 0u, 0u};
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = wave; s < steps; s += NW) {
        const int b = s * 8 + 2 * g;                                     // this lane's blocks: b, b + 1
        const int have = blocks - b;
        const uint32_t mask = have >= 2 ? 0xFFFFu : have == 1 ? 0xFFu : 0u;
        const u32x4 *p = reinterpret_cast<const u32x4 *>(wc + wr * pitch + b * 16);
        const u32x4 a0 = have >= 1 ? p[0] : zero, a1 = have >= 2 ? p[1] : zero;
        const uint32_t sa = *reinterpret_cast<const uint16_t *>(ws + ((int64_t)s * n_out + wr) * 8 + 2 * g) & mask;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int xr = min(m0 + t * 16 + r, m - 1);
            const u32x4 *q = reinterpret_cast<const u32x4 *>(xc + xr * pitch + b * 16);
            const u32x4 b0 = have >= 1 ? q[0] : zero, b1 = have >= 2 ? q[1] : zero;
            const uint32_t sb = *reinterpret_cast<const uint16_t *>(xs + ((int64_t)s * m + xr) * 8 + 2 * g) & mask;
            acc[t] = mx4_mfma16<0, 0>(a0, b0, acc[t], sa, sb);
            acc[t] = mx4_mfma16<1, 1>(a1, b1, acc[t], sa, sb);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 256; i += 64 * NW) {
        const int t = i / 256, row = i / 16 % 16, ch = i % 16;           // x row, channel
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += part[w][t][ch / 4 * 16 + row][ch % 4];
        if (m0 + t * 16 + row < m && n0 + ch < n_out)
            y[(int64_t)(m0 + t * 16 + row) * n_out + n0 + ch] = Mx4Type<TYPE>::store(sum);
    }
}

}  // namespace

hipError_t mx4_launch_matmul(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int64_t m,
                             int64_t n_out, int64_t k, int type, void *y, hipStream_t stream)
{
    const dim3 grid((unsigned)((n_out + 15) / 16), (unsigned)((m + 63) / 64));
    if (type == MX4_F16)
        mx4_rows_kernel<MX4_F16, 4, 4><<<grid, 256, 0, stream>>>(xc, xs, wc, ws, (int)m, (int)n_out, (int)k, (uint16_t *)y);
    else
        mx4_rows_kernel<MX4_BF16, 4, 4><<<grid, 256, 0, stream>>>(xc, xs, wc, ws, (int)m, (int)n_out, (int)k, (uint16_t *)y);
    return hipGetLastError();
}
