// Test kernel: what a raw buffer load to LDS reads when part of its address is the scalar offset.  64 lanes
// load 16 bytes each from `records` bytes at p; the caller's memory holds all that could be addressed however the
// range is checked (soffset + 1024 bytes), so no address is outside it.
#include <hip/hip_runtime.h>
#include <stdint.h>

__global__ __launch_bounds__(64) void buffer_range_kernel(const uint32_t *p, uint32_t records, uint32_t soffset, uint32_t *out)
{
    __shared__ __attribute__((aligned(16))) uint32_t lds[256];
    const int lane = threadIdx.x;
    for (int i = 0; i < 4; ++i) lds[lane * 4 + i] = 0xEEEEEEEEu;
    __syncthreads();
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t *>(p), (short)0, (int)records, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, lane * 16, (int)soffset, 0, 0);
    __syncthreads();
    for (int i = 0; i < 4; ++i) out[lane * 4 + i] = lds[lane * 4 + i];
}

extern "C" int buffer_range(const uint32_t *p, uint32_t records, uint32_t soffset, uint32_t *out, void *stream)
{
    buffer_range_kernel<<<1, 64, 0, (hipStream_t)stream>>>(p, records, soffset, out);
    return (int)hipGetLastError();
}
