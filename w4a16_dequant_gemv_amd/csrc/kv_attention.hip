// kv_attention.hip -- attention over the paged INT8 cache (kv_codec.h): its kernels, and which one a call gets.
#include "kv_attend.h"

namespace {

template <int D, int QT, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void kv_attend_split_kernel(Args a) { attend_split<D, QT>(a); }

template <int D, int QT, int OCC>
__global__ __launch_bounds__(64, OCC) void kv_attend_wave_kernel(Args a) { attend_wave<D, QT>(a); }

template <int D, int QT, int NW>
__global__ __launch_bounds__(64 * NW) void kv_join_kernel(Args a) { join_parts<D, QT, NW>(a); }

template <int D, int NW, int QT>
__global__ __launch_bounds__(64 * NW, 2) void kv_attend_rows_kernel(Args a, int splits)
{
    attend_rows<D, NW, QT, false>(a, splits);
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv_join_rows_kernel(Args a, int splits) { join_rows<D>(a, splits); }

template <int D, int QT>
hipError_t launch_split(const Args &a, const Plan &p, const Target &to)
{
    const hipStream_t stream = to.stream;
    const unsigned groups = (unsigned)(a.workers * a.cache.n_kv);
    constexpr int OCC = split_occupancy(D, QT);
    // with 16 parts a sequence or more, four waves join a row (1 x 131k tokens, 64 heads on
    // 8: 53 us, 59 with one wave; 32 x 4k: 55, 53 with one)
    const int join = a.workers >= 16 * a.batch.batch ? 4 : 1;
    if (to.name) {
        if (p.alone == 1) return to.report("kv_attend_wave_kernel<%d, %d, %d>", D, QT, OCC);
        if (a.whole) return to.report("kv_attend_split_kernel<%d, %d, %d>, whole row blocks", D, QT, OCC);
        return to.report("kv_attend_split_kernel<%d, %d, %d>, kv_join_kernel<%d, %d, %d>", D, QT, OCC, D, QT, join);
    }
    if (p.alone == 1) {
        kv_attend_wave_kernel<D, QT, OCC><<<groups, 64, 0, stream>>>(a);
        return hipGetLastError();
    }
    kv_attend_split_kernel<D, QT, OCC><<<groups, kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole) return e;
    if (join == 4) kv_join_kernel<D, QT, 4><<<groups * 16 * QT, 256, 0, stream>>>(a);
    else kv_join_kernel<D, QT, 1><<<groups * 16 * QT, 64, 0, stream>>>(a);
    return hipGetLastError();
}

template <int D, int NW, int QT>
hipError_t launch_rows(const Args &a, const Plan &p, const Target &to)
{
    const hipStream_t stream = to.stream;
    if (to.name) {
        if (p.splits == 1) return to.report("kv_attend_rows_kernel<%d, %d, %d>", D, NW, QT);
        return to.report("kv_attend_rows_kernel<%d, %d, %d>, kv_join_rows_kernel<%d>, %d cuts", D, NW, QT, D, p.splits);
    }
    constexpr int LDS = 2 * (8 * ((D + 63) / 64) + D / 8) * 1024;
    if (LDS > 65536) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kv_attend_rows_kernel<D, NW, QT>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
        if (e != hipSuccess) return e;
    }
    kv_attend_rows_kernel<D, NW, QT><<<(unsigned)(p.items * a.cache.n_kv * p.splits), 64 * NW, LDS, stream>>>(a, p.splits);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t threads = a.batch.tokens * a.n_q * (D / 4);
    kv_join_rows_kernel<D><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a, p.splits);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const Args &a, const Plan &p, const Target &to)
{
    if (p.qt == 1) return launch_split<D, 1>(a, p, to);
    if constexpr (D == 256) {
        return launch_rows<D, 8, 1>(a, p, to);
    } else {
        if (p.qt == 2) return launch_split<D, 2>(a, p, to);
        if (p.qt == 3) return launch_split<D, 3>(a, p, to);
        return p.waves == 8 ? launch_rows<D, 8, 2>(a, p, to) : launch_rows<D, 4, 2>(a, p, to);
    }
}

}  // namespace

int64_t kv_attention_workspace(int64_t tokens, int batch, int n_q, int n_kv, int d)
{
    const Plan p = plan_for(tokens, batch, n_q, n_kv, d, int64_t(1) << 40, int64_t(1) << 40);
    return p.parts * (d + 2) * 4 + (int64_t)(p.workers + 1) * 16;
}

hipError_t kv_launch_attention(const kv_paged_cache &cache, const kv_paged_batch &batch, const uint16_t *q,
                               int64_t q_stride, int n_q, float scale, int window, int sinks, void *workspace,
                               uint16_t *out, hipStream_t stream, char *name, int64_t name_len)
{
    const int64_t most = (int64_t)batch.table_cols * cache.page;
    const Plan p = plan_for(batch.tokens, batch.batch, n_q, cache.n_kv, cache.d, most,
                            window > 0 ? (int64_t)window + sinks : most);
    float *part = (float *)workspace;
    float *stats = part + p.parts * cache.d;
    const Args a = {cache, batch, q, q_stride, n_q, n_q / cache.n_kv, scale * 1.44269504f, window, sinks,
                    __builtin_ctz(cache.page), p.workers, p.alone == kWaves, p.workers ? 1.0 / p.workers : 0.0, part, stats,
                    reinterpret_cast<int32_t *>(stats + p.parts * 2), out};
    const Target to = {stream, name, name_len};
    switch (cache.d) {
    case 64: return launch<64>(a, p, to);
    case 96: return launch<96>(a, p, to);
    case 128: return launch<128>(a, p, to);
    case 256: return launch<256>(a, p, to);
    default: return hipErrorInvalidValue;
    }
}
