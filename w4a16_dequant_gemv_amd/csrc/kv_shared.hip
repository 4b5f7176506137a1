// kv_shared.hip -- attention over the paged INT8 cache for sequences that share their first
// pages (kv_codec.h): the shared pages' parts of every row, then every sequence's own tokens.
#include "kv_attend.h"

namespace {

// The parts of the shared pages where a group has few rows: a workgroup has a block of 16 QT
// rows of a kv head and one of `pre_splits` runs of the tiles, which its waves take in turn.
template <int D, int QT, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void kv_shared_split_kernel(SharedArgs a)
{
    constexpr int DT = D / 16, RB = 16 * QT, PAD = D + 4, PER = D / 4;
    __shared__ float joint[kWaves][16 * PAD], stat_m[kWaves][RB], stat_l[kWaves][RB];
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = blockIdx.x % a.cache.n_kv, split = blockIdx.x / a.cache.n_kv % a.pre_splits;
    note_others(a);
    int group, b;
    int64_t rb;
    if (!locate_group<RB>(a, blockIdx.x / a.cache.n_kv / a.pre_splits, group, rb)) return;
    const KvSeq seq = group_rows(a, group, h == 0 && split == 0 && rb == 0, b);
    const int rows = seq.n * a.group, row0 = (int)rb * RB;
    const Tiles tiles = {0, 0, seq.total() / kTile};
    if (tiles.count == 0) return;
    const int t0 = (int)((int64_t)tiles.count * split / a.pre_splits), t1 = (int)((int64_t)tiles.count * (split + 1) / a.pre_splits);
    Wave<D, QT> s;
    begin(s, a, seq, h, (int)rb);
    attend_tiles<kWaves>(s, a, seq, b, h, tiles, t0 + wave, t1, 1 << 30, 1 << 30);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float l = column_sum(s.l[t]);
        if (g == 0) {
            stat_m[wave][t * 16 + m16] = s.m[t];
            stat_l[wave][t * 16 + m16] = l;
        }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float top = kNone;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) top = fmaxf(top, stat_m[v][t * 16 + m16]);
        const float f = __builtin_amdgcn_exp2f(s.m[t] - top);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<f32x4 *>(&joint[wave][m16 * PAD + d * 16 + g * 4]) = s.o[t][d] * f;
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * PER; i += kThreads) {
            const int row = i / PER, ch = i % PER * 4, r = row0 + t * 16 + row;
            if (r >= rows) continue;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
            float m = kNone, l = 0.0f;
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                o += *reinterpret_cast<const f32x4 *>(&joint[v][row * PAD + ch]);
                m = fmaxf(m, stat_m[v][t * 16 + row]);
            }
#pragma unroll
            for (int v = 0; v < kWaves; ++v)
                l += stat_l[v][t * 16 + row] * __builtin_amdgcn_exp2f(stat_m[v][t * 16 + row] - m);
            const int tok = r / a.group;
            const int64_t to = ((int64_t)(seq.q0 + tok) * a.n_q + h * a.group + r - tok * a.group) * a.pre_splits + split;
            *reinterpret_cast<f32x4 *>(a.pre_part + to * D + ch) = o;
            if (ch == 0) {
                a.pre_stats[to * 2] = m;
                a.pre_stats[to * 2 + 1] = l;
            }
        }
        __syncthreads();
    }
}

// The parts of the shared pages where a group has many rows.
template <int D, int NW, int QT>
__global__ __launch_bounds__(64 * NW, 2) void kv_shared_rows_kernel(SharedArgs a)
{
    attend_rows<D, NW, QT, true>(a, a.pre_splits);
}

// The sequences' own tokens.
template <int D, int QT, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void kv_own_split_kernel(SharedArgs a) { attend_split<D, QT>(a); }

template <int D, int QT, int OCC>
__global__ __launch_bounds__(64, OCC) void kv_own_wave_kernel(SharedArgs a) { attend_wave<D, QT>(a); }

template <int D, int QT, int NW>
__global__ __launch_bounds__(64 * NW) void kv_own_join_kernel(SharedArgs a) { join_parts<D, QT, NW>(a); }

template <int D, int NW, int QT>
__global__ __launch_bounds__(64 * NW, 2) void kv_own_rows_kernel(SharedArgs a, int splits)
{
    attend_rows<D, NW, QT, false>(a, splits);
}

template <int D>
__global__ __launch_bounds__(kThreads) void kv_own_join_rows_kernel(SharedArgs a, int splits) { join_rows<D>(a, splits); }

// How the shared pages' parts are computed: qt > 0 by kv_shared_split_kernel, otherwise by kv_shared_rows_kernel with
// `waves` waves; in `splits` runs of tiles.
struct SharedPlan {
    int qt, waves, splits;
    int64_t items;               // row blocks (an upper bound)
};

// Groups have `rows` rows a kv head on average and share at most `tiles` tiles.
SharedPlan shared_plan(int64_t tokens, int groups, int n_q, int n_kv, int d, int64_t tiles)
{
    SharedPlan p = {};
    const int64_t group = n_q / n_kv, rows = (tokens + groups - 1) / groups * group;
    double best = 0.0;
    auto offer = [&](int qt, int waves, int64_t rb, int64_t slots, auto cost) {
        const int64_t blocks = (rows + rb - 1) / rb * groups * n_kv;
        for (int cuts = 1; cuts <= 64 && cuts <= tiles && (cuts == 1 || blocks * cuts <= 4 * slots); ++cuts) {
            const double c = cost(blocks * cuts, (double)tiles / cuts) + (double)(tokens * n_q) * cuts * d * 8 / 4e6;
            if (p.splits == 0 || c < best) {
                best = c;
                p = {qt, waves, cuts, tokens * group / rb + groups};
            }
        }
    };
    for (int qt = 1; qt <= (d <= 128 ? 3 : 1); ++qt) {
        const int64_t slots = 256 * split_occupancy(d, qt);
        const double tile = split_occupancy(d, qt) == 2 ? 0.45 : 0.8;
        offer(qt, 0, 16 * qt, slots, [&](int64_t n, double run) {
            return std::max(1.0, (double)n / slots) * (6.0 + tile * std::max(run, (double)kWaves));
        });
    }
    for (int waves = d == 256 ? 8 : 4; waves <= 8; waves += 4) {
        const int64_t places = waves == 4 ? 512 : 256;
        offer(0, waves, (d == 256 ? 16 : 32) * waves, places, [&](int64_t n, double run) {
            const int64_t full = n / places, rest = n % places;
            const double pair = waves == 4 ? 2.3 : 2.0, last = waves == 4 && rest <= 256 ? 1.3 : pair;
            return (double)full * (8.0 + run * pair) + (rest ? 8.0 + run * last : 0.0);
        });
    }
    return p;
}

template <int D, int QT>
hipError_t launch_shared_split(const SharedArgs &a, const SharedPlan &p, const Target &to)
{
    constexpr int OCC = split_occupancy(D, QT);
    if (to.name) return to.report("kv_shared_split_kernel<%d, %d, %d>, %d cuts", D, QT, OCC, p.splits);
    kv_shared_split_kernel<D, QT, OCC><<<(unsigned)(p.items * a.cache.n_kv * p.splits), kThreads, 0, to.stream>>>(a);
    return hipGetLastError();
}

constexpr int rows_lds(int d) { return 2 * (8 * ((d + 63) / 64) + d / 8) * 1024; }

template <typename K>
hipError_t allow_lds(K kernel, int bytes)
{
    if (bytes <= 65536) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, int NW, int QT>
hipError_t launch_shared_rows(const SharedArgs &a, const SharedPlan &p, const Target &to)
{
    if (to.name) return to.report("kv_shared_rows_kernel<%d, %d, %d>, %d cuts", D, NW, QT, p.splits);
    auto kernel = kv_shared_rows_kernel<D, NW, QT>;
    if (hipError_t e = allow_lds(kernel, rows_lds(D))) return e;
    kernel<<<(unsigned)(p.items * a.cache.n_kv * p.splits), 64 * NW, rows_lds(D), to.stream>>>(a);
    return hipGetLastError();
}

template <int D, int QT>
hipError_t launch_own_split(const SharedArgs &a, const Plan &p, const Target &to)
{
    const unsigned groups = (unsigned)(a.workers * a.cache.n_kv);
    constexpr int OCC = split_occupancy(D, QT);
    const int join = a.workers >= 16 * a.batch.batch ? 4 : 1;
    if (to.name) {
        if (p.alone == 1) return to.report("kv_own_wave_kernel<%d, %d, %d>", D, QT, OCC);
        if (a.whole) return to.report("kv_own_split_kernel<%d, %d, %d>, whole row blocks", D, QT, OCC);
        return to.report("kv_own_split_kernel<%d, %d, %d>, kv_own_join_kernel<%d, %d, %d>", D, QT, OCC, D, QT, join);
    }
    if (p.alone == 1) {
        kv_own_wave_kernel<D, QT, OCC><<<groups, 64, 0, to.stream>>>(a);
        return hipGetLastError();
    }
    kv_own_split_kernel<D, QT, OCC><<<groups, kThreads, 0, to.stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole) return e;
    if (join == 4) kv_own_join_kernel<D, QT, 4><<<groups * 16 * QT, 256, 0, to.stream>>>(a);
    else kv_own_join_kernel<D, QT, 1><<<groups * 16 * QT, 64, 0, to.stream>>>(a);
    return hipGetLastError();
}

template <int D, int NW, int QT>
hipError_t launch_own_rows(const SharedArgs &a, const Plan &p, const Target &to)
{
    if (to.name) {
        if (p.splits == 1) return to.report("kv_own_rows_kernel<%d, %d, %d>", D, NW, QT);
        return to.report("kv_own_rows_kernel<%d, %d, %d>, kv_own_join_rows_kernel<%d>, %d cuts", D, NW, QT, D, p.splits);
    }
    auto kernel = kv_own_rows_kernel<D, NW, QT>;
    if (hipError_t e = allow_lds(kernel, rows_lds(D))) return e;
    kernel<<<(unsigned)(p.items * a.cache.n_kv * p.splits), 64 * NW, rows_lds(D), to.stream>>>(a, p.splits);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t threads = a.batch.tokens * a.n_q * (D / 4);
    kv_own_join_rows_kernel<D><<<(unsigned)((threads + kThreads - 1) / kThreads), kThreads, 0, to.stream>>>(a, p.splits);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const SharedArgs &a, const SharedPlan &s, const Plan &p, Target to)
{
    hipError_t e;
    if (s.qt == 1) e = launch_shared_split<D, 1>(a, s, to);
    else if constexpr (D == 256) e = launch_shared_rows<D, 8, 1>(a, s, to);
    else if (s.qt == 2) e = launch_shared_split<D, 2>(a, s, to);
    else if (s.qt == 3) e = launch_shared_split<D, 3>(a, s, to);
    else e = s.waves == 8 ? launch_shared_rows<D, 8, 2>(a, s, to) : launch_shared_rows<D, 4, 2>(a, s, to);
    if (e != hipSuccess) return e;
    to.go_on();
    if (p.qt == 1) return launch_own_split<D, 1>(a, p, to);
    if constexpr (D == 256) {
        return launch_own_rows<D, 8, 1>(a, p, to);
    } else {
        if (p.qt == 2) return launch_own_split<D, 2>(a, p, to);
        if (p.qt == 3) return launch_own_split<D, 3>(a, p, to);
        return p.waves == 8 ? launch_own_rows<D, 8, 2>(a, p, to) : launch_own_rows<D, 4, 2>(a, p, to);
    }
}

// Bytes of the parts and of the notes of skipped tiles, each a multiple of 16.
int64_t parts_bytes(int64_t rows, int d) { return (rows * (d + 2) * 4 + 15) / 16 * 16; }
int64_t skips_bytes(int batch) { return ((int64_t)batch * 4 + 15) / 16 * 16; }

}  // namespace

int64_t kv_shared_workspace(int64_t tokens, int batch, int groups, int max_pages, int page, int n_q, int n_kv, int d)
{
    const SharedPlan s = shared_plan(tokens, groups, n_q, n_kv, d, (int64_t)max_pages * page / kTile);
    return parts_bytes(tokens * n_q * s.splits, d) + skips_bytes(batch) + kv_attention_workspace(tokens, batch, n_q, n_kv, d);
}

hipError_t kv_launch_shared(const kv_paged_cache &cache, const kv_paged_batch &batch, const kv_shared_prefix &prefix,
                            const uint16_t *q, int64_t q_stride, int n_q, float scale, void *workspace, uint16_t *out,
                            hipStream_t stream, char *name, int64_t name_len)
{
    const SharedPlan s = shared_plan(batch.tokens, prefix.groups, n_q, cache.n_kv, cache.d,
                                     (int64_t)prefix.max_pages * cache.page / kTile);
    // what the table has room for behind the shared pages stands for the sequences' own tokens
    const int64_t most = (int64_t)std::max(batch.table_cols - prefix.max_pages, 1) * cache.page;
    const Plan p = plan_for(batch.tokens, batch.batch, n_q, cache.n_kv, cache.d, most, most);
    const int64_t rows = batch.tokens * n_q * s.splits;
    float *pre_part = (float *)workspace, *pre_stats = pre_part + rows * cache.d;
    int32_t *skips = reinterpret_cast<int32_t *>((char *)workspace + parts_bytes(rows, cache.d));
    float *part = reinterpret_cast<float *>((char *)skips + skips_bytes(batch.batch)), *stats = part + p.parts * cache.d;
    SharedArgs a;
    static_cast<Args &>(a) = {cache, batch, q, q_stride, n_q, n_q / cache.n_kv, scale * 1.44269504f, 0, 0,
                              __builtin_ctz(cache.page), p.workers, p.alone == kWaves, p.workers ? 1.0 / p.workers : 0.0,
                              part, stats, reinterpret_cast<int32_t *>(stats + p.parts * 2), out};
    a.cu_seqs = prefix.cu_seqs;
    a.pages = prefix.pages;
    a.groups = prefix.groups;
    a.max_pages = prefix.max_pages;
    a.pre_splits = s.splits;
    a.pre_part = pre_part;
    a.pre_stats = pre_stats;
    a.skips = skips;
    const Target to = {stream, name, name_len};
    switch (cache.d) {
    case 64: return launch<64>(a, s, p, to);
    case 96: return launch<96>(a, s, p, to);
    case 128: return launch<128>(a, s, p, to);
    case 256: return launch<256>(a, s, p, to);
    default: return hipErrorInvalidValue;
    }
}
