// kv_shared.hip -- attention over the paged INT8 cache for sequences that share their first
// pages (kv_codec.h).
//
// Mathematics.  A row's softmax over two sets of tokens is joined from a part for each: with (O, m, l) as in
// kv_attend.h, top = max(m_1, m_2), o = (O_1 2^(m_1 - top) + O_2 2^(m_2 - top)) / (l_1 2^(m_1 - top) + l_2 2^(m_2 - top)).
// All rows of a group of sequences are rows of one matrix product with the shared pages, which are so
// read once; what each sequence has of its own is read by its own rows.
// Both go out as parts in binary32 and are joined by a second launch.  (Joining within the first one would take a wait between
// workgroups; one workgroup for a row block's shared and own tokens takes them one after the other, and was slower on
// every size tried for d <= 128.)  Measured, replayed, 64 heads on 8, d = 128, with and without shared pages: 64 sequences
// with up to 1000 tokens of their own behind 4096 47 and 69 us, 32 with 500 behind 131072 225 and 681,
// 64 with 1000 behind 32768 131 and 344; 4 of 32 heads on 32 with 100 behind 512 11.0 and 13.7.
#include "kv_attend.h"

namespace {

// Four channels of a row's part.
template <int D>
__device__ __forceinline__ void put_part(const SharedArgs &a, int64_t row, int place, int ch, f32x4 o, float m, float l)
{
    const int64_t to = row * a.places() + place;
    *reinterpret_cast<f32x4 *>(a.part + to * D + ch) = o;
    if (ch == 0) {
        a.stats[to * 2] = m;
        a.stats[to * 2 + 1] = l;
    }
}

// Bytes of LDS for put_rows.
constexpr int joint_lds(int d) { return (kWaves * 16 * (d + 4) + 2 * kWaves * 16) * 4; }

// 16 rows, whose tiles `share` waves side by side (1, 2 or 4) took in turn, as one part of each.
// Every thread of the workgroup calls this; those with nothing are not `live`.
template <int D, typename F>
__device__ __forceinline__ void put_rows(const SharedArgs &a, Wave<D, 1> &s, float *smem, int share, bool live, int many,
                                         int place, F row_of)
{
    constexpr int DT = D / 16, PAD = D + 4, PER = D / 4;
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), turn = wave % share, lead = wave - turn;
    float *joint = smem, *stat_m = smem + kWaves * 16 * PAD, *stat_l = stat_m + kWaves * 16;
    if (live) s.l[0] = column_sum(s.l[0]);
    if (share == 1) {
        if (!live || m16 >= many) return;
        const int64_t row = row_of(m16);
#pragma unroll
        for (int d = 0; d < DT; ++d) put_part<D>(a, row, place, d * 16 + g * 4, s.o[0][d], s.m[0], s.l[0]);
        return;
    }
    if (live && g == 0) {
        stat_m[wave * 16 + m16] = s.m[0];
        stat_l[wave * 16 + m16] = s.l[0];
    }
    __syncthreads();
    if (live) {
        float top = kNone;
        for (int v = 0; v < share; ++v) top = fmaxf(top, stat_m[(lead + v) * 16 + m16]);
        const float f = __builtin_amdgcn_exp2f(s.m[0] - top);
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<f32x4 *>(&joint[(wave * 16 + m16) * PAD + d * 16 + g * 4]) = s.o[0][d] * f;
    }
    __syncthreads();
    if (!live) return;
    for (int i = turn * 64 + lane; i < 16 * PER; i += 64 * share) {
        const int row = i / PER, ch = i % PER * 4;
        if (row >= many) continue;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        float m = kNone, l = 0.0f;
        for (int v = lead; v < lead + share; ++v) {
            o += *reinterpret_cast<const f32x4 *>(&joint[(v * 16 + row) * PAD + ch]);
            m = fmaxf(m, stat_m[v * 16 + row]);
        }
        for (int v = lead; v < lead + share; ++v) l += stat_l[v * 16 + row] * __builtin_amdgcn_exp2f(stat_m[v * 16 + row] - m);
        put_part<D>(a, row_of(row), place, ch, o, m, l);
    }
}

// The parts of the shared pages, 16 rows of a group and kv head a workgroup, and one of `splits` runs
// of the tiles, which its waves take in turn from memory.  Bound by the chain of a wave's tiles, 0.39 us each at d = 128 and
// 0.85 with two workgroups on a CU; with many rows attend_rows has 128 of them share a tile by way of LDS, 1.9 and 3.0 us a
// tile.  (Tried while weights were one fp16 part there, 1.5 and 2.3 us a tile: 64 rows, 1.1, no faster in all; 256 rows of eight
// waves, in a launch of their own, 32 sequences behind 131072 tokens 166 us against 175, all others slower.)
template <int D>
__device__ __forceinline__ void shared_rows(const SharedArgs &a, float *smem, int block)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = block % a.cache.n_kv, split = block / a.cache.n_kv % a.splits;
    int b;
    int64_t rb;
    KvSeq seq;
    if (!group_rows<16>(a, block / a.cache.n_kv / a.splits, seq, b, rb)) return;
    const Tiles tiles = {0, 0, seq.total() / kTile};
    const int t0 = (int)((int64_t)tiles.count * split / a.splits), t1 = (int)((int64_t)tiles.count * (split + 1) / a.splits);
    Wave<D, 1> s;
    begin(s, a, seq, h, (int)rb);
    attend_tiles<kWaves>(s, a, seq, b, h, tiles, t0 + wave, t1, 1 << 30, 1 << 30);
    const int row0 = (int)rb * 16;
    put_rows(a, s, smem, kWaves, true, seq.n * a.group - row0, split, [&](int row) {
        const int tok = (row0 + row) / a.group;
        return (int64_t)(seq.q0 + tok) * a.n_q + h * a.group + row0 + row - tok * a.group;
    });
}

// A sequence's own tokens, 16 of its rows of a kv head and a run of `chunk` tiles (the last run: all that are
// left) at a time; `share` waves of a workgroup take a run's tiles in turn, so that a workgroup has 4 / share runs.
// Row block `item` of a kv head is found without a pass over the sequences: sequence b's numbers begin
// at rows_before(b) / 16 + b, which leaves each of them room enough.
template <int D>
__device__ __forceinline__ void own_rows(const SharedArgs &a, float *smem, int block, int per_chunk, int share)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), turn = wave % share;
    const int chunk = block / per_chunk, unit = (block - chunk * per_chunk) * (kWaves / share) + wave / share;
    const int h = unit % a.cache.n_kv, item = unit / a.cache.n_kv;
    const SharedArgs::Named all = a.named();
    auto number = [&](int before, int b) { return (int64_t)min(max(before, 0), (int)a.batch.tokens) * a.group / 16 + b; };
    int b = 0, many = a.batch.batch;                         // the last sequence that begins at or before `item`
    while (many > 64) {
        const int step = (many + 63) / 64, p = lane * step;
        const int n = __popcll(__ballot(p < many && number(a.batch.cu_q[b + p], b + p) <= item));
        b += max(n - 1, 0) * step;
        many = min(step, many - max(n - 1, 0) * step);
    }
    const int mine = b + min(lane, many - 1), from = a.batch.cu_q[mine];
    const KvSeq s64 = kv_seq(a.batch, mine, a.cache.slots, a.page_shift);
    const int before = __popcll(__ballot(lane < many && number(from, mine) <= item)), f = max(before - 1, 0);
    b += f;
    const KvSeq seq = {__builtin_amdgcn_readlane(s64.q0, f), __builtin_amdgcn_readlane(s64.n, f),
                       __builtin_amdgcn_readlane(s64.ctx, f), __builtin_amdgcn_readlane(s64.slot, f)};
    const int rows = seq.n * a.group, rb = item - (int)number(__builtin_amdgcn_readlane(from, f), b);
    const Tiles tiles = visible_tiles(a, seq, a.skip(seq, b, all));
    const int t0 = chunk * a.chunk, t1 = chunk + 1 < a.chunks ? min(t0 + a.chunk, tiles.count) : tiles.count;
    // of a sequence, not between two; and the run is not empty
    const bool live = before > 0 && rb >= 0 && rb < (rows + 15) / 16 && t0 < tiles.count;
    Wave<D, 1> s;
    if (live) {
        const int at_min = seq.ctx + rb * 16 / a.group, at_max = seq.ctx + (min(rb * 16 + 16, rows) - 1) / a.group;
        begin(s, a, seq, h, rb);
        if (share == 4) attend_tiles<4>(s, a, seq, b, h, tiles, t0 + turn, t1, at_min, at_max);
        else if (share == 2) attend_tiles<2>(s, a, seq, b, h, tiles, t0 + turn, t1, at_min, at_max);
        else attend_tiles<1>(s, a, seq, b, h, tiles, t0, t1, at_min, at_max);
    }
    put_rows(a, s, smem, share, live, rows - rb * 16, a.splits + chunk, [&](int row) {
        const int tok = (rb * 16 + row) / a.group;
        return (int64_t)(seq.q0 + tok) * a.n_q + h * a.group + rb * 16 + row - tok * a.group;
    });
}

// Shared pages and own tokens in one launch: the first `first` workgroups compute the shared pages' parts (MANY: 128
// rows each, otherwise 16), bound by the matrix cores, and the others, bound by memory, run beside them.
template <int D, bool MANY, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void kv_shared_kernel(SharedArgs a, int first, int per_chunk, int share)
{
    extern __shared__ __attribute__((aligned(16))) float shared_smem[];
    const int block = blockIdx.x;
    if (block < first) {
        if constexpr (MANY) attend_rows<D, 4, 2, true>(a, a.splits, block, first);
        else shared_rows<D>(a, shared_smem, block);
    } else {
        own_rows<D>(a, shared_smem, block - first, per_chunk, share);
    }
}

// The shared pages alone, for d = 256: 128 rows take the LDS of a whole CU, and eight waves.
template <int D, int NW, int QT>
__global__ __launch_bounds__(64 * NW, 2) void kv_shared_rows_kernel(SharedArgs a)
{
    attend_rows<D, NW, QT, true>(a, a.splits, blockIdx.x, gridDim.x);
}

// Joins each row's parts: D / 4 threads a row, four channels each, eight parts on their way.
// A workgroup takes rows of one sequence, `per` workgroups a sequence.  4 to 6 us, most of it the launch and two loads one
// after the other; 13 for 33 parts of 2048 rows (35 MB).
template <int D>
__global__ __launch_bounds__(kThreads) void kv_shared_join_kernel(SharedArgs a, int per)
{
    constexpr int PER = D / 4, SIDE = kThreads / PER;
    const int b = blockIdx.x / per, turn = blockIdx.x % per, ch = threadIdx.x % PER * 4;
    const KvSeq seq = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
    if (threadIdx.x >= PER * SIDE || seq.n == 0) return;
    const int skip = a.skip(seq, b, a.named()), count = visible_tiles(a, seq, skip).count;
    const int p0 = skip > 0 ? 0 : a.splits, p1 = a.splits + min((count + a.chunk - 1) / a.chunk, a.chunks);
    const int64_t end = (int64_t)(seq.q0 + seq.n) * a.n_q;
    for (int64_t row = (int64_t)seq.q0 * a.n_q + turn * SIDE + threadIdx.x / PER; row < end; row += per * SIDE) {
        const float *stats = a.stats + row * a.places() * 2;
        const float *part = a.part + row * a.places() * D + ch;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
        float m = kNone, l = 0.0f;
        for (int p = p0; p < p1; p += 8) {
            f32x4 x[8];
            float pm[8], pl[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                pm[i] = kNone;
                pl[i] = 0.0f;
                x[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (p + i < p1) {
                    pm[i] = stats[2 * (p + i)];
                    pl[i] = stats[2 * (p + i) + 1];
                    x[i] = *reinterpret_cast<const f32x4 *>(part + (int64_t)(p + i) * D);
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, pm[i]);
            const float keep = __builtin_amdgcn_exp2f(m - top);
            o *= keep;
            l *= keep;
            m = top;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = __builtin_amdgcn_exp2f(pm[i] - m);
                o += x[i] * f;
                l += pl[i] * f;
            }
        }
        store_out(a.out + row * D + ch, o, l);
    }
}

// How a call is run.
struct SharedPlan {
    bool alone;                  // as without shared pages
    int many;                    // rows of the shared pages' workgroups: 16, or 128 (d = 256: in a launch of their own)
    int splits, chunks, chunk, share;
    int64_t items, own;          // row blocks of the shared pages and of the own tokens (upper bounds)
};

constexpr int64_t kMaxBlocks = (int64_t(1) << 32) / kThreads - 1;

// Workgroups of a chunk of the own tokens.
int64_t own_blocks(const SharedPlan &p, int n_kv)
{
    const int64_t each = kWaves / p.share;
    return (p.own * n_kv + each - 1) / each;
}

// Groups share at most `tiles` tiles; sequences have at most `own` tiles besides.
SharedPlan shared_plan(int64_t tokens, int batch, int groups, int n_q, int n_kv, int d, int64_t tiles, int64_t own)
{
    SharedPlan p = {};
    const int64_t group = n_q / n_kv, rows = (tokens + groups - 1) / groups * group, one = (tokens + batch - 1) / batch * group;
    // With many rows of its own a sequence is bound by the matrix rate whoever reads the pages (16 x 16 tokens behind 8k,
    // 64 heads on 8: 101 us shared, 90 not; 32 x 32 behind 2k 106 and 78).
    p.alone = one > 64;
    if (p.alone) return p;
    // Waves of a row block: more of them end a long sequence sooner, fewer need fewer workgroups, of which the CUs hold
    // 512 (us with 1, 2 and 4: 64 heads on 8, 16 x 500 tokens behind 8k 37, 27.6, 24.9; 64 x 1000 behind 4k 61.5, 46.4,
    // 47.3; 256 x 500 behind 8k 159, 153, 162; 128 x 300 behind four times 1k 35.2, 37.3, 42.7; d = 64, 40 x 5 tokens 28.9,
    // 27.3, 22.1).
    const int64_t blocks = (one + 15) / 16 * batch * n_kv;
    p.share = blocks * d <= 50000 ? 4 : own <= 8 ? 1 : 2;
    p.own = tokens * group / 16 + batch;
    p.chunks = (int)std::min<int64_t>((own + 31) / 32, 8);
    p.chunk = (int)((own + p.chunks - 1) / p.chunks);
    // What a choice costs, in us: a start, then the longest run of tiles or, where that is more, all the work shared out to the
    // workgroups that the CUs hold at once, and the parts' way out and back.  A tile of the shared pages takes a workgroup
    // `alone` us with a CU to itself, `full` with two on each.  (With 1, 2, 4, 6, 8, 12 runs: 64 sequences behind 4k, 16
    // rows a workgroup 51, 53, 60, 68, 75, 95, 128 rows 134, 76, 49, 45, 49, 56; 16 of 32 heads on 8 behind 8k 58, 36, 24,
    // 22, 22, 23 and 250, 130, 72, 54, 45, 37.)  The 128 rows' constants are below what their tiles take, 1.9 and 3.0 us: what
    // they choose takes 2.3 % longer than the best choice on average at 38 sizes, 27 % at most, with 1.9 and 3.0 3.1 %, since the
    // 16 rows' are low too.
    const double size = (double)d / 128;
    const double slots = d <= 128 ? 512 : 256;
    const double own_work = (double)(blocks * p.share) / 4 * (6.0 + 1.1 * size * (double)std::min<int64_t>(own, p.chunk) / p.share);
    double best = 0.0;
    auto offer = [&](int rb, double start, double alone, double full) {
        const int64_t n_blocks = (rows + rb - 1) / rb * groups * n_kv;
        for (const int cuts : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64}) {
            if (cuts > 1 && (cuts > tiles || (double)(n_blocks * cuts) > 4 * slots)) break;
            const double n = (double)(n_blocks * cuts), run = (double)tiles / cuts;
            const double tile = alone + (full - alone) * std::min(1.0, std::max(0.0, 2 * n / slots - 1.0));
            const double chain = tile * (rb == 16 ? std::max(run, (double)kWaves) : run) * std::max(1.0, n / slots);
            const double parts = (double)(tokens * n_q) * cuts * d * 8 / 2e6;
            const bool apart = d == 256 && rb == 128;                            // in a launch of its own
            const double work = apart ? chain + own_work / slots : std::max(chain, (n * run * full + own_work) / slots);
            if (p.splits == 0 || start + work + parts < best) {
                best = start + work + parts;
                p.many = rb;
                p.splits = cuts;
                p.items = std::max<int64_t>(tokens * group - groups, 0) / rb + groups;
            }
        }
    };
    offer(16, 8.0, 0.1 + 0.29 * size, 0.1 + 0.75 * size);
    if (d <= 128) offer(128, 10.0, 1.48, 2.3);
    else offer(128, 16.0, 2.6, 2.6);
    // A launch has less than 2^32 threads: so many row blocks take their own tokens in fewer chunks.  (One always has room:
    // batch n_kv is at most 2^21 and rows n_kv 64 times that.)
    const int64_t most = (kMaxBlocks - p.items * n_kv * p.splits) / own_blocks(p, n_kv);
    if (p.chunks > most) {
        p.chunks = (int)std::max<int64_t>(most, 1);
        p.chunk = (int)((own + p.chunks - 1) / p.chunks);
    }
    return p;
}

// The parts of a row.
int places(const SharedPlan &p) { return p.splits + p.chunks; }

// Tiles that the table has room for behind the shared pages, which stand for the sequences' own tokens.
int64_t own_tiles(int64_t table_cols, int64_t max_pages, int64_t page)
{
    return std::max<int64_t>(table_cols - max_pages, 1) * page / kTile;
}

constexpr int rows_lds(int d) { return 2 * (8 * ((d + 63) / 64) + d / 8) * 1024; }

template <typename K>
hipError_t allow_lds(K kernel, int bytes)
{
    if (bytes <= 65536) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int D, bool MANY>
hipError_t launch_kernel(const SharedArgs &a, const SharedPlan &p, int64_t first, const Target &to)
{
    constexpr int OCC = D <= 128 ? 2 : 1, LDS = MANY ? std::max(rows_lds(D), joint_lds(D)) : joint_lds(D);
    auto kernel = kv_shared_kernel<D, MANY, OCC>;
    if (hipError_t e = allow_lds(kernel, LDS)) return e;
    const int64_t per_chunk = own_blocks(p, a.cache.n_kv);
    kernel<<<(unsigned)(first + per_chunk * p.chunks), kThreads, LDS, to.stream>>>(a, (int)first, (int)per_chunk, p.share);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const SharedArgs &a, const SharedPlan &p, const Target &to)
{
    const int64_t first = p.items * a.cache.n_kv * p.splits;
    if (to.name) {
        const char *many = p.many == 16 ? "false" : "true";
        if (D == 256 && p.many == 128)
            return to.report("kv_shared_rows_kernel<256, 8, 1>, kv_shared_kernel<256, false, 1>, kv_shared_join_kernel<256>, "
                             "%d cuts, %d waves, %d chunks", p.splits, p.share, p.chunks);
        return to.report("kv_shared_kernel<%d, %s, %d>, kv_shared_join_kernel<%d>, %d cuts, %d waves, %d chunks", D, many,
                         D <= 128 ? 2 : 1, D, p.splits, p.share, p.chunks);
    }
    hipError_t e;
    if constexpr (D == 256) {
        if (p.many == 128) {
            auto kernel = kv_shared_rows_kernel<D, 8, 1>;
            if (hipError_t f = allow_lds(kernel, rows_lds(D))) return f;
            kernel<<<(unsigned)first, 512, rows_lds(D), to.stream>>>(a);
            if (hipError_t f = hipGetLastError()) return f;
        }
        e = launch_kernel<D, false>(a, p, p.many == 128 ? 0 : first, to);
    } else {
        e = p.many == 128 ? launch_kernel<D, true>(a, p, first, to) : launch_kernel<D, false>(a, p, first, to);
    }
    if (e != hipSuccess) return e;
    constexpr int SIDE = kThreads / (D / 4);
    const int64_t rows = (a.batch.tokens + a.batch.batch - 1) / a.batch.batch * a.n_q;       // of a sequence on average
    const int per = (int)std::min((rows + SIDE - 1) / SIDE, kMaxBlocks / a.batch.batch);
    kv_shared_join_kernel<D><<<(unsigned)per * (unsigned)a.batch.batch, kThreads, 0, to.stream>>>(a, per);
    return hipGetLastError();
}

}  // namespace

int64_t kv_shared_workspace(int64_t tokens, int batch, int groups, int max_pages, int table_cols, int page, int n_q, int n_kv,
                            int d)
{
    const SharedPlan p = shared_plan(tokens, batch, groups, n_q, n_kv, d, (int64_t)max_pages * page / kTile,
                                     own_tiles(table_cols, max_pages, page));
    if (p.alone) return kv_attention_workspace(tokens, batch, n_q, n_kv, d);
    return tokens * n_q * places(p) * (d + 2) * 4;
}

hipError_t kv_launch_shared(const kv_paged_cache &cache, const kv_paged_batch &batch, const kv_shared_prefix &prefix,
                            const uint16_t *q, int64_t q_stride, int n_q, float scale, void *workspace, uint16_t *out,
                            hipStream_t stream, char *name, int64_t name_len)
{
    const SharedPlan p = shared_plan(batch.tokens, batch.batch, prefix.groups, n_q, cache.n_kv, cache.d,
                                     (int64_t)prefix.max_pages * cache.page / kTile,
                                     own_tiles(batch.table_cols, prefix.max_pages, cache.page));
    if (p.alone)
        return kv_launch_attention(cache, batch, q, q_stride, n_q, scale, 0, 0, workspace, out, stream, name, name_len);
    float *part = (float *)workspace;
    SharedArgs a;
    static_cast<Args &>(a) = {cache, batch, q, q_stride, n_q, n_q / cache.n_kv, scale * 1.44269504f, 0, 0,
                              __builtin_ctz(cache.page), 0, false, 0.0, part, part + batch.tokens * n_q * places(p) * cache.d,
                              nullptr, out};
    a.cu_seqs = prefix.cu_seqs;
    a.pages = prefix.pages;
    a.groups = prefix.groups;
    a.max_pages = prefix.max_pages;
    a.splits = p.splits;
    a.chunks = p.chunks;
    a.chunk = p.chunk;
    const Target to = {stream, name, name_len};
    switch (cache.d) {
    case 64: return launch<64>(a, p, to);
    case 96: return launch<96>(a, p, to);
    case 128: return launch<128>(a, p, to);
    case 256: return launch<256>(a, p, to);
    default: return hipErrorInvalidValue;
    }
}
