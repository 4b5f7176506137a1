// kv_attention.hip -- attention over the paged INT8 cache (kv_codec.h): its kernels, and which of them a call gets.
#include "kv_attend.h"

namespace {

// The split kernel's work as numbered units: sequence after sequence, its row
// blocks of RB rows one after the other, each with kStart units for the latency
// of beginning it and then one for each of the sequence's tiles.  Lane i of a
// wave holds sequence 64 chunk + i.
template <int RB>
struct Roster {
    int chunk = -1;
    KvSeq s;
    int64_t units, end;          // the sequence's units, and their sum up to it within the chunk

    __device__ void load(const Args &a, int c)
    {
        chunk = c;
        const int b = c * 64 + (threadIdx.x & 63);
        units = 0;
        s = {0, 0, 0, 0};
        if (b < a.batch.batch) {
            s = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
            if (s.n) units = (int64_t)((s.n * a.group + RB - 1) / RB) * (a.whole ? 1 : visible_tiles(a, s).count + kStart);
        }
        end = kv_wave_scan(units);
    }
    __device__ KvSeq get(int i) const
    {
        return {__builtin_amdgcn_readlane(s.q0, i), __builtin_amdgcn_readlane(s.n, i),
                __builtin_amdgcn_readlane(s.ctx, i), __builtin_amdgcn_readlane(s.slot, i)};
    }
};

// One kv head's work is cut into equal runs of units, one for each worker (a
// workgroup), whatever the sequences' lengths (or, with few tokens, a worker takes a
// row block as a whole: then the row blocks are the units); a worker's four waves take its
// tiles in turn and join at the end of each row block.  A row block that one
// worker has whole is finished there; the others' parts go to the workspace: the
// run's first row block to place 0, its last to place 1.  The worker that has a
// shared row block's first tile leaves a note for the kernel that joins them.
// Bound by HBM with many tokens (32 x 32k, 64 query heads on 8: 377 us, 5.7 TB/s; 64
// ragged sequences of 4k on average: 67 us, 4.7 TB/s, where a fixed number of cuts for
// each sequence took 89), by latency with few (1 x 500 tokens: 9.1 us, uncut).
// Pages go from memory to operand registers: no wave shares a tile with another, so
// LDS would add a trip and a barrier.  P is used as two fp16 parts, whose second one
// costs little here (5 rows of 8 sequences: 21.8 us, 20.0 without it).
template <int D, int QT, int OCC>
__global__ __launch_bounds__(kThreads, OCC) void kv_attend_split_kernel(Args a)
{
    constexpr int DT = D / 16, RB = 16 * QT;
    constexpr int PAD = D + 4;                       // floats a row of the joining buffer: four banks on per row
    __shared__ float joint[kWaves][16 * PAD], stat_m[kWaves][RB], stat_l[kWaves][RB];
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);          // a scalar: its branches are uniform
    const int h = blockIdx.x % a.cache.n_kv, worker = blockIdx.x / a.cache.n_kv;

    // how many units there are, and what a worker takes: no less than a tile for each wave
    Roster<RB> roster;
    int64_t run = 1, units = worker + 1;
    if (!a.whole) {
        units = 0;
        for (int c = 0; c * 64 < a.batch.batch; ++c) {
            roster.load(a, c);
            units += kv_lane(roster.end, 63);
        }
        run = (int64_t)((double)units * a.inv_workers);
        while (run * a.workers < units) ++run;
        run = max(run, (int64_t)kWaves);
    }
    int64_t u = run * worker;
    const int64_t end = min(u + run, units);
    int note_row = 0, note_rows = 0, note_parts = 0, note_place = 0;

    // the sequence with unit u
    int b = a.batch.batch;
    int64_t off = u;
    for (int c = 0; u < end && c * 64 < a.batch.batch; ++c) {
        if (roster.chunk != c) roster.load(a, c);
        const uint64_t hit = __ballot(off < roster.end);
        if (hit) {
            const int i = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
            b = c * 64 + i;
            off -= kv_lane(roster.end - roster.units, i);
            break;
        }
        off -= kv_lane(roster.end, 63);
    }

    for (int place = 0; u < end && b < a.batch.batch;) {
        if (roster.chunk != b >> 6) roster.load(a, b >> 6);
        if (off >= kv_lane(roster.units, b & 63)) {          // done with this one, or it has no rows
            off = 0;
            ++b;
            continue;
        }
        const KvSeq seq = roster.get(b & 63);
        const Tiles tiles = visible_tiles(a, seq);
        const int rows = seq.n * a.group;
        const int per_block = a.whole ? 1 : tiles.count + kStart, rb = (int)(off / per_block), at = (int)(off - (int64_t)rb * per_block);
        const int take = (int)min((int64_t)(per_block - at), end - u);
        const int t0 = max(at - kStart, 0), count = a.whole ? tiles.count : max(at + take - kStart, 0) - t0;
        const int64_t last = u - at + per_block - 1;         // the row block's last unit
        u += take;
        off += take;
        if (count == 0) continue;                            // only the beginning is this worker's

        Wave<D, QT> s;
        begin(s, a, seq, h, rb);
        const int at_min = seq.ctx + rb * RB / a.group;
        const int at_max = seq.ctx + (min(rb * RB + RB, rows) - 1) / a.group;
        attend_tiles<kWaves>(s, a, seq, b, h, tiles, t0 + wave, t0 + count, at_min, at_max);

        // join the waves
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const float l = column_sum(s.l[t]);
            if (g == 0) {
                stat_m[wave][t * 16 + m16] = s.m[t];
                stat_l[wave][t * 16 + m16] = l;
            }
        }
        __syncthreads();
        const bool whole = t0 == 0 && count == tiles.count;
        const int64_t slot = ((int64_t)worker * 2 + place) * a.cache.n_kv + h;
        if (t0 == 0 && !whole) {
            note_row = seq.q0 * a.group + rb * RB;
            note_rows = min(RB, rows - rb * RB);
            note_parts = (int)(last / run) - worker + 1;
            note_place = place;
        }
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
            constexpr int PER = D / 4;                   // threads of a row, four channels each
            for (int i = threadIdx.x; i < 16 * PER; i += kThreads) {
                const int row = i / PER, ch = i % PER * 4, r = rb * RB + t * 16 + row;
                if (r >= rows) continue;
                f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int v = 0; v < kWaves; ++v) o += *reinterpret_cast<const f32x4 *>(&joint[v][row * PAD + ch]);
                float mm = kNone, l = 0.0f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) mm = fmaxf(mm, stat_m[v][t * 16 + row]);
#pragma unroll
                for (int v = 0; v < kWaves; ++v)
                    l += stat_l[v][t * 16 + row] * __builtin_amdgcn_exp2f(stat_m[v][t * 16 + row] - mm);
                if (whole) {
                    const int tok = r / a.group, hq = h * a.group + r - tok * a.group;
                    store_out(a.out + ((int64_t)(seq.q0 + tok) * a.n_q + hq) * D + ch, o, l);
                } else {
                    const int64_t to = slot * RB + t * 16 + row;
                    *reinterpret_cast<f32x4 *>(a.part + to * D + ch) = o;
                    if (ch == 0) {
                        a.stats[to * 2] = mm;
                        a.stats[to * 2 + 1] = l;
                    }
                }
            }
            __syncthreads();
        }
        place = 1;
    }
    if (!a.whole && h == 0 && threadIdx.x == 0) {
        int32_t *n = a.notes + worker * 4;
        n[0] = note_row;
        n[1] = note_rows;
        n[2] = note_parts;
        n[3] = note_place;
    }
}

// Many row blocks with few tokens each: a wave takes one to itself, so nothing is
// joined and no wave waits for another.  Row block `item` of a kv head is found without
// a pass over the sequences: sequence b's numbers begin at rows_before(b) / RB + b, which
// leaves each of them room enough.
template <int D, int QT, int OCC>
__global__ __launch_bounds__(64, OCC) void kv_attend_wave_kernel(Args a)
{
    constexpr int DT = D / 16, RB = 16 * QT;
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
    const int h = blockIdx.x % a.cache.n_kv, item = blockIdx.x / a.cache.n_kv;
    auto number = [&](int b) {
        const int before = min(max(a.batch.cu_q[b], 0), (int)a.batch.tokens);
        return (int64_t)before * a.group / RB + b;
    };
    int b = 0;                                               // the last sequence that begins at or before `item`
    for (int many = a.batch.batch; many > 0;) {
        const int step = (many + 63) / 64, p = lane * step;
        const int n = __popcll(__ballot(p < many && number(b + p) <= item));
        if (n == 0) return;                                  // before the first one: padding
        b += (n - 1) * step;
        many = step > 1 ? min(step, many - (n - 1) * step) : 0;
    }
    const KvSeq seq = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
    const int rows = seq.n * a.group, rb = item - (int)number(b);
    if (rb < 0 || rb * RB >= rows) return;
    const Tiles tiles = visible_tiles(a, seq);
    Wave<D, QT> s;
    begin(s, a, seq, h, rb);
    attend_tiles<1>(s, a, seq, b, h, tiles, 0, tiles.count, seq.ctx + rb * RB / a.group,
                    seq.ctx + (min(rb * RB + RB, rows) - 1) / a.group);
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = rb * RB + t * 16 + m16, tok = r / a.group;
        const float l = column_sum(s.l[t]);
        if (r >= rows) continue;
        uint16_t *to = a.out + ((int64_t)(seq.q0 + tok) * a.n_q + h * a.group + r - tok * a.group) * D + g * 4;
#pragma unroll
        for (int d = 0; d < DT; ++d) store_out(to + d * 16, s.o[t][d], l);
    }
}

// Joins the parts of a row block that several workers shared: a workgroup per
// row, D / 4 lanes side by side, the parts dealt out to its NW waves and to as
// many places in a wave as there is room for.  Bound by latency (a note, then the
// parts, eight at a time): 3 to 5 us.
template <int D, int QT, int NW>
__global__ __launch_bounds__(64 * NW) void kv_join_kernel(Args a)
{
    constexpr int RB = 16 * QT, PER = D / 4, SIDE = 64 / PER;
    __shared__ float wave_m[NW], wave_l[NW];
    __shared__ f32x4 wave_o[NW][PER];
    const int row = blockIdx.x % RB, h = blockIdx.x / RB % a.cache.n_kv, worker = blockIdx.x / RB / a.cache.n_kv;
    const int32_t *n = a.notes + worker * 4;
    const int parts = n[2];
    if (row >= n[1] || parts == 0) return;
    const int r = n[0] + row, tok = r / a.group, hq = h * a.group + r - tok * a.group, place = n[3];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, ch = lane % PER * 4;
    auto slot = [&](int p) {
        return (((int64_t)(worker + p) * 2 + (p == 0 ? place : 0)) * a.cache.n_kv + h) * RB + row;
    };
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float m = kNone, l = 0.0f;
    if (lane < PER * SIDE) {
        // eight parts on their way at a time, each group against its own maximum
        for (int p0 = wave * SIDE + lane / PER; p0 < parts; p0 += 8 * NW * SIDE) {
            f32x4 x[8];
            float pm[8], pl[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int p = p0 + i * NW * SIDE;
                pm[i] = kNone;
                pl[i] = 0.0f;
                x[i] = f32x4{0.f, 0.f, 0.f, 0.f};
                if (p < parts) {
                    const int64_t s = slot(p);
                    pm[i] = a.stats[s * 2];
                    pl[i] = a.stats[s * 2 + 1];
                    x[i] = *reinterpret_cast<const f32x4 *>(a.part + s * D + ch);
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
    }
    // the places of a wave, then the waves
    float top = m;
#pragma unroll
    for (int i = 1; i < SIDE; ++i) top = fmaxf(top, __shfl(m, (lane % PER) + i * PER));
    top = fmaxf(top, __shfl(m, lane % PER));
    const float f = __builtin_amdgcn_exp2f(m - top);
    o *= f;
    l *= f;
    f32x4 sum = o;
    float sum_l = l;
#pragma unroll
    for (int i = 1; i < SIDE; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += __shfl(o[e], lane + i * PER);
        sum_l += __shfl(l, lane + i * PER);
    }
    if (lane < PER) {
        wave_o[wave][lane] = sum;
        if (lane == 0) {
            wave_m[wave] = top;
            wave_l[wave] = sum_l;
        }
    }
    __syncthreads();
    if (threadIdx.x >= PER) return;
    top = kNone;
#pragma unroll
    for (int v = 0; v < NW; ++v) top = fmaxf(top, wave_m[v]);
    sum = f32x4{0.f, 0.f, 0.f, 0.f};
    sum_l = 0.0f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
        const float w = __builtin_amdgcn_exp2f(wave_m[v] - top);
        sum += wave_o[v][lane] * w;
        sum_l += wave_l[v] * w;
    }
    store_out(a.out + ((int64_t)tok * a.n_q + hq) * D + ch, sum, sum_l);
}

template <int D, int NW, int QT>
__global__ __launch_bounds__(64 * NW, 2) void kv_attend_rows_kernel(Args a, int splits)
{
    attend_rows<D, NW, QT, false>(a, splits, blockIdx.x, gridDim.x);
}

// Joins the `splits` parts of every row of the batch's sequences: D / 4 threads a row,
// four channels each, bound by the parts' way in (512 queries of 64 heads, two cuts of
// d = 128: 9.3 us).
template <int D>
__global__ __launch_bounds__(kThreads) void kv_join_rows_kernel(Args a, int splits)
{
    constexpr int PER = D / 4;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x, row = i / PER;
    const int ch = (int)(i - row * PER) * 4;
    if (row >= a.batch.tokens * a.n_q) return;
    const int tok = (int)(row / a.n_q);
    // a row of no sequence, or of one that was skipped, is left as it was
    int lo = 0, hi = a.batch.batch;                        // the last sequence that starts at or before the row
    while (lo + 1 < hi) {
        const int mid = (lo + hi) / 2;
        if (a.batch.cu_q[mid] <= tok) lo = mid; else hi = mid;
    }
    const KvSeq s = kv_seq(a.batch, lo, a.cache.slots, a.page_shift);
    if (tok < s.q0 || tok >= s.q0 + s.n) return;
    float m = kNone;
    for (int p = 0; p < splits; ++p) m = fmaxf(m, a.stats[(row * splits + p) * 2]);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.0f;
    for (int p = 0; p < splits; ++p) {
        const float f = __builtin_amdgcn_exp2f(a.stats[(row * splits + p) * 2] - m);
        l += a.stats[(row * splits + p) * 2 + 1] * f;
        o += *reinterpret_cast<const f32x4 *>(a.part + (row * splits + p) * D + ch) * f;
    }
    store_out(a.out + row * D + ch, o, l);
}

// Waves per SIMD that the split kernel's registers allow (three would fit for d = 64 and
// one block of rows, but take longer: 32 ragged sequences of 8000 tokens 34.8 us, 37.2).
constexpr int split_occupancy(int d, int qt) { return (d <= 64 && qt <= 2) || (d <= 128 && qt == 1) ? 2 : 1; }

// How a call is run.  qt > 0: the split kernel with qt blocks of 16 rows, as many
// as an average sequence fills.  qt == 0: the rows kernel with `waves` waves and
// `splits` runs of tiles.
struct Plan {
    int qt, waves, splits, workers;
    int alone;                   // waves that have a row block to themselves, 0: none, workers' runs share them
    int64_t items, parts;        // row blocks of the rows kernel (an upper bound); rows of workspace, whatever the lengths
};

// Sequences have about `most` tokens at most, and a row sees at most `span` of them.
Plan plan_for(int64_t tokens, int batch, int n_q, int n_kv, int d, int64_t most, int64_t span)
{
    Plan p = {};
    const int64_t group = n_q / n_kv, rows = (tokens + batch - 1) / batch * group;
    // the rows kernel with these would be half idle (8 x 5 rows of 8 query heads on 4000
    // tokens: 40 us, 42 in the rows kernel; 3 rows 32 and 43; d = 64 with 20 rows on 8000 29 and 42)
    if (rows <= (d <= 128 ? 48 : 16)) {
        p.qt = (int)(rows + 15) / 16;
        const int groups = 256 * split_occupancy(d, p.qt);       // workgroups that the 256 CUs hold at once
        p.workers = n_kv < groups ? (groups + n_kv - 1) / n_kv : 1;
        p.parts = (int64_t)p.workers * n_kv * 2 * 16 * p.qt;
        // Where rows see few tokens, a row block is left whole, which saves the second launch:
        // a workgroup for each or, with many, a wave.  By what each costs (us; a round is what
        // the CUs hold): 32 heads and 500 tokens, cut, a workgroup, a wave: 10.4, 9.1, 15.7;
        // 1000 tokens 10.6, 12.4; 64 x 250 tokens on average, 8 kv heads 21.3, 11.6, 13.6;
        // 256 x 250 49.6, 47.5, 26.7; 1024 x 250 216, 335, 122; 128 x 1000 46, 42, 48.
        // Only up to 32 tiles: the host sees no more than what the table holds, and one long
        // sequence among short ones would keep its wave busy alone.
        const int rb = 16 * p.qt;
        const double all = (double)((rows + rb - 1) / rb * batch * n_kv) / groups;           // in rounds
        const double tiles = (double)std::min(most, span + rb / group + 2 * kTile) / kTile;
        const double tile = split_occupancy(d, p.qt) == 2 ? 0.45 : 0.8;
        const double cut = 9.5 + tile * std::max((tiles + kStart) * all, (double)kWaves);
        const double group4 = std::max(all, 1.0) * (6.0 + tile * tiles);
        const double one = std::max(all / 4, 1.0) * (6.0 + 4 * tile * tiles);
        if (tiles <= 32 && std::min(group4, one) < cut) {
            p.alone = one < group4 ? 1 : kWaves;
            p.workers = (int)(tokens * group / rb + batch);
        }
        return p;
    }
    // Waves and cuts by what they cost: a workgroup takes 8 us and 2 a tile, one of four
    // waves 2.3 where two share a CU and 1.3 alone; cuts cost a second launch and the
    // parts' way out and back at 4 TB/s.  (64 query heads on 8, four against eight waves:
    // 512 queries on 8k tokens 157 and 139 us, 2048 on 6144 467 and 410, 512 on none 20.7
    // and 25.5, 32 x 40 on 2000 124 and 130.  Cuts: 512 on 8k uncut 310, in
    // two 159; 2 x 1500 in a window of 1024, d = 256, 102 and 120; 32 x 8 on 2k 52 and 62.)
    // No more than four rounds of cut ones: the parts, at most 2^18 rows, stay small (16
    // cuts of 100000 rows of 64 heads would be 53 GB), and an uneven end among more
    // rounds costs little.
    double best = 0.0;
    for (int waves = d == 256 ? 8 : 4; waves <= 8; waves += 4) {
        const int64_t rb = (d == 256 ? 16 : 32) * waves, places = waves == 4 ? 512 : 256;
        const int64_t groups = (rows + rb - 1) / rb * batch * n_kv;
        const double tiles = (double)std::min(most, span + rb / group + 2 * kTile) / kTile;
        for (int cuts = 1; cuts <= 16 && (cuts == 1 || groups * cuts <= 4 * places); ++cuts) {
            const int64_t full = groups * cuts / places, rest = groups * cuts % places;
            const double pair = waves == 4 ? 2.3 : 2.0, last = waves == 4 && rest <= 256 ? 1.3 : pair;
            const double run = tiles / cuts, cost = (double)full * (8.0 + run * pair) + (rest ? 8.0 + run * last : 0.0) +
                (cuts > 1 ? 5.0 + (double)(tokens * n_q) * cuts * d * 8 / 4e6 : 0.0);
            if (p.waves == 0 || cost < best) {
                best = cost;
                p.waves = waves;
                p.splits = cuts;
            }
            if (cuts > 1) p.parts = std::max(p.parts, tokens * n_q * cuts);
        }
    }
    p.items = tokens * group / ((d == 256 ? 16 : 32) * p.waves) + batch;
    return p;
}

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
