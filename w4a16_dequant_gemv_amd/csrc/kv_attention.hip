// kv_attention.hip -- attention over the paged INT8 cache (kv_codec.h).
//
// Mathematics.  With page scales ks, vs and codes a, c the output row is
//   o = sum_j p_j vs c_j / sum_j p_j,   p_j = 2^(x_j),  x_j = log2(e) scale ks q . a_j.
// The products q . a_j use the fp16 query and the exact integer codes; the
// scales are applied to the fp32 sums.  vs goes into the exponent: with
// e_j = x_j + log2(vs) and a running maximum m of the e_j, P_j = 2^(e_j - m),
//   O = sum P_j c_j,  l = sum P_j / vs,  o = O / l,
// so the second product also takes plain integer codes, and pages of very
// different scales cannot overflow P.  The unfinished page is read from the
// fp16 ring with ks = vs = 1.
//
// Layout.  A wave takes tiles of 64 tokens.  S^T = K Q^T with
// v_mfma_f32_16x16x32_f16: a lane holds scores of one query (column lane % 16)
// and of tokens 16 g + 4 a + i (g = lane / 16).  The second product O^T = V^T P^T
// wants from the same lane P of the same query and 8 consecutive tokens of
// 16 g .. 16 g + 15 at a time: its own registers, since K rows are stored in the
// order that puts them there (kv_k_index).  P never leaves the lane, and K and
// V pages are read straight into operand registers in contiguous 16-byte loads.
#include "kv_device.h"
#include "q4_launch.h"

namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kTile = 64;                  // tokens
constexpr float kNone = -1e30f;            // running maximum before any token: below every score
constexpr float kLift = 14.0f;             // P is at most 2^14: fp16 keeps weights down to 2^-28 of the largest normal

// 16 codes of a lane as two operands, channel or token order kept.  The byte
// c + 128 under the exponent of 1024 is the fp16 value 1152 + c, exactly.
__device__ __forceinline__ void codes_to_half(u32x4 w, f16x8 &lo, f16x8 &hi)
{
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = w[i] ^ 0x80808080u;
        const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
        const f16x2 p = bitcast<f16x2>(__builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias;
        const f16x2 q = bitcast<f16x2>(__builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias;
        if (i < 2) { a[2 * i] = bitcast<uint32_t>(p); a[2 * i + 1] = bitcast<uint32_t>(q); }
        else { b[2 * i - 4] = bitcast<uint32_t>(p); b[2 * i - 3] = bitcast<uint32_t>(q); }
    }
    lo = bitcast<f16x8>(a);
    hi = bitcast<f16x8>(b);
}

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Over the four lanes that hold one query's tokens.
__device__ __forceinline__ float column_max(float v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(bitcast<uint32_t>(v), bitcast<uint32_t>(v), false, false);
    v = fmaxf(bitcast<float>(a[0]), bitcast<float>(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(v), bitcast<uint32_t>(v), false, false);
    return fmaxf(bitcast<float>(b[0]), bitcast<float>(b[1]));
}

__device__ __forceinline__ float column_sum(float v)
{
    const auto a = __builtin_amdgcn_permlane16_swap(bitcast<uint32_t>(v), bitcast<uint32_t>(v), false, false);
    v = bitcast<float>(a[0]) + bitcast<float>(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(bitcast<uint32_t>(v), bitcast<uint32_t>(v), false, false);
    return bitcast<float>(b[0]) + bitcast<float>(b[1]);
}

struct Args {
    kv_paged_cache cache;
    kv_paged_batch batch;
    const uint16_t *q;
    int64_t q_stride;
    int n_q, group;              // query heads, and those per kv head
    float scale;                 // times log2(e)
    int window, sinks, page_shift;
    int workers;                 // per kv head
    float *stats, *part;         // of unfinished row blocks
    uint16_t *out;
};

// The tiles that some row of a sequence sees: the first `head` ones and those
// from `first` to the end (`count` in all).
struct Tiles {
    int head, first, count;
    __device__ int at(int i) const { return i < head ? i : i - head + first; }
};

__device__ __forceinline__ Tiles visible_tiles(const Args &a, const KvSeq &s)
{
    Tiles t = {0, 0, (s.total() + kTile - 1) / kTile};
    if (a.window > 0) {
        const int lo = max(s.ctx - a.window + 1, 0);               // the first row's first token
        t.first = lo / kTile;
        t.head = min((min(a.sinks, lo) + kTile - 1) / kTile, t.first);
        t.count -= t.first - t.head;
    }
    return t;
}

// A run of row blocks' tiles as numbered units: sequence after sequence, its row
// blocks of RB rows one after the other, each with the sequence's tiles.
template <int RB>
__device__ __forceinline__ int64_t seq_units(const Args &a, int b)
{
    const KvSeq s = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
    return s.n ? (int64_t)((s.n * a.group + RB - 1) / RB) * visible_tiles(a, s).count : 0;
}

template <int RB>
__device__ __forceinline__ int64_t all_units(const Args &a)
{
    const int lane = threadIdx.x & 63;
    int64_t n = 0;
    for (int b = lane; b < a.batch.batch; b += 64) n += seq_units<RB>(a, b);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
    return n;
}

// How many workers of a kv head share `units` of work: no fewer than four tiles
// (one for each wave) for a worker.
__device__ __forceinline__ int64_t used_workers(const Args &a, int64_t units)
{
    return max(min((int64_t)a.workers, (units + kWaves - 1) / kWaves), (int64_t)1);
}

// One wave's state for QT blocks of 16 rows.
template <int D, int QT>
struct Wave {
    static constexpr int DT = D / 16, KS = (D + 63) / 64;
    f16x8 q[QT][2 * KS];
    f32x4 o[QT][DT];
    float m[QT], l[QT];
    int at[QT];                  // the row's index in its sequence
};

// Scores to weights: masks, running maximum, P in two fp16 parts.  c1 = scale
// log2(e) ks, w = log2(vs), inv = 1 / vs.
template <int D, int QT>
__device__ __forceinline__ void weights(Wave<D, QT> &s, int t, f32x4 x[4], const Args &a, bool masked, int tile0,
                                        float c1, float w, float inv, f16x8 hi[2], f16x8 lo[2])
{
    constexpr int DT = D / 16;
    const int g = (threadIdx.x & 63) >> 4;
    float top = kNone;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float e = x[i][j] * c1 + w;
            if (masked) {
                const int tok = tile0 + 16 * g + 4 * i + j;
                const bool see = tok <= s.at[t] && (a.window == 0 || s.at[t] - tok < a.window || tok < a.sinks);
                e = see ? e : -INFINITY;
            }
            x[i][j] = e;
            top = fmaxf(top, e);
        }
    const float m = fmaxf(s.m[t], column_max(top));
    const float keep = __builtin_amdgcn_exp2f(s.m[t] - m);
    s.m[t] = m;
    const float sub = m - kLift;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = __builtin_amdgcn_exp2f(x[i][j] - sub);
            sum += p;
            const _Float16 h = (_Float16)p;
            hi[i >> 1][(i & 1) * 4 + j] = h;
            lo[i >> 1][(i & 1) * 4 + j] = (_Float16)(p - (float)h);
        }
    s.l[t] = s.l[t] * keep + sum * inv;
    if (__ballot(keep != 1.0f)) {
#pragma unroll
        for (int d = 0; d < DT; ++d) s.o[t][d] *= keep;
    }
}

// Tiles t0, t0 + 4, ... < t1 of one row block, into the wave's state.
template <int D, int QT>
__device__ __forceinline__ void attend_tiles(Wave<D, QT> &s, const Args &a, const KvSeq &seq, int b, int h,
                                             const Tiles &tiles, int t0, int t1, int at_min, int at_max)
{
    constexpr int DT = D / 16, KS = (D + 63) / 64;
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
    const int n_kv = a.cache.n_kv, page = 1 << a.page_shift, head = page * D;
    const int full = seq.total() >> a.page_shift << a.page_shift;      // tokens in finished pages
    const bool mine = 4 * (KS - 1) + g < DT;                           // the last K load's channels exist (D = 96)
    int n = t1 > t0 ? (t1 - t0 + kWaves - 1) / kWaves : 0;

    // byte offsets inside a tile's K and V
    const int k_lane = (g * 16 + m16) * 16, v_lane = (g * D + m16) * 16;

    for (int base = 0; base < n; base += 64) {
        // lane i: the tile base + i of the wave
        int tok0 = 0, id = 0;
        float c1 = 0.0f, w = -INFINITY, inv = 0.0f;
        const int many = min(n - base, 64);
        if (lane < many) {
            tok0 = tiles.at(t0 + (base + lane) * kWaves) * kTile;
            if (tok0 < full) {
                const int e = a.batch.block_table[(int64_t)b * a.batch.table_cols + (tok0 >> a.page_shift)];
                if (e >= 0 && e < a.cache.pages) {
                    id = e;
                    const float vs = a.cache.v_scale[(int64_t)e * n_kv + h];
                    c1 = a.scale * a.cache.k_scale[(int64_t)e * n_kv + h];
                    w = __builtin_amdgcn_logf(vs);
                    inv = 1.0f / vs;
                }
            }
        }
        const int in_pages = __popcll(__ballot(lane < many && tok0 < full));

        u32x4 kr[4][KS], vr[DT];
        auto load_k = [&](int i) {
            const int t = __builtin_amdgcn_readlane(tok0, i) & (page - 1);
            const int8_t *p = a.cache.k + ((int64_t)__builtin_amdgcn_readlane(id, i) * n_kv + h) * head + t * D;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < KS; ++c) {
                    kr[j][c] = u32x4{0u, 0u, 0u, 0u};
                    if (c < KS - 1 || D % 64 == 0 || mine)
                        kr[j][c] = *reinterpret_cast<const u32x4 *>(p + k_lane + (j * DT + c * 4) * 256);
                }
        };
        auto load_v = [&](int i) {
            const int t = __builtin_amdgcn_readlane(tok0, i) & (page - 1);
            const int8_t *p = a.cache.v + ((int64_t)__builtin_amdgcn_readlane(id, i) * n_kv + h) * head + t * D;
#pragma unroll
            for (int d = 0; d < DT; ++d) vr[d] = *reinterpret_cast<const u32x4 *>(p + v_lane + d * 256);
        };
        auto is_masked = [&](int tile0) {
            return tile0 + kTile - 1 > at_min ||
                   (a.window > 0 && at_max - tile0 >= a.window && tile0 + kTile > a.sinks);
        };

        if (in_pages) {
            load_k(0);
            load_v(0);
        }
        for (int i = 0; i < in_pages; ++i) {
            const int tile0 = __builtin_amdgcn_readlane(tok0, i);
            const float c = bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(c1), i));
            const float lw = bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(w), i));
            const float iv = bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(inv), i));
            f32x4 x[QT][4];
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) x[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < KS; ++e) {
                    f16x8 lo, hi;
                    codes_to_half(kr[j][e], lo, hi);
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        x[t][j] = mfma(lo, s.q[t][2 * e], x[t][j]);
                        x[t][j] = mfma(hi, s.q[t][2 * e + 1], x[t][j]);
                    }
                }
            if (i + 1 < in_pages) load_k(i + 1);
            const bool masked = is_masked(tile0);
            f16x8 ph[QT][2], pl[QT][2];
#pragma unroll
            for (int t = 0; t < QT; ++t) weights<D, QT>(s, t, x[t], a, masked, tile0, c, lw, iv, ph[t], pl[t]);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                f16x8 lo, hi;
                codes_to_half(vr[d], lo, hi);
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    s.o[t][d] = mfma(lo, ph[t][0], s.o[t][d]);
                    s.o[t][d] = mfma(hi, ph[t][1], s.o[t][d]);
                    s.o[t][d] = mfma(lo, pl[t][0], s.o[t][d]);
                    s.o[t][d] = mfma(hi, pl[t][1], s.o[t][d]);
                }
            }
            if (i + 1 < in_pages) load_v(i + 1);
        }

        // tiles of the unfinished page, from the ring
        for (int i = in_pages; i < many; ++i) {
            const int tile0 = __builtin_amdgcn_readlane(tok0, i);
            const int64_t at = ((int64_t)seq.slot * 2 + (tile0 >> a.page_shift & 1)) * n_kv + h;
            const uint16_t *kp = a.cache.k_tail + at * head + (tile0 & (page - 1)) * D + k_lane;
            const uint16_t *vp = a.cache.v_tail + at * head + (tile0 & (page - 1)) * D + v_lane;
            f32x4 x[QT][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int t = 0; t < QT; ++t) x[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < KS; ++e) {
                    u32x4 lo = {0u, 0u, 0u, 0u}, hi = {0u, 0u, 0u, 0u};
                    if (e < KS - 1 || D % 64 == 0 || mine) {
                        lo = *reinterpret_cast<const u32x4 *>(kp + (j * DT + e * 4) * 256);
                        hi = *reinterpret_cast<const u32x4 *>(kp + (j * DT + e * 4) * 256 + 8);
                    }
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        x[t][j] = mfma(bitcast<f16x8>(lo), s.q[t][2 * e], x[t][j]);
                        x[t][j] = mfma(bitcast<f16x8>(hi), s.q[t][2 * e + 1], x[t][j]);
                    }
                }
            }
            f16x8 ph[QT][2], pl[QT][2];
#pragma unroll
            for (int t = 0; t < QT; ++t) weights<D, QT>(s, t, x[t], a, true, tile0, a.scale, 0.0f, 1.0f, ph[t], pl[t]);
            // places behind the last token hold anything: zero them, 0 * NaN is not 0
            const int left = seq.total() - tile0 - 16 * g;
            u32x4 keep[2];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                keep[e >> 2][e & 3] = left >= 2 * e + 2 ? 0xFFFFFFFFu : left == 2 * e + 1 ? 0xFFFFu : 0u;
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(vp + d * 256) & keep[0];
                const u32x4 hi = *reinterpret_cast<const u32x4 *>(vp + d * 256 + 8) & keep[1];
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    s.o[t][d] = mfma(bitcast<f16x8>(lo), ph[t][0], s.o[t][d]);
                    s.o[t][d] = mfma(bitcast<f16x8>(hi), ph[t][1], s.o[t][d]);
                    s.o[t][d] = mfma(bitcast<f16x8>(lo), pl[t][0], s.o[t][d]);
                    s.o[t][d] = mfma(bitcast<f16x8>(hi), pl[t][1], s.o[t][d]);
                }
            }
        }
    }
}

// One kv head's work is cut into equal runs of units, one for each worker (a
// workgroup), whatever the sequences' lengths; a worker's four waves take its
// tiles in turn and join at the end of each row block.  A row block that one
// worker has whole is finished there; the others' parts go to the workspace.
template <int D, int QT>
__global__ __launch_bounds__(kThreads, QT == 1 && D <= 128 ? 2 : 1) void kv_attend_split_kernel(Args a)
{
    constexpr int DT = D / 16, KS = (D + 63) / 64, RB = 16 * QT;
    constexpr int PAD = D + 4;                       // floats a row of the joining buffer: four banks on per row
    __shared__ float joint[kWaves][16 * PAD], stat_m[kWaves][RB], stat_l[kWaves][RB];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, m16 = lane & 15;
    const int h = blockIdx.x % a.cache.n_kv, worker = blockIdx.x / a.cache.n_kv;

    const int64_t units = all_units<RB>(a), used = used_workers(a, units);
    if (worker >= used) return;
    int64_t u = units * worker / used;
    const int64_t end = units * (worker + 1) / used;
    int b;
    int64_t off;
    if (u >= end || !kv_locate(a.batch.batch, u, [&](int i) { return seq_units<RB>(a, i); }, b, off)) return;

    for (bool fresh = true; u < end && b < a.batch.batch; fresh = false) {
        KvSeq seq = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
        if (seq.n == 0) { ++b; off = 0; continue; }
        const Tiles tiles = visible_tiles(a, seq);
        const int rows = seq.n * a.group, blocks = (rows + RB - 1) / RB;
        if (off >= (int64_t)blocks * tiles.count) { ++b; off = 0; continue; }
        const int rb = (int)(off / tiles.count), t0 = (int)(off - (int64_t)rb * tiles.count);
        const int count = (int)min((int64_t)(tiles.count - t0), end - u);

        Wave<D, QT> s;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = rb * RB + t * 16 + m16, tok = r / a.group;
            s.at[t] = seq.ctx + tok;
            s.m[t] = kNone;
            s.l[t] = 0.0f;
#pragma unroll
            for (int d = 0; d < DT; ++d) s.o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
            const uint16_t *row = a.q + (int64_t)(seq.q0 + tok) * a.q_stride + (h * a.group + r - tok * a.group) * D;
#pragma unroll
            for (int e = 0; e < 2 * KS; ++e) {
                const int ch = (e >> 1) * 64 + g * 16 + (e & 1) * 8;
                u32x4 v = {0u, 0u, 0u, 0u};
                if (r < rows && ch < D) v = *reinterpret_cast<const u32x4 *>(row + ch);
                s.q[t][e] = bitcast<f16x8>(v);
            }
        }
        const int at_min = seq.ctx + rb * RB / a.group;
        const int at_max = seq.ctx + (min(rb * RB + RB, rows) - 1) / a.group;
        attend_tiles<D, QT>(s, a, seq, b, h, tiles, t0 + wave, t0 + count, at_min, at_max);

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
        const int64_t slot = ((int64_t)worker * 2 + (fresh ? 0 : 1)) * a.cache.n_kv + h;
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
                    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                    const int tok = r / a.group, hq = h * a.group + r - tok * a.group;
                    const f16x2 x = {(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)};
                    const f16x2 y = {(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)};
                    *reinterpret_cast<u32x2 *>(a.out + ((int64_t)(seq.q0 + tok) * a.n_q + hq) * D + ch) =
                        u32x2{bitcast<uint32_t>(x), bitcast<uint32_t>(y)};
                } else {
                    *reinterpret_cast<f32x4 *>(a.part + (slot * RB + t * 16 + row) * D + ch) = o;
                    if (ch == 0) {
                        a.stats[(slot * RB + t * 16 + row) * 2] = mm;
                        a.stats[(slot * RB + t * 16 + row) * 2 + 1] = l;
                    }
                }
            }
            __syncthreads();
        }
        u += count;
        off += count;
    }
}

// Joins the parts of row blocks that several workers shared: one workgroup per
// query row and head, eight threads' worth of parts at a time.
template <int D, int QT>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(Args a)
{
    constexpr int RB = 16 * QT, PER = D / 4, LANES = kThreads / PER;     // parts read side by side
    __shared__ float sum[LANES][D], sum_l[LANES];
    const int64_t item = blockIdx.x;
    const int hq = (int)(item % a.n_q), row_of_call = (int)(item / a.n_q), h = hq / a.group;
    int b = 0;
    int64_t off = 0;
    // the sequence that holds the row
    const int lane = threadIdx.x & 63;
    bool found = false;
    int64_t before = 0, units = 0;
    for (int c = 0; c < a.batch.batch; c += 64) {
        const int i = c + lane;
        int64_t n = 0;
        bool hit = false;
        if (i < a.batch.batch) {
            const KvSeq s = kv_seq(a.batch, i, a.cache.slots, a.page_shift);
            if (s.n) {
                n = seq_units<RB>(a, i);
                hit = row_of_call >= s.q0 && row_of_call < s.q0 + s.n;
            }
        }
        int64_t incl = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t up = __shfl_up(incl, o);
            if (lane >= o) incl += up;
        }
        const uint64_t any = __ballot(hit);
        if (any && !found) {
            found = true;
            const int f = __ffsll((unsigned long long)any) - 1;
            b = c + f;
            before = units + __shfl(incl - n, f);
        }
        units += __shfl(incl, 63);
    }
    if (!found) return;
    const KvSeq seq = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
    const int count = visible_tiles(a, seq).count;
    const int r = (row_of_call - seq.q0) * a.group + hq - h * a.group, rb = r / RB;
    off = before + (int64_t)rb * count;
    const int64_t used = used_workers(a, units);
    // the workers that have its units [off, off + count): worker w starts at units * w / used
    auto owner = [&](int64_t x) {
        int64_t w = x * used / units;
        while (units * (w + 1) / used <= x) ++w;
        while (units * w / used > x) --w;
        return w;
    };
    const int64_t w0 = owner(off), w1 = owner(off + count - 1);
    if (w0 == w1) return;                                    // one worker had it whole
    const int part = threadIdx.x / PER, ch = threadIdx.x % PER * 4;
    auto slot_of = [&](int64_t w) {
        // a worker's first row block of the run goes to place 0, its last to 1
        const bool first = w > w0 || units * w / used == off;
        return ((w * 2 + (first ? 0 : 1)) * a.cache.n_kv + h) * RB + r - rb * RB;
    };
    float m = kNone;
    for (int64_t w = w0 + lane; w <= w1; w += 64) m = fmaxf(m, a.stats[slot_of(w) * 2]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.0f;
    if (part < LANES) {
        for (int64_t w = w0 + part; w <= w1; w += LANES) {
            const int64_t s = slot_of(w);
            const float f = __builtin_amdgcn_exp2f(a.stats[s * 2] - m);
            l += a.stats[s * 2 + 1] * f;
            o += *reinterpret_cast<const f32x4 *>(a.part + s * D + ch) * f;
        }
        *reinterpret_cast<f32x4 *>(&sum[part][ch]) = o;
        if (ch == 0) sum_l[part] = l;
    }
    __syncthreads();
    if (threadIdx.x < PER) {
        o = f32x4{0.f, 0.f, 0.f, 0.f};
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < LANES; ++i) {
            o += *reinterpret_cast<const f32x4 *>(&sum[i][ch]);
            l += sum_l[i];
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        const f16x2 x = {(_Float16)(o[0] * inv), (_Float16)(o[1] * inv)};
        const f16x2 y = {(_Float16)(o[2] * inv), (_Float16)(o[3] * inv)};
        *reinterpret_cast<u32x2 *>(a.out + ((int64_t)row_of_call * a.n_q + hq) * D + ch) =
            u32x2{bitcast<uint32_t>(x), bitcast<uint32_t>(y)};
    }
}

// Blocks of 16 rows that a wave holds: as many as an average sequence fills,
// within the registers (D = 256 leaves room for two).
int row_blocks(int64_t tokens, int batch, int group, int d)
{
    const int64_t rows = (tokens + batch - 1) / batch * group;
    return rows <= 16 ? 1 : rows <= 32 || d > 128 ? 2 : 4;
}

// Two workgroups per CU: 512 on the 256 CUs, shared by the kv heads.
int workers(int n_kv) { return n_kv < 512 ? (512 + n_kv - 1) / n_kv : 1; }

template <int D, int QT>
hipError_t launch(const Args &a, hipStream_t stream)
{
    kv_attend_split_kernel<D, QT><<<(unsigned)(a.workers * a.cache.n_kv), kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    kv_join_kernel<D, QT><<<(unsigned)(a.batch.tokens * a.n_q), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t kv_attention_workspace(int64_t tokens, int batch, int n_q, int n_kv, int d)
{
    const int64_t rows = (int64_t)workers(n_kv) * n_kv * 2 * 16 * row_blocks(tokens, batch, n_q / n_kv, d);
    return rows * (d + 2) * 4;
}

hipError_t kv_launch_attention(const kv_paged_cache &cache, const kv_paged_batch &batch, const uint16_t *q,
                               int64_t q_stride, int n_q, float scale, int window, int sinks, void *workspace,
                               uint16_t *out, hipStream_t stream)
{
    Args a = {cache, batch, q, q_stride, n_q, n_q / cache.n_kv, scale * 1.44269504f, window, sinks,
              __builtin_ctz(cache.page), workers(cache.n_kv), nullptr, nullptr, out};
    const int qt = row_blocks(batch.tokens, batch.batch, a.group, cache.d);
    a.part = (float *)workspace;
    a.stats = a.part + (int64_t)a.workers * cache.n_kv * 2 * 16 * qt * cache.d;
    switch (cache.d * 8 + qt) {
    case 64 * 8 + 1: return launch<64, 1>(a, stream);
    case 64 * 8 + 2: return launch<64, 2>(a, stream);
    case 64 * 8 + 4: return launch<64, 4>(a, stream);
    case 96 * 8 + 1: return launch<96, 1>(a, stream);
    case 96 * 8 + 2: return launch<96, 2>(a, stream);
    case 96 * 8 + 4: return launch<96, 4>(a, stream);
    case 128 * 8 + 1: return launch<128, 1>(a, stream);
    case 128 * 8 + 2: return launch<128, 2>(a, stream);
    case 128 * 8 + 4: return launch<128, 4>(a, stream);
    case 256 * 8 + 1: return launch<256, 1>(a, stream);
    case 256 * 8 + 2: return launch<256, 2>(a, stream);
    default: return hipErrorInvalidValue;
    }
}
