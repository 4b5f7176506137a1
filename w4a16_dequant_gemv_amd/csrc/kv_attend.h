// kv_attend.h -- attention over the paged INT8 cache (kv_codec.h): what the kernels of
// kv_attention.hip and, for sequences that share their first pages, of kv_shared.hip have in common.
//
// Mathematics.  With page scales ks, vs and codes a, c the output row is
//   o = sum_j p_j vs c_j / sum_j p_j,   p_j = 2^(x_j),  x_j = log2(e) scale ks q . a_j.
// The products q . a_j use the fp16 query and the exact integer codes; the
// scales are applied to the fp32 sums.  vs goes into the exponent: with
// e_j = x_j + log2(vs) and m a little below the running maximum of the e_j, P_j = 2^(e_j - m),
//   O = sum P_j c_j,  l = sum P_j / vs,  o = O / l,
// so the second product also takes plain integer codes, and pages of very
// different scales cannot overflow P.  The unfinished page is read from the
// fp16 ring with ks = vs = 1.  Scores are scaled first and hidden tokens set to -inf
// after that, so whatever a page's scales are (infinite or NaN where an infinity or
// NaN was quantized), a row that sees none of its tokens gets weights of 0 from it.
//
// Layout.  A wave takes tiles of 64 tokens.  S^T = K Q^T with
// v_mfma_f32_16x16x32_f16: a lane holds scores of one query (column lane % 16)
// and of tokens 16 g + 4 a + i (g = lane / 16).  The second product O^T = V^T P^T
// wants from the same lane P of the same query and 8 consecutive tokens of
// 16 g .. 16 g + 15 at a time: its own registers, since K rows are stored in the
// order that puts them there (kv_k_index).  P never leaves the lane, and K and
// V pages are read straight into operand registers in contiguous 16-byte loads.
#pragma once

#include <stdio.h>

#include <algorithm>

#include "kv_device.h"
#include "q4_launch.h"

namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kTile = 64;                  // tokens
constexpr int kStart = 4;                  // what a row block's beginning costs, in tiles
constexpr float kNone = -1e30f;            // m before any token: below every score
constexpr float kLift = 10.0f;             // m is put this many powers of two below the maximum, and raised only when the
constexpr float kSlack = 5.0f;             // maximum is this many more above it: P is at most 2^15, and fp16 keeps weights
                                           // down to 2^-34 of the largest
constexpr float kFar = 0x1p18f;            // m beyond this: an exponent and m are both rounded before they meet

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

// Four channels of o = O / l to fp16; a row that saw nothing gives zeros.
__device__ __forceinline__ void store_out(uint16_t *to, f32x4 o, float l)
{
    const float f = l == 0.0f ? 0.0f : 1.0f / l;
    const f16x2 x = {(_Float16)(o[0] * f), (_Float16)(o[1] * f)}, y = {(_Float16)(o[2] * f), (_Float16)(o[3] * f)};
    *reinterpret_cast<u32x2 *>(to) = u32x2{bitcast<uint32_t>(x), bitcast<uint32_t>(y)};
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

// Infinities and NaN among the ring's V.  In the matrix product a row would get NaN
// from a token that it does not see (0 * NaN); so they are replaced by finite values
// there, and the rows that do see such a token get NaN by their sum.  `trace` turns
// to NaN at their places.
__device__ __forceinline__ f16x8 finite(const u32x4 &x, f16x8 &trace)
{
    const f16x8 v = bitcast<f16x8>(x), zero = {}, most = {65504, 65504, 65504, 65504, 65504, 65504, 65504, 65504};
    trace = __builtin_elementwise_fma(v, zero, trace);
    return __builtin_elementwise_min(__builtin_elementwise_max(v, -most), most);
}

// Whether any of 16 weights, in the order of tokens, is of a token in the mask.
__device__ __forceinline__ bool sees(const f16x8 p[2], const u32x4 bad[2])
{
    const u32x4 x = (bitcast<u32x4>(p[0]) & bad[0]) | (bitcast<u32x4>(p[1]) & bad[1]);
    return (x[0] | x[1] | x[2] | x[3]) != 0u;
}

struct Args {
    kv_paged_cache cache;
    kv_paged_batch batch;
    const uint16_t *q;
    int64_t q_stride;
    int n_q, group;              // query heads, and those per kv head
    float scale;                 // times log2(e)
    int window, sinks, page_shift;
    int workers;                 // per kv head, of the split kernel
    bool whole;                  // a worker has a row block to itself
    double inv_workers;
    float *part, *stats;         // sums and (m, l) of unfinished row blocks
    int32_t *notes;              // [workers][4]: what the joining kernel has to do
    uint16_t *out;
};

// Sequences cu_seqs[g] .. cu_seqs[g + 1] - 1 have their first pages in common.  What all their
// rows get from those pages is computed apart, as `splits` parts of each row (all rows of a
// group against one reading of the pages); a sequence attends to its other tiles by itself, in up to
// `chunks` parts, and each row is joined from its parts: part and stats are [row of out][splits + chunks].
struct SharedArgs : Args {
    const int32_t *cu_seqs, *pages;
    int groups, max_pages;
    int splits, chunks;          // a row's parts of the shared pages, and of its sequence's own tokens
    int chunk;                   // tiles of each of these but the last

    __device__ int pages_of(int g) const { return min(min(max(pages[g], 0), max_pages), batch.table_cols); }
    // What is known of the groups before a sequence is: the sequences that they name, and the first one's pages.
    struct Named {
        int lo, hi, pages;
    };
    __device__ Named named() const { return {cu_seqs[0], cu_seqs[groups], pages_of(0)}; }
    __device__ int places() const { return splits + chunks; }
    // The tiles of sequence b that its parts of the shared pages hold: none where it has not finished the shared pages.
    __device__ int skip(const KvSeq &s, int b, const Named &all) const
    {
        if (s.n <= 0 || b < all.lo || b >= all.hi) return 0;
        int p = all.pages;
        if (groups > 1) {
            int lo = 0, hi = groups;                           // cu_seqs[lo] <= b < cu_seqs[hi]
            while (lo + 1 < hi) {
                const int mid = (lo + hi) / 2;
                if (cu_seqs[mid] <= b) lo = mid; else hi = mid;
            }
            p = pages_of(lo);
        }
        return s.ctx >> page_shift >= p ? p << (page_shift - 6) : 0;
    }
};

// The tiles that some of a sequence's rows at places lo .. hi sees: the first
// `head` ones and those from `first` on (`count` in all); with no window those from `skip` on.
struct Tiles {
    int head, first, count;
    __device__ int at(int i) const { return i < head ? i : i - head + first; }
};

__device__ __forceinline__ Tiles visible_tiles(const Args &a, int lo, int hi, int skip = 0)
{
    Tiles t = {0, skip, hi / kTile + 1 - skip};
    if (a.window > 0) {
        const int first = max(lo - a.window + 1, 0);               // the first token that the window shows
        t.first = first / kTile;
        t.head = min((min(a.sinks, first) + kTile - 1) / kTile, t.first);
        t.count -= t.first - t.head;
    }
    return t;
}

__device__ __forceinline__ Tiles visible_tiles(const Args &a, const KvSeq &s, int skip = 0)
{
    return visible_tiles(a, s.ctx, s.total() - 1, skip);
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

// Exponents x[a][i] of one query (row index `at`): those of tokens that it does not
// see become -inf.
__device__ __forceinline__ void hide(f32x4 x[4], const Args &a, int at, int tile0)
{
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tok = tile0 + 16 * g + 4 * i + j;
            const bool see = tok <= at && (a.window == 0 || at - tok < a.window || tok < a.sinks);
            x[i][j] = see ? x[i][j] : -INFINITY;
        }
}

// Scores to exponents: c1 = scale log2(e) ks > 0, w = log2(vs).
__device__ __forceinline__ void scale_scores(f32x4 x[4], float c1, float w)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = __builtin_fmaf(x[i][j], c1, w);
}

// Scores to weights.  First m, which follows the maximum of the exponents x c1 + w only
// in steps (each step costs a pass over O); returns the factor for what was summed before,
// 1 nearly always.  Where m's own units are large, kLift below the maximum may come out
// as more than kLift: then m is the maximum.
__device__ __forceinline__ float weigh_max(const f32x4 x[4], float c1, float w, float &m_run)
{
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, x[i][j]);
    const float now = __builtin_fmaf(column_max(top), c1, w), low = now - kLift;
    const float m = now - m_run > kLift + kSlack ? now - low > kLift + 1.0f ? now : low : m_run;
    const float keep = __builtin_amdgcn_exp2f(m_run - m);
    m_run = m;
    return keep;
}

// Then P in fp16, and where `lo` is given the rest of P there, for the tokens of
// the second product's step `half`; sum gets this lane's sum of P.  add = w - m: its
// rounding moves a tile's weights together by up to half a unit of m, so where that counts
// (beyond kFar) the scores have been scaled before, c1 is 1, and e - m is exact for the largest.
__device__ __forceinline__ void weigh_exp(const f32x4 x[4], int half, float c1, float add, f16x8 hi[2], float &sum,
                                          f16x8 *lo = nullptr)
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * half + i][j], c1, add));
            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[2 * half + i][j + 1], c1, add));
            sum += p0 + p1;
            const f16x2 h = {(_Float16)p0, (_Float16)p1};
            hi[half][i * 4 + j] = h[0];
            hi[half][i * 4 + j + 1] = h[1];
            if (lo) {
                lo[half][i * 4 + j] = (_Float16)(p0 - (float)h[0]);
                lo[half][i * 4 + j + 1] = (_Float16)(p1 - (float)h[1]);
            }
        }
}

template <int D, int QT>
__device__ __forceinline__ void weigh(Wave<D, QT> &s, int t, f32x4 x[4], const Args &a, bool masked, int tile0, float c1,
                                      float w, float inv, f16x8 hi[2], f16x8 lo[2])
{
    scale_scores(x, c1, w);
    if (masked) hide(x, a, s.at[t], tile0);
    const float keep = weigh_max(x, 1.0f, 0.0f, s.m[t]);
    float sum = 0.0f;
    weigh_exp(x, 0, 1.0f, -s.m[t], hi, sum, lo);
    weigh_exp(x, 1, 1.0f, -s.m[t], hi, sum, lo);
    s.l[t] = s.l[t] * keep + sum * inv;
    if (__ballot(keep != 1.0f)) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d) s.o[t][d] *= keep;
    }
}

__device__ __forceinline__ float lane_value(float v, int i)
{
    return bitcast<float>(__builtin_amdgcn_readlane(bitcast<int>(v), i));
}

// What a tile's page contributes to the scores.  A page that is not there has weight
// 2^-inf.  Scales that are not finite give NaN to every token of the page (and nothing
// to rows that see none: w and inv stay finite).  A page that nobody filled has scales
// of 0 and counts as zeros: for V, 2^-100 stands for 0 and vanishes in every output.
struct PageScales {
    float c1, w, inv;
    __device__ PageScales() : c1(1.0f), w(-INFINITY), inv(0.0f) {}
    __device__ void set(float scale, float ks, float vs)
    {
        const bool finite = ks < INFINITY && vs < INFINITY;
        vs = finite ? fmaxf(vs, 0x1p-100f) : 1.0f;
        c1 = finite ? scale * ks : NAN;
        w = __builtin_amdgcn_logf(vs);
        inv = 1.0f / vs;
    }
};

// A row block's state before its first tile: row block rb of the sequence for kv head h.
template <int D, int QT>
__device__ __forceinline__ void begin(Wave<D, QT> &s, const Args &a, const KvSeq &seq, int h, int rb)
{
    constexpr int DT = D / 16, KS = (D + 63) / 64, RB = 16 * QT;
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
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
            if (r < seq.n * a.group && ch < D) v = *reinterpret_cast<const u32x4 *>(row + ch);
            s.q[t][e] = bitcast<f16x8>(v);
        }
    }
}

// Tiles t0, t0 + STEP, ... < t1 of one row block, into the wave's state.
template <int STEP, int D, int QT>
__device__ __forceinline__ void attend_tiles(Wave<D, QT> &s, const Args &a, const KvSeq &seq, int b, int h,
                                             const Tiles &tiles, int t0, int t1, int at_min, int at_max)
{
    constexpr int DT = D / 16, KS = (D + 63) / 64;
    const int lane = threadIdx.x & 63, g = lane >> 4, m16 = lane & 15;
    const int n_kv = a.cache.n_kv, page = 1 << a.page_shift, head = page * D;
    const int full = seq.total() >> a.page_shift << a.page_shift;      // tokens in finished pages
    const bool mine = 4 * (KS - 1) + g < DT;                           // the last K load's channels exist (D = 96)
    int n = t1 > t0 ? (t1 - t0 + STEP - 1) / STEP : 0;

    // byte offsets inside a tile's K and V
    const int k_lane = (g * 16 + m16) * 16, v_lane = (g * D + m16) * 16;

    for (int base = 0; base < n; base += 64) {
        // lane i: the tile base + i of the wave
        int tok0 = 0, id = -1;
        const int many = min(n - base, 64);
        if (lane < many) {
            tok0 = tiles.at(t0 + (base + lane) * STEP) * kTile;
            if (tok0 < full) id = a.batch.block_table[(int64_t)b * a.batch.table_cols + (tok0 >> a.page_shift)];
        }
        const bool there = id >= 0 && id < a.cache.pages;
        id = there ? id : 0;                                           // a page that is not there: read page 0, weigh it 0
        const float ks = a.cache.k_scale[(int64_t)id * n_kv + h], vs = a.cache.v_scale[(int64_t)id * n_kv + h];
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
        PageScales ps;                                                 // waits for its loads behind the first tile's
        if (there) ps.set(a.scale, ks, vs);
        for (int i = 0; i < in_pages; ++i) {
            const int tile0 = __builtin_amdgcn_readlane(tok0, i);
            const float c = lane_value(ps.c1, i);
            const float lw = lane_value(ps.w, i);
            const float iv = lane_value(ps.inv, i);
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
            for (int t = 0; t < QT; ++t) weigh<D, QT>(s, t, x[t], a, masked, tile0, c, lw, iv, ph[t], pl[t]);
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
            for (int t = 0; t < QT; ++t) weigh<D, QT>(s, t, x[t], a, true, tile0, a.scale, 0.0f, 1.0f, ph[t], pl[t]);
            // places behind the last token hold anything: zero them, 0 * NaN is not 0
            const int left = seq.total() - tile0 - 16 * g;
            u32x4 keep[2];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                keep[e >> 2][e & 3] = left >= 2 * e + 2 ? 0xFFFFFFFFu : left == 2 * e + 1 ? 0xFFFFu : 0u;
            f16x8 trace[2] = {};                                       // NaN at tokens with an infinity or NaN
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const f16x8 lo = finite(*reinterpret_cast<const u32x4 *>(vp + d * 256) & keep[0], trace[0]);
                const f16x8 hi = finite(*reinterpret_cast<const u32x4 *>(vp + d * 256 + 8) & keep[1], trace[1]);
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    s.o[t][d] = mfma(lo, ph[t][0], s.o[t][d]);
                    s.o[t][d] = mfma(hi, ph[t][1], s.o[t][d]);
                    s.o[t][d] = mfma(lo, pl[t][0], s.o[t][d]);
                    s.o[t][d] = mfma(hi, pl[t][1], s.o[t][d]);
                }
            }
            u32x4 bad[2] = {bitcast<u32x4>(trace[0] != trace[0]), bitcast<u32x4>(trace[1] != trace[1])};
            const u32x4 both = bad[0] | bad[1];
            if (__ballot((both[0] | both[1] | both[2] | both[3]) != 0u)) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 4; ++e)                        // over the channels, the lanes of a group
#pragma unroll
                        for (int o = 1; o < 16; o <<= 1) bad[half][e] |= (uint32_t)__shfl_xor((int)bad[half][e], o);
#pragma unroll
                for (int t = 0; t < QT; ++t) s.l[t] = sees(ph[t], bad) ? NAN : s.l[t];
            }
        }
    }
}

// Row block `item` of RB rows, counted through all groups: the rows of its group's sequences, which lie side
// by side, as one sequence that sees all of the shared pages, the block's place there, and `b`, which
// has the pages in its block table: the group's first sequence that has finished them.  Every thread of the
// workgroup calls this.  False if there are not that many blocks, or no such sequence.
template <int RB>
__device__ __forceinline__ bool group_rows(const SharedArgs &a, int64_t item, KvSeq &seq, int &b, int64_t &rb)
{
    __shared__ int first;
    const int lane = threadIdx.x & 63, T = (int)a.batch.tokens;
    int lo = 0, hi = 0, q0 = 0, n = 0, pages = 0;
    int64_t base = 0;
    bool found = false;
    for (int c = 0; c < a.groups && !found; c += 64) {
        int64_t blocks = 0;
        const int g = min(c + lane, a.groups - 1);
        lo = min(max(a.cu_seqs[g], 0), a.batch.batch);
        hi = min(max(a.cu_seqs[g + 1], lo), a.batch.batch);
        pages = a.pages_of(g);
        q0 = min(max(a.batch.cu_q[lo], 0), T);
        n = max(min(a.batch.cu_q[hi], T) - q0, 0);
        if (c + lane < a.groups) blocks = ((int64_t)n * a.group + RB - 1) / RB;
        const int64_t incl = kv_wave_scan(blocks);
        const uint64_t hit = __ballot(item < base + incl);
        if (hit) {
            const int f = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
            rb = item - base - kv_lane(incl - blocks, f);
            lo = __builtin_amdgcn_readlane(lo, f);
            hi = __builtin_amdgcn_readlane(hi, f);
            q0 = __builtin_amdgcn_readlane(q0, f);
            n = __builtin_amdgcn_readlane(n, f);
            pages = __builtin_amdgcn_readlane(pages, f);
            found = true;
        }
        base += kv_lane(incl, 63);
    }
    if (!found || pages == 0) return false;
    if (threadIdx.x == 0) first = hi;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += blockDim.x) {
        const int i = i0 + threadIdx.x;
        bool has = false;
        if (i < hi) {
            const KvSeq s = kv_seq(a.batch, i, a.cache.slots, a.page_shift);
            has = s.n > 0 && s.ctx >> a.page_shift >= pages;
        }
        if (has) atomicMin(&first, i);
        if (__syncthreads_or(has)) break;
    }
    b = __builtin_amdgcn_readfirstlane(first);
    seq = {q0, n, (pages << a.page_shift) - n, 0};
    return b < hi;
}

// Many rows of a sequence: a workgroup of NW waves holds 16 QT NW rows (a wave QT
// blocks of 16; one for D = 256, whose sums fill the registers) and walks the tiles
// they see; each tile is converted to fp16 once, into LDS, in the order of the operands
// (a wave reads 1 KiB in a row).  Two buffers each for K and V; the tiles after them
// are on their way in registers.  Bound by the matrix cores: 2048 queries, 64 heads on
// 8, over 8192 tokens 420 us, 1.14 PFLOP/s (562 us with all waves in step).
// P goes into the second product as one fp16 value, off by up to 2^-11 of itself, where
// the kernels of few rows add the rest as a second one; l is summed from P in binary32.
// A second part here would be half as much matrix work again: 576 us for 420 above, 120
// for 103 at d = 256 (2 x 1500 in a window of 1024).  The outputs' error against 64 bits
// is 2.9e-4 of their size this way and 2.07e-4 that way, their own rounding to fp16.
// With PARTS, where a sequence may have a single row, the second part is there: a row's weights are then as exact as
// without shared pages, whichever kernel takes these (a tile 1.9 us for 1.5 with a CU to itself, 3.0 for 2.3 with two
// workgroups on each, d = 128).
// A wave's matrix work (a tile's scores, the last one's second product) and its
// vector work (weights, conversion of tiles) do not overlap by themselves, and
// waves that meet at barriers do the same at the same time; so with eight waves
// the two that share a SIMD take turns: waves 4 .. 7 run half a tile behind, and
// each barrier hands the matrix cores to the other wave.  With few row blocks the tiles
// are cut into `splits` runs and joined by kv_join_rows_kernel.
// (kv_attend_rows_kernel.  With PARTS the rows are a group's, on its shared pages, and all of them
// go out as parts: workgroup `block` of `blocks`.)
template <int D, int NW, int QT, bool PARTS, typename A>
__device__ __forceinline__ void attend_rows(const A &a, int splits, int block, int blocks)
{
    constexpr int DT = D / 16, KS = (D + 63) / 64, RB = 16 * QT * NW, THREADS = 64 * NW;
    constexpr int UNITS = 4 * D, UN = (UNITS + THREADS - 1) / THREADS;     // 16-byte units of a tile's K (and V)
    constexpr int KF = 8 * KS, VF = 2 * DT;                                // operands of 1 KiB
    extern __shared__ f16x8 k_tile[];                      // [2][KF][64], then V's [2][VF][64]
    f16x8 *v_tile = k_tile + 2 * KF * 64;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);                  // a scalar: its branches are uniform
    const int n_kv = a.cache.n_kv, page = 1 << a.page_shift, head = page * D;
    const int h = block % n_kv, split = block / n_kv % splits;
    int b;
    int64_t rb64;
    // the last row blocks, which see the most tokens, first: the short ones fill the gaps
    // at the end (2048 queries on an empty cache: 89 us, 108 in the other order)
    const int64_t item = (int64_t)(blocks - 1 - block) / n_kv / splits;
    KvSeq seq;
    if constexpr (PARTS) {
        if (!group_rows<RB>(a, item, seq, b, rb64)) return;
    } else {
        if (!kv_locate(a.batch.batch, item, [&](int i) {
                return (int64_t)((kv_seq(a.batch, i, a.cache.slots, a.page_shift).n * a.group + RB - 1) / RB);
            }, b, rb64))
            return;
        seq = kv_seq(a.batch, b, a.cache.slots, a.page_shift);
    }
    const int rows = seq.n * a.group, row0 = (int)rb64 * RB, full = seq.total() >> a.page_shift << a.page_shift;
    Tiles tiles = {0, 0, full / kTile};
    if constexpr (!PARTS)
        tiles = visible_tiles(a, seq.ctx + row0 / a.group, seq.ctx + (min(row0 + RB, rows) - 1) / a.group);
    const int t0 = (int)((int64_t)tiles.count * split / splits), t1 = (int)((int64_t)tiles.count * (split + 1) / splits);

    // this wave's rows
    const int first = row0 + wave * 16 * QT;
    const int turn = NW > 4 && wave >= 4 ? 1 : 0;
    const int at_min = PARTS ? 1 << 30 : seq.ctx + first / a.group;
    const int at_max = seq.ctx + (min(first + 16 * QT, rows) - 1) / a.group;
    f16x8 q[QT][2 * KS];
    f32x4 o[QT][DT];
    float m[QT], l[QT];
    int at[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = first + t * 16 + m16, tok = r / a.group;
        at[t] = seq.ctx + tok;
        m[t] = kNone;
        l[t] = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[t][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        const uint16_t *row = a.q + (int64_t)(seq.q0 + tok) * a.q_stride + (h * a.group + r - tok * a.group) * D;
#pragma unroll
        for (int e = 0; e < 2 * KS; ++e) {
            const int ch = (e >> 1) * 64 + g * 16 + (e & 1) * 8;
            u32x4 v = {0u, 0u, 0u, 0u};
            if (r < rows && ch < D) v = *reinterpret_cast<const u32x4 *>(row + ch);
            q[t][e] = bitcast<f16x8>(v);
        }
    }
    if (D % 64 != 0) {                                     // channels that a last K operand has beyond D
        for (int i = tid; i < 2 * KF * 64; i += THREADS) k_tile[i] = f16x8{};
        __syncthreads();
    }

    // Four operands each: for K tiles a = 2 jp, 2 jp + 1 of 16 tokens and 64 channels,
    // for V 32 channels.
    auto read_k = [&](int i, int n, f16x8 f[4]) {
        const f16x8 *from = k_tile + (i & 1) * KF * 64 + lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = from[((n / KS * 2 + (e >> 1)) * 2 * KS + n % KS * 2 + (e & 1)) * 64];
    };
    auto read_v = [&](int i, int n, f16x8 f[4]) {
        const f16x8 *from = v_tile + (i & 1) * VF * 64 + n * 256 + lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = from[e * 64];
    };
    // where unit u of a tile goes
    auto k_place = [&](int i, int unit) {
        const int c = unit / 16 % DT, ka = unit / 16 / DT;
        return k_tile + (i & 1) * KF * 64 + (ka * KS + (c >> 2)) * 128 + (c & 3) * 16 + (unit & 15);
    };
    auto v_place = [&](int i, int unit) {
        const int ch = unit % D;
        return v_tile + (i & 1) * VF * 64 + ch / 16 * 128 + unit / D * 16 + (ch & 15);
    };
    f32x4 x[QT][4];
    f16x8 p[QT][2], rest[QT][2];                           // P, and with PARTS what is left of it
    // O += P V of tile i - 1, and the scores of tile i.  Operands are read ahead, and
    // an accumulator comes up again after one or three others.  `between` is run twice, after two
    // pieces of the scores.
    auto matrix_work = [&](int i, bool second, bool first, auto between) {
        // two pieces ahead; one for d = 96 in four waves, whose registers two pieces overflow
        // (8 x 300 queries on 2000 tokens 136 us, 140 with two; 512 on 2000 72 and 73)
        constexpr int VP = DT / 2, NP = VP + 2 * KS, AHEAD = D % 64 != 0 && NW == 4 ? 1 : 2;
        f16x8 f[AHEAD + 1][4];
        auto fetch = [&](int n) {
            if (n < VP) { if (second) read_v(i - 1, n, f[n % (AHEAD + 1)]); }
            else if (n < NP) { if (first) read_k(i, n - VP, f[n % (AHEAD + 1)]); }
        };
        __builtin_amdgcn_s_setprio(1);                     // before the SIMD's other wave, whose work is long enough
#pragma unroll
        for (int n = second ? 0 : VP, k = 0; k < AHEAD; ++k) fetch(n + k);
#pragma unroll
        for (int n = second ? 0 : VP; n < (first ? NP : VP); ++n) {
            fetch(n + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 0; e < (PARTS && n < VP ? 8 : 4); ++e) {
                const int one = e & 1, half = e >> 1 & 1;              // operand 2 one + half
                const f16x8 v = f[n % (AHEAD + 1)][2 * one + half];
                if (n < VP) {
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        const f16x8 w = PARTS && e >= 4 ? rest[t][half] : p[t][half];
                        o[t][2 * n + one] = mfma(v, w, o[t][2 * n + one]);
                    }
                } else {
                    const int j = (n - VP) / KS * 2 + one, c = (n - VP) % KS * 2 + half;
                    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int t = 0; t < QT; ++t) x[t][j] = mfma(v, q[t][c], c == 0 ? zero : x[t][j]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            if (n == NP - (KS == 1 ? 2 : 4)) between(0);
            if (n == NP - (KS == 1 ? 1 : 2)) between(1);
        }
        __builtin_amdgcn_s_setprio(0);
    };
    // x to p
    bool far = false;                                      // m of some row is beyond kFar
    auto vector_work = [&](int tile0, float c1, float w, float inv) {
        if (!PARTS && (tile0 + kTile - 1 > at_min || (a.window > 0 && at_max - tile0 >= a.window && tile0 + kTile > a.sinks))) {
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                scale_scores(x[t], c1, w);
                hide(x[t], a, at[t], tile0);
            }
            c1 = 1.0f;                                     // all other tiles are scaled on the way to exp2 (425 us
            w = 0.0f;                                      // on 2048 queries over 8192 tokens, 449 in a step apart)
        }
        float keep[QT];
        bool moved = false;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            keep[t] = weigh_max(x[t], c1, w, m[t]);
            moved |= keep[t] != 1.0f;
        }
        if (__ballot(moved)) {
            bool out = false;
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                l[t] *= keep[t];
                out |= fabsf(m[t]) >= kFar && m[t] != kNone;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[t][d] *= keep[t];
            }
            far = __ballot(out) != 0;
        }
        if (far) {
#pragma unroll
            for (int t = 0; t < QT; ++t) scale_scores(x[t], c1, w);
            c1 = 1.0f;
            w = 0.0f;
        }
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float sum = 0.0f;
            weigh_exp(x[t], 0, c1, w - m[t], p[t], sum, PARTS ? rest[t] : nullptr);
            weigh_exp(x[t], 1, c1, w - m[t], p[t], sum, PARTS ? rest[t] : nullptr);
            l[t] += sum * inv;
        }
    };

    // finished pages
    int base = t0;
    for (bool more = true; more && base < t1;) {
        int tok0 = 0, id = -1;
        if (base + lane < t1) {
            tok0 = tiles.at(base + lane) * kTile;
            if (tok0 < full) id = a.batch.block_table[(int64_t)b * a.batch.table_cols + (tok0 >> a.page_shift)];
        }
        const int many = __popcll(__ballot(base + lane < t1 && tok0 < full));
        if (many == 0) break;
        const bool there = id >= 0 && id < a.cache.pages;
        id = there ? id : 0;                               // a page that is not there: read page 0, weigh it 0
        PageScales ps;
        if (there) ps.set(a.scale, a.cache.k_scale[(int64_t)id * n_kv + h], a.cache.v_scale[(int64_t)id * n_kv + h]);
        const int64_t at0 = ((int64_t)id * n_kv + h) * head + (tok0 & (page - 1)) * D;

        // tile i's codes into registers, and from there into its buffer; behind the last
        // tile the last one once more, which nothing reads
        u32x4 kr[UN], vr[UN];
        auto load = [&](const int8_t *pool, int i, u32x4 r[UN]) {
            const int8_t *from = pool + kv_lane(at0, min(i, many - 1)) + tid * 16;
#pragma unroll
            for (int u = 0; u < UN; ++u)
                if (UNITS % THREADS == 0 || tid + u * THREADS < UNITS)
                    r[u] = *reinterpret_cast<const u32x4 *>(from + u * THREADS * 16);
        };
        auto put_k = [&](int i) {
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                if (UNITS % THREADS != 0 && tid + u * THREADS >= UNITS) continue;
                f16x8 lo, hi, *to = k_place(i, tid + u * THREADS);
                codes_to_half(kr[u], lo, hi);
                to[0] = lo;
                to[64] = hi;
            }
        };
        auto put_v = [&](int i) {
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                if (UNITS % THREADS != 0 && tid + u * THREADS >= UNITS) continue;
                f16x8 lo, hi, *to = v_place(i, tid + u * THREADS);
                codes_to_half(vr[u], lo, hi);
                to[0] = lo;
                to[64] = hi;
            }
        };
        // the tiles after tile i, in two parts of its matrix work
        auto move_on = [&](int i, int part) {
            if (part == 0) {
                put_k(i + 1);
                load(a.cache.k, i + 2, kr);
            }
            if (part == 1) {
                put_v(i);
                load(a.cache.v, i + 1, vr);
            }
        };

        load(a.cache.k, 0, kr);
        load(a.cache.v, 0, vr);
        __syncthreads();                                   // the tiles before have been read
        put_k(0);
        load(a.cache.k, 1, kr);
        __syncthreads();
        if (turn) __syncthreads();
        matrix_work(0, false, true, [&](int part) { move_on(0, part); });
        __syncthreads();
        for (int i = 0; i < many; ++i) {
            vector_work(__builtin_amdgcn_readlane(tok0, i), lane_value(ps.c1, i), lane_value(ps.w, i), lane_value(ps.inv, i));
            if (NW > 4) __syncthreads();
            // behind the last tile the scores are computed from old values and not used
            matrix_work(i + 1, true, true, [&](int part) { move_on(i + 1, part); });
            __syncthreads();
        }
        if (NW > 4 && !turn) __syncthreads();
        base += many;
        more = many == 64;
    }
    // the unfinished page, from the ring
    for (; !PARTS && base < t1; ++base) {
        const int tile0 = tiles.at(base) * kTile;
        const int64_t at0 = (((int64_t)seq.slot * 2 + (tile0 >> a.page_shift & 1)) * n_kv + h) * head +
                            (tile0 & (page - 1)) * D;
        __shared__ uint32_t bad_tokens[4][8];              // all ones for such tokens, by group of 16
        __syncthreads();                                   // the tile before has been read
        if (tid < 32) bad_tokens[tid >> 3][tid & 7] = 0;
        __syncthreads();
        bool any = false;
        for (int unit = tid; unit < UNITS; unit += THREADS) {
            const u32x4 *kp = reinterpret_cast<const u32x4 *>(a.cache.k_tail + at0 + unit * 16);
            const u32x4 *vp = reinterpret_cast<const u32x4 *>(a.cache.v_tail + at0 + unit * 16);
            f16x8 *to = k_place(0, unit);
            to[0] = bitcast<f16x8>(kp[0]);
            to[64] = bitcast<f16x8>(kp[1]);
            // places behind the last token hold anything: zero them
            const int left = seq.total() - tile0 - 16 * (unit / D);
            u32x4 lo = vp[0], hi = vp[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[e] &= left >= 2 * e + 2 ? 0xFFFFFFFFu : left == 2 * e + 1 ? 0xFFFFu : 0u;
                hi[e] &= left >= 2 * e + 10 ? 0xFFFFFFFFu : left == 2 * e + 9 ? 0xFFFFu : 0u;
            }
            f16x8 trace[2] = {};
            to = v_place(0, unit);
            to[0] = finite(lo, trace[0]);
            to[64] = finite(hi, trace[1]);
            lo = bitcast<u32x4>(trace[0] != trace[0]);
            hi = bitcast<u32x4>(trace[1] != trace[1]);
            const u32x4 both = lo | hi;
            if (both[0] | both[1] | both[2] | both[3]) {
                any = true;
                for (int e = 0; e < 4; ++e) {
                    atomicOr(&bad_tokens[unit / D][e], lo[e]);
                    atomicOr(&bad_tokens[unit / D][e + 4], hi[e]);
                }
            }
        }
        const bool found = __syncthreads_or(any);
        matrix_work(0, false, true, [](int) {});
        vector_work(tile0, a.scale, 0.0f, 1.0f);
        if (found) {
            u32x4 bad[2];
            for (int e = 0; e < 8; ++e) bad[e >> 2][e & 3] = bad_tokens[g][e];
#pragma unroll
            for (int t = 0; t < QT; ++t) l[t] = sees(p[t], bad) ? NAN : l[t];
        }
        matrix_work(1, true, false, [](int) {});           // its V is in buffer 0
    }

#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = first + t * 16 + m16;
        const float sum = column_sum(l[t]);
        if (r >= rows) continue;
        const int tok = r / a.group;
        const int64_t at_out = (int64_t)(seq.q0 + tok) * a.n_q + h * a.group + r - tok * a.group;
        if (!PARTS && splits == 1) {
#pragma unroll
            for (int d = 0; d < DT; ++d) store_out(a.out + at_out * D + d * 16 + g * 4, o[t][d], sum);
        } else {
            int64_t slot = at_out * splits + split;
            if constexpr (PARTS) slot = at_out * a.places() + split;
#pragma unroll
            for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4 *>(a.part + slot * D + d * 16 + g * 4) = o[t][d];
            if (g == 0) {
                a.stats[slot * 2] = m[t];
                a.stats[slot * 2 + 1] = sum;
            }
        }
    }
}

// Where a call goes: to a stream, or with `name` nowhere, and the kernels that would have
// been launched are written there.
struct Target {
    hipStream_t stream;
    char *name;
    int64_t name_len;
    template <typename... V>
    hipError_t report(const char *format, V... values) const
    {
        snprintf(name, (size_t)name_len, format, values...);
        return hipSuccess;
    }
};

}  // namespace
