// kv_append.hip -- the paged INT8 cache's writer: rotation of new queries and
// keys, the fp16 ring, quantization of pages that become full; and the
// dequantization of listed pages.
//
// Rotation.  a' = a cos - b sin in binary64: an fp16 value times an fp32 cosine
// is exact there, so the sum is rounded once (2^-53) and then once more to
// fp16; a result in binary32 would cross the border between two codes for
// about one value in 2^12.  Pages then hold the codes of exactly the values
// that the ring holds, however the tokens were split over calls.
//
// Work split.  Per sequence and kv head one workgroup for K and one for V finish
// the page that ctx_lens ends in (old tokens from the ring, new ones from the
// call) and write the ring: where the call's last page may replace the finished
// one there, the reads come before the writes in one workgroup, so no order
// between workgroups is needed.  Pages made of new tokens only are two workgroups
// each, and q is a grid of its own behind them, all in one launch.  Bound by memory
// with many tokens (3 prompts of 5000, 64 + 2 x 8 heads of 128: 90 us, 4.4 TB/s
// with the pages read back), by latency with one (8 us: table, loads, scale, codes).
#include "kv_device.h"
#include "q4_launch.h"

namespace {

constexpr int kThreads = 256;

struct Rope {
    const float *table;          // [rows][dim / 2][2], or null
    const int32_t *positions;
    int64_t rows;
    int dim, interleaved;
};

// binary64 to fp16 with one rounding: the upper 32 bits with the lower ones
// folded into the last (rounding to odd) keep ten bits more than fp16 has, so
// the two conversions that follow round only once.
__device__ __forceinline__ _Float16 to_half_once(double x)
{
    const uint64_t b = bitcast<uint64_t>(x);
    const uint32_t hi = (uint32_t)(b >> 32) | ((uint32_t)b != 0u ? 1u : 0u);
    return (_Float16)(float)bitcast<double>((uint64_t)hi << 32);
}

struct Chunk {                   // 16 channels
    u32x4 lo, hi;
};

__device__ __forceinline__ float half_at(const Chunk &x, int e)
{
    const uint32_t w = e < 8 ? x.lo[e >> 1] : x.hi[(e - 8) >> 1];
    return half_bits_to_float((uint16_t)(w >> (16 * (e & 1))));
}

__device__ __forceinline__ Chunk load_chunk(const uint16_t *p)
{
    return {*reinterpret_cast<const u32x4 *>(p), *reinterpret_cast<const u32x4 *>(p + 8)};
}

__device__ __forceinline__ void store_chunk(uint16_t *p, const Chunk &x)
{
    *reinterpret_cast<u32x4 *>(p) = x.lo;
    *reinterpret_cast<u32x4 *>(p + 8) = x.hi;
}

__device__ __forceinline__ uint32_t pack_once(double a, double b)
{
    const f16x2 h = {to_half_once(a), to_half_once(b)};
    return bitcast<uint32_t>(h);
}

// Rotation works on units of 16 channels of a head: pairs 8 pc .. 8 pc + 7 as their
// two halves, channels c0 .. c0 + 7 and c1 .. c1 + 7 (with interleaved pairs, and
// for the channels behind rope.dim that are only copied, 16 neighbours).
struct Unit {
    int c0, c1;
    bool turned;
    __device__ Unit(const Rope &rope, int pc)
    {
        const int half = rope.dim / 2;
        turned = pc * 8 < half;
        c0 = turned && !rope.interleaved ? pc * 8 : pc * 16;
        c1 = turned && !rope.interleaved ? c0 + half : c0 + 8;
    }
};

struct Angles {                  // of a unit's pairs at one position
    double co[8], si[8];
    bool nan;
};

__device__ __forceinline__ Angles load_angles(const Rope &rope, int64_t row, int pc)
{
    Angles r;
    const int64_t pos = rope.positions[row];
    r.nan = pos < 0 || pos >= rope.rows;
    const float *cs = rope.table + (r.nan ? 0 : pos) * rope.dim + pc * 16;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const f32x4 t = *reinterpret_cast<const f32x4 *>(cs + 2 * j);
        r.co[j] = t[0], r.si[j] = t[1], r.co[j + 1] = t[2], r.si[j + 1] = t[3];
    }
    return r;
}

__device__ __forceinline__ Chunk load_unit(const uint16_t *x, const Unit &u)
{
    return {*reinterpret_cast<const u32x4 *>(x + u.c0), *reinterpret_cast<const u32x4 *>(x + u.c1)};
}

// The products are exact in binary64, so each fma rounds once.
__device__ __forceinline__ Chunk turn(const Chunk &x, const Angles &t, bool interleaved)
{
    Chunk r;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        double u[2], v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = 2 * w + i, at = interleaved ? 2 * j : j, bt = interleaved ? 2 * j + 1 : j + 8;
            const double a = half_at(x, at), b = half_at(x, bt);
            u[i] = __builtin_fma(a, t.co[j], -(b * t.si[j]));
            v[i] = __builtin_fma(b, t.co[j], a * t.si[j]);
        }
        if (interleaved) {
            const uint32_t p0 = pack_once(u[0], v[0]), p1 = pack_once(u[1], v[1]);
            if (w < 2) r.lo[2 * w] = p0, r.lo[2 * w + 1] = p1;
            else r.hi[2 * w - 4] = p0, r.hi[2 * w - 3] = p1;
        } else {
            r.lo[w] = pack_once(u[0], u[1]);
            r.hi[w] = pack_once(v[0], v[1]);
        }
    }
    if (t.nan) r.lo = r.hi = u32x4{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
    return r;
}

// A unit of one row of one head.
__device__ __forceinline__ Chunk rotated_unit(const uint16_t *x, int64_t row, int pc, const Unit &u, const Rope &rope)
{
    const Chunk r = load_unit(x, u);
    return u.turned ? turn(r, load_angles(rope, row, pc), rope.interleaved) : r;
}

// The largest magnitude, of two values each in x, joined to `top`.  Magnitudes are
// compared as bit patterns, in whose order NaN stands above infinity: a page with a
// NaN gets NaN for its scale.
using u16x2 = uint16_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ u16x2 join_max(u16x2 top, const u32x4 &x)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __builtin_elementwise_max(top, bitcast<u16x2>(x[i] & 0x7FFF7FFFu));
    return top;
}

// The same over the workgroup, as a value; `red` holds one pattern per wave.
__device__ __forceinline__ float block_max(u16x2 top, uint32_t *red)
{
    uint32_t a = max((uint32_t)top[0], (uint32_t)top[1]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o));
    __syncthreads();                                   // earlier readers of red are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    return half_bits_to_float((uint16_t)max(max(red[0], red[1]), max(red[2], red[3])));
}

// Page `page_no` of sequence s, all of its tokens at hand: the first
// ctx - page_no * T from the ring page, the rest from the call's rows of one head
// (src, `stride` apart).
template <int D, int T>
__device__ void quantize_k_page(const uint16_t *src, int64_t stride, const KvSeq &s, const Rope &rope, int page_no,
                                const uint16_t *ring, int8_t *codes, float *scale_out, uint32_t *red)
{
    constexpr int DC = D / 16, KU = T * DC, KN = (KU + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    const int old = max(s.ctx - page_no * T, 0);               // tokens of the page that the ring holds
    const int64_t row0 = (int64_t)s.q0 + page_no * T - s.ctx;  // row of the page's token 0
    auto place = [](int tok, int c) { return kv_k_index(tok, c >> 4, DC) + (c & 15); };
    Chunk x[KN];
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        // four tokens, whose codes lie side by side, in neighbouring threads
        const int u = tid + i * kThreads, pc = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
        if (u < KU) {
            const Unit unit(rope, pc);
            if (tok < old)
                x[i] = {*reinterpret_cast<const u32x4 *>(ring + place(tok, unit.c0)),
                        *reinterpret_cast<const u32x4 *>(ring + place(tok, unit.c1))};
            else
                x[i] = rotated_unit(src + (row0 + tok) * stride, row0 + tok, pc, unit, rope);
            top = join_max(join_max(top, x[i].lo), x[i].hi);
        }
    }
    const float scale = kv_scale(block_max(top, red), 127.0f), r = __builtin_amdgcn_rcpf(scale);
    if (tid == 0) *scale_out = scale;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int u = tid + i * kThreads, pc = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
        if (u < KU) {
            const Unit unit(rope, pc);
            u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e >> 2] |= kv_code(half_at(x[i], e), scale, r, 127.0f) << (8 * (e & 3));
            *reinterpret_cast<u32x2 *>(codes + place(tok, unit.c0)) = u32x2{w[0], w[1]};
            *reinterpret_cast<u32x2 *>(codes + place(tok, unit.c1)) = u32x2{w[2], w[3]};
        }
    }
}

// 16 tokens' values of four channels, each channel's in the order of tokens; those
// of tokens before `old` come from `x` as it is.
__device__ __forceinline__ void gather_v(Chunk x[4], const uint16_t *src, int64_t stride, int from, int to)
{
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if (j < from || j >= to) continue;
        const u32x2 w = *reinterpret_cast<const u32x2 *>(src + j * stride);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
            uint32_t v = j < 8 ? x[e].lo[j >> 1] : x[e].hi[(j - 8) >> 1];
            v = j & 1 ? (v & 0xFFFFu) | h << 16 : (v & 0xFFFF0000u) | h;
            if (j < 8) x[e].lo[j >> 1] = v;
            else x[e].hi[(j - 8) >> 1] = v;
        }
    }
}

template <int D, int T>
__device__ void quantize_v_page(const uint16_t *src, int64_t stride, const KvSeq &s, int page_no, const uint16_t *ring,
                                int8_t *codes, float *scale_out, uint32_t *red)
{
    constexpr int VU = T / 16 * (D / 4), VN = (VU + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    const int old = max(s.ctx - page_no * T, 0);
    const int64_t row0 = (int64_t)s.q0 + page_no * T - s.ctx;
    // 16 tokens of four channels: x[i][channel] holds the tokens in order
    Chunk x[VN][4];
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * kThreads, ch = u % (D / 4) * 4, t0 = u / (D / 4) * 16;
        if (u >= VU) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[i][e].lo = x[i][e].hi = u32x4{0u, 0u, 0u, 0u};
            if (t0 < old) x[i][e] = load_chunk(ring + kv_v_index(t0, ch + e, D));
        }
        gather_v(x[i], src + (row0 + t0) * stride + ch, stride, old - t0, 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = join_max(join_max(top, x[i][e].lo), x[i][e].hi);
    }
    const float scale = kv_scale(block_max(top, red), 127.0f), r = __builtin_amdgcn_rcpf(scale);
    if (tid == 0) *scale_out = scale;
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * kThreads, ch = u % (D / 4) * 4, t0 = u / (D / 4) * 16;
        if (u >= VU) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j >> 2] |= kv_code(half_at(x[i][e], j), scale, r, 127.0f) << (8 * (j & 3));
            *reinterpret_cast<u32x4 *>(codes + kv_v_index(t0, ch + e, D)) = w;
        }
    }
}

// The new tokens of the sequence's last two pages, into the ring (its half 0 at
// `ring`, half 1 `other` values on).
template <int D, int T>
__device__ void ring_k(const uint16_t *src, int64_t stride, const KvSeq &s, const Rope &rope, uint16_t *ring, int64_t other)
{
    constexpr int DC = D / 16;
    const int first = max(s.ctx, ((s.total() - 1) / T - 1) * T), count = s.total() - first;
    const int64_t row0 = (int64_t)s.q0 + first - s.ctx;
#pragma unroll 2
    for (int u = threadIdx.x; u < count * DC; u += kThreads) {
        const int i = u / DC, pc = u - i * DC, tok = first + i;
        const Unit unit(rope, pc);
        const Chunk x = rotated_unit(src + (row0 + i) * stride, row0 + i, pc, unit, rope);
        uint16_t *to = ring + (tok / T & 1) * other;
        *reinterpret_cast<u32x4 *>(to + kv_k_index(tok & (T - 1), unit.c0 >> 4, DC) + (unit.c0 & 15)) = x.lo;
        *reinterpret_cast<u32x4 *>(to + kv_k_index(tok & (T - 1), unit.c1 >> 4, DC) + (unit.c1 & 15)) = x.hi;
    }
}

// V in groups of 16 tokens and four channels: a whole group's tokens are one store
// for each channel, a part of one is stored value by value.
template <int D, int T>
__device__ void ring_v(const uint16_t *src, int64_t stride, const KvSeq &s, uint16_t *ring, int64_t other)
{
    const int first = max(s.ctx, ((s.total() - 1) / T - 1) * T), g0 = first / 16, groups = (s.total() + 15) / 16 - g0;
    const int64_t row0 = (int64_t)s.q0 - s.ctx;                // row of token 0, were it in the call
    for (int u = threadIdx.x; u < groups * (D / 4); u += kThreads) {
        const int t0 = (g0 + u / (D / 4)) * 16, ch = u % (D / 4) * 4;
        const int from = max(first - t0, 0), to = min(s.total() - t0, 16);
        uint16_t *out = ring + (t0 / T & 1) * other + kv_v_index(t0 & (T - 1), ch, D);
        const uint16_t *in = src + (row0 + t0) * stride + ch;
        if (to - from == 16) {
            Chunk x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e].lo = x[e].hi = u32x4{0u, 0u, 0u, 0u};
            gather_v(x, in, stride, 0, 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) store_chunk(out + e * 16, x[e]);
        } else {
            for (int j = from; j < to; ++j) {
                const u32x2 w = *reinterpret_cast<const u32x2 *>(in + j * stride);
#pragma unroll
                for (int e = 0; e < 4; ++e) out[e * 16 + j] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
}

struct Source {                  // the call's rows
    const uint16_t *k, *v, *q;
    int64_t k_stride, v_stride, q_stride;
    int n_q, q_heads;            // heads of q, and how many of them a thread rotates
};

// Unit pc of a row's heads head, head + step, ...: the angles are read and widened
// once for all of them.
template <int D>
__device__ __forceinline__ void rotate_q(const Source &src, const Rope &rope, int64_t row, int pc, int head, int step,
                                         uint16_t *out)
{
    const Unit unit(rope, pc);
    Angles t = {};
    if (unit.turned) t = load_angles(rope, row, pc);
    const uint16_t *from = src.q + row * src.q_stride;
    uint16_t *to = out + row * src.n_q * D;
    for (int h = head; h < src.n_q; h += step) {
        Chunk x = load_unit(from + h * D, unit);
        if (unit.turned) x = turn(x, t, rope.interleaved);
        *reinterpret_cast<u32x4 *>(to + h * D + unit.c0) = x.lo;
        *reinterpret_cast<u32x4 *>(to + h * D + unit.c1) = x.hi;
    }
}

template <int D, int T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(kv_paged_cache cache, kv_paged_batch batch, Source src,
                                                             Rope rope, uint16_t *__restrict__ q_out, int edge_groups,
                                                             int page_groups, int mix)
{
    constexpr int PC = D / 16, SHIFT = T == 64 ? 6 : T == 128 ? 7 : 8;
    constexpr int PAGE = D * T;
    __shared__ uint32_t red[4];
    const int n_kv = cache.n_kv;
    int g = blockIdx.x - edge_groups;                          // behind the edges, pages and q mixed: every
    int page_item = -1;                                        // `mix`-th workgroup is a page's while there are any
    if (g >= 0) {
        if (g % mix == 0 && g / mix < page_groups) page_item = g / mix;
        else g -= min(page_groups, g / mix + 1);
    }
    if (g >= 0 && page_item < 0) {
        const int64_t u = (int64_t)g * kThreads + threadIdx.x;
        const int step = (src.n_q + src.q_heads - 1) / src.q_heads;            // threads that share a row's pairs
        const int64_t row = u / (PC * step);
        if (row >= batch.tokens) return;
        const int i = (int)(u - row * (PC * step));
        rotate_q<D>(src, rope, row, i % PC, i / PC, step, q_out);
        return;
    }

    const bool edge = page_item < 0;
    g = edge ? blockIdx.x : page_item;
    const bool of_v = g & 1;
    const int h = g / 2 % n_kv;
    int b = g / 2 / n_kv, page_no = 0;
    if (!edge) {                                               // the page of new tokens with this number
        int64_t off;
        const int64_t item = b;
        if (!kv_locate(batch.batch, item, [&](int i) {
                const KvSeq t = kv_seq(batch, i, cache.slots, SHIFT);
                return t.n ? max((t.total() >> SHIFT) - (t.ctx >> SHIFT) - 1, 0) : 0;
            }, b, off))
            return;
        page_no = (int)off;
    }
    const KvSeq s = kv_seq(batch, b, cache.slots, SHIFT);
    if (s.n == 0) return;
    page_no += (s.ctx >> SHIFT) + (edge ? 0 : 1);
    const uint16_t *from = (of_v ? src.v : src.k) + h * D;
    const int64_t stride = of_v ? src.v_stride : src.k_stride, other = (int64_t)n_kv * PAGE;
    uint16_t *ring = (of_v ? cache.v_tail : cache.k_tail) + ((int64_t)s.slot * 2 * n_kv + h) * PAGE;

    auto keep_new = [&]() {
        if (of_v) ring_v<D, T>(from, stride, s, ring, other);
        else ring_k<D, T>(from, stride, s, rope, ring, other);
    };
    // With a last page no further than the next, the writes leave the old tokens alone
    // and go first: nothing waits for them.
    const bool apart = (s.total() - 1) >> SHIFT <= page_no + 1;
    if (edge && apart) keep_new();
    if (page_no < s.total() >> SHIFT) {
        const int64_t id = batch.block_table[(int64_t)b * batch.table_cols + page_no];
        if (id >= 0 && id < cache.pages) {
            const int64_t at = id * n_kv + h;
            const uint16_t *old = ring + (page_no & 1) * other;
            if (of_v)
                quantize_v_page<D, T>(from, stride, s, page_no, old, cache.v + at * PAGE, cache.v_scale + at, red);
            else
                quantize_k_page<D, T>(from, stride, s, rope, page_no, old, cache.k + at * PAGE, cache.k_scale + at, red);
        }
    }
    if (!edge || apart) return;
    __syncthreads();                                           // the ring's old page has been read
    keep_new();
}

// K or V of one page of one head in the order of tokens: three bytes moved a value, no
// arithmetic to speak of (2 pages of 32 heads 4 us, all of it latency).
template <int D, int T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(kv_paged_cache cache, const int32_t *__restrict__ ids,
                                                           uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out)
{
    constexpr int DC = D / 16, PAGE = D * T;
    const int h = blockIdx.x / 2 % cache.n_kv;
    const int64_t i = blockIdx.x / 2 / cache.n_kv, id = ids[i];
    if (id < 0 || id >= cache.pages) return;
    const int64_t at = id * cache.n_kv + h, to = (i * cache.n_kv + h) * PAGE;
    auto value = [](const u32x4 &w, int e, float s) {
        return bitcast<uint16_t>((_Float16)((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))) * s));
    };
    if (blockIdx.x & 1) {
        const float s = cache.v_scale[at];
        const int8_t *codes = cache.v + at * PAGE;
        for (int u = threadIdx.x; u < T / 16 * (D / 4); u += kThreads) {
            const int ch = u % (D / 4) * 4, t0 = u / (D / 4) * 16;
            u32x4 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const u32x4 *>(codes + kv_v_index(t0, ch + e, D));
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const u32x2 r = {value(w[0], j, s) | (uint32_t)value(w[1], j, s) << 16,
                                 value(w[2], j, s) | (uint32_t)value(w[3], j, s) << 16};
                *reinterpret_cast<u32x2 *>(v_out + to + (t0 + j) * D + ch) = r;
            }
        }
        return;
    }
    const float s = cache.k_scale[at];
    const int8_t *codes = cache.k + at * PAGE;
#pragma unroll 4
    for (int u = threadIdx.x; u < T * DC; u += kThreads) {
        const int c = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
        const u32x4 w = *reinterpret_cast<const u32x4 *>(codes + kv_k_index(tok, c, DC));
        Chunk r;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            r.lo[e >> 1] = value(w, e, s) | (uint32_t)value(w, e + 1, s) << 16;
            r.hi[e >> 1] = value(w, e + 8, s) | (uint32_t)value(w, e + 9, s) << 16;
        }
        store_chunk(k_out + to + tok * D + c * 16, r);
    }
}

// Calls fn with the head dimension and page size as compile-time values.
template <typename F>
hipError_t by_size(int d, int page, F fn)
{
    auto with_d = [&](auto D) {
        switch (page) {
        case 64: return fn(D, std::integral_constant<int, 64>{});
        case 128: return fn(D, std::integral_constant<int, 128>{});
        case 256: return fn(D, std::integral_constant<int, 256>{});
        default: return hipErrorInvalidValue;
        }
    };
    switch (d) {
    case 64: return with_d(std::integral_constant<int, 64>{});
    case 96: return with_d(std::integral_constant<int, 96>{});
    case 128: return with_d(std::integral_constant<int, 128>{});
    case 256: return with_d(std::integral_constant<int, 256>{});
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t kv_launch_append(const kv_paged_cache &cache, const kv_paged_batch &batch, const uint16_t *k,
                            int64_t k_stride, const uint16_t *v, int64_t v_stride, const uint16_t *q, int64_t q_stride,
                            int n_q, const float *rope, int64_t rope_rows, int rope_dim, bool interleaved,
                            const int32_t *positions, uint16_t *q_out, hipStream_t stream)
{
    const Rope r = {rope, positions, rope_rows, rope ? rope_dim : 0, interleaved};
    // four heads a thread, which share the angles, once that leaves half of the card's
    // threads (2048 on each CU) to run: 64 heads, 15000 tokens 153 us, 198 with one head a
    // thread; 2048 tokens 29.6 and 33.7; 1024 tokens 27.8 and 27.3
    const int64_t threads = q ? batch.tokens * n_q * (cache.d / 16) : 0;
    const int per = threads >= int64_t(2) * 2048 * 256 ? 4 : 1;
    const Source src = {k, v, q, k_stride, v_stride, q_stride, n_q, per};
    const int edge = batch.batch * cache.n_kv * 2, pages = (int)(batch.tokens / cache.page) * cache.n_kv * 2;
    const int64_t rows = q ? (batch.tokens * ((n_q + per - 1) / per) * (cache.d / 16) + kThreads - 1) / kThreads : 0;
    // pages are bound by their arithmetic, q by memory: one in `mix` workgroups a page's
    // (3 prompts of 5000 tokens, read back: 102.6 us, 104.1 with the pages first)
    const int mix = pages > 0 ? (int)((pages + rows) / pages) : 1;
    return by_size(cache.d, cache.page, [&](auto D, auto T) {
        kv_append_kernel<D.value, T.value><<<(unsigned)(edge + pages + rows), kThreads, 0, stream>>>(
            cache, batch, src, r, q_out, edge, pages, mix);
        return hipGetLastError();
    });
}

hipError_t kv_launch_read(const kv_paged_cache &cache, const int32_t *ids, int64_t n, uint16_t *k_out, uint16_t *v_out,
                          hipStream_t stream)
{
    return by_size(cache.d, cache.page, [&](auto D, auto T) {
        kv_read_kernel<D.value, T.value><<<(unsigned)(n * cache.n_kv * 2), kThreads, 0, stream>>>(cache, ids, k_out, v_out);
        return hipGetLastError();
    });
}
