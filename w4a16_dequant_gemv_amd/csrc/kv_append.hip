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
// each, and q is a grid of its own behind them, all in one launch.
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

// Channels 16c .. 16c + 15 of one head's row, rotated to `row`'s position.
__device__ __forceinline__ Chunk rotated_chunk(const uint16_t *x, int c, int64_t row, const Rope &rope)
{
    const Chunk own = load_chunk(x + c * 16);
    if (!rope.table || c * 16 >= rope.dim) return own;
    const int64_t pos = rope.positions[row];
    if (pos < 0 || pos >= rope.rows) {
        const u32x4 nan = {0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
        return {nan, nan};
    }
    const int half = rope.dim / 2;
    const float *cs = rope.table + pos * rope.dim;
    Chunk r;
    if (rope.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const double co = cs[(c * 8 + j) * 2], si = cs[(c * 8 + j) * 2 + 1];
            const double a = half_at(own, 2 * j), b = half_at(own, 2 * j + 1);
            const uint32_t w = pack_once(__builtin_fma(a, co, -(b * si)), __builtin_fma(b, co, a * si));
            if (j < 4) r.lo[j] = w; else r.hi[j - 4] = w;
        }
        return r;
    }
    const bool first = c * 16 < half;
    const Chunk other = load_chunk(x + (first ? c * 16 + half : c * 16 - half));
    cs += (first ? c * 16 : c * 16 - half) * 2;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const f32x4 t = *reinterpret_cast<const f32x4 *>(cs + 4 * j);      // two pairs' cosine and sine
        double v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const double co = t[2 * i], si = t[2 * i + 1];
            const double a = half_at(own, 2 * j + i), b = half_at(other, 2 * j + i);
            v[i] = __builtin_fma(a, co, first ? -(b * si) : b * si);        // the product is exact
        }
        const uint32_t w = pack_once(v[0], v[1]);
        if (j < 4) r.lo[j] = w; else r.hi[j - 4] = w;
    }
    return r;
}

// Largest of a value over the workgroup; `red` holds one float per wave.
__device__ __forceinline__ float block_max(float a, float *red)
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) a = fmaxf(a, __shfl_xor(a, o));
    __syncthreads();                                   // earlier readers of red are done
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = a;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// Page `page_no` of sequence s, all of its tokens at hand: the first
// ctx - page_no * T from the ring page, the rest from the call's rows of one head
// (src, `stride` apart).
template <int D, int T>
__device__ void quantize_k_page(const uint16_t *src, int64_t stride, const KvSeq &s, const Rope &rope, int page_no,
                                const uint16_t *ring, int8_t *codes, float *scale_out, float *red)
{
    constexpr int DC = D / 16, KU = T * DC, KN = (KU + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    const int old = max(s.ctx - page_no * T, 0);               // tokens of the page that the ring holds
    const int64_t row0 = (int64_t)s.q0 + page_no * T - s.ctx;  // row of the page's token 0
    Chunk x[KN];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int u = tid + i * kThreads, c = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
        if (u < KU) {
            x[i] = tok < old ? load_chunk(ring + kv_k_index(tok, c, DC))
                             : rotated_chunk(src + (row0 + tok) * stride, c, row0 + tok, rope);
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(half_at(x[i], e)));
        }
    }
    const float scale = kv_scale(block_max(amax, red), 127.0f), r = __builtin_amdgcn_rcpf(scale);
    if (tid == 0) *scale_out = scale;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int u = tid + i * kThreads, c = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
        if (u < KU) {
            u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e >> 2] |= kv_code(half_at(x[i], e), scale, r, 127.0f) << (8 * (e & 3));
            *reinterpret_cast<u32x4 *>(codes + kv_k_index(tok, c, DC)) = w;
        }
    }
}

template <int D, int T>
__device__ void quantize_v_page(const uint16_t *src, int64_t stride, const KvSeq &s, int page_no, const uint16_t *ring,
                                int8_t *codes, float *scale_out, float *red)
{
    constexpr int VU = T / 16 * (D / 4), VN = (VU + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    const int old = max(s.ctx - page_no * T, 0);
    const int64_t row0 = (int64_t)s.q0 + page_no * T - s.ctx;
    // 16 tokens of four channels: x[i][channel] holds the tokens in order
    Chunk x[VN][4];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * kThreads, ch = u % (D / 4) * 4, t0 = u / (D / 4) * 16;
        if (u >= VU) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[i][e].lo = x[i][e].hi = u32x4{0u, 0u, 0u, 0u};
            if (t0 < old) x[i][e] = load_chunk(ring + kv_v_index(t0, ch + e, D));
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if (t0 + j < old) continue;
            const u32x2 w = *reinterpret_cast<const u32x2 *>(src + (row0 + t0 + j) * stride + ch);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t h = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                uint32_t &to = j < 8 ? reinterpret_cast<uint32_t *>(&x[i][e].lo)[j >> 1]
                                     : reinterpret_cast<uint32_t *>(&x[i][e].hi)[(j - 8) >> 1];
                to = j & 1 ? (to & 0xFFFFu) | h << 16 : (to & 0xFFFF0000u) | h;
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(half_at(x[i][e], j)));
    }
    const float scale = kv_scale(block_max(amax, red), 127.0f), r = __builtin_amdgcn_rcpf(scale);
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
    for (int u = threadIdx.x; u < count * DC; u += kThreads) {
        const int i = u / DC, c = u - i * DC, tok = first + i;
        store_chunk(ring + (tok / T & 1) * other + kv_k_index(tok & (T - 1), c, DC),
                    rotated_chunk(src + (row0 + i) * stride, c, row0 + i, rope));
    }
}

template <int D, int T>
__device__ void ring_v(const uint16_t *src, int64_t stride, const KvSeq &s, uint16_t *ring, int64_t other)
{
    constexpr int DC = D / 16;
    const int first = max(s.ctx, ((s.total() - 1) / T - 1) * T), count = s.total() - first;
    const int64_t row0 = (int64_t)s.q0 + first - s.ctx;
    for (int u = threadIdx.x; u < count * DC; u += kThreads) {
        const int i = u / DC, c = u - i * DC, tok = first + i;
        const Chunk x = load_chunk(src + (row0 + i) * stride + c * 16);
        uint16_t *to = ring + (tok / T & 1) * other + kv_v_index(tok & (T - 1), c * 16, D);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t w = e < 8 ? x.lo[e >> 1] : x.hi[(e - 8) >> 1];
            to[e * 16] = (uint16_t)(w >> (16 * (e & 1)));
        }
    }
}

struct Source {                  // the call's rows
    const uint16_t *k, *v, *q;
    int64_t k_stride, v_stride, q_stride;
    int n_q, q_heads;            // heads of q, and how many of them a thread rotates
};

// Pairs 8 pc .. 8 pc + 7 of a row's heads head, head + step, ...: the angles are
// read and widened once for all of them.
template <int D>
__device__ __forceinline__ void rotate_q(const Source &src, const Rope &rope, int64_t row, int pc, int head, int step,
                                         uint16_t *out)
{
    // the two chunks of 8 channels: the pairs' first and second halves, or one after the other
    const int half = rope.dim / 2;
    const bool turned = pc * 8 < half;
    int c0, c1;
    if (!turned) c0 = rope.dim + (pc * 8 - half) * 2, c1 = c0 + 8;             // channels that are only copied
    else if (rope.interleaved) c0 = pc * 16, c1 = c0 + 8;
    else c0 = pc * 8, c1 = c0 + half;
    double co[8], si[8];
    bool nan = false;
    if (turned) {
        const int64_t pos = rope.positions[row];
        nan = pos < 0 || pos >= rope.rows;
        const float *cs = rope.table + (nan ? 0 : pos) * rope.dim + pc * 16;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const f32x4 t = *reinterpret_cast<const f32x4 *>(cs + 2 * j);
            co[j] = t[0], si[j] = t[1], co[j + 1] = t[2], si[j + 1] = t[3];
        }
    }
    const uint16_t *from = src.q + row * src.q_stride;
    uint16_t *to = out + row * src.n_q * D;
    for (int h = head; h < src.n_q; h += step) {
        Chunk x = {*reinterpret_cast<const u32x4 *>(from + h * D + c0), *reinterpret_cast<const u32x4 *>(from + h * D + c1)};
        if (turned) {
            Chunk r;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                double u[2], v[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // interleaved: pairs lie in neighbouring channels, four of them in each chunk
                    const int j = 2 * w + i, at = rope.interleaved ? 2 * j : j, bt = rope.interleaved ? 2 * j + 1 : j + 8;
                    const double a = half_at(x, at), b = half_at(x, bt);
                    u[i] = __builtin_fma(a, co[j], -(b * si[j]));                // the products are exact
                    v[i] = __builtin_fma(b, co[j], a * si[j]);
                }
                if (rope.interleaved) {
                    const uint32_t p0 = pack_once(u[0], v[0]), p1 = pack_once(u[1], v[1]);
                    if (w < 2) r.lo[2 * w] = p0, r.lo[2 * w + 1] = p1;
                    else r.hi[2 * w - 4] = p0, r.hi[2 * w - 3] = p1;
                } else {
                    r.lo[w] = pack_once(u[0], u[1]);
                    r.hi[w] = pack_once(v[0], v[1]);
                }
            }
            x = r;
            if (nan) x.lo = x.hi = u32x4{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
        }
        *reinterpret_cast<u32x4 *>(to + h * D + c0) = x.lo;
        *reinterpret_cast<u32x4 *>(to + h * D + c1) = x.hi;
    }
}

template <int D, int T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(kv_paged_cache cache, kv_paged_batch batch, Source src,
                                                             Rope rope, uint16_t *__restrict__ q_out, int edge_groups,
                                                             int page_groups)
{
    constexpr int PC = D / 16, SHIFT = T == 64 ? 6 : T == 128 ? 7 : 8;
    constexpr int PAGE = D * T;
    __shared__ float red[4];
    const int n_kv = cache.n_kv;
    int g = blockIdx.x;

    if (g >= edge_groups + page_groups) {
        const int64_t u = (int64_t)(g - edge_groups - page_groups) * kThreads + threadIdx.x;
        const int step = (src.n_q + src.q_heads - 1) / src.q_heads;            // threads that share a row's pairs
        const int64_t row = u / (PC * step);
        if (row >= batch.tokens) return;
        const int i = (int)(u - row * (PC * step));
        rotate_q<D>(src, rope, row, i % PC, i / PC, step, q_out);
        return;
    }

    const bool edge = g < edge_groups;
    if (!edge) g -= edge_groups;
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

// One page of one head in the order of tokens.
template <int D, int T>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(kv_paged_cache cache, const int32_t *__restrict__ ids,
                                                           uint16_t *__restrict__ k_out, uint16_t *__restrict__ v_out)
{
    constexpr int DC = D / 16, PAGE = D * T;
    const int h = blockIdx.x % cache.n_kv;
    const int64_t i = blockIdx.x / cache.n_kv, id = ids[i];
    if (id < 0 || id >= cache.pages) return;
    const int64_t at = id * cache.n_kv + h, to = (i * cache.n_kv + h) * PAGE;
    const float ks = cache.k_scale[at], vs = cache.v_scale[at];
    const int8_t *kp = cache.k + at * PAGE, *vp = cache.v + at * PAGE;
    auto value = [](const u32x4 &w, int e, float s) {
        return bitcast<uint16_t>((_Float16)((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))) * s));
    };
    for (int u = threadIdx.x; u < T * DC; u += kThreads) {
        const int c = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
        const u32x4 w = *reinterpret_cast<const u32x4 *>(kp + kv_k_index(tok, c, DC));
        Chunk r;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            r.lo[e >> 1] = value(w, e, ks) | (uint32_t)value(w, e + 1, ks) << 16;
            r.hi[e >> 1] = value(w, e + 8, ks) | (uint32_t)value(w, e + 9, ks) << 16;
        }
        store_chunk(k_out + to + tok * D + c * 16, r);
    }
    for (int u = threadIdx.x; u < T / 16 * (D / 4); u += kThreads) {
        const int ch = u % (D / 4) * 4, t0 = u / (D / 4) * 16;
        u32x4 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = *reinterpret_cast<const u32x4 *>(vp + kv_v_index(t0, ch + e, D));
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const u32x2 r = {value(w[0], j, vs) | (uint32_t)value(w[1], j, vs) << 16,
                             value(w[2], j, vs) | (uint32_t)value(w[3], j, vs) << 16};
            *reinterpret_cast<u32x2 *>(v_out + to + (t0 + j) * D + ch) = r;
        }
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
    // four heads a thread once that still fills the card (2048 threads on each CU)
    const int64_t threads = q ? batch.tokens * n_q * (cache.d / 16) : 0;
    const int per = threads >= int64_t(4) * 2048 * 256 ? 4 : 1;
    const Source src = {k, v, q, k_stride, v_stride, q_stride, n_q, per};
    const int edge = batch.batch * cache.n_kv * 2, pages = (int)(batch.tokens / cache.page) * cache.n_kv * 2;
    const int64_t rows = q ? (batch.tokens * ((n_q + per - 1) / per) * (cache.d / 16) + kThreads - 1) / kThreads : 0;
    return by_size(cache.d, cache.page, [&](auto D, auto T) {
        kv_append_kernel<D.value, T.value><<<(unsigned)(edge + pages + rows), kThreads, 0, stream>>>(
            cache, batch, src, r, q_out, edge, pages);
        return hipGetLastError();
    });
}

hipError_t kv_launch_read(const kv_paged_cache &cache, const int32_t *ids, int64_t n, uint16_t *k_out, uint16_t *v_out,
                          hipStream_t stream)
{
    return by_size(cache.d, cache.page, [&](auto D, auto T) {
        kv_read_kernel<D.value, T.value><<<(unsigned)(n * cache.n_kv), kThreads, 0, stream>>>(cache, ids, k_out, v_out);
        return hipGetLastError();
    });
}
