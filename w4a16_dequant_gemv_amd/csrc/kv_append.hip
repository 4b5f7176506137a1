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
// Work split.  Per sequence and kv head one workgroup finishes the page that
// ctx_lens ends in (old tokens from the ring, new ones from the call) and then
// writes the ring: the reads of the finished page come before the writes that
// may replace it, in one workgroup, so no order between workgroups is needed.
// Pages made of new tokens only are one workgroup each, and q is a grid of its
// own behind them, all in one launch.
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
            const uint32_t w = pack_once(a * co - b * si, b * co + a * si);
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
            v[i] = first ? a * co - b * si : a * co + b * si;
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

struct Source {                  // the call's new tokens of one kv head
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;
};

// Page `page_no` of sequence s, all of its tokens at hand: the first
// ctx - page_no * T from the ring page kt / vt, the rest from the call.
template <int D, int T>
__device__ void quantize_page(const Source &src, const KvSeq &s, const Rope &rope, int page_no, const uint16_t *kt,
                              const uint16_t *vt, int8_t *kp, int8_t *vp, float *ks, float *vs, float *red)
{
    constexpr int DC = D / 16;
    constexpr int KU = T * DC, KN = (KU + kThreads - 1) / kThreads;
    constexpr int VU = T / 16 * (D / 4), VN = (VU + kThreads - 1) / kThreads;
    const int tid = threadIdx.x;
    const int old = max(s.ctx - page_no * T, 0);               // tokens of the page that the ring holds
    const int64_t row0 = (int64_t)s.q0 + page_no * T - s.ctx;  // row of the page's token 0
    {
        Chunk x[KN];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int u = tid + i * kThreads, c = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
            if (u < KU) {
                x[i] = tok < old ? load_chunk(kt + kv_k_index(tok, c, DC))
                                 : rotated_chunk(src.k + (row0 + tok) * src.k_stride, c, row0 + tok, rope);
#pragma unroll
                for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(half_at(x[i], e)));
            }
        }
        const float scale = kv_scale(block_max(amax, red), 127.0f), r = __builtin_amdgcn_rcpf(scale);
        if (tid == 0) *ks = scale;
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int u = tid + i * kThreads, c = (u >> 2) % DC, tok = (u >> 2) / DC * 4 + (u & 3);
            if (u < KU) {
                u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e >> 2] |= kv_code(half_at(x[i], e), scale, r, 127.0f) << (8 * (e & 3));
                *reinterpret_cast<u32x4 *>(kp + kv_k_index(tok, c, DC)) = w;
            }
        }
    }
    {
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
                if (t0 < old) x[i][e] = load_chunk(vt + kv_v_index(t0, ch + e, D));
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (t0 + j < old) continue;
                const u32x2 w = *reinterpret_cast<const u32x2 *>(src.v + (row0 + t0 + j) * src.v_stride + ch);
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
        if (tid == 0) *vs = scale;
#pragma unroll
        for (int i = 0; i < VN; ++i) {
            const int u = tid + i * kThreads, ch = u % (D / 4) * 4, t0 = u / (D / 4) * 16;
            if (u >= VU) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u32x4 w = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j >> 2] |= kv_code(half_at(x[i][e], j), scale, r, 127.0f) << (8 * (j & 3));
                *reinterpret_cast<u32x4 *>(vp + kv_v_index(t0, ch + e, D)) = w;
            }
        }
    }
}

template <int D, int T>
__global__ __launch_bounds__(kThreads) void kv_append_kernel(kv_paged_cache cache, kv_paged_batch batch, Source src,
                                                             const uint16_t *__restrict__ q, int64_t q_stride, int n_q,
                                                             Rope rope, uint16_t *__restrict__ q_out, int edge_groups,
                                                             int page_groups)
{
    constexpr int DC = D / 16, SHIFT = T == 64 ? 6 : T == 128 ? 7 : 8;
    constexpr int PAGE = D * T;
    __shared__ float red[4];
    const int n_kv = cache.n_kv;
    int g = blockIdx.x;

    if (g >= edge_groups + page_groups) {                      // rotation of q: 16 channels a thread
        const int64_t u = (int64_t)(g - edge_groups - page_groups) * kThreads + threadIdx.x;
        const int64_t per_row = (int64_t)n_q * DC, row = u / per_row;
        if (row >= batch.tokens) return;
        const int i = (int)(u - row * per_row), head = i / DC, c = i - head * DC;
        store_chunk(q_out + (row * n_q + head) * D + c * 16,
                    rotated_chunk(q + row * q_stride + head * D, c, row, rope));
        return;
    }

    const bool edge = g < edge_groups;
    if (!edge) g -= edge_groups;
    const int h = g % n_kv;
    int b = g / n_kv, page_no = 0;
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
    src.k += h * D;
    src.v += h * D;
    const int64_t ring = ((int64_t)s.slot * 2 * n_kv + h) * PAGE;          // its half 0; half 1 is n_kv pages on

    if (page_no < s.total() >> SHIFT) {
        const int64_t id = batch.block_table[(int64_t)b * batch.table_cols + page_no];
        if (id >= 0 && id < cache.pages) {
            const int64_t at = id * n_kv + h, r = ring + (int64_t)(page_no & 1) * n_kv * PAGE;
            quantize_page<D, T>(src, s, rope, page_no, cache.k_tail + r, cache.v_tail + r, cache.k + at * PAGE,
                                cache.v + at * PAGE, cache.k_scale + at, cache.v_scale + at, red);
        }
    }
    if (!edge) return;
    __syncthreads();                                           // the ring's old page has been read

    // The new tokens of the sequence's last two pages go into the ring.
    const int first = max(s.ctx, (((s.total() - 1) >> SHIFT) - 1) * T), count = s.total() - first;
    const int64_t row0 = (int64_t)s.q0 + first - s.ctx;
    for (int u = threadIdx.x; u < count * DC; u += kThreads) {
        const int i = u / DC, c = u - i * DC, tok = first + i;
        const int64_t at = ring + (int64_t)(tok >> SHIFT & 1) * n_kv * PAGE;
        store_chunk(cache.k_tail + at + kv_k_index(tok & (T - 1), c, DC),
                    rotated_chunk(src.k + (row0 + i) * src.k_stride, c, row0 + i, rope));
        const Chunk x = load_chunk(src.v + (row0 + i) * src.v_stride + c * 16);
        uint16_t *to = cache.v_tail + at + kv_v_index(tok & (T - 1), c * 16, D);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t w = e < 8 ? x.lo[e >> 1] : x.hi[(e - 8) >> 1];
            to[e * 16] = (uint16_t)(w >> (16 * (e & 1)));
        }
    }
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
    const Rope r = {rope, positions, rope_rows, rope_dim, interleaved};
    const Source src = {k, v, k_stride, v_stride};
    const int edge = batch.batch * cache.n_kv, pages = (int)(batch.tokens / cache.page) * cache.n_kv;
    const int64_t rows = q ? (batch.tokens * n_q * (cache.d / 16) + kThreads - 1) / kThreads : 0;
    return by_size(cache.d, cache.page, [&](auto D, auto T) {
        kv_append_kernel<D.value, T.value><<<(unsigned)(edge + pages + rows), kThreads, 0, stream>>>(
            cache, batch, src, q, q_stride, n_q, r, q_out, edge, pages);
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
