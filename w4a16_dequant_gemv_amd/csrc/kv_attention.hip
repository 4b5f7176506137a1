// kv_attention.hip -- attention over the paged INT8 cache (kv_codec.h).
#include "kv_device.h"
#include "q4_launch.h"

namespace {

constexpr int kThreads = 256;

// One workgroup per (row, query head): tiles of 64 tokens, one pass with the
// running maximum and sum.
__global__ __launch_bounds__(kThreads) void kv_attend_simple_kernel(kv_paged_cache cache, kv_paged_batch batch,
                                                                    const uint16_t *__restrict__ q, int64_t q_stride,
                                                                    int n_q, float scale, int window, int sinks,
                                                                    int page_shift, uint16_t *__restrict__ out)
{
    __shared__ float qs[256], p[64];
    const int d = cache.d, tid = threadIdx.x, page = 1 << page_shift, dc = d / 16;
    const int row = blockIdx.x / n_q, hq = blockIdx.x % n_q, h = hq / (n_q / cache.n_kv);
    int b;
    int64_t off;
    // the last sequence that starts at or before the row and holds it
    bool found = false;
    KvSeq s;
    for (b = 0; b < batch.batch; ++b) {
        s = kv_seq(batch, b, cache.slots, page_shift);
        if (row >= s.q0 && row < s.q0 + s.n) { found = true; break; }
    }
    (void)off;
    if (!found) return;
    const int at = s.ctx + row - s.q0, total = s.total(), full = total >> page_shift << page_shift;
    if (tid < d) qs[tid] = half_bits_to_float(q[row * q_stride + hq * d + tid]);
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int t0 = 0; t0 <= at; t0 += 64) {
        const int page_no = t0 >> page_shift;
        const bool ring = t0 >= full;
        int64_t id = 0;
        if (!ring) {
            id = batch.block_table[(int64_t)b * batch.table_cols + page_no];
            if (id < 0 || id >= cache.pages) continue;
        }
        const int64_t pg = ring ? ((int64_t)s.slot * 2 + (page_no & 1)) * cache.n_kv + h : id * cache.n_kv + h;
        const float ks = ring ? 1.0f : cache.k_scale[pg], vs = ring ? 1.0f : cache.v_scale[pg];
        const int64_t base = pg * page * d;
        __syncthreads();
        if (tid < 64) {
            const int j = t0 + tid, jp = j & (page - 1);
            float x = -INFINITY;
            if (j <= at && (window == 0 || at - j < window || j < sinks)) {
                x = 0.0f;
                for (int c = 0; c < d; ++c) {
                    const int64_t i = base + kv_k_index(jp, c >> 4, dc) + (c & 15);
                    x += qs[c] * (ring ? half_bits_to_float(cache.k_tail[i]) : (float)cache.k[i]);
                }
                x *= scale * ks;
            }
            p[tid] = x;
        }
        __syncthreads();
        float mt = m;
        for (int j = 0; j < 64; ++j) mt = fmaxf(mt, p[j]);
        if (mt == -INFINITY) continue;
        const float f = __expf(m - mt);
        m = mt;
        l *= f;
        o *= f;
        for (int j = 0; j < 64; ++j) {
            if (p[j] == -INFINITY) continue;
            const float w = __expf(p[j] - m);
            l += w;
            if (tid < d) {
                const int64_t i = base + kv_v_index((t0 + j) & (page - 1), tid, d);
                o += w * vs * (ring ? half_bits_to_float(cache.v_tail[i]) : (float)cache.v[i]);
            }
        }
    }
    if (tid < d) out[((int64_t)row * n_q + hq) * d + tid] = bitcast<uint16_t>((_Float16)(l > 0.0f ? o / l : 0.0f));
}

}  // namespace

int64_t kv_attention_workspace(int64_t tokens, int batch, int n_q, int n_kv, int d) { return 256; }

hipError_t kv_launch_attention(const kv_paged_cache &cache, const kv_paged_batch &batch, const uint16_t *q,
                               int64_t q_stride, int n_q, float scale, int window, int sinks, void *workspace,
                               uint16_t *out, hipStream_t stream)
{
    kv_attend_simple_kernel<<<(unsigned)(batch.tokens * n_q), kThreads, 0, stream>>>(
        cache, batch, q, q_stride, n_q, scale, window, sinks, __builtin_ctz(cache.page), out);
    return hipGetLastError();
}
