/*
 * kv_codec.h -- C ABI of the KV-cache codec in the same library (libw4a16.so):
 * symmetric INT8 / INT4 quantization of attention keys per channel and of
 * values per token, their dequantization, and the flush of FP16 window blocks
 * into a pool of quantized blocks; and of the paged INT8 cache (kv_paged_*):
 * rotating and appending new tokens, and attention over what it holds.
 *
 * Sources (cited by page title and section):
 *   [Guide] "27届大模型面试准备十九 模型量化全攻略 -- INT8/INT4、GPTQ、AWQ、
 *           SmoothQuant 与 KV Cache 量化" (dksg.cn), §6 KV Cache 量化:
 *           K quantized per channel (its outliers sit in fixed channels), V per
 *           token; the most recent tokens (about 128) kept in FP16; the
 *           per-token listing: qmax = 2^(b-1) - 1, scale = max|v| / qmax
 *           floored at 1e-8, q = clamp(round(v / scale), -qmax - 1, qmax) as
 *           int8.
 *   [Intro] "大模型量化技术入门：为什么我们需要量化？" (devpress.csdn.net),
 *           §3.2: separate scale factors for K and V.
 *
 * Conventions (shared with w4a16.h: status codes, streams, ownership)
 * -------------------------------------------------------------------
 *  - Pointers are caller-owned device pointers; the library never allocates,
 *    frees or synchronizes; work is enqueued on `stream` (a hipStream_t).
 *  - Cached values are fp16 bit patterns; codes are int8 (two's complement)
 *    for both widths; scales are fp32.
 *  - Every step is one IEEE binary32 operation with round-to-nearest-even on
 *    the exactly widened fp16 inputs (correctly rounded division), so codes
 *    and scales are bit-exact and independent of the launch configuration.
 *    Dequantized values are fp16(q * scale), the binary32 product rounded
 *    once more to fp16.
 *  - Head dimension d: a multiple of 8 in [8, 512].  bits: 4 or 8 (INT4
 *    codes lie in [-8, 7], one per byte).  Per-channel blocks hold t tokens
 *    with 1 <= t <= 32 * (2048 / d) (t <= 512 at d = 128).
 *  - Alignment: fp16 and int8 arrays 16 bytes; scale arrays 4 bytes (16 for
 *    kv_dequant_channels).  Violations return Q4_ERR_ALIGN; bad sizes or bits
 *    Q4_ERR_SHAPE; NULL pointers Q4_ERR_NULL; all before any HIP call.
 *  - Inputs containing NaN or Inf give unspecified (memory-safe) results.
 */
#ifndef KV_CODEC_H
#define KV_CODEC_H

#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Per-token quantization (the V side): x fp16 [rows][d] -> q int8 [rows][d],
 * scale fp32 [rows], one symmetric scale per row over its d values
 * ([Guide] §6, quant_kv_per_token).  A [B][H][S][D] cache is rows = B*H*S.
 */
int kv_quant_tokens(const uint16_t *x, int64_t rows, int32_t d, int32_t bits,
                    int8_t *q, float *scale, void *stream);

/*
 * Per-channel quantization (the K side): x fp16 [blocks][t][d] -> q int8
 * [blocks][t][d], scale fp32 [blocks][d]; channel j of a block gets one
 * symmetric scale over the block's t tokens ([Guide] §6: K per channel).  A
 * block is t consecutive tokens of one head, e.g. the 128 tokens that leave
 * the FP16 window together.
 */
int kv_quant_channels(const uint16_t *x, int64_t blocks, int32_t t, int32_t d,
                      int32_t bits, int8_t *q, float *scale, void *stream);

/* out fp16 [rows][d] = fp16(q * scale[row]). */
int kv_dequant_tokens(const int8_t *q, const float *scale, int64_t rows, int32_t d,
                      uint16_t *out, void *stream);

/* out fp16 [blocks][t][d] = fp16(q * scale[block][channel]). */
int kv_dequant_channels(const int8_t *q, const float *scale, int64_t blocks, int32_t t,
                        int32_t d, uint16_t *out, void *stream);

/*
 * Flush of FP16 window blocks into a block pool in one launch: block p of k
 * and v (fp16 [blocks][t][d] each) is quantized -- K per channel, V per token
 * -- into pool slot dst[p] (int32 device array [blocks]): k_pool / v_pool
 * int8 [pool_blocks][t][d], k_scale fp32 [pool_blocks][d], v_scale fp32
 * [pool_blocks][t].  Entries of dst outside [0, pool_blocks) are skipped
 * (their slots are not written); two entries naming the same slot race.
 * Slots not named by dst are left unchanged.
 */
int kv_flush_blocks(const uint16_t *k, const uint16_t *v, int64_t blocks, int32_t t,
                    int32_t d, int32_t bits, const int32_t *dst, int64_t pool_blocks,
                    int8_t *k_pool, float *k_scale, int8_t *v_pool, float *v_scale,
                    void *stream);

/*
 * The paged INT8 cache
 * --------------------
 * One layer's keys and values of many sequences.  A page holds `page`
 * consecutive tokens of one sequence for one kv head, as int8 codes with one
 * fp32 scale for K and one for V (scale and codes by the map above, taken over
 * all page * d values: scale = max|x| / 127 floored at 1e-8, codes =
 * clamp(rint(x / scale), -128, 127), each step one binary32 operation; with a NaN
 * among the values the scale is NaN, with an infinity infinite, whatever the codes).  A
 * page's scale needs all of its tokens, so the newest tokens stay in fp16: a
 * slot per sequence holds the two highest pages that it has reached (the ring;
 * page p of the sequence in half p % 2), a page that becomes full is quantized
 * into the pool as well, and readers take the unfinished page from the ring.
 *
 * A sequence can be shortened (drafted tokens taken back) by calling again with a
 * smaller ctx_lens, no further than to the first token of the page before the
 * highest one that it has reached, in however many steps: the ring gave page p's
 * place to page p + 2 and does not get it back.  Beyond that only to a multiple of
 * `page` (0 among them), where no page is unfinished, and from then on no further
 * back than there.  The library cannot tell: a sequence that is shortened further
 * reads a later page's tokens from the ring.
 *
 * Both pools have the order in which the attention kernels read them: inside
 * a page of one head, K is [page / 64][4][d / 16][16][16] -- token
 * 64 i + 16 (m / 4) + 4 a + m % 4, channel 16 c + e at [i][a][c][m][e] -- and V
 * is [page / 16][d][16], token 16 i + j at [i][channel][j].  Ring pages have the
 * same order in fp16.
 *
 *  - page: 64, 128 or 256.  d: 64, 96, 128 or 256.  n_kv in [1, 1024], n_q a
 *    multiple of n_kv, at most 1024; query head i reads kv head
 *    i / (n_q / n_kv).  batch: at most 65536, and batch * n_kv at most 2^21.
 *    A sequence's tokens (table_cols * page) end before 2^30.
 *  - Alignment: k, v, k_tail, v_tail, q, k, v of new tokens and out 16 bytes,
 *    the rest 4 (the rotation table 16).
 */
typedef struct kv_paged_cache {
    int8_t *k, *v;              /* [pages][n_kv][page * d], in the order above */
    float *k_scale, *v_scale;   /* [pages][n_kv] */
    uint16_t *k_tail, *v_tail;  /* fp16 [slots][2][n_kv][page * d] */
    int64_t pages, slots;
    int32_t n_kv, d, page;
} kv_paged_cache;

/*
 * The sequences of one call: rows cu_q[b] .. cu_q[b + 1] - 1 of the new tokens
 * (or queries) belong to sequence b, which holds ctx_lens[b] tokens before
 * them; its page p is pool page block_table[b][p] and its ring is slots[b].
 * Rows before cu_q[0] and from cu_q[batch] on (padding) belong to none.  All
 * four arrays are int32 device arrays, read when the kernels run; how attention is
 * run goes by the sizes below, table_cols standing for the length of the sequences
 * (a narrower table for short ones is faster).  A sequence
 * with ctx_lens[b] < 0, slots[b] outside [0, cache.slots) or more than
 * table_cols full pages is skipped as if it had no rows.  cu_q must not
 * decrease (a decreasing one gives unspecified, memory-safe results); two
 * sequences of one call must not share a slot, nor a page that the call fills.
 */
typedef struct kv_paged_batch {
    const int32_t *cu_q;         /* [batch + 1] */
    const int32_t *ctx_lens;     /* [batch] */
    const int32_t *block_table;  /* [batch][table_cols] */
    const int32_t *slots;        /* [batch] */
    int64_t tokens;              /* rows of the call */
    int32_t batch, table_cols;
} kv_paged_batch;

/*
 * Appends k and v (fp16 [tokens][n_kv][d], row strides in elements) behind
 * each sequence's ctx_lens tokens.  With `rope`, k and q (fp16
 * [tokens][n_q][d], optional) are rotated first: rope is fp32
 * [rope_rows][rope_dim / 2][2], cosine and sine of pair j at a position;
 * row r has position positions[r] (int32 device array, required with rope).
 * Pair j is channels (j, j + rope_dim / 2), or (2 j, 2 j + 1) if `interleaved`;
 * channels from rope_dim on are copied.  a' = a cos - b sin, b' = b cos + a sin
 * in binary64, rounded once to fp16.  A position outside [0, rope_rows) gives
 * NaN.  q_out is fp16 [tokens][n_q][d], contiguous; rows of no sequence are
 * rotated as well.  Pages whose block_table entry is outside [0, pages) are
 * not stored.  Strides: multiples of 8 (at least n_kv * d, n_q * d).
 * rope_dim: a multiple of 32, at most d.  q NULL: n_q is not read.
 */
int kv_paged_append(const kv_paged_cache *cache, const kv_paged_batch *batch, const uint16_t *k, int64_t k_stride,
                    const uint16_t *v, int64_t v_stride, const uint16_t *q, int64_t q_stride, int32_t n_q,
                    const float *rope, int64_t rope_rows, int32_t rope_dim, int32_t interleaved,
                    const int32_t *positions, uint16_t *q_out, void *stream);

/*
 * Pages ids[0 .. n) of the pool, dequantized in the order of tokens: k_out,
 * v_out fp16 [n][n_kv][page][d] = fp16(code * scale).  Entries of ids outside
 * [0, pages) are skipped (their outputs are not written).
 */
int kv_paged_read(const kv_paged_cache *cache, const int32_t *ids, int64_t n, uint16_t *k_out, uint16_t *v_out,
                  void *stream);

/* Workspace bytes of kv_paged_attention; no HIP call is made. */
int64_t kv_paged_attention_workspace_size(int64_t tokens, int32_t batch, int32_t n_q, int32_t n_kv, int32_t d);

/*
 * Attention of q (fp16 [tokens][n_q][d], row stride in elements) over the
 * cache, whose last tokens are the batch's own (append first): row i of a
 * sequence stands at index ctx_lens[b] + i and sees the tokens j <= that
 * index, with window > 0 only those with index - j < window and the first
 * `sinks` tokens.  out fp16 [tokens][n_q][d], contiguous:
 * softmax_j(scale * q . k_j) v, with scores, sums and statistics in binary32 and
 * the output rounded once; in calls of many rows a sequence each weight of the
 * second product is rounded to fp16 too (2^-11; in others to two fp16 parts, 2^-22).
 * Pages whose block_table entry is outside [0, pages) are not visible (pages that
 * no row sees are not looked up at all); a row that sees nothing gives zeros.  Rows
 * of no sequence are left as they were.  An infinity or NaN in the k or v of a
 * token that is read from the ring gives NaN in the rows that see the token (with a
 * weight above zero) and reaches no other; one that was quantized has spoiled its
 * page for its kv head: NaN in the rows that see any of the page's tokens, and in
 * no other.  A page with scales of 0 (nobody filled it) counts as zeros.
 * `workspace`: device memory of at least kv_paged_attention_workspace_size bytes,
 * 16-byte aligned, overwritten; calls sharing a workspace must not overlap.
 * Results are deterministic for given inputs and sizes; a row's last bits depend on
 * the sizes of its call (tokens, batch, table_cols, window), which choose how it is
 * run.
 */
int kv_paged_attention(const kv_paged_cache *cache, const kv_paged_batch *batch, const uint16_t *q, int64_t q_stride,
                       int32_t n_q, float scale, int32_t window, int32_t sinks, void *workspace,
                       int64_t workspace_bytes, uint16_t *out, void *stream);

/*
 * Kernel selection report, for tests and profiling: writes to `name` the kernels
 * that kv_paged_attention launches for these sizes, in the form in which profilers
 * print their names ("kv_attend_split_kernel<128, 1, 2>, kv_join_kernel<128, 1, 1>"),
 * NUL-terminated and truncated to name_len bytes.  Nothing is launched and no HIP
 * call is made.  Returns the status that kv_paged_attention would return for these
 * sizes (Q4_ERR_NULL without a name, Q4_ERR_SHAPE for name_len < 1).
 */
int kv_paged_attention_config(int64_t tokens, int32_t batch, int32_t table_cols, int32_t page, int32_t n_q, int32_t n_kv,
                              int32_t d, int32_t window, int32_t sinks, char *name, int64_t name_len);

/*
 * Groups of a batch's sequences that begin with the same tokens (a system prompt, a
 * document): sequences cu_seqs[g] .. cu_seqs[g + 1] - 1 have the same pool pages in the
 * first pages[g] columns of their block tables.  Both are int32 device arrays, read when
 * the kernels run.  A sequence that no group names shares nothing.  cu_seqs must not
 * decrease (a decreasing one gives unspecified, memory-safe results).
 */
typedef struct kv_shared_prefix {
    const int32_t *cu_seqs;      /* [groups + 1] */
    const int32_t *pages;        /* [groups] */
    int32_t groups, max_pages;   /* 1 .. 65536 groups, groups * n_kv at most 2^21; no group shares more than max_pages,
                                    which is in [1, 2^24] */
} kv_shared_prefix;

/* Workspace bytes of kv_paged_attention_shared; no HIP call is made. */
int64_t kv_paged_attention_shared_workspace_size(int64_t tokens, int32_t batch, int32_t table_cols, int32_t page,
                                                 int32_t groups, int32_t max_pages, int32_t n_q, int32_t n_kv, int32_t d);

/*
 * kv_paged_attention without a window, with the shared pages read and scored once for each
 * group, all of its rows at a time: the same result but for the order of sums, each weight of the
 * second product in two fp16 parts (2^-22).  Of a group's pages the first
 * min(pages[g], max_pages) are taken together, from the block table of its first
 * sequence that has rows and has finished them (ctx_lens[b] / page); a sequence that has not
 * attends to all of its tokens by itself.  A call of more than 64 rows a kv head for each
 * sequence on average (tokens / batch, rounded up, times n_q / n_kv) is run as
 * kv_paged_attention in all of its sequences.  How others are run goes by max_pages for the
 * shared pages and table_cols - max_pages for the sequences' own tokens.
 */
int kv_paged_attention_shared(const kv_paged_cache *cache, const kv_paged_batch *batch, const kv_shared_prefix *prefix,
                              const uint16_t *q, int64_t q_stride, int32_t n_q, float scale, void *workspace,
                              int64_t workspace_bytes, uint16_t *out, void *stream);

/* Kernel selection report of kv_paged_attention_shared, as kv_paged_attention_config. */
int kv_paged_attention_shared_config(int64_t tokens, int32_t batch, int32_t table_cols, int32_t page, int32_t groups,
                                     int32_t max_pages, int32_t n_q, int32_t n_kv, int32_t d, char *name, int64_t name_len);

#ifdef __cplusplus
}
#endif

#endif /* KV_CODEC_H */
