// kv_device.h -- the symmetric quantization map of the KV codec and of the paged
// cache, and the paged cache's page order and sequence bookkeeping.  Units that
// quantize are built without FMA contraction and with correctly rounded division.
#pragma once

#include "kv_codec.h"
#include "q4_device.h"

__device__ __forceinline__ float kv_scale(float amax, float qmax)
{
    float s = amax / qmax;
    return s < 1e-8f ? 1e-8f : s;
}

// round(v / s) clamped to [-qmax - 1, qmax], as the byte of an int8.  The
// product with r, the hardware reciprocal of s (within 1 ulp), is within
// 2^-21.5 * |v / s| of the correctly rounded quotient; for |v / s| < 2^7 that
// is below 2^-14, so both round to the same integer unless the product lies
// within 2^-14 of a half-integer.  There, and for larger quotients, the
// correctly rounded division decides: the code is the one round(v / s)
// gives, bit for bit.
__device__ __forceinline__ uint32_t kv_code(float v, float s, float r, float qmax)
{
    const float a = v * r;
    float c = __builtin_rintf(a);
    if (fabsf(a - c) > 0.5f - 0x1p-14f || fabsf(a) >= 128.0f) c = __builtin_rintf(v / s);
    c = fminf(fmaxf(c, -qmax - 1.0f), qmax);
    return (uint32_t)(int32_t)c & 0xFFu;
}

// Order of a page of one head (kv_codec.h): offset of token tok's channels
// 16c .. 16c + 15 in a K page, and of token tok, channel ch in a V page.  Token
// and channel orders are those of the matrix cores' operands: a wave's 16-byte
// loads of a page are contiguous.
__device__ __forceinline__ int kv_k_index(int tok, int c, int chunks)
{
    return ((((tok >> 6) * 4 + ((tok & 15) >> 2)) * chunks + c) * 16 + ((tok & 63) >> 4) * 4 + (tok & 3)) * 16;
}

__device__ __forceinline__ int kv_v_index(int tok, int ch, int d) { return ((tok >> 4) * d + ch) * 16 + (tok & 15); }

// One sequence of a call: rows [q0, q0 + n), ctx tokens before them.  n is 0
// for sequences that the call skips.  Rows are clipped to the call's tokens
// whatever cu_q holds.
struct KvSeq {
    int q0, n, ctx, slot;
    __device__ int total() const { return ctx + n; }
};

__device__ __forceinline__ KvSeq kv_seq(const kv_paged_batch &p, int b, int64_t n_slots, int page_shift)
{
    KvSeq s;
    const int T = (int)p.tokens;
    s.q0 = min(max(p.cu_q[b], 0), T);
    s.n = max(min(p.cu_q[b + 1], T) - s.q0, 0);
    s.ctx = p.ctx_lens[b];
    s.slot = p.slots[b];
    if (s.ctx < 0 || s.slot < 0 || s.slot >= n_slots || ((int64_t)s.ctx + s.n) >> page_shift > p.table_cols) s.n = 0;
    return s;
}

// Inclusive sum over the lanes of a wave: row shifts, then broadcasts of the
// last lane of a row of 16 and of the first half, all on the VALU.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t kv_scan_step(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
    return v + (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ int64_t kv_wave_scan(int64_t v)
{
    v = kv_scan_step<0x111, 0xF>(v);       // row_shr:1
    v = kv_scan_step<0x112, 0xF>(v);       // row_shr:2
    v = kv_scan_step<0x114, 0xF>(v);       // row_shr:4
    v = kv_scan_step<0x118, 0xF>(v);       // row_shr:8
    v = kv_scan_step<0x142, 0xA>(v);       // row_bcast:15 into rows 1 and 3
    return kv_scan_step<0x143, 0xC>(v);    // row_bcast:31 into rows 2 and 3
}

// The value of v in lane i, the same i in every lane.
__device__ __forceinline__ int64_t kv_lane(int64_t v, int i)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, i);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), i);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Finds which of the batch's sequences item `u` falls in when sequence b has
// count(b) items: every lane of a wave calls it, 64 sequences a step.  False if
// there are not that many.
template <typename F>
__device__ __forceinline__ bool kv_locate(int batch, int64_t u, F count, int &b, int64_t &off)
{
    const int lane = threadIdx.x & 63;
    int64_t base = 0;
    for (int c = 0; c < batch; c += 64) {
        const int64_t n = c + lane < batch ? (int64_t)count(c + lane) : 0, incl = kv_wave_scan(n);
        const uint64_t hit = __ballot(u < base + incl);
        if (hit) {
            const int f = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
            b = c + f;
            off = u - base - kv_lane(incl - n, f);
            return true;
        }
        base += kv_lane(incl, 63);
    }
    return false;
}
