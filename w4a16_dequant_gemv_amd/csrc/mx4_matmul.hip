// mx4_matmul.hip -- products of MXFP4 operands on the matrix cores (mxfp4.h).
#include <stdio.h>
#include <algorithm>
#include <type_traits>

#include "gemm_tile.h"
#include "mx4_device.h"
#include "q4_launch.h"

namespace {

constexpr int kRowWaves = 8;

// Few rows of x: a workgroup has 16 rows of W and all of x, its waves take steps of 256
// elements in turn and are summed at the end.  W goes from memory to operand registers, two
// steps ahead; x lies in LDS, `chunk` steps of it at a time, and comes there as codes or, with
// X the type of its elements, is quantized on the way.  What lies behind a row's last block
// is zero in x and so does not matter in W.
template <int TYPE, int MT, int X>
__global__ __launch_bounds__(64 * kRowWaves, 4) void mx4_rows_kernel(const void *__restrict__ x, const uint8_t *__restrict__ xs,
                                                           int64_t stride, const uint8_t *__restrict__ wc,
                                                           const uint8_t *__restrict__ ws, int m, int n_out, int k,
                                                           int chunk, uint16_t *__restrict__ y)
{
    constexpr int NW = kRowWaves;
    extern __shared__ __attribute__((aligned(16))) char smem[];          // [chunk][m][128], then scales [chunk][m][8]
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = blockIdx.x * 16, steps = (k + 255) / 256, blocks = k / 32, pitch = k / 2;
    const int wr = min(n0 + r, n_out - 1);
    const uint8_t *wrow = wc + (int64_t)wr * pitch, *wscale = ws + (int64_t)wr * 8 + 2 * g;
    char *xscale = smem + chunk * m * 128;

    constexpr int U = 2;
    u32x4 a[U][2];
    uint32_t sa[U];
    auto load = [&](int s, int u) {
        const int b = s * 8 + 2 * g;                                     // this lane's blocks: b, b + 1
        a[u][0] = *reinterpret_cast<const u32x4 *>(wrow + (int64_t)min(b, blocks - 1) * 16);
        a[u][1] = *reinterpret_cast<const u32x4 *>(wrow + (int64_t)min(b + 1, blocks - 1) * 16);
        sa[u] = *reinterpret_cast<const uint16_t *>(wscale + (int64_t)s * n_out * 8);
    };
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (wave + u * NW < steps) load(wave + u * NW, u);

    for (int c0 = 0; c0 < steps; c0 += chunk) {
        const int have = min(chunk, steps - c0);
        if (c0) __syncthreads();                                         // the chunk before has been read
        if constexpr (X < 0) {
            const uint8_t *xc = static_cast<const uint8_t *>(x);
            for (int i = tid; i < have * m * 8; i += 64 * NW) {
                const int row = (i >> 3) % m, s = (i >> 3) / m, b = (c0 + s) * 8 + (i & 7);
                u32x4 v = {0u, 0u, 0u, 0u};
                if (b < blocks) v = *reinterpret_cast<const u32x4 *>(xc + (int64_t)row * pitch + b * 16);
                *reinterpret_cast<u32x4 *>(smem + (s * m + row) * 128 + (((i & 7) ^ swz(row)) * 16)) = v;
            }
            for (int i = tid; i < have * m; i += 64 * NW) {
                const int left = blocks - (c0 + i / m) * 8;
                const uint64_t v = *reinterpret_cast<const uint64_t *>(xs + ((int64_t)c0 * m + i) * 8);
                *reinterpret_cast<uint64_t *>(xscale + i * 8) = left < 8 ? v & ~0ull >> (64 - 8 * left) : v;
            }
        } else {
            typedef typename Mx4Type<X>::T T;
            for (int i = tid; i < have * m * 32; i += 64 * NW) {         // eight elements, four lanes a block
                const int row = (i >> 5) % m, s = (i >> 5) / m, c = i & 31, at = (c0 + s) * 256 + c * 8;
                float v[8] = {};
                if (at < k) mx4_load8<X>(static_cast<const T *>(x) + row * stride + at, v);
                uint32_t top = mx4_top8(v);
                top = max(top, (uint32_t)__shfl_xor((int)top, 1));
                top = max(top, (uint32_t)__shfl_xor((int)top, 2));
                const int e = mx4_scale(top);
                *reinterpret_cast<uint32_t *>(smem + (s * m + row) * 128 + (((c >> 2) ^ swz(row)) * 16) + (c & 3) * 4) =
                    mx4_codes8(v, e);
                if ((c & 3) == 0) xscale[(s * m + row) * 8 + (c >> 2)] = (char)e;
            }
        }
        __syncthreads();
        for (int s = wave; s < have; s += U * NW)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = s + u * NW;
                if (at >= have) break;
                const int left = blocks - (c0 + at) * 8 - 2 * g;
                const uint32_t sw = left >= 2 ? sa[u] : left == 1 ? sa[u] & 0xFFu : 0u;
                const u32x4 w0 = a[u][0], w1 = a[u][1];
                if (c0 + at + U * NW < steps) load(c0 + at + U * NW, u);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int row = min(t * 16 + r, m - 1);
                    const char *p = smem + (at * m + row) * 128;
                    const u32x4 b0 = *reinterpret_cast<const u32x4 *>(p + (((2 * g) ^ swz(row)) * 16));
                    const u32x4 b1 = *reinterpret_cast<const u32x4 *>(p + (((2 * g + 1) ^ swz(row)) * 16));
                    const uint32_t sx = *reinterpret_cast<const uint16_t *>(xscale + (at * m + row) * 8 + 2 * g);
                    acc[t] = mx4_mfma16<0, 0>(w0, b0, acc[t], sw, sx);
                    acc[t] = mx4_mfma16<1, 1>(w1, b1, acc[t], sw, sx);
                }
            }
    }
    __syncthreads();
    f32x4 *part = reinterpret_cast<f32x4 *>(smem);
#pragma unroll
    for (int t = 0; t < MT; ++t) part[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    const float *sums = reinterpret_cast<const float *>(smem);
    for (int i = tid; i < MT * 256; i += 64 * NW) {
        const int t = i / 256, row = i / 16 % 16, ch = i % 16;           // x row, channel
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) sum += sums[((w * MT + t) * 64 + ch / 4 * 16 + row) * 4 + ch % 4];
        if (t * 16 + row < m && n0 + ch < n_out)
            y[(int64_t)(t * 16 + row) * n_out + n0 + ch] = Mx4Type<TYPE>::store(sum);
    }
}

// 64 lanes x 16 bytes from memory to LDS at `lds` (lane after lane), without a stop in
// registers.  In assembly, since the compiler makes every LDS read of a wave wait for all
// such loads that the wave has on their way; the barrier that ends a stage waits for them.
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff)
{
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" : : "{m0}"(lds), "v"(voff), "s"(rsrc), "s"(soff) : "memory");
}

__device__ __forceinline__ u32x4 buffer_of(const void *p, uint32_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xFFFFu,
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)kBufferFlags};
}

// Many rows of x: a workgroup has BM = 64 TM rows of x and BN = 64 TN of W, each of its four
// waves (one a SIMD, two by two) a quarter of them as TM x TN blocks of 32 x 32.  A stage is
// 256 elements of every row, 128 bytes, and their scales; two stages in LDS.  A wave reads
// the operands of the next 64 elements between the matrix instructions of these ones.  In
// the middle of a stage's last ones every wave has all it needs of the stage and the next one
// has come in: one barrier, and the stage after that is sent for, a whole stage ahead.  Where k ends inside a stage,
// the codes behind it are the next row's or zeros; their scales are made 2^-127 on both sides, and such products vanish
// in any sum.
template <int TYPE, int TM, int TN, int NB>
__global__ __launch_bounds__(256, 1) void mx4_tile_kernel(const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xs,
                                                          const uint8_t *__restrict__ wc, const uint8_t *__restrict__ ws,
                                                          int m, int n_out, int k, uint16_t *__restrict__ y, int tiles_m,
                                                          int tiles_n)
{
    constexpr int BM = 64 * TM, BN = 64 * TN;
    constexpr int XSL = (BM + 127) / 128, WSL = (BN + 127) / 128;        // loads of scales: 128 rows each
    constexpr int X = 0, W = BM * 128, XS = W + BN * 128, WS = XS + XSL * 1024, STAGE = WS + WSL * 1024;
    constexpr int XL = BM / 32, WL = BN / 32;                            // loads of a wave: 8 rows each
    extern __shared__ __attribute__((aligned(16))) char smem[];
    int tile_m, tile_n;
    xcd_tile<4>(blockIdx.x, tiles_m, tiles_n, tile_m, tile_n);
    const int m0 = tile_m * BM, n0 = tile_n * BN;
    const int rows_m = min(BM, m - m0), rows_n = min(BN, n_out - n0);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pitch = k / 2, steps = (k + 255) / 256;

    // Loading: lane i of a load puts 16 bytes at row i / 8, place i % 8, where swz puts another chunk of the row.
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
    const u32x4 xr = buffer_of(xc + (int64_t)m0 * pitch, (uint32_t)rows_m * pitch);
    const u32x4 wr = buffer_of(wc + (int64_t)n0 * pitch, (uint32_t)rows_n * pitch);
    uint32_t xoff[XL], woff[WL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
        const int r = (wave * XL + i) * 8 + (lane >> 3);
        xoff[i] = (uint32_t)min(r, rows_m - 1) * pitch + ((lane & 7) ^ swz(r)) * 16;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
        const int r = (wave * WL + i) * 8 + (lane >> 3);
        woff[i] = (uint32_t)min(r, rows_n - 1) * pitch + ((lane & 7) ^ swz(r)) * 16;
    }
    // Piece p of stage s; behind the last stage the buffers are empty and nothing is read.
    constexpr int PIECES = XL + WL + 1;
    auto load = [&](int s, int buf, int p) {
        const uint32_t at = lds0 + buf * STAGE;
        const bool there = s < steps;
        if (p < XL) {
            u32x4 b = xr;
            b[2] = there ? b[2] : 0u;
            load_to_lds(b, at + X + (wave * XL + p) * 1024, xoff[p], s * 128);
        } else if (p < XL + WL) {
            u32x4 b = wr;
            b[2] = there ? b[2] : 0u;
            load_to_lds(b, at + W + (wave * WL + p - XL) * 1024, woff[p - XL], s * 128);
        } else {
            // what lies behind the tile's rows comes as zeros; a wave with no part of its own repeats one, so
            // that all have as many loads on their way
            const int turn = wave % (XSL + WSL);
            const bool of_x = turn < XSL;
            const int part = of_x ? turn : turn - XSL;
            const uint8_t *from = of_x ? xs + ((int64_t)s * m + m0) * 8 : ws + ((int64_t)s * n_out + n0) * 8;
            load_to_lds(buffer_of(from, there ? (of_x ? rows_m : rows_n) * 8 : 0), at + (of_x ? XS : WS) + part * 1024,
                        part * 1024 + lane * 16, 0);
        }
    };

    // Operands: lane (r, g) has blocks 4 g + j of its row for the j-th quarter of a stage, their scales in a word.
    const int r = lane & 31, g = lane >> 5, wm = wave >> 1, wn = wave & 1;
    const uint32_t xrow = wm * 32 * TM + r, wrow = wn * 32 * TN + r;
    struct Frag {
        u32x4 x[TM], w[TN];
    };
    struct Scale {
        uint32_t x[TM], w[TN];
    };
    auto read = [&](Frag &f, int buf, int j, int i) {                    // the i-th of TM + TN
        const uint32_t c = ((4 * g + j) ^ swz(r)) * 16;
        if (i < TM) f.x[i] = *reinterpret_cast<const u32x4 *>(smem + buf * STAGE + X + (xrow + 32 * i) * 128 + c);
        else f.w[i - TM] = *reinterpret_cast<const u32x4 *>(smem + buf * STAGE + W + (wrow + 32 * (i - TM)) * 128 + c);
    };
    const int left = k / 32 - (steps - 1) * 8 - 4 * g;                   // blocks of the last stage for this lane
    const uint32_t tail = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << 8 * left) - 1;
    auto read_scale = [&](Scale &f, int buf, int i) {
        if (i < TM) f.x[i] = *reinterpret_cast<const uint32_t *>(smem + buf * STAGE + XS + (xrow + 32 * i) * 8 + 4 * g);
        else f.w[i - TM] = *reinterpret_cast<const uint32_t *>(smem + buf * STAGE + WS + (wrow + 32 * (i - TM)) * 8 + 4 * g);
    };
    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    constexpr int ALL = TM * TN, PART = TM + TN;
    auto mma = [&](auto J, const Frag &f, const Scale &s, int t) {
        constexpr int j = decltype(J)::value;
        const int a = t / TN, b = t % TN;
        acc[a][b] = mx4_mfma32<j, j>(f.w[b], f.x[a], acc[a][b], s.w[b], s.x[a]);
    };
    // the products of quarter J, between them the reads of the next quarter and pieces LO .. HI - 1 of stage `to`
    constexpr int FIRST = PIECES / 3;
    auto quarter = [&](auto J, const Frag &f, const Scale &s, Frag &next, int buf, int to, int into, int lo, int hi) {
        constexpr int j = decltype(J)::value;
#pragma unroll
        for (int t = 0; t < ALL; ++t) {
            mma(J, f, s, t);
#pragma unroll
            for (int i = t * PART / ALL; i < (t + 1) * PART / ALL; ++i) read(next, buf, j + 1, i);
#pragma unroll
            for (int i = lo + t * (hi - lo) / ALL; i < lo + (t + 1) * (hi - lo) / ALL; ++i) load(to, into, i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    using Q0 = std::integral_constant<int, 0>;
    using Q1 = std::integral_constant<int, 1>;
    using Q2 = std::integral_constant<int, 2>;
    using Q3 = std::integral_constant<int, 3>;

    Frag f0, f1;
    Scale s0, s1;
    // stage s in buffer `buf`, `last` and `after` being the buffers around it
    auto stage = [&](int s, int last, int buf, int after, Scale &now, Scale &next) {
        if (s + 1 == steps) {
#pragma unroll
            for (int i = 0; i < TM; ++i) now.x[i] &= tail;
#pragma unroll
            for (int i = 0; i < TN; ++i) now.w[i] &= tail;
        }
        quarter(Q0{}, f0, now, f1, buf, s + NB - 1, last, FIRST, PIECES);
        quarter(Q1{}, f1, now, f0, buf, 0, 0, 0, 0);
        quarter(Q2{}, f0, now, f1, buf, 0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < ALL / 2; ++t) {
            mma(Q3{}, f1, now, t);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vmem<(NB - 2) * PIECES>();
        barrier_keep_vmem();
        // behind the last stage old values are read and not used
#pragma unroll
        for (int t = ALL / 2; t < ALL; ++t) {
            constexpr int HALF = ALL - ALL / 2;
            const int u = t - ALL / 2;
#pragma unroll
            for (int i = u * PART / HALF; i < (u + 1) * PART / HALF; ++i) {
                read(f0, after, 0, i);
                read_scale(next, after, i);
            }
            mma(Q3{}, f1, now, t);
#pragma unroll
            for (int i = u * FIRST / HALF; i < (u + 1) * FIRST / HALF; ++i) load(s + NB, buf, i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    {
#pragma unroll
        for (int s = 0; s < NB - 1; ++s)
#pragma unroll
            for (int i = 0; i < PIECES; ++i) load(s, s, i);
        wait_vmem<(NB - 2) * PIECES>();
        barrier_keep_vmem();
#pragma unroll
        for (int i = 0; i < FIRST; ++i) load(NB - 1, NB - 1, i);
#pragma unroll
        for (int i = 0; i < PART; ++i) {
            read(f0, 0, 0, i);
            read_scale(s0, 0, i);
        }
        int s = 0, last = NB - 1, buf = 0, after = 1;
        auto on = [&] {
            last = buf;
            buf = after;
            after = after + 1 == NB ? 0 : after + 1;
        };
        for (; s + 2 <= steps; s += 2) {
            stage(s, last, buf, after, s0, s1);
            on();
            stage(s + 1, last, buf, after, s1, s0);
            on();
        }
        if (s < steps) stage(s, last, buf, after, s0, s1);
        wait_vmem<0>();
    }
    // y goes through LDS (rows padded to YS bytes) and leaves as 16-byte pieces of whole rows.
    constexpr int YS = BN * 2 + 16;
    static_assert(BM * YS <= NB * STAGE, "output tile exceeds LDS");
    __syncthreads();
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x16 &v = acc[a][b];
                const uint32_t lo = Mx4Type<TYPE>::store(v[4 * q]) | (uint32_t)Mx4Type<TYPE>::store(v[4 * q + 1]) << 16;
                const uint32_t hi = Mx4Type<TYPE>::store(v[4 * q + 2]) | (uint32_t)Mx4Type<TYPE>::store(v[4 * q + 3]) << 16;
                *reinterpret_cast<u32x2 *>(smem + (xrow + 32 * a) * YS + (wn * 32 * TN + 32 * b + 8 * q + 4 * g) * 2) =
                    u32x2{lo, hi};
            }
    __syncthreads();
    const int cols = min(BN, n_out - n0);
    uint16_t *out = y + (int64_t)m0 * n_out + n0;
    if ((reinterpret_cast<uintptr_t>(y) & 15) == 0 && (n_out & 7) == 0) {
        constexpr int CPR = BN / 8;
#pragma unroll 4
        for (int i = tid; i < rows_m * CPR; i += 256) {
            const int row = i / CPR, c = i % CPR * 8;
            if (c < cols)
                *reinterpret_cast<u32x4 *>(out + (int64_t)row * n_out + c) = *reinterpret_cast<const u32x4 *>(smem + row * YS + c * 2);
        }
    } else {
        // rows that begin anywhere: a wave's stores are still side by side
#pragma unroll 8
        for (int i = tid; i < rows_m * BN; i += 256) {
            const int row = i / BN, c = i % BN;
            if (c < cols) out[(int64_t)row * n_out + c] = *reinterpret_cast<const uint16_t *>(smem + row * YS + c * 2);
        }
    }
}

template <int TYPE, int TM, int TN, int NB>
hipError_t launch_tiles(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int m, int n_out,
                        int k, uint16_t *y, hipStream_t stream)
{
    constexpr int LDS = NB * (64 * (TM + TN) * 128 + ((TM + 1) / 2 + (TN + 1) / 2) * 1024);
    auto kernel = mx4_tile_kernel<TYPE, TM, TN, NB>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (e != hipSuccess) return e;
    const int tiles_m = (m + 64 * TM - 1) / (64 * TM), tiles_n = (n_out + 64 * TN - 1) / (64 * TN);
    kernel<<<(unsigned)(tiles_m * tiles_n), 256, LDS, stream>>>(xc, xs, wc, ws, m, n_out, k, y, tiles_m, tiles_n);
    return hipGetLastError();
}

template <int TYPE, int MT, int X>
hipError_t launch_rows(const void *x, const uint8_t *xs, int64_t stride, const uint8_t *wc, const uint8_t *ws, int m,
                       int n_out, int k, uint16_t *y, hipStream_t stream)
{
    constexpr int NW = kRowWaves, ROUND = 2 * NW;                                        // steps of one round of the waves
    const int steps = (k + 255) / 256, most = std::max(1, 80 * 1024 / (m * 136) / ROUND) * ROUND;
    const int chunk = std::min(most, steps);
    const int lds = std::max(chunk * m * 136, NW * MT * 1024);
    auto kernel = mx4_rows_kernel<TYPE, MT, X>;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<(unsigned)((n_out + 15) / 16), 64 * NW, lds, stream>>>(x, xs, stride, wc, ws, m, n_out, k, chunk, y);
    return hipGetLastError();
}

// How a product is run: by mx4_rows_kernel (tm == 0; at most 32 rows of x), or by tiles of 64 tm x 64 tn
// with nb stages in LDS.
struct Plan {
    int tm, tn, nb;
};

struct TileCost {
    Plan plan;
    int slots;                       // workgroups that the 256 CUs hold
    double start, alone, full;       // us: a tile's beginning and end; a stage with few and with all CUs busy
};

// Measured with 64 to 4096 rows of x, n_out from 1024 to 28672, k from 1024 to 8192; off by 10 % at most where it
// matters.  (us, the kernels below in order: 64 x 8192 x 8192 12.5, 15.3, 18.2, 26.9, 37.3, 42.3; 512 x 11008 x 4096
// 30.9, 21.7, 22.7, 18.3, 22.2, 25.8; 2048 x 11008 x 4096 94.8, 70.8, 67.0, 57.6, 53.0, 58.4; 8192^3 497, 398, 358, 306,
// 271, 244.)
constexpr TileCost kTiles[] = {
    {{1, 1, 4}, 512, 3.0, 0.20, 0.47}, {{2, 1, 3}, 512, 3.3, 0.25, 0.74}, {{2, 2, 3}, 256, 3.7, 0.38, 0.60},
    {{2, 2, 2}, 512, 4.0, 0.50, 1.10}, {{3, 4, 2}, 256, 5.0, 0.80, 1.38}, {{4, 4, 2}, 256, 6.0, 1.00, 1.78},
};

Plan plan_for(int64_t m, int64_t n_out, int64_t k)
{
    const double steps = (double)((k + 255) / 256);
    const double memory = (double)(n_out * k) * 17 / 32 / 4.6e6;         // us, W at what a stream of it reaches
    Plan best = {};
    double least = 1e30;
    for (const TileCost &t : kTiles) {
        const int64_t bm = 64 * t.plan.tm, bn = 64 * t.plan.tn;
        const int64_t tiles = ((m + bm - 1) / bm) * ((n_out + bn - 1) / bn), full = tiles / t.slots, rest = tiles % t.slots;
        double cost = (double)full * (t.start + steps * t.full);
        if (rest) cost += t.start + steps * (t.alone + (t.full - t.alone) * (double)rest / t.slots);
        cost = std::max(cost, memory);
        if (cost < least) {
            least = cost;
            best = t.plan;
        }
    }
    // 16 rows of W a workgroup: most workgroups where there are few rows of x, but x comes once for each (1 x 4096 x
    // 4096 4.3 us against 7.0 in the smallest tiles, 16 x 1024 x 16384 11.3 and 18.1, 16 x 8192 x 8192 12.6 and 10.9).
    if (m <= 32) {
        const double groups = (double)((n_out + 15) / 16), rounds = std::max(1.0, groups / 512);
        const double slope = (0.065 + 0.0043 * (double)m) * (1.0 + 1.3 * std::min(1.0, groups / 512));
        const double cost = 2.5 + steps * slope * rounds + 0.8 * (rounds - 1.0);
        if (std::max(cost, memory) < least) best = {0, 0, 0};
    }
    return best;
}

// x is quantized by the product's own workgroups where that costs less than a launch of its own (2 us): each does it for
// itself (1 x 8192 x 8192 10.9 us, 12.4 in two launches; 4 x 4096 x 4096 6.0 and 6.4; 8 x 4096 x 4096 8.0 and 6.8).
bool quantizes_itself(const Plan &p, int64_t m, int64_t k) { return p.tm == 0 && m * k <= 16384; }

template <int TYPE>
hipError_t launch(const Plan &p, const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int m,
                  int n_out, int k, uint16_t *y, hipStream_t stream)
{
    if (p.tm == 0)
        return m <= 16 ? launch_rows<TYPE, 1, -1>(xc, xs, 0, wc, ws, m, n_out, k, y, stream)
                       : launch_rows<TYPE, 2, -1>(xc, xs, 0, wc, ws, m, n_out, k, y, stream);
    switch (p.tm * 100 + p.tn * 10 + p.nb) {
    case 114: return launch_tiles<TYPE, 1, 1, 4>(xc, xs, wc, ws, m, n_out, k, y, stream);
    case 213: return launch_tiles<TYPE, 2, 1, 3>(xc, xs, wc, ws, m, n_out, k, y, stream);
    case 223: return launch_tiles<TYPE, 2, 2, 3>(xc, xs, wc, ws, m, n_out, k, y, stream);
    case 222: return launch_tiles<TYPE, 2, 2, 2>(xc, xs, wc, ws, m, n_out, k, y, stream);
    case 342: return launch_tiles<TYPE, 3, 4, 2>(xc, xs, wc, ws, m, n_out, k, y, stream);
    case 442: return launch_tiles<TYPE, 4, 4, 2>(xc, xs, wc, ws, m, n_out, k, y, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int TYPE>
hipError_t launch_linear(const void *x, int64_t stride, const uint8_t *wc, const uint8_t *ws, int m, int n_out, int k,
                         uint8_t *codes, uint8_t *scales, uint16_t *y, hipStream_t stream)
{
    const Plan p = plan_for(m, n_out, k);
    if (quantizes_itself(p, m, k))
        return m <= 16 ? launch_rows<TYPE, 1, TYPE>(x, nullptr, stride, wc, ws, m, n_out, k, y, stream)
                       : launch_rows<TYPE, 2, TYPE>(x, nullptr, stride, wc, ws, m, n_out, k, y, stream);
    const hipError_t e = mx4_launch_quantize(x, TYPE, m, k, stride, codes, scales, stream);
    return e != hipSuccess ? e : launch<TYPE>(p, codes, scales, wc, ws, m, n_out, k, y, stream);
}

}  // namespace

hipError_t mx4_launch_matmul(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int64_t m,
                             int64_t n_out, int64_t k, int type, void *y, hipStream_t stream)
{
    auto f = type == MX4_F16 ? launch<MX4_F16> : launch<MX4_BF16>;
    return f(plan_for(m, n_out, k), xc, xs, wc, ws, (int)m, (int)n_out, (int)k, (uint16_t *)y, stream);
}

hipError_t mx4_launch_linear(const void *x, int type, int64_t stride, const uint8_t *wc, const uint8_t *ws, int64_t m,
                             int64_t n_out, int64_t k, uint8_t *codes, uint8_t *scales, void *y, hipStream_t stream)
{
    auto f = type == MX4_F16 ? launch_linear<MX4_F16> : launch_linear<MX4_BF16>;
    return f(x, stride, wc, ws, (int)m, (int)n_out, (int)k, codes, scales, (uint16_t *)y, stream);
}

bool mx4_linear_needs_room(int64_t m, int64_t n_out, int64_t k) { return !quantizes_itself(plan_for(m, n_out, k), m, k); }

void mx4_linear_name(int64_t m, int64_t n_out, int64_t k, int type, bool linear, char *name, int64_t name_len)
{
    const Plan p = plan_for(m, n_out, k);
    const bool self = linear && quantizes_itself(p, m, k);
    const char *first = "";
    if (linear && !self) first = type == MX4_F16 ? "mx4_quantize_kernel<0>, " : "mx4_quantize_kernel<1>, ";
    if (p.tm == 0) snprintf(name, (size_t)name_len, "%smx4_rows_kernel<%d, %d, %d>", first, type, m <= 16 ? 1 : 2, self ? type : -1);
    else snprintf(name, (size_t)name_len, "%smx4_tile_kernel<%d, %d, %d, %d>", first, type, p.tm, p.tn, p.nb);
}
