// mx4_matmul.hip -- products of MXFP4 operands on the matrix cores (mxfp4.h).
//
// y[i][j] = sum over blocks b of 2^(sx + sw - 254) sum over the block of cx cw: the matrix instructions take both
// operands' codes and scales as they are and add up in binary32.  A dozen rows of x or fewer are bound by W's way from
// HBM, thousands by the matrix cores, what lies between by the L2 caches and LDS.
#include <stdio.h>
#include <algorithm>
#include <type_traits>

#include "gemm_tile.h"
#include "mx4_device.h"
#include "q4_launch.h"

namespace {

constexpr int kRowWaves = 8;

// Few rows of x: a workgroup has 16 rows of W and all of x, its waves take steps of 256
// elements in turn and are summed at the end.  W goes from memory to operand registers, U
// steps ahead; x lies in LDS, `chunk` steps of it at a time, and comes there as codes or, with
// X the type of its elements, is quantized on the way.  What lies behind a row's last block
// is zero in x and so does not matter in W.  The 16 x 16 x 128 form: half as much padding with few rows of x
// as the 32 x 32 one.  Replayed with W from the Infinity Cache or HBM, 1 x 4096 x 4096 takes 4.2 us, of which a launch and
// the first loads are 2.9, 1 x 8192 x 8192 8.2 (4.3 TB/s), 1 x 28672 x 8192 23.7 (5.3 TB/s), 8 x 8192 x 28672 28.0 (4.5 TB/s).
template <int TYPE, int MT, int X, int U>
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
// such loads that the wave has on their way; the barrier that ends a stage waits for them.  A load may not take a
// scalar register that a vector instruction (readfirstlane) wrote less than five instructions before, which the compiler does
// not see to here: PAUSE of them for a buffer that was just made, none for one that is `fixed`.
// The range check counts both offsets, dword by dword, and the scalar one may exceed the buffer's bytes: what lies
// at or behind its end is not read and comes as zero (tests/test_gpu_buffer_range.py holds that).  With the stage's place in
// the vector offset, which needs an addition for each load, the tiles took 1 to 6 % longer (on quantized normal numbers 8192^3 230
// and 233 us, 333 x 4096 x 8192 13.9 and 14.8).
template <int PAUSE>
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t lds, uint32_t voff, uint32_t soff)
{
    asm volatile("s_nop %4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 : : "{m0}"(lds), "v"(voff), "s"(rsrc), "s"(soff), "n"(PAUSE) : "memory");
}

__device__ __forceinline__ u32x4 buffer_of(const void *p, uint32_t bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xFFFFu,
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)kBufferFlags};
}

// The same value, in scalar registers from here on.
__device__ __forceinline__ u32x4 fixed(u32x4 rsrc)
{
    asm volatile("s_nop 4" : "+s"(rsrc));
    return rsrc;
}

// What the kernels of many rows have in LDS: a tile of BM rows of x and BN of W, of which a stage is 256
// elements of every row, 128 bytes, and their scales.  Four waves load it in PIECES instructions each.
template <int BM, int BN>
struct Stages {
    static constexpr int XSL = (BM + 127) / 128, WSL = (BN + 127) / 128;                        // loads of scales: 128 rows each
    static constexpr int X = 0, W = BM * 128, XS = W + BN * 128, WS = XS + XSL * 1024, SIZE = WS + WSL * 1024;
    static constexpr int XL = BM / 32, WL = BN / 32, PIECES = XL + WL + 1;                      // loads of a wave: 8 rows each
    int m0, n0, rows_m, rows_n, steps, lane, wave;
    uint32_t lds0;
    u32x4 xr, wr;
    uint32_t xoff[XL], woff[WL];
    const uint8_t *scales;               // of this wave's load of scales: its rows', a step's distance, how many there are
    int64_t scale_step;
    uint32_t scale_bytes, scale_part, scale_at;

    // Lane i of a load puts 16 bytes at row i / 8, place i % 8, where swz puts another chunk of the row.
    __device__ __forceinline__ Stages(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int m, int n_out,
                                      int k, int tile_m, int tile_n, char *smem)
        : m0(tile_m * BM), n0(tile_n * BN)
    {
        rows_m = min(BM, m - m0);
        rows_n = min(BN, n_out - n0);
        steps = (k + 255) / 256;
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;
        const int pitch = k / 2;
        xr = fixed(buffer_of(xc + (int64_t)m0 * pitch, (uint32_t)rows_m * pitch));
        wr = fixed(buffer_of(wc + (int64_t)n0 * pitch, (uint32_t)rows_n * pitch));
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
        // a wave with no part of its own repeats one, so that all have as many loads on their way
        const int turn = wave % (XSL + WSL);
        const bool of_x = turn < XSL;
        scale_part = (of_x ? turn : turn - XSL) * 1024;
        scale_at = (of_x ? XS : WS) + scale_part;
        scales = of_x ? xs + (int64_t)m0 * 8 : ws + (int64_t)n0 * 8;
        scale_step = (int64_t)(of_x ? m : n_out) * 8;
        scale_bytes = (of_x ? rows_m : rows_n) * 8;
    }

    // Piece p of stage s; from stage `end` on the buffers are empty and nothing is read.  Behind a row's end the next
    // row's codes come, or, for the tile's last row, the zeros of the range check.
    __device__ __forceinline__ void load(int s, int end, int buf, int p) const
    {
        const uint32_t at = lds0 + buf * SIZE;
        const bool there = s < end;
        if (p < XL) {
            u32x4 b = xr;
            b[2] = there ? b[2] : 0u;
            load_to_lds<0>(b, at + X + (wave * XL + p) * 1024, xoff[p], s * 128);
        } else if (p < XL + WL) {
            u32x4 b = wr;
            b[2] = there ? b[2] : 0u;
            load_to_lds<0>(b, at + W + (wave * WL + p - XL) * 1024, woff[p - XL], s * 128);
        } else {
            // what lies behind the tile's rows comes as zeros
            load_to_lds<4>(buffer_of(scales + s * scale_step, there ? scale_bytes : 0), at + scale_at, scale_part + lane * 16, 0);
        }
    }
};

// Rows of a tile of y go through LDS (padded, so that a wave's rows lie in different banks) and leave as 16-byte pieces.
template <int BN>
constexpr int kRowOfY = BN * 2 + 16;

// Four sums, channels c .. c + 3 of row `row` of the tile.
template <int TYPE, int BN>
__device__ __forceinline__ void put_y(char *tile, int row, int c, float a, float b, float d, float e)
{
    const uint32_t lo = Mx4Type<TYPE>::store(a) | (uint32_t)Mx4Type<TYPE>::store(b) << 16;
    const uint32_t hi = Mx4Type<TYPE>::store(d) | (uint32_t)Mx4Type<TYPE>::store(e) << 16;
    *reinterpret_cast<u32x2 *>(tile + row * kRowOfY<BN> + c * 2) = u32x2{lo, hi};
}

template <int BN>
__device__ __forceinline__ void write_y(const char *tile, uint16_t *y, int m0, int n0, int rows_m, int n_out)
{
    const int cols = min(BN, n_out - n0);
    uint16_t *out = y + (int64_t)m0 * n_out + n0;
    if ((reinterpret_cast<uintptr_t>(y) & 15) == 0 && (n_out & 7) == 0) {
        constexpr int CPR = BN / 8;
#pragma unroll 4
        for (int i = threadIdx.x; i < rows_m * CPR; i += 256) {
            const int row = i / CPR, c = i % CPR * 8;
            if (c < cols)
                *reinterpret_cast<u32x4 *>(out + (int64_t)row * n_out + c) =
                    *reinterpret_cast<const u32x4 *>(tile + row * kRowOfY<BN> + c * 2);
        }
    } else {
        // rows that begin anywhere: a wave's stores are still side by side
#pragma unroll 8
        for (int i = threadIdx.x; i < rows_m * BN; i += 256) {
            const int row = i / BN, c = i % BN;
            if (c < cols) out[(int64_t)row * n_out + c] = *reinterpret_cast<const uint16_t *>(tile + row * kRowOfY<BN> + c * 2);
        }
    }
}

// Many rows of x, on the 32 x 32 x 64 form: a loop of nothing else reaches 6.5 PFLOP/s on random codes here, and 5.4 in the
// 16 x 16 form.  A workgroup has BM = 64 TM rows of x and BN = 64 TN of W, each of its four
// waves (one a SIMD, two by two) a quarter of them as TM x TN blocks of 32 x 32; NB stages in LDS.  A wave reads
// the operands of the next 64 elements between the matrix instructions of these ones.  In
// the middle of a stage's last ones every wave has all it needs of the stage and the next one
// has come in: one barrier, and the stage after that is sent for, a whole stage ahead.  Where k ends inside a stage,
// the codes behind it are the next row's or zeros; their scales are made 2^-127 on both sides, and such products vanish
// in any sum.
// Large tiles are bound by the matrix cores and the card's power: 8192^3 in tiles of 256 x 256 takes 244 us (4.5 PFLOP/s), 210
// without the loop's loads, 168 without its reads of LDS too (6.6 PFLOP/s).  Small ones are bound by what a CU can load:
// 18 KB in 0.26 us, 0.53 with two of them on each (PARTS: more CUs for a long k, each with a part of the stages, its sums
// left for mx4_join_kernel).
template <int TYPE, int TM, int TN, int NB, bool PARTS>
__global__ __launch_bounds__(256, 1) void mx4_tile_kernel(const uint8_t *__restrict__ xc, const uint8_t *__restrict__ xs,
                                                          const uint8_t *__restrict__ wc, const uint8_t *__restrict__ ws,
                                                          int m, int n_out, int k, void *__restrict__ to, int tiles_m,
                                                          int tiles_n, int splits)
{
    typedef Stages<64 * TM, 64 * TN> S;
    constexpr int STAGE = S::SIZE, X = S::X, W = S::W, XS = S::XS, WS = S::WS, PIECES = S::PIECES;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tiles = tiles_m * tiles_n, tile = PARTS ? (int)blockIdx.x % tiles : (int)blockIdx.x;
    int tile_m, tile_n;
    xcd_tile<4>(tile, tiles_m, tiles_n, tile_m, tile_n);
    const S st(xc, xs, wc, ws, m, n_out, k, tile_m, tile_n, smem);
    const int lane = st.lane, wave = st.wave, steps = st.steps;
    const int split = PARTS ? (int)blockIdx.x / tiles : 0;               // stages first .. end - 1 are this workgroup's
    const int first = PARTS ? split * steps / splits : 0, end = PARTS ? (split + 1) * steps / splits : steps;
    auto load = [&](int s, int buf, int p) { st.load(s, end, buf, p); };

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
    constexpr int FIRST = PIECES / 3, EARLY = ALL > 1 ? ALL / 2 : 1, MEET = ALL / 4;
    auto quarter = [&](auto J, const Frag &f, const Scale &s, Frag &next, int buf, int to, int into, int lo, int hi) {
        constexpr int j = decltype(J)::value;
#pragma unroll
        for (int t = 0; t < ALL; ++t) {
#pragma unroll
            for (int i = t * PART / EARLY; i < min((t + 1) * PART / EARLY, PART); ++i) read(next, buf, j + 1, i);
            mma(J, f, s, t);
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
        for (int t = 0; t < MEET; ++t) {
            mma(Q3{}, f1, now, t);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vmem<(NB - 2) * PIECES>();
        barrier_keep_vmem();
        // behind the last stage old values are read and not used
#pragma unroll
        for (int t = MEET; t < ALL; ++t) {
            constexpr int HALF = ALL - MEET;
            const int u = t - MEET;
#pragma unroll
            for (int i = u * PART / EARLY; i < min((u + 1) * PART / EARLY, PART); ++i) {
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
            for (int i = 0; i < PIECES; ++i) load(first + s, s, i);
        wait_vmem<(NB - 2) * PIECES>();
        barrier_keep_vmem();
#pragma unroll
        for (int i = 0; i < FIRST; ++i) load(first + NB - 1, NB - 1, i);
#pragma unroll
        for (int i = 0; i < PART; ++i) {
            read(f0, 0, 0, i);
            read_scale(s0, 0, i);
        }
        int s = first, last = NB - 1, buf = 0, after = 1;
        auto on = [&] {
            last = buf;
            buf = after;
            after = after + 1 == NB ? 0 : after + 1;
        };
        for (; s + 2 <= end; s += 2) {
            stage(s, last, buf, after, s0, s1);
            on();
            stage(s + 1, last, buf, after, s1, s0);
            on();
        }
        if (s < end) stage(s, last, buf, after, s0, s1);
        wait_vmem<0>();
    }
    if constexpr (PARTS) {
        // the sums as the lanes have them, block after block of 32 x 32
#pragma unroll
        for (int q = 0; q < 4; ++q)
            static_cast<f32x4 *>(to)[(((int64_t)blockIdx.x * 4 + wave) * 4 + q) * 64 + lane] =
                f32x4{acc[0][0][4 * q], acc[0][0][4 * q + 1], acc[0][0][4 * q + 2], acc[0][0][4 * q + 3]};
        return;
    }
    static_assert(!PARTS || ALL == 1, "the joining kernel takes tiles of 64 x 64");
    static_assert(64 * TM * kRowOfY<64 * TN> <= NB * STAGE, "output tile exceeds LDS");
    __syncthreads();
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
        for (int b = 0; b < TN; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x16 &v = acc[a][b];
                put_y<TYPE, 64 * TN>(smem, xrow + 32 * a, wn * 32 * TN + 32 * b + 8 * q + 4 * g, v[4 * q], v[4 * q + 1], v[4 * q + 2],
                                     v[4 * q + 3]);
            }
    __syncthreads();
    write_y<64 * TN>(smem, static_cast<uint16_t *>(to), st.m0, st.n0, st.rows_m, n_out);
}

// y from the sums of mx4_tile_kernel<TYPE, 1, 1, NB, true>, always added up in this order: a workgroup has a block of 32 x 32,
// a thread four sums of each part, which it reads side by side.  2 to 4 us: the launch, then 0.6 us for each MB of sums.
template <int TYPE>
__global__ __launch_bounds__(256) void mx4_join_kernel(const f32x4 *__restrict__ parts, int splits, int m, int n_out,
                                                       uint16_t *__restrict__ y, int tiles_m, int tiles_n)
{
    const int64_t next = (int64_t)tiles_m * tiles_n * 1024;
    const f32x4 *p = parts + (int64_t)blockIdx.x * 256 + threadIdx.x;
    f32x4 sum = p[0];
#pragma unroll 8
    for (int i = 1; i < splits; ++i) {
        const f32x4 v = p[i * next];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += v[e];
    }
    int tile_m, tile_n;
    xcd_tile<4>(blockIdx.x / 4, tiles_m, tiles_n, tile_m, tile_n);
    const int wave = blockIdx.x & 3, lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int row = tile_m * 64 + (wave >> 1) * 32 + (lane & 31), c = tile_n * 64 + (wave & 1) * 32 + q * 8 + (lane >> 5) * 4;
    if (row >= m || c >= n_out) return;
    uint16_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = Mx4Type<TYPE>::store(sum[e]);
    uint16_t *to = y + (int64_t)row * n_out + c;
    if ((reinterpret_cast<uintptr_t>(y) & 7) == 0 && (n_out & 3) == 0) {
        *reinterpret_cast<u32x2 *>(to) = u32x2{(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < n_out) to[e] = v[e];
    }
}

template <int TYPE, int TM, int TN, int NB>
hipError_t launch_tiles(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int m, int n_out,
                        int k, uint16_t *y, hipStream_t stream)
{
    constexpr int LDS = NB * Stages<64 * TM, 64 * TN>::SIZE;
    auto kernel = mx4_tile_kernel<TYPE, TM, TN, NB, false>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (e != hipSuccess) return e;
    const int tiles_m = (m + 64 * TM - 1) / (64 * TM), tiles_n = (n_out + 64 * TN - 1) / (64 * TN);
    kernel<<<(unsigned)(tiles_m * tiles_n), 256, LDS, stream>>>(xc, xs, wc, ws, m, n_out, k, y, tiles_m, tiles_n, 1);
    return hipGetLastError();
}

template <int TYPE>
hipError_t launch_parts(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int m, int n_out,
                        int k, int splits, f32x4 *parts, uint16_t *y, hipStream_t stream)
{
    constexpr int LDS = 4 * Stages<64, 64>::SIZE;
    auto kernel = mx4_tile_kernel<TYPE, 1, 1, 4, true>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (e != hipSuccess) return e;
    const int tiles_m = (m + 63) / 64, tiles_n = (n_out + 63) / 64, tiles = tiles_m * tiles_n;
    kernel<<<(unsigned)(tiles * splits), 256, LDS, stream>>>(xc, xs, wc, ws, m, n_out, k, parts, tiles_m, tiles_n, splits);
    mx4_join_kernel<TYPE><<<(unsigned)(tiles * 4), 256, 0, stream>>>(parts, splits, m, n_out, y, tiles_m, tiles_n);
    return hipGetLastError();
}

template <int TYPE, int MT, int X, int U>
hipError_t launch_rows_ahead(const void *x, const uint8_t *xs, int64_t stride, const uint8_t *wc, const uint8_t *ws, int m,
                       int n_out, int k, uint16_t *y, hipStream_t stream)
{
    constexpr int NW = kRowWaves, ROUND = U * NW;                                        // steps of one round of the waves
    const int steps = (k + 255) / 256, most = std::max(1, 80 * 1024 / (m * 136) / ROUND) * ROUND;
    const int chunk = std::min(most, steps);
    const int lds = std::max(chunk * m * 136, NW * MT * 1024);
    auto kernel = mx4_rows_kernel<TYPE, MT, X, U>;
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    kernel<<<(unsigned)((n_out + 15) / 16), 64 * NW, lds, stream>>>(x, xs, stride, wc, ws, m, n_out, k, chunk, y);
    return hipGetLastError();
}

// Steps of W that a wave has on their way: four where it has that many (us with two and with four: 1 x 8192 x 8192 9.7 and 8.2,
// 16 x 8192 x 8192 12.7 and 11.3, 1 x 28672 x 8192 27.6 and 23.7; but 1 x 28672 x 4096 14.7 and 16.9), and at most 16 rows, with
// which x is in LDS in one piece or two.
int rows_ahead(int64_t m, int64_t k) { return m <= 16 && (k + 255) / 256 >= 4 * kRowWaves ? 4 : 2; }

template <int TYPE, int X>
hipError_t launch_rows(const void *x, const uint8_t *xs, int64_t stride, const uint8_t *wc, const uint8_t *ws, int m,
                       int n_out, int k, uint16_t *y, hipStream_t stream)
{
    if (m > 16) return launch_rows_ahead<TYPE, 2, X, 2>(x, xs, stride, wc, ws, m, n_out, k, y, stream);
    return rows_ahead(m, k) == 4 ? launch_rows_ahead<TYPE, 1, X, 4>(x, xs, stride, wc, ws, m, n_out, k, y, stream)
                                 : launch_rows_ahead<TYPE, 1, X, 2>(x, xs, stride, wc, ws, m, n_out, k, y, stream);
}

// How a product is run: by mx4_rows_kernel (tm == 0; at most 32 rows of x), or by tiles of 64 tm x 64 tn
// with nb stages in LDS, in `splits` parts of k that mx4_join_kernel adds up.
struct Plan {
    int tm, tn, nb, splits;
};

struct TileCost {
    Plan plan;
    int slots;                       // workgroups that the 256 CUs hold
    double start, alone, full;       // us: a tile's beginning and end; a stage with few and with all CUs busy
};

// Measured at 790 sizes: 17 to 4096 rows of x, n_out from 39 to 28672, k from 32 to 28672.  What these costs choose takes
// 0.7 % longer than the fastest of all, 26 % at most.  (us, the tiles below in order: 64 x 8192 x 8192 12.5, 15.3,
// 18.2, 26.9, 37.3, 42.3; 512 x 11008 x 4096 28.6, 22.6, 23.0, 19.7, 22.2, 25.8; 2048 x 11008 x 4096 94.8, 70.8, 67.0, 57.6, 53.0, 58.4;
// 8192^3 497, 398, 358, 306, 271, 244.)
constexpr TileCost kTiles[] = {
    {{1, 1, 4, 1}, 512, 3.3, 0.25, 0.55}, {{2, 1, 3, 1}, 512, 3.3, 0.28, 1.10}, {{2, 2, 3, 1}, 256, 3.3, 0.46, 0.69},
    {{2, 2, 2, 1}, 512, 3.0, 0.66, 1.30}, {{3, 4, 2, 1}, 256, 5.1, 1.30, 1.70}, {{4, 4, 2, 1}, 256, 7.1, 1.40, 2.00},
};

Plan plan_for(int64_t m, int64_t n_out, int64_t k)
{
    const int64_t stages = (k + 255) / 256;
    const double steps = (double)stages;
    const double memory = (double)(n_out * k) * 17 / 32 / 4.6e6;         // us, W at what a stream of it reaches
    Plan best = {};
    double least = 1e30;
    for (const TileCost &t : kTiles) {
        const int64_t bm = 64 * t.plan.tm, bn = 64 * t.plan.tn;
        const int64_t tiles = ((m + bm - 1) / bm) * ((n_out + bn - 1) / bn), full = tiles / t.slots, rest = tiles % t.slots;
        // CUs that share an L2 get into each other's way the more the more of them are busy
        const double part = (double)rest / t.slots;
        double cost = (double)full * (t.start + steps * t.full);
        if (rest) cost += t.start + steps * (t.alone + (t.full - t.alone) * part * part);
        cost = std::max(cost, memory);
        if (cost < least) {
            least = cost;
            best = t.plan;
        }
    }
    // Few tiles and a long k: one CU's loads bound a tile (64 x 64 x 256 elements in 0.26 us, whether two or seven stages are
    // on their way), so more of them take parts of k, at the cost of a second launch and of their sums' way through memory
    // (64 x 256 x 28672 32.0 us, in 12 parts 9.2; 64 x 8192 x 28672 41.7, in 2 parts 30.4; 64 x 4096 x 4096 7.6, in 2 parts 8.7).
    const int64_t tiles = ((m + 63) / 64) * ((n_out + 63) / 64);
    for (const int splits : {2, 3, 4, 6, 8, 12, 16}) {
        if (tiles * splits > 512 || splits > stages) break;
        const double part = (double)(tiles * splits) / 512;
        const double one = 3.3 + (double)((stages + splits - 1) / splits) * (0.25 + 0.30 * part * part);
        const double cost = std::max(one, memory) + 1.7 + 0.13 * splits + 4.3 * part;
        if (cost < least) {
            least = cost;
            best = {1, 1, 4, splits};
        }
    }
    // 16 rows of W a workgroup: most workgroups where there are few rows of x, but x comes once for each (1 x 4096 x
    // 4096 4.3 us against 7.0 in the smallest tiles, 16 x 1024 x 16384 11.3 and 18.1, 16 x 8192 x 8192 12.6 and 10.9).
    if (m <= 32) {
        const double groups = (double)((n_out + 15) / 16), rounds = std::max(1.0, groups / 512);
        const double slope = (0.065 + 0.0043 * (double)m) * (1.0 + 1.3 * std::min(1.0, groups / 512));
        const double cost = 2.5 + steps * slope * rounds + 0.8 * (rounds - 1.0);
        const double stream = rows_ahead(m, k) == 4 ? 0.87 * memory : memory;
        if (std::max(cost, stream) < least) best = {0, 0, 0, 1};
    }
    return best;
}

// x is quantized by the product's own workgroups where that costs less than a launch of its own (2 us): each does it for
// itself, 2.2 us for 16384 elements, and 512 at a time (1 x 8192 x 8192 9.2 us, 10.1 in two launches; 4 x 4096 x 4096 6.0 and
// 6.4; 8 x 4096 x 4096 8.0 and 6.8; 1 x 28672 x 8192 28.0 and 25.5).
bool quantizes_itself(const Plan &p, int64_t m, int64_t n_out, int64_t k)
{
    return p.tm == 0 && (double)(m * k) * std::max(1.0, (double)((n_out + 15) / 16) / 512) <= 16384;
}

// Bytes of the parts' sums.
int64_t part_bytes(const Plan &p, int64_t m, int64_t n_out)
{
    return p.splits > 1 ? p.splits * ((m + 63) / 64) * ((n_out + 63) / 64) * 16384 : 0;
}

template <int TYPE>
hipError_t launch(const Plan &p, const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int m,
                  int n_out, int k, void *parts, uint16_t *y, hipStream_t stream)
{
    if (p.splits > 1) return launch_parts<TYPE>(xc, xs, wc, ws, m, n_out, k, p.splits, (f32x4 *)parts, y, stream);
    if (p.tm == 0) return launch_rows<TYPE, -1>(xc, xs, 0, wc, ws, m, n_out, k, y, stream);
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
                         uint8_t *codes, uint8_t *scales, void *parts, uint16_t *y, hipStream_t stream)
{
    const Plan p = plan_for(m, n_out, k);
    if (quantizes_itself(p, m, n_out, k))
        return launch_rows<TYPE, TYPE>(x, nullptr, stride, wc, ws, m, n_out, k, y, stream);
    const hipError_t e = mx4_launch_quantize(x, TYPE, m, k, stride, codes, scales, stream);
    return e != hipSuccess ? e : launch<TYPE>(p, codes, scales, wc, ws, m, n_out, k, parts, y, stream);
}

}  // namespace

hipError_t mx4_launch_matmul(const uint8_t *xc, const uint8_t *xs, const uint8_t *wc, const uint8_t *ws, int64_t m,
                             int64_t n_out, int64_t k, int type, void *parts, void *y, hipStream_t stream)
{
    auto f = type == MX4_F16 ? launch<MX4_F16> : launch<MX4_BF16>;
    return f(plan_for(m, n_out, k), xc, xs, wc, ws, (int)m, (int)n_out, (int)k, parts, (uint16_t *)y, stream);
}

hipError_t mx4_launch_linear(const void *x, int type, int64_t stride, const uint8_t *wc, const uint8_t *ws, int64_t m,
                             int64_t n_out, int64_t k, uint8_t *codes, uint8_t *scales, void *parts, void *y, hipStream_t stream)
{
    auto f = type == MX4_F16 ? launch_linear<MX4_F16> : launch_linear<MX4_BF16>;
    return f(x, stride, wc, ws, (int)m, (int)n_out, (int)k, codes, scales, parts, (uint16_t *)y, stream);
}

Mx4Room mx4_room(int64_t m, int64_t n_out, int64_t k)
{
    const Plan p = plan_for(m, n_out, k);
    return {!quantizes_itself(p, m, n_out, k), part_bytes(p, m, n_out)};
}

void mx4_linear_name(int64_t m, int64_t n_out, int64_t k, int type, bool linear, char *name, int64_t name_len)
{
    const Plan p = plan_for(m, n_out, k);
    const bool self = linear && quantizes_itself(p, m, n_out, k);
    const char *first = "";
    if (linear && !self) first = type == MX4_F16 ? "mx4_quantize_kernel<0>, " : "mx4_quantize_kernel<1>, ";
    if (p.tm == 0) snprintf(name, (size_t)name_len, "%smx4_rows_kernel<%d, %d, %d, %d>", first, type, m <= 16 ? 1 : 2, self ? type : -1, rows_ahead(m, k));
    else if (p.splits > 1) snprintf(name, (size_t)name_len, "%smx4_tile_kernel<%d, 1, 1, 4, true>, mx4_join_kernel<%d>", first, type, type);
    else snprintf(name, (size_t)name_len, "%smx4_tile_kernel<%d, %d, %d, %d, false>", first, type, p.tm, p.tn, p.nb);
}
