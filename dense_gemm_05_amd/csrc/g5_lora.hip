// g5_lora.hip -- a shared projection with low-rank adapters of many requests:
//
//   C[m] = X[m] Wt^T + s_a (X[m] A_a^T) B_a^T,   a = idx[m]
//
// in two launches: the low-rank values v[m] = s_a X[m] A_a^T (R per row, in
// FP32 or as two bf16 parts) into the workspace, then the product, whose
// kernels add v B_a^T to the FP32 sums before they are rounded once.  An
// adapter adds 2 R (K + N) flops and R (K + N) elements to a row's 2 N K: both
// are small beside the projection, so the product is organized as without
// adapters (up to 16 rows and up to 128 the weights' stream, beyond the ring
// kernel's tiles) and the adapters join at its end, where rows of different
// adapters may stand next to each other in any order.
#include <hip/hip_runtime.h>

#include "g5_device.h"
#include "g5_kernels.h"
#include "g5_stream.h"

namespace g5 {

namespace {

constexpr int kShrinkWaves = 8;

// The adapter of row m, or -1: rows without one, past M, or whose index
// names no adapter.
__device__ __forceinline__ int lora_adapter(const LoraArgs &q, int64_t m, int64_t M)
{
    const int a = m < M ? q.idx[m] : -1;
    return a >= 0 && a < q.L ? a : -1;
}

// Two values as packed pairs of bf16, v = hi + lo to 2^-16 of it (an infinite
// value has no rest).
__device__ __forceinline__ void two_parts(float v0, float v1, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(v0, v1);
    lo = pack_bf16x2((hi & 0x7f80u) == 0x7f80u ? 0.f : v0 - bf16_lo(hi),
                     (hi & 0x7f800000u) == 0x7f800000u ? 0.f : v1 - bf16_hi(hi));
}

// Calls f(a, mine) for every adapter among 16 rows, in the order of their
// first rows; the lane's row is lane % 16 and its adapter `a_row`.
template <class F>
__device__ __forceinline__ void each_adapter(int a_row, F f)
{
    uint64_t todo = __ballot(a_row >= 0) & 0xffffull;
    for (int ordinal = 0; todo; ++ordinal) {
        const int a = __builtin_amdgcn_readlane(a_row, __builtin_ctzll(todo));
        f(a, a_row == a, ordinal);
        todo &= ~__ballot(a_row == a);
    }
}

}  // namespace

// v of 16 rows and 16 ranks over one of q.splits slices of K.  Workgroup
// (x: row block, y: rank group, z: adapter turn * splits + slice) takes every
// q.turns-th adapter of its rows; its eight waves divide the slice, their sums
// are added in wave order.  The adapter's rows of A are the matrix core's
// 16-row operand, X's rows the other: a row's sums are its own whatever
// stands in the other rows, and only rows of this adapter keep them.  Bound by
// what one CU reads (about 35 GB/s beside the latency): with K = 4096 in four
// slices 4.4 us for one row, 5.4 for 16 rows of 16 adapters and 6.7 for 77, in
// one slice 11 us for 1024 rows in runs; where rows of 64 adapters are mixed,
// so that a block's adapters follow each other, 34 us, and 118 at rank 64 (30
// in runs).  The ring kernels take one slice all the same:
// adding four at their ends cost them 10 us and saved 3 here.  Sixteen waves,
// or eight steps in flight, measured no faster.  WHOLE: K is a
// multiple of 8.
template <bool WHOLE>
__global__ void __launch_bounds__(kShrinkWaves * 64) k_lora_shrink(GemmArgs p, LoraArgs q)
{
    __shared__ f32x4 red[kShrinkWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    const int64_t m = (int64_t)blockIdx.x * 16 + li;
    const int r0 = blockIdx.y * 16, rank = r0 + li;
    const int slice = blockIdx.z % q.splits, turn = blockIdx.z / q.splits;
    const int a_row = lora_adapter(q, m, p.M);
    const int K = (int)p.K, steps = (K + 31) / 32;
    const int b0 = steps / q.splits * slice, b1 = slice + 1 < q.splits ? b0 + steps / q.splits : steps;
    const int s0 = b0 + (int)((unsigned)((b1 - b0) * wave) / kShrinkWaves);
    const int s1 = b0 + (int)((unsigned)((b1 - b0) * (wave + 1)) / kShrinkWaves);
    // (rows without an adapter and ranks past R read row 0: not kept)
    const uint16_t *xrow = (const uint16_t *)p.A + (a_row >= 0 ? m : 0) * p.lda;
    const int64_t ra = (int64_t)(rank < q.R ? rank : 0) * q.lda;
    each_adapter(a_row, [&](int a, bool mine, int ordinal) {
        if (ordinal % q.turns != turn) return;        // uniform over the workgroup
        const uint16_t *arow = q.A + (int64_t)a * q.strideA + ra;
        const float sc = q.scale ? q.scale[a] : 1.0f;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        constexpr int D = 4;
        for (int s = s0; s < s1; s += D) {
            u32x4 w[D], x[D];
#pragma unroll
            for (int j = 0; j < D; ++j) {
                const int col = (s + j) * 32 + g * 8;
                const bool in = s + j < s1 && col < K;
                w[j] = x[j] = u32x4{0u, 0u, 0u, 0u};
                if constexpr (WHOLE) {
                    // (a lane or step past the end reads the wave's first again)
                    const uint32_t at = in ? col : s0 * 32;
                    const u32x4 lw = load16(arow + at), lx = load16(xrow + at);
                    if (in) {
                        w[j] = lw;
                        x[j] = lx;
                    }
                } else if (in && col + 8 <= K) {
                    w[j] = load16(arow + col);
                    x[j] = load16(xrow + col);
                } else if (in) {
                    w[j] = load_part8(arow + col, K - col);
                    x[j] = load_part8(xrow + col, K - col);
                }
            }
#pragma unroll
            for (int j = 0; j < D; ++j)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[j]),
                                                              __builtin_bit_cast(bf16x8, x[j]), acc, 0, 0, 0);
        }
        __syncthreads();                              // (the adapter before has been read)
        red[wave][lane] = acc;
        __syncthreads();
        if (wave == 0 && mine && r0 + 4 * g < q.ranks) {
            f32x4 v = red[0][lane];
#pragma unroll
            for (int w2 = 1; w2 < kShrinkWaves; ++w2) v += red[w2][lane];
            v = v * sc;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (r0 + 4 * g + i >= q.R) v[i] = 0.f;
            if (q.V) {
                *(f32x4 *)(q.V + ((int64_t)slice * p.M + m) * q.ranks + r0 + 4 * g) = v;
            } else {
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) two_parts(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
                uint16_t *dst = q.V2 + m * 2 * q.ranks + r0 + 4 * g;
                *(u32x2 *)dst = u32x2{hi[0], hi[1]};
                *(u32x2 *)(dst + q.ranks) = u32x2{lo[0], lo[1]};
            }
        }
    });
}

namespace {

// Ranks 8 c .. 8 c + 7 of v[m], the slices added in order.
__device__ __forceinline__ void lora_v8(const LoraArgs &q, int64_t M, int64_t m, int c, f32x4 (&v)[2])
{
    const float *src = q.V + m * q.ranks + 8 * c;
    v[0] = *(const f32x4 *)src;
    v[1] = *(const f32x4 *)(src + 4);
    for (int s = 1; s < q.splits; ++s) {
        src += M * q.ranks;
        v[0] += *(const f32x4 *)src;
        v[1] += *(const f32x4 *)(src + 4);
    }
}

// Ranks 8 c .. 8 c + 7 of a row of B (zeros past R).  WHOLE: R is a multiple
// of 8.
template <bool WHOLE>
__device__ __forceinline__ u32x4 lora_b8(const LoraArgs &q, const uint16_t *row, int c)
{
    if (WHOLE || 8 * c + 8 <= q.R) return load16(row + 8 * c);
    return load_part8(row + 8 * c, (int)q.R - 8 * c);
}

// acc += v B^T for the rows and columns of a ring tile, 16 rows at a time.
//  - Sixteen rows of one adapter: matrix-core products of the adapter's rows
//    of B with the rows' values, which are stored as two bf16 parts behind
//    each other (v = hi + lo to 2^-16 of it): 2 R deep, both parts against
//    the same rows of B.  Rows of B stay in registers while the adapter stays.
//  - Any other sixteen rows: each lane forms its own outputs from its row's
//    values and its adapter's rows of B, R products each, with nothing shared
//    between the rows.  That grows with M N R: this kernel at N = 12288, K =
//    4096 with 64 adapters, mixed rows against runs of rows, 512 rows of rank
//    16 139 / 115 us, 1024 of rank 16 149 / 124, 512 of rank 64 590 / 202,
//    1024 of rank 64 1162 / 201.
template <class RT, int WGN, bool WHOLE>
__device__ __forceinline__ void lora_expand(const GemmArgs &p, const LoraArgs &q, typename RT::Acc &acc, int wave,
                                            int64_t m0, int64_t n0)
{
    const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
    const int64_t mw = m0 + (wave / WGN) * RT::TM, nw = n0 + (wave % WGN) * RT::TN;
    const int chunks = q.ranks / 8, depth = (2 * chunks + 3) / 4;     // 8-rank chunks; 32-deep steps
    int a_row[RT::FM], one[RT::FM];      // the lane's adapter; all sixteen rows' or -1
#pragma unroll
    for (int fm = 0; fm < RT::FM; ++fm) a_row[fm] = lora_adapter(q, mw + fm * 16 + li, p.M);
#pragma unroll
    for (int fm = 0; fm < RT::FM; ++fm) {
        const int a = __builtin_amdgcn_readfirstlane(a_row[fm]);
        one[fm] = __ballot(a_row[fm] != a) ? -1 : a;
    }
    for (int k = 0; k < depth; ++k) {
        const int kc = 4 * k + g, c = kc < chunks ? kc : kc - chunks;
        u32x4 x[RT::FM], b[RT::FN];
#pragma unroll
        for (int fm = 0; fm < RT::FM; ++fm) {
            x[fm] = u32x4{0u, 0u, 0u, 0u};
            if (one[fm] >= 0 && c < chunks)
                x[fm] = *(const u32x4 *)(q.V2 + (mw + fm * 16 + li) * 2 * q.ranks + 8 * kc);
        }
        int held = -1;
#pragma unroll
        for (int fm = 0; fm < RT::FM; ++fm) {
            if (one[fm] < 0) continue;
            if (one[fm] != held) {
                held = one[fm];
#pragma unroll
                for (int fn = 0; fn < RT::FN; ++fn) {
                    // (a column past N reads another, c past the chunks the
                    // first, which meets zeros of x: but not if it is NaN)
                    const int64_t n = nw + fn * 16 + li;
                    b[fn] = lora_b8<WHOLE>(q, q.B + (int64_t)held * q.strideB + (n < p.N ? n : 0) * q.ldb,
                                          c < chunks ? c : 0);
                    if (c >= chunks) b[fn] = u32x4{0u, 0u, 0u, 0u};
                }
            }
#pragma unroll
            for (int fn = 0; fn < RT::FN; ++fn)
                acc[fn][fm] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[fn]),
                                                                      __builtin_bit_cast(bf16x8, x[fm]), acc[fn][fm], 0, 0, 0);
        }
    }
#pragma unroll
    for (int fm = 0; fm < RT::FM; ++fm) {
        if (one[fm] >= 0 || a_row[fm] < 0) continue;
        // (addresses formed anew for each sixteen rows: kept for all of them
        // they would not fit beside the sums)
        int lane_g = g;
        asm volatile("" : "+v"(lane_g));
        const uint16_t *Ba = q.B + (int64_t)a_row[fm] * q.strideB;
        for (int c = 0; c < chunks; ++c) {
            const uint16_t *src = q.V2 + (mw + fm * 16 + li) * 2 * q.ranks + 8 * c;
            const u32x4 hi = *(const u32x4 *)src, lo = *(const u32x4 *)(src + q.ranks);
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(hi[i]) + bf16_lo(lo[i]);
                v[2 * i + 1] = bf16_hi(hi[i]) + bf16_hi(lo[i]);
            }
#pragma unroll
            for (int fn = 0; fn < RT::FN; ++fn) {
                u32x4 b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = nw + fn * 16 + 4 * lane_g + i;
                    b[i] = lora_b8<WHOLE>(q, Ba + (n < p.N ? n : 0) * q.ldb, c);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float d = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        d = __builtin_fmaf(v[2 * j], bf16_lo(b[i][j]), d);
                        d = __builtin_fmaf(v[2 * j + 1], bf16_hi(b[i][j]), d);
                    }
                    acc[fn][fm][i] += d;
                }
            }
        }
    }
}

}  // namespace

// The ring kernel on Bt (k_bf16_ms) with the adapters joined to its finished
// sums: 1024 x 12288 x 4096 with eight adapters of rank 16 in runs of rows
// 101 to 104 us (1.0 PFLOP/s), the product alone 102; 64 adapters of rank 16
// 124, of rank 64 201 (mixed rows: above).
template <int BM, int BN, int WGM, int WGN, bool MASKED, bool SK, bool WHOLE>
__global__ void __launch_bounds__(WGM *WGN * 64, BM == 128 ? 4 : 2) k_lora_ms(GemmArgs p, LoraArgs q)
{
    using R = RingTile<BM, BN, WGM, WGN, 4, 4, 16, MASKED, EPI_NONE, true, false, false>;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[R::LDS_BYTES / 2];
    const int64_t ntiles = p.tiles_m * p.tiles_n;
    const int64_t wg = SK ? (int64_t)blockIdx.x % ntiles : (int64_t)blockIdx.x;
    const int slice = SK ? (int)((int64_t)blockIdx.x / ntiles) : 0;
    const TileCoord tc = tile_map(wg, 1, p.tiles_m, p.tiles_n, p.group_m);
    const int64_t kbase = SK ? (int64_t)slice * p.kt_per * R::KS : 0;
    const int64_t Kpart = SK && slice < p.ksplit - 1 ? (int64_t)p.kt_per * R::KS : p.K - kbase;
    typename R::Acc acc;
    R::zero(acc);
    R::accumulate(p, smem, tc, kbase, Kpart, acc);
    if constexpr (SK) {
        if (!R::join_slices(p, wg, slice, acc)) return;
    }
    lora_expand<R, WGN, WHOLE>(p, q, acc, threadIdx.x >> 6, tc.tm * BM, tc.tn * BN);
    R::store(p, smem, tc, acc);
}

// M <= 16: the weights' stream on NW waves, and NX more waves that form v B^T
// of the workgroup's 16 RB columns meanwhile, an output at a time per thread
// (R products in rank order); the last pass adds both.  Bound by the stream:
// 12288 x 4096 for one row 22 to 24 us (4.2 to 4.5 TB/s), for 16 rows of 16
// adapters of rank 16 26 to 28 us (the product alone 22.0 and 24.2).  At rank
// 64 the values of v, which every output reads and adds up from K's slices
// anew, weigh more: 31 and 40 us.  One row takes a
// block of 16 weight rows per workgroup and four steps in flight, more rows
// three blocks, which share X (the product alone: 23.8 us, 29.2 with one).
template <int NW, int NX, int RB, int D>
__global__ void __launch_bounds__((NW + NX) * 64) k_lora_decode(GemmArgs p, LoraArgs q)
{
    __shared__ f32x4 red[NW][RB][64];
    __shared__ float extra[16][16 * RB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, li = lane & 15;
    const int64_t M = p.M, N = p.N;
    const int64_t n0 = (int64_t)blockIdx.x * 16 * RB;
    if (wave >= NW) {
        const int chunks = q.ranks / 8;
        for (int o = tid - NW * 64; o < (int)M * 16 * RB; o += NX * 64) {
            const int m = o / (16 * RB), c0 = o - m * (16 * RB);
            const int64_t n = n0 + c0;
            const int a = lora_adapter(q, m, M);
            float d = 0.f;
            if (a >= 0 && n < N) {
                const uint16_t *brow = q.B + (int64_t)a * q.strideB + n * q.ldb;
                for (int c = 0; c < chunks; ++c) {
                    const u32x4 b = lora_b8<false>(q, brow, c);
                    f32x4 v[2];
                    lora_v8(q, M, m, c, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d = __builtin_fmaf(v[i >> 1][2 * (i & 1)], bf16_lo(b[i]), d);
                        d = __builtin_fmaf(v[i >> 1][2 * (i & 1) + 1], bf16_hi(b[i]), d);
                    }
                }
            }
            extra[m][c0] = d;
        }
    } else {
        // (a block's rows lie within 2 GiB of its first; rows past N read a
        // row that is there, rows past M the first: not stored)
        const char *wbase[RB];
        uint32_t woff[RB];
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            const int64_t n = n0 + 16 * r < N ? n0 + 16 * r : n0;
            wbase[r] = (const char *)p.B + n * p.ldb * 2;
            woff[r] = (uint32_t)(n + li < N ? li : 0) * (uint32_t)(p.ldb * 2) + 16 * g;
        }
        auto tokens = [&](uint32_t (&off)[1], bool (&ok)[1]) {
            ok[0] = true;
            off[0] = (uint32_t)(li < M ? li : 0) * (uint32_t)(p.lda * 2) + x_lane<false>(g);
        };
        const int K = (int)p.K, steps = (K + kStep<false> - 1) / kStep<false>;
        RowStream<false, RB, 1, D> b;
        f32x4 acc[RB][1];
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r][0] = f32x4{0.f, 0.f, 0.f, 0.f};
        b.run(wbase, woff, (const char *)p.A, tokens, steps * wave / NW, steps * (wave + 1) / NW, K, g, acc);
#pragma unroll
        for (int r = 0; r < RB; ++r) red[wave][r][lane] = acc[r][0];
    }
    __syncthreads();
    if (tid < 64 * RB) {
        const int r = tid >> 6, t = tid & 63;
        f32x4 sum = red[0][r][t];
#pragma unroll
        for (int w2 = 1; w2 < NW; ++w2) sum += red[w2][r][t];
        const int m = t & 15, gg = t >> 4;
        if (m < M) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t n = n0 + 16 * r + 4 * gg + i;
                if (n >= N) continue;
                store_out(p, 0, m, n, sum[i] + extra[m][16 * r + 4 * gg + i]);
            }
        }
    }
}

// 16 < M <= 16 NC rows: the weight rows still go from HBM straight into the
// matrix core, once for all rows of X, whose part of a phase (2 ST steps of K)
// the workgroup stages in LDS.  A workgroup has 64 weight rows and one of
// q.slices slices of K: wave (kh, rw) multiplies its 16 rows rw with half kh of
// every phase.  The halves meet in LDS.  There v B^T is added, 8 ranks (32 for
// sixteen rows of X with one adapter, on the matrix core) to a slice in turn.
// The slices meet in the workspace as in RingTile::join_slices.  Bound by
// what a CU takes in, the weights and about as much of X again from L2, and by
// the latencies of the few phases that each workgroup has: 77 x 4104 x 4100 with 16
// adapters of rank 24 28 to 30 us (the weights alone 6.6 us at 5.1 TB/s),
// where the ring kernel took 33 and the copies of its unaligned rows 17 more.
template <int NC, int ST>
__global__ void __launch_bounds__(512, 4) k_lora_rows(GemmArgs p, LoraArgs q)
{
    constexpr int KC = 2 * ST * 64, LD = KC * 2 + 16;     // (16: rows start four banks apart)
    // a wave stages RP rows at a time, 16 bytes per lane
    constexpr int CPR = KC / 8, RP = CPR <= 32 ? 2 : 1, XT = 2 * NC / RP;
    static_assert(CPR * RP <= 64 && 2 * NC % RP == 0, "whole rows per wave");
    __shared__ __attribute__((aligned(16))) char xs[16 * NC * LD];
    __shared__ unsigned arrived;
    static_assert(16 * NC * LD >= 8 * NC * 64 * 16, "the halves' sums fit");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int g = lane >> 4, li = lane & 15, rw = wave & 3, kh = wave >> 2;
    const int wv = __builtin_amdgcn_readfirstlane(wave);
    const int xr = RP == 2 ? lane >> 5 : 0, xl = RP == 2 ? lane & 31 : lane, xc = xl < CPR ? xl : CPR - 1;
    const int block = (int)(blockIdx.x % (unsigned)p.tiles_n), slice = (int)(blockIdx.x / (unsigned)p.tiles_n);
    const int M = (int)p.M, K = (int)p.K;
    const int64_t nb = (int64_t)block * 64, nw = nb + 16 * rw;
    const int k0 = slice * q.per * KC, k1 = slice + 1 < q.slices ? k0 + q.per * KC : K;
    // (rows past N read the block's first, rows past M the first: not stored)
    const uint16_t *wrow = (const uint16_t *)p.B + (nw + li < p.N ? nw + li : nb) * p.ldb;
    f32x4 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k = k0; k < k1; k += KC) {
        u32x4 w[ST][2];
        const int kw = k + kh * ST * 64 + 8 * g;
        const uint16_t *xcol = (const uint16_t *)p.A + (k + 8 * xc);
        char *const to = xs + (wv * RP + xr) * LD + xc * 16;
        if (k + KC <= K) {
            u32x4 x[XT];
#pragma unroll
            for (int i = 0; i < XT; ++i) {
                const int row = (8 * i + wv) * RP + xr;
                x[i] = load16(xcol + (row < M ? row : 0) * p.lda);
            }
#pragma unroll
            for (int j = 0; j < ST; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) w[j][h] = load16(wrow + (kw + 64 * j + 32 * h));
            __syncthreads();             // (the phase before has been read)
#pragma unroll
            for (int i = 0; i < XT; ++i)
                if (CPR * RP == 64 || xl < CPR) *(u32x4 *)(to + 8 * i * RP * LD) = x[i];
        } else {
            const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < ST; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = kw + 64 * j + 32 * h, left = K - at;
                    w[j][h] = left >= 8 ? load16(wrow + at) : left > 0 ? load_part8(wrow + at, left) : zero;
                }
            __syncthreads();
            const int left = K - k - 8 * xc;
#pragma unroll 2
            for (int i = 0; i < XT; ++i) {
                const int row = (8 * i + wv) * RP + xr;
                const uint16_t *src = xcol + (row < M ? row : 0) * p.lda;
                const u32x4 x = left >= 8 ? load16(src) : left > 0 ? load_part8(src, left) : zero;
                if (CPR * RP == 64 || xl < CPR) *(u32x4 *)(to + 8 * i * RP * LD) = x;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ST; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const u32x4 xf = *(const u32x4 *)(xs + (16 * c + li) * LD + ((kh * ST + j) * 64 + 32 * h + 8 * g) * 2);
                    acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[j][h]),
                                                                     __builtin_bit_cast(bf16x8, xf), acc[c], 0, 0, 0);
                }
    }
    // the halves, each keeping every other 16 rows of X, and v B^T (kept in
    // LDS and not unrolled: the sums of all rows and the adapters' addresses
    // do not fit the registers together)
    f32x4 *const red = (f32x4 *)xs;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < NC; ++c) red[(wave * NC + c) * 64 + lane] = acc[c];
    __syncthreads();
    const int n_left = (int)(p.N - nw < 16 ? p.N - nw : 16);
#pragma unroll 1
    for (int c = kh; c < NC; c += 2) {
        f32x4 *const mine = red + (rw * NC + c) * 64 + lane;
        f32x4 sum = mine[0] + mine[4 * NC * 64];
        const int m = 16 * c + li, a = lora_adapter(q, m, M), one = __builtin_amdgcn_readfirstlane(a);
        // (a lane without an adapter reads one that is there and keeps nothing)
        const uint16_t *Ba = q.B + (int64_t)(a >= 0 ? a : 0) * q.strideB + (n_left > 0 ? nw : nb) * q.ldb;
        if (one >= 0 && !__ballot(m < M && a != one)) {
            // rows of one adapter: the matrix core, 32 ranks at a time, each
            // value as two bf16 parts
            const uint16_t *Bo = q.B + (int64_t)one * q.strideB + (n_left > 0 ? nw + (li < n_left ? li : 0) : nb) * q.ldb;
            for (int c8 = 4 * slice + g; c8 - g < q.ranks / 8; c8 += 4 * q.slices) {
                u32x4 b = {0u, 0u, 0u, 0u};
                uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
                if (c8 < q.ranks / 8) {
                    f32x4 v[2];
                    b = lora_b8<false>(q, Bo, c8);
                    lora_v8(q, M, m < M ? m : 0, c8, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) two_parts(v[i >> 1][2 * (i & 1)], v[i >> 1][2 * (i & 1) + 1], hi[i], lo[i]);
                }
                const u32x4 vh = {hi[0], hi[1], hi[2], hi[3]}, vl = {lo[0], lo[1], lo[2], lo[3]};
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, vh),
                                                              sum, 0, 0, 0);
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, vl),
                                                              sum, 0, 0, 0);
            }
        } else for (int c8 = slice; c8 < q.ranks / 8; c8 += q.slices) {
            u32x4 b[4];
            f32x4 v[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = lora_b8<false>(q, Ba + (4 * g + i < n_left ? 4 * g + i : 0) * q.ldb, c8);
            lora_v8(q, M, a >= 0 ? m : 0, c8, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float d = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d = __builtin_fmaf(v[j >> 1][2 * (j & 1)], bf16_lo(b[i][j]), d);
                    d = __builtin_fmaf(v[j >> 1][2 * (j & 1) + 1], bf16_hi(b[i][j]), d);
                }
                if (a >= 0) sum[i] += d;
            }
        }
        *mine = sum;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if ((c & 1) == kh) acc[c] = red[(rw * NC + c) * 64 + lane];
    if (q.slices > 1) {
        constexpr int TILE = 4 * NC * 64 * 16;
        char *const tile = (char *)q.part + (int64_t)block * q.slices * TILE;
        const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(tile + (int64_t)slice * TILE, 0, TILE, 0x00020000);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if ((c & 1) == kh)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[c]), wr,
                                                       ((rw * NC + c) * 64 + lane) * 16, 0, 16);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) arrived = __hip_atomic_fetch_add(q.count + block, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (arrived != (unsigned)(q.slices - 1)) return;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
        for (int s = 0; s < q.slices; ++s) {
            const __amdgpu_buffer_rsrc_t rr = __builtin_amdgcn_make_buffer_rsrc(tile + (int64_t)s * TILE, 0, TILE, 0x00020000);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if ((c & 1) == kh)
                    acc[c] += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                        rr, ((rw * NC + c) * 64 + lane) * 16, 0, 16));
        }
        if (tid == 0) __hip_atomic_store(q.count + block, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int m = 16 * c + li;
        if ((c & 1) != kh || m >= M) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = nw + 4 * g + i;
            if (n < p.N) store_out(p, 0, m, n, acc[c][i]);
        }
    }
}

hipError_t launch_lora_shrink(const GemmArgs &a, const LoraArgs &q, hipStream_t s)
{
    const dim3 g((unsigned)((a.M + 15) / 16), (unsigned)((q.ranks + 15) / 16), (unsigned)(q.turns * q.splits));
    if (a.K % 8 == 0)
        hipLaunchKernelGGL((k_lora_shrink<true>), g, dim3(kShrinkWaves * 64), 0, s, a, q);
    else
        hipLaunchKernelGGL((k_lora_shrink<false>), g, dim3(kShrinkWaves * 64), 0, s, a, q);
    return hipGetLastError();
}

template <int BM, int BN, int WGM, int WGN, bool MASKED, bool SK>
static hipError_t launch_lora_tile(const GemmArgs &a, const LoraArgs &q, int64_t grid, hipStream_t s)
{
    const dim3 g((unsigned)grid), b(WGM * WGN * 64);
    if (q.R % 8 == 0)
        hipLaunchKernelGGL((k_lora_ms<BM, BN, WGM, WGN, MASKED, SK, true>), g, b, 0, s, a, q);
    else
        hipLaunchKernelGGL((k_lora_ms<BM, BN, WGM, WGN, MASKED, SK, false>), g, b, 0, s, a, q);
    return hipGetLastError();
}

template <int BM, int BN, int WGM, int WGN>
static hipError_t launch_lora_ring(const GemmArgs &a, const LoraArgs &q, int variant, int64_t grid, hipStream_t s)
{
    if constexpr (BM == 128 && BN == 128) {
        if (a.ksplit > 1)
            return variant == 1 ? launch_lora_tile<BM, BN, WGM, WGN, false, true>(a, q, grid, s)
                                : launch_lora_tile<BM, BN, WGM, WGN, true, true>(a, q, grid, s);
    }
    return variant == 1 ? launch_lora_tile<BM, BN, WGM, WGN, false, false>(a, q, grid, s)
                        : launch_lora_tile<BM, BN, WGM, WGN, true, false>(a, q, grid, s);
}

hipError_t launch_lora(int config_id, const GemmArgs &a, const LoraArgs &q, int variant, int64_t grid, hipStream_t s)
{
    if (config_id == CFG_DECODE_NT && a.M > 16) {
        const dim3 gr((unsigned)(grid * q.slices)), bl(512);
        if (a.M <= 48) hipLaunchKernelGGL((k_lora_rows<3, kLoraSteps48>), gr, bl, 0, s, a, q);
        else if (a.M <= 80) hipLaunchKernelGGL((k_lora_rows<5, kLoraSteps80>), gr, bl, 0, s, a, q);
        else hipLaunchKernelGGL((k_lora_rows<8, kLoraSteps128>), gr, bl, 0, s, a, q);
        return hipGetLastError();
    }
    if (config_id == CFG_DECODE_NT) {
        // (fill_grid: three 16-row blocks of Wt per workgroup when M > 1)
        if (a.M > 1) hipLaunchKernelGGL((k_lora_decode<8, 4, 3, 2>), dim3((unsigned)grid), dim3(12 * 64), 0, s, a, q);
        else hipLaunchKernelGGL((k_lora_decode<8, 1, 1, 4>), dim3((unsigned)grid), dim3(9 * 64), 0, s, a, q);
        return hipGetLastError();
    }
    if (variant != 1 && variant != 2) return hipErrorInvalidValue;
    switch (config_id) {
    case CFG_BF16_256x192: return launch_lora_ring<256, 192, 2, 4>(a, q, variant, grid, s);
    case CFG_BF16_256x256: return launch_lora_ring<256, 256, 2, 4>(a, q, variant, grid, s);
    case CFG_BF16_128x128: return launch_lora_ring<128, 128, 4, 2>(a, q, variant, grid, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace g5
