// g5_stream.h -- weight rows streamed from HBM straight into the matrix core
// for a few token rows: the inner loop of the small-M kernels of the expert
// layer and of the projection with adapters.
#pragma once

#include "g5_device.h"

namespace g5 {

namespace {

// 16 bytes at any address: one load or store instruction (global memory takes
// any alignment; one that crosses a line is slower).
__device__ __forceinline__ u32x4 load16(const void *p)
{
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ void store16(void *p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// 8 bf16 (16 codes) of which the first `n` lie in the row, zeros behind them.
__device__ __forceinline__ u32x4 load_part8(const uint16_t *p, int n)
{
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? (uint32_t)p[i] : 0u;
    return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
}
__device__ __forceinline__ u32x4 load_part16(const uint8_t *p, int n)
{
    u32x4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = 4 * w + i < n ? (uint32_t)p[4 * w + i] : 0u;
        v[w] = e[0] | e[1] << 8 | e[2] << 16 | e[3] << 24;
    }
    return v;
}

// 16 E4M3FN codes as 16 bf16 values (each exact), in order.
__device__ __forceinline__ void codes16_to_bf16(u32x4 c, u32x4 &lo, u32x4 &hi)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], false);
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[i], true);
        u32x4 &d = i < 2 ? lo : hi;
        d[2 * (i & 1)] = pack_bf16x2(a[0], a[1]);
        d[2 * (i & 1) + 1] = pack_bf16x2(b[0], b[1]);
    }
}

// A step is a 128-byte line of every weight row, read in two pieces: lane
// group g (of four) takes bytes 16 g .. 16 g + 15 of each half.  The halves
// are loaded one right after the other and with ordinary loads: the bytes in
// flight exceed an XCD's L2, so of the lines whose second half is asked for
// later some are fetched again (the halves of D steps behind each other: 1.01
// to 1.09 times the bytes and 1.04 to 1.21 times the time in the expert
// layer's kernels), and loads marked non-temporal give them up sooner (16
// tokens, down rows: 170 us against 132).  Piece h meets the same elements of
// the token's row (8 of bf16, or 16 codes in two products).
template <bool CODES>
constexpr int kStep = CODES ? 128 : 64;       // elements
template <bool CODES>
constexpr int kPieces = CODES ? 4 : 2;        // 8-element pieces of a token row per lane and step

// Where piece q of a token's row starts in a step, for lane group g: bf16 has
// one per half, codes two.
template <bool CODES>
__device__ __forceinline__ int x_piece(int q, int g)
{
    return CODES ? 64 * (q >> 1) + 16 * g + 8 * (q & 1) : 32 * q + 8 * g;
}

// The lane group's part of that, in bytes.
template <bool CODES>
__device__ __forceinline__ uint32_t x_lane(int g)
{
    return (CODES ? 32u : 16u) * g;
}

// D steps of RB weight rows and of NC token rows in registers, and their
// products: step s in place j is multiplied and step s + D loaded
// over it, so D steps stay in flight.
template <bool CODES, int RB, int NC, int D>
struct RowStream {
    static constexpr int XP = kPieces<CODES>, KS = kStep<CODES>;
    u32x4 w[D][RB][2], x[D][NC][XP];

    // Whole step s: wave-uniform bases and the lane's byte offsets (its row
    // and 16 g).  A lane without a token leaves its x
    // as it is (its column of the product is never read).
    __device__ __forceinline__ void load_w(int j, const char *const (&wbase)[RB], const uint32_t (&woff)[RB], int s)
    {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[j][r][h] = load16((wbase[r] + (int64_t)s * 128 + 64 * h) + woff[r]);
    }
    __device__ __forceinline__ void load_x(int j, const char *xbase, const uint32_t (&xoff)[NC], const bool (&xok)[NC], int s)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (xok[c]) {
#pragma unroll
                for (int q = 0; q < XP; ++q)
                    x[j][c][q] = load16((xbase + ((int64_t)s * KS + x_piece<CODES>(q, 0)) * 2) + xoff[c]);
            }
    }

    // The last, partial step: zeros past K.
    __device__ __forceinline__ void load_tail(const char *const (&wbase)[RB], const uint32_t (&woff)[RB], const char *xbase,
                                              const uint32_t (&xoff)[NC], const bool (&xok)[NC], int s, int K, int g)
    {
        const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = s * 128 + 64 * h;                     // + 16 g, in woff
            const int left = K - (int)(at + 16 * g) / (CODES ? 1 : 2);
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                const char *p = wbase[r] + (woff[r] + at);
                w[0][r][h] = zero;
                if (left >= (CODES ? 16 : 8)) w[0][r][h] = load16(p);
                else if (left > 0) w[0][r][h] = CODES ? load_part16((const uint8_t *)p, left) : load_part8((const uint16_t *)p, left);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int q = 0; q < XP; ++q) {
                const int left = xok[c] ? K - s * KS - x_piece<CODES>(q, g) : 0;
                const char *p = xbase + (xoff[c] + 2 * (uint32_t)(s * KS + x_piece<CODES>(q, 0)));
                x[0][c][q] = zero;
                if (left >= 8) x[0][c][q] = load16(p);
                else if (left > 0) x[0][c][q] = load_part8((const uint16_t *)p, left);
            }
    }

    __device__ __forceinline__ void mma(int j, f32x4 (&acc)[RB][NC]) const
    {
#pragma unroll
        for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                u32x4 b[2] = {w[j][r][h], w[j][r][h]};
                if constexpr (CODES) codes16_to_bf16(w[j][r][h], b[0], b[1]);
#pragma unroll
                for (int q = 0; q < XP / 2; ++q)
#pragma unroll
                    for (int c = 0; c < NC; ++c)
                        acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, b[q]), __builtin_bit_cast(bf16x8, x[j][c][h * (XP / 2) + q]),
                            acc[r][c], 0, 0, 0);
            }
    }

    // Steps s0 .. s1 - 1 of K (the last may be partial).
    // tokens(xoff, xok) gives the lane's token rows, asked for when the first
    // weights are on their way.
    template <class F>
    __device__ __forceinline__ void run(const char *const (&wbase)[RB], const uint32_t (&woff)[RB], const char *xbase, F tokens, int s0,
                                        int s1, int K, int g, f32x4 (&acc)[RB][NC])
    {
        const int whole = K / KS, sw = s1 < whole ? s1 : whole;
        uint32_t xoff[NC];
        bool xok[NC];
        int s = s0;
        if (s + D <= sw) {
#pragma unroll
            for (int j = 0; j < D; ++j) load_w(j, wbase, woff, s + j);
            tokens(xoff, xok);
#pragma unroll
            for (int j = 0; j < D; ++j) load_x(j, xbase, xoff, xok, s + j);
            for (; s + 2 * D <= sw; s += D) {
#pragma unroll
                for (int j = 0; j < D; ++j) {
                    mma(j, acc);
                    load_w(j, wbase, woff, s + D + j);
                    load_x(j, xbase, xoff, xok, s + D + j);
                }
            }
            // the last whole group, and behind it the fewer than D steps left
#pragma unroll
            for (int j = 0; j < D; ++j) {
                mma(j, acc);
                if (j < D - 1 && s + D + j < sw) {
                    load_w(j, wbase, woff, s + D + j);
                    load_x(j, xbase, xoff, xok, s + D + j);
                }
            }
            s += D;
        } else {
            tokens(xoff, xok);
#pragma unroll
            for (int j = 0; j < D - 1; ++j)
                if (s + j < sw) {
                    load_w(j, wbase, woff, s + j);
                    load_x(j, xbase, xoff, xok, s + j);
                }
        }
#pragma unroll
        for (int j = 0; j < D - 1; ++j)
            if (s + j < sw) mma(j, acc);
        if (s0 < s1 && s1 > whole) {
            load_tail(wbase, woff, xbase, xoff, xok, whole, K, g);
            mma(0, acc);
        }
    }
};

}  // namespace

}  // namespace g5
