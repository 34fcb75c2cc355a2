// g5_ping.h -- the main loop of large bf16 tiles: two groups of waves that
// take turns at the matrix cores and at memory.
#pragma once

#include <type_traits>

#include "g5_device.h"

namespace g5 {

// A 256 x 256 output tile by eight waves as 2 x 4 (wave tile 128 x 64), with
// RingTile's operand layouts (BT: B given as Bt [N, K]; AT: A given as At [K,
// M]), masks, accumulators and epilogues.
//
// K goes in stages of 64 through two LDS buffers.  A wave multiplies a stage
// in two phases of 32 MFMAs: A0, its upper 64 rows, by both halves B0 and B1 of
// its columns, then A1, its lower 64, by the same.  Before each phase it reads
// the fragments that the phase lacks (all but A1's, then A1's) and copies its
// part of the stages ahead.  The waves with the tile's upper rows and those
// with the lower rows, one of each on every SIMD, are kept half a phase apart
// by one more barrier at the start: while one feeds the matrix core, the other
// reads and copies.
//
// What a phase read is free behind the next barrier that both groups passed:
// the second phase of stage t copies A0, B0 and B1 of stage t + 2 and the first
// of stage t + 1 A1, each four phases before it is read.  With two copies per
// region and wave vmcnt(8) says at the end of either phase's copies that the
// next phase's regions have landed.
//
// LDS.  A K-contiguous operand's stage has rows of 128 bytes (a copy
// instruction moves eight whole lines), 16-byte chunks at chunk ^ (row & 7).
// One given across K is kept as its two regions, each 64 rows (k) of the 128
// columns that the waves' halves hold, chunks at chunk ^ swz_bn(k), and read by
// the transposing read.
//
// Against the ring's 32-deep stages, in which all waves read at once and then
// multiply at once: 4096 x 131072 x 4096 with the loss's epilogue 3150 us for
// 3550 (that epilogue's targets listed by lane since: 2918, 1507 TFLOP/s; the
// platform's library without any 3081).  Four phases of 16
// MFMAs 3215, raised wave priority around the MFMAs 1 to 2 % slower, copies
// ahead of the reads 3 % slower; workgroups that walk over several tiles and
// copy the next one's first stage under the epilogue 2 to 20 % slower.
template <bool BT, bool AT>
struct PingTile : RingTile<256, 256, 2, 4, 4, 4, 16, true, EPI_NONE, BT, false, AT> {
    using R = RingTile<256, 256, 2, 4, 4, 4, 16, true, EPI_NONE, BT, false, AT>;
    using typename R::Acc;
    static constexpr int KSTAGE = 64, BUF = 256 * 64, REGION = BUF / 2;      // elements
    static_assert(R::LDS_BYTES == 4 * BUF * 2, "two buffers of A and of B");

    // Rows of q.A (q.M of them) and columns of q.B (q.N) from the tile's first
    // on, K summed elements.  Rows start at any multiple of 4 bytes, which is
    // what the copies of 16 need (16000 rows in 16 groups by 1540 x 4098 240 us,
    // 424 with both operands copied to rows of 4104 first); those of an operand
    // across K have an even length: a copy past the last one's end brings zeros
    // for the dwords outside.  The LDS must be free on entry; it is free again
    // behind the caller's next barrier.
    __device__ static __forceinline__ void accumulate(const GemmArgs &p, uint16_t *smem, const int64_t K, Acc &acc)
    {
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 2, wn = wave & 3;
        const int g = lane >> 4, li = lane & 15;
        const char *A = (const char *)p.A, *B = (const char *)p.B;
        // (in whole dwords: the range check is per dword)
        auto even = [](int64_t n) { return (n + 1) & ~(int64_t)1; };
        const uint32_t a_bytes = (uint32_t)((AT ? (p.K - 1) * p.lda + even(p.M) : (p.M - 1) * p.lda + even(p.K)) * 2);
        const uint32_t b_bytes = (uint32_t)((BT ? (p.N - 1) * p.ldb + even(p.K) : (p.K - 1) * p.ldb + even(p.N)) * 2);

        // Copies: region r of a stage (0: A0, 1: B0, 2: B1, 3: A1) is 16 blocks
        // of 1 KiB, two for each wave: eight rows, or four of the region's k.
        constexpr auto of_a = [](int r) { return r == 0 || r == 3; };
        constexpr auto across = [](bool a) { return a ? AT : !BT; };
        auto place = [&](int r, int i) {       // of the block, in KiB of the stage's buffer
            const int b = 2 * wave + i, h = r >= 2;
            if (across(of_a(r))) return h * 16 + b;
            return of_a(r) ? (b >> 3) * 16 + h * 8 + (b & 7) : (b >> 2) * 8 + h * 4 + (b & 3);
        };
        uint32_t voff[4][2];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool a = of_a(r);
                const int64_t ld = a ? p.lda : p.ldb, limit = a ? p.M : p.N;
                if (across(a)) {
                    const int k = 4 * (2 * wave + i) + (lane >> 4), col = ((lane & 15) ^ swz_bn<128>(k)) * 8, h = r >= 2;
                    const int at = a ? (col >> 6) * 128 + h * 64 + (col & 63) : (col >> 5) * 64 + h * 32 + (col & 31);
                    voff[r][i] = (uint32_t)((k * ld + at) * 2);
                } else {
                    const int row = 8 * place(r, i) + (lane >> 3), chunk = (lane & 7) ^ (row & 7);
                    voff[r][i] = row >= limit ? 0x80000000u : (uint32_t)(row * ld * 2 + chunk * 16);
                }
            }
        // The last stage may be a partial one.  Of an operand across K the rows
        // from K on lie past its descriptor and arrive as zeros; one along K
        // brings what follows its rows, cleared in the fragments.
        const int KT = (int)((K + KSTAGE - 1) / KSTAGE), KF = AT && !BT ? KT : (int)(K / KSTAGE);
        // (a stage past the last copies the last one again, into a place that
        // is read no more)
        auto copy = [&](int r, int t) {
            const int kt = t < KT ? t : KT - 1;
            const bool a = of_a(r);
            const int64_t adv = (int64_t)kt * KSTAGE * 2 * (across(a) ? (a ? p.lda : p.ldb) : 1);
            const i32x4_t d = make_rsrc((a ? A : B) + adv, (a ? a_bytes : b_bytes) - (uint32_t)adv);
            uint16_t *to = smem + (a ? 0 : 2 * BUF) + (t & 1) * BUF;
#pragma unroll
            for (int i = 0; i < 2; ++i) dma<16>(d, voff[r][i], 0, to + place(r, i) * 512);
        };

        // Fragments: lane (g, li) holds K elements 8 g .. 8 g + 7 of row li, in
        // steps s of 32.  K-contiguous: chunk (4 s + g) ^ (row & 7) of the row.
        bf16x8 a0[4][2], a1[4][2], b0[2][2], b1[2][2];
        const int at = li * 64 + ((g ^ (li & 7)) * 8), at1 = at ^ 32;
        // Across K: two transposing reads of four k each.
        const int k0 = g * 8 + (li >> 2);
        int at_a[4], at_b[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) at_a[i] = k0 * 128 + (((wm * 8 + i * 2 + ((li & 3) >> 1)) ^ swz_bn<128>(k0)) * 8) + (li & 1) * 4;
#pragma unroll
        for (int j = 0; j < 2; ++j) at_b[j] = k0 * 128 + (((wn * 4 + j * 2 + ((li & 3) >> 1)) ^ swz_bn<128>(k0)) * 8) + (li & 1) * 4;
        auto transposed = [&](const uint16_t *s) {
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(G5_LDS(i16x4, s));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(G5_LDS(i16x4, s + 4 * 128));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        };
        auto read_a = [&](bf16x8 (&f)[4][2], int t, int h) {
            const uint16_t *s = smem + (t & 1) * BUF;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if constexpr (AT) f[i][q] = transposed(s + h * REGION + at_a[i] + q * 32 * 128);
                    else f[i][q] = __builtin_bit_cast(bf16x8, *(const u32x4 *)(s + (wm * 128 + h * 64) * 64 + (q ? at1 : at) + i * 1024));
                }
        };
        auto read_b = [&](bf16x8 (&f)[2][2], int t, int h) {
            const uint16_t *s = smem + (2 + (t & 1)) * BUF;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if constexpr (!BT) f[j][q] = transposed(s + h * REGION + at_b[j] + q * 32 * 128);
                    else f[j][q] = __builtin_bit_cast(bf16x8, *(const u32x4 *)(s + (wn * 64 + h * 32) * 64 + (q ? at1 : at) + j * 1024));
                }
        };
        auto mma = [&](const bf16x8 (&a)[4][2], const bf16x8 (&b)[2][2], int ha, int hb) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[hb * 2 + j][ha * 4 + i] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][q], a[i][q], acc[hb * 2 + j][ha * 4 + i], 0, 0, 0);
        };
        // of a lane's fragments the elements from the n-th of step 0 on
        auto clear = [&](auto &f, int n) {
            for (auto &row : f)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    u32x4 v = __builtin_bit_cast(u32x4, row[q]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int left = n - 32 * q - 2 * i;
                        v[i] = left >= 2 ? v[i] : left == 1 ? v[i] & 0xffffu : 0u;
                    }
                    row[q] = __builtin_bit_cast(bf16x8, v);
                }
        };
        auto barrier = [&]() {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        // the end of a phase's reads and copies: the reads are done, and the
        // copies of what the next phase (of either group) reads have landed
        auto landed = [&]() {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(8, 0));
            barrier();
        };

        if (KT > 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) copy(r, 0);
#pragma unroll
            for (int r = 0; r < 3; ++r) copy(r, 1);
            landed();
            if (wm == 1) barrier();
            auto stage = [&](int t, auto last) {
                constexpr bool LAST = decltype(last)::value;
                const int n = (int)(K - (int64_t)t * KSTAGE) - 8 * g;
                read_a(a0, t, 0);
                read_b(b0, t, 0);
                read_b(b1, t, 1);
                copy(3, t + 1);
                landed();
                if constexpr (LAST && !AT) clear(a0, n);
                if constexpr (LAST && BT) {
                    clear(b0, n);
                    clear(b1, n);
                }
                mma(a0, b0, 0, 0);
                mma(a0, b1, 0, 1);
                barrier();
                read_a(a1, t, 1);
                copy(0, t + 2);
                copy(1, t + 2);
                copy(2, t + 2);
                landed();
                if constexpr (LAST && !AT) clear(a1, n);
                mma(a1, b1, 1, 1);
                mma(a1, b0, 1, 0);
                barrier();
            };
            constexpr std::integral_constant<bool, false> whole{};
            constexpr std::integral_constant<bool, true> partial{};
            int t = 0;
            for (; t + 1 < KF; t += 2) {
                stage(t, whole);
                stage(t + 1, whole);
            }
            if (t < KF) stage(t++, whole);
            if constexpr (!AT || BT) {
                if (t < KT) stage(t, partial);
            }
            if (wm == 0) barrier();
        }
        __builtin_amdgcn_s_waitcnt(0);
    }
};

// The product of a tile whose operands' bases are at its own first row and
// column: 256 x 256 tiles by two groups of waves in turn, others on the ring.
template <class R, int BM, int BN, bool BT, bool AT>
__device__ __forceinline__ void multiply_tile(const GemmArgs &q, uint16_t *smem, int64_t K, typename R::Acc &acc)
{
    if constexpr (BM == 256 && BN == 256) PingTile<BT, AT>::accumulate(q, smem, K, acc);
    else R::accumulate(q, smem, TileCoord{0, 0, 0}, 0, K, acc);
}

typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));

// A tile's sums to q's rows of C from the tile's first on, of any alignment and
// length: staged through LDS as C's type, RP rows at a time, then 16 bytes per
// lane, which a store takes at any address, consecutive lanes on consecutive
// ones (16 groups' gradients of 1540 x 4101 from 16000 rows 380 us for 630 with
// rows not aligned stored from the registers, a loss's dW of 32003 x 1028 bf16
// from 1000 rows 98 for 111).
template <class R, int BM, int BN, int WGM, int WGN, typename TOut>
__device__ __forceinline__ void store_rows_as(const GemmArgs &q, uint16_t *smem, const typename R::Acc &acc)
{
    constexpr int ESZ = sizeof(TOut), PER = 16 / ESZ, PITCH = BN * ESZ + 16, CPR = BN / PER, NT = WGM * WGN * 64;
    constexpr int FITS = R::LDS_BYTES / PITCH, RP = FITS >= BM ? BM : FITS >= BM / 2 ? BM / 2 : BM / 4;
    static_assert(RP % 16 == 0 && RP * PITCH <= R::LDS_BYTES, "staging passes");
    using at_any = std::conditional_t<ESZ == 4, u32x4_at4, u32x4_at2>;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, wave = tid >> 6, wm = wave / WGN, wn = wave % WGN, g = lane >> 4, li = lane & 15;
    char *L = (char *)smem;
#pragma unroll
    for (int pass = 0; pass < BM / RP; ++pass) {
        __syncthreads();
#pragma unroll
        for (int fm = 0; fm < R::FM; ++fm) {
            const int row = wm * R::TM + fm * 16;
            if (row / RP != pass) continue;
#pragma unroll
            for (int fn = 0; fn < R::FN; ++fn) {
                char *to = L + (row - pass * RP + li) * PITCH + (wn * R::TN + fn * 16 + g * 4) * ESZ;
                const f32x4 v = acc[fn][fm];
                if constexpr (ESZ == 4) *(f32x4 *)to = v;
                else *(u32x2 *)to = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            }
        }
        __syncthreads();
        for (int i = tid; i < RP * CPR; i += NT) {
            const int r = i / CPR, c = i % CPR, left = (int)q.N - c * PER;
            if (pass * RP + r >= q.M || left <= 0) continue;
            const char *from = L + r * PITCH + c * 16;
            TOut *to = (TOut *)q.C + (pass * RP + r) * q.ldc + c * PER;
            if (left >= PER) {
                __builtin_nontemporal_store(*(const u32x4 *)from, (at_any *)to);      // C is written once
            } else {
                for (int j = 0; j < left; ++j) to[j] = ((const TOut *)from)[j];
            }
        }
    }
}
template <class R, int BM, int BN, int WGM, int WGN>
__device__ __forceinline__ void store_rows(const GemmArgs &q, uint16_t *smem, const typename R::Acc &acc)
{
    if (q.out_f32) store_rows_as<R, BM, BN, WGM, WGN, float>(q, smem, acc);
    else store_rows_as<R, BM, BN, WGM, WGN, uint16_t>(q, smem, acc);
}

}  // namespace g5
