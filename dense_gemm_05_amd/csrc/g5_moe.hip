// g5_moe.hip -- a mixture-of-experts SwiGLU layer for a few tokens.
//
//   ids, gates: for each token the topk largest router logits (ties to the
//     lowest index; -inf and NaN never), gate_s = exp(l_s - max) / sum, the
//     sum over the chosen experts or over all
//   z_s = silu(x Wg_e^T) (.) (x Wu_e^T),  e = ids[s]
//   y   = sum_s gate_s (z_s Wd_e^T)
//
// With few tokens every weight of a chosen expert is used by a handful of
// rows: the layer is bound by reading those weights once from HBM (3 I H
// elements per expert), at 2 n flops per weight element for n tokens.  So
// the work is divided by weight rows: a workgroup owns 32 rows of one
// expert's matrices and streams them once, its waves on contiguous pieces of
// K, straight from HBM into the matrix core as the 16-row operand; the tokens
// that chose the expert are gathered as the other operand, 16 at a time.  Sums are FP32 throughout; z is kept as the sum of two bf16 (hi +
// lo, to 2^-16 of it), each multiplied on its own, so no rounding but the
// output's is seen in y.
#include <hip/hip_runtime.h>

#include "g5_device.h"
#include "g5_kernels.h"
#include "g5_stream.h"

namespace g5 {

namespace {

constexpr int kMoeWaves = 4;
constexpr int kMoeThreads = kMoeWaves * 64;

// A logit as a key that orders like it: 0 for -inf and NaN (never chosen),
// the same for both zeros.
__device__ __forceinline__ uint32_t logit_key(float x)
{
    if (!(x > -__builtin_inff())) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v)
{
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false);
    return o > v ? o : v;
}
// The largest of the wave's keys, in every lane: lane i takes the maximum
// with lanes i - 1, i - 2, i - 4, i - 8 of its row of 16, then with the rows
// before, so that lane 63 has all.
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v)
{
    v = max_dpp<0x111, 0xf>(v);
    v = max_dpp<0x112, 0xf>(v);
    v = max_dpp<0x114, 0xf>(v);
    v = max_dpp<0x118, 0xf>(v);
    v = max_dpp<0x142, 0xa>(v);
    v = max_dpp<0x143, 0xc>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// One token's routing, by one wave: lane l holds logits l, l + 64, ...
// (NV of them).  Each of the topk turns takes the largest remaining key, the
// lowest index among equals; lane s ends up with slot s: its expert (-1:
// none) and gate.
template <int NV>
__device__ __forceinline__ void route_token(const MoeArgs &a, const float (&x)[NV], int lane, int &id, float &gate)
{
    uint32_t v[NV], my = 0u;
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = logit_key(x[j]);
    float m = 0.f;
    id = -1;
    for (int s = 0; s < a.topk; ++s) {
        uint32_t best = v[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) best = v[j] > best ? v[j] : best;
        best = wave_max_key(best);
        if (best == 0u) break;              // nothing left to choose
        if (s == 0) m = key_logit(best);
        int at = -1;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint64_t eq = __ballot(v[j] == best);
            if (at < 0 && eq) at = 64 * j + __builtin_ctzll(eq);
        }
        if (lane == s) {
            my = best;
            id = at;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at == lane + 64 * j) v[j] = 0u;
    }
    const float p = id >= 0 ? expf(key_logit(my) - m) : 0.f;
    float all = p;
    if (!a.renormalize) {
        all = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) all += x[j] > -__builtin_inff() ? expf(x[j] - m) : 0.f;
    }
    const float sum = wave_sum(all);
    gate = id >= 0 ? p / sum : 0.f;
}

// Routing, by one workgroup: a wave per token (and every 16th after), then
// the pairs (token * topk + slot) sorted by expert, tokens in order: a bit
// per token and expert, the experts' counts added up, and each pair's place
// is its expert's first place plus the bits below its own.  The work items of
// the kernels below are runs of at most a.chunk pairs of one expert.  Latency
// only: of 64 experts 8 for one token 4.8 us, for 16 tokens 5.9, for 64 11.3.
template <int NV>
__global__ void __launch_bounds__(1024) k_moe_route(MoeArgs a)
{
    __shared__ unsigned long long mask[NV * 64];             // tokens of each expert
    __shared__ int first[NV * 64], ids[kMoeMaxPairs];
    __shared__ int sums[2][16];
    static_assert(kMoeMaxTokens == 64 && NV * 64 <= 1024, "a word of bits per expert, a thread per expert");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
    // the logits of all the wave's tokens first
    constexpr int PER = kMoeMaxTokens / 16;
    const int waves = threads / 64;          // T, or 16 for more tokens
    float v[PER][NV];
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int t = wave + i * waves, e = lane + 64 * j;
            v[i][j] = t < (int)a.T && e < (int)a.E ? a.logits[t * a.ldl + e] : -__builtin_inff();
        }
    for (int i = tid; i < NV * 64; i += threads) mask[i] = 0ull;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int t = wave + i * waves;
        if (t >= (int)a.T) break;
        int id;
        float gate;
        route_token<NV>(a, v[i], lane, id, gate);
        if (lane < a.topk) {
            const int p = t * a.topk + lane;
            ids[p] = id;
            a.w_ids[p] = id;
            a.w_gates[p] = gate;
            if (a.ids) a.ids[p] = id;
            if (a.gates) a.gates[p] = gate;
            if (id >= 0) atomicOr(&mask[id], 1ull << t);
        }
    }
    __syncthreads();
    // experts in turns of one per thread: pairs before, items before
    int pr0 = 0, ch0 = 0;
    for (int e0 = 0; e0 < NV * 64; e0 += threads) {
        const int e = e0 + tid;
        const int cnt = e < NV * 64 ? __builtin_popcountll(mask[e]) : 0;
        int pr = cnt, ch = (cnt + a.chunk - 1) / a.chunk;
        const int mine = ch;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(pr, o, 64), y = __shfl_up(ch, o, 64);
            if (lane >= o) {
                pr += x;
                ch += y;
            }
        }
        if (lane == 63) {
            sums[0][wave] = pr;
            sums[1][wave] = ch;
        }
        __syncthreads();
        int pr_all = pr0, ch_all = ch0;
        for (int w = 0; w < threads / 64; ++w) {
            if (w == wave) {
                pr += pr_all;
                ch += ch_all;
            }
            pr_all += sums[0][w];
            ch_all += sums[1][w];
        }
        if (cnt > 0) {
            first[e] = pr - cnt;
            for (int i = 0; i < mine; ++i) {
                const int left = cnt - i * a.chunk;
                a.items[ch - mine + i] = MoeItem{e, pr - cnt + i * a.chunk, left < a.chunk ? left : a.chunk, 0};
            }
        }
        pr0 = pr_all;
        ch0 = ch_all;
        __syncthreads();
    }
    if (tid == 0) *a.n_items = ch0;
    if (a.cols == 32)
        for (int i = tid; i < (int)(a.H + 31) / 32; i += threads) a.arrived[i] = 0u;
    for (int p = tid; p < (int)a.T * a.topk; p += threads) {
        const int e = ids[p];
        if (e >= 0) a.pairs[first[e] + __builtin_popcountll(mask[e] & ((1ull << (p / a.topk)) - 1))] = p;
    }
}

// (the same item in every lane)
__device__ __forceinline__ MoeItem uniform_item(const MoeItem &it)
{
    return MoeItem{__builtin_amdgcn_readfirstlane(it.expert), __builtin_amdgcn_readfirstlane(it.first),
                   __builtin_amdgcn_readfirstlane(it.count), 0};
}

// The waves' partial sums of chunk c, added in order by the first 64 threads:
// s[r] is block r's sum of rows 4 (t / 16) .. + 3, token t % 16.
template <int NC>
__device__ __forceinline__ void moe_join(f32x4 (&red)[kMoeWaves][2][64], const f32x4 (&acc)[2][NC], int c,
                                         f32x4 (&s)[2])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();             // (the chunk before has been read)
    red[wave][0][lane] = acc[0][c];
    red[wave][1][lane] = acc[1][c];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s[r] = red[0][r][lane];
#pragma unroll
            for (int w = 1; w < kMoeWaves; ++w) s[r] += red[w][r][lane];
        }
    }
}

// z of 16 inner columns for the tokens of one work item (at most 16 NC): gate
// rows i0 .. i0 + 15 and the up rows of the same columns.  Bound by the
// weights' stream from HBM: 8 experts of 2 x 1536 x 4096 for one token 36 us
// (5.6 TB/s), 56 experts for 16 tokens 242 to 250 us (5.6 to 5.8 TB/s; a copy
// reaches 5.1),
// 64 in codes for 64 tokens 172 to 182 us (4.4 to 4.7 TB/s: half the bytes per
// matrix-core step, and 32 tokens' x beside them).
template <bool CODES, int NC, int D>
__device__ __forceinline__ void moe_gate_up(const MoeArgs &a, const MoeItem &it, int i0,
                                            f32x4 (&red)[kMoeWaves][2][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    constexpr int EB = CODES ? 1 : 2, KS = kStep<CODES>;
    const char *W = (const char *)a.Wgu + (int64_t)it.expert * a.strideGu * EB;
    const bool wok = i0 + li < a.I;
    bool xok[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        xok[c] = 16 * c + li < it.count;
        pair[c] = xok[c] ? a.pairs[it.first + 16 * c + li] : 0;
    }
    f32x4 acc[2][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = acc[1][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int K = (int)a.H, steps = (K + KS - 1) / KS;
    const int s0 = steps * wave / kMoeWaves, s1 = steps * (wave + 1) / kMoeWaves;
    RowStream<CODES, 2, NC, D> b;
    // (a row past I repeats the block's first and is not stored; a block's
    // rows, and all token rows, lie within 2 GiB of their first)
    const char *const wbase[2] = {W + (int64_t)i0 * a.ldgu * EB, W + (a.I + i0) * a.ldgu * EB};
    const uint32_t off = (uint32_t)(wok ? li : 0) * (uint32_t)(a.ldgu * EB) + 16 * g, woff[2] = {off, off};
    auto tokens = [&](uint32_t (&xoff)[NC], bool (&ok)[NC]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            ok[c] = xok[c];
            xoff[c] = (uint32_t)(pair[c] / a.topk) * (uint32_t)(a.ldx * 2) + x_lane<CODES>(g);
        }
    };
    b.run(wbase, woff, (const char *)a.X, tokens, s0, s1, K, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (16 * c >= it.count) break;       // uniform
        f32x4 s[2];
        moe_join<NC>(red, acc, c, s);
        if (wave == 0 && xok[c]) {
            const int64_t p = pair[c], i = i0 + 4 * g;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (i + q >= a.I) break;
                float gt = s[0][q], up = s[1][q];
                if (a.scale_gu) {
                    const float *sc = a.scale_gu + (int64_t)it.expert * 2 * a.I;
                    gt *= sc[i + q];
                    up *= sc[a.I + i + q];
                }
                const float z = silu_f32(gt) * up;
                const uint32_t hi = bf16_rne(z);
                const float rest = z - __uint_as_float(hi << 16);
                a.z[p * a.ldz + i + q] = (uint16_t)hi;
                // (an infinite z has no rest)
                a.z[a.zplane + p * a.ldz + i + q] = (uint16_t)((hi & 0x7f80u) == 0x7f80u ? 0u : bf16_rne(rest));
            }
        }
    }
}

// (128 registers per lane: four workgroups per CU; MANY: items of up to 32
// tokens)
template <bool CODES, bool MANY>
__global__ void __launch_bounds__(kMoeThreads, 4) k_moe_gate_up(MoeArgs a)
{
    __shared__ f32x4 red[kMoeWaves][2][64];
    const int strips = (int)(a.I + 15) / 16, ordinal = blockIdx.x / strips;
    if (ordinal >= *a.n_items) return;
    const MoeItem it = uniform_item(a.items[ordinal]);
    const int i0 = (blockIdx.x - ordinal * strips) * 16;
    if (MANY && it.count > 16) moe_gate_up<CODES, 2, CODES ? 1 : 2>(a, it, i0, red);
    else moe_gate_up<CODES, 1, CODES ? 2 : 3>(a, it, i0, red);
}

// The down rows.  A workgroup owns `cols` (at most 16) hidden columns for
// every expert, so a token's slots meet in its LDS and nothing else is joined:
// its sixteen waves take pieces (work item, half of K) one after the other,
// the next free one each, and leave each pair's sums in the piece's own
// places.  The order in which pieces are taken does not matter: the slots of
// each half are added in order, then the halves, here and in the kernel for
// many tokens below, so a token's bits do not depend on the number of tokens.
// 8 experts of 4096 x 1536 for one token 22 to 24 us (4.2 to 4.6 TB/s), 56 for
// 16 tokens 128 to 131 us (5.4 to 5.5 TB/s).
constexpr int kDownWaves = 16, kDownSlices = 2, kMoeMaxItems = kMoeMaxPairs;
// A piece's products for its tokens, 8 to a block of the matrix core's 16
// columns: columns 0 .. 7 take z's hi parts, 8 .. 15 the lo parts, and the two
// sums are added at the end.
template <bool CODES, int RB, int NB, int D>
__device__ __forceinline__ void moe_down(const MoeArgs &a, const MoeItem &it, int from, int slice, int n0,
                                         const int *pairs, float (*part)[16 * RB])
{
    constexpr int EB = CODES ? 1 : 2, KS = kStep<CODES>;
    const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
    const int K = (int)a.I, steps = (K + KS - 1) / KS;
    const int s0 = steps * slice / kDownSlices, s1 = steps * (slice + 1) / kDownSlices;
    // (columns past the workgroup's or H repeat its first: not stored)
    const char *wbase[RB];
    uint32_t woff[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int n = n0 + 16 * r < (int)a.H ? n0 + 16 * r : n0;
        wbase[r] = (const char *)a.Wd + ((int64_t)it.expert * a.strideD + (int64_t)n * a.ldd) * EB;
        woff[r] = (uint32_t)(16 * r + li < a.cols && n + li < (int)a.H ? li : 0) * (uint32_t)(a.ldd * EB) + 16 * g;
    }
    bool zok[NB];
    int pair[NB];
    f32x4 acc[RB][NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) {
        const int i = from + 8 * c + (li & 7);
        zok[c] = i < it.count;
        pair[c] = zok[c] ? pairs[it.first + i] : 0;
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    RowStream<CODES, RB, NB, D> b;
    auto tokens = [&](uint32_t (&off)[NB], bool (&ok)[NB]) {
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            ok[c] = zok[c];
            off[c] = 2 * ((uint32_t)pair[c] * (uint32_t)a.ldz + (li < 8 ? 0u : (uint32_t)a.zplane)) + x_lane<CODES>(g);
        }
    };
    b.run(wbase, woff, (const char *)a.z, tokens, s0, s1, K, g, acc);
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            f32x4 v = acc[r][c];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], 8, 64);
            if (zok[c] && li < 8) *(f32x4 *)&part[pair[c]][16 * r + 4 * g] = v;
        }
}

// A piece has 16 tokens at most: a work item's SUB chunks are pieces of their
// own.
template <bool CODES, int SUB>
__global__ void __launch_bounds__(kDownWaves * 64, 4) k_moe_down(MoeArgs a)
{
    __shared__ __attribute__((aligned(16))) float part[kDownSlices][kMoeMaxPairs][16];
    __shared__ MoeItem items[kMoeMaxItems];
    __shared__ int pairs[kMoeMaxPairs], next;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n0 = blockIdx.x * a.cols;
    const int n_items = *a.n_items;
    for (int i = threadIdx.x; i < n_items; i += kDownWaves * 64) items[i] = a.items[i];
    for (int i = threadIdx.x; i < (int)a.T * a.topk; i += kDownWaves * 64) pairs[i] = a.pairs[i];
    if (threadIdx.x == 0) next = kDownWaves;
    __syncthreads();
    for (int piece = wave; piece < n_items * (kDownSlices * SUB);) {
        const MoeItem it = uniform_item(items[piece / (kDownSlices * SUB)]);
        const int slice = piece % kDownSlices, from = piece / kDownSlices % SUB * 16;
        if (it.count - from > 8) moe_down<CODES, 1, 2, CODES ? 2 : 3>(a, it, from, slice, n0, pairs, part[slice]);
        else if (it.count > from) moe_down<CODES, 1, 1, CODES ? 3 : 5>(a, it, from, slice, n0, pairs, part[slice]);
        int p = 0;
        if (lane == 0) p = atomicAdd(&next, 1);
        piece = __builtin_amdgcn_readfirstlane(p);
    }
    __syncthreads();
    // a thread per token and column
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15, n = n0 + c;
    if (t >= (int)a.T || c >= a.cols || n >= (int)a.H) return;
    float half[kDownSlices] = {0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.topk; ++s) {
        const int p = t * a.topk + s, e = a.w_ids[p];
        if (e < 0) continue;
        const float gate = a.w_gates[p], scale = a.scale_d ? a.scale_d[(int64_t)e * a.H + n] : 1.0f;
#pragma unroll
        for (int h = 0; h < kDownSlices; ++h) half[h] = __builtin_fmaf(gate, part[h][p][c] * scale, half[h]);
    }
    const float y = half[0] + half[1];
    if (a.out_f32) ((float *)a.Y)[t * a.ldy + n] = y;
    else ((uint16_t *)a.Y)[t * a.ldy + n] = (uint16_t)bf16_rne(y);
}

// The same for many tokens, where every workgroup's z (64 tokens, topk 8: 3 MB
// from L2) is as much as its weights, or twice with codes: a workgroup owns 32 columns and one half of K, so z is read half
// as often, and the two halves' outputs (FP32, the workgroup's own part of
// a.halves) are added by whichever comes second, the first half first.  Stores
// and loads of the halves go to the device's coherence point, and the wait and
// barrier retire the stores before the arrival is counted, as in
// RingTile::join_slices; the routing kernel sets the counts to zero.  64
// experts of 4096 x 1536 in codes for 64 tokens: 113 to 116 us (3.5 TB/s; 145
// with all of K in a workgroup, 103 with none of z's loads).
template <bool CODES>
__global__ void __launch_bounds__(kDownWaves * 64, 4) k_moe_down_halves(MoeArgs a)
{
    __shared__ __attribute__((aligned(16))) float part[kMoeMaxPairs][32];
    __shared__ MoeItem items[kMoeMaxItems];
    __shared__ int pairs[kMoeMaxPairs], next;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int block = blockIdx.x >> 1, half = blockIdx.x & 1, n0 = block * 32;
    const int n_items = *a.n_items;
    for (int i = threadIdx.x; i < n_items; i += kDownWaves * 64) items[i] = a.items[i];
    for (int i = threadIdx.x; i < (int)a.T * a.topk; i += kDownWaves * 64) pairs[i] = a.pairs[i];
    if (threadIdx.x == 0) next = kDownWaves;
    __syncthreads();
    for (int piece = wave; piece < n_items * 2;) {
        const MoeItem it = uniform_item(items[piece >> 1]);
        const int from = (piece & 1) * 16;
        if (it.count - from > 8) moe_down<CODES, 2, 2, CODES ? 1 : 2>(a, it, from, half, n0, pairs, part);
        else if (it.count > from) moe_down<CODES, 2, 1, 2>(a, it, from, half, n0, pairs, part);
        int p = 0;
        if (lane == 0) p = atomicAdd(&next, 1);
        piece = __builtin_amdgcn_readfirstlane(p);
    }
    __syncthreads();
    // a thread per column and two tokens
    constexpr int TILE = kMoeMaxTokens * 32;
    const int c = threadIdx.x & 31, n = n0 + c;
    float y[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = (threadIdx.x >> 5) + 32 * j;
        if (t >= (int)a.T || n >= (int)a.H) continue;
#pragma unroll 4
        for (int s = 0; s < a.topk; ++s) {
            const int p = t * a.topk + s, e = a.w_ids[p];
            if (e < 0) continue;
            float v = part[p][c];
            if (a.scale_d) v *= a.scale_d[(int64_t)e * a.H + n];
            y[j] = __builtin_fmaf(a.w_gates[p], v, y[j]);
        }
    }
    float *const mine = a.halves + (int64_t)blockIdx.x * TILE;
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(mine, 0, TILE * 4, 0x00020000);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[j]), wr, (int)(threadIdx.x + 1024 * j) * 4, 0, 16);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0)
        next = (int)__hip_atomic_fetch_add(a.arrived + block, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (next != 1) return;
    const __amdgpu_buffer_rsrc_t rr = __builtin_amdgcn_make_buffer_rsrc(a.halves + (int64_t)(blockIdx.x ^ 1) * TILE, 0,
                                                                        TILE * 4, 0x00020000);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = (threadIdx.x >> 5) + 32 * j;
        const float other = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rr, (int)(threadIdx.x + 1024 * j) * 4, 0, 16));
        const float v = half ? other + y[j] : y[j] + other;
        if (t >= (int)a.T || n >= (int)a.H) continue;
        if (a.out_f32) ((float *)a.Y)[t * a.ldy + n] = v;
        else ((uint16_t *)a.Y)[t * a.ldy + n] = (uint16_t)bf16_rne(v);
    }
}

}  // namespace

template <bool CODES, bool MANY>
static hipError_t launch_moe_weights(const MoeArgs &a, hipStream_t s)
{
    const dim3 gg((unsigned)(moe_items(a.T, a.E, a.topk) * ((a.I + 15) / 16)));
    const dim3 gd((unsigned)((a.H + a.cols - 1) / a.cols)), bg(kMoeThreads), bd(kDownWaves * 64);
    if (a.I > 0) {      // (no inner columns: the down kernel's sums are empty)
        hipLaunchKernelGGL((k_moe_gate_up<CODES, MANY>), gg, bg, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (MANY && a.cols == 32) hipLaunchKernelGGL((k_moe_down_halves<CODES>), dim3(2 * gd.x), bd, 0, s, a);
    else hipLaunchKernelGGL((k_moe_down<CODES, MANY ? 2 : 1>), gd, bd, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs &args, bool codes, hipStream_t s)
{
    MoeArgs a = args;
    a.chunk = moe_chunk(a.T);
    // hidden columns per workgroup of the down kernel: as many workgroups as
    // the 256 CUs, 16 columns at most and 4 at least
    a.cols = moe_halves(a.T, a.H) ? 32 : a.H > 2048 ? 16 : a.H > 1024 ? 8 : 4;
    const dim3 rg(1), rb((unsigned)(a.T < 16 ? a.T * 64 : 1024));
    if (a.E <= 64) hipLaunchKernelGGL((k_moe_route<1>), rg, rb, 0, s, a);
    else if (a.E <= 128) hipLaunchKernelGGL((k_moe_route<2>), rg, rb, 0, s, a);
    else if (a.E <= 256) hipLaunchKernelGGL((k_moe_route<4>), rg, rb, 0, s, a);
    else hipLaunchKernelGGL((k_moe_route<kMoeMaxExperts / 64>), rg, rb, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.H == 0) return e;
    if (a.chunk > 16)
        return codes ? launch_moe_weights<true, true>(a, s) : launch_moe_weights<false, true>(a, s);
    return codes ? launch_moe_weights<true, false>(a, s) : launch_moe_weights<false, false>(a, s);
}

}  // namespace g5
