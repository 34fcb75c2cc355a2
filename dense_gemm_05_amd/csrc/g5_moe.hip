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
// expert's matrix and streams them once, its eight waves on contiguous
// pieces of K, straight from HBM into the matrix core as the 16-row operand;
// the tokens that chose the expert are gathered as the other operand, 16 at
// a time.  Sums are FP32 throughout; z is kept as the sum of two bf16 (hi +
// lo, to 2^-16 of it), each multiplied on its own, so no rounding but the
// output's is seen in y.
#include <hip/hip_runtime.h>

#include "g5_device.h"
#include "g5_kernels.h"

namespace g5 {

namespace {

constexpr int kMoeWaves = 8;
constexpr int kMoeThreads = kMoeWaves * 64;

template <int CTRL, int ROWS>
__device__ __forceinline__ float max_dpp(float v)
{
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, ROWS, 0xf,
                                                               false)));
}
// The largest of the wave's values, in every lane.
__device__ __forceinline__ float wave_max_dpp(float v)
{
    // lane i takes the maximum with lanes i - 1, i - 2, i - 4, i - 8 of its
    // row of 16, then with the rows before: lane 63 has all
    v = max_dpp<0x111, 0xf>(v);
    v = max_dpp<0x112, 0xf>(v);
    v = max_dpp<0x114, 0xf>(v);
    v = max_dpp<0x118, 0xf>(v);
    v = max_dpp<0x142, 0xa>(v);
    v = max_dpp<0x143, 0xc>(v);
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// One token's routing, by one wave: lane l holds logits l, l + 64, ...
// (NV of them).  Each of the topk turns takes the largest remaining one, the
// lowest index among equals; lane s ends up with slot s: its expert (-1:
// none) and gate.
template <int NV>
__device__ __forceinline__ void route_token(const MoeArgs &a, int64_t t, int lane, int &id, float &gate)
{
    const float *lg = a.logits + t * a.ldl;
    const float ninf = -__builtin_inff();
    float v[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane + 64 * j;
        const float x = e < a.E ? lg[e] : ninf;
        v[j] = x == x ? x : ninf;
    }
    float m = 0.f, all = 0.f, my = ninf;
    id = -1;
    for (int s = 0; s < a.topk; ++s) {
        float best = v[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) best = fmaxf(best, v[j]);
        best = wave_max_dpp(best);
        if (!(best > ninf)) break;          // nothing left to choose
        if (s == 0) {
            m = best;
            if (!a.renormalize) {
#pragma unroll
                for (int j = 0; j < NV; ++j) all += v[j] > ninf ? expf(v[j] - m) : 0.f;
            }
        }
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
            if (at == lane + 64 * j) v[j] = ninf;
    }
    const float p = id >= 0 ? expf(my - m) : 0.f;
    const float sum = wave_sum(a.renormalize ? p : all);
    gate = id >= 0 ? p / sum : 0.f;
}

// Routing, by one workgroup: a wave per token (and every 16th after), then
// the pairs (token * topk + slot) sorted by expert, tokens in order: a bit
// per token and expert, the experts' counts added up, and each pair's place
// is its expert's first place plus the bits below its own.
template <int NV>
__global__ void __launch_bounds__(1024) k_moe_route(MoeArgs a)
{
    __shared__ unsigned long long mask[NV * 64];             // tokens of each expert
    __shared__ int first[NV * 64], ids[kMoeMaxPairs];
    __shared__ int sums[2][16];
    static_assert(kMoeMaxTokens == 64 && NV * 64 <= 1024, "a word of bits per expert, a thread per expert");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, threads = blockDim.x;
    for (int i = tid; i < NV * 64; i += threads) mask[i] = 0ull;
    __syncthreads();
    for (int t = wave; t < (int)a.T; t += threads / 64) {
        int id;
        float gate;
        route_token<NV>(a, t, lane, id, gate);
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
    // experts in turns of one per thread: pairs before, chosen experts before
    int pr0 = 0, ch0 = 0;
    for (int e0 = 0; e0 < NV * 64; e0 += threads) {
        const int e = e0 + tid;
        const int cnt = e < NV * 64 ? __builtin_popcountll(mask[e]) : 0;
        int pr = cnt, ch = cnt > 0;
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
            a.items[ch - 1] = MoeItem{e, pr - cnt, cnt, 0};
        }
        pr0 = pr_all;
        ch0 = ch_all;
        __syncthreads();
    }
    if (tid == 0) *a.chosen = ch0;
    for (int p = tid; p < (int)a.T * a.topk; p += threads) {
        const int e = ids[p];
        if (e >= 0) a.pairs[first[e] + __builtin_popcountll(mask[e] & ((1ull << (p / a.topk)) - 1))] = p;
    }
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

// Waves per SIMD: three workgroups per CU for bf16 weights and at most 16
// tokens (80 registers), two for the others, whose larger steps need 128.
constexpr int moe_occupancy(bool codes, bool many) { return codes || many ? 4 : 6; }

// acc[r][c] += rows of W block r (RB blocks of 16 rows) times the token
// rows of chunk c (16 of them), over slice ks of KW of K.  wrow[r]: the
// lane's row (li) of block r; xrow[c]: the lane's row of chunk c in plane 0,
// plane 1 at + xplane (PL == 2).  A step is 64 bytes of every row: lane
// group g takes bytes 16 g .. 16 g + 15; D steps' loads are issued before the
// first is used.
template <bool CODES, int PL, int RB, int NC, int KW, int REGS, bool VEC>
__device__ __forceinline__ void moe_stream(const void *const (&wrow)[RB], const bool (&wok)[RB], int align_w,
                                           const uint16_t *const (&xrow)[NC], const bool (&xok)[NC], int64_t xplane,
                                           int align_x, int64_t K, int ks, int g, f32x4 (&acc)[RB][NC])
{
    constexpr int KS = CODES ? 64 : 32;
    constexpr int XQ = CODES ? 2 : 1;              // 8-element pieces of x per lane and step
    // as many steps as REGS registers hold (4 per piece of W and of x)
    constexpr int fit = REGS / (4 * RB + 4 * NC * PL * XQ);
    constexpr int D = fit < 1 ? 1 : fit < 8 ? fit : 8;
    const int whole = (int)(K / KS);
    const int s0 = whole * ks / KW, s1 = whole * (ks + 1) / KW;
    auto load_w = [&](int r, int s, bool in) -> u32x4 {
        if (!wok[r] || !in) return u32x4{0u, 0u, 0u, 0u};
        if constexpr (VEC) return __builtin_nontemporal_load((const u32x4 *)((const char *)wrow[r] + s * 64 + g * 16));
        if constexpr (CODES) return load_chunk16_u8((const uint8_t *)wrow[r], s * KS + g * 16, K, true, align_w);
        else return load_chunk8_bf16((const uint16_t *)wrow[r], s * KS + g * 8, K, true, align_w);
    };
    auto load_x = [&](int c, int pl, int q, int s, bool in) -> u32x4 {
        const int col = s * KS + (CODES ? g * 16 + q * 8 : g * 8);
        const uint16_t *row = xrow[c] + pl * xplane;
        if constexpr (VEC) return xok[c] && in ? *(const u32x4 *)(row + col) : u32x4{0u, 0u, 0u, 0u};
        return load_chunk8_bf16(row, col, K, xok[c] && in, align_x);
    };
    auto mma = [&](const u32x4 (&w)[RB], const u32x4 (&x)[NC][PL][XQ]) {
#pragma unroll
        for (int r = 0; r < RB; ++r) {
            u32x4 b[2] = {w[r], w[r]};
            if constexpr (CODES) codes16_to_bf16(w[r], b[0], b[1]);
#pragma unroll
            for (int q = 0; q < XQ; ++q)
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int pl = 0; pl < PL; ++pl)
                        acc[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b[q]),
                                                                            __builtin_bit_cast(bf16x8, x[c][pl][q]),
                                                                            acc[r][c], 0, 0, 0);
        }
    };
    for (int s = s0; s < s1; s += D) {
        u32x4 w[D][RB], x[D][NC][PL][XQ];
#pragma unroll
        for (int j = 0; j < D; ++j)
#pragma unroll
            for (int r = 0; r < RB; ++r) w[j][r] = load_w(r, s + j, s + j < s1);
#pragma unroll
        for (int j = 0; j < D; ++j)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                    for (int q = 0; q < XQ; ++q) x[j][c][pl][q] = load_x(c, pl, q, s + j, s + j < s1);
#pragma unroll
        for (int j = 0; j < D; ++j) mma(w[j], x[j]);
    }
    if (ks == KW - 1 && K % KS != 0) {
        // the rest of K, zero-filled past it
        u32x4 w[RB], x[NC][PL][XQ];
#pragma unroll
        for (int r = 0; r < RB; ++r)
            w[r] = CODES ? load_chunk16_u8((const uint8_t *)wrow[r], whole * KS + g * 16, K, wok[r], align_w)
                         : load_chunk8_bf16((const uint16_t *)wrow[r], whole * KS + g * 8, K, wok[r], align_w);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                for (int q = 0; q < XQ; ++q)
                    x[c][pl][q] = load_chunk8_bf16(xrow[c] + pl * xplane,
                                                   whole * KS + (CODES ? g * 16 + q * 8 : g * 8), K, xok[c], align_x);
        mma(w, x);
    }
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

// z of 16 inner columns: gate rows i0 .. i0 + 15 and the up rows of the same
// columns, for tokens base .. base + 16 NC - 1 of the expert's pairs.
template <bool CODES, bool VEC, int NC, bool MANY>
__device__ __forceinline__ void moe_gate_up_tokens(const MoeArgs &a, const MoeItem &it, int i0, int base,
                                                   f32x4 (&red)[kMoeWaves][2][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    constexpr int EB = CODES ? 1 : 2;
    const char *W = (const char *)a.Wgu + (int64_t)it.expert * a.strideGu * EB;
    const bool wok[2] = {i0 + li < a.I, i0 + li < a.I};
    const int64_t row = wok[0] ? i0 + li : 0;
    const void *const wrow[2] = {W + row * a.ldgu * EB, W + (a.I + row) * a.ldgu * EB};
    const uint16_t *xrow[NC];
    bool xok[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        xok[c] = base + 16 * c + li < it.count;
        pair[c] = xok[c] ? a.pairs[it.first + base + 16 * c + li] : 0;
        xrow[c] = a.X + (int64_t)(pair[c] / a.topk) * a.ldx;
    }
    f32x4 acc[2][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = acc[1][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_stream<CODES, 1, 2, NC, kMoeWaves, moe_occupancy(CODES, MANY) == 6 ? 48 : 64, VEC>(wrow, wok, a.align_gu, xrow, xok, 0, a.align_x, a.H, wave, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (base + 16 * c >= it.count) break;       // uniform
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

// MANY: an expert may have more than 16 tokens (T > 16), taken 32 at a time
// (the weights come from the caches after the first).
template <bool CODES, bool VEC, bool MANY>
__global__ void __launch_bounds__(kMoeThreads, moe_occupancy(CODES, MANY)) k_moe_gate_up(MoeArgs a)
{
    __shared__ f32x4 red[kMoeWaves][2][64];
    const int strips = (int)((a.I + 15) / 16), ordinal = blockIdx.x / strips;
    if (ordinal >= *a.chosen) return;
    const MoeItem it = a.items[ordinal];
    const int i0 = (blockIdx.x - ordinal * strips) * 16;
    if constexpr (!MANY) {
        moe_gate_up_tokens<CODES, VEC, 1, MANY>(a, it, i0, 0, red);
    } else {
        for (int base = 0; base < it.count; base += 32) {
            if (it.count - base <= 16) moe_gate_up_tokens<CODES, VEC, 1, MANY>(a, it, i0, base, red);
            else moe_gate_up_tokens<CODES, VEC, 2, MANY>(a, it, i0, base, red);
        }
    }
}

// The down rows.  A workgroup owns `cols` (at most 16) hidden columns for
// every expert, so a token's slots meet in its LDS and nothing else is joined:
// its sixteen waves take pieces (expert, half of K) one after the other, the
// next free one each, and leave each pair's sums in the piece's own places.
// The order in which pieces are taken does not matter; the halves and the
// slots are added in order.
constexpr int kDownWaves = 16, kDownSlices = 2;
template <bool CODES, bool VEC, int NC, bool MANY>
__device__ __forceinline__ void moe_down_tokens(const MoeArgs &a, const MoeItem &it, int n0, int slice, int base,
                                                float (&part)[kDownSlices][kMoeMaxPairs][16])
{
    const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
    constexpr int EB = CODES ? 1 : 2;
    const char *W = (const char *)a.Wd + (int64_t)it.expert * a.strideD * EB;
    const bool wok[1] = {li < a.cols && n0 + li < a.H};
    const void *const wrow[1] = {W + (wok[0] ? n0 + li : 0) * a.ldd * EB};
    const uint16_t *zrow[NC];
    bool zok[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        zok[c] = base + 16 * c + li < it.count;
        pair[c] = zok[c] ? a.pairs[it.first + base + 16 * c + li] : 0;
        zrow[c] = a.z + (int64_t)pair[c] * a.ldz;
    }
    f32x4 acc[1][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_stream<CODES, 2, 1, NC, kDownSlices, MANY ? 64 : CODES ? 80 : 96, VEC>(wrow, wok, a.align_d, zrow, zok, a.zplane, 16, a.I,
                                                                  slice, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c)
        if (zok[c]) *(f32x4 *)&part[slice][pair[c]][4 * g] = acc[0][c];
}

template <bool CODES, bool VEC, bool MANY>
__global__ void __launch_bounds__(kDownWaves * 64, 4) k_moe_down(MoeArgs a)
{
    __shared__ __attribute__((aligned(16))) float part[kDownSlices][kMoeMaxPairs][16];
    __shared__ int next;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n0 = blockIdx.x * a.cols;
    if (threadIdx.x == 0) next = kDownWaves;
    __syncthreads();
    const int pieces = *a.chosen * kDownSlices;
    for (int piece = wave; piece < pieces;) {
        const MoeItem it = a.items[piece / kDownSlices];
        const int slice = piece % kDownSlices;
        if constexpr (!MANY) {
            moe_down_tokens<CODES, VEC, 1, MANY>(a, it, n0, slice, 0, part);
        } else {
            for (int base = 0; base < it.count; base += 32) {
                if (it.count - base <= 16) moe_down_tokens<CODES, VEC, 1, MANY>(a, it, n0, slice, base, part);
                else moe_down_tokens<CODES, VEC, 2, MANY>(a, it, n0, slice, base, part);
            }
        }
        int p = 0;
        if (lane == 0) p = atomicAdd(&next, 1);
        piece = __builtin_amdgcn_readfirstlane(p);
    }
    __syncthreads();
    // a thread per token and column
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15, n = n0 + c;
    if (t >= (int)a.T || c >= a.cols || n >= (int)a.H) return;
    float y = 0.f;
#pragma unroll 4
    for (int s = 0; s < a.topk; ++s) {
        const int p = t * a.topk + s, e = a.w_ids[p];
        if (e < 0) continue;
        float v = part[0][p][c] + part[1][p][c];
        if (a.scale_d) v *= a.scale_d[(int64_t)e * a.H + n];
        y = __builtin_fmaf(a.w_gates[p], v, y);
    }
    if (a.out_f32) ((float *)a.Y)[t * a.ldy + n] = y;
    else ((uint16_t *)a.Y)[t * a.ldy + n] = (uint16_t)bf16_rne(y);
}

}  // namespace

template <bool CODES, bool MANY>
static hipError_t launch_moe_weights(const MoeArgs &a, bool vec_gu, bool vec_d, hipStream_t s)
{
    const int64_t chosen = a.E < a.T * a.topk ? a.E : a.T * a.topk;   // experts at most
    const dim3 gg((unsigned)(chosen * ((a.I + 15) / 16))), gd((unsigned)((a.H + a.cols - 1) / a.cols));
    const dim3 b(kMoeThreads), bd(kDownWaves * 64);
    if (a.I > 0) {      // (no inner columns: the down kernel's sums are empty)
        if (vec_gu) hipLaunchKernelGGL((k_moe_gate_up<CODES, true, MANY>), gg, b, 0, s, a);
        else hipLaunchKernelGGL((k_moe_gate_up<CODES, false, MANY>), gg, b, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (vec_d) hipLaunchKernelGGL((k_moe_down<CODES, true, MANY>), gd, bd, 0, s, a);
    else hipLaunchKernelGGL((k_moe_down<CODES, false, MANY>), gd, bd, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs &args, bool codes, bool vec_gu, bool vec_d, hipStream_t s)
{
    MoeArgs a = args;
    // hidden columns per workgroup of the down kernel: as many workgroups as
    // the 256 CUs, 16 columns at most and 4 at least
    a.cols = a.H > 2048 ? 16 : a.H > 1024 ? 8 : 4;
    const dim3 rg(1), rb((unsigned)(a.T < 16 ? a.T * 64 : 1024));
    if (a.E <= 64) hipLaunchKernelGGL((k_moe_route<1>), rg, rb, 0, s, a);
    else if (a.E <= 128) hipLaunchKernelGGL((k_moe_route<2>), rg, rb, 0, s, a);
    else if (a.E <= 256) hipLaunchKernelGGL((k_moe_route<4>), rg, rb, 0, s, a);
    else hipLaunchKernelGGL((k_moe_route<kMoeMaxExperts / 64>), rg, rb, 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.H == 0) return e;
    if (a.T > 16)
        return codes ? launch_moe_weights<true, true>(a, vec_gu, vec_d, s)
                     : launch_moe_weights<false, true>(a, vec_gu, vec_d, s);
    return codes ? launch_moe_weights<true, false>(a, vec_gu, vec_d, s)
                 : launch_moe_weights<false, false>(a, vec_gu, vec_d, s);
}

}  // namespace g5
