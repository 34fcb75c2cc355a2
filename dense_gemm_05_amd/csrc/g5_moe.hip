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

// One token's routing, by one wave: lane l holds logits l, l + 64, ...
// (NV of them).  Each of the topk turns takes the largest remaining one, the
// lowest index among equals.
template <int NV>
__device__ __forceinline__ void route_token(const MoeArgs &a, int64_t t, int lane)
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
    float m = v[0];
#pragma unroll
    for (int j = 1; j < NV; ++j) m = fmaxf(m, v[j]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    float all = 0.f;
    if (!a.renormalize) {
#pragma unroll
        for (int j = 0; j < NV; ++j) all += v[j] > ninf ? expf(v[j] - m) : 0.f;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o, 64);
    }
    // lane s ends up with slot s
    float my = ninf, sum = 0.f;
    int my_id = -1;
    for (int s = 0; s < a.topk; ++s) {
        float best = v[0];
        int at = lane;
#pragma unroll
        for (int j = 1; j < NV; ++j)
            if (v[j] > best) {
                best = v[j];
                at = lane + 64 * j;
            }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const float ov = __shfl_xor(best, o, 64);
            const int oi = __shfl_xor(at, o, 64);
            if (ov > best || (ov == best && oi < at)) {
                best = ov;
                at = oi;
            }
        }
        if (!(best > ninf)) break;          // uniform: nothing left to choose
        if (lane == s) {
            my = best;
            my_id = at;
        }
        sum += expf(best - m);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at == lane + 64 * j) v[j] = ninf;
    }
    if (lane < a.topk) {
        const float gate = my_id >= 0 ? expf(my - m) / (a.renormalize ? sum : all) : 0.f;
        const int64_t p = t * a.topk + lane;
        __hip_atomic_store(a.w_ids + p, my_id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        a.w_gates[p] = gate;
        if (a.ids) a.ids[p] = my_id;
        if (a.gates) a.gates[p] = gate;
    }
}

// Routing: four waves, a token each.  The workgroup that arrives last then
// sorts the pairs (token * topk + slot) by expert, tokens in order: a bit per
// token and expert (OR-ed in any order), the experts' counts added up, and
// each pair's place is its expert's first place plus the bits below its own.
// Other workgroups' ids are read at the device's coherence point: written and
// read with device-scope accesses, the writes complete (the wait) before the
// arrival is counted.
constexpr int kMaskWords = kMoeMaxTokens / 32;
template <int NV>
__global__ void __launch_bounds__(256) k_moe_route(MoeArgs a)
{
    __shared__ unsigned mask[NV * 64][kMaskWords + 1];      // [expert][token / 32]; the last word: first place
    __shared__ unsigned arrived, sums[2][4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t < a.T) route_token<NV>(a, t, lane);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0) arrived = __hip_atomic_fetch_add(a.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = tid; i < NV * 64 * (kMaskWords + 1); i += 256) (&mask[0][0])[i] = 0u;
    __syncthreads();
    if (arrived != gridDim.x - 1) return;
    const int pairs = (int)a.T * a.topk;
    for (int p = tid; p < pairs; p += 256) {
        const int e = __hip_atomic_load(a.w_ids + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int tok = p / a.topk;
        if (e >= 0) atomicOr(&mask[e][tok >> 5], 1u << (tok & 31));
    }
    __syncthreads();
    // thread i sums experts NV / 4 i ..: pairs before, chosen experts before
    constexpr int EPT = NV * 64 / 256 > 0 ? NV * 64 / 256 : 1;
    unsigned cnt[EPT], pr = 0, ch = 0;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const int e = tid * EPT + j;
        cnt[j] = 0;
        if (e < NV * 64)
            for (int w = 0; w < kMaskWords; ++w) cnt[j] += __builtin_popcount(mask[e][w]);
        pr += cnt[j];
        ch += cnt[j] > 0;
    }
    unsigned pr_to = pr, ch_to = ch;         // inclusive over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const unsigned x = __shfl_up(pr_to, o, 64), y = __shfl_up(ch_to, o, 64);
        if (lane >= o) {
            pr_to += x;
            ch_to += y;
        }
    }
    if (lane == 63) {
        sums[0][wave] = pr_to;
        sums[1][wave] = ch_to;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        pr_to += sums[0][w];
        ch_to += sums[1][w];
    }
    unsigned first = pr_to - pr, ordinal = ch_to - ch;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
        const int e = tid * EPT + j;
        if (cnt[j] > 0) {
            a.items[ordinal] = MoeItem{e, (int)first, (int)cnt[j], 0};
            mask[e][kMaskWords] = first;
            ++ordinal;
            first += cnt[j];
        }
    }
    if (tid == 255) *a.chosen = (int)ch_to;
    __syncthreads();
    for (int p = tid; p < pairs; p += 256) {
        const int e = __hip_atomic_load(a.w_ids + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (e < 0) continue;
        const int tok = p / a.topk;
        unsigned at = mask[e][kMaskWords] + __builtin_popcount(mask[e][tok >> 5] & ((1u << (tok & 31)) - 1u));
        for (int w = 0; w < (tok >> 5); ++w) at += __builtin_popcount(mask[e][w]);
        a.pairs[at] = p;
    }
    if (tid == 0) __hip_atomic_store(a.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// acc[r][c] += rows of W block r (two blocks of 16 rows) times the token
// rows of chunk c (16 of them), over slice ks of KW of K.  wrow[r]: the
// lane's row (li) of block r; xrow[c]: the lane's row of chunk c in plane 0,
// plane 1 at + xplane (PL == 2).  A step is 64 bytes of every row: lane
// group g takes bytes 16 g .. 16 g + 15; D steps' loads are issued before the
// first is used.
template <bool CODES, int PL, int NC, int KW, bool VEC, bool MANY>
__device__ __forceinline__ void moe_stream(const void *const (&wrow)[2], const bool (&wok)[2], int align_w,
                                           const uint16_t *const (&xrow)[NC], const bool (&xok)[NC], int64_t xplane,
                                           int align_x, int64_t K, int ks, int g, f32x4 (&acc)[2][NC])
{
    constexpr int KS = CODES ? 64 : 32;
    constexpr int XQ = CODES ? 2 : 1;              // 8-element pieces of x per lane and step
    // as many steps as the kernel's registers hold (8 words of W and 4 per
    // piece of x each): moe_occupancy leaves 80 or 128 registers per lane
    constexpr int fit = (moe_occupancy(CODES, MANY) == 6 ? 48 : CODES ? 72 : 80) / (8 + 4 * NC * PL * XQ);
    constexpr int D = fit < 1 ? 1 : fit < 4 ? fit : 4;
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
    auto mma = [&](const u32x4 (&w)[2], const u32x4 (&x)[NC][PL][XQ]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
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
        u32x4 w[D][2], x[D][NC][PL][XQ];
#pragma unroll
        for (int j = 0; j < D; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) w[j][r] = load_w(r, s + j, s + j < s1);
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
        u32x4 w[2], x[NC][PL][XQ];
#pragma unroll
        for (int r = 0; r < 2; ++r)
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

// The KW slices' partial sums of chunk c, added in order by the first
// 64 * 8 / KW threads (64 per group of rows): s[r] is block r's sum of rows
// 4 (t % 64 / 16) .. + 3, token t % 16.
template <int NC, int KW>
__device__ __forceinline__ void moe_join(f32x4 (&red)[kMoeWaves][2][64], const f32x4 (&acc)[2][NC], int c,
                                         f32x4 (&s)[2])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();             // (the chunk before has been read)
    red[wave][0][lane] = acc[0][c];
    red[wave][1][lane] = acc[1][c];
    __syncthreads();
    if (wave < kMoeWaves / KW) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s[r] = red[wave * KW][r][lane];
#pragma unroll
            for (int w = 1; w < KW; ++w) s[r] += red[wave * KW + w][r][lane];
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
    moe_stream<CODES, 1, NC, kMoeWaves, VEC, MANY>(wrow, wok, a.align_gu, xrow, xok, 0, a.align_x, a.H, wave, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (base + 16 * c >= it.count) break;       // uniform
        f32x4 s[2];
        moe_join<NC, kMoeWaves>(red, acc, c, s);
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

constexpr int kDownK = 4;                                  // K slices of the down kernel's waves
constexpr int kDownCols = 32 * (kMoeWaves / kDownK);       // hidden columns per workgroup

// gate * (z Wd^T) of the workgroup's hidden columns for the expert's tokens,
// each pair's into its own row of `part`.
template <bool CODES, bool VEC, int NC, bool MANY>
__device__ __forceinline__ void moe_down_tokens(const MoeArgs &a, const MoeItem &it, int n0, int base,
                                                f32x4 (&red)[kMoeWaves][2][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    constexpr int EB = CODES ? 1 : 2;
    const char *W = (const char *)a.Wd + (int64_t)it.expert * a.strideD * EB;
    const int nw = n0 + 32 * (wave / kDownK);
    const bool wok[2] = {nw + li < a.H, nw + 16 + li < a.H};
    const void *const wrow[2] = {W + (wok[0] ? nw + li : 0) * a.ldd * EB, W + (wok[1] ? nw + 16 + li : 0) * a.ldd * EB};
    const uint16_t *zrow[NC];
    bool zok[NC];
    int pair[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        zok[c] = base + 16 * c + li < it.count;
        pair[c] = zok[c] ? a.pairs[it.first + base + 16 * c + li] : 0;
        zrow[c] = a.z + (int64_t)pair[c] * a.ldz;
    }
    f32x4 acc[2][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = acc[1][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_stream<CODES, 2, NC, kDownK, VEC, MANY>(wrow, wok, a.align_d, zrow, zok, a.zplane, 16, a.I, wave % kDownK, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (base + 16 * c >= it.count) break;       // uniform
        f32x4 s[2];
        moe_join<NC, kDownK>(red, acc, c, s);
        if (wave < kMoeWaves / kDownK && zok[c]) {
            const int64_t p = pair[c];
            const float gate = a.w_gates[p];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t n = n0 + 32 * wave + 16 * r + 4 * g + q;
                    if (n >= a.H) break;
                    const float sc = a.scale_d ? a.scale_d[(int64_t)it.expert * a.H + n] : 1.0f;
                    __hip_atomic_store(a.part + p * a.H + n, gate * (s[r][q] * sc), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
                }
        }
    }
}

// The last of a column strip's workgroups (one per chosen expert) adds each
// token's pairs in slot order: the parts are written and read at the device's
// coherence point, complete before the arrival is counted.
template <bool CODES, bool VEC, bool MANY>
__global__ void __launch_bounds__(kMoeThreads, moe_occupancy(CODES, MANY)) k_moe_down(MoeArgs a)
{
    __shared__ f32x4 red[kMoeWaves][2][64];
    __shared__ unsigned arrived;
    const int strips = (int)((a.H + kDownCols - 1) / kDownCols), ordinal = blockIdx.x / strips;
    const int strip = blockIdx.x - ordinal * strips, n0 = strip * kDownCols;
    const int chosen = *a.chosen;
    if (ordinal >= chosen && !(chosen == 0 && ordinal == 0)) return;
    if (chosen > 0) {
        const MoeItem it = a.items[ordinal];
        if constexpr (!MANY) {
            moe_down_tokens<CODES, VEC, 1, MANY>(a, it, n0, 0, red);
        } else {
            for (int base = 0; base < it.count; base += 32) {
                if (it.count - base <= 16) moe_down_tokens<CODES, VEC, 1, MANY>(a, it, n0, base, red);
                else moe_down_tokens<CODES, VEC, 2, MANY>(a, it, n0, base, red);
            }
        }
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        unsigned *c = a.counter + 1 + strip;
        if (threadIdx.x == 0) arrived = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (arrived != (unsigned)(chosen - 1)) return;
        if (threadIdx.x == 0) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    for (int o = threadIdx.x; o < (int)a.T * kDownCols; o += kMoeThreads) {
        const int64_t t = o / kDownCols, n = n0 + o % kDownCols;
        if (n >= a.H) continue;
        float y = 0.f;
#pragma unroll 4
        for (int s = 0; s < a.topk; ++s) {
            const int64_t p = t * a.topk + s;
            if (a.w_ids[p] >= 0)
                y += __hip_atomic_load(a.part + p * a.H + n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        if (a.out_f32) ((float *)a.Y)[t * a.ldy + n] = y;
        else ((uint16_t *)a.Y)[t * a.ldy + n] = (uint16_t)bf16_rne(y);
    }
}

}  // namespace

template <bool CODES, bool MANY>
static hipError_t launch_moe_weights(const MoeArgs &a, bool vec_gu, bool vec_d, hipStream_t s)
{
    const int64_t chosen = a.E < a.T * a.topk ? a.E : a.T * a.topk;   // experts at most
    const dim3 gg((unsigned)(chosen * ((a.I + 15) / 16))), gd((unsigned)(chosen * ((a.H + kDownCols - 1) / kDownCols)));
    const dim3 b(kMoeThreads);
    if (a.I > 0) {      // (no inner columns: the down kernel's sums are empty)
        if (vec_gu) hipLaunchKernelGGL((k_moe_gate_up<CODES, true, MANY>), gg, b, 0, s, a);
        else hipLaunchKernelGGL((k_moe_gate_up<CODES, false, MANY>), gg, b, 0, s, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (vec_d) hipLaunchKernelGGL((k_moe_down<CODES, true, MANY>), gd, b, 0, s, a);
    else hipLaunchKernelGGL((k_moe_down<CODES, false, MANY>), gd, b, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs &a, bool codes, bool vec_gu, bool vec_d, hipStream_t s)
{
    const dim3 rg((unsigned)((a.T + 3) / 4)), rb(256);
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
