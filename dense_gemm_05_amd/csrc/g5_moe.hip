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
        a.w_ids[p] = my_id;
        a.w_gates[p] = gate;
        if (a.ids) a.ids[p] = my_id;
        if (a.gates) a.gates[p] = gate;
    }
}

template <int NV>
__global__ void __launch_bounds__(64) k_moe_route(MoeArgs a)
{
    route_token<NV>(a, blockIdx.x, threadIdx.x);
}

// The tokens of the `ordinal`-th expert (by index) that any token chose:
// their pairs (token * topk + slot) in order into list[], their number into
// *count; returns the expert, or -1 when fewer experts were chosen.
struct MoeList {
    unsigned chosen[kMoeMaxExperts / 32];
    int pair[kMoeMaxTokens];
    int count;
};
__device__ __forceinline__ int moe_tokens(const MoeArgs &a, int ordinal, MoeList &l)
{
    const int tid = threadIdx.x, pairs = (int)a.T * a.topk;
    const int words = (int)((a.E + 31) / 32);
    for (int i = tid; i < words; i += kMoeThreads) l.chosen[i] = 0u;
    __syncthreads();
    for (int p = tid; p < pairs; p += kMoeThreads) {
        const int e = a.w_ids[p];
        if (e >= 0) atomicOr(&l.chosen[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    int e = -1, left = ordinal;
    for (int i = 0; i < words && e < 0; ++i) {
        unsigned w = l.chosen[i];
        const int n = __builtin_popcount(w);
        if (left >= n) {
            left -= n;
            continue;
        }
        for (; left > 0; --left) w &= w - 1;
        e = 32 * i + __builtin_ctz(w);
    }
    if (e < 0) return -1;       // the same in every thread
    if (tid < 64) {
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += 64) {
            const int p = p0 + tid;
            const bool mine = p < pairs && a.w_ids[p] == e;
            const uint64_t b = __ballot(mine);
            if (mine) l.pair[n + __builtin_popcountll(b & ((1ull << tid) - 1))] = p;
            n += __builtin_popcountll(b);
        }
        if (tid == 0) l.count = n;
    }
    __syncthreads();
    return e;
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

// acc[r][c] += rows of W block r (two blocks of 16 rows) times the token
// rows of chunk c (16 of them), over this wave's piece of K.  wrow[r]: the
// lane's row (li) of block r; xrow[c]: the lane's row of chunk c in plane 0,
// plane 1 at + xplane (PL == 2).  A step is 64 bytes of every row: lane
// group g takes bytes 16 g .. 16 g + 15.
template <bool CODES, int PL, int NC, bool VEC>
__device__ __forceinline__ void moe_stream(const void *const (&wrow)[2], const bool (&wok)[2], int align_w,
                                           const uint16_t *const (&xrow)[NC], const bool (&xok)[NC], int64_t xplane,
                                           int align_x, int64_t K, int wave, int g, f32x4 (&acc)[2][NC])
{
    constexpr int KS = CODES ? 64 : 32;
    constexpr int XQ = CODES ? 2 : 1;              // 8-element pieces of x per lane and step
    constexpr int D = NC == 1 ? 4 : NC == 2 ? 2 : 1;   // steps of W in flight
    const int64_t whole = K / KS;
    const int64_t s0 = whole * wave / kMoeWaves, s1 = whole * (wave + 1) / kMoeWaves;
    auto load_w = [&](int r, int64_t s) -> u32x4 {
        if (!wok[r]) return u32x4{0u, 0u, 0u, 0u};
        if constexpr (VEC) return __builtin_nontemporal_load((const u32x4 *)((const char *)wrow[r] + s * 64 + g * 16));
        if constexpr (CODES) return load_chunk16_u8((const uint8_t *)wrow[r], s * KS + g * 16, K, true, align_w);
        else return load_chunk8_bf16((const uint16_t *)wrow[r], s * KS + g * 8, K, true, align_w);
    };
    auto load_x = [&](int c, int pl, int q, int64_t s) -> u32x4 {
        const int64_t col = s * KS + (CODES ? g * 16 + q * 8 : g * 8);
        const uint16_t *row = xrow[c] + pl * xplane;
        if constexpr (VEC) return xok[c] ? *(const u32x4 *)(row + col) : u32x4{0u, 0u, 0u, 0u};
        return load_chunk8_bf16(row, col, K, xok[c], align_x);
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
    auto load_xs = [&](int64_t s, u32x4 (&x)[NC][PL][XQ]) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int pl = 0; pl < PL; ++pl)
#pragma unroll
                for (int q = 0; q < XQ; ++q) x[c][pl][q] = load_x(c, pl, q, s);
    };
    int64_t s = s0;
    for (; s + D <= s1; s += D) {
        u32x4 w[D][2], x[D][NC][PL][XQ];
#pragma unroll
        for (int j = 0; j < D; ++j)
#pragma unroll
            for (int r = 0; r < 2; ++r) w[j][r] = load_w(r, s + j);
#pragma unroll
        for (int j = 0; j < D; ++j) load_xs(s + j, x[j]);
#pragma unroll
        for (int j = 0; j < D; ++j) mma(w[j], x[j]);
    }
    for (; s < s1; ++s) {
        u32x4 x[NC][PL][XQ];
        const u32x4 w[2] = {load_w(0, s), load_w(1, s)};
        load_xs(s, x);
        mma(w, x);
    }
    if (wave == kMoeWaves - 1 && K % KS != 0) {
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

// The waves' partial sums of chunk c, added in wave order by the first 64
// threads: s[r] is block r's sum of rows 4 (t / 16) .. + 3, token t % 16.
template <int NC>
__device__ __forceinline__ void moe_join(f32x4 (&red)[kMoeWaves][2][64], const f32x4 (&acc)[2][NC], int c,
                                         f32x4 (&s)[2])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();             // (the chunk before has been read)
    red[wave][0][lane] = acc[0][c];
    red[wave][1][lane] = acc[1][c];
    __syncthreads();
    if (threadIdx.x < 64) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s[r] = red[0][r][lane];
#pragma unroll
            for (int w = 1; w < kMoeWaves; ++w) s[r] += red[w][r][lane];
        }
    }
}

// z of 16 inner columns: gate rows i0 .. i0 + 15 and the up rows of the same
// columns, for tokens base .. base + 16 NC - 1 of the expert's list.
template <bool CODES, bool VEC, int NC>
__device__ __forceinline__ void moe_gate_up_tokens(const MoeArgs &a, int e, int64_t i0, const MoeList &l, int base,
                                                   f32x4 (&red)[kMoeWaves][2][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    constexpr int EB = CODES ? 1 : 2;
    const char *W = (const char *)a.Wgu + (int64_t)e * a.strideGu * EB;
    const bool wok[2] = {i0 + li < a.I, i0 + li < a.I};
    const int64_t row = wok[0] ? i0 + li : 0;
    const void *const wrow[2] = {W + row * a.ldgu * EB, W + (a.I + row) * a.ldgu * EB};
    const uint16_t *xrow[NC];
    bool xok[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        xok[c] = base + 16 * c + li < l.count;
        xrow[c] = a.X + (xok[c] ? (int64_t)(l.pair[base + 16 * c + li] / a.topk) : 0) * a.ldx;
    }
    f32x4 acc[2][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = acc[1][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_stream<CODES, 1, NC, VEC>(wrow, wok, a.align_gu, xrow, xok, 0, a.align_x, a.H, wave, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (base + 16 * c >= l.count) break;       // uniform
        f32x4 s[2];
        moe_join<NC>(red, acc, c, s);
        const int tok = base + 16 * c + li;
        if (threadIdx.x < 64 && tok < l.count) {
            const int64_t p = l.pair[tok], i = i0 + 4 * g;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (i + q >= a.I) break;
                float gt = s[0][q], up = s[1][q];
                if (a.scale_gu) {
                    const float *sc = a.scale_gu + (int64_t)e * 2 * a.I;
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

template <bool CODES, bool VEC>
__global__ void __launch_bounds__(kMoeThreads) k_moe_gate_up(MoeArgs a)
{
    __shared__ MoeList l;
    __shared__ f32x4 red[kMoeWaves][2][64];
    const int strips = (int)((a.I + 15) / 16);
    const int e = moe_tokens(a, blockIdx.x / strips, l);
    if (e < 0) return;
    const int64_t i0 = (int64_t)(blockIdx.x % strips) * 16;
    for (int base = 0; base < l.count; base += 64) {
        const int n = l.count - base;
        if (n <= 16) moe_gate_up_tokens<CODES, VEC, 1>(a, e, i0, l, base, red);
        else if (n <= 32) moe_gate_up_tokens<CODES, VEC, 2>(a, e, i0, l, base, red);
        else moe_gate_up_tokens<CODES, VEC, 4>(a, e, i0, l, base, red);
    }
}

// gate * (z Wd^T) of 32 hidden columns for the expert's tokens, each pair's
// into its own row of `part`.
template <bool CODES, bool VEC, int NC>
__device__ __forceinline__ void moe_down_tokens(const MoeArgs &a, int e, int64_t n0, const MoeList &l, int base,
                                                f32x4 (&red)[kMoeWaves][2][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    constexpr int EB = CODES ? 1 : 2;
    const char *W = (const char *)a.Wd + (int64_t)e * a.strideD * EB;
    const bool wok[2] = {n0 + li < a.H, n0 + 16 + li < a.H};
    const void *const wrow[2] = {W + (wok[0] ? n0 + li : 0) * a.ldd * EB, W + (wok[1] ? n0 + 16 + li : 0) * a.ldd * EB};
    const uint16_t *zrow[NC];
    bool zok[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        zok[c] = base + 16 * c + li < l.count;
        zrow[c] = a.z + (zok[c] ? (int64_t)l.pair[base + 16 * c + li] : 0) * a.ldz;
    }
    f32x4 acc[2][NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[0][c] = acc[1][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    moe_stream<CODES, 2, NC, VEC>(wrow, wok, a.align_d, zrow, zok, a.zplane, 16, a.I, wave, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        if (base + 16 * c >= l.count) break;       // uniform
        f32x4 s[2];
        moe_join<NC>(red, acc, c, s);
        const int tok = base + 16 * c + li;
        if (threadIdx.x < 64 && tok < l.count) {
            const int64_t p = l.pair[tok];
            const float gate = a.w_gates[p];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t n = n0 + 16 * r + 4 * g + q;
                    if (n >= a.H) break;
                    const float sc = a.scale_d ? a.scale_d[(int64_t)e * a.H + n] : 1.0f;
                    a.part[p * a.H + n] = gate * (s[r][q] * sc);
                }
        }
    }
}

template <bool CODES, bool VEC>
__global__ void __launch_bounds__(kMoeThreads) k_moe_down(MoeArgs a)
{
    __shared__ MoeList l;
    __shared__ f32x4 red[kMoeWaves][2][64];
    const int strips = (int)((a.H + 31) / 32);
    const int e = moe_tokens(a, blockIdx.x / strips, l);
    if (e < 0) return;
    const int64_t n0 = (int64_t)(blockIdx.x % strips) * 32;
    for (int base = 0; base < l.count; base += 64) {
        const int n = l.count - base;
        if (n <= 16) moe_down_tokens<CODES, VEC, 1>(a, e, n0, l, base, red);
        else if (n <= 32) moe_down_tokens<CODES, VEC, 2>(a, e, n0, l, base, red);
        else moe_down_tokens<CODES, VEC, 4>(a, e, n0, l, base, red);
    }
}

// y[t][n]: the token's pairs added in slot order.
__global__ void __launch_bounds__(256) k_moe_combine(MoeArgs a)
{
    const int64_t t = blockIdx.y, n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n >= a.H) return;
    float y = 0.f;
    for (int s = 0; s < a.topk; ++s) {
        const int64_t p = t * a.topk + s;
        if (a.w_ids[p] >= 0) y += a.part[p * a.H + n];
    }
    if (a.out_f32) ((float *)a.Y)[t * a.ldy + n] = y;
    else ((uint16_t *)a.Y)[t * a.ldy + n] = (uint16_t)bf16_rne(y);
}

}  // namespace

hipError_t launch_moe(const MoeArgs &a, bool codes, bool vec_gu, bool vec_d, hipStream_t s)
{
    const int64_t chosen = a.E < a.T * a.topk ? a.E : a.T * a.topk;   // experts at most
    const dim3 rg((unsigned)a.T), rb(64), b(kMoeThreads);
    if (a.E <= 64) hipLaunchKernelGGL((k_moe_route<1>), rg, rb, 0, s, a);
    else if (a.E <= 128) hipLaunchKernelGGL((k_moe_route<2>), rg, rb, 0, s, a);
    else if (a.E <= 256) hipLaunchKernelGGL((k_moe_route<4>), rg, rb, 0, s, a);
    else hipLaunchKernelGGL((k_moe_route<kMoeMaxExperts / 64>), rg, rb, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.H == 0) return e;
    const dim3 gg((unsigned)(chosen * ((a.I + 15) / 16))), gd((unsigned)(chosen * ((a.H + 31) / 32)));
    if (a.I == 0) {
        // no inner columns: the down kernel's sums are empty
    } else if (codes) {
        if (vec_gu) hipLaunchKernelGGL((k_moe_gate_up<true, true>), gg, b, 0, s, a);
        else hipLaunchKernelGGL((k_moe_gate_up<true, false>), gg, b, 0, s, a);
    } else {
        if (vec_gu) hipLaunchKernelGGL((k_moe_gate_up<false, true>), gg, b, 0, s, a);
        else hipLaunchKernelGGL((k_moe_gate_up<false, false>), gg, b, 0, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (codes) {
        if (vec_d) hipLaunchKernelGGL((k_moe_down<true, true>), gd, b, 0, s, a);
        else hipLaunchKernelGGL((k_moe_down<true, false>), gd, b, 0, s, a);
    } else {
        if (vec_d) hipLaunchKernelGGL((k_moe_down<false, true>), gd, b, 0, s, a);
        else hipLaunchKernelGGL((k_moe_down<false, false>), gd, b, 0, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(k_moe_combine, dim3((unsigned)((a.H + 255) / 256), (unsigned)a.T), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace g5
