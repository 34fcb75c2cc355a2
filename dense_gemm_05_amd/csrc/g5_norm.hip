// g5_norm.hip -- the RMS norm that stands before a projection, with the
// residual's addition and a bf16 or E4M3FN output, and its gradient.
//
//   h = bf16(x + r)                       (or h = x without a residual)
//   rstd = 1 / sqrt(sum_j h_j^2 / cols + eps)
//   y_j = bf16(h_j rstd w_j)              (codes: y's row quantized as
//                                          k_quant_rows_e4m3 quantizes it)
//
// Sums and rstd are FP32.  h is rounded once because it is stored as the
// residual stream, and the norm reads what is stored; y is rounded to bf16
// before it is quantized, so the codes are those of the unfused program.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "g5_device.h"
#include "g5_kernels.h"
#include "g5_stream.h"

namespace g5 {

namespace {

// Chunks of 8 elements of rows of any alignment, one instruction each; WHOLE:
// cols is a multiple of 8.  Else the row's last chunk either ends with the row
// (`lap`: it repeats `dup` elements of the chunk before, which the row's sums
// leave out and which are stored twice with the same value), so that no load
// waits on a condition; or, for rows of less than a chunk and for a sum formed
// in place (whose elements may be read once only), it goes element by element.
struct NormCols {
    int64_t cols;
    bool lap;
    __device__ __forceinline__ int64_t at(int64_t col) const { return lap && col + 8 > cols ? cols - 8 : col; }
    __device__ __forceinline__ int dup(int64_t col) const { return lap && col + 8 > cols ? (int)(col + 8 - cols) : 0; }
};
// v without its first n elements.
__device__ __forceinline__ u32x4 drop_first(u32x4 v, int n)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] &= (2 * i < n ? 0u : 0xffffu) | (2 * i + 1 < n ? 0u : 0xffff0000u);
    return v;
}

template <bool WHOLE>
__device__ __forceinline__ u32x4 norm_load(const uint16_t *row, int64_t col, int64_t cols)
{
    if (WHOLE || col + 8 <= cols) return load16(row + col);
    return load_part8(row + col, (int)(cols - col));
}

template <bool WHOLE>
__device__ __forceinline__ void norm_store(uint16_t *row, int64_t col, int64_t cols, u32x4 v)
{
    if (WHOLE || col + 8 <= cols) {
        store16(row + col, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < cols) row[col + i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
    }
}

template <bool WHOLE>
__device__ __forceinline__ void norm_store_codes(uint8_t *row, int64_t col, int64_t cols, uint32_t w0, uint32_t w1)
{
    if (WHOLE || col + 8 <= cols) {
        const u32x2 v = {w0, w1};
        __builtin_memcpy(row + col, &v, 8);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < cols) row[col + i] = (uint8_t)((i < 4 ? w0 : w1) >> (8 * (i & 3)));
    }
}

__device__ __forceinline__ u32x4 add8_bf16(u32x4 x, u32x4 r)
{
    u32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack_bf16x2(bf16_lo(x[i]) + bf16_lo(r[i]), bf16_hi(x[i]) + bf16_hi(r[i]));
    return h;
}

__device__ __forceinline__ float sumsq8(float s, u32x4 h)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = __builtin_fmaf(bf16_lo(h[i]), bf16_lo(h[i]), s);
        s = __builtin_fmaf(bf16_hi(h[i]), bf16_hi(h[i]), s);
    }
    return s;
}

// h w rstd.  h takes rstd's power of two first, which is exact: then neither
// h 2^e, whatever the row's scale, nor its product with w (exact too, two bf16)
// leaves FP32's range unless y does, and y is rounded once in FP32 by rstd's
// mantissa.  (rstd 0, infinite or NaN: the mantissa is 1 or NaN.)
__device__ __forceinline__ u32x4 scale8(u32x4 h, float rstd, u32x4 w, bool has_w)
{
    const uint32_t bits = __float_as_uint(rstd);
    const float two_e = __uint_as_float(bits & 0x7f800000u);
    const float man = rstd != rstd ? rstd : __uint_as_float((bits & 0x007fffffu) | 0x3f800000u);
    u32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = has_w ? bf16_lo(h[i]) * two_e * bf16_lo(w[i]) * man : bf16_lo(h[i]) * rstd;
        const float hi = has_w ? bf16_hi(h[i]) * two_e * bf16_hi(w[i]) * man : bf16_hi(h[i]) * rstd;
        y[i] = pack_bf16x2(lo, hi);
    }
    return y;
}

__device__ __forceinline__ float absmax8(float m, u32x4 c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf16_lo(c[i])), fabsf(bf16_hi(c[i]))));
    return m;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

__device__ __forceinline__ float rstd_of(float ss, int64_t cols, float eps)
{
    return 1.0f / sqrtf(ss / (float)cols + eps);
}

}  // namespace

// Rows of up to WPR * NCH * 512 elements, held in registers between the
// passes: WPR waves share a row (part p holds its chunks p, p + WPR, ... of
// 512 elements), in workgroups of four waves, or eight for the longest.  Each
// wave sums in a fixed order (chunk, element, butterfly), the parts are
// added in order, so a row's result does not depend on the others.
// Bound by HBM (2 bytes per element each for x, r, h and y, one for codes):
// 16384 x 8192 with a residual 194 us, 5.5 TB/s, to codes 173 us, 5.4 TB/s;
// 1024 x 4096 to codes 9.5 us, 3.1 TB/s, of which about 3 us are the launch and
// one load's latency, all that 1 x 4096 takes (3.1 us).
template <int WPR, int NCH, bool CODES, bool WHOLE>
__global__ void __launch_bounds__(WPR > 4 ? WPR * 64 : 256, 4) k_rms_norm(NormArgs a)
{
    constexpr int ROWS = WPR > 4 ? 1 : 4 / WPR;              // per workgroup
    __shared__ float red[2][WPR > 4 ? WPR : 4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, part = wv % WPR, w0 = wv - part;
    const int64_t r = (int64_t)blockIdx.x * ROWS + wv / WPR;
    const bool r_ok = r < a.rows;
    if (WPR == 1 && !r_ok) return;        // a whole wave; nothing below joins waves
    const int64_t rr = r_ok ? r : 0;
    auto col_of = [&](int j) { return (int64_t)lane * 8 + (int64_t)(j * WPR + part) * 512; };
    const NormCols cc{a.cols, !WHOLE && a.cols >= 8 && (!a.H || (a.H != a.X && a.H != a.R))};
    auto at_of = [&](int j) { return WHOLE ? col_of(j) : cc.at(col_of(j)); };
    u32x4 h[NCH], w[NCH];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        h[j] = w[j] = u32x4{0u, 0u, 0u, 0u};
        if (r_ok && col_of(j) < a.cols) h[j] = norm_load<WHOLE>(a.X + rr * a.ldx, at_of(j), a.cols);
    }
    if (a.R) {
        u32x4 q[NCH];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            q[j] = u32x4{0u, 0u, 0u, 0u};
            if (r_ok && col_of(j) < a.cols) q[j] = norm_load<WHOLE>(a.R + rr * a.ldr, at_of(j), a.cols);
        }
#pragma unroll
        for (int j = 0; j < NCH; ++j) h[j] = add8_bf16(h[j], q[j]);
        if (a.H) {
#pragma unroll
            for (int j = 0; j < NCH; ++j)
                if (r_ok && col_of(j) < a.cols) norm_store<WHOLE>(a.H + rr * a.ldh, at_of(j), a.cols, h[j]);
        }
    }
    if (a.W) {
#pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (col_of(j) < a.cols) w[j] = norm_load<WHOLE>(a.W, at_of(j), a.cols);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) ss = sumsq8(ss, WHOLE ? h[j] : drop_first(h[j], cc.dup(col_of(j))));
    ss = wave_sum(ss);
    if constexpr (WPR > 1) {
        if (lane == 0) red[0][wv] = ss;
        __syncthreads();
        ss = red[0][w0];
#pragma unroll
        for (int k = 1; k < WPR; ++k) ss += red[0][w0 + k];
    }
    const float rstd = rstd_of(ss, a.cols, a.eps);
    if (a.rstd && r_ok && part == 0 && lane == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int j = 0; j < NCH; ++j) h[j] = scale8(h[j], rstd, w[j], a.W != nullptr);
    if constexpr (!CODES) {
#pragma unroll
        for (int j = 0; j < NCH; ++j)
            if (r_ok && col_of(j) < a.cols)
                norm_store<WHOLE>((uint16_t *)a.Y + rr * a.ldy, at_of(j), a.cols, h[j]);
    } else {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) amax = absmax8(amax, h[j]);
        amax = wave_max(amax);
        if constexpr (WPR > 1) {
            if (lane == 0) red[1][wv] = amax;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < WPR; ++k) amax = fmaxf(amax, red[1][w0 + k]);
        }
        if (!r_ok) return;
        if (part == 0 && lane == 0) a.scale[r] = amax / 448.0f;
        const E4m3Quot qz(amax);
        auto emit = [&](auto fast) {
            constexpr bool F = decltype(fast)::value;
#pragma unroll
            for (int j = 0; j < NCH; ++j)
                if (col_of(j) < a.cols)
                    norm_store_codes<WHOLE>((uint8_t *)a.Y + rr * a.ldy, at_of(j), a.cols,
                                          qz.code4<F>(h[j][0], h[j][1]), qz.code4<F>(h[j][2], h[j][3]));
        };
        if (qz.fast) emit(std::true_type{});
        else emit(std::false_type{});
    }
}

// Longer rows: a workgroup per row reads it again in each pass.  Each thread
// reads back only elements of H that it stored itself.
template <bool CODES>
__global__ void __launch_bounds__(256) k_rms_norm_long(NormArgs a)
{
    __shared__ float red[2][4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t r = blockIdx.x;
    const uint16_t *x = a.X + r * a.ldx, *q = a.R ? a.R + r * a.ldr : nullptr;
    uint16_t *hrow = a.R && a.H ? a.H + r * a.ldh : nullptr;
    float ss = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += 2048) {
        u32x4 h = norm_load<false>(x, c, a.cols);
        if (q) h = add8_bf16(h, norm_load<false>(q, c, a.cols));
        if (hrow) norm_store<false>(hrow, c, a.cols, h);
        ss = sumsq8(ss, h);
    }
    ss = wave_sum(ss);
    if (lane == 0) red[0][wv] = ss;
    __syncthreads();
    const float rstd = rstd_of(((red[0][0] + red[0][1]) + red[0][2]) + red[0][3], a.cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    auto y_of = [&](int64_t c) {
        u32x4 h;
        if (hrow) {
            h = norm_load<false>(hrow, c, a.cols);
        } else {
            h = norm_load<false>(x, c, a.cols);
            if (q) h = add8_bf16(h, norm_load<false>(q, c, a.cols));
        }
        const u32x4 w = a.W ? norm_load<false>(a.W, c, a.cols) : u32x4{0u, 0u, 0u, 0u};
        return scale8(h, rstd, w, a.W != nullptr);
    };
    if constexpr (!CODES) {
        for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += 2048)
            norm_store<false>((uint16_t *)a.Y + r * a.ldy, c, a.cols, y_of(c));
    } else {
        float amax = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += 2048) amax = absmax8(amax, y_of(c));
        amax = wave_max(amax);
        if (lane == 0) red[1][wv] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3]));
        if (threadIdx.x == 0) a.scale[r] = amax / 448.0f;
        const E4m3Quot qz(amax);
        for (int64_t c = (int64_t)threadIdx.x * 8; c < a.cols; c += 2048) {
            const u32x4 y = y_of(c);
            const uint32_t w0 = qz.fast ? qz.code4<true>(y[0], y[1]) : qz.code4<false>(y[0], y[1]);
            const uint32_t w1 = qz.fast ? qz.code4<true>(y[2], y[3]) : qz.code4<false>(y[2], y[3]);
            norm_store_codes<false>((uint8_t *)a.Y + r * a.ldy, c, a.cols, w0, w1);
        }
    }
}

template <int WPR, int NCH>
static hipError_t launch_norm_held(const NormArgs &a, bool codes, hipStream_t s)
{
    const bool whole = a.cols % 8 == 0;
    constexpr int ROWS = WPR > 4 ? 1 : 4 / WPR;
    const dim3 g((unsigned)((a.rows + ROWS - 1) / ROWS)), b(WPR > 4 ? WPR * 64 : 256);
    if (codes) {
        if (whole) hipLaunchKernelGGL((k_rms_norm<WPR, NCH, true, true>), g, b, 0, s, a);
        else hipLaunchKernelGGL((k_rms_norm<WPR, NCH, true, false>), g, b, 0, s, a);
    } else {
        if (whole) hipLaunchKernelGGL((k_rms_norm<WPR, NCH, false, true>), g, b, 0, s, a);
        else hipLaunchKernelGGL((k_rms_norm<WPR, NCH, false, false>), g, b, 0, s, a);
    }
    return hipGetLastError();
}

static hipError_t launch_norm_rows(const NormArgs &a, bool codes, hipStream_t s)
{
    // A wave for rows of up to 512 elements, four up to 8192 (past 1536 all
    // of them at work), then eight: 131072 x 512 takes 48 us with a wave per
    // row and 104 with four (three of them idle), 16384 x 4096 44 us with four
    // and 46 with eight.
    if (a.cols <= 512) return launch_norm_held<1, 1>(a, codes, s);
    if (a.cols <= 2048) return launch_norm_held<4, 1>(a, codes, s);
    if (a.cols <= 4096) return launch_norm_held<4, 2>(a, codes, s);
    if (a.cols <= 8192) return launch_norm_held<4, 4>(a, codes, s);
    if (a.cols <= 16384) return launch_norm_held<8, 4>(a, codes, s);
    if (codes) hipLaunchKernelGGL((k_rms_norm_long<true>), dim3((unsigned)a.rows), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_rms_norm_long<false>), dim3((unsigned)a.rows), dim3(256), 0, s, a);
    return hipGetLastError();
}

// (a launch holds fewer than 2^32 threads: 2^22 rows at a time)
hipError_t launch_rms_norm(const NormArgs &a, bool codes, hipStream_t s)
{
    constexpr int64_t kRows = (int64_t)1 << 22;
    for (int64_t r = 0; r < a.rows; r += kRows) {
        NormArgs b = a;
        b.X += r * a.ldx;
        if (b.R) b.R += r * a.ldr;
        if (b.H) b.H += r * a.ldh;
        b.Y = (char *)a.Y + r * a.ldy * (codes ? 1 : 2);
        if (b.scale) b.scale += r;
        if (b.rstd) b.rstd += r;
        b.rows = a.rows - r < kRows ? a.rows - r : kRows;
        const hipError_t e = launch_norm_rows(b, codes, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// ------------------------------------------------------------- the gradient
//
// With xh = h rstd and g = dy w, element by element:
//   dX_j = rstd (g_j - xh_j * sum_i(g_i xh_i) / cols) + dH_j
//   dW_j = sum over rows of dy_j xh_j
// One pass: workgroup b takes rows b, b + gridDim.x, ...; a thread owns the
// same columns in every row, so dW's sums over the workgroup's rows stay in
// its registers (NCH > 0) and go out once, as row b of `part`; a second
// kernel adds the workgroups' rows in order.  The next row is loaded while
// this one is summed.  Bound by HBM (8 bytes per element with dH): 8192 x 4096
// 46 us, 5.8 TB/s, and 4.9 us for dW; 1000 x 4100 without dH, whose rows start
// at any 8 bytes, 13.5 and 5.4 us, where a workgroup has two rows, the latency
// of its first load shows, and the 512 rows of `part` are 8.4 MB written and
// read again beside 24.6 MB of rows.
template <int NCH, int NW, bool WHOLE>
__global__ void __launch_bounds__(NW * 64) k_rms_norm_grad(NormGradArgs a)
{
    __shared__ float red[2][NW];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    auto col_of = [&](int j) { return (int64_t)threadIdx.x * 8 + (int64_t)j * (NW * 512); };
    const NormCols cc{a.cols, !WHOLE && a.cols >= 8};
    auto at_of = [&](int j) { return WHOLE ? col_of(j) : cc.at(col_of(j)); };
    u32x4 w[NCH];
    float dw[NCH][8];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
        w[j] = u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};   // ones
        if (a.W && col_of(j) < a.cols) w[j] = norm_load<WHOLE>(a.W, at_of(j), a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
    }
    struct Row {
        u32x4 dy[NCH], h[NCH], dh[NCH];
        float rstd;
    };
    auto load = [&](int64_t r, Row &w) {
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            w.dy[j] = w.h[j] = w.dh[j] = u32x4{0u, 0u, 0u, 0u};
            if (col_of(j) < a.cols) {
                w.dy[j] = norm_load<WHOLE>(a.dY + r * a.lddy, at_of(j), a.cols);
                w.h[j] = norm_load<WHOLE>(a.H + r * a.ldh, at_of(j), a.cols);
                if (a.dH) w.dh[j] = norm_load<WHOLE>(a.dH + r * a.lddh, at_of(j), a.cols);
            }
        }
        w.rstd = a.rstd[r];
    };
    // the next row's loads go out before this row is worked on
    Row cur, nxt;
    load(blockIdx.x, cur);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
        load(r + gridDim.x < a.rows ? r + gridDim.x : r, nxt);
        const u32x4 (&dy)[NCH] = cur.dy, (&h)[NCH] = cur.h, (&dh)[NCH] = cur.dh;
        const float rstd = cur.rstd;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            // (w too: zero times an infinite weight would be NaN)
            const u32x4 dk = WHOLE ? dy[j] : drop_first(dy[j], cc.dup(col_of(j)));
            const u32x4 wk = WHOLE ? w[j] : drop_first(w[j], cc.dup(col_of(j)));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float plo = bf16_lo(dk[i]) * (bf16_lo(h[j][i]) * rstd);
                const float phi = bf16_hi(dk[i]) * (bf16_hi(h[j][i]) * rstd);
                dw[j][2 * i] += plo;
                dw[j][2 * i + 1] += phi;
                dot = __builtin_fmaf(plo, bf16_lo(wk[i]), dot);
                dot = __builtin_fmaf(phi, bf16_hi(wk[i]), dot);
            }
        }
        dot = wave_sum(dot);
        // (two sets of slots in turn: one barrier per row)
        if (lane == 0) red[turn][wv] = dot;
        __syncthreads();
        float c = red[turn][0];
#pragma unroll
        for (int k = 1; k < NW; ++k) c += red[turn][k];
        c /= (float)a.cols;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            u32x4 dx;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float glo = bf16_lo(dy[j][i]) * bf16_lo(w[j][i]), ghi = bf16_hi(dy[j][i]) * bf16_hi(w[j][i]);
                const float xlo = bf16_lo(h[j][i]) * rstd, xhi = bf16_hi(h[j][i]) * rstd;
                dx[i] = pack_bf16x2(__builtin_fmaf(rstd, glo - xlo * c, bf16_lo(dh[j][i])),
                                    __builtin_fmaf(rstd, ghi - xhi * c, bf16_hi(dh[j][i])));
            }
            if (col_of(j) < a.cols) norm_store<WHOLE>(a.dX + r * a.lddx, at_of(j), a.cols, dx);
        }
        cur = nxt;
    }
    if (a.part) {
        float *part = a.part + (int64_t)blockIdx.x * a.cols;
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (col_of(j) >= a.cols) continue;
            float *at = part + at_of(j);
            if (WHOLE || col_of(j) + 8 <= a.cols) {
                store16(at, __builtin_bit_cast(u32x4, f32x4{dw[j][0], dw[j][1], dw[j][2], dw[j][3]}));
                store16(at + 4, __builtin_bit_cast(u32x4, f32x4{dw[j][4], dw[j][5], dw[j][6], dw[j][7]}));
            } else {
                const int dup = cc.dup(col_of(j));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i >= dup && at_of(j) + i < a.cols) at[i] = dw[j][i];
            }
        }
    }
}

// Rows past 16384 elements: each is read twice, and a workgroup's row of
// `part` holds its running sums (each element read and written by one
// thread only).
__global__ void __launch_bounds__(256) k_rms_norm_grad_long(NormGradArgs a)
{
    __shared__ float red[2][4];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    float *part = a.part ? a.part + (int64_t)blockIdx.x * a.cols : nullptr;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
        const uint16_t *dyr = a.dY + r * a.lddy, *hr = a.H + r * a.ldh;
        const float rstd = a.rstd[r];
        float dot = 0.f;
        for (int64_t col = threadIdx.x; col < a.cols; col += 256) {
            const float p = __uint_as_float((uint32_t)dyr[col] << 16) * (__uint_as_float((uint32_t)hr[col] << 16) * rstd);
            const float w = a.W ? __uint_as_float((uint32_t)a.W[col] << 16) : 1.0f;
            dot = __builtin_fmaf(p, w, dot);
            if (part) part[col] = r == (int64_t)blockIdx.x ? p : part[col] + p;
        }
        dot = wave_sum(dot);
        if (lane == 0) red[turn][wv] = dot;
        __syncthreads();
        const float c = (((red[turn][0] + red[turn][1]) + red[turn][2]) + red[turn][3]) / (float)a.cols;
        for (int64_t col = threadIdx.x; col < a.cols; col += 256) {
            const float w = a.W ? __uint_as_float((uint32_t)a.W[col] << 16) : 1.0f;
            const float g = __uint_as_float((uint32_t)dyr[col] << 16) * w;
            const float xh = __uint_as_float((uint32_t)hr[col] << 16) * rstd;
            const float dh = a.dH ? __uint_as_float((uint32_t)a.dH[r * a.lddh + col] << 16) : 0.f;
            a.dX[r * a.lddx + col] = (uint16_t)bf16_rne(__builtin_fmaf(rstd, g - xh * c, dh));
        }
    }
}

// dW[n] = sum of rows 0 .. parts - 1 (`stride` floats apart) of `part`: a workgroup owns 16 columns
// (64 bytes of a row), 64 rows in flight at once; thread (row r, column c)
// adds rows r, r + 64, ..., and the 64 sums are joined in order of a tree.
__global__ void __launch_bounds__(1024) k_norm_dw(const float *part, int parts, int64_t stride, int64_t cols, float *dW)
{
    __shared__ float red[64][17];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int64_t n = (int64_t)blockIdx.x * 16 + c;
    float s = 0.f;
    if (n < cols) {
#pragma unroll 8
        for (int p = r; p < parts; p += 64) s += part[(int64_t)p * stride + n];
    }
    red[r][c] = s;
    __syncthreads();
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        if (r < o) red[r][c] += red[r + o][c];
        __syncthreads();
    }
    if (r == 0 && n < cols) dW[n] = red[0][c];
}

// (a launch holds fewer than 2^32 threads, 64 per column: 2^25 columns at a time)
hipError_t launch_norm_dw(const float *part, int parts, int64_t cols, float *dW, hipStream_t s)
{
    constexpr int64_t kCols = (int64_t)1 << 25;
    for (int64_t n = 0; n < cols; n += kCols) {
        const int64_t c = cols - n < kCols ? cols - n : kCols;
        hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)((c + 15) / 16)), dim3(1024), 0, s, part ? part + n : nullptr, parts,
                           cols, c, dW + n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int NCH, int NW>
static void launch_norm_grad_held(const NormGradArgs &a, int grid, hipStream_t s)
{
    if (a.cols % 8 == 0) hipLaunchKernelGGL((k_rms_norm_grad<NCH, NW, true>), dim3(grid), dim3(NW * 64), 0, s, a);
    else hipLaunchKernelGGL((k_rms_norm_grad<NCH, NW, false>), dim3(grid), dim3(NW * 64), 0, s, a);
}

// Two workgroups per CU, four for rows of up to 1024 elements, which leave
// more of a workgroup's time to the loads' latency: 16384 x 1024 27.2 us with
// 1024 workgroups, 34.8 with 512 and 56.7 with 256, while 8192 x 4096 takes
// 42.7 with 512, 44.0 with 256 and 46.1 with 1024 (no dH).
int norm_grad_parts(int64_t rows, int64_t cols)
{
    const int64_t most = cols <= 1024 ? 1024 : 512;
    return (int)(rows < most ? rows : most);
}

hipError_t launch_rms_norm_grad(const NormGradArgs &a, hipStream_t s)
{
    const int grid = norm_grad_parts(a.rows, a.cols);
    // (up to 226 registers per lane: rows past 6144 elements take eight waves)
    if (a.cols <= 2048) launch_norm_grad_held<1, 4>(a, grid, s);
    else if (a.cols <= 4096) launch_norm_grad_held<2, 4>(a, grid, s);
    else if (a.cols <= 6144) launch_norm_grad_held<3, 4>(a, grid, s);
    else if (a.cols <= 8192) launch_norm_grad_held<2, 8>(a, grid, s);
    else if (a.cols <= 16384) launch_norm_grad_held<4, 8>(a, grid, s);
    else hipLaunchKernelGGL(k_rms_norm_grad_long, dim3(grid), dim3(256), 0, s, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || !a.dW ? e : launch_norm_dw(a.part, grid, a.cols, a.dW, s);
}

}  // namespace g5
