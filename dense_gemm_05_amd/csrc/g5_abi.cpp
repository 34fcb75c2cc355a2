// g5_abi.cpp -- C entry points of the dense-GEMM library: argument
// validation, the tile-configuration selector and kernel dispatch.
//
// Validation and selection run on the host only and touch no GPU state, so
// they are usable (through gemm_plan_query) without a device.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "../../include/gemm05.h"
#include "g5_common.h"
#include "g5_kernels.h"

namespace g5 {
namespace {

// ------------------------------------------------------------ config table
const ConfigInfo kConfigs[CFG_COUNT] = {
    {CFG_NONE, GEMM_FAMILY_NONE, 0, 0, 0, 0, 0, "none"},
    {CFG_ZERO, GEMM_FAMILY_ZERO, 0, 0, 0, 256, 0, "zero"},
    {CFG_BF16_256x192, GEMM_FAMILY_BF16_MFMA, 256, 192, 64, 256, 2 * (256 * 64 + 64 * 192) * 2, "bf16_256x192"},
    {CFG_BF16_128x128, GEMM_FAMILY_BF16_MFMA, 128, 128, 64, 256, 2 * (128 * 64 + 64 * 128) * 2, "bf16_128x128"},
    {CFG_BF16_256x128, GEMM_FAMILY_BF16_MFMA, 256, 128, 64, 256, 2 * (256 * 64 + 64 * 128) * 2, "bf16_256x128"},
    {CFG_BF16_256x256, GEMM_FAMILY_BF16_MFMA, 256, 256, 64, 256, 2 * (256 * 64 + 64 * 256) * 2, "bf16_256x256"},
    {CFG_F32_128x128, GEMM_FAMILY_F32_MFMA, 128, 128, 32, 256, 2 * (128 * 32 + 32 * 132) * 4, "f32_128x128"},
    {CFG_F32_64x64, GEMM_FAMILY_F32_MFMA, 64, 64, 32, 256, 2 * (64 * 32 + 32 * 68) * 4, "f32_64x64"},
    {CFG_F32_32x32_WK, GEMM_FAMILY_F32_MFMA, 32, 32, 256, 256, 8 * (32 * 32 + 32 * 36) * 4, "f32_32x32_wholek"},
    {CFG_DECODE_64, GEMM_FAMILY_DECODE, 16, 64, 32, 1024, 16 * 64 * 17 * 4, "decode_64"},
    {CFG_DECODE_SPLIT, GEMM_FAMILY_DECODE, 16, 128, 32, 1024, 16 * 64 * 33 * 4 + 4, "decode_splitk"},
    {CFG_DECODE_NT, GEMM_FAMILY_DECODE, 16, 16, 32, 512, 8 * 64 * 16, "decode_nt"},
    {CFG_GENERIC, GEMM_FAMILY_GENERIC, 16, 16, 16, 256, 2 * 16 * 17 * 4, "generic"},
};

// MI355X figures used by the selector's cost model.
constexpr int kNumCU = 256;
constexpr int64_t kLdsPerCU = 160 * 1024;
constexpr double kHbmBytesPerS = 8.0e12;
constexpr double kCopyBytesPerCUperS = 40.8e9;   // measured, LDS-ring kernels (see model_time)
constexpr double kBf16FlopsPerCUperS = 2.5166e15 / kNumCU;
constexpr double kF32FlopsPerCUperS = 157.3e12 / kNumCU;

struct Problem {
    int op;  // gemm_op
    int64_t batch, M, N, K;
    uint64_t a, b, c;
    int64_t lda, ldb, ldc, sA, sB, sC;
    int c_type;
    uint64_t scale_a = 0, scale_b = 0;   // fp8: dequantization factors (float), 0 = none
    // affine epilogue: C := alpha * (A.B) + bias[n] + beta * C
    float alpha = 1.0f, beta = 0.0f;
    uint64_t bias = 0;                   // bf16 [N], 0 = none
    // SwiGLU with c_type GEMM_OUT_E4M3: the fixed range that maps to 448
    float out_amax = 0.0f;
    // GEMM_OP_BF16_NT with low-rank adapters joined to its sums (NULL: none)
    const LoraArgs *lora = nullptr;
};

struct Plan {
    int config = CFG_NONE;
    bool even = false;       // no edge masking
    int variant = 0;         // kernel variant passed to launch_config
    int64_t grid = 0;
    int64_t tiles_m = 0, tiles_n = 0, group_m = 1;
    int align_a = 2, align_b = 2, align_c = 2;
    int ks = 1;              // K slices of the split small-M path
    int ksplit = 1;          // K slices of a tiled bf16 call (128x128 ring kernel)
    bool realign_a = false;  // copy A's rows to 16-byte aligned ones first
    int64_t lda2 = 0;        // row stride of that copy (elements)
    bool realign_b = false;  // the same for the rows of a transposed B (Bt [N, K])
    int64_t ldb2 = 0;
    bool streamk = false;    // tiled bf16 call on the persistent stream-K schedule (grid = kNumCU)
    double model_bytes = 0.0;
};

// K slices per strip of the split small-M path: enough workgroups for the
// 256 CUs (at most 8 slices, each at least 16 steps of 32 rows).
int decode_slices(int64_t strips, int64_t K)
{
    int64_t ks = 256 / (strips > 0 ? strips : 1);
    const int64_t by_k = K / (32 * 16);
    if (ks > by_k) ks = by_k;
    if (ks > 8) ks = 8;
    return ks < 1 ? 1 : (int)ks;
}

// E4M3FN operands (A and Bt codes with per-row factors).
bool is_fp8(const Problem &p) { return p.op == GEMM_OP_FP8_NT || p.op == GEMM_OP_FP8_NT_AFFINE; }
int elem_a(const Problem &p) { return p.op == GEMM_OP_SGEMM ? 4 : is_fp8(p) ? 1 : 2; }
// K per stage of the LDS-ring kernels: 64-byte slot rows of bf16 or fp8.
int stage_k(const Problem &p) { return is_fp8(p) ? 64 : 32; }
// Batch strides of the fp8 factors (floats): an operand shared by every
// batch entry (stride 0, or a single entry) shares its factors too; else
// entry b's factors follow entry b-1's (M of A's rows, N of Bt's).
int64_t scale_stride_a(const Problem &p) { return p.batch > 1 && p.sA != 0 ? p.M : 0; }
int64_t scale_stride_b(const Problem &p) { return p.batch > 1 && p.sB != 0 ? p.N : 0; }
// Fused epilogue of an operation (EPI_NONE for the plain products).
int epi_of(const Problem &p)
{
    return p.op == GEMM_OP_BF16_SILU     ? EPI_SILU
           : p.op == GEMM_OP_BF16_SWIGLU ? EPI_SWIGLU
           : p.op == GEMM_OP_BF16_AFFINE || p.op == GEMM_OP_BF16_NT_AFFINE || p.op == GEMM_OP_BF16_TN_AFFINE ||
                   p.op == GEMM_OP_FP8_NT_AFFINE
               ? EPI_AFFINE
               : EPI_NONE;
}
bool is_affine(const Problem &p) { return epi_of(p) == EPI_AFFINE; }
// The output type of the generic entry points: FP32 for SGEMM, bf16 for
// SiLU, bf16 or (when asked for) E4M3FN codes for SwiGLU, else the caller's.
int op_c_type(int op, int c_type)
{
    if (op == GEMM_OP_SGEMM) return GEMM_OUT_F32;
    if (op == GEMM_OP_BF16_SILU) return GEMM_OUT_BF16;
    if (op == GEMM_OP_BF16_SWIGLU) return c_type == GEMM_OUT_E4M3 ? GEMM_OUT_E4M3 : GEMM_OUT_BF16;
    return c_type;
}
// An affine call with no product to form (alpha == 0: A and B are not read).
bool no_product(const Problem &p) { return is_affine(p) && p.alpha == 0.0f; }
// B is given transposed, Bt [N, K].
bool b_trans(const Problem &p)
{
    return p.op == GEMM_OP_BF16_NT || is_fp8(p) || p.op == GEMM_OP_BF16_NT_AFFINE;
}
// A is given transposed, At [K, M].
bool a_trans(const Problem &p) { return p.op == GEMM_OP_BF16_TN || p.op == GEMM_OP_BF16_TN_AFFINE; }
// Rows and columns of the A operand as stored: [M, K] or At [K, M].
int64_t a_rows(const Problem &p) { return a_trans(p) ? p.K : p.M; }
int64_t a_cols(const Problem &p) { return a_trans(p) ? p.M : p.K; }
// Rows and columns of the B operand as stored: [K, N], Bt [N, K], or the
// merged gate|up weight [K, 2N] of SwiGLU.
int64_t b_rows(const Problem &p) { return b_trans(p) ? p.N : p.K; }
int64_t b_cols(const Problem &p) { return b_trans(p) ? p.K : p.op == GEMM_OP_BF16_SWIGLU ? 2 * p.N : p.N; }
// Calls only the LDS-ring kernels can run (variants 1-3) when they take a
// tiled config (the affine epilogue also runs in the small-M kernels).
bool ring_only(const Problem &p) { return epi_of(p) != EPI_NONE || b_trans(p) || a_trans(p); }
bool tiled(int config) { return kConfigs[config].family == GEMM_FAMILY_BF16_MFMA; }
// Output columns per tile of a tiled config (SwiGLU: half the B columns).
int64_t out_tile_n(const Problem &p, const ConfigInfo &c)
{
    return p.op == GEMM_OP_BF16_SWIGLU ? c.tile_n / 2 : c.tile_n;
}
int elem_c(const Problem &p)
{
    return p.c_type == GEMM_OUT_E4M3 ? 1 : (p.op == GEMM_OP_SGEMM || p.c_type == GEMM_OUT_F32) ? 4 : 2;
}

// Largest power of two <= 16 dividing the address of every row start of an
// operand (pointer, row stride and batch stride all in bytes).
int row_alignment(uint64_t ptr, int64_t ld, int64_t stride, int64_t batch, int esz)
{
    uint64_t bits = ptr | (uint64_t)(ld * esz);
    if (batch > 1) bits |= (uint64_t)(stride * esz);
    int a = 16;
    while (a > 1 && (bits % (uint64_t)a) != 0) a >>= 1;
    return a;
}

// [lo, hi) byte range touched by an operand with rows x cols elements.
struct Range {
    __int128 lo, hi;
};
Range extent(uint64_t ptr, int64_t batch, int64_t rows, int64_t cols, int64_t ld, int64_t stride, int esz)
{
    __int128 last = (__int128)(batch - 1) * stride + (__int128)(rows - 1) * ld + cols;
    return Range{(__int128)ptr, (__int128)ptr + last * esz};
}
bool overlap(const Range &x, const Range &y) { return x.lo < y.hi && y.lo < x.hi; }

int validate(const Problem &p)
{
    if (p.op != GEMM_OP_SGEMM && p.op != GEMM_OP_BF16 && p.op != GEMM_OP_BF16_SILU && p.op != GEMM_OP_BF16_SWIGLU &&
        p.op != GEMM_OP_BF16_NT && p.op != GEMM_OP_FP8_NT && p.op != GEMM_OP_BF16_AFFINE && p.op != GEMM_OP_BF16_TN &&
        p.op != GEMM_OP_BF16_NT_AFFINE && p.op != GEMM_OP_BF16_TN_AFFINE && p.op != GEMM_OP_FP8_NT_AFFINE)
        return GEMM_ERR_INVALID_ARG;
    if (p.batch < 0 || p.M < 0 || p.N < 0 || p.K < 0) return GEMM_ERR_INVALID_ARG;
    if ((p.op == GEMM_OP_BF16 || p.op == GEMM_OP_BF16_NT || is_fp8(p) || is_affine(p) ||
         p.op == GEMM_OP_BF16_TN) &&
        p.c_type != GEMM_OUT_BF16 && p.c_type != GEMM_OUT_F32)
        return GEMM_ERR_INVALID_ARG;
    if (is_fp8(p) && ((p.scale_a % 4) || (p.scale_b % 4))) return GEMM_ERR_INVALID_ARG;
    if (p.op == GEMM_OP_BF16_SILU && p.c_type != GEMM_OUT_BF16) return GEMM_ERR_INVALID_ARG;
    // SwiGLU writes bf16, or E4M3FN codes against a finite positive range
    if (p.op == GEMM_OP_BF16_SWIGLU && p.c_type != GEMM_OUT_BF16 &&
        (p.c_type != GEMM_OUT_E4M3 || !std::isfinite(p.out_amax) || !(p.out_amax > 0.0f)))
        return GEMM_ERR_INVALID_ARG;
    if (is_affine(p) && (!std::isfinite(p.alpha) || !std::isfinite(p.beta) || (p.bias % 2)))
        return GEMM_ERR_INVALID_ARG;
    if (p.sA < 0 || p.sB < 0 || p.sC < 0) return GEMM_ERR_INVALID_ARG;
    if (p.batch == 0 || p.M == 0 || p.N == 0) return GEMM_OK;  // nothing to do
    if (p.ldc < p.N || p.c == 0) return GEMM_ERR_INVALID_ARG;
    if (p.batch > 1 && (__int128)p.sC < (__int128)(p.M - 1) * p.ldc + p.N) return GEMM_ERR_INVALID_ARG;
    const Range rc = extent(p.c, p.batch, p.M, p.N, p.ldc, p.sC, elem_c(p));
    if (rc.hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
    if (p.bias && overlap(rc, Range{(__int128)p.bias, (__int128)p.bias + 2 * (__int128)p.N})) return GEMM_ERR_INVALID_ARG;
    if (p.K == 0 || no_product(p)) return GEMM_OK;
    if (p.lda < a_cols(p) || p.ldb < b_cols(p) || p.a == 0 || p.b == 0) return GEMM_ERR_INVALID_ARG;
    const Range ra = extent(p.a, p.batch, a_rows(p), a_cols(p), p.lda, p.sA, elem_a(p));
    const Range rb = extent(p.b, p.batch, b_rows(p), b_cols(p), p.ldb, p.sB, elem_a(p));
    if (ra.hi > ((__int128)1 << 63) || rb.hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
    if (overlap(rc, ra) || overlap(rc, rb)) return GEMM_ERR_INVALID_ARG;
    const __int128 na = (__int128)(p.batch - 1) * scale_stride_a(p) + p.M;
    const __int128 nb = (__int128)(p.batch - 1) * scale_stride_b(p) + p.N;
    if (p.scale_a && overlap(rc, Range{(__int128)p.scale_a, (__int128)p.scale_a + 4 * na})) return GEMM_ERR_INVALID_ARG;
    if (p.scale_b && overlap(rc, Range{(__int128)p.scale_b, (__int128)p.scale_b + 4 * nb})) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Cost model of a tiled config (seconds), page "Operator & Runtime" §5.4.5
// (estimate first, then correct by measurement).  The interface traffic of
// §5.2.2 -- every tile reads its A row panel and B column panel and writes
// its C block -- is on gfx950 served mostly by the L2 and the Infinity Cache,
// and what it limits is each CU's copy path: a tile's operand bytes pass
// through one CU at the measured copy rate of the LDS-ring kernels (about
// 41 GB/s per CU: 3.77 MB per 256x192 tile of the FFN projection in a
// ~92 us main loop).  A CU that runs n tiles pays n times the slower of its
// matrix-core time and its copy time; the whole call is never faster than
// reading the operands and writing C once from HBM.  The result is divided
// by a relative efficiency measured per tile shape.
double model_time(const Problem &p, const ConfigInfo &c, double eff)
{
    const int64_t tm = cdiv(p.M, c.tile_m), tn = cdiv(p.N, out_tile_n(p, c));
    const int64_t tiles = p.batch * tm * tn;
    const int64_t per_cu = cdiv(tiles, (int64_t)kNumCU);
    // (E4M3 operands: the double-rate fp8 matrix instruction)
    const double rate = p.op == GEMM_OP_SGEMM ? kF32FlopsPerCUperS
                        : is_fp8(p)           ? 2.0 * kBf16FlopsPerCUperS
                                              : kBf16FlopsPerCUperS;
    const double kpad = (double)cdiv(p.K, c.tile_k) * c.tile_k;
    const double t_mfma = (2.0 * c.tile_m * c.tile_n * kpad) / rate;
    const double tile_bytes =
        (double)(c.tile_m + c.tile_n) * kpad * elem_a(p) + (double)c.tile_m * out_tile_n(p, c) * elem_c(p);
    const double t_copy = tile_bytes / kCopyBytesPerCUperS;
    const double t_tiles = (double)per_cu * (t_mfma > t_copy ? t_mfma : t_copy);
    const double once =
        (double)p.batch * ((double)elem_a(p) * (p.M * p.K + p.K * b_cols(p)) + (double)elem_c(p) * p.M * p.N);
    const double t_hbm = once / kHbmBytesPerS;
    return (t_tiles > t_hbm ? t_tiles : t_hbm) / eff;
}

// The same for the 128x128 ring kernel with K split into S slices: each
// tile's S workgroups run 1/S of the stages, each publishes its FP32 tile
// and the last reads the other S-1 back (both through the CU's copy path).
double model_time_split(const Problem &p, const ConfigInfo &c, int S, double eff)
{
    Problem q = p;
    q.K = cdiv(cdiv(p.K, stage_k(p)), S) * stage_k(p);
    q.batch = p.batch * S;
    const double combine = (double)S * c.tile_m * c.tile_n * 4 / kCopyBytesPerCUperS;
    return model_time(q, c, eff) + combine / eff;
}

int find_config_by_name(const char *name)
{
    for (int i = 0; i < CFG_COUNT; ++i)
        if (std::strcmp(kConfigs[i].name, name) == 0) return i;
    return -1;
}

// Configurations compiled with the fused epilogues (and with fp8 operands).
bool has_epilogues(int id) { return id == CFG_BF16_256x192 || id == CFG_BF16_256x256 || id == CFG_BF16_128x128; }

// The small-M kernels of the projection with adapters: rows of any alignment;
// up to 16 rows they add 32-bit byte offsets of 16 rows.  Past 16 rows every
// 64 weight rows read all of X again, M N K / 32 bytes, which the ring kernels
// do not: measured with 16 adapters of rank 16, mixed, K = 4096, streaming
// against ring, N = 4096: 22 / 36 us for 32 rows, 31 / 40 for 80, 40 / 45 for
// 128; N = 12288: 43 / 53 for 48 rows, 56 / 54 for 64, 77 / 62 for 128.  So up
// to M N = 64 x 12288 (and columns that 32 bits count).  At that bound the
// other K and ranks are, 64 x 12288 and 128 x 4096: K = 1024 27 / 29 and 27 /
// 31, K = 8192 91 / 82 and 57 / 59, rank 64 at K = 4096 97 / 78 and 62 / 98
// (in runs of rows 88 / 67 and 50 / 59): the rule takes the slower side by up
// to a quarter where the columns are many and the rank is high.  (Up to 16 rows a launch
// has up to 36 threads per weight row, and fewer than 2^32.)
bool lora_streams(const Problem &p)
{
    if (p.M <= 16) return p.lda < (1 << 27) && p.ldb < (1 << 27) && p.N <= 1 << 26;
    return p.M <= kLoraStreamRows && p.N <= 64 * 12288 / p.M && p.K <= 1 << 30;
}

bool config_fits(const Problem &p, int id)
{
    const ConfigInfo &c = kConfigs[id];
    if (epi_of(p) != EPI_NONE && c.family == GEMM_FAMILY_DECODE) {   // the small-M kernels apply them too
        if (a_trans(p)) return false;
        if (b_trans(p)) return id == CFG_DECODE_NT && p.M <= 16 && p.batch <= 65535;   // (affine only)
        return (id == CFG_DECODE_64 || id == CFG_DECODE_SPLIT) && p.M <= 16 && p.batch <= 65535;
    }
    if (p.lora) return has_epilogues(id) || (id == CFG_DECODE_NT && lora_streams(p));   // g5_lora.hip's kernels
    if (epi_of(p) != EPI_NONE) return has_epilogues(id);
    if (p.op == GEMM_OP_FP8_NT && id == CFG_DECODE_NT) return p.M <= 16 && p.batch <= 65535;   // k_decode_nt_f8
    if (p.op == GEMM_OP_FP8_NT) return has_epilogues(id);         // fp8 ring kernels: 256x192, 256x256, 128x128
    if (a_trans(p)) return has_epilogues(id);                       // transposed-A ring kernels: the same three
    if (b_trans(p)) return c.family == GEMM_FAMILY_BF16_MFMA;   // the ring kernels of every bf16 tile config
    switch (c.family) {
    case GEMM_FAMILY_BF16_MFMA: return p.op == GEMM_OP_BF16;
    case GEMM_FAMILY_F32_MFMA: return p.op == GEMM_OP_SGEMM;
    case GEMM_FAMILY_DECODE:
        if (id == CFG_DECODE_NT) return p.op == GEMM_OP_BF16_NT && p.M <= 16 && p.batch <= 65535;
        return p.op == GEMM_OP_BF16 && p.M <= 16 && p.batch <= 65535;
    case GEMM_FAMILY_GENERIC: return true;
    default: return false;
    }
}

void fill_grid(const Problem &p, Plan &pl, bool ws)
{
    const ConfigInfo &c = kConfigs[pl.config];
    switch (c.family) {
    case GEMM_FAMILY_ZERO: {
        const int64_t total = p.batch * p.M * p.N;
        int64_t g = cdiv(total, 256);
        if (g > 4096) g = 4096;
        pl.grid = g;
        break;
    }
    case GEMM_FAMILY_DECODE:
        pl.tiles_m = 1;
        // (decode_nt: three 16-row blocks per workgroup when M > 1)
        pl.tiles_n = cdiv(p.N, c.tile_n * (pl.config == CFG_DECODE_NT && p.M > 1 ? 3 : 1));
        // (adapters, more than 16 rows: 64 weight rows per workgroup and slice of K)
        if (p.lora && p.M > 16) pl.tiles_n = cdiv(p.N, 64);
        pl.grid = pl.tiles_n;  // x; batch goes to grid y
        if (pl.config == CFG_DECODE_SPLIT) {
            // (SwiGLU: a strip's gate and up columns are read by separate workgroups)
            // (one slice, a direct store, without a workspace)
            const int64_t groups = pl.tiles_n * (p.op == GEMM_OP_BF16_SWIGLU ? 2 : 1);
            pl.ks = ws ? decode_slices(groups * p.batch, p.K) : 1;
            pl.grid = groups * pl.ks;
        }
        break;
    default:
        pl.tiles_m = cdiv(p.M, c.tile_m);
        pl.tiles_n = cdiv(p.N, out_tile_n(p, c));
        pl.grid = p.batch * pl.tiles_m * pl.tiles_n * pl.ksplit;
        break;
    }
    // Column bands as tall as the whole M extent when it is only a few tiles
    // (each XCD then owns whole column panels of B), else 8 tiles tall.
    pl.group_m = pl.tiles_m <= 8 ? (pl.tiles_m > 0 ? pl.tiles_m : 1) : 8;
    // diagnostic: the orders the map is measured against (GEMM_TILE_ORDER =
    // "rowmajor": tile w for workgroup w; "bands": the same column bands
    // without gathering each XCD's workgroups)
    if (const char *o = std::getenv("GEMM_TILE_ORDER")) {
        if (std::strcmp(o, "rowmajor") == 0) pl.group_m = 0;
        else if (std::strcmp(o, "bands") == 0) pl.group_m = -pl.group_m;
    }
    pl.model_bytes = (c.tile_m > 0 && p.K > 0)
                         ? p.batch * gemm_model_traffic_bytes(p.M, p.N, p.K, c.tile_m, c.tile_n, elem_a(p))
                         : 0.0;
}

// Tiled kernel variant for a config (see launch_config): the aligned ring
// kernel when the problem is whole tiles with 16-byte rows, the masked ring
// kernel when B rows are 16-byte and A rows at least 4-byte aligned and each
// operand's byte extent fits 31 bits (32-bit buffer offsets), else the fully
// general kernel.
int pick_variant(const Problem &p, const Plan &pl, bool *even)
{
    const ConfigInfo &c = kConfigs[pl.config];
    *even = false;
    if (pl.config == CFG_F32_32x32_WK) {     // all of K at once: whole tiles and slabs only
        *even = !(p.M % 32 || p.N % 32 || p.K % 32) && p.K <= 256 && pl.align_a >= 16 && pl.align_b >= 16 &&
                pl.align_c >= 16;
        return *even ? 1 : -1;
    }
    if (c.family == GEMM_FAMILY_F32_MFMA) {
        *even = !(p.M % c.tile_m || p.N % c.tile_n || p.K % c.tile_k) && pl.align_a >= 16 && pl.align_b >= 16 &&
                pl.align_c >= 16;
        return *even ? 1 : 0;
    }
    if (pl.config == CFG_DECODE_NT) {      // 16-byte loads of Bt rows; 3 row blocks per workgroup for M > 1
        *even = p.lora || pl.align_b >= 16;
        return *even ? (p.M > 1 ? 2 : 1) : -1;
    }
    if (c.family == GEMM_FAMILY_DECODE) {
        *even = (p.N % c.tile_n == 0) && pl.align_b >= 8 && pl.align_a >= 16;
        if (pl.config == CFG_DECODE_SPLIT)     // 16-byte loads of whole steps only
            return (*even && pl.align_b >= 16 && p.K % 32 == 0) ? 1 : -1;
        return *even ? 1 : 0;
    }
    if (c.family != GEMM_FAMILY_BF16_MFMA) return 0;
    // (At: the masked copy reads the last row up to M rounded up to 8)
    const __int128 a_bytes = ((__int128)(a_rows(p) - 1) * p.lda + (a_trans(p) ? (p.M + 7) / 8 * 8 : p.K)) * 2;
    const __int128 b_bytes = ((__int128)(b_rows(p) - 1) * p.ldb + b_cols(p)) * 2;
    const bool fits = a_bytes < ((__int128)1 << 31) && b_bytes < ((__int128)1 << 31);
    // N % 8: every 16-byte chunk of B lies wholly inside or wholly past the
    // descriptor extent (no partially out-of-range copies).
    // (Bt's chunks run along K like A's: no condition on N.)
    if (!fits || pl.align_b < 16 || pl.align_a < 4 || (!b_trans(p) && p.N % 8 != 0)) return 0;
    // At is copied 16 bytes per lane in whole chunks: aligned rows, and M % 8
    // == 0 unless the rows are the padded copy.
    if (a_trans(p) && (pl.align_a < 16 || (p.M % 8 != 0 && !pl.realign_a))) return 0;
    const int ring_k = stage_k(p);
    const bool c_ok = pl.align_c >= (elem_c(p) == 4 ? 16 : 8);
    *even = !(p.M % c.tile_m || p.N % out_tile_n(p, c) || p.K % ring_k) && pl.align_a >= 16 && c_ok;
    if (*even) return 1;
    return pl.align_a >= 16 ? 2 : 3;
}

// A K split into S slices of whole 32-deep stages, each at least 4 stages,
// with partial tiles addressable by 32-bit buffer offsets per tile.
bool split_ok(const Problem &p, int S)
{
    const int64_t kt = p.K / stage_k(p);
    return S >= 2 && S <= 8 && kt >= 4 * S && p.batch * cdiv(p.M, 128) * cdiv(p.N, 128) * S <= ((int64_t)1 << 24);
}

// Stages per slice of a K split (the last slice also takes the rest of K).
int split_kt_per(const Problem &p, int S) { return (int)((p.K / stage_k(p)) / S); }

// Counters live in the first kCounterBytes of a workspace: a split call
// needs one per output tile (tiled kernels) or per strip (small-M path), or
// one exchange slot per output (small-M path with two slices).
constexpr size_t kCounterBytes = GEMM_WORKSPACE_COUNTER_BYTES;
constexpr int64_t kMaxCounters = (int64_t)(kCounterBytes / sizeof(unsigned));

// The plan of a call.  `ws`: a caller workspace will be passed, so the
// paths that need scratch memory (K split over workgroups, the split small-M
// path, realigned row copies) may be chosen; without one they are not.
// The persistent stream-K schedule runs plain bf16 products (A as [M, K], B
// as [K, N], no fused epilogue) on the 256x256 and 256x192 ring kernels with
// 16-byte rows (variants 1 and 2), whole 32-deep stages, a workspace and at
// most one counter per tile in its counter region.
bool streamk_ok(const Problem &p, const Plan &pl, bool ws)
{
    return ws && p.op == GEMM_OP_BF16 && (pl.config == CFG_BF16_256x256 || pl.config == CFG_BF16_256x192) &&
           (pl.variant == 1 || pl.variant == 2) && !pl.realign_a && p.K % 32 == 0 && p.K > 0 &&
           p.batch * pl.tiles_m * pl.tiles_n <= kMaxCounters;
}

// Returns GEMM_OK or GEMM_ERR_UNSUPPORTED.
int select_plan(const Problem &p, Plan &pl, bool ws)
{
    pl = Plan();
    if (p.batch == 0 || p.M == 0 || p.N == 0) {
        pl.config = CFG_NONE;
        return GEMM_OK;
    }
    const int ea = elem_a(p), ec = elem_c(p);
    pl.align_a = row_alignment(p.a, p.lda, p.sA, p.batch, ea);
    pl.align_b = row_alignment(p.b, p.ldb, p.sB, p.batch, ea);
    pl.align_c = row_alignment(p.c, p.ldc, p.sC, p.batch, ec);
    if (p.K == 0 || no_product(p)) {
        pl.config = CFG_ZERO;
        fill_grid(p, pl, ws);
        return GEMM_OK;
    }

    // The fused epilogues run in the LDS-staged store of the ring kernels:
    // 16-byte aligned output rows and whole 16-byte output chunks.
    if (epi_of(p) != EPI_NONE && (pl.align_c < 16 || p.N % 8 != 0)) return GEMM_ERR_UNSUPPORTED;
    const char *force = std::getenv("GEMM_FORCE_CONFIG");
    if (force && *force) {
        const int id = find_config_by_name(force);
        if (id < 0 || !config_fits(p, id) || kConfigs[id].family == GEMM_FAMILY_ZERO ||
            kConfigs[id].family == GEMM_FAMILY_NONE)
            return GEMM_ERR_UNSUPPORTED;
        pl.config = id;
    } else if (p.op == GEMM_OP_SGEMM && p.K <= 256 && cdiv(p.M, 64) * cdiv(p.N, 64) * p.batch < kNumCU &&
               [&] { Plan t = pl; t.config = CFG_F32_32x32_WK; bool ev; return pick_variant(p, t, &ev) == 1; }()) {
        // A small FP32 problem with few slabs: 32x32 tiles with all of K
        // staged at once (one load latency per tile instead of one per slab;
        // 256^3 measured 9.4 us with the double-buffered 64x64 kernel).
        pl.config = CFG_F32_32x32_WK;
    } else if ((p.op == GEMM_OP_BF16_NT || p.op == GEMM_OP_BF16_NT_AFFINE || is_fp8(p)) &&
               (p.lora ? lora_streams(p) : p.M <= 16 && p.batch <= 65535 && pl.align_b >= 16)) {
        // Small M with B transposed: a GEMV over the contiguous rows of Bt.
        pl.config = CFG_DECODE_NT;
    } else if ((p.op == GEMM_OP_BF16 || p.op == GEMM_OP_BF16_AFFINE || p.op == GEMM_OP_BF16_SILU ||
                p.op == GEMM_OP_BF16_SWIGLU) &&
               p.M <= 16 && p.batch <= 65535) {
        // The split path (128-column strips, 256 bytes of each W row) when
        // its preconditions hold and it would use more than one slice, or
        // enough whole-K strips to occupy most CUs on their own (one slice:
        // no partial sums, no workspace); SwiGLU always combines its gate and
        // up workgroups, so it needs the workspace.  Else whole-K strips of
        // 64 columns.
        pl.config = CFG_DECODE_SPLIT;
        bool ev = false;
        const bool glu = p.op == GEMM_OP_BF16_SWIGLU;
        const int64_t strips = cdiv(p.N, 128) * p.batch;
        const int ks = ws ? decode_slices(strips * (glu ? 2 : 1), p.K) : 1;
        const bool split = glu ? ws : (ks >= 2 || strips >= kNumCU * 3 / 4);
        if (!split || pick_variant(p, pl, &ev) < 0 || strips > kMaxCounters) pl.config = CFG_DECODE_64;
    } else {
        // Candidates with their measured relative efficiency; the model
        // picks the fastest (page "Operator & Runtime" §5.4.5: feasibility,
        // then an estimate, then measurement).
        struct Cand {
            int id;
            double eff;
        };
        // 256x256 tiles move the fewest bytes per flop through the copy
        // path and LDS, and carry the same measured per-flop rate as 256x192
        // when the tile count fills whole waves: bf16 4096^3 116.6 us
        // against 164.9 us for 256x192 (352 tiles, 2 waves); the FFN shape
        // (192 tiles of 256x256, a 0.75 wave) 115.7 against 97.9 us.
        static const Cand bf16c[] = {{CFG_BF16_256x192, 1.0}, {CFG_BF16_256x256, 1.0}, {CFG_BF16_256x128, 0.95},
                                     {CFG_BF16_128x128, 0.85}};
        // With only a few 32-deep stages per tile, a tile's time is mostly
        // its first-load latency and its epilogue, which a second resident
        // workgroup per CU hides: the 128x128 ring kernel (64 KiB of LDS,
        // two per CU) measured 1.12x faster than 256x128 (96 KiB, one per
        // CU) on 32 x 1024x1024x128 with FP32 output.
        static const Cand bf16_short_k[] = {{CFG_BF16_256x192, 0.7}, {CFG_BF16_256x256, 0.65}, {CFG_BF16_256x128, 0.75},
                                            {CFG_BF16_128x128, 1.0}};
        static const Cand f32c[] = {{CFG_F32_128x128, 1.0}, {CFG_F32_64x64, 0.8}};
        // FP8 ring kernels (256x192, 256x256, 128x128): the 256x256 one runs
        // single-rate stages (its registers do not hold stage pairs) and is
        // half as fast; two co-resident 128x128 workgroups per CU beat the
        // model's copy rate (measured: 4096x1536x4096 39.2 against 51.6 us
        // for 256x192, 4096^3 90.3 against 105.7 us for 256x256, while the
        // FFN's one tile per CU stays on 256x192, 58.8 against 67.6 us).
        static const Cand fp8c[] = {{CFG_BF16_256x192, 1.0}, {CFG_BF16_256x256, 0.5}, {CFG_BF16_128x128, 1.4}};
        const bool bf16 = p.op != GEMM_OP_SGEMM;
        const Cand *cands = is_fp8(p) ? fp8c : bf16 ? (p.K <= 8 * 32 ? bf16_short_k : bf16c) : f32c;
        const int nc = is_fp8(p) ? 3 : bf16 ? 4 : 2;
        double best = 0.0;
        for (int i = 0; i < nc; ++i) {
            if (!config_fits(p, cands[i].id)) continue;
            Plan trial = pl;
            trial.config = cands[i].id;
            bool ev = false;
            const int var = pick_variant(p, trial, &ev);
            // measured relative speed of the kernel variants
            const double veff = var == 1 ? 1.0 : (var == 2 || var == 3) ? 0.85 : 0.3;
            const double t = model_time(p, kConfigs[cands[i].id], cands[i].eff * veff);
            if (pl.config == CFG_NONE || t < best) {
                best = t;
                pl.config = cands[i].id;
            }
        }
        // An output with fewer tiles than CUs: K split over workgroups of
        // 128x128 tiles when the model gives it the shortest time
        // (page "Operator & Runtime" §5.2.4 splits the reduction dimension
        // to occupy the device).
        if (ws && bf16 && (epi_of(p) == EPI_NONE || epi_of(p) == EPI_AFFINE) &&
            p.batch * cdiv(p.M, 128) * cdiv(p.N, 128) < kNumCU) {
            Plan t = pl;
            t.config = CFG_BF16_128x128;
            bool ev = false;
            int var = pick_variant(p, t, &ev);
            if (b_trans(p) && var == 0 && pl.align_b < 16) var = 2;   // Bt rows realigned below
            if (a_trans(p) && var == 0) var = 2;                          // At rows realigned below
            for (int S = 2; S <= 8 && var >= 1; ++S) {
                if (!split_ok(p, S)) continue;
                // (the 128x128 entry of the candidate table above)
                const double base = is_fp8(p) ? 1.4 : p.K <= 8 * 32 ? 1.0 : 0.85;
                const double eff = base * (var == 1 ? 1.0 : 0.85);
                const double tm = model_time_split(p, kConfigs[CFG_BF16_128x128], S, eff);
                if (tm < best) {
                    best = tm;
                    pl.config = CFG_BF16_128x128;
                    pl.ksplit = S;
                }
            }
        }
    }
    if (const char *fk = std::getenv("GEMM_FORCE_KSPLIT")) {
        // diagnostic: force the K split of the 128x128 ring kernel (1 = none)
        const int S = std::atoi(fk);
        if (S >= 1 && pl.config == CFG_BF16_128x128 && (epi_of(p) == EPI_NONE || epi_of(p) == EPI_AFFINE)) {
            if (S > 1 && (!ws || !split_ok(p, S) || p.batch * cdiv(p.M, 128) * cdiv(p.N, 128) > kMaxCounters))
                return GEMM_ERR_UNSUPPORTED;
            pl.ksplit = S;
        }
    }
    fill_grid(p, pl, ws);
    if (pl.grid <= 0 || pl.grid > (int64_t)1 << 24) return GEMM_ERR_UNSUPPORTED;
    // (a forced split path that would need partial sums without a workspace)
    if (pl.config == CFG_DECODE_SPLIT && !ws && p.op == GEMM_OP_BF16_SWIGLU) return GEMM_ERR_UNSUPPORTED;
    pl.variant = pick_variant(p, pl, &pl.even);
    if (pl.variant < 0) return GEMM_ERR_UNSUPPORTED;   // forced split path without its preconditions
    // A large bf16 product whose A rows are not 16-byte aligned: multiply
    // from a copy of A with aligned rows when that lets the ring kernel copy
    // A 16 bytes per lane (the copy costs 2 x M x K x 2 bytes of traffic,
    // small next to the product from 2^30 multiply-adds on).
    // The fused epilogues and a transposed B exist only in the ring kernels,
    // so such a call whose rows no ring variant takes is realigned at any
    // size: Bt's rows first, then A's.
    if (ws && kConfigs[pl.config].family == GEMM_FAMILY_BF16_MFMA && b_trans(p) && !is_fp8(p) &&
        pl.align_b < 16) {
        pl.realign_b = true;
        pl.ldb2 = (p.K + 7) / 8 * 8;
        pl.align_b = 16;
        Problem q = p;
        q.ldb = pl.ldb2;
        q.sB = p.N * pl.ldb2;
        pl.variant = pick_variant(q, pl, &pl.even);
    }
    if (ws && kConfigs[pl.config].family == GEMM_FAMILY_BF16_MFMA && !is_fp8(p) &&
        (pl.align_a < 16 || (a_trans(p) && p.M % 8 != 0)) &&
        ((double)p.batch * p.M * p.N * p.K >= (double)(1 << 30) || (ring_only(p) && pl.variant == 0) ||
         (p.lora && pl.variant == 3))) {
        Problem q = p;
        if (pl.realign_b) {
            q.ldb = pl.ldb2;
            q.sB = p.N * pl.ldb2;
        }
        q.lda = (a_cols(p) + 7) / 8 * 8;
        q.sA = a_rows(p) * q.lda;
        Plan t = pl;
        t.align_a = 16;
        t.realign_a = true;
        bool ev = false;
        const int v = pick_variant(q, t, &ev);
        if (v == 1 || v == 2) {
            pl.realign_a = true;
            pl.lda2 = q.lda;
            pl.align_a = 16;
            pl.variant = v;
            pl.even = ev;
        }
    }
    // fused epilogues and a transposed B exist in the ring kernels only (variants 1-3)
    if (ring_only(p) && tiled(pl.config) && pl.variant == 0) return GEMM_ERR_UNSUPPORTED;
    if (p.lora && tiled(pl.config) && pl.variant == 3) return GEMM_ERR_UNSUPPORTED;   // (16-byte copies only)
    // (k_lora_shrink: 512 threads for 16 rows, fewer than 2^32 in a launch)
    if (p.lora && p.M > ((int64_t)1 << 27) - 16) return GEMM_ERR_UNSUPPORTED;
    if (const char *fs = std::getenv("GEMM_FORCE_STREAMK")) {
        // diagnostic: the persistent stream-K schedule for the chosen tile
        if (*fs == '1') {
            if (!streamk_ok(p, pl, ws)) return GEMM_ERR_UNSUPPORTED;
            pl.streamk = true;
            pl.ksplit = 1;
            const int64_t units = p.batch * pl.tiles_m * pl.tiles_n * (p.K / 32);
            pl.grid = units < kNumCU ? units : kNumCU;
        }
    }
    return GEMM_OK;
}

size_t realign_bytes(const Problem &p, const Plan &pl)
{
    return pl.realign_a ? (size_t)p.batch * a_rows(p) * pl.lda2 * 2 : 0;
}
size_t realign_b_bytes(const Problem &p, const Plan &pl)
{
    return pl.realign_b ? (size_t)p.batch * p.N * pl.ldb2 * 2 : 0;
}

// The split small-M path with one workgroup per strip stores C directly
// (no partial sums, no counters).
bool decode_split_direct(const Problem &p, const Plan &pl)
{
    return pl.config == CFG_DECODE_SPLIT && pl.ks == 1 && p.op != GEMM_OP_BF16_SWIGLU;
}

// Two workgroups per strip (two K slices, or SwiGLU's gate and up with one
// slice each) whose outputs fit the counter region as exchange slots (one
// 32-bit word per output, zero between calls): the split small-M path pairs
// their partial sums by atomic exchange instead of counters and a
// partial-sum buffer (the same sums, in the same order).
bool decode_split_pair(const Problem &p, const Plan &pl)
{
    const bool two = p.op == GEMM_OP_BF16_SWIGLU ? pl.ks == 1 : pl.ks == 2;
    if (const char *e = std::getenv("GEMM_DECODE_PAIR"))    // diagnostic: 0 = counters and partial sums
        if (std::strcmp(e, "0") == 0) return false;
    return pl.config == CFG_DECODE_SPLIT && two && (uint64_t)p.batch * p.M * p.N * 4 <= kCounterBytes;
}

// Partial sums of the split small-M path: one slot of 16 x 128 FP32 per
// (batch entry, strip, K slice); of a K-split tiled call: ksplit FP32 tiles
// per output tile.  The arrival counters (one per strip or tile) are in the
// workspace's counter region.
size_t partial_bytes(const Problem &p, const Plan &pl)
{
    if (pl.config == CFG_DECODE_SPLIT)
        return decode_split_direct(p, pl) || decode_split_pair(p, pl)
                   ? 0
                   : (size_t)p.batch * pl.tiles_n * pl.ks * (p.op == GEMM_OP_BF16_SWIGLU ? 2 : 1) * 16 * 128 *
                         sizeof(float);
    const ConfigInfo &c = kConfigs[pl.config];
    if (pl.streamk) return (size_t)2 * pl.grid * c.tile_m * c.tile_n * 4;
    return pl.ksplit > 1 ? (size_t)p.batch * pl.tiles_m * pl.tiles_n * pl.ksplit * c.tile_m * c.tile_n * 4 : 0;
}

// Workspace layout (byte offsets from its start, each region 256-byte
// aligned): [0, kCounterBytes) arrival counters, then the partial sums,
// then the realigned copy of A, then that of Bt.  A plan that needs none of
// them and no counters (or exchange slots) needs no workspace (0 bytes).
size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }
struct WsLayout {
    size_t part = 0, rows_a = 0, rows_b = 0, total = 0;
};
int64_t counters_used(const Problem &p, const Plan &pl);

WsLayout ws_layout(const Problem &p, const Plan &pl)
{
    WsLayout L;
    const size_t pb = partial_bytes(p, pl), ab = realign_bytes(p, pl), bb = realign_b_bytes(p, pl);
    if (pb == 0 && ab == 0 && bb == 0 && counters_used(p, pl) == 0) return L;
    L.part = kCounterBytes;
    L.rows_a = L.part + round256(pb);
    L.rows_b = L.rows_a + round256(ab);
    L.total = L.rows_b + round256(bb);
    return L;
}

void fill_public_plan(const Problem &p, const Plan &pl, gemm_plan *out)
{
    if (!out) return;
    std::memset(out, 0, sizeof *out);
    const ConfigInfo &c = kConfigs[pl.config];
    out->family = c.family;
    out->config_id = pl.config;
    out->tile_m = c.tile_m;
    out->tile_n = c.tile_n;
    out->tile_k = c.tile_k;
    out->threads = c.threads;
    out->vec_a = pl.align_a;
    out->vec_b = pl.align_b;
    out->even = pl.even ? 1 : 0;
    out->variant = pl.variant;
    out->grid = pl.grid * (c.family == GEMM_FAMILY_DECODE ? p.batch : 1);
    out->lds_bytes = c.lds_bytes;
    if (c.family == GEMM_FAMILY_BF16_MFMA && pl.variant >= 1 && pl.variant <= 3) {
        // LDS-ring kernels: 8 waves, 4 slots of a 32-deep K slab of A and B
        out->threads = 512;
        out->tile_k = 32;
        out->lds_bytes = 4 * (c.tile_m * 32 + 32 * c.tile_n) * 2;
    }
    out->model_bytes = pl.model_bytes;
    std::snprintf(out->name, sizeof out->name, "%s", c.name);
    out->workspace_bytes = (int64_t)ws_layout(p, pl).total;
    out->ksplit = pl.ksplit;
    out->streamk = pl.streamk ? 1 : 0;
}

// ------------------------------------------------------------ device check
std::mutex g_dev_mu;
int g_dev_state[64];  // 0 unknown, 1 gfx950, -1 another architecture (no usable device)

int check_device()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return GEMM_ERR_NO_DEVICE;
    if (dev >= 64) return GEMM_OK;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (g_dev_state[dev] == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_ERR_NO_DEVICE;
        g_dev_state[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : -1;
    }
    return g_dev_state[dev] == 1 ? GEMM_OK : GEMM_ERR_NO_DEVICE;
}

bool log_enabled()
{
    static int v = -1;
    if (v < 0) {
        const char *e = std::getenv("GEMM_LOG");
        v = (e && *e && *e != '0') ? 1 : 0;
    }
    return v == 1;
}

// Arrival counters, or exchange slots, a plan uses (32-bit words at the
// start of the workspace, zero between calls).
int64_t counters_used(const Problem &p, const Plan &pl)
{
    if (pl.config == CFG_DECODE_SPLIT)
        return decode_split_direct(p, pl) ? 0 : decode_split_pair(p, pl) ? p.batch * p.M * p.N : p.batch * pl.tiles_n;
    if (pl.ksplit > 1 || pl.streamk) return p.batch * pl.tiles_m * pl.tiles_n;
    return 0;
}

// The plan a call runs: with the workspace paths when the caller passes a
// workspace (which must then hold what the plan needs), else without.
int plan_for_call(const Problem &p, const void *ws, size_t ws_bytes, Plan &pl, WsLayout &L)
{
    int st = select_plan(p, pl, ws != nullptr);
    if (st != GEMM_OK) return st;
    L = ws_layout(p, pl);
    if (ws != nullptr && L.total > ws_bytes) return GEMM_ERR_WORKSPACE;
    if (ws != nullptr && ((uintptr_t)ws % 256) != 0) return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

// The adapters' values v follow the product's own scratch.  For the small-M
// kernels K is cut into up to 4 slices of at least 512 (by K alone, so a row's
// result does not depend on the other rows up to 16); the adapters of a row
// block are shared out while the grid stays within one workgroup per CU of the
// ring kernels' calls, four where the slices make the work short.
// Past 16 rows the streaming kernel's own slices of K follow: as many as give
// every CU a workgroup, at most 8 and at least one phase each.  (Whole
// calls, 80 x 4104 x 4100: 33.9 us, 36.2 with two workgroups per CU and 43.9
// with three; 128 x 4096 x 4096 39.7, 43.8 and 43.4: the join takes longer.)
size_t lora_layout(const Problem &p, const Plan &pl, const WsLayout &L, LoraArgs &q, size_t *total)
{
    const bool small = pl.config == CFG_DECODE_NT, rows = small && p.M > 16;
    const int64_t splits = p.K / 512 < 4 ? p.K / 512 : 4;
    q.splits = small && splits > 1 ? (int)splits : 1;
    const int64_t room = (rows ? 4 * kNumCU / q.splits : kNumCU) / (cdiv(p.M, 16) * cdiv(q.R, 16));
    int64_t turns = p.M < 16 ? p.M : 16;
    if (turns > q.L) turns = q.L;
    if ((!small || rows) && turns > room) turns = room;
    q.turns = turns < 1 ? 1 : (int)turns;
    q.ranks = (int)((q.R + 7) / 8 * 8);
    const size_t at = L.total > kCounterBytes ? L.total : kCounterBytes;
    *total = at + round256((size_t)q.splits * p.M * q.ranks * 4);
    q.slices = q.per = 1;
    if (rows) {
        const int64_t phases = cdiv(p.K, 128 * lora_steps(p.M));
        int64_t s = kNumCU / pl.tiles_n;
        s = s > 8 ? 8 : s < 1 ? 1 : s;
        q.per = (int)cdiv(phases, s);
        q.slices = (int)cdiv(phases, q.per);
        if (q.slices > 1) *total += (size_t)pl.tiles_n * q.slices * 4 * lora_row_blocks(p.M) * 1024;
    }
    return at;
}

// Validate, plan and enqueue one call.  `ws`: the caller's workspace (NULL:
// none); no memory is allocated, freed, copied or waited for here.
int run(const Problem &p, void *stream, void *ws = nullptr, size_t ws_bytes = 0)
{
    int st = validate(p);
    if (st != GEMM_OK) return st;
    Plan pl;
    WsLayout L;
    st = plan_for_call(p, ws, ws_bytes, pl, L);
    if (st != GEMM_OK) return st;
    if (pl.config == CFG_NONE) return GEMM_OK;
    LoraArgs lora{};
    if (p.lora && pl.config != CFG_ZERO) {
        lora = *p.lora;
        size_t need = 0;
        const size_t at = lora_layout(p, pl, L, lora, &need);
        if (!ws || need > ws_bytes) return GEMM_ERR_WORKSPACE;
        if (pl.config == CFG_DECODE_NT) lora.V = (float *)((char *)ws + at);
        else lora.V2 = (uint16_t *)((char *)ws + at);
        lora.part = (float *)((char *)ws + at + round256((size_t)lora.splits * p.M * lora.ranks * 4));
        lora.count = (unsigned *)ws;
    }
    st = check_device();
    if (st != GEMM_OK) return st;
    char *wsb = (char *)ws;
    unsigned *counters = (unsigned *)wsb;
    if (log_enabled())
        std::fprintf(stderr, "[gemm05] op=%d batch=%lld M=%lld N=%lld K=%lld -> %s variant=%d grid=%lld align=(%d,%d,%d)\n",
                     p.op, (long long)p.batch, (long long)p.M, (long long)p.N, (long long)p.K,
                     kConfigs[pl.config].name, pl.variant, (long long)pl.grid, pl.align_a, pl.align_b,
                     pl.align_c);
    GemmArgs a;
    a.A = (const void *)p.a;
    a.B = (const void *)p.b;
    a.C = (void *)p.c;
    a.M = p.M;
    a.N = p.N;
    a.K = p.K;
    a.lda = p.lda;
    a.ldb = p.ldb;
    a.ldc = p.ldc;
    a.sA = p.sA;
    a.sB = p.sB;
    a.sC = p.sC;
    a.batch = p.batch;
    a.tiles_m = pl.tiles_m;
    a.tiles_n = pl.tiles_n;
    a.group_m = pl.group_m;
    a.align_a = pl.align_a;
    a.align_b = pl.align_b;
    a.align_c = pl.align_c;
    a.out_f32 = elem_c(p) == 4 ? 1 : 0;
    a.ksplit = 1;
    a.kt_per = 0;
    a.b_trans = b_trans(p) ? 1 : 0;
    a.fp8 = is_fp8(p) ? 1 : 0;
    a.scale_a = (const float *)p.scale_a;
    a.scale_b = (const float *)p.scale_b;
    a.s_scale_a = scale_stride_a(p);
    a.s_scale_b = scale_stride_b(p);
    a.alpha = p.alpha;
    a.beta = p.beta;
    a.bias = (const uint16_t *)p.bias;
    a.align_bias = row_alignment(p.bias, 0, 0, 1, 2);
    a.affine = is_affine(p) ? 1 : 0;
    a.a_trans = a_trans(p) ? 1 : 0;
    a.epi = epi_of(p);
    a.c_e4m3 = p.c_type == GEMM_OUT_E4M3 ? 1 : 0;
    a.c_amax = p.out_amax;
    if (pl.realign_b) {
        uint16_t *B2 = (uint16_t *)(wsb + L.rows_b);
        const hipError_t e = launch_realign_rows((const uint16_t *)p.b, p.ldb, p.sB, p.batch, p.N, p.K,
                                                 row_alignment(p.b, p.ldb, p.sB, p.batch, 2), B2, pl.ldb2,
                                                 (hipStream_t)stream);
        if (e != hipSuccess) return GEMM_ERR_LAUNCH;
        a.B = B2;
        a.ldb = pl.ldb2;
        a.sB = p.N * pl.ldb2;
        a.align_b = 16;
    }
    a.ws_part = nullptr;
    a.ws_cnt = nullptr;
    if (pl.ksplit > 1 || pl.streamk) {
        a.ksplit = pl.ksplit;
        a.kt_per = pl.ksplit > 1 ? split_kt_per(p, pl.ksplit) : 0;
        a.ws_part = (float *)(wsb + L.part);
        a.ws_cnt = counters;
    }
    if (pl.streamk) {
        const hipError_t e = launch_streamk(pl.config, a, pl.variant, pl.grid, (hipStream_t)stream);
        return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    if (pl.realign_a) {
        uint16_t *A2 = (uint16_t *)(wsb + L.rows_a);
        const hipError_t e = launch_realign_rows((const uint16_t *)p.a, p.lda, p.sA, p.batch, a_rows(p), a_cols(p),
                                                 row_alignment(p.a, p.lda, p.sA, p.batch, 2), A2, pl.lda2,
                                                 (hipStream_t)stream);
        if (e != hipSuccess) return GEMM_ERR_LAUNCH;
        a.A = A2;
        a.lda = pl.lda2;
        a.sA = a_rows(p) * pl.lda2;
        a.align_a = 16;
    }
    if (p.lora && pl.config != CFG_ZERO) {
        hipError_t e = launch_lora_shrink(a, lora, (hipStream_t)stream);
        if (e == hipSuccess) e = launch_lora(pl.config, a, lora, pl.variant, pl.grid, (hipStream_t)stream);
        return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    if (pl.config == CFG_DECODE_SPLIT) {
        const bool pair = decode_split_pair(p, pl);
        const hipError_t e = launch_decode_split(a, pair ? nullptr : (float *)(wsb + L.part), counters, pl.ks,
                                                 pair ? counters : nullptr, (hipStream_t)stream);
        return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    const hipError_t e =
        pl.config == CFG_ZERO ? (is_affine(p) ? launch_affine_no_product(a, pl.grid, (hipStream_t)stream)
                                                             : launch_config(pl.config, false, a, 0, pl.grid, (hipStream_t)stream))
        : epi_of(p) == EPI_NONE || !tiled(pl.config)
            ? launch_config(pl.config, p.op == GEMM_OP_SGEMM, a, pl.variant, pl.grid, (hipStream_t)stream)
                                : launch_fused(pl.config, epi_of(p), a, pl.variant, pl.grid, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

}  // namespace
}  // namespace g5

using g5::Problem;

extern "C" {

int gemm_sgemm(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B, int64_t ldb,
               float *C, int64_t ldc, void *stream)
{
    const Problem p{GEMM_OP_SGEMM, 1, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc, 0, 0, 0,
                    GEMM_OUT_F32};
    return g5::run(p, stream);
}

int gemm_bf16(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
              void *C, int64_t ldc, int c_type, void *stream)
{
    const Problem p{GEMM_OP_BF16, 1, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc, 0, 0, 0,
                    c_type};
    return g5::run(p, stream);
}

int gemm_bf16_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                      int64_t strideA, const uint16_t *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc,
                      int64_t strideC, int c_type, void *stream)
{
    const Problem p{GEMM_OP_BF16, batch, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc,
                    strideA, strideB, strideC, c_type};
    return g5::run(p, stream);
}

int gemm_bf16_nt(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, const uint16_t *Bt, int64_t ldbt,
                 void *C, int64_t ldc, int c_type, void *stream)
{
    const Problem p{GEMM_OP_BF16_NT, 1, M, N, K, (uint64_t)A, (uint64_t)Bt, (uint64_t)C, lda, ldbt, ldc, 0, 0, 0,
                    c_type};
    return g5::run(p, stream);
}

int gemm_bf16_nt_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                         int64_t strideA, const uint16_t *Bt, int64_t ldbt, int64_t strideBt, void *C, int64_t ldc,
                         int64_t strideC, int c_type, void *stream)
{
    const Problem p{GEMM_OP_BF16_NT, batch, M, N, K, (uint64_t)A, (uint64_t)Bt, (uint64_t)C, lda, ldbt, ldc,
                    strideA, strideBt, strideC, c_type};
    return g5::run(p, stream);
}

int gemm_fp8_nt(int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda, const float *scale_a,
                const uint8_t *Bt, int64_t ldbt, const float *scale_b, void *C, int64_t ldc, int c_type, void *stream)
{
    Problem p{GEMM_OP_FP8_NT, 1, M, N, K, (uint64_t)A, (uint64_t)Bt, (uint64_t)C, lda, ldbt, ldc, 0, 0, 0, c_type};
    p.scale_a = (uint64_t)scale_a;
    p.scale_b = (uint64_t)scale_b;
    return g5::run(p, stream);
}

int gemm_fp8_nt_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                        int64_t strideA, const float *scale_a, const uint8_t *Bt, int64_t ldbt, int64_t strideBt,
                        const float *scale_b, void *C, int64_t ldc, int64_t strideC, int c_type, void *stream)
{
    Problem p{GEMM_OP_FP8_NT, batch, M, N, K, (uint64_t)A, (uint64_t)Bt, (uint64_t)C, lda, ldbt, ldc, strideA,
              strideBt, strideC, c_type};
    p.scale_a = (uint64_t)scale_a;
    p.scale_b = (uint64_t)scale_b;
    return g5::run(p, stream);
}

int gemm_fp8_nt_affine(int64_t batch, int64_t M, int64_t N, int64_t K, const uint8_t *A, int64_t lda,
                       int64_t strideA, const float *scale_a, const uint8_t *Bt, int64_t ldbt, int64_t strideBt,
                       const float *scale_b, float alpha, const uint16_t *bias, float beta, void *C, int64_t ldc,
                       int64_t strideC, int c_type, void *stream)
{
    Problem p{GEMM_OP_FP8_NT_AFFINE, batch, M, N, K, (uint64_t)A, (uint64_t)Bt, (uint64_t)C, lda, ldbt, ldc, strideA,
              strideBt, strideC, c_type};
    p.scale_a = (uint64_t)scale_a;
    p.scale_b = (uint64_t)scale_b;
    p.alpha = alpha;
    p.beta = beta;
    p.bias = (uint64_t)bias;
    return g5::run(p, stream);
}

int gemm_fp8_nt_quant_a(int64_t M, int64_t N, int64_t K, const uint16_t *X, int64_t ldx, float *scale_x,
                        const uint8_t *Bt, int64_t ldbt, const float *scale_b, void *C, int64_t ldc, int c_type,
                        void *workspace, uint64_t workspace_bytes, void *stream)
{
    using g5::Range;
    if (M < 0 || N < 0 || K < 0 || M > 0x7fffffff) return GEMM_ERR_INVALID_ARG;
    if (c_type != GEMM_OUT_BF16 && c_type != GEMM_OUT_F32) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!X || !Bt || !C || !scale_x || ldx < K || ldbt < K || ldc < N) return GEMM_ERR_INVALID_ARG;
    if (((uint64_t)scale_x % 4) || ((uint64_t)scale_b % 4) || ((uint64_t)X % 2)) return GEMM_ERR_INVALID_ARG;
    const int ec = c_type == GEMM_OUT_F32 ? 4 : 2;
    const Range rx = g5::extent((uint64_t)X, 1, M, K > 0 ? K : 1, ldx, 0, 2);
    const Range rb = g5::extent((uint64_t)Bt, 1, N, K > 0 ? K : 1, ldbt, 0, 1);
    const Range rc = g5::extent((uint64_t)C, 1, M, N, ldc, 0, ec);
    const Range rs{(__int128)(uint64_t)scale_x, (__int128)(uint64_t)scale_x + 4 * (__int128)M};
    // the row maxima go after the workspace's arrival counters, which other
    // calls sharing the workspace expect to find at zero
    const Range rw{(__int128)(uint64_t)workspace + (__int128)g5::kCounterBytes,
                   (__int128)(uint64_t)workspace + (__int128)g5::kCounterBytes + 4 * (__int128)M};
    if (g5::overlap(rc, rx) || g5::overlap(rc, rb) || g5::overlap(rc, rs) || g5::overlap(rs, rx) || g5::overlap(rs, rb))
        return GEMM_ERR_INVALID_ARG;
    if (scale_b && g5::overlap(rc, Range{(__int128)(uint64_t)scale_b, (__int128)(uint64_t)scale_b + 4 * (__int128)N}))
        return GEMM_ERR_INVALID_ARG;
    // whole 64-deep stages, 16-byte rows of X and Bt, 32-bit buffer offsets
    if (K == 0 || K % 64 != 0 || g5::row_alignment((uint64_t)X, ldx, 0, 1, 2) < 16 ||
        g5::row_alignment((uint64_t)Bt, ldbt, 0, 1, 1) < 16 || rx.hi - rx.lo >= ((__int128)1 << 31) ||
        rb.hi - rb.lo >= ((__int128)1 << 31))
        return GEMM_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < g5::kCounterBytes + 4 * (uint64_t)M) return GEMM_ERR_WORKSPACE;
    if (((uint64_t)workspace % 256) || g5::overlap(rw, rx) || g5::overlap(rw, rb) || g5::overlap(rw, rc) ||
        g5::overlap(rw, rs))
        return GEMM_ERR_INVALID_ARG;
    const int st = g5::check_device();
    if (st != GEMM_OK) return st;
    g5::GemmArgs a{};
    a.A = X;
    a.B = Bt;
    a.C = C;
    a.M = M;
    a.N = N;
    a.K = K;
    a.lda = ldx;
    a.ldb = ldbt;
    a.ldc = ldc;
    a.batch = 1;
    // Tile width: 256 columns convert each A element half as often as 128
    // (the conversion, not the MFMAs, bounds the loop), at one workgroup
    // per CU instead of two.  Per-CU costs measured with K = 4096 (both
    // scale with K alike): one 128x256 tile 72 us; two 128x128 tiles
    // sharing a CU 87 us, one alone 50 us.  The width with the smaller
    // estimate for the busiest CU is taken (e.g. 4096x1536: 256, one tile
    // per CU on 192 CUs; 1024x12288: 128, three tiles per CU against two
    // rounds of the wider ones).  GEMM_QA_TILE_N=128|256 forces one
    // (diagnostic).
    const int64_t tm = (M + 127) / 128;
    const int64_t k256 = (tm * ((N + 255) / 256) + g5::kNumCU - 1) / g5::kNumCU;
    const int64_t k128 = (tm * ((N + 127) / 128) + g5::kNumCU - 1) / g5::kNumCU;
    int tile_n = 72.0 * k256 < 87.0 * (k128 / 2) + 50.0 * (k128 % 2) ? 256 : 128;
    if (const char *f = std::getenv("GEMM_QA_TILE_N")) {
        if (std::strcmp(f, "128") == 0) tile_n = 128;
        else if (std::strcmp(f, "256") == 0) tile_n = 256;
    }
    a.tiles_m = tm;
    a.tiles_n = (N + tile_n - 1) / tile_n;
    a.group_m = a.tiles_m <= 8 ? a.tiles_m : 8;
    a.align_a = 16;
    a.align_b = 16;
    a.align_c = g5::row_alignment((uint64_t)C, ldc, 0, 1, ec);
    a.out_f32 = ec == 4 ? 1 : 0;
    a.ksplit = 1;
    a.b_trans = 1;
    a.fp8 = 1;
    a.scale_a = scale_x;
    a.scale_b = scale_b;
    a.alpha = 1.0f;
    const hipError_t e = g5::launch_fp8_quant_a(a, (float *)((char *)workspace + g5::kCounterBytes), tile_n,
                                                a.tiles_m * a.tiles_n, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_fp8_quantize_rows(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, uint8_t *Q, int64_t ldq,
                           float *scale, void *stream)
{
    if (rows < 0 || cols < 0 || rows > 0x7fffffff) return GEMM_ERR_INVALID_ARG;
    if (rows == 0) return GEMM_OK;
    if (!scale || ((uint64_t)scale % 4)) return GEMM_ERR_INVALID_ARG;
    if (cols > 0 && (!X || !Q || ldx < cols || ldq < cols)) return GEMM_ERR_INVALID_ARG;
    const g5::Range rs{(__int128)(uint64_t)scale, (__int128)(uint64_t)scale + 4 * (__int128)rows};
    if (cols > 0) {
        const g5::Range rx = g5::extent((uint64_t)X, 1, rows, cols, ldx, 0, 2);
        const g5::Range rq = g5::extent((uint64_t)Q, 1, rows, cols, ldq, 0, 1);
        if (g5::overlap(rx, rq) || g5::overlap(rs, rx) || g5::overlap(rs, rq)) return GEMM_ERR_INVALID_ARG;
    }
    int st = g5::check_device();
    if (st != GEMM_OK) return st;
    const hipError_t e = g5::launch_quant_rows_e4m3(X, ldx, rows, cols, g5::row_alignment((uint64_t)X, ldx, 0, 1, 2),
                                                    Q, ldq, g5::row_alignment((uint64_t)Q, ldq, 0, 1, 1), scale,
                                                    (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_act_chain(int step, int64_t M, int64_t N, const uint16_t *in0, int64_t ld0, const uint16_t *in1,
                   int64_t ld1, void *out, int64_t ldo, float amax, void *stream)
{
    if (step < GEMM_ACT_SILU || step > GEMM_ACT_SWIGLU_E4M3 || M < 0 || N < 0) return GEMM_ERR_INVALID_ARG;
    const bool two = step == GEMM_ACT_MUL || step == GEMM_ACT_SWIGLU || step == GEMM_ACT_SWIGLU_E4M3;
    const bool codes = step == GEMM_ACT_QUANT || step == GEMM_ACT_SWIGLU_E4M3;
    if (codes && !(std::isfinite(amax) && amax > 0.0f)) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GEMM_OK;
    const int eo = codes ? 1 : 2;
    if (!in0 || !out || (two && !in1) || ld0 < N || ldo < N || (two && ld1 < N)) return GEMM_ERR_INVALID_ARG;
    if (((uint64_t)in0 % 2) || (two && ((uint64_t)in1 % 2)) || ((uint64_t)out % eo)) return GEMM_ERR_INVALID_ARG;
    const g5::Range r0 = g5::extent((uint64_t)in0, 1, M, N, ld0, 0, 2);
    const g5::Range ro = g5::extent((uint64_t)out, 1, M, N, ldo, 0, eo);
    if (r0.hi > ((__int128)1 << 63) || ro.hi > ((__int128)1 << 63) || g5::overlap(r0, ro)) return GEMM_ERR_INVALID_ARG;
    if (two) {
        const g5::Range r1 = g5::extent((uint64_t)in1, 1, M, N, ld1, 0, 2);
        if (r1.hi > ((__int128)1 << 63) || g5::overlap(r1, ro)) return GEMM_ERR_INVALID_ARG;
    }
    int st = g5::check_device();
    if (st != GEMM_OK) return st;
    // 16-byte chunks when every row holds whole chunks at aligned starts
    const bool vec = N % 8 == 0 && (__int128)M * (N / 8) < ((__int128)1 << 31) &&
                     g5::row_alignment((uint64_t)in0, ld0, 0, 1, 2) >= 16 &&
                     (!two || g5::row_alignment((uint64_t)in1, ld1, 0, 1, 2) >= 16) &&
                     g5::row_alignment((uint64_t)out, ldo, 0, 1, eo) >= 8 * eo;
    const bool contig = ld0 == N && ldo == N && (!two || ld1 == N);
    const g5::ActArgs a{in0, two ? in1 : nullptr, out, M, N, ld0, two ? ld1 : N, ldo, codes ? amax : 1.0f};
    const hipError_t e = g5::launch_act_chain(step, a, vec, contig, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_fp8_quantize_cols(int64_t K, int64_t N, const uint16_t *W, int64_t ldw, uint8_t *Qt, int64_t ldq,
                           float *scale, void *stream)
{
    if (K < 0 || N < 0 || N > ((int64_t)1 << 36)) return GEMM_ERR_INVALID_ARG;
    if (N == 0) return GEMM_OK;
    if (!scale || ((uint64_t)scale % 4)) return GEMM_ERR_INVALID_ARG;
    if (K > 0 && (!W || !Qt || ((uint64_t)W % 2) || ldw < N || ldq < K)) return GEMM_ERR_INVALID_ARG;
    const g5::Range rs{(__int128)(uint64_t)scale, (__int128)(uint64_t)scale + 4 * (__int128)N};
    if (K > 0) {
        const g5::Range rw = g5::extent((uint64_t)W, 1, K, N, ldw, 0, 2);
        const g5::Range rq = g5::extent((uint64_t)Qt, 1, N, K, ldq, 0, 1);
        if (g5::overlap(rw, rq) || g5::overlap(rs, rw) || g5::overlap(rs, rq)) return GEMM_ERR_INVALID_ARG;
    }
    int st = g5::check_device();
    if (st != GEMM_OK) return st;
    const hipError_t e = g5::launch_quant_cols_e4m3(W, ldw, K, N, g5::row_alignment((uint64_t)W, ldw, 0, 1, 2), Qt, ldq,
                                                    g5::row_alignment((uint64_t)Qt, ldq, 0, 1, 1), scale,
                                                    (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_bf16_silu(int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                   uint16_t *C, int64_t ldc, void *stream)
{
    const Problem p{GEMM_OP_BF16_SILU, 1, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc, 0, 0, 0,
                    GEMM_OUT_BF16};
    return g5::run(p, stream);
}

int gemm_bf16_swiglu(int64_t M, int64_t N, int64_t K, const uint16_t *X, int64_t ldx, const uint16_t *Wgu,
                     int64_t ldw, uint16_t *Z, int64_t ldz, void *stream)
{
    const Problem p{GEMM_OP_BF16_SWIGLU, 1, M, N, K, (uint64_t)X, (uint64_t)Wgu, (uint64_t)Z, ldx, ldw, ldz, 0, 0,
                    0, GEMM_OUT_BF16};
    return g5::run(p, stream);
}

int gemm_bf16_swiglu_e4m3(int64_t M, int64_t N, int64_t K, const uint16_t *X, int64_t ldx, const uint16_t *Wgu,
                          int64_t ldw, uint8_t *Zq, int64_t ldz, float amax, void *stream)
{
    Problem p{GEMM_OP_BF16_SWIGLU, 1, M, N, K, (uint64_t)X, (uint64_t)Wgu, (uint64_t)Zq, ldx, ldw, ldz, 0, 0,
              0, GEMM_OUT_E4M3};
    p.out_amax = amax;
    return g5::run(p, stream);
}

int gemm_bf16_silu_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                           int64_t strideA, const uint16_t *B, int64_t ldb, int64_t strideB, uint16_t *C, int64_t ldc,
                           int64_t strideC, void *stream)
{
    const Problem p{GEMM_OP_BF16_SILU, batch, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc,
                    strideA, strideB, strideC, GEMM_OUT_BF16};
    return g5::run(p, stream);
}

int gemm_bf16_swiglu_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *X, int64_t ldx,
                             int64_t strideX, const uint16_t *Wgu, int64_t ldw, int64_t strideW, uint16_t *Z,
                             int64_t ldz, int64_t strideZ, void *stream)
{
    const Problem p{GEMM_OP_BF16_SWIGLU, batch, M, N, K, (uint64_t)X, (uint64_t)Wgu, (uint64_t)Z, ldx, ldw, ldz,
                    strideX, strideW, strideZ, GEMM_OUT_BF16};
    return g5::run(p, stream);
}

int gemm_bf16_swiglu_e4m3_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *X, int64_t ldx,
                                  int64_t strideX, const uint16_t *Wgu, int64_t ldw, int64_t strideW, uint8_t *Zq,
                                  int64_t ldz, int64_t strideZ, float amax, void *stream)
{
    Problem p{GEMM_OP_BF16_SWIGLU, batch, M, N, K, (uint64_t)X, (uint64_t)Wgu, (uint64_t)Zq, ldx, ldw, ldz,
              strideX, strideW, strideZ, GEMM_OUT_E4M3};
    p.out_amax = amax;
    return g5::run(p, stream);
}

int gemm_bf16_tn(int64_t M, int64_t N, int64_t K, const uint16_t *At, int64_t ldat, const uint16_t *B, int64_t ldb,
                 void *C, int64_t ldc, int c_type, void *stream)
{
    const Problem p{GEMM_OP_BF16_TN, 1, M, N, K, (uint64_t)At, (uint64_t)B, (uint64_t)C, ldat, ldb, ldc, 0, 0, 0,
                    c_type};
    return g5::run(p, stream);
}

int gemm_bf16_tn_batched(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *At, int64_t ldat,
                         int64_t strideAt, const uint16_t *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc,
                         int64_t strideC, int c_type, void *stream)
{
    const Problem p{GEMM_OP_BF16_TN, batch, M, N, K, (uint64_t)At, (uint64_t)B, (uint64_t)C, ldat, ldb, ldc,
                    strideAt, strideB, strideC, c_type};
    return g5::run(p, stream);
}

int gemm_bf16_affine(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda, int64_t strideA,
                     const uint16_t *B, int64_t ldb, int64_t strideB, float alpha, const uint16_t *bias, float beta,
                     void *C, int64_t ldc, int64_t strideC, int c_type, void *stream)
{
    Problem p{GEMM_OP_BF16_AFFINE, batch, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc,
              strideA, strideB, strideC, c_type};
    p.alpha = alpha;
    p.beta = beta;
    p.bias = (uint64_t)bias;
    return g5::run(p, stream);
}

int gemm_bf16_tn_affine(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *At, int64_t ldat,
                        int64_t strideAt, const uint16_t *B, int64_t ldb, int64_t strideB, float alpha,
                        const uint16_t *bias, float beta, void *C, int64_t ldc, int64_t strideC, int c_type,
                        void *stream)
{
    Problem p{GEMM_OP_BF16_TN_AFFINE, batch, M, N, K, (uint64_t)At, (uint64_t)B, (uint64_t)C, ldat, ldb, ldc,
              strideAt, strideB, strideC, c_type};
    p.alpha = alpha;
    p.beta = beta;
    p.bias = (uint64_t)bias;
    return g5::run(p, stream);
}

int gemm_bf16_nt_affine(int64_t batch, int64_t M, int64_t N, int64_t K, const uint16_t *A, int64_t lda,
                        int64_t strideA, const uint16_t *Bt, int64_t ldbt, int64_t strideBt, float alpha,
                        const uint16_t *bias, float beta, void *C, int64_t ldc, int64_t strideC, int c_type,
                        void *stream)
{
    Problem p{GEMM_OP_BF16_NT_AFFINE, batch, M, N, K, (uint64_t)A, (uint64_t)Bt, (uint64_t)C, lda, ldbt, ldc,
              strideA, strideBt, strideC, c_type};
    p.alpha = alpha;
    p.beta = beta;
    p.bias = (uint64_t)bias;
    return g5::run(p, stream);
}

// ---- RMS norm: the arguments' checks, shared shape of the entries below
// [lo, hi) of a vector of n elements of esz bytes (empty for NULL).
static g5::Range vec_range(const void *v, int64_t n, int esz)
{
    if (!v) return g5::Range{0, 0};
    return g5::Range{(__int128)(uint64_t)v, (__int128)(uint64_t)v + (__int128)esz * n};
}
// Whether any output range overlaps an input or another output.
static bool outputs_overlap(const g5::Range *out, int n_out, const g5::Range *in, int n_in)
{
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (g5::overlap(out[i], in[j])) return true;
        for (int j = i + 1; j < n_out; ++j)
            if (g5::overlap(out[i], out[j])) return true;
    }
    return false;
}

int gemm_rms_norm(int64_t rows, int64_t cols, const uint16_t *X, int64_t ldx, const uint16_t *R, int64_t ldr,
                  uint16_t *H, int64_t ldh, const uint16_t *W, float eps, void *Y, int64_t ldy, int y_type,
                  float *scale, float *rstd, void *stream)
{
    using g5::Range;
    const bool codes = y_type == GEMM_OUT_E4M3;
    if (rows < 0 || cols < 0 || rows > 0x7fffffff) return GEMM_ERR_INVALID_ARG;
    if ((y_type != GEMM_OUT_BF16 && !codes) || !std::isfinite(eps) || eps < 0.0f) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return GEMM_OK;
    if (!X || !Y || (codes && !scale) || (H && !R)) return GEMM_ERR_INVALID_ARG;
    if (ldx < cols || ldy < cols || (R && ldr < cols) || (H && ldh < cols)) return GEMM_ERR_INVALID_ARG;
    const int ey = codes ? 1 : 2;
    if (((uint64_t)X % 2) || ((uint64_t)R % 2) || ((uint64_t)H % 2) || ((uint64_t)W % 2) || ((uint64_t)Y % ey) ||
        (codes && ((uint64_t)scale % 4)) || ((uint64_t)rstd % 4))
        return GEMM_ERR_INVALID_ARG;
    const Range none{0, 0};
    const Range rx = g5::extent((uint64_t)X, 1, rows, cols, ldx, 0, 2);
    const Range rr = R ? g5::extent((uint64_t)R, 1, rows, cols, ldr, 0, 2) : none;
    const Range rh = H ? g5::extent((uint64_t)H, 1, rows, cols, ldh, 0, 2) : none;
    const Range ry = g5::extent((uint64_t)Y, 1, rows, cols, ldy, 0, ey);
    const Range rw = vec_range(W, cols, 2);
    const __int128 top = (__int128)1 << 63;
    if (rx.hi > top || rr.hi > top || rh.hi > top || ry.hi > top || rw.hi > top) return GEMM_ERR_INVALID_ARG;
    // H may be X or R itself (the sum in place): then the two ranges are one
    const bool h_is_x = H && H == X && ldh == ldx, h_is_r = H && H == R && ldh == ldr;
    const Range in[] = {h_is_x ? none : rx, h_is_r ? none : rr, rw};
    const Range out[] = {rh, ry, codes ? vec_range(scale, rows, 4) : none, vec_range(rstd, rows, 4)};
    if (outputs_overlap(out, 4, in, 3)) return GEMM_ERR_INVALID_ARG;
    const int st = g5::check_device();
    if (st != GEMM_OK) return st;
    const g5::NormArgs a{X, R, W, H, Y, codes ? scale : nullptr, rstd, rows, cols, ldx, R ? ldr : cols, H ? ldh : cols,
                         ldy, eps};
    const hipError_t e = g5::launch_rms_norm(a, codes, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_rms_norm_workspace_size(int64_t rows, int64_t cols, uint64_t *bytes)
{
    if (bytes) *bytes = 0;
    if (rows < 0 || cols < 0 || rows > 0x7fffffff || cols > ((int64_t)1 << 40)) return GEMM_ERR_INVALID_ARG;
    if (bytes && rows > 0 && cols > 0)
        *bytes = g5::kCounterBytes + g5::round256((size_t)g5::norm_grad_parts(rows, cols) * (size_t)cols * 4);
    return GEMM_OK;
}

int gemm_rms_norm_backward(int64_t rows, int64_t cols, const uint16_t *dY, int64_t lddy, const uint16_t *H,
                           int64_t ldh, const uint16_t *W, const float *rstd, const uint16_t *dH, int64_t lddh,
                           uint16_t *dX, int64_t lddx, float *dW, void *workspace, uint64_t workspace_bytes,
                           void *stream)
{
    using g5::Range;
    if (rows < 0 || cols < 0 || rows > 0x7fffffff) return GEMM_ERR_INVALID_ARG;
    if (cols == 0 || (rows == 0 && !dW)) return GEMM_OK;
    if (rows == 0) {          // dW := 0, the empty sum
        if ((uint64_t)dW % 4 || vec_range(dW, cols, 4).hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
        const int st = g5::check_device();
        if (st != GEMM_OK) return st;
        return g5::launch_norm_dw(nullptr, 0, cols, dW, (hipStream_t)stream) == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    if (!dY || !H || !rstd || !dX || lddy < cols || ldh < cols || lddx < cols || (dH && lddh < cols))
        return GEMM_ERR_INVALID_ARG;
    if (((uint64_t)dY % 2) || ((uint64_t)H % 2) || ((uint64_t)W % 2) || ((uint64_t)dH % 2) || ((uint64_t)dX % 2) ||
        ((uint64_t)rstd % 4) || ((uint64_t)dW % 4))
        return GEMM_ERR_INVALID_ARG;
    const Range none{0, 0};
    const Range rdy = g5::extent((uint64_t)dY, 1, rows, cols, lddy, 0, 2);
    const Range rh = g5::extent((uint64_t)H, 1, rows, cols, ldh, 0, 2);
    const Range rdh = dH ? g5::extent((uint64_t)dH, 1, rows, cols, lddh, 0, 2) : none;
    const Range rdx = g5::extent((uint64_t)dX, 1, rows, cols, lddx, 0, 2);
    const __int128 top = (__int128)1 << 63;
    if (rdy.hi > top || rh.hi > top || rdh.hi > top || rdx.hi > top) return GEMM_ERR_INVALID_ARG;
    const Range in[] = {rdy, rh, rdh, vec_range(W, cols, 2), vec_range(rstd, rows, 4)};
    uint64_t need = 0;
    if (dW && gemm_rms_norm_workspace_size(rows, cols, &need) != GEMM_OK) return GEMM_ERR_INVALID_ARG;
    const Range rws = dW && workspace ? Range{(__int128)(uint64_t)workspace, (__int128)(uint64_t)workspace + need} : none;
    const Range out[] = {rdx, vec_range(dW, cols, 4), rws};
    if (outputs_overlap(out, 3, in, 5)) return GEMM_ERR_INVALID_ARG;
    if (dW && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
    if (dW && ((uint64_t)workspace % 256)) return GEMM_ERR_INVALID_ARG;
    const int st = g5::check_device();
    if (st != GEMM_OK) return st;
    const g5::NormGradArgs a{dY, H, W, dH, rstd, dX, dW ? (float *)((char *)workspace + g5::kCounterBytes) : nullptr, dW,
                             rows, cols, lddy, ldh, dH ? lddh : cols, lddx};
    const hipError_t e = g5::launch_rms_norm_grad(a, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

// ---- mixture-of-experts layer for a few tokens
// Scratch after the counter region, each part 256-byte aligned.
struct MoeLayout {
    size_t ids, gates, n_items, items, pairs, z, halves, arrived, total;
    int64_t ldz, zplane;
};
static MoeLayout moe_layout(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk)
{
    MoeLayout L;
    const size_t pairs = (size_t)T * topk;
    L.ldz = (I + 127) / 128 * 128;      // rows start on 256 bytes; columns from I on are neither written nor read
    L.zplane = (int64_t)pairs * L.ldz;
    L.ids = g5::kCounterBytes;
    L.gates = L.ids + g5::round256(pairs * 4);
    L.n_items = L.gates + g5::round256(pairs * 4);
    L.items = L.n_items + 256;
    L.pairs = L.items + g5::round256((size_t)g5::moe_items(T, E, topk) * sizeof(g5::MoeItem));
    L.z = L.pairs + g5::round256(pairs * 4);
    L.halves = L.z + g5::round256((size_t)L.zplane * 4);
    const size_t blocks = g5::moe_halves(T, H) ? (size_t)(H + 31) / 32 : 0;
    L.arrived = L.halves + blocks * 2 * g5::kMoeMaxTokens * 32 * 4;
    L.total = L.arrived + g5::round256(blocks * 4);
    return L;
}
static bool moe_sizes_ok(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk)
{
    return T >= 0 && T <= g5::kMoeMaxTokens && H >= 0 && H <= g5::kMoeMaxWidth && I >= 0 && I <= g5::kMoeMaxWidth &&
           E >= 1 && E <= g5::kMoeMaxExperts && topk >= 1 && topk <= g5::kMoeMaxTopk && topk <= E;
}

int gemm_moe_workspace_size(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, uint64_t *bytes)
{
    if (bytes) *bytes = 0;
    if (!moe_sizes_ok(T, H, I, E, topk)) return GEMM_ERR_INVALID_ARG;
    if (bytes && T > 0) *bytes = moe_layout(T, H, I, E, topk).total;
    return GEMM_OK;
}

int gemm_moe_swiglu(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, int renormalize, const uint16_t *X,
                    int64_t ldx, const float *logits, int64_t ldl, int w_type, const void *Wgu, int64_t ldgu,
                    int64_t strideGu, const float *scale_gu, const void *Wd, int64_t ldd, int64_t strideD,
                    const float *scale_d, void *Y, int64_t ldy, int c_type, int32_t *ids, float *gates,
                    void *workspace, uint64_t workspace_bytes, void *stream)
{
    using g5::Range;
    const bool codes = w_type == GEMM_OUT_E4M3;
    if (!moe_sizes_ok(T, H, I, E, topk)) return GEMM_ERR_INVALID_ARG;
    if ((w_type != GEMM_OUT_BF16 && !codes) || (c_type != GEMM_OUT_BF16 && c_type != GEMM_OUT_F32))
        return GEMM_ERR_INVALID_ARG;
    if (T == 0) return GEMM_OK;
    const int ew = codes ? 1 : 2, ec = c_type == GEMM_OUT_F32 ? 4 : 2;
    if (!logits || ldl < E || ((uint64_t)logits % 4) || ((uint64_t)ids % 4) || ((uint64_t)gates % 4))
        return GEMM_ERR_INVALID_ARG;
    if (H > 0 && (!X || !Y || ldx < H || ldy < H || ((uint64_t)X % 2) || ((uint64_t)Y % ec))) return GEMM_ERR_INVALID_ARG;
    if (((uint64_t)scale_gu % 4) || ((uint64_t)scale_d % 4) || (!codes && (scale_gu || scale_d)))
        return GEMM_ERR_INVALID_ARG;
    const bool weights = H > 0 && I > 0;
    if (weights && (!Wgu || !Wd || ldgu < H || ldd < I || strideGu < 0 || strideD < 0 || ((uint64_t)Wgu % ew) ||
                    ((uint64_t)Wd % ew)))
        return GEMM_ERR_INVALID_ARG;
    const Range none{0, 0};
    const Range in[] = {H > 0 ? g5::extent((uint64_t)X, 1, T, H, ldx, 0, 2) : none,
                        g5::extent((uint64_t)logits, 1, T, E, ldl, 0, 4),
                        weights ? g5::extent((uint64_t)Wgu, E, 2 * I, H, ldgu, strideGu, ew) : none,
                        weights ? g5::extent((uint64_t)Wd, E, H, I, ldd, strideD, ew) : none,
                        vec_range(scale_gu, E * 2 * I, 4), vec_range(scale_d, E * H, 4)};
    const MoeLayout L = moe_layout(T, H, I, E, topk);
    const Range out[] = {H > 0 ? g5::extent((uint64_t)Y, 1, T, H, ldy, 0, ec) : none, vec_range(ids, T * topk, 4),
                         vec_range(gates, T * topk, 4),
                         workspace ? Range{(__int128)(uint64_t)workspace, (__int128)(uint64_t)workspace + (__int128)L.total}
                                   : none};
    for (const Range &r : in)
        if (r.hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
    if (out[0].hi > ((__int128)1 << 63) || outputs_overlap(out, 4, in, 6)) return GEMM_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < L.total) return GEMM_ERR_WORKSPACE;
    if ((uint64_t)workspace % 256) return GEMM_ERR_INVALID_ARG;
    // (the kernels add 32-bit byte offsets of 16 weight rows and of the token rows)
    if (weights && (ldgu * ew >= (1 << 27) || ldd * ew >= (1 << 27) || ldx * 2 >= (1 << 25))) return GEMM_ERR_UNSUPPORTED;
    const int st = g5::check_device();
    if (st != GEMM_OK) return st;
    char *ws = (char *)workspace;
    g5::MoeArgs a{};
    a.X = X;
    a.logits = logits;
    a.Wgu = Wgu;
    a.Wd = Wd;
    a.scale_gu = scale_gu;
    a.scale_d = scale_d;
    a.Y = Y;
    a.ids = ids;
    a.gates = gates;
    a.T = T;
    a.H = H;
    a.I = I;
    a.E = E;
    a.ldx = ldx;
    a.ldl = ldl;
    a.ldgu = ldgu;
    a.strideGu = strideGu;
    a.ldd = ldd;
    a.strideD = strideD;
    a.ldy = ldy;
    a.topk = (int)topk;
    a.renormalize = renormalize != 0;
    a.out_f32 = ec == 4;
    a.n_items = (int *)(ws + L.n_items);
    a.items = (g5::MoeItem *)(ws + L.items);
    a.pairs = (int32_t *)(ws + L.pairs);
    a.w_ids = (int32_t *)(ws + L.ids);
    a.w_gates = (float *)(ws + L.gates);
    a.z = (uint16_t *)(ws + L.z);
    a.ldz = L.ldz;
    a.zplane = L.zplane;
    a.halves = (float *)(ws + L.halves);
    a.arrived = (unsigned *)(ws + L.arrived);
    const hipError_t e = g5::launch_moe(a, codes, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

// ---- low-rank adapters beside a projection
static int lora_sizes_ok(int64_t L, int64_t R) { return L >= 0 && L <= 0x7fffffff && R >= 0 && R <= 4096; }

int gemm_lora_workspace_size(int64_t M, int64_t N, int64_t K, int64_t L, int64_t R, uint64_t x_addr, int64_t ldx,
                             uint64_t w_addr, int64_t ldw, uint64_t c_addr, int64_t ldc, int c_type, uint64_t *bytes)
{
    if (bytes) *bytes = 0;
    if (!lora_sizes_ok(L, R)) return GEMM_ERR_INVALID_ARG;
    g5::LoraArgs q{};
    q.L = L;
    q.R = R;
    Problem p{GEMM_OP_BF16_NT, 1, M, N, K, x_addr, w_addr, c_addr, ldx, ldw, ldc, 0, 0, 0, c_type};
    if (L > 0 && R > 0) p.lora = &q;
    int st = g5::validate(p);
    if (st != GEMM_OK) return st;
    g5::Plan pl;
    st = g5::select_plan(p, pl, true);
    if (st != GEMM_OK || !bytes || pl.config == g5::CFG_NONE || pl.config == g5::CFG_ZERO) return st;
    const g5::WsLayout W = g5::ws_layout(p, pl);
    size_t need = W.total;
    if (p.lora) g5::lora_layout(p, pl, W, q, &need);
    *bytes = need;
    return GEMM_OK;
}

int gemm_bf16_nt_lora(int64_t M, int64_t N, int64_t K, const uint16_t *X, int64_t ldx, const uint16_t *Wt, int64_t ldw,
                      int64_t L, int64_t R, const uint16_t *A, int64_t lda, int64_t strideA, const uint16_t *B,
                      int64_t ldb, int64_t strideB, const float *scale, const int32_t *idx, void *C, int64_t ldc,
                      int c_type, void *workspace, uint64_t workspace_bytes, void *stream)
{
    using g5::Range;
    if (!lora_sizes_ok(L, R)) return GEMM_ERR_INVALID_ARG;
    Problem p{GEMM_OP_BF16_NT, 1, M, N, K, (uint64_t)X, (uint64_t)Wt, (uint64_t)C, ldx, ldw, ldc, 0, 0, 0, c_type};
    const int st = g5::validate(p);
    if (st != GEMM_OK) return st;
    const bool some = M > 0 && N > 0 && K > 0;
    g5::LoraArgs q{};
    Range in[6] = {};
    if (some) {
        in[0] = g5::extent((uint64_t)X, 1, M, K, ldx, 0, 2);
        in[1] = g5::extent((uint64_t)Wt, 1, N, K, ldw, 0, 2);
    }
    if (some && L > 0 && R > 0) {
        if (!A || !B || !idx || lda < K || ldb < R || strideA < 0 || strideB < 0) return GEMM_ERR_INVALID_ARG;
        if (((uint64_t)A % 2) || ((uint64_t)B % 2) || ((uint64_t)scale % 4) || ((uint64_t)idx % 4))
            return GEMM_ERR_INVALID_ARG;
        in[2] = g5::extent((uint64_t)A, L, R, K, lda, strideA, 2);
        in[3] = g5::extent((uint64_t)B, L, N, R, ldb, strideB, 2);
        in[4] = vec_range(scale, L, 4);
        in[5] = vec_range(idx, M, 4);
        if (in[2].hi > ((__int128)1 << 63) || in[3].hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
        q = g5::LoraArgs{A, B, scale, idx, L, R, lda, strideA, ldb, strideB, 0, 0, 0, nullptr, nullptr, 0, 0, nullptr, nullptr};
        p.lora = &q;
    }
    if (some) {
        uint64_t need = 0;
        const int ws = gemm_lora_workspace_size(M, N, K, L, R, p.a, ldx, p.b, ldw, p.c, ldc, c_type, &need);
        if (ws != GEMM_OK) return ws;
        const Range out[] = {g5::extent((uint64_t)C, 1, M, N, ldc, 0, g5::elem_c(p)),
                             workspace ? Range{(__int128)(uint64_t)workspace, (__int128)(uint64_t)workspace + need}
                                       : Range{0, 0}};
        if (outputs_overlap(out, 2, in, 6)) return GEMM_ERR_INVALID_ARG;
        if (need > 0 && (!workspace || workspace_bytes < need)) return GEMM_ERR_WORKSPACE;
        if ((uint64_t)workspace % 256) return GEMM_ERR_INVALID_ARG;
    }
    return g5::run(p, stream, workspace, (size_t)workspace_bytes);
}

// ---- products grouped by expert
// The part of a workspace that a call of `need` bytes may write (a smaller one
// is refused as such, not as an overlap with what lies behind it).
static g5::Range scratch_range(const void *workspace, uint64_t bytes, uint64_t need)
{
    const __int128 at = (__int128)(uint64_t)workspace;
    return g5::Range{at, at + (__int128)(bytes < need ? bytes : need)};
}

namespace {
struct GroupedPlan {
    int tile = g5::GROUPED_128;
    bool copy_a = false, copy_b = false;
    int64_t lda2 = 0, ldb2 = 0, batch_b = 1, rows_b = 0, cols_a = 0;
    int slices = 1;                      // of a group's rows (TN)
    size_t at_a = 0, at_b = 0, at_sums = 0, total = 0;
};
}  // namespace

static bool grouped_sizes_ok(int kind, int64_t E, int64_t rows, int64_t M, int64_t N, int64_t K)
{
    const int64_t top = (int64_t)1 << 30;
    return kind >= g5::GROUPED_NT && kind <= g5::GROUPED_TN && E >= 0 && E <= g5::kGroupedMaxGroups && rows >= 0 &&
           rows <= 0x7fffffff && M >= 0 && N >= 0 && K >= 0 && M <= top && N <= top && K <= top;
}

// Tile and row copies of a call with work in it.
static int grouped_plan(int kind, int64_t E, int64_t rows, int64_t M, int64_t N, int64_t K, uint64_t a, int64_t lda,
                        uint64_t b, int64_t ldb, int64_t sB, GroupedPlan &pl)
{
    const bool tn = kind == g5::GROUPED_TN, nt = kind == g5::GROUPED_NT;
    pl = GroupedPlan();
    pl.cols_a = tn ? M : K;
    pl.rows_b = nt ? N : tn ? rows : K;
    const int64_t cols_b = nt ? K : N;
    pl.batch_b = tn || sB == 0 ? 1 : E;
    pl.copy_a = g5::row_alignment(a, lda, 0, 1, 2) < 4 || (tn && M % 2 != 0);
    pl.copy_b = g5::row_alignment(b, ldb, sB, pl.batch_b, 2) < 4 || (!nt && N % 2 != 0);
    const bool stream = nt && lda < (1 << 24) && ldb < (1 << 26);
    // The projection of few rows streams the weights past them.  Measured,
    // stream against 128-row tiles: 64 experts of 1536 x 4096, 8 rows each
    // 140 / 142 us, 16 rows 183 / 148; 16 of them 37 / 37 and 55 / 38.  Where
    // tiles leave most CUs idle it carries further (one of 4096 x 4096, 125
    // rows 26 / 37, 200 rows 47 / 36; 4 of 4096 x 1030, 48 rows 14 / 16, 63 rows
    // 20 / 16; 16 of 700 x 1100, 63 rows 14 / 18, 90 rows 23 / 21), and where
    // they would need the weights copied (32 of 1001 x 2001, 31 rows 75 / 101,
    // 48 rows 121 / 104).
    const int64_t tiles = E * g5::cdiv(N, 128);
    const int far = tiles <= g5::kNumCU / 4 ? 128 : tiles <= g5::kNumCU / 2 ? 48 : pl.copy_b ? 32 : 8;
    // Streams past more than 16 rows in the mean: 64 weight rows a workgroup
    // read the group's rows half as often as 32 do, where that leaves a
    // workgroup per CU (16 of 1540 x 4100, 31 rows each 52 us for 64; one of
    // 4096 x 4096, 128 rows 33 for 26).
    const int streamed = rows <= 16 * E                               ? g5::GROUPED_STREAM
                         : E * g5::cdiv(N, 64) >= g5::kNumCU ? g5::GROUPED_STREAM_64x64
                                                                      : g5::GROUPED_STREAM_64x32;
    // Tiles of 256 rows where they keep most CUs busy (128 / 256): 64 experts
    // of 1536 x 4096, 48 rows each 195 / 183 us, 90 rows 202 / 191, 125 rows 239
    // / 195; 8 of 12288 x 4096, 63 rows 169 / 186, 125 rows 241 / 195; 16 of 1540
    // x 4100, 63 rows 56 / 79, 125 rows 105 / 85; 40 of 512 x 1024, 200 rows 22 /
    // 25; the input gradient to 4096 columns, 64 rows each 196 / 167, 16 rows
    // 150 / 144.
    const char *force = std::getenv("GEMM_FORCE_CONFIG");
    if (force && *force) {
        const int id = g5::find_config_by_name(force);
        if (id == g5::CFG_BF16_256x256) pl.tile = g5::GROUPED_256;
        else if (id == g5::CFG_DECODE_NT && stream) pl.tile = streamed;
        else if (id != g5::CFG_BF16_128x128) return GEMM_ERR_UNSUPPORTED;
    } else if (stream && rows <= far * E) {
        pl.tile = streamed;
    } else if (tn ? E * g5::cdiv(M, 256) * g5::cdiv(N, 256) >= g5::kNumCU
                  : rows >= (nt ? 96 : 32) * E && (E + rows / 256) * g5::cdiv(N, 256) >= g5::kNumCU * 5 / 8) {
        pl.tile = g5::GROUPED_256;
    }
    if (g5::grouped_grid(kind, E, rows, M, N, pl.tile) > (int64_t)1 << 22) return GEMM_ERR_UNSUPPORTED;
    // A weight gradient with few tiles over many rows: the rows of a group in
    // slices of at least 512 in the mean, two tiles a CU, as many as 64, whose
    // planes of FP32 sums stay within 24 MiB (one slice / these, us: one group of
    // 30000 rows 64 x 64 282 / 19, 512 x 512 290 / 43, 1024 x 1024 290 / 90; 4528
    // rows 224 x 88 49 / 15; where the rule stays with one, 3000 rows in 4 groups
    // 1000 x 1000 19 / 27, 600 rows 128 x 128 12 / 14).
    if (tn && pl.tile == g5::GROUPED_128) {
        const double plane = 4.0 * E * M * ((N + 3) / 4 * 4);
        int64_t s = 2 * g5::kNumCU / g5::grouped_grid(kind, E, rows, M, N, pl.tile);
        if (s > rows / E / 512) s = rows / E / 512;
        if (s > 64) s = 64;
        if (plane * s > 3 << 23) s = (int64_t)((3 << 23) / plane);
        pl.slices = s < 1 ? 1 : (int)s;
    }
    if (pl.tile != g5::GROUPED_128 && pl.tile != g5::GROUPED_256) {
        pl.copy_a = pl.copy_b = false;
        return GEMM_OK;
    }
    // The tiles copy dwords: rows that start elsewhere, or that end inside one
    // where they lie across the summed axis, are copied to padded ones first.
    pl.lda2 = pl.copy_a ? (pl.cols_a + 7) / 8 * 8 : lda;
    pl.ldb2 = pl.copy_b ? (cols_b + 7) / 8 * 8 : ldb;
    // (32-bit offsets from a tile's own first row: 256 rows, or a piece of 64
    // along the summed axis)
    if (pl.lda2 > (1 << 21) || pl.ldb2 > (1 << 21)) return GEMM_ERR_UNSUPPORTED;
    if (pl.copy_a || pl.copy_b || pl.slices > 1) {
        pl.at_a = g5::kCounterBytes;
        pl.at_b = pl.at_a + (pl.copy_a ? g5::round256((size_t)rows * pl.lda2 * 2) : 0);
        pl.at_sums = pl.at_b + (pl.copy_b ? g5::round256((size_t)pl.batch_b * pl.rows_b * pl.ldb2 * 2) : 0);
        pl.total = pl.at_sums + (pl.slices > 1 ? g5::round256((size_t)pl.slices * E * M * ((N + 3) / 4 * 4) * 4) : 0);
    }
    return GEMM_OK;
}

int gemm_grouped_workspace_size(int kind, int64_t E, int64_t rows, int64_t M, int64_t N, int64_t K, uint64_t a_addr,
                                int64_t lda, uint64_t b_addr, int64_t ldb, int64_t strideB, uint64_t *bytes)
{
    if (bytes) *bytes = 0;
    if (!grouped_sizes_ok(kind, E, rows, M, N, K)) return GEMM_ERR_INVALID_ARG;
    if (E == 0 || N == 0 || rows == 0 || (kind == g5::GROUPED_TN ? M : K) == 0) return GEMM_OK;
    GroupedPlan pl;
    const int st = grouped_plan(kind, E, rows, M, N, K, a_addr, lda, b_addr, ldb, strideB, pl);
    if (st == GEMM_OK && bytes) *bytes = pl.total;
    return st;
}

// M: output rows of TN (else unused); K: the summed axis of NT and NN.
static int grouped_run(int kind, int64_t E, int64_t rows, int64_t M, int64_t N, int64_t K, const int32_t *offsets,
                       const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb, int64_t sB, void *C,
                       int64_t ldc, int64_t sC, int c_type, void *workspace, uint64_t workspace_bytes, void *stream)
{
    using g5::Range;
    const bool tn = kind == g5::GROUPED_TN, nt = kind == g5::GROUPED_NT;
    if (!grouped_sizes_ok(kind, E, rows, M, N, K)) return GEMM_ERR_INVALID_ARG;
    if (c_type != GEMM_OUT_BF16 && c_type != GEMM_OUT_F32) return GEMM_ERR_INVALID_ARG;
    if (E == 0 || N == 0 || (tn ? M == 0 : rows == 0)) return GEMM_OK;
    const int ec = c_type == GEMM_OUT_F32 ? 4 : 2;
    if (!offsets || !C || ((uint64_t)offsets % 4) || ((uint64_t)C % ec) || ldc < N || sB < 0 || sC < 0)
        return GEMM_ERR_INVALID_ARG;
    if (tn && E > 1 && (__int128)sC < (__int128)(M - 1) * ldc + N) return GEMM_ERR_INVALID_ARG;
    const bool some = tn ? rows > 0 : K > 0;        // (else: empty sums)
    const int64_t cols_a = tn ? M : K, rows_b = nt ? N : tn ? rows : K, cols_b = nt ? K : N;
    if (some && (!A || !B || lda < cols_a || ldb < cols_b || ((uint64_t)A % 2) || ((uint64_t)B % 2)))
        return GEMM_ERR_INVALID_ARG;
    const Range none{0, 0};
    const Range in[] = {some ? g5::extent((uint64_t)A, 1, rows, cols_a, lda, 0, 2) : none,
                        some ? g5::extent((uint64_t)B, tn ? 1 : E, rows_b, cols_b, ldb, sB, 2) : none,
                        vec_range(offsets, E + 1, 4)};
    GroupedPlan pl;
    if (some) {
        const int st = grouped_plan(kind, E, rows, M, N, K, (uint64_t)A, lda, (uint64_t)B, ldb, sB, pl);
        if (st != GEMM_OK) return st;
    } else if (g5::grouped_grid(kind, E, rows, M, N, pl.tile) > (int64_t)1 << 22) {
        return GEMM_ERR_UNSUPPORTED;
    }
    const Range out[] = {g5::extent((uint64_t)C, tn ? E : 1, tn ? M : rows, N, ldc, sC, ec),
                         pl.total && workspace
                             ? scratch_range(workspace, workspace_bytes, pl.total)
                             : none};
    for (const Range &r : in)
        if (r.hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
    if (out[0].hi > ((__int128)1 << 63) || outputs_overlap(out, 2, in, 3)) return GEMM_ERR_INVALID_ARG;
    if (pl.total && (!workspace || workspace_bytes < pl.total)) return GEMM_ERR_WORKSPACE;
    if (pl.total && ((uint64_t)workspace % 256)) return GEMM_ERR_INVALID_ARG;
    const int st = g5::check_device();
    if (st != GEMM_OK) return st;
    g5::GroupedArgs a{};
    a.A = A;
    a.B = B;
    a.C = C;
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.M = M;
    a.N = N;
    a.K = K;
    a.lda = some ? lda : 0;
    a.ldb = some ? ldb : 0;
    a.sB = some ? sB : 0;
    a.ldc = ldc;
    a.sC = sC;
    a.align_a = pl.copy_a || !some ? 16 : g5::row_alignment((uint64_t)A, lda, 0, 1, 2);
    a.align_b = pl.copy_b || !some ? 16 : g5::row_alignment((uint64_t)B, ldb, sB, tn ? 1 : E, 2);
    a.align_c = g5::row_alignment((uint64_t)C, ldc, sC, tn ? E : 1, ec);
    a.out_f32 = ec == 4;
    char *ws = (char *)workspace;
    a.slices = pl.slices;
    a.sums = (float *)(ws + pl.at_sums);
    a.ld_sums = (N + 3) / 4 * 4;
    if (pl.copy_a) {
        uint16_t *A2 = (uint16_t *)(ws + pl.at_a);
        if (g5::launch_realign_rows(A, lda, 0, 1, rows, pl.cols_a, g5::row_alignment((uint64_t)A, lda, 0, 1, 2), A2, pl.lda2,
                                    (hipStream_t)stream) != hipSuccess)
            return GEMM_ERR_LAUNCH;
        a.A = A2;
        a.lda = pl.lda2;
    }
    if (pl.copy_b) {
        uint16_t *B2 = (uint16_t *)(ws + pl.at_b);
        if (g5::launch_realign_rows(B, ldb, sB, pl.batch_b, pl.rows_b, cols_b,
                                    g5::row_alignment((uint64_t)B, ldb, sB, pl.batch_b, 2), B2, pl.ldb2,
                                    (hipStream_t)stream) != hipSuccess)
            return GEMM_ERR_LAUNCH;
        a.B = B2;
        a.ldb = pl.ldb2;
        a.sB = pl.batch_b > 1 ? pl.rows_b * pl.ldb2 : 0;
    }
    const int64_t widest = tn && a.lda > a.ldb ? a.lda : a.ldb;
    a.piece = widest > 0 ? (((int64_t)1 << 29) / widest) / 64 * 64 : 32;
    const hipError_t e = g5::launch_grouped(kind, a, pl.tile, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

int gemm_bf16_grouped_nt(int64_t E, int64_t M, int64_t N, int64_t K, const int32_t *offsets, const uint16_t *A,
                         int64_t lda, const uint16_t *Bt, int64_t ldbt, int64_t strideBt, void *C, int64_t ldc,
                         int c_type, void *workspace, uint64_t workspace_bytes, void *stream)
{
    return grouped_run(g5::GROUPED_NT, E, M, 0, N, K, offsets, A, lda, Bt, ldbt, strideBt, C, ldc, 0, c_type, workspace,
                       workspace_bytes, stream);
}

int gemm_bf16_grouped(int64_t E, int64_t M, int64_t N, int64_t K, const int32_t *offsets, const uint16_t *A,
                      int64_t lda, const uint16_t *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc, int c_type,
                      void *workspace, uint64_t workspace_bytes, void *stream)
{
    return grouped_run(g5::GROUPED_NN, E, M, 0, N, K, offsets, A, lda, B, ldb, strideB, C, ldc, 0, c_type, workspace,
                       workspace_bytes, stream);
}

int gemm_bf16_grouped_tn(int64_t E, int64_t rows, int64_t M, int64_t N, const int32_t *offsets, const uint16_t *At,
                         int64_t ldat, const uint16_t *B, int64_t ldb, void *C, int64_t ldc, int64_t strideC,
                         int c_type, void *workspace, uint64_t workspace_bytes, void *stream)
{
    return grouped_run(g5::GROUPED_TN, E, rows, M, N, 0, offsets, At, ldat, B, ldb, 0, C, ldc, strideC, c_type, workspace,
                       workspace_bytes, stream);
}

// ---- the loss over a vocabulary behind the last projection
namespace {
// Scratch of a call, behind the counter region, each part 256-byte aligned.
struct VocabPlan {
    int tile = 128;                      // 256, 128, or 0: the stream (forward)
    int64_t piece = 0, parts = 0;        // vocabulary rows at a time; column tiles (forward)
    bool copy_x = false, copy_w = false;
    int64_t ld2 = 0;                     // row length of the copies
    int parts_d = 1;                     // of D (gradient)
    int tile_x = 128, tile_w = 128;      // of dX's and dW's products
    int slices = 1, w_slices = 1;        // of a piece's tokens in dX's product, of the rows in dW's
    int64_t per = 0, w_per = 0;          // tokens, rows in each
    size_t x2 = 0, w2 = 0, part = 0, zt = 0, d = 0, sums = 0, w_sums = 0, ids = 0, q = 0, has = 0, weight = 0, alpha = 0, total = 0;
};
struct VocabCall {
    bool grad;
    int64_t M, V, K, topk;
    uint64_t x;
    int64_t ldx;
    uint64_t w;
    int64_t ldw;
};
}  // namespace

static bool vocab_sizes_ok(const VocabCall &c)
{
    return c.M >= 0 && c.M <= 1 << 24 && c.V >= 1 && c.V <= 0x7fffffff - 256 && c.K >= 1 && c.K <= 1 << 21 && c.topk >= 1 &&
           c.topk <= g5::kVocabMaxTopk;
}

// The tile with the shorter time: rounds of workgroups (one of 256 rows per CU,
// two of 128) times what a tile takes beside its stages of 64 and per stage,
// in us, fitted to the measured (tiles of 128 / 256): the loss's logits of 3594
// x 4740 x 128 20 / 25, 300 x 100000 x 128 29 / 36, 4096 x 32768 x 512 177 / 135,
// 700 x 9000 x 700 22 / 27, 3000 x 3000 x 1000 42 / 36; D of the first 24 / 36,
// of the third 198 / 188; dW of 131072 x 4096 from 2, 120, 500 and 1000 rows 242
// / 276, 420 / 347, 853 / 689 and 1410 / 1101.
enum VocabProduct { VOCAB_STATS, VOCAB_D, VOCAB_DW };
static int vocab_tile(VocabProduct what, int64_t M, int64_t N, int64_t K)
{
    struct Cost {
        double start, tile, stage, rest;     // per kernel, tile, stage of 64, and a K that ends inside one
    };
    static const Cost kBig[] = {{8, 4, 1.45, 5}, {8, 9, 1.45, 5}, {0, 8.3, 1.63, 0}};
    static const Cost kSmall[] = {{6, 2.3, 1.05, 5}, {6, 3.6, 1.05, 5}, {0, 3.8, 1.15, 0}};
    const double stages = (double)g5::cdiv(K, 64), rest = K % 64 != 0;
    const int64_t t256 = g5::cdiv(M, 256) * g5::cdiv(N, 256), t128 = g5::cdiv(M, 128) * g5::cdiv(N, 128);
    const Cost &b = kBig[what], &s = kSmall[what];
    const double big = b.start + (double)g5::cdiv(t256, g5::kNumCU) * (b.tile + b.stage * stages + b.rest * rest);
    // (a CU with one tile of 128 goes through it faster than one with two)
    const double small = s.start + (double)g5::cdiv(t128, 2 * g5::kNumCU) *
                                       (s.tile + (t128 <= g5::kNumCU ? 0.75 : s.stage) * stages + s.rest * rest);
    return big < small ? 256 : 128;
}

static int vocab_plan(const VocabCall &c, VocabPlan &pl)
{
    pl = VocabPlan();
    pl.ld2 = (c.K + 7) / 8 * 8;
    const int align_x = g5::row_alignment(c.x, c.ldx, 0, 1, 2), align_w = g5::row_alignment(c.w, c.ldw, 0, 1, 2);
    const size_t CR = g5::kCounterBytes;
    size_t at = CR;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += g5::round256(bytes);
        return here;
    };
    const bool stream = c.M <= g5::kVocabStreamRows && c.ldx < (1 << 24) && c.ldw < (1 << 26);
    const char *force = std::getenv("GEMM_FORCE_CONFIG");
    int forced = -1;                     // 0: the stream
    if (force && *force) {
        const int id = g5::find_config_by_name(force);
        forced = id == g5::CFG_BF16_256x256 ? 256 : id == g5::CFG_BF16_128x128 ? 128 : id == g5::CFG_DECODE_NT ? 0 : -1;
        if (forced < 0 || (forced == 0 && !stream)) return GEMM_ERR_UNSUPPORTED;
    }
    pl.tile = forced >= 0 ? forced : stream ? 0 : vocab_tile(c.grad ? VOCAB_D : VOCAB_STATS, c.M, c.V, c.K);
    if (!c.grad && pl.tile == 0) {
        pl.piece = c.V;
        pl.parts = g5::cdiv(c.V, 32);
        if (pl.parts > (int64_t)1 << 23) return GEMM_ERR_UNSUPPORTED;
    } else {
        pl.copy_x = c.grad || align_x < 4;
        // (dX's product reads W's rows in whole dwords)
        pl.copy_w = align_w < 4 || (c.grad && c.K % 2 != 0);
        const int64_t ldw = pl.copy_w ? pl.ld2 : c.ldw;
        if (c.ldx > 1 << 21 || ldw > 1 << 21) return GEMM_ERR_UNSUPPORTED;
        // A piece: D of 2^27 elements (256 MiB, the Infinity Cache's size), the
        // copy of W as many, and W's rows and 64 of D's within 32-bit offsets
        // (each such limit at least 256 tokens, the rounding's).
        int64_t rows = c.V;
        const int64_t cache = (int64_t)1 << 27;
        if (c.grad && c.M > 0 && rows > cache / c.M) rows = cache / c.M;
        if (pl.copy_w && rows > cache / pl.ld2) rows = cache / pl.ld2;
        if (c.grad && rows > g5::kVocabReach / ldw) rows = g5::kVocabReach / ldw;
        if (c.grad && rows > g5::kVocabMaxPiece) rows = g5::kVocabMaxPiece;
        if (rows < c.V) rows = rows < 256 ? 256 : rows / 256 * 256;
        pl.piece = rows < c.V ? rows : c.V;
        pl.parts = pl.tile ? g5::cdiv(c.V, pl.tile) : 0;
        if (g5::cdiv(c.M, 128) * g5::cdiv(pl.piece, 128) > (int64_t)1 << 22 ||
            g5::cdiv(pl.piece, 128) * g5::cdiv(c.K, 128) > (int64_t)1 << 22)
            return GEMM_ERR_UNSUPPORTED;
    }
    if (c.grad) {
        pl.parts_d = c.M <= g5::kVocabSplitRows ? 2 : 1;
        const int64_t rows = c.M * pl.parts_d;
        pl.tile_w = forced > 0 ? forced : vocab_tile(VOCAB_DW, pl.piece, c.K, rows);
        pl.tile_x = forced > 0 ? forced : rows > 128 ? 256 : 128;
        // Output tiles shared out over slices of the summed axis until every
        // CU has one (two of 128): dX's, as many as 64 of at least 256 tokens,
        // and dW's, as many as 16 of at least 512 rows, while the planes of
        // sums stay within a quarter of the Infinity Cache.
        const auto slots = [](int tile) { return (tile == 256 ? 1 : 2) * (int64_t)g5::kNumCU; };
        const auto slices = [](int64_t most, int64_t tiles, int64_t slots, int64_t len, int64_t least, double plane) {
            int64_t s = slots / tiles;
            if (s > len / least) s = len / least;
            if (plane * s > (1 << 26)) s = (int64_t)((1 << 26) / plane);
            return s > most ? most : s < 1 ? 1 : s;
        };
        const int64_t tiles_x = g5::cdiv(rows, pl.tile_x) * g5::cdiv(pl.ld2, pl.tile_x);
        const int64_t sx = slices(64, tiles_x, slots(pl.tile_x), pl.piece, 256, 4.0 * rows * pl.ld2);
        pl.per = g5::cdiv(g5::cdiv(pl.piece, sx), 32) * 32;
        pl.slices = (int)g5::cdiv(pl.piece, pl.per);
        const int64_t tiles_w = g5::cdiv(pl.piece, pl.tile_w) * g5::cdiv(c.K, pl.tile_w);
        const int64_t sw = slices(16, tiles_w, slots(pl.tile_w), rows, 512, 4.0 * pl.piece * pl.ld2);
        pl.w_per = g5::cdiv(g5::cdiv(rows, sw), 64) * 64;
        pl.w_slices = (int)g5::cdiv(rows, pl.w_per);
        if (tiles_x * pl.slices > (int64_t)1 << 22) return GEMM_ERR_UNSUPPORTED;
    }
    if (pl.copy_x) pl.x2 = take((size_t)c.M * pl.parts_d * pl.ld2 * 2);
    if (pl.copy_w) pl.w2 = take((size_t)pl.piece * pl.ld2 * 2);
    if (!c.grad) {
        pl.part = take((size_t)pl.parts * c.M * 8);
        pl.zt = take((size_t)c.M * c.topk * 4);
    } else {
        pl.d = take((size_t)c.M * pl.parts_d * ((pl.piece + 7) / 8 * 8) * 2);
        pl.sums = take((size_t)pl.slices * c.M * pl.parts_d * pl.ld2 * 4);
        if (pl.w_slices > 1) pl.w_sums = take((size_t)pl.w_slices * pl.piece * pl.ld2 * 4);
        pl.ids = take((size_t)c.M * c.topk * 4);
        pl.q = take((size_t)c.M * c.topk * 4);
        pl.has = take((size_t)c.M * 4);
        pl.weight = take((size_t)c.M * 4);
        pl.alpha = take(4);
    }
    pl.total = at;
    return GEMM_OK;
}

int gemm_linear_loss_workspace_size(int backward, int64_t M, int64_t V, int64_t K, int64_t topk, uint64_t x_addr,
                                    int64_t ldx, uint64_t w_addr, int64_t ldw, uint64_t *bytes)
{
    if (bytes) *bytes = 0;
    const VocabCall c{backward != 0, M, V, K, topk, x_addr, ldx, w_addr, ldw};
    if (!vocab_sizes_ok(c)) return GEMM_ERR_INVALID_ARG;
    if (M == 0) return GEMM_OK;
    VocabPlan pl;
    const int st = vocab_plan(c, pl);
    if (st == GEMM_OK && bytes) *bytes = pl.total;
    return st;
}

// teacher NULL: ids are labels (topk 1).
static int vocab_check(const VocabCall &c, const uint16_t *X, const uint16_t *W, float scale, const void *ids,
                       int id_bytes, g5::Range (&in)[6], const float *teacher)
{
    if (!vocab_sizes_ok(c) || !std::isfinite(scale) || !(scale > 0.0f) || (id_bytes != 4 && id_bytes != 8))
        return GEMM_ERR_INVALID_ARG;
    if (c.M > 0 && (!X || !W || !ids || c.ldx < c.K || c.ldw < c.K || (c.x % 2) || (c.w % 2) ||
                    ((uint64_t)ids % id_bytes) || ((uint64_t)teacher % 4)))
        return GEMM_ERR_INVALID_ARG;
    if (c.M == 0) return GEMM_OK;
    in[0] = g5::extent(c.x, 1, c.M, c.K, c.ldx, 0, 2);
    in[1] = g5::extent(c.w, 1, c.V, c.K, c.ldw, 0, 2);
    in[2] = vec_range(ids, c.M * c.topk, id_bytes);
    in[3] = vec_range(teacher, c.M * c.topk, 4);
    return in[0].hi > ((__int128)1 << 63) || in[1].hi > ((__int128)1 << 63) ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

static g5::VocabArgs vocab_args(const VocabCall &c, const uint16_t *X, const uint16_t *W, float scale, const void *ids,
                                int id_bytes, const float *teacher)
{
    g5::VocabArgs a{};
    a.X = X;
    a.W = W;
    a.M = c.M;
    a.V = a.vocab = c.V;
    a.K = c.K;
    a.ldx = c.ldx;
    a.ldw = c.ldw;
    a.align_x = g5::row_alignment(c.x, c.ldx, 0, 1, 2);
    a.scale = scale;
    a.ids = ids;
    a.ids64 = id_bytes == 8;
    a.topk = (int)c.topk;
    a.teacher = teacher;
    return a;
}

// The rows of W of the piece that starts at v0, as they are or copied.
static hipError_t vocab_piece(const VocabCall &c, const VocabPlan &pl, char *ws, const uint16_t *W, int64_t v0,
                              g5::VocabArgs &a, hipStream_t s)
{
    a.v0 = v0;
    a.align_w = pl.copy_w ? 16 : g5::row_alignment(c.w, c.ldw, 0, 1, 2);
    a.V = c.V - v0 < pl.piece ? c.V - v0 : pl.piece;
    a.W = W + v0 * c.ldw;
    a.ldw = c.ldw;
    if (!pl.copy_w) return hipSuccess;
    uint16_t *W2 = (uint16_t *)(ws + pl.w2);
    const hipError_t e = g5::launch_realign_rows(a.W, c.ldw, 0, 1, a.V, c.K, g5::row_alignment(c.w, c.ldw, 0, 1, 2), W2,
                                                 pl.ld2, s);
    a.W = W2;
    a.ldw = pl.ld2;
    return e;
}

static int vocab_forward(const VocabCall &c, const uint16_t *X, const uint16_t *W, float scale, const void *ids,
                         int id_bytes, const float *teacher, float *loss, float *lse, void *workspace,
                         uint64_t workspace_bytes, void *stream)
{
    using g5::Range;
    Range in[6] = {};
    int st = vocab_check(c, X, W, scale, ids, id_bytes, in, teacher);
    if (st != GEMM_OK || c.M == 0) return st;
    if (!loss || ((uint64_t)loss % 4) || ((uint64_t)lse % 4)) return GEMM_ERR_INVALID_ARG;
    VocabPlan pl;
    st = vocab_plan(c, pl);
    if (st != GEMM_OK) return st;
    const Range out[] = {vec_range(loss, c.M, 4), vec_range(lse, c.M, 4),
                         workspace ? scratch_range(workspace, workspace_bytes, pl.total)
                                   : Range{0, 0}};
    if (outputs_overlap(out, 3, in, 4)) return GEMM_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < pl.total) return GEMM_ERR_WORKSPACE;
    if ((uint64_t)workspace % 256) return GEMM_ERR_INVALID_ARG;
    st = g5::check_device();
    if (st != GEMM_OK) return st;
    char *ws = (char *)workspace;
    const hipStream_t s = (hipStream_t)stream;
    g5::VocabArgs a = vocab_args(c, X, W, scale, ids, id_bytes, teacher);
    a.part = (float2 *)(ws + pl.part);
    a.zt = (float *)(ws + pl.zt);
    a.parts = pl.parts;
    a.loss = loss;
    a.lse_out = lse;
    if (pl.copy_x) {
        uint16_t *X2 = (uint16_t *)(ws + pl.x2);
        if (g5::launch_realign_rows(X, c.ldx, 0, 1, c.M, c.K, g5::row_alignment(c.x, c.ldx, 0, 1, 2), X2, pl.ld2, s) !=
            hipSuccess)
            return GEMM_ERR_LAUNCH;
        a.X = X2;
        a.ldx = pl.ld2;
        a.align_x = 16;
    }
    for (int64_t v0 = 0; v0 < c.V; v0 += pl.piece) {
        if (vocab_piece(c, pl, ws, W, v0, a, s) != hipSuccess) return GEMM_ERR_LAUNCH;
        a.tile0 = pl.tile ? v0 / pl.tile : 0;
        if (g5::launch_vocab_stats(a, pl.tile, s) != hipSuccess) return GEMM_ERR_LAUNCH;
    }
    return g5::launch_vocab_join(a, s) == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}

static int vocab_backward(const VocabCall &c, const uint16_t *X, const uint16_t *W, float scale, const void *ids,
                          int id_bytes, const float *teacher, const float *dloss, const float *lse, uint16_t *dX,
                          int64_t lddx, void *dW, int64_t lddw, int dw_type, void *workspace,
                          uint64_t workspace_bytes, void *stream)
{
    using g5::Range;
    Range in[6] = {};
    int st = vocab_check(c, X, W, scale, ids, id_bytes, in, teacher);
    if (st != GEMM_OK) return st;
    if (dw_type != GEMM_OUT_BF16 && dw_type != GEMM_OUT_F32) return GEMM_ERR_INVALID_ARG;
    const int ew = dw_type == GEMM_OUT_F32 ? 4 : 2;
    if (c.M == 0) dX = nullptr;
    if (!dX && !dW) return GEMM_OK;
    if ((c.M > 0 && (!dloss || !lse || ((uint64_t)dloss % 4) || ((uint64_t)lse % 4))) || (dX && (lddx < c.K || ((uint64_t)dX % 2))) ||
        (dW && (lddw < c.K || ((uint64_t)dW % ew))))
        return GEMM_ERR_INVALID_ARG;
    const Range none{0, 0};
    in[4] = c.M > 0 ? vec_range(dloss, c.M, 4) : none;
    in[5] = c.M > 0 ? vec_range(lse, c.M, 4) : none;
    VocabPlan pl;
    if (c.M > 0) {
        st = vocab_plan(c, pl);
        if (st != GEMM_OK) return st;
    } else if (g5::cdiv(c.V, 128) * g5::cdiv(c.K, 128) > (int64_t)1 << 22) {
        return GEMM_ERR_UNSUPPORTED;
    }
    const Range out[] = {dX ? g5::extent((uint64_t)dX, 1, c.M, c.K, lddx, 0, 2) : none,
                         dW ? g5::extent((uint64_t)dW, 1, c.V, c.K, lddw, 0, ew) : none,
                         c.M > 0 && workspace
                             ? scratch_range(workspace, workspace_bytes, pl.total)
                             : none};
    for (const Range &r : out)
        if (r.hi > ((__int128)1 << 63)) return GEMM_ERR_INVALID_ARG;
    if (outputs_overlap(out, 3, in, 6)) return GEMM_ERR_INVALID_ARG;
    if (c.M > 0 && (!workspace || workspace_bytes < pl.total)) return GEMM_ERR_WORKSPACE;
    if (c.M > 0 && ((uint64_t)workspace % 256)) return GEMM_ERR_INVALID_ARG;
    st = g5::check_device();
    if (st != GEMM_OK) return st;
    char *ws = (char *)workspace;
    const hipStream_t s = (hipStream_t)stream;
    g5::VocabArgs a = vocab_args(c, X, W, scale, ids, id_bytes, teacher);
    g5::VocabGrad b{};
    b.dX = dX;
    b.lddx = lddx;
    b.dW = dW;
    b.lddw = lddw;
    b.dw_f32 = ew == 4;
    b.ldx2 = (c.K + 7) / 8 * 8;
    b.rows_at_once = b.w_per = 64;
    b.parts = b.w_slices = 1;
    if (c.M == 0) {                  // the empty sum
        a.V = c.V;
        return g5::launch_vocab_dw(a, b, 128, s) == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
    }
    b.dloss = dloss;
    b.lse = lse;
    b.ids = (int32_t *)(ws + pl.ids);
    b.has = (int32_t *)(ws + pl.has);
    b.q = (float *)(ws + pl.q);
    b.weight = (float *)(ws + pl.weight);
    b.alpha = (float *)(ws + pl.alpha);
    b.X2 = (uint16_t *)(ws + pl.x2);
    b.D = (uint16_t *)(ws + pl.d);
    b.ldd = (pl.piece + 7) / 8 * 8;
    b.parts = pl.parts_d;
    b.sums = (float *)(ws + pl.sums);
    b.slices = pl.slices;
    b.per = pl.per;
    b.w_slices = pl.w_slices;
    b.w_per = pl.w_per;
    b.w_sums = (float *)(ws + pl.w_sums);
    const int64_t widest = b.ldd > b.ldx2 ? b.ldd : b.ldx2;
    b.rows_at_once = g5::kVocabReach / widest / 64 * 64;     // (64 at least: neither exceeds kVocabMaxPiece)
    if (g5::launch_vocab_prep(a, b, s) != hipSuccess) return GEMM_ERR_LAUNCH;
    a.X = b.X2;                       // (the stream's rows of X too: at most kVocabStreamRows of them)
    a.ldx = b.ldx2;
    a.align_x = 16;
    for (int64_t v0 = 0; v0 < c.V; v0 += pl.piece) {
        if (vocab_piece(c, pl, ws, W, v0, a, s) != hipSuccess) return GEMM_ERR_LAUNCH;
        if (g5::launch_vocab_dlogits(a, b, pl.tile, s) != hipSuccess) return GEMM_ERR_LAUNCH;
        if (dW && g5::launch_vocab_dw(a, b, pl.tile_w, s) != hipSuccess) return GEMM_ERR_LAUNCH;
        b.more = v0 > 0;
        if (dX && g5::launch_vocab_sums(a, b, pl.tile_x, s) != hipSuccess) return GEMM_ERR_LAUNCH;
    }
    if (dX && g5::launch_vocab_dx(a, b, s) != hipSuccess) return GEMM_ERR_LAUNCH;
    return GEMM_OK;
}

int gemm_linear_cross_entropy(int64_t M, int64_t V, int64_t K, const uint16_t *X, int64_t ldx, const uint16_t *Wt,
                              int64_t ldw, float scale, const void *targets, int index_bytes, float *loss, float *lse,
                              void *workspace, uint64_t workspace_bytes, void *stream)
{
    const VocabCall c{false, M, V, K, 1, (uint64_t)X, ldx, (uint64_t)Wt, ldw};
    return vocab_forward(c, X, Wt, scale, targets, index_bytes, nullptr, loss, lse, workspace, workspace_bytes, stream);
}

int gemm_linear_cross_entropy_backward(int64_t M, int64_t V, int64_t K, const uint16_t *X, int64_t ldx,
                                       const uint16_t *Wt, int64_t ldw, float scale, const void *targets,
                                       int index_bytes, const float *dloss, const float *lse, uint16_t *dX,
                                       int64_t lddx, void *dW, int64_t lddw, int dw_type, void *workspace,
                                       uint64_t workspace_bytes, void *stream)
{
    const VocabCall c{true, M, V, K, 1, (uint64_t)X, ldx, (uint64_t)Wt, ldw};
    return vocab_backward(c, X, Wt, scale, targets, index_bytes, nullptr, dloss, lse, dX, lddx, dW, lddw, dw_type, workspace,
                          workspace_bytes, stream);
}

int gemm_linear_distill(int64_t M, int64_t V, int64_t K, const uint16_t *X, int64_t ldx, const uint16_t *Wt,
                        int64_t ldw, float scale, int64_t topk, const void *ids, int index_bytes,
                        const float *teacher, float *loss, float *lse, void *workspace, uint64_t workspace_bytes,
                        void *stream)
{
    const VocabCall c{false, M, V, K, topk, (uint64_t)X, ldx, (uint64_t)Wt, ldw};
    if (M > 0 && !teacher) return GEMM_ERR_INVALID_ARG;
    return vocab_forward(c, X, Wt, scale, ids, index_bytes, teacher, loss, lse, workspace, workspace_bytes, stream);
}

int gemm_linear_distill_backward(int64_t M, int64_t V, int64_t K, const uint16_t *X, int64_t ldx, const uint16_t *Wt,
                                 int64_t ldw, float scale, int64_t topk, const void *ids, int index_bytes,
                                 const float *teacher, const float *dloss, const float *lse, uint16_t *dX,
                                 int64_t lddx, void *dW, int64_t lddw, int dw_type, void *workspace,
                                 uint64_t workspace_bytes, void *stream)
{
    const VocabCall c{true, M, V, K, topk, (uint64_t)X, ldx, (uint64_t)Wt, ldw};
    if (M > 0 && !teacher) return GEMM_ERR_INVALID_ARG;
    return vocab_backward(c, X, Wt, scale, ids, index_bytes, teacher, dloss, lse, dX, lddx, dW, lddw, dw_type, workspace,
                          workspace_bytes, stream);
}

const char *gemm_status_string(int status)
{
    switch (status) {
    case GEMM_OK: return "GEMM_OK: success";
    case GEMM_ERR_INVALID_ARG: return "GEMM_ERR_INVALID_ARG: invalid size, stride, pointer, output type or overlap";
    case GEMM_ERR_UNSUPPORTED: return "GEMM_ERR_UNSUPPORTED: no compiled kernel configuration can run this call";
    case GEMM_ERR_LAUNCH: return "GEMM_ERR_LAUNCH: kernel launch failed";
    case GEMM_ERR_NO_DEVICE: return "GEMM_ERR_NO_DEVICE: no usable HIP device is current (none, or not gfx950)";
    case GEMM_ERR_WORKSPACE:
        return "GEMM_ERR_WORKSPACE: the workspace passed is smaller than the call needs (gemm_workspace_size)";
    default: return "unknown gemm status";
    }
}

static int plan_query_impl(int with_workspace, int op, int64_t batch, int64_t M, int64_t N, int64_t K,
                           uint64_t a_addr, int64_t lda, int64_t strideA, uint64_t b_addr, int64_t ldb,
                           int64_t strideB, uint64_t c_addr, int64_t ldc, int64_t strideC, int c_type,
                           gemm_plan *out)
{
    Problem p{op, batch, M, N, K, a_addr, b_addr, c_addr, lda, ldb, ldc, strideA, strideB, strideC,
              g5::op_c_type(op, c_type)};
    if (p.c_type == GEMM_OUT_E4M3) p.out_amax = 1.0f;   // (the range does not change the plan)
    int st = g5::validate(p);
    if (st != GEMM_OK) return st;
    g5::Plan pl;
    st = g5::select_plan(p, pl, with_workspace != 0);
    if (st != GEMM_OK) return st;
    g5::fill_public_plan(p, pl, out);
    return GEMM_OK;
}

int gemm_plan_query(int op, int64_t batch, int64_t M, int64_t N, int64_t K, uint64_t a_addr, int64_t lda,
                    int64_t strideA, uint64_t b_addr, int64_t ldb, int64_t strideB, uint64_t c_addr, int64_t ldc,
                    int64_t strideC, int c_type, gemm_plan *out)
{
    return plan_query_impl(1, op, batch, M, N, K, a_addr, lda, strideA, b_addr, ldb, strideB, c_addr, ldc, strideC,
                           c_type, out);
}

int gemm_plan_query_ex(int with_workspace, int op, int64_t batch, int64_t M, int64_t N, int64_t K, uint64_t a_addr,
                       int64_t lda, int64_t strideA, uint64_t b_addr, int64_t ldb, int64_t strideB, uint64_t c_addr,
                       int64_t ldc, int64_t strideC, int c_type, gemm_plan *out)
{
    return plan_query_impl(with_workspace, op, batch, M, N, K, a_addr, lda, strideA, b_addr, ldb, strideB, c_addr,
                           ldc, strideC, c_type, out);
}

int gemm_workspace_size(int op, int64_t batch, int64_t M, int64_t N, int64_t K, uint64_t a_addr, int64_t lda,
                        int64_t strideA, uint64_t b_addr, int64_t ldb, int64_t strideB, uint64_t c_addr, int64_t ldc,
                        int64_t strideC, int c_type, uint64_t *bytes)
{
    gemm_plan pl;
    const int st = plan_query_impl(1, op, batch, M, N, K, a_addr, lda, strideA, b_addr, ldb, strideB, c_addr, ldc,
                                   strideC, c_type, &pl);
    if (bytes) *bytes = st == GEMM_OK ? (uint64_t)pl.workspace_bytes : 0;
    return st;
}

static g5::Problem run_problem(int op, int64_t batch, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                               int64_t strideA, const void *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc,
                               int64_t strideC, int c_type, float alpha, const uint16_t *bias, float beta,
                               const float *scale_a, const float *scale_b)
{
    Problem p{op, batch, M, N, K, (uint64_t)A, (uint64_t)B, (uint64_t)C, lda, ldb, ldc, strideA, strideB, strideC,
              g5::op_c_type(op, c_type)};
    if (p.c_type == GEMM_OUT_E4M3) p.out_amax = alpha;   // SwiGLU's fixed range
    if (op == GEMM_OP_FP8_NT || op == GEMM_OP_FP8_NT_AFFINE) {
        p.scale_a = (uint64_t)scale_a;
        p.scale_b = (uint64_t)scale_b;
    }
    if (op == GEMM_OP_BF16_AFFINE || op == GEMM_OP_BF16_NT_AFFINE || op == GEMM_OP_BF16_TN_AFFINE ||
        op == GEMM_OP_FP8_NT_AFFINE) {
        p.alpha = alpha;
        p.beta = beta;
        p.bias = (uint64_t)bias;
    }
    return p;
}

int gemm_run(int op, int64_t batch, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda, int64_t strideA,
             const void *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc, int64_t strideC, int c_type,
             float alpha, const uint16_t *bias, float beta, const float *scale_a, const float *scale_b,
             void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (op < GEMM_OP_SGEMM || op > GEMM_OP_FP8_NT_AFFINE) return GEMM_ERR_INVALID_ARG;
    if (op == GEMM_OP_SGEMM && batch != 1) return GEMM_ERR_INVALID_ARG;
    const Problem p = run_problem(op, batch, M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, c_type, alpha,
                                  bias, beta, scale_a, scale_b);
    return g5::run(p, stream, workspace, (size_t)workspace_bytes);
}

int gemm_run_noalloc(int op, int64_t batch, int64_t M, int64_t N, int64_t K, const void *A, int64_t lda,
                     int64_t strideA, const void *B, int64_t ldb, int64_t strideB, void *C, int64_t ldc,
                     int64_t strideC, int c_type, float alpha, const uint16_t *bias, float beta,
                     const float *scale_a, const float *scale_b, void *stream)
{
    if (op < GEMM_OP_SGEMM || op > GEMM_OP_FP8_NT_AFFINE) return GEMM_ERR_INVALID_ARG;
    if (op == GEMM_OP_SGEMM && batch != 1) return GEMM_ERR_INVALID_ARG;
    const Problem p = run_problem(op, batch, M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, c_type, alpha,
                                  bias, beta, scale_a, scale_b);
    int st = g5::validate(p);
    if (st != GEMM_OK) return st;
    g5::Plan pl;
    st = g5::select_plan(p, pl, true);
    if (st != GEMM_OK) return st;
    if (pl.config == g5::CFG_NONE) return GEMM_OK;
    if (g5::ws_layout(p, pl).total > g5::kScratchBytes) return GEMM_ERR_WORKSPACE;
    st = g5::check_device();
    if (st != GEMM_OK) return st;
    void *scratch = nullptr;
    if (g5::noalloc_scratch(&scratch) != hipSuccess) return GEMM_ERR_LAUNCH;
    // The scratch keeps the last call's contents: the arrival counters this
    // call uses are cleared first (every call leaves them zero, but a call
    // that overlapped another on this GPU may not have).
    if (g5::launch_clear_counters(scratch, g5::counters_used(p, pl), (hipStream_t)stream) != hipSuccess)
        return GEMM_ERR_LAUNCH;
    return g5::run(p, stream, scratch, g5::kScratchBytes);
}

int64_t gemm_model_local_bytes(int64_t m, int64_t n, int64_t k, int64_t elem_bytes)
{
    return elem_bytes * m * k + elem_bytes * k * n + 4 * m * n;
}

double gemm_model_traffic_bytes(int64_t M, int64_t N, int64_t K, int64_t m, int64_t n, int64_t elem_bytes)
{
    if (m <= 0 || n <= 0) return 0.0;
    const double e = (double)elem_bytes;
    return e * M * K * (double)((N + n - 1) / n) + e * K * N * (double)((M + m - 1) / m) + e * M * N;
}

void gemm_model_quant_traffic(int64_t M, int64_t N, int64_t K, int64_t m, int64_t n, int64_t in_bytes,
                              int64_t q_bytes, int64_t w_bytes, int64_t out_bytes, double *separate, double *fused)
{
    double sep = 0.0, fus = 0.0;
    if (m > 0 && n > 0 && M >= 0 && N >= 0 && K >= 0) {
        const double in = (double)in_bytes * M * K, q = (double)q_bytes * M * K;
        const double col_blocks = (double)((N + n - 1) / n), row_blocks = (double)((M + m - 1) / m);
        const double common = row_blocks * w_bytes * (double)K * N + (double)out_bytes * M * N;
        sep = in + q + col_blocks * q + common;     // read once, write the codes, each column block reads them
        fus = in + col_blocks * in + common;        // read once for the factors, each column block re-reads it
    }
    if (separate) *separate = sep;
    if (fused) *fused = fus;
}

double gemm_model_act_chain_bytes(int step, int64_t M, int64_t N)
{
    // bytes per element: the inputs read plus the output written
    static const int kPerElem[5] = {2 + 2, 2 + 2 + 2, 2 + 2 + 2, 2 + 1, 2 + 2 + 1};
    if (step < GEMM_ACT_SILU || step > GEMM_ACT_SWIGLU_E4M3 || M < 0 || N < 0) return 0.0;
    return (double)kPerElem[step] * (double)M * (double)N;
}

int gemm_tile_map(int64_t wg, int64_t batch, int64_t tiles_m, int64_t tiles_n, int64_t group_m, int64_t *b,
                  int64_t *tm, int64_t *tn)
{
    if (batch <= 0 || tiles_m <= 0 || tiles_n <= 0 || group_m < -tiles_m || wg < 0 ||
        wg >= batch * tiles_m * tiles_n || !b || !tm || !tn)
        return -1;
    const g5::TileCoord t = g5::tile_map(wg, batch, tiles_m, tiles_n, group_m);
    *b = t.b;
    *tm = t.tm;
    *tn = t.tn;
    return 0;
}

}  // extern "C"
