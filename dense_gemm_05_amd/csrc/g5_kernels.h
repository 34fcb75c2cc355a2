// g5_kernels.h -- launch entry of the gfx950 kernels (host side).
#pragma once

#include <hip/hip_runtime.h>

#include "g5_common.h"

namespace g5 {

// Enqueue compiled configuration `config_id` on stream `s` with `grid`
// workgroups.  `variant` selects the kernel variant (tiled configs: 0 fully
// general, 1 aligned without edge masking, 2/3 masked ring kernel copying A in
// 16- or 4-byte pieces); the caller guarantees its preconditions.  Returns the
// launch status.
hipError_t launch_config(int config_id, bool f32_inputs, const GemmArgs &a, int variant, int64_t grid,
                         hipStream_t s);

// The bf16 ring kernels with B given transposed (a.b_trans): variants 1-3
// of the configs 256x192, 256x256, 256x128 and 128x128, the last also with
// K split (a.ksplit > 1).
hipError_t launch_ring_bt(int config_id, const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// The bf16 ring kernels with A given transposed (a.a_trans): variants 1 and
// 2 of the configs 256x192, 256x256 and 128x128, the last also with K split.
hipError_t launch_ring_at(int config_id, const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// The ring kernels on E4M3FN operands (a.fp8, a.b_trans): variants 1-3 of
// the configs 256x192, 256x256 and 128x128, the last also with K split.
hipError_t launch_ring_fp8(int config_id, const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// The same with the affine epilogue applied to the dequantized sums.
hipError_t launch_ring_fp8_affine(int config_id, const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// The FP8 product with A quantized on load: each bf16 row's largest
// magnitude into amax[M] (device scratch) and its factor into a.scale_a,
// then 128 x tile_n tiles (tile_n 128 or 256; grid of them) that convert A
// to codes in LDS.  a.A
// holds bf16 rows (16-byte aligned), a.B the Bt codes; K % 64 == 0.
hipError_t launch_fp8_quant_a(const GemmArgs &a, float *amax, int tile_n, int64_t grid, hipStream_t s);

// Small M (<= 16) on E4M3FN operands with B given transposed: variant 1
// one 16-row block of Bt per workgroup, 2 three (grid = blocks of Bt rows).
hipError_t launch_decode_nt_f8(const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// Per-row E4M3FN quantization of `rows` bf16 rows of `cols` elements (row
// strides ldx, ldq; align_x, align_q the byte alignments of the row starts)
// into codes Q and dequantization factors scale[rows].
hipError_t launch_quant_rows_e4m3(const uint16_t *X, int64_t ldx, int64_t rows, int64_t cols, int align_x,
                                  uint8_t *Q, int64_t ldq, int align_q, float *scale, hipStream_t s);

// Per-column E4M3FN quantization of W [K, N] (bf16, row stride ldw, rows
// `align_w`-byte aligned) into the rows of Qt [N, K] (row stride ldq, rows
// `align_q`-byte aligned) with the factors scale[N].
hipError_t launch_quant_cols_e4m3(const uint16_t *W, int64_t ldw, int64_t K, int64_t N, int align_w, uint8_t *Qt,
                                  int64_t ldq, int align_q, float *scale, hipStream_t s);

// The same for a bf16 product with a fused epilogue (EPI_SILU, EPI_SWIGLU
// or EPI_AFFINE; ring kernel variants 1-3 of the configs 256x192, 256x256
// and 128x128, the last also with K split for EPI_AFFINE, with a.tiles_n
// counting output tiles of tile_n / 2 columns for EPI_SWIGLU).
hipError_t launch_fused(int config_id, int epi, const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// The affine epilogue alone (K == 0 or alpha == 0): C := bias[n] + beta * C
// over a.batch x a.M x a.N, reading C only when a.beta != 0.
hipError_t launch_affine_no_product(const GemmArgs &a, int64_t grid, hipStream_t s);

// Copy batch x M rows of K bf16 elements (row stride lda, batch stride sA,
// rows `align`-byte aligned) into A2 with row stride lda2 (a multiple of 8,
// >= K) and batch stride M x lda2, zero-filling columns K..lda2-1.
hipError_t launch_realign_rows(const uint16_t *A, int64_t lda, int64_t sA, int64_t batch, int64_t M, int64_t K,
                               int align, uint16_t *A2, int64_t lda2, hipStream_t s);

// Small-M path with K split over `ks` workgroups per 128-column strip
// (a.tiles_n strips; 2 ks for a.epi == EPI_SWIGLU: ks on the gate columns,
// ks on the up columns): `ws` holds batch x strips x (ks or 2 ks) x 16 x 128
// floats of partial sums, `cnt` batch x strips counters that are zero on
// entry and left zero on exit.  With `pair` (ks == 2, or ks == 1 for
// SwiGLU: two members per strip): no partial sums or counters, but
// batch x M x N 32-bit exchange slots, zero on entry and left zero.
// Requires N % 128 == 0, K % 32 == 0, 16-byte aligned rows of X and W.
hipError_t launch_decode_split(const GemmArgs &a, float *ws, unsigned *cnt, int ks, unsigned *pair, hipStream_t s);

// The bf16 ring kernel on a persistent stream-K schedule (variants 1 and 2
// of the configs 256x256 and 256x192; `grid` workgroups, a multiple of 8):
// a.ws_part holds 2 x grid partial tiles of FP32, a.ws_cnt one counter per
// output tile (zero on entry, left zero).  Requires K % 32 == 0.
hipError_t launch_streamk(int config_id, const GemmArgs &a, int variant, int64_t grid, hipStream_t s);

// The library's own scratch memory (gemm_run_noalloc): kScratchBytes of
// device memory per GPU, in a file-scope device array.  noalloc_scratch
// returns the current device's copy (its address looked up once per
// device); launch_clear_counters zeroes its first n arrival counters.
constexpr size_t kScratchBytes = (size_t)16 << 20;
hipError_t noalloc_scratch(void **ptr);
hipError_t launch_clear_counters(void *base, int64_t n, hipStream_t s);

// The activation chain on stored bf16 operands (g5_act.hip): steps of page
// "Operator & Runtime" §5.3.1, Example 5-4, each alone or fused.
enum ActStep {
    ACT_SILU = 0,         // in0 = G -> out = T = bf16(SiLU(g))
    ACT_MUL = 1,          // in0 = T, in1 = U -> out = Z = bf16(t * u)
    ACT_SWIGLU = 2,       // in0 = G, in1 = U -> out = Z (SiLU and product fused)
    ACT_QUANT = 3,        // in0 = Z -> out = E4M3FN codes against amax
    ACT_SWIGLU_E4M3 = 4   // in0 = G, in1 = U -> out = the codes of Z (all three fused)
};
struct ActArgs {
    const uint16_t *in0;
    const uint16_t *in1;     // NULL for the one-input steps
    void *out;               // bf16, or E4M3FN codes (bytes) for the quantizing steps
    int64_t M, N;
    int64_t ld0, ld1, ldo;   // row strides in elements
    float amax;              // the quantizing steps' range (> 0)
};
// vec: N % 8 == 0, 16-byte aligned input rows, 16-byte (bf16) or 8-byte
// (codes) aligned output rows and M * N / 8 < 2^32; contig additionally every
// ld == N.  Else one element per thread.
hipError_t launch_act_chain(int step, const ActArgs &a, bool vec, bool contig, hipStream_t s);

// The RMS norm with the residual's addition (g5_norm.hip).  Strides in
// elements (Y: bytes for codes); rows of any alignment.
struct NormArgs {
    const uint16_t *X, *R, *W;   // R (residual) and W (weight) or NULL
    uint16_t *H;                 // bf16(X + R), or NULL
    void *Y;                     // bf16, or E4M3FN codes with factors scale[rows]
    float *scale, *rstd;         // rstd or NULL
    int64_t rows, cols, ldx, ldr, ldh, ldy;
    float eps;
};
hipError_t launch_rms_norm(const NormArgs &a, bool codes, hipStream_t s);

// Its gradient: dX and, when dW is given, the weight's through `part`
// (norm_grad_parts(rows, cols) rows of cols floats, written before they are
// read).
struct NormGradArgs {
    const uint16_t *dY, *H, *W, *dH;   // W and dH (the residual branch's gradient) or NULL
    const float *rstd;
    uint16_t *dX;
    float *part, *dW;
    int64_t rows, cols, lddy, ldh, lddh, lddx;
};
int norm_grad_parts(int64_t rows, int64_t cols);
// dW[n] := the sum of `parts` rows of `part` (0: zeros, `part` not read).
hipError_t launch_norm_dw(const float *part, int parts, int64_t cols, float *dW, hipStream_t s);
hipError_t launch_rms_norm_grad(const NormGradArgs &a, hipStream_t s);

// The mixture-of-experts SwiGLU layer for a few tokens (g5_moe.hip).
// Weights bf16, or E4M3FN codes with factors per row; strides in elements.
constexpr int kMoeMaxTokens = 64, kMoeMaxExperts = 1024, kMoeMaxTopk = 16, kMoeMaxWidth = 65536;
constexpr int kMoeMaxPairs = kMoeMaxTokens * kMoeMaxTopk;
struct MoeItem {
    int expert, first, count, pad;   // its pairs: first .. first + count - 1 of the sorted list
};
// Tokens per work item (the matrix core's 16 columns once or twice), and the
// most items a call can have: one per chosen expert and one more per whole
// chunk, never more than pairs.  Twice where an expert may have more than 16
// tokens, so that its weights are read once for 32: 64 tokens on 8 experts
// (topk 2, 4096 x 1536) 94 us against 110 with 16, on 64 experts (topk 8, six
// or eight tokens each) 485 against 491.
inline int moe_chunk(int64_t T) { return T > 16 ? 32 : 16; }
inline int64_t moe_items(int64_t T, int64_t E, int64_t topk)
{
    const int64_t pairs = T * topk, most = E + pairs / moe_chunk(T);
    return most < pairs ? most : pairs;
}
// Whether the down kernel's workgroups take half of K each (whole calls,
// 4096 x 1536, halves against whole): 64 tokens on 64 experts, topk 8, bf16
// 451 / 486 us, codes 288 / 324; 64 on 8, topk 2, bf16 89 / 96; 17 on 64,
// topk 8, bf16 372 / 365, codes 205 / 225.  Up to 2048 columns the whole form
// has the more workgroups.
inline bool moe_halves(int64_t T, int64_t H) { return T > 16 && H > 2048; }
struct MoeArgs {
    const uint16_t *X;
    const float *logits;
    const void *Wgu, *Wd;
    const float *scale_gu, *scale_d;   // [E, 2I], [E, H] or NULL
    void *Y;
    int32_t *ids;                      // [T, topk] or NULL
    float *gates;
    int64_t T, H, I, E, ldx, ldl, ldgu, strideGu, ldd, strideD, ldy;
    int topk, renormalize, out_f32;
    int cols;                          // hidden columns per workgroup of the down kernel
    int chunk;                         // moe_chunk(T)
    // scratch: the routing [T * topk], the number of work items, the items by
    // expert and the pairs sorted by expert; z as two bf16 planes of
    // rows of ldz
    int *n_items;
    MoeItem *items;
    int32_t *pairs;
    int32_t *w_ids;
    float *w_gates;
    uint16_t *z;
    int64_t ldz, zplane;
    // moe_halves: each half's outputs (64 x 32 floats per workgroup) and a count
    // per 32 columns
    float *halves;
    unsigned *arrived;
};
// Rows of any alignment; 16 rows of Wgu or Wd and the T rows of X span less
// than 2 GiB.
hipError_t launch_moe(const MoeArgs &a, bool codes, hipStream_t s);

// The low-rank adapters beside a bf16 product with B given transposed
// (g5_lora.hip): adapter a has A at A + a strideA [R, K] and B at
// B + a strideB [N, R]; row m of the product uses adapter idx[m] (none when
// outside [0, L)); rows of any alignment.
struct LoraArgs {
    const uint16_t *A, *B;
    const float *scale;          // [L] or NULL
    const int32_t *idx;          // [M]
    int64_t L, R, lda, strideA, ldb, strideB;
    int ranks;                   // R rounded up to 8: the row length of V
    int splits, turns;           // K slices of V; workgroups sharing a row block's adapters
    // scratch for the values v (rows without an adapter unused): FP32
    // [splits, M, ranks] for the small-M kernel, else (V NULL, splits 1) two
    // bf16 parts per row, [M, 2, ranks]
    float *V;
    uint16_t *V2;
    // 16 < M <= kLoraStreamRows on the small-M config: slices of `per` phases
    // of K, their partial sums and one counter per 64 weight rows
    int slices, per;
    float *part;
    unsigned *count;
};
// Steps (64 elements of K) of each of a phase's two halves, by the rows of X:
// a phase of X fits twice in a CU's LDS (48 rows: 50 KB, 80: 63, 128: 68).
constexpr int kLoraStreamRows = 128, kLoraSteps48 = 4, kLoraSteps80 = 3, kLoraSteps128 = 2;
constexpr int lora_steps(int64_t M) { return M <= 48 ? kLoraSteps48 : M <= 80 ? kLoraSteps80 : kLoraSteps128; }
constexpr int lora_row_blocks(int64_t M) { return M <= 48 ? 3 : M <= 80 ? 5 : 8; }
hipError_t launch_lora_shrink(const GemmArgs &a, const LoraArgs &q, hipStream_t s);
// The product with v B^T joined: configs 256x192, 256x256, 128x128 (also
// with K split; variants 1 and 2) and the small-M CFG_DECODE_NT.
hipError_t launch_lora(int config_id, const GemmArgs &a, const LoraArgs &q, int variant, int64_t grid, hipStream_t s);

}  // namespace g5
