// g5_vocab.hip -- the loss over a large vocabulary behind the last projection,
// and its gradient, without the logits in memory.
//
//   z = X . Wt^T, l = scale z, lse_m = log sum_v exp(l_mv)
//   loss_m = sum_j q_mj (log q_mj - l_m,id(m,j) + lse_m)
//
// with the targets q: one token of weight 1 (cross entropy), or a teacher's
// best tokens, q_m = softmax of its logits there (distillation).
//
// Forward: an output tile of the product keeps its logits in registers and
// leaves, for each of its rows, their maximum and the sum of exp(l - maximum)
// (one pass: a later tile's maximum rescales the sum) and the logits of the
// row's targets that lie in it; a second kernel joins the tiles.
//
// Backward, vocabulary piece by piece: the logits again, from them
// D = g (exp(l - lse) - q) in bf16, then dW = D^T X of the piece and dX += D W.
#include <hip/hip_runtime.h>

#include "g5_device.h"
#include "g5_kernels.h"
#include "g5_ping.h"
#include "g5_stream.h"

namespace g5 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ int64_t target_id(const VocabArgs &p, int64_t i)
{
    return p.ids64 ? ((const int64_t *)p.ids)[i] : (int64_t)((const int32_t *)p.ids)[i];
}

// A part of a row: its maximum and the sum of exp2(c (z - maximum)) without the
// maximum's own 1, so that a loss near 0, log(1 + rest), does not lose what 1 +
// rest rounds off.  A part without finite logits has maximum -inf and rest -1
// (or NaN, which stays).
struct Part {
    float top, rest;
};
__device__ __forceinline__ Part join_part(Part a, Part b, float c)
{
    const Part hi = a.top >= b.top ? a : b, lo = a.top >= b.top ? b : a;
    const float base = hi.top == -__builtin_inff() ? 0.f : hi.top;
    return Part{hi.top, hi.rest + (1.f + lo.rest) * __builtin_amdgcn_exp2f(c * (lo.top - base))};
}

// The tile's operands, bases moved to its first row and column.
template <int BM, int BN>
__device__ __forceinline__ GemmArgs tile_args(const VocabArgs &p, int64_t m0, int64_t n0)
{
    GemmArgs q{};
    q.A = p.X + m0 * p.ldx;
    q.B = p.W + n0 * p.ldw;
    q.M = p.M - m0 < BM ? p.M - m0 : BM;
    q.N = p.V - n0 < BN ? p.V - n0 : BN;
    q.K = p.K;
    q.lda = p.ldx;
    q.ldb = p.ldw;
    q.align_a = p.align_x;
    q.align_b = p.align_w;
    return q;
}

// Rows of the accumulators go through LDS as FP32, RP at a time.
template <class R, int BM, int BN>
struct Staged {
    static constexpr int PITCH = BN + 4;                                  // floats; (4: bank conflicts)
    static constexpr int FITS = R::LDS_BYTES / (PITCH * 4);
    static constexpr int RP = FITS >= BM ? BM : FITS >= BM / 2 ? BM / 2 : BM / 4;
    static_assert(RP * PITCH * 4 <= R::LDS_BYTES && RP % 16 == 0, "staging passes");

    __device__ static __forceinline__ void put(const typename R::Acc &acc, float *L, int pass, int wm, int wn, int g, int li)
    {
#pragma unroll
        for (int fm = 0; fm < R::FM; ++fm) {
            const int row = wm * R::TM + fm * 16;
            if (row / RP != pass) continue;
#pragma unroll
            for (int fn = 0; fn < R::FN; ++fn)
                *(f32x4 *)(L + (row - pass * RP + li) * PITCH + wn * R::TN + fn * 16 + g * 4) = acc[fn][fm];
        }
    }
};

// The targets of a tile's rows that lie in its columns [first, first + cols),
// found by all threads: pair i = tid + NT k (of row i / topk) sets bit k % 64.
// Few pairs do, so the scan asks for sixteen ids at once, unconditionally, and
// what is done with them walks the bits.
template <int NT, class T>
__device__ __forceinline__ uint64_t scan_ids(const T *ids, int tid, int pairs, T first, int cols)
{
    uint64_t bits = 0;
    for (int i = tid, k = 0; i < pairs; i += NT * 16, k += 16) {
        T id[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) id[j] = ids[i + NT * j < pairs ? i + NT * j : i];
        uint32_t found = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const T col = id[j] - first;
            found |= (uint32_t)((i + NT * j < pairs) & (id[j] >= 0) & (col >= 0) & (col < (T)cols)) << j;
        }
        bits |= (uint64_t)found << (k & 63);
    }
    return bits;
}
template <int NT, class Do>
__device__ __forceinline__ void each_target(int tid, int pairs, uint64_t bits, Do act)
{
    for (; bits; bits &= bits - 1)
        for (int i = tid + NT * __builtin_ctzll(bits); i < pairs; i += NT * 64) act(i);
}

// They are then listed for the wave that holds the logit, each of whose lanes
// takes its own, one after the other, out of all its registers.  A tile with
// more for one wave than the list holds is staged through LDS instead.
template <class R, int WGM, int WGN>
struct TargetList {
    static constexpr int PER = 64;
    int count[WGM * WGN];
    uint32_t at[WGM * WGN][PER];         // pair << 16 | row << 8 | column

    __device__ __forceinline__ void clear(int tid)
    {
        if (tid < WGM * WGN) count[tid] = 0;
    }
    __device__ __forceinline__ void add(int i, int row, int col)
    {
        const int w = row / R::TM * WGN + col / R::TN, k = atomicAdd(&count[w], 1);
        if (k < PER) at[w][k] = (uint32_t)i << 16 | (uint32_t)row << 8 | (uint32_t)col;
    }
    __device__ __forceinline__ bool over() const
    {
        bool o = false;
#pragma unroll
        for (int w = 0; w < WGM * WGN; ++w) o |= count[w] > PER;
        return o;
    }
    // act(place, pair), by all lanes of the wave together: the lane's target
    // lies in element place % 4 of acc[place / 4 / FM][place / 4 % FM] (place -1:
    // it has none this time).
    template <class Do>
    __device__ __forceinline__ void each(int wave, int lane, Do act) const
    {
        const int n = __builtin_amdgcn_readfirstlane(count[wave]);
        uint64_t mine = 0;
#pragma unroll 4
        for (int k = 0; k < n; ++k) {
            const uint32_t e = at[wave][k], row = e >> 8 & 255, col = e & 255;
            mine |= (uint64_t)(lane == (int)(col % 16 / 4 * 16 + row % 16)) << k;
        }
        while (__any(mine != 0)) {
            int place = -1, pair = 0;
            if (mine) {
                const uint32_t e = at[wave][__builtin_ctzll(mine)], row = e >> 8 & 255, col = e & 255;
                mine &= mine - 1;
                place = (int)((col % R::TN / 16 * R::FM + row % R::TM / 16) * 4 + col % 4);
                pair = (int)(e >> 16);
            }
            act(place, pair);
        }
    }
};

// Forward by tiles.  The tile's epilogue is registers but for the join of
// the four waves side by side, and tiles that hold a target.  Bound by the
// matrix cores: 4096 rows by 131072 tokens of 4096 2918 us (1507 TFLOP/s), 2048
// by 32768 with 32 targets a row 384 us (1432); 1000 by 32003 of 1028 72 us
// (916: two rounds of tiles of 17 stages, a launch and their ends).
template <int BM, int BN, int WGM, int WGN>
__global__ void __launch_bounds__(WGM *WGN * 64, 2) k_vocab_stats(VocabArgs p)
{
    using R = RingTile<BM, BN, WGM, WGN, 4, 4, 16, true, EPI_NONE, true>;
    using S = Staged<R, BM, BN>;
    constexpr int NT = WGM * WGN * 64;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[R::LDS_BYTES / 2];
    const TileCoord tc = tile_map(blockIdx.x, 1, p.tiles_m, p.tiles_n, p.group_m);
    const int64_t m0 = tc.tm * BM, n0 = tc.tn * BN;
    const GemmArgs q = tile_args<BM, BN>(p, m0, n0);
    f32x4 acc[R::FN][R::FM];
    R::zero(acc);
    multiply_tile<R, BM, BN, true, false>(q, smem, q.K, acc);

    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, wave = tid >> 6, wm = wave / WGN, wn = wave % WGN, g = lane >> 4, li = lane & 15;
    const float c = p.scale * kLog2e;
    if (q.N < BN) {
#pragma unroll
        for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (wn * R::TN + fn * 16 + g * 4 + i >= q.N) {
#pragma unroll
                    for (int fm = 0; fm < R::FM; ++fm) acc[fn][fm][i] = -__builtin_inff();
                }
    }
    __syncthreads();
    Part *st = (Part *)smem;                       // [WGN][BM]
    TargetList<R, WGM, WGN> &list = *(TargetList<R, WGM, WGN> *)(st + WGN * BM);
    static_assert(WGN * BM * sizeof(Part) + sizeof(list) <= R::LDS_BYTES, "behind the ring");
    list.clear(tid);
    // targets in this tile
    const int64_t first = p.v0 + n0;
    const int pairs = (int)q.M * p.topk;
    auto col_of = [&](int i) { return target_id(p, m0 * p.topk + i) - first; };
    auto in = [&](int64_t col) { return col >= 0 && col < q.N; };
    const uint64_t bits = p.ids64 ? scan_ids<NT>((const int64_t *)p.ids + m0 * p.topk, tid, pairs, first, (int)q.N)
                                  : scan_ids<NT>((const int32_t *)p.ids + m0 * p.topk, tid, pairs, (int32_t)first, (int)q.N);
#pragma unroll
    for (int fm = 0; fm < R::FM; ++fm) {
        float top = -__builtin_inff();
#pragma unroll
        for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, acc[fn][fm][i]);
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float base = top == -__builtin_inff() ? 0.f : top;
        // (the difference first: it is exact near the maximum, where it counts)
        float whole = 0.f;
#pragma unroll
        for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
            for (int i = 0; i < 4; ++i) whole += __builtin_amdgcn_exp2f(c * (acc[fn][fm][i] - base));
        whole += __shfl_xor(whole, 16, 64);
        whole += __shfl_xor(whole, 32, 64);
        float rest = whole - 1.f;
        // Where little stands beside the maximum, once more without it: the
        // one term that is 1 has no fraction.
        // (4096 x 32768 x 512 with ordinary logits: none 142 us, so 145; always,
        // 12 us more than none.)
        const bool near = rest < 0.0625f && whole > 0.f;
        if (__any(near)) {
            float small = 0.f;
#pragma unroll
            for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    small += __builtin_amdgcn_fractf(__builtin_amdgcn_exp2f(c * (acc[fn][fm][i] - base)));
            small += __shfl_xor(small, 16, 64);
            small += __shfl_xor(small, 32, 64);
            if (near) rest = small;
        }
        if (g == 0) st[wn * BM + wm * R::TM + fm * 16 + li] = Part{top, rest};
    }
    __syncthreads();
    each_target<NT>(tid, pairs, bits, [&](int i) {
        const int64_t col = col_of(i);
        if (in(col)) list.add(i, i / p.topk, (int)col);
    });
    if (tid < q.M) {
        Part s = st[tid];
#pragma unroll
        for (int w = 1; w < WGN; ++w) s = join_part(s, st[w * BM + tid], c);
        p.part[(m0 + tid) * p.parts + p.tile0 + tc.tn] = float2{s.top, s.rest};
    }
    __syncthreads();
    if (!list.over()) {
        list.each(wave, lane, [&](int place, int pair) {
            float v = 0.f;
#pragma unroll
            for (int c = 0; c < R::FN * R::FM * 4; ++c) v = c == place ? acc[c / 4 / R::FM][c / 4 % R::FM][c % 4] : v;
            if (place >= 0) p.zt[m0 * p.topk + pair] = v;
        });
        return;
    }
    float *L = (float *)smem;
    for (int pass = 0; pass < BM / S::RP; ++pass) {
        __syncthreads();
        // (the accumulators' places are compile-time constants)
#pragma unroll
        for (int k = 0; k < BM / S::RP; ++k)
            if (k == pass) S::put(acc, L, k, wm, wn, g, li);
        __syncthreads();
        each_target<NT>(tid, pairs, bits, [&](int i) {
            const int64_t col = col_of(i);
            const int r = i / p.topk - pass * S::RP;
            if (in(col) && r >= 0 && r < S::RP) p.zt[m0 * p.topk + i] = L[r * S::PITCH + (int)col];
        });
    }
}

// Up to 32 rows: bound by reading the weight once, so a workgroup owns 32 rows
// of it, streamed from HBM into the matrix core by four waves on contiguous
// pieces of K, and one wave joins them: forward the statistics and the targets'
// logits, GRAD the rows' D, in two bf16 parts.  One row of 4096 by 32768 tokens
// 42.7 us (6.3 TB/s), 16 of 2048 by 128003 100 us (5.2); D of 3 rows of 3712
// by 1302 tokens 12 us for 34 in tiles of 128.
constexpr int kVocabWaves = 4, kVocabCols = 32;

template <int NC, int D, bool GRAD>
__global__ void __launch_bounds__(kVocabWaves * 64, 4) k_vocab_stream(VocabArgs p, VocabGrad b)
{
    __shared__ f32x4 red[kVocabWaves][2][64];
    __shared__ float tile[kVocabCols][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    const int64_t n0 = (int64_t)blockIdx.x * kVocabCols;
    f32x4 acc[2][NC];
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) acc[0][cc] = acc[1][cc] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int K = (int)p.K, steps = (K + 63) / 64, M = (int)p.M;
    const int s0 = steps * wave / kVocabWaves, s1 = steps * (wave + 1) / kVocabWaves;
    // (rows past V repeat the block's first and are masked below)
    const char *wbase[2];
    uint32_t woff[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int64_t n = n0 + 16 * r < p.V ? n0 + 16 * r : n0;
        wbase[r] = (const char *)(p.W + n * p.ldw);
        woff[r] = (uint32_t)(n + li < p.V ? li : 0) * (uint32_t)(p.ldw * 2) + 16 * g;
    }
    RowStream<false, 2, NC, D> rows_of_w;
    auto tokens = [&](uint32_t (&xoff)[NC], bool (&ok)[NC]) {
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
            ok[cc] = 16 * cc + li < M;
            xoff[cc] = (uint32_t)(ok[cc] ? 16 * cc + li : 0) * (uint32_t)(p.ldx * 2) + x_lane<false>(g);
        }
    };
    rows_of_w.run(wbase, woff, (const char *)p.X, tokens, s0, s1, K, g, acc);
    const float c = p.scale * kLog2e;
#pragma unroll
    for (int cc = 0; cc < NC; ++cc) {
        if (16 * cc >= M) break;         // uniform
        __syncthreads();                 // (the chunk before has been read)
        red[wave][0][lane] = acc[0][cc];
        red[wave][1][lane] = acc[1][cc];
        __syncthreads();
        if (wave != 0) continue;
        const int m = 16 * cc + li, rows = M - 16 * cc < 16 ? M - 16 * cc : 16;
        f32x4 s[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            s[r] = red[0][r][lane];
#pragma unroll
            for (int w = 1; w < kVocabWaves; ++w) s[r] += red[w][r][lane];
        }
        if constexpr (GRAD) {
            const bool some = m < M && b.has[m] != 0;
            const float lse = some ? b.lse[m] : 0.f, weight = some ? b.weight[m] : 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    tile[16 * r + 4 * g + i][li] = __builtin_amdgcn_exp2f(kLog2e * __builtin_fmaf(p.scale, s[r][i], -lse));
            // (one wave writes and reads the tile: in order)
            __builtin_amdgcn_wave_barrier();
#pragma unroll 8
            for (int i = lane; i < rows * p.topk; i += 64) {
                const int64_t at = (int64_t)16 * cc * p.topk + i;
                const int id = b.ids[at], col = id - (int)(p.v0 + n0);
                if (id >= 0 && col >= 0 && col < kVocabCols) tile[col][i / p.topk] -= b.q[at];
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t n = n0 + 16 * r + 4 * g;
                if (m >= M || n >= b.ldd) continue;      // (columns from V on are padding)
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = some ? weight * tile[16 * r + 4 * g + i][li] : 0.f;
                const u32x2 d = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                const u32x2 rest = {pack_bf16x2(v[0] - bf16_lo(d[0]), v[1] - bf16_hi(d[0])),
                                    pack_bf16x2(v[2] - bf16_lo(d[1]), v[3] - bf16_hi(d[1]))};
                *(u32x2 *)(b.D + m * b.ldd + n) = d;
                *(u32x2 *)(b.D + (M + m) * b.ldd + n) = rest;
            }
            __builtin_amdgcn_wave_barrier();
        } else {
            float top = -__builtin_inff(), rest = 0.f, ones = -1.f;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (n0 + 16 * r + 4 * g + i >= p.V) s[r][i] = -__builtin_inff();
                    top = fmaxf(top, s[r][i]);
                    tile[16 * r + 4 * g + i][li] = s[r][i];
                }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float base = top == -__builtin_inff() ? 0.f : top;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(c * (s[r][i] - base));
                    ones += e == 1.f ? 1.f : 0.f;
                    rest += e == 1.f ? 0.f : e;
                }
            if (g != 0) ones += 1.f;         // (the one taken off once)
#pragma unroll
            for (int o = 16; o < 64; o <<= 1) {
                rest += __shfl_xor(rest, o, 64);
                ones += __shfl_xor(ones, o, 64);
            }
            if (g == 0 && m < M) p.part[m * p.parts + blockIdx.x] = float2{top, ones + rest};
            // (one wave writes and reads the tile: in order)
            __builtin_amdgcn_wave_barrier();
#pragma unroll 8
            for (int i = lane; i < rows * p.topk; i += 64) {
                const int64_t at = (int64_t)16 * cc * p.topk + i, col = target_id(p, at) - n0;
                if (col >= 0 && col < kVocabCols && n0 + col < p.V) p.zt[at] = tile[col][i / p.topk];
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

// A teacher's entry: a token of the vocabulary whose logit is not -inf.
__device__ __forceinline__ bool has_entry(int64_t id, int64_t vocab, float t)
{
    return id >= 0 && id < vocab && !(t == -__builtin_inff());
}
__device__ __forceinline__ float max64(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
__device__ __forceinline__ float sum64(float v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

constexpr int kTopkPer = kVocabMaxTopk / 64;

// A row's targets, by one wave: lane j holds entries j, j + 64, ...: their
// weights (0: none) and, for the loss, log q.  False where the row has none.
struct RowTargets {
    int64_t id[kTopkPer];
    float q[kTopkPer], logq[kTopkPer];
};
__device__ __forceinline__ bool row_targets(const VocabArgs &p, int64_t m, int lane, RowTargets &t)
{
    bool has[kTopkPer];
    float v[kTopkPer], top = -__builtin_inff();
    bool some = false;
#pragma unroll
    for (int j = 0; j < kTopkPer; ++j) {
        const int at = lane + 64 * j;
        t.id[j] = at < p.topk ? target_id(p, m * p.topk + at) : -1;
        v[j] = at < p.topk && p.teacher ? p.teacher[m * p.topk + at] : 0.f;
        has[j] = has_entry(t.id[j], p.vocab, v[j]);
        some |= has[j];
        if (has[j]) top = fmaxf(top, v[j]);
    }
    const bool any = __any(some);
    top = max64(top);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kTopkPer; ++j) {
        t.logq[j] = has[j] ? p.scale * (v[j] - top) : 0.f;
        t.q[j] = has[j] ? expf(t.logq[j]) : 0.f;
        sum += t.q[j];
    }
    sum = sum64(sum);
    const float log_sum = logf(sum);
#pragma unroll
    for (int j = 0; j < kTopkPer; ++j) {
        if (!has[j]) t.id[j] = -1;
        else t.q[j] /= sum;
        t.logq[j] -= log_sum;
    }
    return any;
}

// The tiles' parts of a row joined by a workgroup, then its loss.  Always the
// same parts in the same order: the same call gives the same bits.  Latency: one
// row of 1024 parts 4.6 us, 4096 rows of 512 parts 11 us (16 MiB of parts,
// against the 1 GiB of logits in bf16 that are not written).
constexpr int kJoinWaves = 4;
__global__ void __launch_bounds__(kJoinWaves * 64) k_vocab_join(VocabArgs p)
{
    __shared__ Part st[kJoinWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float c = p.scale * kLog2e;
    for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
        Part s{-__builtin_inff(), -1.f};
#pragma unroll 8
        for (int64_t i = threadIdx.x; i < p.parts; i += kJoinWaves * 64) {
            const float2 v = p.part[m * p.parts + i];
            s = join_part(s, Part{v.x, v.y}, c);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) s = join_part(s, Part{__shfl_xor(s.top, o, 64), __shfl_xor(s.rest, o, 64)}, c);
        __syncthreads();                 // (the row before has been read)
        if (lane == 0) st[wave] = s;
        __syncthreads();
        if (wave != 0) continue;
        s = st[0];
#pragma unroll
        for (int w = 1; w < kJoinWaves; ++w) s = join_part(s, st[w], c);
        const float top = s.top, log_sum = log1pf(s.rest);
        if (lane == 0 && p.lse_out) p.lse_out[m] = p.scale * top + log_sum;
        float loss = 0.f;
        if (!p.teacher) {
            const int64_t id = target_id(p, m);
            // (the difference of the logits first: exact where the loss is small)
            if (id >= 0 && id < p.vocab) loss = p.scale * (top - p.zt[m]) + log_sum;
        } else {
            RowTargets q;
            if (row_targets(p, m, lane, q)) {
#pragma unroll
                for (int j = 0; j < kTopkPer; ++j)
                    // (a weight of 0 adds nothing, however low its log is; NaN stays)
                    if (q.id[j] >= 0 && q.q[j] != 0.f)
                        loss += q.q[j] * (q.logq[j] + (p.scale * (top - p.zt[m * p.topk + lane + 64 * j]) + log_sum));
                loss = sum64(loss);
            }
        }
        if (lane == 0) p.loss[m] = loss;
    }
}

// Before the gradient, a wave per row: its targets as int32 ids, each once
// (one listed twice has both weights at its first place), their weights,
// whether there are any, and its row of X with zero padding, all zeros for a
// row without targets, whose contents must not reach dW (twice with b.parts 2:
// D's two parts meet it one after the other).  4096 rows of 4096 13.6 us (67 MB,
// 4.9 TB/s).
struct PrepRow {
    int ids[kVocabMaxTopk];
    float qs[kVocabMaxTopk];
};
// The row's weight, 0 where it has no target.
__device__ __forceinline__ float prep_row(const VocabArgs &p, const VocabGrad &b, int64_t m, int lane, PrepRow &l)
{
    bool some;
    if (!p.teacher) {
        const int64_t id = target_id(p, m);
        some = id >= 0 && id < p.vocab;
        if (lane == 0) {
            b.ids[m] = some ? (int32_t)id : -1;
            b.q[m] = 1.f;
        }
    } else {
        RowTargets t;
        some = row_targets(p, m, lane, t);
#pragma unroll
        for (int j = 0; j < kTopkPer; ++j) {
            l.ids[lane + 64 * j] = (int)t.id[j];
            l.qs[lane + 64 * j] = t.q[j];
        }
        // (one wave writes and reads its row: in order)
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < kTopkPer; ++j) {
            const int at = lane + 64 * j, id = l.ids[at];
            if (at >= p.topk) break;
            bool again = id < 0;
            float q = 0.f;
            for (int i = 0; i < p.topk; ++i) {
                const bool same = l.ids[i] == id;
                again |= same && i < at;
                if (same && i >= at) q += l.qs[i];
            }
            b.ids[m * p.topk + at] = again ? -1 : id;
            b.q[m * p.topk + at] = q;
        }
    }
    if (lane == 0) b.has[m] = some;
    const uint16_t *x = p.X + m * p.ldx;
    for (int64_t col = lane * 8; col < b.ldx2; col += 512) {
        const u32x4 v = load_chunk8_bf16(x, col, p.K, some, p.align_x);
        *(u32x4 *)(b.X2 + m * b.ldx2 + col) = v;
        if (b.parts == 2) *(u32x4 *)(b.X2 + (p.M + m) * b.ldx2 + col) = v;
    }
    return some ? b.dloss[m] : 0.f;
}
// The factor that the weights are divided by, from their largest size: 1
// where there is no weight at all, or an infinite one.
__device__ __forceinline__ float weight_factor(float top) { return top > 0.f && top < __builtin_inff() ? top : 1.f; }

constexpr int kPrepWaves = 4;
template <bool ALPHA>
__global__ void __launch_bounds__(kPrepWaves * 64) k_vocab_prep(VocabArgs p, VocabGrad b)
{
    __shared__ PrepRow rows[kPrepWaves];
    __shared__ float tops[kPrepWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = (int64_t)blockIdx.x * kPrepWaves + wave;
    float a = 1.f;
    if constexpr (ALPHA) {
        float top = 0.f;
        const int pairs = (int)p.M * p.topk;
#pragma unroll 4
        for (int i = threadIdx.x; i < pairs; i += kPrepWaves * 64) {
            const float d = fabsf(b.dloss[i / p.topk]), t = p.teacher ? p.teacher[i] : 0.f;
            top = fmaxf(top, has_entry(target_id(p, i), p.vocab, t) ? d : 0.f);
        }
        top = max64(top);
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        for (int w = 0; w < kPrepWaves; ++w) top = fmaxf(top, tops[w]);
        a = weight_factor(top);
        if (blockIdx.x == 0 && threadIdx.x == 0) *b.alpha = a;
    }
    if (m >= p.M) return;                 // (a wave works alone)
    const float w = prep_row(p, b, m, lane, rows[wave]);
    if (lane == 0) b.weight[m] = w / a;
}

// The largest |dloss| of the rows with targets into alpha, every row's weight
// divided by it.  D holds weight (p - q) and the products multiply their sums
// by alpha: where all weights are alike (a mean over the rows) they are then
// exactly 1 and D's rounding to bf16 does not round that common factor, which
// would move whole gradients by up to 2^-8 at once.  One workgroup: 5 us of
// latency for 4096 rows, once per call.
__global__ void __launch_bounds__(1024) k_vocab_weights(float *weight, int64_t M, float *alpha)
{
    __shared__ float tops[16];
    const int tid = threadIdx.x;
    float top = 0.f;
    for (int64_t m = tid; m < M; m += 1024) top = fmaxf(top, fabsf(weight[m]));
    top = max64(top);
    if ((tid & 63) == 0) tops[tid >> 6] = top;
    __syncthreads();
    top = 0.f;
    for (int w = 0; w < 16; ++w) top = fmaxf(top, tops[w]);
    const float a = weight_factor(top);
    for (int64_t m = tid; m < M; m += 1024) weight[m] = weight[m] / a;
    if (tid == 0) *alpha = a;
}

// Both in one launch: for up to 16 rows, a wave each (3 rows: 3.6 us for 2.2 +
// 1.8 and the gap between them), and for up to kPrepScan entries, where every
// workgroup of k_vocab_prep looks at all of them (262 rows 3.8 us for 3.2 + 1.8
// and the gap, 1000 rows 5.4 for 3.9 + 1.8; 2000 entries of 100 rows 9.5 for 5.7
// + 1.6).
constexpr int kPrepScan = 1024;
constexpr int kPrepFew = 16;
__global__ void __launch_bounds__(kPrepFew * 64) k_vocab_prep_few(VocabArgs p, VocabGrad b)
{
    __shared__ PrepRow rows[kPrepFew];
    __shared__ float weights[kPrepFew];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, M = (int)p.M;     // as many waves as rows
    const float w = prep_row(p, b, wave, lane, rows[wave]);
    if (lane == 0) weights[wave] = w;
    __syncthreads();
    if (wave != 0) return;
    const float v = lane < M ? weights[lane] : 0.f, a = weight_factor(max64(fabsf(v)));
    if (lane < M) b.weight[lane] = v / a;
    if (lane == 0) *b.alpha = a;
}

// D of a piece: exp(l - lse) in registers, the targets' weights taken off where
// they lie, then weighted and rounded to bf16.  Many targets in a tile, and
// b.parts 2 (few rows: the rounding's rest, as a bf16 of its own, follows in
// rows M .. 2 M - 1), go through LDS as FP32.  Bound by the matrix cores and the
// epilogue behind them: 4096 rows by a piece of 32768 tokens of 4096 780 us
// (1410 TFLOP/s; the same logits alone take 730), 2048 by 50001 of 2048 with 64
// targets a row 406 us (1034).
template <int BM, int BN, int WGM, int WGN>
__global__ void __launch_bounds__(WGM *WGN * 64, 2) k_vocab_dlogits(VocabArgs p, VocabGrad b)
{
    using R = RingTile<BM, BN, WGM, WGN, 4, 4, 16, true, EPI_NONE, true>;
    using S = Staged<R, BM, BN>;
    constexpr int NT = WGM * WGN * 64;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[R::LDS_BYTES / 2];
    const TileCoord tc = tile_map(blockIdx.x, 1, p.tiles_m, p.tiles_n, p.group_m);
    const int64_t m0 = tc.tm * BM, n0 = tc.tn * BN;
    const GemmArgs q = tile_args<BM, BN>(p, m0, n0);
    f32x4 acc[R::FN][R::FM];
    R::zero(acc);
    multiply_tile<R, BM, BN, true, false>(q, smem, q.K, acc);

    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, wave = tid >> 6, wm = wave / WGN, wn = wave % WGN, g = lane >> 4, li = lane & 15;
#pragma unroll
    for (int fm = 0; fm < R::FM; ++fm) {
        const int r = wm * R::TM + fm * 16 + li;
        const float lse = r < q.M ? b.lse[m0 + r] : 0.f;
#pragma unroll
        for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[fn][fm][i] = __builtin_amdgcn_exp2f(kLog2e * __builtin_fmaf(p.scale, acc[fn][fm][i], -lse));
    }
    const int pairs = (int)q.M * p.topk;
    const int first = (int)(p.v0 + n0);
    auto col_of = [&](int i) {
        const int id = b.ids[m0 * p.topk + i];
        return id < 0 ? -1 : id - first;
    };
    auto in = [&](int col) { return col >= 0 && col < q.N; };
    const uint64_t bits = scan_ids<NT>(b.ids + m0 * p.topk, tid, pairs, (int32_t)first, (int)q.N);
    __syncthreads();
    if (b.parts == 1) {
        TargetList<R, WGM, WGN> &list = *(TargetList<R, WGM, WGN> *)smem;
        list.clear(tid);
        __syncthreads();
        each_target<NT>(tid, pairs, bits, [&](int i) {
            const int col = col_of(i);
            if (in(col)) list.add(i, i / p.topk, col);
        });
        __syncthreads();
        if (!list.over()) {
            list.each(wave, lane, [&](int place, int pair) {
                const float t = place >= 0 ? b.q[m0 * p.topk + pair] : 0.f;
#pragma unroll
                for (int c = 0; c < R::FN * R::FM * 4; ++c) acc[c / 4 / R::FM][c / 4 % R::FM][c % 4] -= c == place ? t : 0.f;
            });
#pragma unroll
            for (int fm = 0; fm < R::FM; ++fm) {
                const int r = wm * R::TM + fm * 16 + li;
                const bool some = r < q.M && b.has[m0 + r] != 0;
                const float w = some ? b.weight[m0 + r] : 0.f;
#pragma unroll
                for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[fn][fm][i] = some ? w * acc[fn][fm][i] : 0.f;
            }
            __syncthreads();
            GemmArgs out = q;
            out.C = b.D + m0 * b.ldd + n0;
            out.ldc = b.ldd;
            out.N = b.ldd - n0 < BN ? b.ldd - n0 : BN;       // (padding columns too: whole chunks)
            out.align_c = 16;
            R::store(out, smem, TileCoord{0, 0, 0}, acc);
            return;
        }
    }
    float *L = (float *)smem;
    for (int pass = 0; pass < BM / S::RP; ++pass) {
        if (pass * S::RP >= q.M) break;          // uniform
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BM / S::RP; ++k)
            if (k == pass) S::put(acc, L, k, wm, wn, g, li);
        __syncthreads();
        each_target<NT>(tid, pairs, bits, [&](int i) {
            const int col = col_of(i), r = i / p.topk - pass * S::RP;
            if (col >= 0 && col < q.N && r >= 0 && r < S::RP) L[r * S::PITCH + col] -= b.q[m0 * p.topk + i];
        });
        __syncthreads();
#pragma unroll 2
        for (int i = tid; i < S::RP * (BN / 8); i += NT) {
            const int r = i / (BN / 8), ch = i % (BN / 8) * 8, row = pass * S::RP + r;
            if (row >= q.M || ch >= q.N) continue;
            const float w = b.weight[m0 + row];
            const bool some = b.has[m0 + row] != 0;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = some ? w * L[r * S::PITCH + ch + j] : 0.f;
            const u32x4 d = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
            uint16_t *out = b.D + (m0 + row) * b.ldd + n0 + ch;
            *(u32x4 *)out = d;
            if (b.parts == 2) {
                u32x4 rest;
#pragma unroll
                for (int j = 0; j < 4; ++j) rest[j] = pack_bf16x2(v[2 * j] - bf16_lo(d[j]), v[2 * j + 1] - bf16_hi(d[j]));
                *(u32x4 *)(out + p.M * b.ldd) = rest;
            }
        }
    }
}

// dW rows of a piece: scale alpha D^T X2, summed over the rows in pieces whose
// 32-bit offsets fit.  Few output tiles over many rows: b.w_slices parts of the
// rows, each part's sums as FP32 in a plane of its own (k_vocab_total).  A
// piece of 32768 tokens from 4096 rows of 4096 804 us (1367 TFLOP/s), 50001
// tokens from 2048 rows of 2048 388 us (1080: a tile's 32 stages, then its 128
// KiB stored behind them); few rows are bound by writing dW (131072 x 4096 bf16
// from two rows 242 us, 4.4 TB/s).
template <int BM, int BN, int WGM, int WGN>
__global__ void __launch_bounds__(WGM *WGN * 64, 2) k_vocab_dw(VocabArgs p, VocabGrad b)
{
    using R = RingTile<BM, BN, WGM, WGN, 4, 4, 16, true, EPI_NONE, false, false, true>;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[R::LDS_BYTES / 2];
    const TileCoord tc = tile_map(blockIdx.x, b.w_slices, p.tiles_m, p.tiles_n, p.group_m);
    const int64_t m0 = tc.tm * BM, n0 = tc.tn * BN;          // vocabulary, hidden
    const int64_t all = p.M * b.parts;
    const int64_t from = tc.b * b.w_per < all ? tc.b * b.w_per : all, to = all - from < b.w_per ? all : from + b.w_per;
    GemmArgs q{};
    if (b.w_slices == 1) {
        q.C = (char *)b.dW + ((p.v0 + m0) * b.lddw + n0) * (b.dw_f32 ? 4 : 2);
        q.ldc = b.lddw;
        q.out_f32 = b.dw_f32;
    } else {
        q.C = b.w_sums + (tc.b * p.V + m0) * b.ldx2 + n0;
        q.ldc = b.ldx2;
        q.out_f32 = 1;
    }
    q.lda = b.ldd;
    q.ldb = b.ldx2;
    q.align_a = q.align_b = 16;
    q.M = p.V - m0 < BM ? p.V - m0 : BM;
    q.N = b.ldx2 - n0 < BN ? b.ldx2 - n0 : BN;               // (whole padded chunks)
    f32x4 acc[R::FN][R::FM];
    R::zero(acc);
    for (int64_t done = from; done < to;) {
        q.A = b.D + m0 + done * b.ldd;
        q.B = b.X2 + n0 + done * b.ldx2;
        q.K = to - done < b.rows_at_once ? to - done : b.rows_at_once;
        if (done > from) __syncthreads();
        multiply_tile<R, BM, BN, false, true>(q, smem, q.K, acc);
        done += q.K;
    }
    if (b.w_slices == 1) {
        const float a = all > 0 ? p.scale * *b.alpha : 0.f;
#pragma unroll
        for (int fn = 0; fn < R::FN; ++fn)
#pragma unroll
            for (int fm = 0; fm < R::FM; ++fm)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[fn][fm][i] *= a;
        q.N = p.K - n0 < BN ? p.K - n0 : BN;
    }
    store_rows<R, BM, BN, WGM, WGN>(q, smem, acc);
}

// A piece's share of dX before its factor: sums (+)= D W over one of b.slices
// parts of the piece's tokens, each with sums of its own.  Few output tiles
// would leave CUs idle over a long summed axis.  4096 x 4096 from a piece of
// 32768 tokens 778 us (1414 TFLOP/s).
template <int BM, int BN, int WGM, int WGN>
__global__ void __launch_bounds__(WGM *WGN * 64, 2) k_vocab_sums(VocabArgs p, VocabGrad b)
{
    using R = RingTile<BM, BN, WGM, WGN, 4, 4, 16, true>;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[R::LDS_BYTES / 2];
    const TileCoord tc = tile_map(blockIdx.x, b.slices, p.tiles_m, p.tiles_n, p.group_m);
    const int64_t m0 = tc.tm * BM, n0 = tc.tn * BN, rows = p.M * b.parts;
    const int64_t k0 = tc.b * b.per < p.V ? tc.b * b.per : p.V;
    GemmArgs q{};
    q.A = b.D + m0 * b.ldd + k0;
    q.B = p.W + k0 * p.ldw + n0;
    q.C = b.sums + (tc.b * rows + m0) * b.ldx2 + n0;
    q.M = rows - m0 < BM ? rows - m0 : BM;
    // (in whole dwords, as a copy's range check is: W's rows are padded where K is odd)
    q.N = p.K - n0 < BN ? (p.K - n0 + 1) & ~(int64_t)1 : BN;
    q.K = p.V - k0 < b.per ? p.V - k0 : b.per;
    q.lda = b.ldd;
    q.ldb = p.ldw;
    q.ldc = b.ldx2;
    q.align_a = q.align_c = 16;
    q.align_b = p.align_w;
    q.out_f32 = 1;
    f32x4 acc[R::FN][R::FM];
    R::zero(acc);
    if (b.more) {
        // the pieces before
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wm = wave / WGN, wn = wave % WGN;
#pragma unroll
        for (int fm = 0; fm < R::FM; ++fm)
#pragma unroll
            for (int fn = 0; fn < R::FN; ++fn) {
                const int r = wm * R::TM + fm * 16 + (lane & 15), n = wn * R::TN + fn * 16 + (lane >> 4) * 4;
                if (r < q.M && n < q.N) acc[fn][fm] = *(const f32x4 *)((const float *)q.C + r * b.ldx2 + n);
            }
    }
    multiply_tile<R, BM, BN, false, false>(q, smem, q.K, acc);
    q.N = (q.N + 7) & ~(int64_t)7;                 // whole chunks of the padded rows
    R::store(q, smem, TileCoord{0, 0, 0}, acc);
}

// dX or a piece's dW from planes of FP32 sums, added in a fixed order: scale
// alpha sum, rounded to the output's type; zeros for rows that `has` leaves out.
// SHARE threads per 8 columns, each with every SHARE-th plane: more than one
// where the columns alone would leave most CUs idle over many planes (20 x 300
// from 50 planes 6.3 us with four, 11.0 with one; 4096 x 4096 from one 42 and
// 22).
struct Total {
    const float *sums;
    const int32_t *has;          // or NULL
    void *out;
    int64_t rows, cols, ld, ldo, plane;
    int planes, out_f32;
    const float *alpha;
    float scale;
};
template <int SHARE>
__global__ void __launch_bounds__(256) k_vocab_total(Total t)
{
    const int64_t chunks = (t.cols + 7) / 8, total = t.rows * chunks;
    const float a = t.scale * *t.alpha;
    const int share = threadIdx.x % SHARE;
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / SHARE; at < total; at += (int64_t)gridDim.x * (256 / SHARE)) {
        const int64_t m = at / chunks, col = at % chunks * 8;
        const float *s = t.sums + m * t.ld + col;
        f32x4 v[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 8
        for (int i = share; i < t.planes; i += SHARE) {
            v[0] += *(const f32x4 *)(s + i * t.plane);
            v[1] += *(const f32x4 *)(s + i * t.plane + 4);
        }
#pragma unroll
        for (int o = 1; o < SHARE; o <<= 1)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] += __shfl_xor(v[j >> 2][j & 3], o, 64);
        if (share != 0) continue;
        const bool some = !t.has || t.has[m] != 0;
        float r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = some ? a * v[j >> 2][j & 3] : 0.f;
        const int64_t to = m * t.ldo + col;
        const int left = t.cols - col < 8 ? (int)(t.cols - col) : 8;
        if (t.out_f32) {
            float *out = (float *)t.out + to;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < left) out[j] = r[j];
            continue;
        }
        const u32x4 d = {pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7])};
        uint16_t *out = (uint16_t *)t.out + to;
        if (left == 8) {
            store16(out, d);
            continue;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < left) out[i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
    }
}

}  // namespace

static void tiles_of(VocabArgs &p, int64_t M, int64_t N, int tile)
{
    p.tiles_m = (M + tile - 1) / tile;
    p.tiles_n = (N + tile - 1) / tile;
    p.group_m = p.tiles_m < 8 ? p.tiles_m : 8;
}

hipError_t launch_vocab_stats(const VocabArgs &args, int tile, hipStream_t s)
{
    VocabArgs p = args;
    if (tile == 0) {
        const dim3 g((unsigned)((p.V + kVocabCols - 1) / kVocabCols)), b(kVocabWaves * 64);
        if (p.M > 16) hipLaunchKernelGGL((k_vocab_stream<2, 2, false>), g, b, 0, s, p, VocabGrad{});
        else hipLaunchKernelGGL((k_vocab_stream<1, 3, false>), g, b, 0, s, p, VocabGrad{});
        return hipGetLastError();
    }
    tiles_of(p, p.M, p.V, tile);
    const dim3 g((unsigned)(p.tiles_m * p.tiles_n)), b(512);
    if (tile == 256) hipLaunchKernelGGL((k_vocab_stats<256, 256, 2, 4>), g, b, 0, s, p);
    else hipLaunchKernelGGL((k_vocab_stats<128, 128, 4, 2>), g, b, 0, s, p);
    return hipGetLastError();
}

hipError_t launch_vocab_join(const VocabArgs &p, hipStream_t s)
{
    hipLaunchKernelGGL(k_vocab_join, dim3((unsigned)(p.M < 65536 ? p.M : 65536)), dim3(kJoinWaves * 64), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_vocab_prep(const VocabArgs &p, const VocabGrad &b, hipStream_t s)
{
    if (p.M <= kPrepFew) {
        hipLaunchKernelGGL(k_vocab_prep_few, dim3(1), dim3((unsigned)p.M * 64), 0, s, p, b);
        return hipGetLastError();
    }
    const dim3 g((unsigned)((p.M + kPrepWaves - 1) / kPrepWaves)), t(kPrepWaves * 64);
    if (p.M * p.topk <= kPrepScan) {
        hipLaunchKernelGGL(k_vocab_prep<true>, g, t, 0, s, p, b);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_vocab_prep<false>, g, t, 0, s, p, b);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_vocab_weights, dim3(1), dim3(1024), 0, s, b.weight, p.M, b.alpha);
    return hipGetLastError();
}

hipError_t launch_vocab_dlogits(const VocabArgs &args, const VocabGrad &b, int tile, hipStream_t s)
{
    VocabArgs p = args;
    if (tile == 0) {
        const dim3 g((unsigned)((p.V + kVocabCols - 1) / kVocabCols)), t(kVocabWaves * 64);
        if (p.M > 16) hipLaunchKernelGGL((k_vocab_stream<2, 2, true>), g, t, 0, s, p, b);
        else hipLaunchKernelGGL((k_vocab_stream<1, 3, true>), g, t, 0, s, p, b);
        return hipGetLastError();
    }
    tiles_of(p, p.M, p.V, tile);
    const dim3 g((unsigned)(p.tiles_m * p.tiles_n)), t(512);
    if (tile == 256) hipLaunchKernelGGL((k_vocab_dlogits<256, 256, 2, 4>), g, t, 0, s, p, b);
    else hipLaunchKernelGGL((k_vocab_dlogits<128, 128, 4, 2>), g, t, 0, s, p, b);
    return hipGetLastError();
}

static hipError_t launch_total(const Total &t, hipStream_t s)
{
    const int64_t chunks = t.rows * ((t.cols + 7) / 8);
    const int share = chunks <= 8192 && t.planes >= 32 ? 16 : chunks <= 32768 && t.planes >= 8 ? 4 : 1;
    const int64_t groups = (chunks * share + 255) / 256;
    const dim3 g((unsigned)(groups < 65536 ? groups : 65536)), b(256);
    if (share == 16) hipLaunchKernelGGL(k_vocab_total<16>, g, b, 0, s, t);
    else if (share == 4) hipLaunchKernelGGL(k_vocab_total<4>, g, b, 0, s, t);
    else hipLaunchKernelGGL(k_vocab_total<1>, g, b, 0, s, t);
    return hipGetLastError();
}

hipError_t launch_vocab_dw(const VocabArgs &args, const VocabGrad &b, int tile, hipStream_t s)
{
    VocabArgs p = args;
    tiles_of(p, p.V, p.K, tile);
    const dim3 g((unsigned)(b.w_slices * p.tiles_m * p.tiles_n)), t(512);
    if (tile == 256) hipLaunchKernelGGL((k_vocab_dw<256, 256, 2, 4>), g, t, 0, s, p, b);
    else hipLaunchKernelGGL((k_vocab_dw<128, 128, 4, 2>), g, t, 0, s, p, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || b.w_slices == 1) return e;
    return launch_total(Total{b.w_sums, nullptr, (char *)b.dW + p.v0 * b.lddw * (b.dw_f32 ? 4 : 2), p.V, p.K, b.ldx2, b.lddw,
                              p.V * b.ldx2, b.w_slices, b.dw_f32, b.alpha, p.scale},
                        s);
}

hipError_t launch_vocab_sums(const VocabArgs &args, const VocabGrad &b, int tile, hipStream_t s)
{
    VocabArgs p = args;
    tiles_of(p, p.M * b.parts, b.ldx2, tile);
    const dim3 g((unsigned)(b.slices * p.tiles_m * p.tiles_n)), t(512);
    if (tile == 256) hipLaunchKernelGGL((k_vocab_sums<256, 256, 2, 4>), g, t, 0, s, p, b);
    else hipLaunchKernelGGL((k_vocab_sums<128, 128, 4, 2>), g, t, 0, s, p, b);
    return hipGetLastError();
}

hipError_t launch_vocab_dx(const VocabArgs &p, const VocabGrad &b, hipStream_t s)
{
    return launch_total(Total{b.sums, b.has, b.dX, p.M, p.K, b.ldx2, b.lddx, p.M * b.ldx2, b.slices * b.parts, 0, b.alpha, p.scale},
                        s);
}

}  // namespace g5
