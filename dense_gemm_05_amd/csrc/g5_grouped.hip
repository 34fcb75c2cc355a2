// g5_grouped.hip -- products grouped by expert with ragged numbers of rows.
//
// The rows of the token operand stand group behind group; offsets[e] ..
// offsets[e + 1] - 1 are group e's:
//
//   NT  C[r] = A[r] . Bt_e^T      the experts' projection, Bt [E, N, K]
//   NN  C[r] = A[r] . B_e         its input gradient, B [E, K, N]
//   TN  C_e = At_e^T . B_e        its weight gradient, C [E, M, N], the sum
//                                 over the group's rows
//
// The group sizes are known on the device only (a router's counts), so every
// workgroup finds its tile from the offsets itself: a wave takes a lane per
// group and adds up the tiles before it.  The grid is the most tiles that any
// offsets can give; workgroups past the last tile end at once.
#include <hip/hip_runtime.h>

#include "g5_device.h"
#include "g5_kernels.h"
#include "g5_ping.h"
#include "g5_stream.h"

namespace g5 {

namespace {

// 64 groups, a lane each: first row, rows, and tiles of BM rows up to and with
// the group.  Offsets are held to [0, M] and to ascending order (one lower
// than an earlier one counts as that), so that whatever they hold no row lies
// in two groups or outside the operands.  `floor`: the end of the group
// before; becomes the end of the last of these.
struct GroupLanes {
    int first, rows, tiles;
};
__device__ __forceinline__ GroupLanes scan_groups(const GroupedArgs &p, int base, int bm, int &floor)
{
    const int lane = threadIdx.x & 63, e = base + lane, M = (int)p.rows;
    auto held = [&](int v) { return v < 0 ? 0 : v > M ? M : v; };
    const int s = e < p.E ? held(p.offsets[e]) : 0, t = e < p.E ? held(p.offsets[e + 1]) : 0;
    int first = s > floor ? s : floor;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(first, o, 64);
        if (lane >= o && v > first) first = v;
    }
    const int end = t > first ? t : first;
    GroupLanes g{first, end - first, (end - first + bm - 1) / bm};
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(g.tiles, o, 64);
        if (lane >= o) g.tiles += v;
    }
    floor = __builtin_amdgcn_readlane(end, 63);
    return g;
}

// The tile of workgroup `wg`: tiles run group by group, and within a group in
// column bands of up to 8 tiles (the rows of a band meet each column panel of
// the group's weight one after the other), the whole sequence shared out over
// the XCDs in contiguous runs.
struct GroupTile {
    int group, row, rows, tn;      // its first row in A and C, and its rows
};
__device__ __forceinline__ bool find_tile(const GroupedArgs &p, int bm, GroupTile &t)
{
    int total = 0, floor = 0;
    GroupLanes g{};
    for (int base = 0; base < p.E; base += 64) {
        g = scan_groups(p, base, bm, floor);
        total += __builtin_amdgcn_readlane(g.tiles, 63);
    }
    const int64_t all = (int64_t)total * p.tiles_n;
    if ((int64_t)blockIdx.x >= all) return false;
    const int L = (int)tile_map(blockIdx.x, 1, all, 1, 1).tm;
    const int tiles_n = (int)p.tiles_n;
    const int at = L / tiles_n;                // in tiles of BM rows
    int before = 0;
    floor = 0;
    for (int base = 0; base < p.E; base += 64) {
        if (p.E > 64) g = scan_groups(p, base, bm, floor);
        const uint64_t past = __ballot(before + g.tiles > at);
        if (past) {
            const int lane = __builtin_ctzll(past);
            const int first = __builtin_amdgcn_readlane(g.first, lane), rows = __builtin_amdgcn_readlane(g.rows, lane);
            const int tiles = (rows + bm - 1) / bm;
            const int r = L - (before + __builtin_amdgcn_readlane(g.tiles, lane) - tiles) * tiles_n;
            const int band = r / (8 * tiles_n), left = tiles - 8 * band, h = left < 8 ? left : 8;
            const int rr = r - band * 8 * tiles_n, tm = 8 * band + rr % h;
            t.group = base + lane;
            t.row = first + tm * bm;
            t.rows = rows - tm * bm;
            if (t.rows > bm) t.rows = bm;
            t.tn = rr / h;
            return true;
        }
        before += __builtin_amdgcn_readlane(g.tiles, 63);
    }
    return false;
}

// Group e's rows alone.
__device__ __forceinline__ void find_group(const GroupedArgs &p, int e, int &first, int &rows)
{
    int floor = 0;
    for (int base = 0; base <= e; base += 64) {
        const GroupLanes g = scan_groups(p, base, 1, floor);
        if (e - base < 64) {
            first = __builtin_amdgcn_readlane(g.first, e - base);
            rows = __builtin_amdgcn_readlane(g.rows, e - base);
        }
    }
}

// An output tile on the LDS ring (RingTile): q's operand bases are at the
// tile's own first row and column, so that 32-bit offsets span no more than the
// tile's rows.  Where the summed axis walks rows (B of NN, both of TN), it
// goes in pieces of p.piece that keep them so.
template <class R, int KIND, int BM, int BN, int WGM, int WGN>
__device__ __forceinline__ void ring_tile(const GroupedArgs &p, GemmArgs &q, uint16_t *smem, int64_t K, int n0)
{
    q.lda = p.lda;
    q.ldb = p.ldb;
    q.align_a = p.align_a;
    q.align_b = p.align_b;
    // (columns of B in whole dwords: even, or padded by the host)
    const int64_t left = p.N - n0;
    q.N = left < BN ? (KIND == GROUPED_NT ? left : (left + 1) & ~(int64_t)1) : BN;
    typename R::Acc acc;
    R::zero(acc);
    for (int64_t done = 0; done < K;) {
        q.K = KIND != GROUPED_NT && K - done > p.piece ? p.piece : K - done;
        if (done > 0) __syncthreads();            // every wave is through with the ring
        multiply_tile<R, BM, BN, KIND == GROUPED_NT, KIND == GROUPED_TN>(q, smem, q.K, acc);
        done += q.K;
        q.A = (const char *)q.A + q.K * (KIND == GROUPED_TN ? p.lda : 1) * 2;
        q.B = (const char *)q.B + q.K * (KIND == GROUPED_NT ? 1 : p.ldb) * 2;
    }
    q.N = left < BN ? left : BN;
    store_rows<R, BM, BN, WGM, WGN>(q, smem, acc);
}

template <int BM, int BN, int WGM, int WGN, int KIND>
using GroupedRing = RingTile<BM, BN, WGM, WGN, 4, 4, 16, true, EPI_NONE, KIND == GROUPED_NT, false, KIND == GROUPED_TN>;

// HALF: a group's last tile that has no more than BM / 2 rows runs as one of
// that height (a mean of 512 rows in tiles of 256 otherwise multiplies a fifth
// of the rows for nothing).
//
// Measured, 64 groups drawn at random, weights of 1536 x 4096: the projection of
// 32768 rows 394 us (1047 TFLOP/s of the rows that exist; of the multiplied
// ones a ninth are the tails' padding), the input gradient of 16384 rows 258 us
// (799 TFLOP/s and 3.8 TB/s: the weights are read once, 805 MB, under tiles of
// 24 stages), the weight gradient of as many 404 us (4.4 TB/s, nearly all of it
// FP32 written; 473 into outputs that change from call to call).  Workgroups that walk over several tiles were slower (weight gradient
// 567 for 487, projection 418 for 401), and so were half tiles put last (419).
template <int BM, int BN, int WGM, int WGN, int KIND, bool HALF>
__global__ void __launch_bounds__(WGM *WGN * 64, 2) k_grouped(GroupedArgs p)
{
    using R = GroupedRing<BM, BN, WGM, WGN, KIND>;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[R::LDS_BYTES / 2];
    GemmArgs q{};
    q.ldc = p.ldc;
    q.out_f32 = p.out_f32;
    if constexpr (KIND == GROUPED_TN) {
        const TileCoord tc = tile_map(blockIdx.x, p.E * p.slices, p.tiles_m, p.tiles_n, p.group_m);
        const int e = (int)tc.b / p.slices, slice = (int)tc.b % p.slices;
        int first, rows;
        find_group(p, e, first, rows);
        if (p.slices > 1) {
            const int64_t per = (((int64_t)rows + p.slices - 1) / p.slices + 63) & ~(int64_t)63;
            const int from = slice * per < rows ? (int)(slice * per) : rows;
            first += from;
            rows = rows - from < per ? rows - from : (int)per;
        }
        const int m0 = (int)tc.tm * BM, n0 = (int)tc.tn * BN;
        q.A = p.A + (first * p.lda + m0);
        q.B = p.B + (first * p.ldb + n0);
        q.C = (char *)p.C + (e * p.sC + m0 * p.ldc + n0) * (p.out_f32 ? 4 : 2);
        if (p.slices > 1) {
            q.C = p.sums + ((slice * p.E + e) * p.M + m0) * p.ld_sums + n0;
            q.ldc = p.ld_sums;
            q.out_f32 = 1;
        }
        q.M = p.M - m0 < BM ? p.M - m0 : BM;
        ring_tile<R, KIND, BM, BN, WGM, WGN>(p, q, smem, rows, n0);
    } else {
        GroupTile t;
        if (!find_tile(p, BM, t)) return;
        const int n0 = t.tn * BN;
        q.A = p.A + t.row * p.lda;
        q.B = p.B + (t.group * p.sB + (KIND == GROUPED_NT ? n0 * p.ldb : n0));
        q.C = (char *)p.C + (t.row * p.ldc + n0) * (p.out_f32 ? 4 : 2);
        q.M = t.rows;
        if constexpr (HALF) {
            if (t.rows <= BM / 2) {
                ring_tile<GroupedRing<BM / 2, BN, WGM, WGN, KIND>, KIND, BM / 2, BN, WGM, WGN>(p, q, smem, p.K, n0);
                return;
            }
        }
        ring_tile<R, KIND, BM, BN, WGM, WGN>(p, q, smem, p.K, n0);
    }
}

// NT with a few rows per group (a decoding step): bound by reading the
// groups' weights once, so a workgroup owns 32 weight rows of one group,
// streamed from HBM into the matrix core by four waves on contiguous pieces of
// K, and up to 32 of the group's rows.  128 rows over 64 groups of 1536 x 4096
// 108 us (6.5 TB/s of the weights that occur).
constexpr int kStreamWaves = 4;

// NC chunks of 16 of the group's rows, RB blocks of 16 weight rows, D steps of
// 64 of K in flight.
template <int NC, int RB, int D>
__device__ __forceinline__ void stream_tile(const GroupedArgs &p, const GroupTile &t, f32x4 (&red)[kStreamWaves][RB][64])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, li = lane & 15;
    const int n0 = t.tn * (16 * RB), N = (int)p.N;
    const char *const W = (const char *)p.B + t.group * p.sB * 2;
    f32x4 acc[RB][NC];
    bool xok[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        xok[c] = 16 * c + li < t.rows;
#pragma unroll
        for (int r = 0; r < RB; ++r) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const int K = (int)p.K, steps = (K + 63) / 64;
    const int s0 = steps * wave / kStreamWaves, s1 = steps * (wave + 1) / kStreamWaves;
    // (rows past N repeat the tile's first and are not stored)
    const char *wbase[RB];
    uint32_t woff[RB];
#pragma unroll
    for (int r = 0; r < RB; ++r) {
        const int n = n0 + 16 * r < N ? n0 + 16 * r : n0;
        wbase[r] = W + n * p.ldb * 2;
        woff[r] = (uint32_t)(n + li < N ? li : 0) * (uint32_t)(p.ldb * 2) + 16 * g;
    }
    RowStream<false, RB, NC, D> b;
    auto tokens = [&](uint32_t (&xoff)[NC], bool (&ok)[NC]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            ok[c] = xok[c];
            xoff[c] = (uint32_t)(xok[c] ? 16 * c + li : 0) * (uint32_t)(p.lda * 2) + x_lane<false>(g);
        }
    };
    b.run(wbase, woff, (const char *)p.A + t.row * p.lda * 2, tokens, s0, s1, K, g, acc);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        __syncthreads();             // (the chunk before has been read)
#pragma unroll
        for (int r = 0; r < RB; ++r) red[wave][r][lane] = acc[r][c];
        __syncthreads();
        // a wave per block of 16 columns adds the waves' parts in order
        if (wave < RB && xok[c]) {
            f32x4 s = red[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) s += red[w][wave][lane];
            const int64_t n = n0 + 16 * wave + 4 * g;
            if (n < N) store4(p.C, p.out_f32 != 0, p.ldc, t.row + 16 * c + li, n, s, n + 4 <= N, t.row + t.rows, N, p.align_c);
        }
    }
}

// 32 weight rows past up to 32 rows of a group.
__global__ void __launch_bounds__(kStreamWaves * 64, 4) k_grouped_stream(GroupedArgs p)
{
    __shared__ f32x4 red[kStreamWaves][2][64];
    GroupTile t;
    if (!find_tile(p, 32, t)) return;
    if (t.rows > 16) stream_tile<2, 2, 2>(p, t, red);
    else stream_tile<1, 2, 3>(p, t, red);
}

// 16 RB weight rows past up to 64.
template <int RB>
__global__ void __launch_bounds__(kStreamWaves * 64, 2) k_grouped_stream_many(GroupedArgs p)
{
    __shared__ f32x4 red[kStreamWaves][RB][64];
    GroupTile t;
    if (!find_tile(p, 64, t)) return;
    constexpr int D = RB == 4 ? 2 : 3;
    if (t.rows > 48) stream_tile<4, RB, D>(p, t, red);
    else if (t.rows > 32) stream_tile<3, RB, D>(p, t, red);
    else if (t.rows > 16) stream_tile<2, RB, D + 1>(p, t, red);
    else stream_tile<1, RB, D + 1>(p, t, red);
}

// The slices' sums of TN added in order.
__global__ void __launch_bounds__(256) k_grouped_total(GroupedArgs p)
{
    const int64_t chunks = p.ld_sums / 4, rows = p.E * p.M, plane = rows * p.ld_sums;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < rows * chunks; at += (int64_t)gridDim.x * 256) {
        const int64_t row = at / chunks, n = at % chunks * 4, e = row / p.M, m = row % p.M;
        const float *s = p.sums + row * p.ld_sums + n;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int i = 0; i < p.slices; ++i) v += *(const f32x4 *)(s + i * plane);
        store4((char *)p.C + e * p.sC * (p.out_f32 ? 4 : 2), p.out_f32 != 0, p.ldc, m, n, v, n + 4 <= p.N, p.M, p.N, p.align_c);
    }
}

template <int BM, int BN, int WGM, int WGN>
hipError_t launch_kind(int kind, const GroupedArgs &a, int64_t grid, hipStream_t s)
{
    const dim3 g((unsigned)grid), b(WGM * WGN * 64);
    constexpr bool HALF = BM == 256;
    switch (kind) {
    case GROUPED_NT: hipLaunchKernelGGL((k_grouped<BM, BN, WGM, WGN, GROUPED_NT, HALF>), g, b, 0, s, a); break;
    case GROUPED_NN: hipLaunchKernelGGL((k_grouped<BM, BN, WGM, WGN, GROUPED_NN, HALF>), g, b, 0, s, a); break;
    case GROUPED_TN: hipLaunchKernelGGL((k_grouped<BM, BN, WGM, WGN, GROUPED_TN, false>), g, b, 0, s, a); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(int kind, const GroupedArgs &args, int tile, hipStream_t s)
{
    GroupedArgs a = args;
    const int64_t grid = grouped_grid(kind, a.E, a.rows, a.M, a.N, tile, a.slices);
    const int64_t bn = grouped_tile_n(tile);
    a.tiles_n = (a.N + bn - 1) / bn;
    a.tiles_m = (a.M + grouped_tile_m(tile) - 1) / grouped_tile_m(tile);
    a.group_m = a.tiles_m < 8 ? a.tiles_m : 8;
    // Weight gradients: a run of tiles per XCD gives it whole groups, and the
    // one with the longest groups is waited for.  So the tiles go round the XCDs
    // one by one in bands of two (us, run / one by one: 64 groups of 1536 x 4096
    // FP32, 256 rows each 574 / 461, 78 rows 376 / 311; 8 of them, 2048 rows 262
    // / 215), but for short groups whose outputs the Infinity Cache holds (32 of
    // 1024 x 1536, 125 rows 49 / 54; 40 of 700 x 1002, 75 rows 40 / 45).
    if (kind == GROUPED_TN && (a.rows > 128 * a.E || a.E * a.M * a.N * (a.out_f32 ? 4 : 2) > (int64_t)1 << 28)) a.group_m = -2;
    switch (tile) {
    case GROUPED_STREAM:
    case GROUPED_STREAM_64x32:
    case GROUPED_STREAM_64x64: {
        if (kind != GROUPED_NT) return hipErrorInvalidValue;
        const dim3 g((unsigned)grid), b(kStreamWaves * 64);
        if (tile == GROUPED_STREAM) hipLaunchKernelGGL(k_grouped_stream, g, b, 0, s, a);
        else if (tile == GROUPED_STREAM_64x32) hipLaunchKernelGGL(k_grouped_stream_many<2>, g, b, 0, s, a);
        else hipLaunchKernelGGL(k_grouped_stream_many<4>, g, b, 0, s, a);
        return hipGetLastError();
    }
    case GROUPED_128:
    case GROUPED_256: break;
    default: return hipErrorInvalidValue;
    }
    const hipError_t e = tile == GROUPED_256 ? launch_kind<256, 256, 2, 4>(kind, a, grid, s) : launch_kind<128, 128, 4, 2>(kind, a, grid, s);
    if (e != hipSuccess || a.slices == 1) return e;
    const int64_t groups = (a.E * a.M * (a.ld_sums / 4) + 255) / 256;
    hipLaunchKernelGGL(k_grouped_total, dim3((unsigned)(groups < 65536 ? groups : 65536)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace g5
