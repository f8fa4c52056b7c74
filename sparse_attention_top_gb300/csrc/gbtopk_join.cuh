// Shared by the attention kernels: the references of their probabilities, and the
// join of units that span blocks, for the kernels over a paged cache that leave
// partial results.  Not part of the ABI.
#pragma once

#include <cfloat>
#include <cmath>

#include "gbtopk_paged.cuh"

namespace gbtopk {
namespace {

constexpr int kMaxGrid = 160;       // blocks of the attention kernel (workspace bound)

constexpr float kRescale = 8.f;     // rise of a tile's maximum over the reference m (base 2) that rescales O

// fp16 holds 2^-14 .. 2^15 with all its digits and nothing below 2^-25, so
// with m the maximum a key 17 nats above the others (an attention sink) left
// nothing of their P.  There the reference is 2^7 below a tile's maximum (P is
// at most 2^15 before O is rescaled), and it also falls, scaling O and l up,
// where a tile's maximum is more than 2^8 below the one that set it: every
// tile's P then reaches 2^-1 or more, and what its elements below 2^-14 lose is
// 2^-24 of the tile's largest each.  l stays at or below 2^80 (O below 2^127 for
// any values and lengths); what lies further down than that is below the
// smallest fp16 output.  The first reference gives the first tile's largest
// element a P of 2^7, which needs no rounding (with whole numbers as references
// short rows' error was 1.16 times as large); from there it moves by whole
// numbers, so that the many moves of a row add no error of their own to a sum
// that each of them may scale as a whole.  bf16 has the range of the sums.
// 32 requests x 4 drafts over 6000 positions: 129.4 -> 130.6 us; 8 x 64 drafts
// whose tiles' maxima jump by 10 nats at random, so that some row's reference
// moves at nearly every tile: 64.1 -> 69.0, without jumps 63.1 -> 63.2.
template <bool BF16>
constexpr float kLift = BF16 ? 0.f : 7.f;
constexpr float kMostSum = 0x1p80f;

// 2^x of a whole number, exactly (0 below 2^-126).
__device__ __forceinline__ float exp2_whole(float x) {
    return __int_as_float((static_cast<int>(fminf(fmaxf(x, -127.f), 128.f)) + 127) << 23);
}

// 2^(a - b) of two references.  In fp16 kernels the part that it scales down may
// be the larger one all the same (a high sum over a low reference), so what the
// subtraction of the two rounds off counts (Knuth, "The Art of Computer
// Programming", volume 2, 4.2.2, theorem B).
template <bool BF16>
__device__ __forceinline__ float exp2_between(float a, float b) {
    const float d = a - b, e = exp2_fast(d);
    if constexpr (BF16) return e;
    const float bv = __fsub_rn(d, a), rest = __fadd_rn(__fsub_rn(a, __fsub_rn(d, bv)), __fsub_rn(-b, bv));
    return e == 0.f ? 0.f : fmaf(e, rest * kLn2, e);
}

// Log-sum-exp of a row from its reference and sum (fp16: a high sum over a low
// reference, whose large parts cancel before the rest is added).
template <bool BF16>
__device__ __forceinline__ float row_lse(float m, float l) {
    if (l == 0.f) return -INFINITY;
    if constexpr (BF16) return (m + log2f(l)) * kLn2;
    int e;
    const float digits = frexpf(l, &e);
    return (m + static_cast<float>(e) + log2f(digits)) * kLn2;
}

// Joins the partial results of units that span blocks: blocks of 32 rows (a
// lane each) and sixteen warps, of COLS columns each, in GROUPS groups that
// take batches of BATCH parts in turn and are joined in order at the end; grid
// (units, row groups, column groups).  A batch is loaded at once: its latency
// bounds a join of many parts, which few units have.  So the shapes with more
// blocks and more parts in flight are taken as long as their blocks all run at
// once, one an SM by their registers:
//     four columns, four groups of sixteen parts (1 request x 4 drafts, 16
//     heads over one of 128, 65536 positions, 152 parts: 20.1 us a call; one
//     request of 1027 positions over eight heads, 9 tiles: 11.7);
//     four columns, sixteen parts (34.4; 12.2. 1 request x 64 drafts, 32 heads
//     over four, 8192 positions: 26.8);
//     eight columns, eight parts at dimension 128 (44.7; 13.2; 29.0. 4 requests
//     x 32 drafts, 32 heads over four, 8192 positions: 33.9, against 36.6 with
//     the next);
//     all columns, four parts otherwise (8 requests x 32 drafts, 16 heads over
//     two of 256, 4096 positions: 39.7, with four and sixteen 44).
constexpr int kCombineRows = 32, kCombineThreads = 512;

template <bool BF16, int DP, int COLS, int BATCH, int GROUPS>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ AttnParams p, int32_t unit_rows) {
    pdl_wait();
    pdl_release();
    const int2 ends = reinterpret_cast<const int2 *>(p.unit_ends)[blockIdx.x];
    const int32_t c0 = ends.x, c1 = ends.y;
    if (c0 == c1 || c0 < 0 || c1 < c0 || c1 >= kMaxGrid) return;   // whole, or not written by a block that gave up
    const int32_t b = static_cast<int32_t>(blockIdx.x / p.request_units), hm = static_cast<int32_t>(blockIdx.x % p.request_units);
    const int32_t h = hm / p.row_tiles, r0 = (hm - h * p.row_tiles) * unit_rows;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t row = static_cast<int32_t>(blockIdx.y) * kCombineRows + lane;
    const bool mine = row < unit_rows && r0 + row < p.next_n * p.group;
    constexpr int kCols = COLS, kBatch = BATCH, kWarps = kCombineThreads / 32 / GROUPS;   // warps of a group
    const int32_t col = static_cast<int32_t>(blockIdx.z * kWarps + warp % kWarps) * kCols;
    float m = -INFINITY, l = 0.f, acc[kCols] = {};
    // the parts (x: m, y: l) and o of a batch, joined to m, l, acc
    auto join = [&](const float2 *ml, const float (*o)[kCols], int n) {
        float top = m;
#pragma unroll
        for (int k = 0; k < n; ++k) top = fmaxf(top, ml[k].x);
        const float f = l == 0.f ? 0.f : exp2_between<BF16>(m, top);
        m = top;
        l *= f;
#pragma unroll
        for (int d = 0; d < kCols; ++d) acc[d] *= f;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            if (ml[k].y == 0.f) continue;   // (a NaN score leaves it NaN)
            const float fk = exp2_between<BF16>(ml[k].x, top);
            l += ml[k].y * fk;
#pragma unroll
            for (int d = 0; d < kCols; ++d) acc[d] += fk * o[k][d];
        }
    };
    if (mine) {
        for (int32_t g0 = c0 + warp / kWarps * kBatch; g0 <= c1; g0 += GROUPS * kBatch) {
            float2 ml[kBatch];
            float o[kBatch][kCols];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                ml[k] = make_float2(-INFINITY, 0.f);
                if (g0 + k > c1) continue;
                const int64_t part = 2ll * (g0 + k) + (g0 + k == c0 ? 1 : 0);
                ml[k] = p.part_ml[part * unit_rows + row];
#pragma unroll
                for (int d = 0; d < kCols; ++d) o[k][d] = p.part_o[(part * DP + col + d) * unit_rows + row];
            }
            join(ml, o, kBatch);
        }
    }
    if constexpr (GROUPS > 1) {   // the groups' results, in order
        __shared__ float2 group_ml[GROUPS - 1][kWarps][32];
        __shared__ float group_o[GROUPS - 1][kWarps][kCols][32];
        const int g = warp / kWarps - 1, w = warp % kWarps;
        if (g >= 0) {
            group_ml[g][w][lane] = make_float2(m, l);
#pragma unroll
            for (int d = 0; d < kCols; ++d) group_o[g][w][d][lane] = acc[d];
        }
        __syncthreads();
        if (g >= 0) return;
        float2 ml[GROUPS - 1];
        float o[GROUPS - 1][kCols];
#pragma unroll
        for (int k = 0; k < GROUPS - 1; ++k) {
            ml[k] = group_ml[k][w][lane];
#pragma unroll
            for (int d = 0; d < kCols; ++d) o[k][d] = group_o[k][w][d][lane];
        }
        join(ml, o, GROUPS - 1);
    }
    if (!mine) return;
    const int32_t t = (r0 + row) / p.group, gq = r0 + row - t * p.group;
    const int64_t q_at = (static_cast<int64_t>(b) * p.next_n + t) * p.q_heads + h * p.group + gq;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int d = 0; d < kCols; d += 4) {
        if (col + d >= p.dim) break;
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + 2 * (q_at * p.dim + col + d)) =
            make_uint2(Half2<BF16>::down(acc[d] * inv, acc[d + 1] * inv), Half2<BF16>::down(acc[d + 2] * inv, acc[d + 3] * inv));
    }
    if (p.lse && col == 0) p.lse[q_at] = row_lse<BF16>(m, l);
}

inline int dim_class(int32_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

inline size_t partial_rows(int32_t dim) { return static_cast<size_t>(2 * kMaxGrid) * (dim > 128 ? 128 : 256); }
inline size_t unit_bytes(int64_t num_rows, int32_t q_heads) {   // a unit has a row or more
    return (static_cast<size_t>(num_rows) * q_heads * 8 + 255) / 256 * 256;
}

// Lays the units' ends and the parts out in the workspace.
inline void place_parts(AttnParams &p, uint8_t *ws) {
    p.unit_ends = reinterpret_cast<int32_t *>(ws + kWsHeaderBytes);
    p.part_ml = reinterpret_cast<float2 *>(ws + kWsHeaderBytes + unit_bytes(static_cast<int64_t>(p.requests) * p.next_n, p.q_heads));
    p.part_o = reinterpret_cast<float *>(p.part_ml + partial_rows(p.dim));
}

// Joins units of unit_rows rows and tiles of `tile` positions.
template <bool BF16, int DP>
cudaError_t launch_join(const AttnParams &p, int32_t unit_rows, int tile, int sms, cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.next_n) * p.group;
    const int64_t units = static_cast<int64_t>(p.requests) * p.request_units;
    // no unit spans blocks where none has more than one tile
    const int64_t longest = p.seq_lens ? p.pages.cols * p.pages.page.d : p.top_k;
    if (longest <= tile) return cudaSuccess;
    const int64_t each = rows < unit_rows ? rows : unit_rows;
    dim3 blocks(static_cast<unsigned>(units), static_cast<unsigned>((each + kCombineRows - 1) / kCombineRows));
    blocks.z = DP / 16;
    if (units * blocks.y * blocks.z <= sms)
        return launch_pdl(combine_kernel<BF16, DP, 4, 16, 4>, blocks, kCombineThreads, 0, stream, 1, p, unit_rows);
    blocks.z = DP / 64;
    if (units * blocks.y * blocks.z <= sms)
        return launch_pdl(combine_kernel<BF16, DP, 4, 16, 1>, blocks, kCombineThreads, 0, stream, 1, p, unit_rows);
    blocks.z = 1;
    if (DP == 128 && units * blocks.y <= sms)
        return launch_pdl(combine_kernel<BF16, DP, DP / 16, DP == 128 ? 8 : 4, 1>, blocks, kCombineThreads, 0, stream, 1, p, unit_rows);
    return launch_pdl(combine_kernel<BF16, DP, DP / 16, 4, 1>, blocks, kCombineThreads, 0, stream, 1, p, unit_rows);
}

}  // namespace
}  // namespace gbtopk
