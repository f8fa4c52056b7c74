// Shared by the tensor-core kernels over a paged cache (gbtopk_attention.cu,
// gbtopk_weights.cu): their arguments, the equal split of a ragged batch's
// tiles over the blocks, and the copies of cached rows.  Not part of the ABI.
#pragma once

#include <cstdlib>

#include "gbtopk_decode.cuh"
#include "gbtopk_mma.cuh"

namespace gbtopk {

// Limit of the kernels' waits in cycles: kWaitCycles, or the positive value
// of GBTOPK_WAIT_POLLS (read once a process), which lets a test run them out.
inline int64_t wait_cycles() {
    static const int64_t cycles = [] {
        const char *v = std::getenv("GBTOPK_WAIT_POLLS");
        char *end = nullptr;
        const unsigned long x = v && *v ? std::strtoul(v, &end, 10) : 0;
        return x > 0 && *end == '\0' && x < kWaitCycles ? static_cast<int64_t>(x) : static_cast<int64_t>(kWaitCycles);
    }();
    return cycles;
}

struct AttnParams {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_slot, k_head, v_slot, v_head;  // strides in elements
    Paging pages;
    const int32_t *seq_lens;     // null: selected slots
    const int64_t *tree_mask;
    const int32_t *indices;
    int64_t idx_row;
    int32_t top_k;
    int32_t requests;            // selected: rows
    int32_t next_n, q_heads, kv_heads, group, dim;
    int32_t row_tiles;           // row tiles of a (request, kv head)
    int32_t request_units;       // units of a request
    float c;                     // |scale| log2 e
    int32_t negative;            // scale < 0: the products are negated
    void *out;
    float *lse;
    uint32_t *status;
    int64_t wait_cycles;         // limit of each wait
    int32_t *unit_ends;          // first and last block of each unit
    float *part_o;               // [2 grid][rows of a tile][DP]
    float2 *part_ml;             // [2 grid][rows of a tile]
};

// Cached positions of request b, and the first drafted one.
struct Span {
    int32_t n, ctx;
};

__device__ __forceinline__ Span span_of(const AttnParams &p, int32_t b) {
    if (!p.seq_lens) return Span{p.top_k, INT32_MAX};
    const int32_t raw = fetch(p.seq_lens + b);
    const int32_t len = raw > 0 ? raw : 0;
    const int64_t room = p.pages.cols * p.pages.page.d;
    return Span{static_cast<int32_t>(len < room ? len : room), len - p.next_n};
}

// Every request has at least one tile, so that rows that see nothing are
// written too.
template <int KT>
__device__ __forceinline__ int32_t tiles_of(const Span &s) {
    return s.n > KT ? (s.n - 1) / KT + 1 : 1;
}

// A unit's cost beside its tiles (its queries, first products and output), in
// tiles: measured 9,000 to 20,000 cycles against 2,000 to 4,000 a tile.  Shares
// are equal in cost; with equal tile counts the block that held the shortest
// requests took 1.4 times the mean.
constexpr int kUnitCost = 3;

// The block's part of one unit: position tiles t0 .. t1 - 1 of `tiles`.
struct Unit {
    int32_t b, hm, t0, t1, tiles;
    Span span;
};

struct ScanScratch {
    int64_t warps[16], low[16];
    int64_t off;
    int32_t b;
};

// A block's share of the call: `cost` from offset `off` in the units of
// request b on.  A unit's cost is kUnitCost and then one a tile.
struct Share {
    int64_t off, cost;
    int32_t b;
};

// Walks the units of a share that it has tiles of.
template <int KT>
struct Walk {
    const AttnParams &p;
    int64_t left;    // cost of the share behind the present unit
    bool here = false;
    Unit u;
    __device__ Walk(const AttnParams &p, const Share &s) : p(p), left(s.cost) {
        if (left <= 0) return;
        u.b = s.b;
        u.span = span_of(p, u.b);
        u.tiles = tiles_of<KT>(u.span);
        u.hm = static_cast<int32_t>(s.off / (u.tiles + kUnitCost));
        clip(s.off - static_cast<int64_t>(u.hm) * (u.tiles + kUnitCost));
        if (u.t0 == u.t1) next();
    }
    // The part of the unit from offset v on; its cost leaves the share.
    __device__ void clip(int64_t v) {
        const int64_t all = u.tiles + kUnitCost, end = v + left < all ? v + left : all;
        left -= end - v;
        u.t0 = v > kUnitCost ? static_cast<int32_t>(v - kUnitCost) : 0;
        u.t1 = end > kUnitCost ? static_cast<int32_t>(end - kUnitCost) : 0;
        here = u.t1 > u.t0;
    }
    __device__ bool more() const { return here; }
    __device__ void next() {
        here = false;
        while (left > 0 && !here) {
            if (++u.hm == p.request_units) {
                u.hm = 0;
                u.span = span_of(p, ++u.b);
                u.tiles = tiles_of<KT>(u.span);
            }
            clip(0);
        }
    }
};

// Cost of the call, and in *before that of the requests below b, summed by
// the block.
template <int KT, int THREADS>
__device__ int64_t sum_cost(const AttnParams &p, int32_t b, int64_t *before, ScanScratch *scratch) {
    if (!p.seq_lens) {
        const int64_t each = static_cast<int64_t>(tiles_of<KT>(span_of(p, 0)) + kUnitCost) * p.request_units;
        *before = b * each;
        return p.requests * each;
    }
    int64_t all = 0, low = 0;
    for (int32_t x = threadIdx.x; x < p.requests; x += THREADS) {
        const int32_t v = tiles_of<KT>(span_of(p, x)) + kUnitCost;
        all += v;
        low += x < b ? v : 0;
    }
    for (int o = 16; o; o >>= 1) {
        all += __shfl_xor_sync(~0u, all, o);
        low += __shfl_xor_sync(~0u, low, o);
    }
    if ((threadIdx.x & 31) == 0) {
        scratch->warps[threadIdx.x >> 5] = all;
        scratch->low[threadIdx.x >> 5] = low;
    }
    __syncthreads();
    all = low = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        all += scratch->warps[w];
        low += scratch->low[w];
    }
    __syncthreads();
    *before = low * p.request_units;
    return all * p.request_units;
}

// The blockIdx.x-th of gridDim.x equal shares.
template <int KT, int THREADS>
__device__ Share block_share(const AttnParams &p, ScanScratch *scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t before;
    const int64_t total = sum_cost<KT, THREADS>(p, 0, &before, scratch);
    const int64_t per = (total + gridDim.x - 1) / gridDim.x, start = per * blockIdx.x;
    Share s{0, start >= total ? 0 : (start + per < total ? per : total - start), 0};
    if (s.cost == 0) return s;
    if (!p.seq_lens) {
        const int64_t each = static_cast<int64_t>(tiles_of<KT>(span_of(p, 0)) + kUnitCost) * p.request_units;
        s.b = static_cast<int32_t>(start / each);
        s.off = start - s.b * each;
        return s;
    }
    int64_t base = 0;
    for (int32_t b0 = 0; b0 < p.requests; b0 += THREADS) {
        const int32_t b = b0 + static_cast<int32_t>(threadIdx.x);
        const int64_t v = b < p.requests ? static_cast<int64_t>(tiles_of<KT>(span_of(p, b)) + kUnitCost) * p.request_units : 0;
        int64_t inc = v;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) scratch->warps[warp] = inc;
        __syncthreads();
        int64_t all = 0;
        before = base;
        for (int w = 0; w < THREADS / 32; ++w) {
            before += w < warp ? scratch->warps[w] : 0;
            all += scratch->warps[w];
        }
        const int64_t at = before + inc - v;
        if (start >= at && start < at + v) {
            scratch->b = b;
            scratch->off = start - at;
        }
        base += all;
        __syncthreads();
        if (start < base) break;
    }
    s.b = scratch->b;
    s.off = scratch->off;
    return s;
}

// Copies one tile's rows, of which each of four warps has KT / 4: eight lanes
// a row of a 128-byte panel, four rows an instruction, so that a row's address
// is computed once for all its panels.  `slot` is the slot of the warp's row
// `lane`; rows without one, and columns at or beyond `loaded` chunks, become
// zeros.  (One lane group a whole row, two rows an instruction, took 62 cycles
// an instruction and bound the attention kernel at 3.9 TB/s.)
template <int DP, int KT>
__device__ __forceinline__ void copy_tile(uint32_t dst, const uint8_t *base, int64_t slot_bytes, int32_t slot,
                                          int32_t chunks, int32_t loaded, int warp, int lane) {
    constexpr int kMine = KT / 4, kPanels = DP / 64;
    const int c0 = lane & 7, sub = lane >> 3;
    base += c0 * 16;
    dst += (warp * kMine + sub) * 128;
    const uint32_t off[2] = {static_cast<uint32_t>((c0 ^ sub) << 4), static_cast<uint32_t>((c0 ^ (sub + 4)) << 4)};
#pragma unroll
    for (int it = 0; it < kMine / 4; ++it) {
        const int32_t s = __shfl_sync(~0u, slot, it * 4 + sub);
        const uint8_t *src = base + static_cast<int64_t>(s < 0 ? 0 : s) * slot_bytes;
#pragma unroll
        for (int n = 0; n < kPanels; ++n)
            if (n * 8 + c0 < chunks)
                copy16(dst + it * 512 + off[it & 1] + n * (KT * 128), src + n * 128, s >= 0 && n * 8 + c0 < loaded ? 16u : 0u);
    }
}

}  // namespace gbtopk
