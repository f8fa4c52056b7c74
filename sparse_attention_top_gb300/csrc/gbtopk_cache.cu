// Eviction from a paged cache by accumulated weight (gbtopk_cache_evict).
//
// evict_select_kernel: a cluster of 1 to 8 blocks for each (request, weight
// head).  Each block stages the order-preserving keys of its slice of the
// survivors in shared memory, three rounds of 11-bit radix histograms (summed
// over the cluster through distributed shared memory) give the key at the
// budget (8-bit rounds put all weights of one sign and a few binades into a
// handful of bins, whose atomics serialised: 30 us for 17000 weights), and one
// ordered pass (warp segments, prefix sums) writes the kept positions in place.
// evict_move_kernel then copies the kept rows, blocks of about 32 KB of keys
// and values.
//
// The copies are bound by their bytes: 32 requests x 8 heads of 128, 4096 kept
// positions each, 150 us = 7.1 TB/s read and written.  The selection of those
// 256 rows of up to 32768 weights takes 50 us, bound by the instructions of its
// five passes over the keys in shared memory; one row of 5001 weights, both
// kernels, 15 us.
#include <cooperative_groups.h>

#include "gbtopk_decode.cuh"

namespace cg = cooperative_groups;

namespace gbtopk {
namespace {

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kStagedKeys = 49152;   // keys a block can stage (192 KB)
constexpr int kMaxCluster = 8;

struct EvictParams {
    const float *weights;
    const int32_t *seq_lens;
    const int64_t *accept_mask;
    int64_t requests, width;
    int32_t heads, next_n, budget, recent;
    Paging from, to;
    uint8_t *cache[2];
    int64_t slot_bytes[2], head_bytes[2];
    int32_t kv_heads, row_chunks;  // 16-byte chunks of one (slot, head) row
    int32_t *kept, *new_lens;
    float *out_weights;
    int32_t move_rows;     // kept positions a block of evict_move_kernel copies
    int32_t row_blocks;
    int32_t staged;        // keys staged in shared memory (else read again)
};

__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kBins11 = 2048;

// The weight of a key (+0 for either zero).
__device__ __forceinline__ float key_weight(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

struct SelectShared {
    alignas(16) uint32_t hist[kBins11];
    uint32_t scan[kSelectWarps];
    uint32_t gt[kSelectWarps], eq[kSelectWarps];   // kept for sure, equal to the key: by warp, then before each
    uint32_t all_gt[kMaxCluster], all_eq[kMaxCluster];
    int32_t draft[64];
    uint32_t bin, need, count;
};

__global__ void __launch_bounds__(kSelectThreads, 2) evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ __align__(16) uint32_t keys[];
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int size = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_release();
    const int64_t row = blockIdx.x / size, i = row / p.heads;
    const float *w = p.weights + row * p.width;
    int32_t *kept = p.kept + row * p.budget;
    float *out_w = p.out_weights + row * p.width;
    const int32_t raw = p.seq_lens[i], len = raw > 0 ? raw : 0;
    const int64_t room = p.from.cols * p.from.page.d < p.width ? p.from.cols * p.from.page.d : p.width;
    const int32_t lim = static_cast<int32_t>(len < room ? len : room);
    // survivors in order: positions 0 .. a - 1, then draft[0 .. nd - 1]
    int32_t a = lim, nd = 0;
    if (p.accept_mask) {
        const int32_t ctx = len - p.next_n;
        a = ctx < 0 ? 0 : (ctx < lim ? ctx : lim);
        const int32_t lo = ctx < 0 ? -ctx : 0, hi = lim - ctx < p.next_n ? lim - ctx : p.next_n;
        uint64_t bits = static_cast<uint64_t>(p.accept_mask[i]);
        bits = hi > lo ? bits & (~0ull >> (64 - hi)) & (~0ull << lo) : 0;
        nd = __popcll(bits);
        if (tid < 64 && ((bits >> tid) & 1)) sh.draft[__popcll(bits & ((1ull << tid) - 1))] = ctx + tid;
    }
    const int32_t n = a + nd, m = n < p.budget ? n : p.budget;
    const int32_t recent = p.recent < p.budget ? p.recent : p.budget;
    const int32_t cut = n <= p.budget ? 0 : n - recent;   // survivors below the cut compete
    uint32_t need = n <= p.budget ? 0u : static_cast<uint32_t>(p.budget - recent);
    // the block's slice of the survivors
    const int32_t each = (n + size - 1) / size;
    const int32_t s0 = rank * each < n ? rank * each : n, s1 = s0 + each < n ? s0 + each : n;
    const int32_t c1 = s1 < cut ? s1 : (s0 < cut ? cut : s0);   // its competitors: s0 .. c1 - 1
    // also: every block of the cluster runs before any other writes to it
    if (size > 1) cluster.sync();
    else __syncthreads();
    auto pos = [&](int32_t s) { return s < a ? s : sh.draft[s - a]; };
    // keys of the slice's survivors o .. o + 3, o a multiple of 4; those from
    // `end` on hold anything
    auto keys_at = [&](int32_t o, int32_t end) {
        if (p.staged) return o < end ? *reinterpret_cast<const uint4 *>(keys + o) : make_uint4(0, 0, 0, 0);
        uint32_t k[4] = {};
        for (int j = 0; j < 4; ++j)
            if (o + j < end) k[j] = weight_key(w[pos(s0 + o + j)]);
        return make_uint4(k[0], k[1], k[2], k[3]);
    };
    if (p.staged) {   // eight loads in flight a thread
        constexpr int kUnroll = 8;
        for (int32_t b = s0 + tid; b < s1; b += kSelectThreads * kUnroll) {
            float x[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (b + u * kSelectThreads < s1) x[u] = w[pos(b + u * kSelectThreads)];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (b + u * kSelectThreads < s1) keys[b + u * kSelectThreads - s0] = weight_key(x[u]);
        }
        __syncthreads();
    }
    // the key t at the budget: keys above it are kept, and the first `need`
    // equal to it (with `whole` every key of at least t)
    uint32_t t = 0;
    bool whole = false;
    for (int round = 0; round < 3 && need && !whole; ++round) {
        const int shift = 21 - 11 * round < 0 ? 0 : 21 - 11 * round;   // digits of 11, 11 and 10 bits
        const uint32_t digit = round < 2 ? kBins11 - 1 : kBins11 / 2 - 1;
        for (int b = tid; b < kBins11; b += kSelectThreads) sh.hist[b] = 0;
        __syncthreads();
        const uint32_t above_digit = ~(digit | ((1u << shift) - 1) | (digit << shift));
        for (int32_t o = tid * 4; o - tid * 4 < c1 - s0; o += kSelectThreads * 4) {
            const uint4 v = keys_at(o, c1 - s0);
            const uint32_t k[4] = {v.x, v.y, v.z, v.w};
            uint32_t bin[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                bin[j] = o + j < c1 - s0 && ((k[j] ^ t) & above_digit) == 0 ? (k[j] >> shift) & digit : kBins11;
            // a warp of equal keys adds once
            const uint32_t lead = __shfl_sync(~0u, bin[0], 0);
            if (__all_sync(~0u, bin[0] == lead && bin[1] == lead && bin[2] == lead && bin[3] == lead)) {
                if (lane == 0 && lead < kBins11) atomicAdd(&sh.hist[lead], 128u);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (bin[j] < kBins11) atomicAdd(&sh.hist[bin[j]], 1u);
            }
        }
        if (size > 1) cluster.sync();
        else __syncthreads();
        // four bins a thread, the highest in thread 0
        const int hi = kBins11 - 1 - 4 * tid;
        uint32_t h[4] = {}, mine = 0;
        for (int r = 0; r < size; ++r) {
            const uint4 x = *reinterpret_cast<const uint4 *>(cluster.map_shared_rank(sh.hist, r) + hi - 3);
            h[0] += x.w;
            h[1] += x.z;
            h[2] += x.y;
            h[3] += x.x;
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) mine += h[b];
        uint32_t inc = mine;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        uint32_t above = lane < warp ? sh.scan[lane] : 0;   // in higher bins
        for (int o = 16; o; o >>= 1) above += __shfl_xor_sync(~0u, above, o);
        above += inc - mine;
        if (above < need && above + mine >= need) {
            uint32_t left = need - above;
            bool found = false;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (found) continue;
                if (left > h[b]) {
                    left -= h[b];
                    continue;
                }
                found = true;
                sh.bin = static_cast<uint32_t>(hi - b);
                sh.need = left;
                sh.count = h[b];
            }
        }
        if (size > 1) cluster.sync();
        else __syncthreads();
        t |= sh.bin << shift;
        need = sh.need;
        whole = need == sh.count;
    }
    const bool compete = cut > 0 && p.budget > recent;
    // ordered pass: each warp a segment of the slice, four survivors a lane
    const int32_t held = s1 - s0;
    const int32_t seg = ((held + kSelectWarps - 1) / kSelectWarps + 127) / 128 * 128;
    const int32_t b0 = warp * seg < held ? warp * seg : held, b1 = b0 + seg < held ? b0 + seg : held;
    // bits of the four from offset o on: kept for sure, equal to the key
    auto classify = [&](int32_t o, uint32_t *equal) {
        const uint4 v = keys_at(o, b1);
        const uint32_t k[4] = {v.x, v.y, v.z, v.w};
        uint32_t g = 0, e = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (o + j >= b1) continue;
            const bool late = s0 + o + j >= cut;
            g |= static_cast<uint32_t>(late || (compete && (whole ? k[j] >= t : k[j] > t))) << j;
            e |= static_cast<uint32_t>(!late && compete && !whole && k[j] == t) << j;
        }
        *equal = e;
        return g;
    };
    uint32_t gt = 0, eq = 0;
    for (int32_t o = b0 + lane * 4; o < b1; o += 128) {
        uint32_t e;
        gt += __popc(classify(o, &e));
        eq += __popc(e);
    }
    gt = __reduce_add_sync(~0u, gt);
    eq = __reduce_add_sync(~0u, eq);
    if (lane == 0) {
        sh.gt[warp] = gt;
        sh.eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        uint32_t g = lane < kSelectWarps ? sh.gt[lane] : 0, e = lane < kSelectWarps ? sh.eq[lane] : 0, gi = g, ei = e;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(~0u, gi, o), y = __shfl_up_sync(~0u, ei, o);
            if (lane >= o) {
                gi += x;
                ei += y;
            }
        }
        if (lane < kSelectWarps) {
            sh.gt[lane] = gi - g;
            sh.eq[lane] = ei - e;
        }
        if (lane == 31)
            for (int r = 0; r < size; ++r) {
                cluster.map_shared_rank(sh.all_gt, r)[rank] = gi;
                cluster.map_shared_rank(sh.all_eq, r)[rank] = ei;
            }
    }
    if (size > 1) cluster.sync();
    else __syncthreads();
    gt = sh.gt[warp];
    eq = sh.eq[warp];
    for (int r = 0; r < rank; ++r) {
        gt += sh.all_gt[r];
        eq += sh.all_eq[r];
    }
    for (int32_t o0 = b0; o0 < b1; o0 += 128) {
        const int32_t o = o0 + lane * 4;
        uint32_t e;
        const uint32_t g = classify(o, &e), mine = __popc(g) | __popc(e) << 16;
        uint32_t inc = mine;
        for (int i = 1; i < 32; i <<= 1) {
            const uint32_t x = __shfl_up_sync(~0u, inc, i);
            if (lane >= i) inc += x;
        }
        const uint32_t all = __shfl_sync(~0u, inc, 31), before = inc - mine;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t low = (1u << j) - 1, eb = eq + (before >> 16) + __popc(e & low);   // equal keys before this one
            if (((g >> j) & 1) || (((e >> j) & 1) && eb < need)) {
                const uint32_t at = gt + (before & 0xffff) + __popc(g & low) + (eb < need ? eb : need);
                const int32_t q = pos(s0 + o + j);
                kept[at] = q;
                out_w[at] = key_weight(p.staged ? keys[o + j] : weight_key(w[q]));
            }
        }
        gt += all & 0xffff;
        eq += all >> 16;
    }
    for (int64_t j = m + rank * kSelectThreads + tid; j < p.budget; j += size * kSelectThreads) kept[j] = -1;
    for (int64_t j = m + rank * kSelectThreads + tid; j < p.width; j += size * kSelectThreads) out_w[j] = 0.f;
    if (rank == 0 && tid == 0 && row % p.heads == 0) p.new_lens[i] = m;
}

// Copies kept rows: row_blocks blocks of move_rows kept positions for each
// (request, weight head).  Consecutive threads copy consecutive 16-byte chunks of a
// position's heads; two keys' and two values' chunks are in flight a thread.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kUnroll = 2;
    __shared__ int64_t src[64], dst[64];
    pdl_wait();
    pdl_release();
    const int64_t row = blockIdx.x / p.row_blocks, i = row / p.heads;
    const int32_t j0 = static_cast<int32_t>(blockIdx.x % p.row_blocks) * p.move_rows;
    const int32_t m = p.new_lens[i];
    const int32_t rows = m - j0 < p.move_rows ? m - j0 : p.move_rows;
    if (rows <= 0) return;
    if (static_cast<int32_t>(threadIdx.x) < rows) {
        const int32_t j = j0 + static_cast<int32_t>(threadIdx.x);
        src[threadIdx.x] = p.from.slot(i, p.kept[row * p.budget + j]);
        dst[threadIdx.x] = p.to.slot(i, j);
    }
    __syncthreads();
    const int32_t h0 = p.heads == 1 ? 0 : static_cast<int32_t>(row % p.heads), heads = p.heads == 1 ? p.kv_heads : 1;
    const int32_t per = heads * p.row_chunks, total = rows * per;
    for (int32_t x0 = threadIdx.x; x0 < total; x0 += kMoveThreads * kUnroll) {
        uint4 v[kUnroll][2];
        uint8_t *to[kUnroll][2];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t x = x0 + u * kMoveThreads;
            to[u][0] = nullptr;
            if (x >= total) continue;
            const int32_t j = x / per, c = x - j * per, h = h0 + c / p.row_chunks, b = c % p.row_chunks;
            const int64_t s = src[j], d = dst[j];
            if (d < 0) continue;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                uint8_t *base = p.cache[kv] + h * p.head_bytes[kv] + b * 16;
                v[u][kv] = s < 0 ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4 *>(base + s * p.slot_bytes[kv]);
                to[u][kv] = base + d * p.slot_bytes[kv];
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (to[u][0])
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) *reinterpret_cast<uint4 *>(to[u][kv]) = v[u][kv];
    }
}

// Blocks of a selection's cluster: enough for two blocks an SM to stage their
// slices (256 rows of 32768 weights, one block each of 1024 threads: 56 us),
// and for rows that leave half of the SMs idle as many as leave each block 4096
// weights.
int select_cluster(int64_t rows, int64_t width, int sms) {
    int c = 1;
    while (c < kMaxCluster && ((width + c - 1) / c > 24576 || (rows * c * 2 <= sms && width / c > 4096))) c *= 2;
    return c;
}

bool overlap(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" int gbtopk_cache_evict(const float *weights, int64_t num_requests, int32_t weight_heads, int64_t width,
                                  const int32_t *seq_lens, int32_t next_n, const int64_t *accept_mask, int32_t budget,
                                  int32_t recent, void *k_cache, int64_t k_slot_stride, int64_t k_head_stride,
                                  void *v_cache, int64_t v_slot_stride, int64_t v_head_stride, int64_t num_slots,
                                  int32_t kv_heads, int32_t head_dim, int32_t elem_bytes, const int32_t *page_table,
                                  int64_t pt_cols, int64_t pt_row_stride, const int32_t *out_page_table,
                                  int64_t out_pt_cols, int64_t out_pt_row_stride, int32_t page_size, int32_t *kept,
                                  int32_t *new_lens, float *out_weights, void *stream) {
    if (num_requests < 0 || width < 0 || next_n < 1 || budget < 1 || recent < 0 || kv_heads < 1 || head_dim < 1)
        return GBTOPK_EINVAL;
    if (weight_heads != 1 && weight_heads != kv_heads) return GBTOPK_EINVAL;
    if (page_size < 1 || page_size > (1 << 30) || num_slots < 0 || pt_cols < 0 || out_pt_cols < 0) return GBTOPK_EINVAL;
    if (num_requests > 1 && (pt_row_stride < pt_cols || out_pt_row_stride < out_pt_cols)) return GBTOPK_EINVAL;
    if (out_pt_cols < (static_cast<int64_t>(budget) + page_size - 1) / page_size) return GBTOPK_EINVAL;
    if (elem_bytes != 2 && elem_bytes != 4) return GBTOPK_EUNSUPPORTED;
    if (next_n > GBTOPK_MAX_NEXT_N || width > INT32_MAX || num_requests > INT32_MAX / weight_heads || head_dim > (1 << 20) || kv_heads > 65535 ||
        static_cast<int64_t>(kv_heads) * head_dim > (1 << 26))
        return GBTOPK_EUNSUPPORTED;
    if (num_requests == 0) return GBTOPK_OK;
    if ((width > 0 && (!weights || !out_weights)) || !seq_lens || (num_slots > 0 && (!k_cache || !v_cache)) || !kept || !new_lens ||
        (pt_cols > 0 && !page_table) || !out_page_table)
        return GBTOPK_EINVAL;
    if (k_slot_stride < 0 || k_head_stride < 0 || v_slot_stride < 0 || v_head_stride < 0) return GBTOPK_EINVAL;
    const int32_t es = elem_bytes;
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !multiple_of(k_slot_stride * es, 16) ||
        !multiple_of(k_head_stride * es, 16) || !multiple_of(v_slot_stride * es, 16) ||
        !multiple_of(v_head_stride * es, 16) || !multiple_of(static_cast<int64_t>(head_dim) * es, 16) ||
        !aligned_to(weights, 16) || !aligned_to(out_weights, 16) || !aligned_to(kept, 16) || !aligned_to(new_lens, 4) ||
        !aligned_to(seq_lens, 4) || !aligned_to(accept_mask, 8) || !aligned_to(page_table, 4) || !aligned_to(out_page_table, 4))
        return GBTOPK_EALIGN;
    const size_t wbytes = static_cast<size_t>(num_requests) * weight_heads * width * 4;
    if (width > 0 && overlap(weights, wbytes, out_weights, wbytes)) return GBTOPK_EOVERLAP;
    // (a request's heads are separate blocks: one would read what another wrote)
    const size_t lbytes = static_cast<size_t>(num_requests) * 4;
    if (overlap(seq_lens, lbytes, new_lens, lbytes)) return GBTOPK_EOVERLAP;
    EvictParams p{};
    p.weights = weights;
    p.seq_lens = seq_lens;
    p.accept_mask = accept_mask;
    p.requests = num_requests;
    p.width = width;
    p.heads = weight_heads;
    p.next_n = next_n;
    p.budget = budget;
    p.recent = recent;
    p.from.table = page_table;
    p.from.cols = pt_cols < INT32_MAX / page_size ? pt_cols : INT32_MAX / page_size;
    p.from.row_stride = pt_row_stride;
    p.from.num_slots = num_slots;
    p.from.spare = seq_lens;
    p.from.page.init(static_cast<uint32_t>(page_size));
    p.to = p.from;
    p.to.table = out_page_table;
    p.to.cols = out_pt_cols;
    p.to.row_stride = out_pt_row_stride;
    p.cache[0] = static_cast<uint8_t *>(k_cache);
    p.cache[1] = static_cast<uint8_t *>(v_cache);
    p.slot_bytes[0] = k_slot_stride * es;
    p.slot_bytes[1] = v_slot_stride * es;
    p.head_bytes[0] = k_head_stride * es;
    p.head_bytes[1] = v_head_stride * es;
    p.kv_heads = kv_heads;
    p.row_chunks = head_dim * es / 16;
    p.kept = kept;
    p.new_lens = new_lens;
    p.out_weights = out_weights;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t rows = num_requests * weight_heads;
    const int sms = device_sms();
    if (sms == 0) return GBTOPK_ECUDA;
    const int cluster = select_cluster(rows, width, sms);
    const int64_t slice = (width + cluster - 1) / cluster;
    p.staged = slice <= kStagedKeys;
    const size_t smem = p.staged ? static_cast<size_t>((slice + 3) / 4) * 16 : 0;
    // 32 KB of keys and values a block, at most 64 positions
    const int64_t bytes = 2ll * head_dim * es * (weight_heads == 1 ? kv_heads : 1);
    p.move_rows = static_cast<int32_t>(bytes >= 32768 ? 1 : 32768 / bytes > 64 ? 64 : 32768 / bytes);
    p.row_blocks = (budget + p.move_rows - 1) / p.move_rows;
    if (rows * p.row_blocks > INT32_MAX || rows * cluster > INT32_MAX) return GBTOPK_EUNSUPPORTED;
    static std::atomic<uint64_t> allowed{0};
    if (allow_smem(evict_select_kernel, kStagedKeys * 4, allowed) != cudaSuccess) return GBTOPK_ECUDA;
    if (launch_pdl(evict_select_kernel, dim3(static_cast<unsigned>(rows * cluster)), kSelectThreads, smem, s, cluster, p) !=
        cudaSuccess)
        return GBTOPK_ECUDA;
    return launch_pdl(evict_move_kernel, dim3(static_cast<unsigned>(rows * p.row_blocks)), kMoveThreads, 0, s, 1, p) == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}
