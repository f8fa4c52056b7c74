// Eviction from a paged cache by accumulated weight (gbtopk_cache_evict).
#include "gbtopk_decode.cuh"

namespace gbtopk {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kMoveThreads = 256;

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
};

__device__ __forceinline__ uint32_t weight_key(float w) {
    const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sum over the block of `v` and, in *before, the sum over lower threads.
__device__ uint32_t block_scan(uint32_t v, uint32_t *warps, uint32_t *before) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = v;
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(~0u, s, o);
        if (lane >= static_cast<uint32_t>(o)) s += x;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    uint32_t base = 0, all = 0;
    for (uint32_t w = 0; w < kEvictThreads / 32; ++w) {
        base += w < warp ? warps[w] : 0;
        all += warps[w];
    }
    *before = base + s - v;
    return all;
}

// One block for each (request, weight head).
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(EvictParams p) {
    __shared__ uint32_t hist[256], scan[kEvictThreads / 32], pick[2];
    __shared__ int32_t draft[64];
    pdl_wait();
    const int64_t i = blockIdx.x / p.heads, row = blockIdx.x;
    const float *w = p.weights + row * p.width;
    int32_t *kept = p.kept + row * p.budget;
    float *out_w = p.out_weights + row * p.width;
    const int64_t len = p.seq_lens[i] > 0 ? p.seq_lens[i] : 0;
    const int64_t room = p.from.cols * p.from.page.d < p.width ? p.from.cols * p.from.page.d : p.width;
    const int32_t lim = static_cast<int32_t>(len < room ? len : room);
    // survivors in order: positions 0 .. a - 1, then draft[0 .. nd - 1]
    int32_t a = lim, nd = 0;
    if (p.accept_mask) {
        const int32_t ctx = static_cast<int32_t>(len - p.next_n);
        a = ctx < 0 ? 0 : (ctx < lim ? ctx : lim);
        const uint64_t bits = static_cast<uint64_t>(p.accept_mask[i]);
        for (int j = 0; j < p.next_n; ++j) {
            if (!((bits >> j) & 1) || ctx + j < 0 || ctx + j >= lim) continue;
            if (threadIdx.x == 0) draft[nd] = ctx + j;
            ++nd;
        }
        __syncthreads();
    }
    const int32_t n = a + nd, m = n < p.budget ? n : p.budget;
    const int32_t recent = p.recent < p.budget ? p.recent : p.budget;
    const int32_t cut = n <= p.budget ? 0 : n - recent;  // survivors below the cut compete
    uint32_t t = 0, need = static_cast<uint32_t>(n <= p.budget ? 0 : p.budget - recent);
    auto pos = [&](int32_t s) { return s < a ? s : draft[s - a]; };
    for (int shift = 24; shift >= 0 && need; shift -= 8) {
        for (int b = threadIdx.x; b < 256; b += kEvictThreads) hist[b] = 0;
        __syncthreads();
        for (int32_t s = threadIdx.x; s < cut; s += kEvictThreads) {
            const uint32_t k = weight_key(w[pos(s)]);
            if (shift == 24 || (k >> (shift + 8)) == (t >> (shift + 8))) atomicAdd(hist + ((k >> shift) & 255), 1u);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            int b = 255;
            for (; b > 0 && need > hist[b]; --b) need -= hist[b];
            pick[0] = static_cast<uint32_t>(b);
            pick[1] = need;
        }
        __syncthreads();
        t |= pick[0] << shift;
        need = pick[1];
    }
    const bool any = p.budget > recent && cut > 0;  // keys above t, and the first `need` equal to it
    uint32_t ties = 0, at = 0;
    for (int32_t s0 = 0; s0 < n; s0 += kEvictThreads) {
        const int32_t s = s0 + static_cast<int32_t>(threadIdx.x);
        const uint32_t k = s < cut ? weight_key(w[pos(s)]) : 0;
        const bool tie = s < cut && any && k == t;
        uint32_t before, nb;
        const uint32_t all_ties = block_scan(tie ? 1u : 0u, scan, &before);
        const bool keep = s < n && (s >= cut || (any && k > t) || (tie && ties + before < need));
        const uint32_t all = block_scan(keep ? 1u : 0u, scan, &nb);
        if (keep) {
            kept[at + nb] = pos(s);
            out_w[at + nb] = w[pos(s)];
        }
        ties += all_ties;
        at += all;
    }
    for (int64_t j = m + threadIdx.x; j < p.budget; j += kEvictThreads) kept[j] = -1;
    for (int64_t j = m + threadIdx.x; j < p.width; j += kEvictThreads) out_w[j] = 0.f;
    if (threadIdx.x == 0 && row % p.heads == 0) p.new_lens[i] = m;
}

// One thread for each 16-byte chunk of the kept rows of keys and values.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictParams p) {
    pdl_wait();
    const int64_t i = blockIdx.y;
    const int32_t m = p.new_lens[i];
    const int32_t per = p.kv_heads * p.row_chunks;
    const int64_t total = static_cast<int64_t>(m) * per;
    for (int64_t x = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; x < total;
         x += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
        const int32_t j = static_cast<int32_t>(x / per), c = static_cast<int32_t>(x % per);
        const int32_t h = c / p.row_chunks, b = c % p.row_chunks;
        const int32_t pos = p.kept[(i * p.heads + (p.heads == 1 ? 0 : h)) * p.budget + j];
        const int64_t src = p.from.slot(i, pos), dst = p.to.slot(i, j);
        if (dst < 0) continue;
        for (int kv = 0; kv < 2; ++kv) {
            uint8_t *base = p.cache[kv] + h * p.head_bytes[kv] + b * 16;
            const uint4 v = src < 0 ? make_uint4(0, 0, 0, 0)
                                    : *reinterpret_cast<const uint4 *>(base + src * p.slot_bytes[kv]);
            *reinterpret_cast<uint4 *>(base + dst * p.slot_bytes[kv]) = v;
        }
    }
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
    if (next_n > GBTOPK_MAX_NEXT_N || width > INT32_MAX || num_requests > 65535 ||
        num_requests * weight_heads > INT32_MAX || head_dim > (1 << 20) || kv_heads > 65535 ||
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
        !aligned_to(weights, 16) || !aligned_to(out_weights, 16) || !aligned_to(kept, 16) || !aligned_to(new_lens, 4))
        return GBTOPK_EALIGN;
    const size_t wbytes = static_cast<size_t>(num_requests) * weight_heads * width * 4;
    if (width > 0 && overlap(weights, wbytes, out_weights, wbytes)) return GBTOPK_EOVERLAP;
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
    if (launch_pdl(evict_select_kernel, dim3(static_cast<unsigned>(num_requests * weight_heads)), kEvictThreads, 0, s, 1,
                   p) != cudaSuccess)
        return GBTOPK_ECUDA;
    const int64_t most = (static_cast<int64_t>(budget) * kv_heads * p.row_chunks + kMoveThreads - 1) / kMoveThreads;
    const dim3 grid(static_cast<unsigned>(most < 4096 ? most : 4096), static_cast<unsigned>(num_requests));
    return launch_pdl(evict_move_kernel, grid, kMoveThreads, 0, s, 1, p) == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}
