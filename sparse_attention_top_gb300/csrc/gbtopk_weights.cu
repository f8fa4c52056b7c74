// The weight each cached position accumulates (gbtopk_cache_weights).
#include "gbtopk_decode.cuh"

namespace gbtopk {
namespace {

struct WeightParams {
    const void *q, *k, *v;
    int64_t q_row, q_head, k_slot, k_head, v_slot, v_head;
    Paging pages;
    const int32_t *seq_lens;     // null: selected slots
    const int64_t *tree_mask;
    const int64_t *accept_mask;
    const int32_t *indices;
    int64_t top_k, idx_row;
    int64_t num_rows;
    int32_t next_n, q_heads, kv_heads, dim;
    float scale;
    void *out;
    float *lse;
    const float *lse_in;
    float *weights;
    int32_t weight_heads;
    int64_t width;
};

// Positions a row may see: [0, n), slot() < 0 where it sees none.
template <bool SELECTED>
struct Row {
    const WeightParams &p;
    int64_t r, i;
    int32_t ctx, n;
    uint64_t tree;
    __device__ Row(const WeightParams &p, int64_t r) : p(p), r(r) {
        if constexpr (SELECTED) {
            n = static_cast<int32_t>(p.top_k);
        } else {
            i = r / p.next_n;
            const int t = static_cast<int>(r - i * p.next_n);
            const int64_t len = p.seq_lens[i] > 0 ? p.seq_lens[i] : 0;
            ctx = static_cast<int32_t>(len - p.next_n);
            const int64_t room = p.pages.cols * p.pages.page.d;
            n = static_cast<int32_t>(len < room ? len : room);
            tree = p.tree_mask ? static_cast<uint64_t>(p.tree_mask[r]) : (~0ull >> (63 - t));
        }
    }
    __device__ int64_t slot(int32_t pos) const {
        if constexpr (SELECTED) {
            const int32_t s = p.indices[r * p.idx_row + pos];
            return s < p.pages.num_slots ? s : -1;
        } else {
            if (pos >= ctx && !((tree >> (pos - ctx)) & 1)) return -1;
            return p.pages.slot(i, pos);
        }
    }
};

template <bool BF16>
__device__ float dot(const float *q, const uint4 *k, int dim) {
    float s = 0;
    for (int c = 0; c < dim / 8; ++c) {
        const uint4 x = k[c];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        for (int j = 0; j < 4; ++j) {
            const float2 f = Half2<BF16>::up(w[j]);
            s = fmaf(f.x, q[c * 8 + 2 * j], s);
            s = fmaf(f.y, q[c * 8 + 2 * j + 1], s);
        }
    }
    return s;
}

// One thread for each (position, weight head) of a request.
template <bool BF16>
__global__ void __launch_bounds__(128) weights_kernel(WeightParams p) {
    using T = typename Half2<BF16>::T;
    __shared__ float q[GBTOPK_MAX_HEAD_DIM];
    pdl_wait();
    const int64_t i = blockIdx.y;
    const int w = blockIdx.z, group = p.q_heads / p.kv_heads, per = p.q_heads / p.weight_heads;
    const int64_t pos = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    const uint64_t took = p.accept_mask ? static_cast<uint64_t>(p.accept_mask[i]) : ~0ull;
    float sum = 0;
    for (int t = 0; t < p.next_n; ++t) {
        if (!((took >> t) & 1)) continue;
        const int64_t r = i * p.next_n + t;
        const Row<false> row(p, r);
        const int64_t slot = pos < row.n && pos < p.width ? row.slot(static_cast<int32_t>(pos)) : -1;
        for (int h = w * per; h < w * per + per; ++h) {
            __syncthreads();
            for (int d = threadIdx.x; d < p.dim; d += 128)
                q[d] = static_cast<float>(static_cast<const T *>(p.q)[r * p.q_row + h * p.q_head + d]);
            __syncthreads();
            const float lse = p.lse_in[r * p.q_heads + h];
            if (slot < 0 || lse == -INFINITY) continue;
            sum += expf(p.scale * dot<BF16>(q, reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k) +
                                                                               slot * p.k_slot + (h / group) * p.k_head),
                                            p.dim) - lse);
        }
    }
    if (pos < p.width) p.weights[(i * p.weight_heads + w) * p.width + pos] += sum;
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" int gbtopk_cache_weights(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                         int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *k_cache,
                         int64_t k_slot_stride, int64_t k_head_stride, int64_t num_slots, const float *lse,
                         const int32_t *page_table, int64_t pt_cols, int64_t pt_row_stride, int32_t page_size,
                         const int32_t *seq_lens, int32_t next_n, const int64_t *tree_mask,
                         const int64_t *accept_mask, float scale, float *weights, int32_t weight_heads, int64_t width,
                         void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (next_n < 1 || num_rows % next_n != 0 || width < 0) return GBTOPK_EINVAL;
    if (weight_heads != 1 && weight_heads != kv_heads) return GBTOPK_EINVAL;
    if (next_n > GBTOPK_MAX_NEXT_N || width > INT32_MAX) return GBTOPK_EUNSUPPORTED;
    WeightParams p{};
    if ((rc = check_pages(page_table, pt_cols, pt_row_stride, page_size, num_slots, num_rows / next_n, &p.pages)) != GBTOPK_OK)
        return rc;
    if (num_rows == 0 || width == 0) return GBTOPK_OK;
    if (!seq_lens || !lse || !weights) return GBTOPK_EINVAL;
    if ((rc = check_rows(q, q_row_stride, q_head_stride, true)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(k_cache, k_slot_stride, k_head_stride, num_slots > 0)) != GBTOPK_OK) return rc;
    if (!aligned_to(lse, 4) || !aligned_to(weights, 16)) return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < kWsHeaderBytes) return GBTOPK_EWORKSPACE;
    p.q = q;
    p.q_row = q_row_stride;
    p.q_head = q_head_stride;
    p.k = k_cache;
    p.k_slot = k_slot_stride;
    p.k_head = k_head_stride;
    p.num_rows = num_rows;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.dim = head_dim;
    p.scale = scale;
    p.seq_lens = seq_lens;
    p.next_n = next_n;
    p.tree_mask = tree_mask;
    p.accept_mask = accept_mask;
    p.lse_in = lse;
    p.weights = weights;
    p.weight_heads = weight_heads;
    p.width = width;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>((width + 127) / 128), static_cast<unsigned>(num_rows / next_n),
                    static_cast<unsigned>(weight_heads));
    if (grid.y > 65535) return GBTOPK_EUNSUPPORTED;
    return (dtype == GBTOPK_BF16 ? launch_pdl(weights_kernel<true>, grid, 128, 0, s, 1, p)
                                 : launch_pdl(weights_kernel<false>, grid, 128, 0, s, 1, p)) == cudaSuccess
               ? GBTOPK_OK
               : GBTOPK_ECUDA;
}

