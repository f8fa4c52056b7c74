// Attention of drafted tokens over a paged cache (gbtopk_tree_attention),
// over selected slots (gbtopk_selected_attention), and the weight each
// cached position accumulates (gbtopk_cache_weights).
#include "gbtopk_decode.cuh"

namespace gbtopk {
namespace {

struct AttnParams {
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
    const AttnParams &p;
    int64_t r, i;
    int32_t ctx, n;
    uint64_t tree;
    __device__ Row(const AttnParams &p, int64_t r) : p(p), r(r) {
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

__device__ float block_max(float v, float *red) {
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}
__device__ float block_sum(float v, float *red) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// One block of 128 threads for each (row, query head): 128 positions at a
// time, their scores by one thread each, then each thread sums two columns
// of the values.
template <bool BF16, bool SELECTED>
__global__ void __launch_bounds__(128) attention_kernel(AttnParams p) {
    using T = typename Half2<BF16>::T;
    __shared__ float q[GBTOPK_MAX_HEAD_DIM], prob[128], red[4];
    __shared__ int64_t where[128];
    pdl_wait();
    const int64_t r = blockIdx.x;
    const int h = blockIdx.y, g = h / (p.q_heads / p.kv_heads);
    for (int d = threadIdx.x; d < p.dim; d += 128)
        q[d] = static_cast<float>(static_cast<const T *>(p.q)[r * p.q_row + h * p.q_head + d]);
    const Row<SELECTED> row(p, r);
    float m = -INFINITY, l = 0, o[2] = {0, 0};
    for (int32_t p0 = 0; p0 < row.n; p0 += 128) {
        __syncthreads();
        const int32_t pos = p0 + static_cast<int32_t>(threadIdx.x);
        const int64_t slot = pos < row.n ? row.slot(pos) : -1;
        const float s = slot < 0 ? -INFINITY
                                 : p.scale * dot<BF16>(q, reinterpret_cast<const uint4 *>(static_cast<const T *>(p.k) +
                                                                                          slot * p.k_slot + g * p.k_head),
                                                       p.dim);
        const float top = fmaxf(m, block_max(s, red));
        if (top == -INFINITY) continue;
        const float e = expf(s - top), f = expf(m - top);
        prob[threadIdx.x] = e;
        where[threadIdx.x] = slot;
        l = l * f + block_sum(e, red);
        m = top;
        for (int c = 0; c < 2; ++c) {
            const int d = static_cast<int>(threadIdx.x) + 128 * c;
            if (d >= p.dim) break;
            float a = o[c] * f;
            for (int j = 0; j < 128; ++j)
                if (where[j] >= 0)
                    a += prob[j] * static_cast<float>(static_cast<const T *>(p.v)[where[j] * p.v_slot + g * p.v_head + d]);
            o[c] = a;
        }
    }
    for (int c = 0; c < 2; ++c) {
        const int d = static_cast<int>(threadIdx.x) + 128 * c;
        if (d < p.dim)
            static_cast<T *>(p.out)[(r * p.q_heads + h) * p.dim + d] = static_cast<T>(m == -INFINITY ? 0.f : o[c] / l);
    }
    if (p.lse && threadIdx.x == 0) p.lse[r * p.q_heads + h] = m == -INFINITY ? -INFINITY : m + logf(l);
}

// One thread for each (position, weight head) of a request.
template <bool BF16>
__global__ void __launch_bounds__(128) weights_kernel(AttnParams p) {
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

int check_heads(int dtype, int64_t num_rows, int32_t q_heads, int32_t kv_heads, int32_t dim) {
    if (dtype != GBTOPK_F32 && dtype != GBTOPK_BF16 && dtype != GBTOPK_F16) return GBTOPK_EINVAL;
    if (num_rows < 0 || q_heads < 1 || kv_heads < 1 || dim < 1 || q_heads % kv_heads != 0) return GBTOPK_EINVAL;
    if (dtype == GBTOPK_F32 || dim > GBTOPK_MAX_HEAD_DIM || dim % 8 != 0) return GBTOPK_EUNSUPPORTED;
    if (num_rows > INT32_MAX || q_heads > 65535) return GBTOPK_EUNSUPPORTED;
    return GBTOPK_OK;
}

// Rows of 16-bit elements read in 16-byte pieces; `any`: there are some.
int check_rows(const void *base, int64_t a, int64_t b, bool any) {
    if (any && !base) return GBTOPK_EINVAL;
    if (a < 0 || b < 0) return GBTOPK_EINVAL;
    if (!aligned_to(base, 16) || !multiple_of(a, 8) || !multiple_of(b, 8)) return GBTOPK_EALIGN;
    return GBTOPK_OK;
}

int check_pages(const int32_t *table, int64_t cols, int64_t stride, int32_t page, int64_t num_slots,
                int64_t requests, Paging *out) {
    if (page < 1 || page > (1 << 30) || cols < 0 || num_slots < 0 || (requests > 1 && stride < cols)) return GBTOPK_EINVAL;
    if (requests > 0 && cols > 0 && !table) return GBTOPK_EINVAL;
    if (cols > INT32_MAX / page) cols = INT32_MAX / page;  // positions are 31-bit numbers
    out->table = table;
    out->cols = cols;
    out->row_stride = stride;
    out->num_slots = num_slots;
    out->page.init(static_cast<uint32_t>(page));
    return GBTOPK_OK;
}

template <bool BF16>
cudaError_t launch_attention(const AttnParams &p, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.num_rows), static_cast<unsigned>(p.q_heads));
    return p.seq_lens ? launch_pdl(attention_kernel<BF16, false>, grid, 128, 0, stream, 1, p)
                      : launch_pdl(attention_kernel<BF16, true>, grid, 128, 0, stream, 1, p);
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

namespace {

int attend(AttnParams &p, int dtype, const void *q, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
           int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *k_cache, int64_t k_slot_stride,
           int64_t k_head_stride, const void *v_cache, int64_t v_slot_stride, int64_t v_head_stride, float scale,
           void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    int rc;
    const int64_t num_slots = p.pages.num_slots;
    if ((rc = check_rows(q, q_row_stride, q_head_stride, true)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(k_cache, k_slot_stride, k_head_stride, num_slots > 0)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(v_cache, v_slot_stride, v_head_stride, num_slots > 0)) != GBTOPK_OK) return rc;
    if (!out) return GBTOPK_EINVAL;
    if (!aligned_to(out, 16) || !aligned_to(lse, 4)) return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) ||
        workspace_bytes < gbtopk_attention_workspace_bytes(num_rows, q_heads, kv_heads, head_dim))
        return GBTOPK_EWORKSPACE;
    p.q = q;
    p.q_row = q_row_stride;
    p.q_head = q_head_stride;
    p.k = k_cache;
    p.k_slot = k_slot_stride;
    p.k_head = k_head_stride;
    p.v = v_cache;
    p.v_slot = v_slot_stride;
    p.v_head = v_head_stride;
    p.num_rows = num_rows;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.dim = head_dim;
    p.scale = scale;
    p.out = out;
    p.lse = lse;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return (dtype == GBTOPK_BF16 ? launch_attention<true>(p, s) : launch_attention<false>(p, s)) == cudaSuccess
               ? GBTOPK_OK
               : GBTOPK_ECUDA;
}

}  // namespace

extern "C" {

size_t gbtopk_attention_workspace_bytes(int64_t num_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (check_heads(GBTOPK_BF16, num_rows, q_heads, kv_heads, head_dim) != GBTOPK_OK) return 0;
    return kWsHeaderBytes;
}

int gbtopk_tree_attention(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                          int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *k_cache,
                          int64_t k_slot_stride, int64_t k_head_stride, const void *v_cache, int64_t v_slot_stride,
                          int64_t v_head_stride, int64_t num_slots, const int32_t *page_table, int64_t pt_cols,
                          int64_t pt_row_stride, int32_t page_size, const int32_t *seq_lens, int32_t next_n,
                          const int64_t *tree_mask, float scale, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (next_n < 1 || num_rows % next_n != 0) return GBTOPK_EINVAL;
    if (next_n > GBTOPK_MAX_NEXT_N) return GBTOPK_EUNSUPPORTED;
    AttnParams p{};
    if ((rc = check_pages(page_table, pt_cols, pt_row_stride, page_size, num_slots, num_rows / next_n, &p.pages)) != GBTOPK_OK)
        return rc;
    if (num_rows == 0) return GBTOPK_OK;
    if (!seq_lens) return GBTOPK_EINVAL;
    p.seq_lens = seq_lens;
    p.next_n = next_n;
    p.tree_mask = tree_mask;
    return attend(p, dtype, q, num_rows, q_row_stride, q_head_stride, q_heads, kv_heads, head_dim, k_cache, k_slot_stride,
                  k_head_stride, v_cache, v_slot_stride, v_head_stride, scale, out, lse, workspace, workspace_bytes, stream);
}

int gbtopk_selected_attention(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                              int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *k_cache,
                              int64_t k_slot_stride, int64_t k_head_stride, const void *v_cache, int64_t v_slot_stride,
                              int64_t v_head_stride, int64_t num_slots, const int32_t *indices, int64_t top_k,
                              int64_t idx_row_stride, float scale, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (top_k < 0 || num_slots < 0 || (num_rows > 1 && idx_row_stride < top_k)) return GBTOPK_EINVAL;
    if (top_k > INT32_MAX / 2) return GBTOPK_EUNSUPPORTED;
    if (num_rows == 0) return GBTOPK_OK;
    if (top_k > 0 && !indices) return GBTOPK_EINVAL;
    AttnParams p{};
    p.pages.num_slots = num_slots;
    p.indices = indices;
    p.top_k = top_k;
    p.idx_row = idx_row_stride;
    p.next_n = 1;
    return attend(p, dtype, q, num_rows, q_row_stride, q_head_stride, q_heads, kv_heads, head_dim, k_cache, k_slot_stride,
                  k_head_stride, v_cache, v_slot_stride, v_head_stride, scale, out, lse, workspace, workspace_bytes, stream);
}

int gbtopk_cache_weights(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
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
    AttnParams p{};
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

}  // extern "C"
