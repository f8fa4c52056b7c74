// Verification of drafted tokens against the target's distributions
// (gbtopk_verify_drafts).
#include "gbtopk_decode.cuh"

namespace gbtopk {
namespace {

constexpr int kVerifyThreads = 1024;

struct VerifyParams {
    const void *logits;
    int64_t num_rows, vocab, row_stride;
    const int32_t *tokens;
    const float *uniforms, *noise;
    int32_t next_n;
    const int64_t *tree_mask;
    const float *temperature, *draft_probs;
    int32_t *accepted, *path, *next_token;
    int64_t *accept_mask;
    uint8_t *ws;
};

// Of one row of logits: its largest value, that value's lowest index and
// the sum of exp((x - top) / temperature).
struct RowStat {
    float top, sum;
    int32_t first;
};

template <int DT>
__device__ __forceinline__ float logit(const void *x, int64_t at) {
    if constexpr (DT == GBTOPK_F32) return static_cast<const float *>(x)[at];
    if constexpr (DT == GBTOPK_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[at]);
    return __half2float(static_cast<const __half *>(x)[at]);
}

__device__ __forceinline__ void better(float &v, int32_t &i, float v2, int32_t i2) {
    if (v2 > v || (v2 == v && i2 < i)) {
        v = v2;
        i = i2;
    }
}

// Every thread gets the block's largest value (lowest index).
__device__ void block_argmax(float &v, int32_t &i, float *sv, int32_t *si) {
    for (int o = 16; o; o >>= 1) better(v, i, __shfl_xor_sync(~0u, v, o), __shfl_xor_sync(~0u, i, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        sv[threadIdx.x >> 5] = v;
        si[threadIdx.x >> 5] = i;
    }
    __syncthreads();
    v = sv[0];
    i = si[0];
    for (int w = 1; w < kVerifyThreads / 32; ++w) better(v, i, sv[w], si[w]);
}

template <int DT>
__global__ void __launch_bounds__(kVerifyThreads) verify_stat_kernel(VerifyParams p) {
    __shared__ float sv[32];
    __shared__ int32_t si[32];
    pdl_wait();
    const int64_t r = blockIdx.x, base = r * p.row_stride;
    const float t = p.temperature ? p.temperature[r / p.next_n] : 1.f;
    float top = -INFINITY;
    int32_t first = INT32_MAX;
    for (int64_t c = threadIdx.x; c < p.vocab; c += kVerifyThreads)
        better(top, first, logit<DT>(p.logits, base + c), static_cast<int32_t>(c));
    block_argmax(top, first, sv, si);
    float sum = 0;
    if (t > 0 && top > -INFINITY)
        for (int64_t c = threadIdx.x; c < p.vocab; c += kVerifyThreads) sum += expf((logit<DT>(p.logits, base + c) - top) / t);
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sv[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0;
        for (int w = 0; w < kVerifyThreads / 32; ++w) sum += sv[w];
        reinterpret_cast<RowStat *>(p.ws + kWsHeaderBytes)[r] = RowStat{top, sum, first};
    }
}

template <int DT>
__device__ __forceinline__ float prob(const VerifyParams &p, const RowStat &st, int64_t r, float t, int64_t v) {
    if (st.top == -INFINITY) return 0.f;
    if (t <= 0) return v == st.first ? 1.f : 0.f;
    return expf((logit<DT>(p.logits, r * p.row_stride + v) - st.top) / t) / st.sum;
}

template <int DT>
__global__ void __launch_bounds__(kVerifyThreads) verify_walk_kernel(VerifyParams p) {
    __shared__ float sv[32];
    __shared__ int32_t si[32];
    __shared__ int32_t refused[GBTOPK_MAX_NEXT_N], s_refused, s_cur;
    pdl_wait();
    const int64_t i = blockIdx.x, r0 = i * p.next_n;
    const RowStat *stat = reinterpret_cast<const RowStat *>(p.ws + kWsHeaderBytes) + r0;
    const float t = p.temperature ? p.temperature[i] : 1.f;
    if (threadIdx.x == 0) {
        int cur = 0, count = 0, n_ref = 0;
        uint64_t took = 1;
        p.path[r0] = 0;
        float mass = 1.f;
        for (int c = 1; c < p.next_n; ++c) {
            int parent = c - 1;
            if (p.tree_mask) {
                const uint64_t above = static_cast<uint64_t>(p.tree_mask[r0 + c]) & ((1ull << c) - 1);
                parent = above ? 63 - __clzll(static_cast<long long>(above)) : -1;
            }
            if (parent != cur) continue;
            const int32_t x = p.tokens[r0 + c];
            float have = 0, q = mass;
            bool again = false;
            if (x >= 0 && x < p.vocab) {
                for (int k = 0; k < n_ref; ++k) again |= refused[k] == x;
                have = again ? 0.f : prob<DT>(p, stat[cur], r0 + cur, t, x);
                if (p.draft_probs) q = p.draft_probs[(r0 + cur) * p.vocab + x];
            }
            if (p.uniforms[r0 + c] * q < have) {
                cur = c;
                took |= 1ull << c;
                p.path[r0 + ++count] = c;
                n_ref = 0;
                mass = 1.f;
            } else {
                refused[n_ref++] = x;
                mass -= have;
            }
        }
        for (int k = count + 1; k < p.next_n; ++k) p.path[r0 + k] = -1;
        p.accepted[i] = count;
        p.accept_mask[i] = static_cast<int64_t>(took);
        s_cur = cur;
        s_refused = n_ref;
    }
    __syncthreads();
    const int cur = s_cur, n_ref = s_refused;
    const RowStat st = stat[cur];
    float best = 0;
    int32_t token = INT32_MAX;
    for (int64_t v = threadIdx.x; v < p.vocab; v += kVerifyThreads) {
        float rest = prob<DT>(p, st, r0 + cur, t, v);
        if (n_ref) {
            if (p.draft_probs) {
                rest -= p.draft_probs[(r0 + cur) * p.vocab + v];
            } else {
                for (int k = 0; k < n_ref; ++k)
                    if (refused[k] == v) rest = 0;
            }
        }
        if (rest > 0) better(best, token, rest / p.noise[i * p.vocab + v], static_cast<int32_t>(v));
    }
    block_argmax(best, token, sv, si);
    if (threadIdx.x == 0) p.next_token[i] = best > 0 ? token : -1;
}

template <int DT>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t s) {
    const cudaError_t e = launch_pdl(verify_stat_kernel<DT>, dim3(static_cast<unsigned>(p.num_rows)), kVerifyThreads, 0, s, 1, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(verify_walk_kernel<DT>, dim3(static_cast<unsigned>(p.num_rows / p.next_n)), kVerifyThreads, 0, s, 1, p);
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" {

size_t gbtopk_verify_workspace_bytes(int64_t num_rows, int64_t vocab, int32_t next_n) {
    if (num_rows < 0 || vocab < 1 || next_n < 1 || num_rows % next_n != 0 || num_rows > INT32_MAX || vocab > INT32_MAX ||
        next_n > GBTOPK_MAX_NEXT_N)
        return 0;
    return kWsHeaderBytes + static_cast<size_t>(num_rows) * sizeof(RowStat);
}

int gbtopk_verify_drafts(const void *logits, int dtype, int64_t num_rows, int64_t vocab, int64_t row_stride,
                         const int32_t *tokens, const float *uniforms, const float *noise, int32_t next_n,
                         const int64_t *tree_mask, const float *temperature, const float *draft_probs,
                         int32_t *accepted, int32_t *path, int32_t *next_token, int64_t *accept_mask, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (dtype != GBTOPK_F32 && dtype != GBTOPK_BF16 && dtype != GBTOPK_F16) return GBTOPK_EINVAL;
    if (num_rows < 0 || vocab < 1 || next_n < 1 || num_rows % next_n != 0) return GBTOPK_EINVAL;
    if (num_rows > 1 && row_stride < vocab) return GBTOPK_EINVAL;
    if (draft_probs && tree_mask) return GBTOPK_EINVAL;
    const size_t need = gbtopk_verify_workspace_bytes(num_rows, vocab, next_n);
    if (need == 0) return GBTOPK_EUNSUPPORTED;
    if (num_rows == 0) return GBTOPK_OK;
    if (!logits || !tokens || !uniforms || !noise || !accepted || !path || !next_token || !accept_mask)
        return GBTOPK_EINVAL;
    if (!aligned_to(logits, dtype == GBTOPK_F32 ? 4 : 2) || !aligned_to(noise, 4) || !aligned_to(draft_probs, 4) ||
        !aligned_to(accepted, 4) || !aligned_to(path, 4) || !aligned_to(next_token, 4) || !aligned_to(accept_mask, 8))
        return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < need) return GBTOPK_EWORKSPACE;
    VerifyParams p{logits, num_rows, vocab, row_stride, tokens, uniforms, noise, next_n, tree_mask, temperature,
                   draft_probs, accepted, path, next_token, accept_mask, static_cast<uint8_t *>(workspace)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GBTOPK_F32    ? launch_verify<GBTOPK_F32>(p, s)
                          : dtype == GBTOPK_BF16 ? launch_verify<GBTOPK_BF16>(p, s)
                                                 : launch_verify<GBTOPK_F16>(p, s);
    return e == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}

}  // extern "C"
