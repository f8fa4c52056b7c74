// Verification of drafted tokens against the target's distributions
// (gbtopk_verify_drafts).
#include <cooperative_groups.h>

#include "gbtopk_decode.cuh"
#include "gbtopk_mma.cuh"

namespace cg = cooperative_groups;

namespace gbtopk {
namespace {

// Two kernels.  verify_stat_kernel reads every row of logits once: blocks of
// (row, piece of the vocabulary) leave the piece's largest logit and its sum
// of exponentials (a running pair per thread, rescaled when the maximum
// rises), or for greedy requests the largest logit's lowest index.
// verify_walk_kernel runs a cluster of kWalkCluster blocks for each request:
// every block joins the pieces' pairs, looks up the probability that each
// node's parent gives it (one thread a node), walks the tree in shared memory,
// then draws over its part of the vocabulary; the cluster's first block takes
// the best of the parts through distributed shared memory.
constexpr int kStatThreads = 256;
constexpr int kWalkThreads = 512;
constexpr int kWalkCluster = 8;
constexpr int kMaxPieces = 32;
// A piece: 32 KB of a row, so that a block has 16 KB or more in flight and
// the sum of a row's pieces stays short (131073 bf16 logits: 9 pieces).
constexpr int kPieceBytes = 32768;

// Of a row, or a piece of one: the largest logit, its lowest index (greedy
// requests) and the sum of exp((x - top) / temperature).
struct RowStat {
    float top, sum;
    int32_t first;
};

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
    RowStat *stats;      // [num_rows][pieces]
    int32_t pieces;
    int64_t piece;       // logits of a piece
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

// Adds a piece's pair (top, sum) to a running one, exponents scaled by c
// (log2 e / temperature).
__device__ __forceinline__ void join(float &top, float &sum, float t2, float s2, float c) {
    const float t = fmaxf(top, t2);
    const float base = t == -INFINITY ? 0.f : t;
    sum = sum * exp2f((top - base) * c) + s2 * exp2f((t2 - base) * c);
    top = t;
}

template <int DT>
__device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == GBTOPK_F32) {
            x[i] = __uint_as_float(w[i]);
        } else {
            const float2 f = Half2<DT == GBTOPK_BF16>::up(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// grid: pieces of row 0, of row 1, ...
template <int DT>
__global__ void __launch_bounds__(kStatThreads) verify_stat_kernel(const __grid_constant__ VerifyParams p) {
    constexpr int kBytes = DT == GBTOPK_F32 ? 4 : 2, kVec = 16 / kBytes, kUnroll = 4;
    __shared__ float s_top[kStatThreads / 32], s_sum[kStatThreads / 32];
    __shared__ int32_t s_first[kStatThreads / 32];
    pdl_wait();
    pdl_release();
    const int64_t r = blockIdx.x / p.pieces;
    const int32_t piece = static_cast<int32_t>(blockIdx.x % p.pieces);
    const float t = p.temperature ? fetch(p.temperature + r / p.next_n) : 1.f;
    const bool greedy = t <= 0.f;
    const float c = greedy ? 0.f : kLog2e / t;
    const uint8_t *row = static_cast<const uint8_t *>(p.logits) + r * p.row_stride * kBytes;
    // the piece's logits [e0, e1); whole 16-byte vectors from `skip` logits on
    const int64_t e0 = piece * p.piece;
    const int64_t e1 = e0 + p.piece < p.vocab ? e0 + p.piece : p.vocab;
    const int32_t n = static_cast<int32_t>(e1 - e0);
    const uint8_t *base = row + e0 * kBytes;
    int32_t skip = static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / kBytes;
    if (skip > n) skip = n;
    const int32_t vecs = (n - skip) / kVec;
    const uint4 *body = reinterpret_cast<const uint4 *>(base + skip * kBytes);
    float top = -INFINITY, sum = 0.f;
    int32_t first = INT32_MAX;
    auto one = [&](int32_t e) {   // logit e of the piece
        const float x = logit<DT>(base, e);
        if (greedy) better(top, first, x, static_cast<int32_t>(e0) + e);
        else if (x > -INFINITY) join(top, sum, x, 1.f, c);
    };
    if (static_cast<int32_t>(threadIdx.x) < skip) one(threadIdx.x);
    const int32_t tail = skip + vecs * kVec;
    if (static_cast<int32_t>(threadIdx.x) < n - tail) one(tail + threadIdx.x);
    for (int32_t v0 = 0; v0 < vecs; v0 += kStatThreads * kUnroll) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t v = v0 + u * kStatThreads + static_cast<int32_t>(threadIdx.x);
            if (v < vecs) raw[u] = fetch(body + v);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t v = v0 + u * kStatThreads + static_cast<int32_t>(threadIdx.x);
            if (v >= vecs) break;
            float x[kVec];
            unpack<DT>(raw[u], x);
            float m = x[0];
#pragma unroll
            for (int i = 1; i < kVec; ++i) m = fmaxf(m, x[i]);
            if (greedy) {
                if (m >= top) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        better(top, first, x[i], static_cast<int32_t>(e0) + skip + v * kVec + i);
                }
                continue;
            }
            if (m > top) {
                sum *= exp2f((top - m) * c);
                top = m;
            }
            const float base = top == -INFINITY ? 0.f : top;
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) part += exp2_fast((x[i] - base) * c);
            sum += part;
        }
    }
    for (int o = 16; o; o >>= 1) {
        const float t2 = __shfl_xor_sync(~0u, top, o), s2 = __shfl_xor_sync(~0u, sum, o);
        const int32_t f2 = __shfl_xor_sync(~0u, first, o);
        if (greedy) better(top, first, t2, f2);
        else join(top, sum, t2, s2, c);
    }
    if ((threadIdx.x & 31) == 0) {
        s_top[threadIdx.x >> 5] = top;
        s_sum[threadIdx.x >> 5] = sum;
        s_first[threadIdx.x >> 5] = first;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kStatThreads / 32; ++w) {
            if (greedy) better(top, first, s_top[w], s_first[w]);
            else join(top, sum, s_top[w], s_sum[w], c);
        }
        p.stats[r * p.pieces + piece] = RowStat{top, sum, first};
    }
}

struct WalkShared {
    RowStat stat[GBTOPK_MAX_NEXT_N];
    int32_t parent[GBTOPK_MAX_NEXT_N], token[GBTOPK_MAX_NEXT_N];
    float u[GBTOPK_MAX_NEXT_N], have[GBTOPK_MAX_NEXT_N], q[GBTOPK_MAX_NEXT_N];
    int32_t refused[GBTOPK_MAX_NEXT_N], path[GBTOPK_MAX_NEXT_N];
    int32_t n_refused, cur, count;
    uint64_t took;
    float best[kWalkThreads / 32];
    int32_t index[kWalkThreads / 32];
    float all_best[kWalkCluster];      // of the cluster's first block
    int32_t all_index[kWalkCluster];
};

// A cluster of kWalkCluster blocks for each request.
template <int DT>
__global__ void __launch_bounds__(kWalkThreads) verify_walk_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ WalkShared sh;
    const int rank = static_cast<int>(blockIdx.x % kWalkCluster), tid = static_cast<int>(threadIdx.x);
    const int64_t i = blockIdx.x / kWalkCluster, r0 = i * p.next_n;
    pdl_wait();
    pdl_release();
    const float t = p.temperature ? fetch(p.temperature + i) : 1.f;
    const bool greedy = t <= 0.f;
    const float c = greedy ? 0.f : kLog2e / t;
    // p of token v under row n of the request, 1 / sum and top given
    auto prob = [&](int64_t row, float top, float inv, int32_t first, int64_t v) -> float {
        if (top == -INFINITY) return 0.f;
        if (greedy) return v == first ? 1.f : 0.f;
        return exp2f((logit<DT>(p.logits, row * p.row_stride + v) - top) * c) * inv;
    };
    cg::cluster_group cluster = cg::this_cluster();
    // each row's pieces joined, eight lanes a row
    for (int n = tid >> 3; n < p.next_n; n += kWalkThreads / 8) {
        float top = -INFINITY, sum = 0.f;
        int32_t first = INT32_MAX;
        for (int k = tid & 7; k < p.pieces; k += 8) {
            const RowStat st = p.stats[(r0 + n) * p.pieces + k];
            if (greedy) better(top, first, st.top, st.first);
            else join(top, sum, st.top, st.sum, c);
        }
        const uint32_t lanes = 0xffu << (tid & 24);
        for (int o = 4; o; o >>= 1) {
            const float t2 = __shfl_xor_sync(lanes, top, o), s2 = __shfl_xor_sync(lanes, sum, o);
            const int32_t f2 = __shfl_xor_sync(lanes, first, o);
            if (greedy) better(top, first, t2, f2);
            else join(top, sum, t2, s2, c);
        }
        if ((tid & 7) == 0) sh.stat[n] = RowStat{top, sum > 0.f ? 1.f / sum : 0.f, first};
    }
    cluster.sync();   // also: every block of the cluster runs before any other writes to it
    if (tid < p.next_n && tid > 0) {
        int32_t parent = tid - 1;
        if (p.tree_mask) {
            const uint64_t above = static_cast<uint64_t>(fetch(p.tree_mask + r0 + tid)) & ((1ull << tid) - 1);
            parent = above ? 63 - __clzll(static_cast<long long>(above)) : -1;
        }
        const int32_t x = fetch(p.tokens + r0 + tid);
        const bool known = parent >= 0 && x >= 0 && x < p.vocab;
        sh.parent[tid] = parent;
        sh.token[tid] = x;
        sh.u[tid] = fetch(p.uniforms + r0 + tid);
        const RowStat st = sh.stat[parent >= 0 ? parent : 0];
        sh.have[tid] = known ? prob(r0 + parent, st.top, st.sum, st.first, x) : 0.f;
        sh.q[tid] = known && p.draft_probs ? fetch(p.draft_probs + (r0 + parent) * p.vocab + x) : 1.f;
    }
    __syncthreads();
    if (tid == 0) {
        int cur = 0, count = 0, n_ref = 0;
        uint64_t took = 1;
        float mass = 1.f;
        sh.path[0] = 0;
        for (int n = 1; n < p.next_n; ++n) {
            if (sh.parent[n] != cur) continue;
            const int32_t x = sh.token[n];
            float have = sh.have[n];
            for (int k = 0; k < n_ref; ++k)
                if (sh.refused[k] == x) have = 0.f;
            const float q = p.draft_probs ? sh.q[n] : mass;
            if (sh.u[n] * q < have) {
                cur = n;
                took |= 1ull << n;
                sh.path[++count] = n;
                n_ref = 0;
                mass = 1.f;
            } else {
                sh.refused[n_ref++] = x;
                mass -= have;
            }
        }
        sh.cur = cur;
        sh.count = count;
        sh.n_refused = n_ref;
        sh.took = took;
    }
    __syncthreads();
    const int cur = sh.cur, n_ref = sh.n_refused;
    if (rank == 0) {
        if (tid < p.next_n) p.path[r0 + tid] = tid <= sh.count ? sh.path[tid] : -1;
        if (tid == 0) {
            p.accepted[i] = sh.count;
            p.accept_mask[i] = static_cast<int64_t>(sh.took);
        }
    }
    // the draw: this block's part of the vocabulary
    const RowStat st = sh.stat[cur];
    const int64_t row = r0 + cur;
    const int64_t part = (p.vocab + kWalkCluster - 1) / kWalkCluster;
    const int64_t v1 = (rank + 1) * part < p.vocab ? (rank + 1) * part : p.vocab;
    const float *noise = p.noise + i * p.vocab, *q = p.draft_probs && n_ref ? p.draft_probs + row * p.vocab : nullptr;
    float best = 0.f;
    int32_t token = INT32_MAX;
    auto consider = [&](float rest, float e, int64_t v) {
        const float race = rest / e;
        if (rest > 0.f && (race > best || (race == best && v < token))) {
            if (!q)
                for (int k = 0; k < n_ref; ++k)
                    if (sh.refused[k] == v) return;
            best = race;
            token = static_cast<int32_t>(v);
        }
    };
    if (st.top > -INFINITY) {
        constexpr int kUnroll = 8;
        for (int64_t v0 = rank * part + tid; v0 < v1; v0 += kWalkThreads * kUnroll) {
            float x[kUnroll], e[kUnroll], d[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t v = v0 + u * kWalkThreads;
                if (v < v1) {
                    x[u] = logit<DT>(p.logits, row * p.row_stride + v);
                    e[u] = fetch(noise + v);
                    d[u] = q ? fetch(q + v) : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t v = v0 + u * kWalkThreads;
                if (v >= v1) break;
                const float pr = greedy ? (v == st.first ? 1.f : 0.f) : exp2f((x[u] - st.top) * c) * st.sum;
                consider(pr - d[u], e[u], v);
            }
        }
    }
    for (int o = 16; o; o >>= 1) better(best, token, __shfl_xor_sync(~0u, best, o), __shfl_xor_sync(~0u, token, o));
    if ((tid & 31) == 0) {
        sh.best[tid >> 5] = best;
        sh.index[tid >> 5] = token;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWalkThreads / 32; ++w) better(best, token, sh.best[w], sh.index[w]);
        WalkShared *home = cluster.map_shared_rank(&sh, 0);
        home->all_best[rank] = best;
        home->all_index[rank] = token;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
        for (int k = 0; k < kWalkCluster; ++k) better(best, token, sh.all_best[k], sh.all_index[k]);
        p.next_token[i] = best > 0.f ? token : -1;
    }
}

int elem_bytes(int dtype) { return dtype == GBTOPK_F32 ? 4 : 2; }

// Logits of a piece: kPieceBytes of them, more where a row would have over
// kMaxPieces pieces, fewer where a call would have fewer blocks than SMs.
int64_t piece_of(int64_t num_rows, int64_t vocab, int es) {
    int64_t piece = kPieceBytes / es;
    while (piece * kMaxPieces < vocab) piece *= 2;
    while (piece > 4096 / es * 2 && num_rows * ((vocab + piece - 1) / piece) < 152 && piece / 2 * kMaxPieces >= vocab) piece /= 2;
    return piece;
}

template <int DT>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t s) {
    const cudaError_t e = launch_pdl(verify_stat_kernel<DT>, dim3(static_cast<unsigned>(p.num_rows * p.pieces)),
                                     kStatThreads, 0, s, 1, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(verify_walk_kernel<DT>, dim3(static_cast<unsigned>(p.num_rows / p.next_n * kWalkCluster)), kWalkThreads, 0, s,
                      kWalkCluster, p);
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" {

size_t gbtopk_verify_workspace_bytes(int64_t num_rows, int64_t vocab, int32_t next_n) {
    if (num_rows < 0 || vocab < 1 || next_n < 1 || num_rows % next_n != 0 || num_rows > INT32_MAX / kMaxPieces || vocab > INT32_MAX / 2 ||
        next_n > GBTOPK_MAX_NEXT_N)
        return 0;
    return kWsHeaderBytes + static_cast<size_t>(num_rows) * kMaxPieces * sizeof(RowStat);
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
                   draft_probs, accepted, path, next_token, accept_mask,
                   reinterpret_cast<RowStat *>(static_cast<uint8_t *>(workspace) + kWsHeaderBytes), 0, 0};
    p.piece = piece_of(num_rows, vocab, elem_bytes(dtype));
    p.pieces = static_cast<int32_t>((vocab + p.piece - 1) / p.piece);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GBTOPK_F32    ? launch_verify<GBTOPK_F32>(p, s)
                          : dtype == GBTOPK_BF16 ? launch_verify<GBTOPK_BF16>(p, s)
                                                 : launch_verify<GBTOPK_F16>(p, s);
    return e == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}

}  // extern "C"
