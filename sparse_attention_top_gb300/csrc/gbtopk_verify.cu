// Verification of drafted tokens against the target's distributions
// (gbtopk_verify_drafts).
#include <cooperative_groups.h>

#include <cfloat>

#include "gbtopk_decode.cuh"
#include "gbtopk_mma.cuh"

namespace cg = cooperative_groups;

namespace gbtopk {
namespace {

// verify_path_kernel: a cluster of kCluster blocks for each request, every
// block an equal part of the vocabulary.  A step of the walk reads the current
// node's row of logits once (each block its part: a running maximum and sum of
// exponentials per thread, joined over the cluster through distributed shared
// memory), decides its children in order, and goes on from the accepted one;
// the last node's row is then drawn from.  Rows that the path does not reach
// are not read.  For small calls (kLazyBytes) verify_stat_kernel reads all rows
// first, blocks of (row, piece of the vocabulary), and the path kernel only
// joins the pieces.
//
// Measured on one GB300, 64 requests x 16 nodes over 131073 bf16 words.  Greedy,
// nothing accepted: 9.7 us (one step).  Sampled: 32 us, since the draw reads the
// 34 MB of noise and the last row again, in eight rounds of loads a thread; each
// further step adds 5.5 to 6.5 us (15 accepted: 117), and each child refused
// before the draw 2.4 us (15 of them: 69), because every word that leads its
// thread's race is compared with all of them.  Trees of 16 with a third of a
// draft accepted a request: 42 to 47 us, most of it the draw.  One request
// x 4 nodes over 32000 fp32 words with draft probabilities: 8 us.
constexpr int kThreads = 256;
constexpr int kCluster = 8;
constexpr int kMaxPieces = 32;
// A piece: 64 KB of a row, fewer for few rows (see piece_of).
constexpr int kPieceBytes = 65536;
// Bytes of one row of logits of every request, above which the walk reads rows
// as it reaches them.  How far walks go is not known here, and neither order
// is the faster one for all; as (nothing, a quarter, all accepted), walking
// against reading all rows first, us, bf16:
//     64 requests x 16 nodes x 131073 words (16.8 MB a row): 35, 59, 117 / 88
//     64 x  4 x 131073 (16.8 MB):                            35, 41, 51 / 53
//     32 x 16 x 131073 (8.4 MB):                             27, 50, 94 / 65
//     16 x 16 x 131073 (4.2 MB):                             23, 45, 91 / 47
//      8 x 16 x 131073 (2.1 MB):                             23, 36, 89 / 41
//     64 x  8 x  32000 (4.1 MB):                             11, 18, 36 / 25
//    128 x  8 x  32000 fp32 (16.4 MB):                       21, 37, 70 / 39
//      1 x  4 x  32000 fp32 (0.1 MB):                         7,  9, 13 / 8
// Above the bound a walk to the end costs 1.0 to 1.8 times the other order and
// a short one saves up to 60 %; below it a walk to the end costs up to 2.2 times.
constexpr int64_t kLazyBytes = 10 << 20;

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

// log2 e / temperature, neither 0 (its product with -infinity) nor infinite
// (with 0) at the ends of the temperature's range.
__device__ __forceinline__ float exponent_of(float t) { return fminf(fmaxf(kLog2e / t, FLT_MIN), FLT_MAX); }

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

struct StatScratch {
    RowStat warp[kThreads / 32];
};

// The parts' stats as one: the largest logit first, then every sum scaled to
// it, so that the exponentials do not wait for one another.
template <int N>
__device__ __forceinline__ RowStat join_all(const RowStat *part, bool greedy, float c) {
    RowStat st = part[0];
    if (greedy) {
#pragma unroll
        for (int k = 1; k < N; ++k) better(st.top, st.first, part[k].top, part[k].first);
        return st;
    }
#pragma unroll
    for (int k = 1; k < N; ++k) st.top = fmaxf(st.top, part[k].top);
    const float base = st.top == -INFINITY ? 0.f : st.top;
    st.sum = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) st.sum += part[k].sum * exp2f((part[k].top - base) * c);
    return st;
}

// The stat of logits [e0, e1) of a row, by the block (every thread has it).
template <int DT, int UNROLL>
__device__ RowStat block_stat(const uint8_t *row, int64_t e0, int64_t e1, bool greedy, float c, StatScratch &sh) {
    constexpr int kBytes = DT == GBTOPK_F32 ? 4 : 2, kVec = 16 / kBytes, kUnroll = UNROLL;
    const int32_t n = static_cast<int32_t>(e1 - e0), tid = static_cast<int32_t>(threadIdx.x);
    const uint8_t *base = row + e0 * kBytes;
    // whole 16-byte vectors from `skip` logits on
    int32_t skip = static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(base) & 15)) & 15) / kBytes;
    if (skip > n) skip = n;
    const int32_t vecs = (n - skip) / kVec;
    const uint4 *body = reinterpret_cast<const uint4 *>(base + skip * kBytes);
    float top = -INFINITY, sum = 0.f;
    int32_t first = INT32_MAX;
    auto one = [&](int32_t e) {   // logit e of the part
        const float x = logit<DT>(base, e);
        if (greedy) better(top, first, x, static_cast<int32_t>(e0) + e);
        else if (x > -INFINITY) join(top, sum, x, 1.f, c);
    };
    if (tid < skip) one(tid);
    const int32_t tail = skip + vecs * kVec;
    if (tid < n - tail) one(tail + tid);
    for (int32_t v0 = 0; v0 < vecs; v0 += kThreads * kUnroll) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t v = v0 + u * kThreads + tid;
            if (v < vecs) raw[u] = fetch(body + v);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t v = v0 + u * kThreads + tid;
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
                sum *= exp2_fast((top - m) * c);
                top = m;
            }
            const float base_x = top == -INFINITY ? 0.f : top;
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) part += exp2_fast((x[i] - base_x) * c);
            sum += part;
        }
    }
    if (greedy) {
        for (int o = 16; o; o >>= 1) better(top, first, __shfl_xor_sync(~0u, top, o), __shfl_xor_sync(~0u, first, o));
    } else {
        float most = top;
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
        sum *= exp2f((top - (most == -INFINITY ? 0.f : most)) * c);
        top = most;
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    }
    if ((tid & 31) == 0) sh.warp[tid >> 5] = RowStat{top, sum, first};
    __syncthreads();
    return join_all<kThreads / 32>(sh.warp, greedy, c);
}

// grid: pieces of row 0, of row 1, ...
template <int DT>
__global__ void __launch_bounds__(kThreads) verify_stat_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ StatScratch sh;
    pdl_wait();
    pdl_release();
    const int64_t r = blockIdx.x / p.pieces;
    const int32_t piece = static_cast<int32_t>(blockIdx.x % p.pieces);
    const float t = p.temperature ? fetch(p.temperature + r / p.next_n) : 1.f;
    const int64_t e0 = piece * p.piece, e1 = e0 + p.piece < p.vocab ? e0 + p.piece : p.vocab;
    const RowStat st = block_stat<DT, 4>(static_cast<const uint8_t *>(p.logits) + r * p.row_stride * (DT == GBTOPK_F32 ? 4 : 2), e0, e1,
                                      t <= 0.f, t <= 0.f ? 0.f : exponent_of(t), sh);
    if (threadIdx.x == 0) p.stats[r * p.pieces + piece] = st;
}

struct PathShared {
    RowStat part[2][kCluster];         // each block's part of a step's row
    RowStat stat[GBTOPK_MAX_NEXT_N];   // rows' stats (sum: its reciprocal)
    uint64_t children[GBTOPK_MAX_NEXT_N];
    int32_t token[GBTOPK_MAX_NEXT_N];
    float u[GBTOPK_MAX_NEXT_N], have[GBTOPK_MAX_NEXT_N], q[GBTOPK_MAX_NEXT_N];
    int32_t refused[GBTOPK_MAX_NEXT_N], path[GBTOPK_MAX_NEXT_N];
    int32_t n_refused, cur, count;
    uint64_t took;
    StatScratch scratch;
    float best[kThreads / 32];
    int32_t index[kThreads / 32];
    float all_best[kCluster];          // of the cluster's first block
    int32_t all_index[kCluster];
};

template <int DT, bool LAZY>
__global__ void __launch_bounds__(kThreads, 4) verify_path_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ PathShared sh;
    const int rank = static_cast<int>(blockIdx.x % kCluster), tid = static_cast<int>(threadIdx.x);
    const int64_t i = blockIdx.x / kCluster, r0 = i * p.next_n;
    cg::cluster_group cluster = cg::this_cluster();
    if (tid < GBTOPK_MAX_NEXT_N) sh.children[tid] = 0;
    pdl_wait();
    pdl_release();
    const float t = p.temperature ? fetch(p.temperature + i) : 1.f;
    const bool greedy = t <= 0.f;
    const float c = greedy ? 0.f : exponent_of(t);
    const int32_t part = static_cast<int32_t>((p.vocab + kCluster - 1) / kCluster);
    const int32_t v0 = rank * part < p.vocab ? rank * part : static_cast<int32_t>(p.vocab);
    const int32_t v1 = v0 + part < p.vocab ? v0 + part : static_cast<int32_t>(p.vocab);
    // of a logit under a stat whose sum is a reciprocal
    auto prob = [&](const RowStat &st, float x, int32_t v) -> float {
        if (st.top == -INFINITY) return 0.f;
        if (greedy) return v == st.first ? 1.f : 0.f;
        return exp2f((x - st.top) * c) * st.sum;
    };
    __syncthreads();
    int32_t parent = -1;
    if (tid < p.next_n && tid > 0) {
        parent = tid - 1;
        if (p.tree_mask) {
            const uint64_t above = static_cast<uint64_t>(fetch(p.tree_mask + r0 + tid)) & ((1ull << tid) - 1);
            parent = above ? 63 - __clzll(static_cast<long long>(above)) : -1;
        }
        sh.token[tid] = fetch(p.tokens + r0 + tid);
        sh.u[tid] = fetch(p.uniforms + r0 + tid);
        if (parent >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&sh.children[parent]), 1ull << tid);
    }
    if (!LAZY) {   // each row's pieces joined, eight lanes a row
        for (int n = tid >> 3; n < p.next_n; n += kThreads / 8) {
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
    }
    if (tid == 0) {
        sh.cur = sh.count = sh.n_refused = 0;
        sh.took = 1;
        sh.path[0] = 0;
    }
    cluster.sync();   // also: every block of the cluster runs before any other writes to it
    const int32_t x_tok = tid < p.next_n && parent >= 0 ? sh.token[tid] : -1;
    const bool known = x_tok >= 0 && x_tok < p.vocab;
    if (!LAZY) {
        if (parent >= 0) {
            sh.have[tid] = known ? prob(sh.stat[parent], logit<DT>(p.logits, (r0 + parent) * p.row_stride + x_tok), x_tok) : 0.f;
            sh.q[tid] = known && p.draft_probs ? fetch(p.draft_probs + (r0 + parent) * p.vocab + x_tok) : 1.f;
        }
        __syncthreads();
    }
    for (uint32_t step = 0;; ++step) {
        const int cur = sh.cur;
        if (LAZY) {
            // the node's row, and what it gives its children
            const uint8_t *row = static_cast<const uint8_t *>(p.logits) + (r0 + cur) * p.row_stride * (DT == GBTOPK_F32 ? 4 : 2);
            const bool child = parent == cur && known;
            const float x = child ? logit<DT>(row, x_tok) : 0.f;
            const float q = child && p.draft_probs ? fetch(p.draft_probs + (r0 + cur) * p.vocab + x_tok) : 1.f;
            const RowStat mine = block_stat<DT, 8>(row, v0, v1, greedy, c, sh.scratch);
            if (tid < kCluster) cluster.map_shared_rank(&sh, tid)->part[step & 1][rank] = mine;
            cluster.sync();
            RowStat st = join_all<kCluster>(sh.part[step & 1], greedy, c);
            st.sum = st.sum > 0.f ? 1.f / st.sum : 0.f;
            if (tid == 0) sh.stat[cur] = st;
            if (parent == cur) {
                sh.have[tid] = child ? prob(st, x, x_tok) : 0.f;
                sh.q[tid] = q;
            }
            __syncthreads();
        }
        if (tid == 0) {
            int at = cur, count = sh.count, n_ref;
            uint64_t took = sh.took;
            bool moved;
            do {
                moved = false;
                n_ref = 0;
                float mass = 1.f;
                for (uint64_t left = sh.children[at]; left; left &= left - 1) {
                    const int n = __ffsll(static_cast<long long>(left)) - 1;
                    float have = sh.have[n];
                    for (int k = 0; k < n_ref; ++k)
                        if (sh.refused[k] == sh.token[n]) have = 0.f;
                    if (sh.u[n] * (p.draft_probs ? sh.q[n] : mass) < have) {
                        at = n;
                        took |= 1ull << n;
                        sh.path[++count] = n;
                        moved = true;
                        break;
                    }
                    sh.refused[n_ref++] = sh.token[n];
                    mass -= have;
                }
            } while (moved && !LAZY);
            if (moved) n_ref = 0;
            sh.cur = at;
            sh.count = count;
            sh.n_refused = moved ? -1 : n_ref;
            sh.took = took;
        }
        __syncthreads();
        if (sh.n_refused >= 0) break;
    }
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
    const float *noise = p.noise + i * p.vocab, *q = p.draft_probs && n_ref ? p.draft_probs + row * p.vocab : nullptr;
    float best = 0.f;
    int32_t token = INT32_MAX;
    auto refused = [&](int32_t v) {
        for (int k = 0; k < n_ref; ++k)
            if (sh.refused[k] == v) return true;
        return false;
    };
    if (st.top == -INFINITY) {
    } else if (greedy) {   // all of p is at one word
        if (rank == 0 && tid == 0 && (q ? 1.f - fetch(q + st.first) > 0.f : !refused(st.first))) {
            best = 1.f;
            token = st.first;
        }
    } else {
        constexpr int kUnroll = 8;
        for (int32_t b0 = v0 + tid; b0 < v1; b0 += kThreads * kUnroll) {
            float x[kUnroll], e[kUnroll], d[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int32_t v = b0 + u * kThreads;
                x[u] = -INFINITY;
                e[u] = 1.f;
                d[u] = 0.f;
                if (v < v1) {
                    x[u] = logit<DT>(p.logits, row * p.row_stride + v);
                    e[u] = fetch(noise + v);
                    if (q) d[u] = fetch(q + v);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const float rest = exp2_fast((x[u] - st.top) * c) * st.sum - d[u];
                const float race = __fdividef(rest, e[u]);
                const int32_t v = b0 + u * kThreads;
                if (race > best && (q || !refused(v))) {   // a thread's words ascend: ties keep the lowest
                    best = race;
                    token = v;
                }
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
        for (int w = 1; w < kThreads / 32; ++w) better(best, token, sh.best[w], sh.index[w]);
        PathShared *home = cluster.map_shared_rank(&sh, 0);
        home->all_best[rank] = best;
        home->all_index[rank] = token;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
        for (int k = 0; k < kCluster; ++k) better(best, token, sh.all_best[k], sh.all_index[k]);
        p.next_token[i] = best > 0.f ? token : -1;
    }
}

int elem_bytes(int dtype) { return dtype == GBTOPK_F32 ? 4 : 2; }

// Logits of a piece: kPieceBytes of them, more where a row would have over
// kMaxPieces pieces, fewer where a call would have fewer blocks than SMs.
int64_t piece_of(int64_t num_rows, int64_t vocab, int es, int sms) {
    int64_t piece = kPieceBytes / es;
    while (piece * kMaxPieces < vocab) piece *= 2;
    while (piece > 4096 / es * 2 && num_rows * ((vocab + piece - 1) / piece) < sms && piece / 2 * kMaxPieces >= vocab) piece /= 2;
    return piece;
}

template <int DT>
cudaError_t launch_verify(const VerifyParams &p, cudaStream_t s) {
    const dim3 clusters(static_cast<unsigned>(p.num_rows / p.next_n * kCluster));
    if (p.num_rows / p.next_n * p.vocab * (DT == GBTOPK_F32 ? 4 : 2) > kLazyBytes)
        return launch_pdl(verify_path_kernel<DT, true>, clusters, kThreads, 0, s, kCluster, p);
    const cudaError_t e = launch_pdl(verify_stat_kernel<DT>, dim3(static_cast<unsigned>(p.num_rows * p.pieces)), kThreads, 0, s, 1, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(verify_path_kernel<DT, false>, clusters, kThreads, 0, s, kCluster, p);
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
        !aligned_to(accepted, 4) || !aligned_to(path, 4) || !aligned_to(next_token, 4) || !aligned_to(accept_mask, 8) ||
        !aligned_to(tokens, 4) || !aligned_to(uniforms, 4) || !aligned_to(tree_mask, 8) || !aligned_to(temperature, 4))
        return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < need) return GBTOPK_EWORKSPACE;
    VerifyParams p{logits, num_rows, vocab, row_stride, tokens, uniforms, noise, next_n, tree_mask, temperature,
                   draft_probs, accepted, path, next_token, accept_mask,
                   reinterpret_cast<RowStat *>(static_cast<uint8_t *>(workspace) + kWsHeaderBytes), 0, 0};
    const int sms = device_sms();
    if (sms == 0) return GBTOPK_ECUDA;
    p.piece = piece_of(num_rows, vocab, elem_bytes(dtype), sms);
    p.pieces = static_cast<int32_t>((vocab + p.piece - 1) / p.piece);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == GBTOPK_F32    ? launch_verify<GBTOPK_F32>(p, s)
                          : dtype == GBTOPK_BF16 ? launch_verify<GBTOPK_BF16>(p, s)
                                                 : launch_verify<GBTOPK_F16>(p, s);
    return e == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}

}  // extern "C"
