// The weight each cached position accumulates (gbtopk_cache_weights):
// w[p] += sum over rows of 2^(c s(row, p) - lse2(row)), c = |scale| log2 e.
//
// The scores are computed transposed, S^T = K Q^T (tensor core): a tile of
// 128 cached positions is the rows of the matrix, so one thread owns one
// position and sums its rows alone, in a fixed order and without atomics;
// the softmax's sum is known (lse), so one pass over the keys does it and
// the values are not read.  Only accepted rows enter the product.
//
// Work is split as in the attention kernel: block c takes the c-th equal
// share of the list of (request, weight head, position tile).  Within a
// share, up to kSpan tiles of one (request, weight head) at a time: for each
// kv head and each group of up to NQ rows (a phase, one queries' buffer) its
// tiles one after the other (a job each), the even and odd jobs summed by two
// warpgroups, each into its own sums in shared memory.
//
// Bound by the keys' bytes.  Measured on one GB300: 32 requests x 8 drafts over
// 2048..16384 positions, 8 heads of 128, the accepted rows only, 106 us = 5.9
// TB/s; one request of 2049 positions, one weight for all heads, 18 us (17
// blocks, each one tile's eight heads in turn: the sum over heads stays in one
// block, in a fixed order).
#include <cfloat>
#include <cmath>

#include "gbtopk_paged.cuh"

namespace gbtopk {
namespace {

constexpr int kSpan = 16;        // tiles whose sums are held at a time
constexpr int kMaskRing = 8;     // tiles whose validity bits are kept
constexpr int KT = 128;          // positions a tile

struct WeightParams {
    AttnParams a;                // request_units: weight heads
    const int64_t *accept_mask;
    const float *lse;
    float *weights;
    int32_t weight_heads;
    int64_t width;
};

// NQ: query rows of a phase; few rows leave room for the queries of eight
// phases, so that a request's heads (one weight for all) follow one another
// without a wait for each head's queries.
template <int DP, int NQ>
struct Shape {
    static constexpr int kQBufs = NQ == 32 ? (DP == 256 ? 4 : 8) : 2;
    static constexpr int kThreads = 512;                    // 2 summing warpgroups, products, copies
    static constexpr int kQBytes = NQ * DP * 2;             // of a phase
    static constexpr int kStageBytes = KT * DP * 2;
    static constexpr int kSums = 2 * kSpan * KT * 4;
    static constexpr int kFixed = 8192;                     // barriers, slots and masks, lse, trees
    static constexpr int kFit = (static_cast<int>(kMaxSmemBytes) - 1024 - kFixed - kSums - kQBufs * kQBytes) / kStageBytes;
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static constexpr size_t kSmem = 1024 + kFixed + kSums + kQBufs * kQBytes + static_cast<size_t>(kStages) * kStageBytes;
    static_assert(kStages >= 2 && kStages <= kMaskRing && NQ * kQBufs <= 256, "ring");
};

struct Shared {
    uint64_t full[6], empty[6];     // ring stages, one key tile each
    uint64_t slots_full[kMaskRing], slots_empty[kMaskRing];   // slots and validity bits of a job's tile
    uint64_t q_full[8], q_empty[8]; // phase buffers
    uint64_t s_full[2], s_empty[2];
    uint64_t drain;
    uint32_t mask[kMaskRing][4];
    int32_t slots[kMaskRing][KT];   // cache slot of each position, -1 where there is none
    alignas(16) float lse2[256];    // base-2 lse of the phases' rows; +inf: adds nothing
    uint64_t tree[GBTOPK_MAX_NEXT_N];
    alignas(16) uint32_t without[8][4];         // a phase has rows without an lse, by copying warp
    ScanScratch scan;
    uint32_t tmem;
    uint32_t abort;
};
static_assert(sizeof(Shared) <= 8192, "shared block");
static_assert(offsetof(Shared, lse2) % 16 == 0 && offsetof(Shared, without) % 16 == 0, "vector loads");

// One span of a share: tiles t0 .. t1 - 1 of a (request, weight head), and
// its phases.
struct Span16 {
    int32_t b, w, t0, t1, n, ctx;
    uint64_t took;     // accepted tokens
    int32_t rows;      // accepted rows of a kv head
    int32_t groups;    // row groups of a kv head
    int32_t phases;
};

// Walks the spans of the block's share; every role sees the same sequence.
template <int NQ>
struct Spans {
    const WeightParams &p;
    Walk<KT> walk;
    int32_t t;
    __device__ Spans(const WeightParams &p, const Share &s) : p(p), walk(p.a, s), t(walk.more() ? walk.u.t0 : 0) {}
    __device__ bool next(Span16 *s) {
        while (walk.more()) {
            if (t == walk.u.t1) {
                walk.next();
                if (!walk.more()) return false;
                t = walk.u.t0;
            }
            s->b = walk.u.b;
            s->w = walk.u.hm;
            s->n = walk.u.span.n;
            s->ctx = walk.u.span.ctx;
            s->t0 = t;
            s->t1 = walk.u.t1 - t > kSpan ? t + kSpan : walk.u.t1;
            t = s->t1;
            const uint64_t all = ~0ull >> (64 - p.a.next_n);
            s->took = p.accept_mask ? static_cast<uint64_t>(fetch(p.accept_mask + s->b)) & all : all;
            s->rows = __popcll(s->took) * p.a.group;
            s->groups = (s->rows + NQ - 1) / NQ;
            s->phases = s->groups * (p.a.kv_heads / p.weight_heads);
            if (s->phases > 0 && s->n > 0 && static_cast<int64_t>(s->t0) * KT < p.width) return true;
        }
        return false;
    }
};

// The k-th accepted token.
__device__ __forceinline__ int nth_bit(uint64_t bits, int k) {
    for (; k > 0; --k) bits &= bits - 1;
    return __ffsll(static_cast<long long>(bits)) - 1;
}

// Barrier of the two summing warpgroups; true for all when `v` is for one.
__device__ __forceinline__ bool sums_barrier_or(bool v) {
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(v))
        : "memory");
    return any != 0;
}

template <bool BF16, int DP, int NQ>
__global__ void __launch_bounds__(Shape<DP, NQ>::kThreads, 1) weights_kernel(const __grid_constant__ WeightParams p) {
    using Sh = Shape<DP, NQ>;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t q_smem = smem_addr(smem), ring = q_smem + Sh::kQBufs * Sh::kQBytes;
    float *sums = reinterpret_cast<float *>(smem + Sh::kQBufs * Sh::kQBytes + Sh::kStages * Sh::kStageBytes);   // [2][kSpan][KT]
    Shared &sh = *reinterpret_cast<Shared *>(reinterpret_cast<uint8_t *>(sums) + Sh::kSums);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kMmaWarp = 8;
    const AttnParams &a = p.a;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            bar_init(&sh.full[i], 128);
            bar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kMaskRing; ++i) {
            bar_init(&sh.slots_full[i], 1);
            bar_init(&sh.slots_empty[i], 4);
        }
        for (int i = 0; i < Sh::kQBufs; ++i) {
            bar_init(&sh.q_full[i], 128 + 4);   // copies, and the lse values of each copying warp
            bar_init(&sh.q_empty[i], 1 + 8);    // products, and the summing warps
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.s_full[i], 1);
            bar_init(&sh.s_empty[i], 4);
        }
        bar_init(&sh.drain, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&sh.tmem, 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_release();
    const Share share = block_share<KT, Sh::kThreads>(a, &sh.scan);
    const Waits abort{&sh.abort, a.wait_cycles};
    const uint32_t tmem = sh.tmem;
    Spans<NQ> spans(p, share);
    const int32_t per = a.kv_heads / p.weight_heads;   // kv heads of a weight head
    const int32_t chunks = (a.dim + 15) / 16 * 2, loaded = a.dim / 8;
    Span16 s;
    bool ok = true;

    if (warp >= kMmaWarp + 4) {
        // ------------------------------------------------ copies
        const int w = warp - kMmaWarp - 4;
        uint32_t phase = 0, job = 0;
        while (ok && spans.next(&s)) {
            for (int32_t ph = 0; ph < s.phases && ok; ++ph, ++phase) {
                const int32_t h = s.w * per + ph / s.groups, r0 = (ph % s.groups) * NQ;
                const int32_t rows = s.rows - r0 < NQ ? s.rows - r0 : NQ, padded = (rows + 15) / 16 * 16;
                const uint32_t qb = phase % Sh::kQBufs;
                if (phase >= Sh::kQBufs) ok = __all_sync(~0u, bar_wait(&sh.q_empty[qb], (phase / Sh::kQBufs - 1) & 1, abort));
                if (!ok) break;
                for (int x = w * 32 + lane; x < padded * chunks; x += 128) {
                    const int32_t r = x / chunks, c = x - r * chunks;
                    const uint8_t *src = static_cast<const uint8_t *>(a.q);
                    const bool have = r < rows && c < loaded;
                    if (have) {
                        const int32_t k = (r0 + r) / a.group, gq = r0 + r - k * a.group;
                        src += 2 * ((static_cast<int64_t>(s.b) * a.next_n + nth_bit(s.took, k)) * a.q_row + (h * a.group + gq) * a.q_head) + c * 16;
                    }
                    copy16(q_smem + qb * Sh::kQBytes + tile_offset(NQ, r, c), src, have ? 16u : 0u);
                }
                bar_arrive_copies(&sh.q_full[qb]);
                bool none = false;
                for (int r = w * 32 + lane; r < padded; r += 128) {
                    float v = INFINITY;
                    if (r < rows) {
                        const int32_t k = (r0 + r) / a.group, gq = r0 + r - k * a.group;
                        const float lse = fetch(p.lse + (static_cast<int64_t>(s.b) * a.next_n + nth_bit(s.took, k)) * a.q_heads + h * a.group + gq);
                        v = lse == -INFINITY ? INFINITY : lse * kLog2e;
                        none |= lse == -INFINITY;
                    }
                    sh.lse2[qb * NQ + r] = v;
                }
                none = __any_sync(~0u, none);
                if (lane == 0) {
                    sh.without[qb][w] = none;
                    bar_arrive(&sh.q_full[qb]);
                }
                for (int32_t t = s.t0; t < s.t1; ++t, ++job) {
                    ok = __all_sync(~0u, bar_wait(&sh.slots_full[job % kMaskRing], (job / kMaskRing) & 1, abort));
                    if (!ok) break;
                    const int32_t slot = reinterpret_cast<volatile int32_t *>(sh.slots[job % kMaskRing])[w * 32 + lane];
                    const uint32_t stage = job % Sh::kStages;
                    if (job >= Sh::kStages) ok = __all_sync(~0u, bar_wait(&sh.empty[stage], (job / Sh::kStages - 1) & 1, abort));
                    if (!ok) break;
                    copy_tile<DP, KT>(ring + stage * Sh::kStageBytes, static_cast<const uint8_t *>(a.k) + 2 * h * a.k_head, a.k_slot * 2,
                                      slot, chunks, loaded, w, lane);
                    bar_arrive_copies(&sh.full[stage]);
                }
            }
        }
        copies_land();
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------ matrix products
        if (warp == kMmaWarp) {   // all lanes alike, see elect_lane
            const bool lead = elect_lane();
            uint32_t phase = 0, job = 0;
            while (ok && __any_sync(~0u, spans.next(&s))) {
                // broadcasts: values known to be warp-uniform
                s.phases = __shfl_sync(~0u, s.phases, 0);
                s.groups = __shfl_sync(~0u, s.groups, 0);
                s.rows = __shfl_sync(~0u, s.rows, 0);
                s.t0 = __shfl_sync(~0u, s.t0, 0);
                s.t1 = __shfl_sync(~0u, s.t1, 0);
                for (int32_t ph = 0; ph < s.phases && ok; ++ph, ++phase) {
                    const int32_t r0 = (ph % s.groups) * NQ;
                    const int32_t rows = s.rows - r0 < NQ ? s.rows - r0 : NQ, padded = (rows + 15) / 16 * 16;
                    const uint32_t desc = mma_desc(BF16, 128, static_cast<uint32_t>(padded), false, a.negative != 0);
                    const uint32_t qb = phase % Sh::kQBufs, qa = q_smem + qb * Sh::kQBytes;
                    ok = __all_sync(~0u, bar_wait(&sh.q_full[qb], (phase / Sh::kQBufs) & 1, abort));
                    for (int32_t t = s.t0; t < s.t1 && ok; ++t, ++job) {
                        const uint32_t stage = job % Sh::kStages, sb = job & 1;
                        ok = __all_sync(~0u, bar_wait(&sh.full[stage], (job / Sh::kStages) & 1, abort));
                        if (ok && job >= 2) ok = __all_sync(~0u, bar_wait(&sh.s_empty[sb], (job / 2 - 1) & 1, abort));
                        if (!ok) break;
                        fence_async_reads();
                        tc_fence_after();
                        const uint32_t ka = ring + stage * Sh::kStageBytes;
                        if (lead) {
#pragma unroll
                            for (int kk = 0; kk < DP / 16; ++kk)
                                if (kk < chunks / 2)
                                    mma_ss(tmem + sb * 128, smem_desc(ka + (kk >> 2) * (KT * 128) + (kk & 3) * 32, 16, 1024),
                                           smem_desc(qa + (kk >> 2) * (NQ * 128) + (kk & 3) * 32, 16, 1024), desc, kk > 0);
                            tc_commit(&sh.s_full[sb]);
                            tc_commit(&sh.empty[stage]);
                        }
                        __syncwarp();
                    }
                    if (ok && lead) tc_commit(&sh.q_empty[qb]);
                    __syncwarp();
                }
            }
            if (lead) tc_commit(&sh.drain);
            __syncwarp();
            if (!bar_wait(&sh.drain, 0, abort)) {
                const long long t0 = clock64();
                while (!bar_try(&sh.drain, 0) && clock64() - t0 < kWaitCycles) {
                }
            }
        }
        else {
            // -------------------------------------------- slots of the tiles to come, three warps in turn
            const int turn = warp - kMmaWarp - 1;
            uint32_t job = 0;
            while (ok && spans.next(&s)) {
                uint64_t seen = ~0ull;   // drafted tokens that an accepted row sees
                if (a.tree_mask && (s.t1 - 1) * KT > s.ctx - KT) {   // (KT more could pass 31 bits)
                    seen = 0;
                    for (int j = lane; j < a.next_n; j += 32)
                        if ((s.took >> j) & 1) seen |= static_cast<uint64_t>(fetch(a.tree_mask + static_cast<int64_t>(s.b) * a.next_n + j));
                    seen = static_cast<uint64_t>(__reduce_or_sync(~0u, static_cast<uint32_t>(seen >> 32))) << 32 |
                           __reduce_or_sync(~0u, static_cast<uint32_t>(seen));
                }
                for (int32_t ph = 0; ph < s.phases && ok; ++ph)
                    for (int32_t t = s.t0; t < s.t1; ++t, ++job) {
                        if (job % 3 != static_cast<uint32_t>(turn)) continue;
                        const uint32_t r = job % kMaskRing;
                        Paging::Place at[KT / 32];
#pragma unroll
                        for (int k = 0; k < KT / 32; ++k) {
                            const int32_t pos = t * KT + k * 32 + lane;
                            at[k] = a.pages.place(s.b, pos, pos < s.n && pos < p.width && (pos < s.ctx || ((seen >> (pos - s.ctx)) & 1)));
                        }
                        if (job >= kMaskRing) ok = __all_sync(~0u, bar_wait(&sh.slots_empty[r], (job / kMaskRing - 1) & 1, abort));
                        if (!ok) break;
#pragma unroll
                        for (int k = 0; k < KT / 32; ++k) {
                            const int32_t slot = static_cast<int32_t>(a.pages.slot(at[k]));
                            const uint32_t valid = __ballot_sync(~0u, slot >= 0);
                            sh.slots[r][k * 32 + lane] = slot;
                            if (lane == 0) sh.mask[r][k] = valid;
                        }
                        __syncwarp();
                        if (lane == 0) bar_arrive(&sh.slots_full[r]);
                    }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ sums
        const int wg = warp >> 2, key = threadIdx.x & 127;
        const uint32_t t_s = tmem + (static_cast<uint32_t>(warp & 3) << 21) + wg * 128;
        float *mine = sums + wg * kSpan * KT + key;
        uint32_t phase = 0, job = 0;
        while (ok && spans.next(&s)) {
            for (int i = 0; i < s.t1 - s.t0; ++i) mine[i * KT] = 0.f;
            // the span's weights, loaded while its products run
            float *w = p.weights + (static_cast<int64_t>(s.b) * p.weight_heads + s.w) * p.width;
            constexpr int kHeld = kSpan * KT / 256;
            float held[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int64_t pos = static_cast<int64_t>(s.t0) * KT + i * 256 + threadIdx.x;
                if (i * 256 + static_cast<int>(threadIdx.x) < (s.t1 - s.t0) * KT && pos < s.n && pos < p.width) held[i] = w[pos];
            }
            // trees of the accepted tokens, where the span reaches the drafts
            const bool drafts = (s.t1 - 1) * KT > s.ctx - KT;
            if (drafts) {
                sums_barrier_or(false);
                const int k = threadIdx.x;
                if (k < __popcll(s.took)) {
                    const int t = nth_bit(s.took, k);
                    sh.tree[k] = a.tree_mask ? static_cast<uint64_t>(fetch(a.tree_mask + static_cast<int64_t>(s.b) * a.next_n + t))
                                             : ~0ull >> (63 - t);
                }
                sums_barrier_or(false);
            }
            for (int32_t ph = 0; ph < s.phases && ok; ++ph, ++phase) {
                const int32_t r0 = (ph % s.groups) * NQ;
                const int32_t rows = s.rows - r0 < NQ ? s.rows - r0 : NQ, padded = (rows + 15) / 16 * 16;
                const uint32_t qb = phase % Sh::kQBufs;
                const float *lse2 = sh.lse2 + qb * NQ;
                ok = __all_sync(~0u, bar_wait(&sh.q_full[qb], (phase / Sh::kQBufs) & 1, abort));
                const uint4 wo = *reinterpret_cast<const uint4 *>(sh.without[qb]);
                const bool without = (wo.x | wo.y | wo.z | wo.w) != 0;
                for (int32_t t = s.t0; t < s.t1 && ok; ++t, ++job) {
                    if ((job & 1) != static_cast<uint32_t>(wg)) continue;
                    ok = __all_sync(~0u, bar_wait(&sh.slots_full[job % kMaskRing], (job / kMaskRing) & 1, abort) &&
                                             bar_wait(&sh.s_full[wg], (job / 2) & 1, abort));
                    if (!ok) break;
                    tc_fence_after();
                    const bool valid = (reinterpret_cast<volatile uint32_t *>(sh.mask[job % kMaskRing])[warp & 3] >> lane) & 1;
                    const int32_t j = t * KT + key - s.ctx;   // the position's drafted token
                    float add = 0.f;
                    for (int c0 = 0; c0 < padded; c0 += 16) {
                        uint32_t x[16];
                        tmem_load16(t_s + c0, x);
                        float e[16];
#pragma unroll
                        for (int c = 0; c < 16; c += 4) *reinterpret_cast<float4 *>(e + c) = *reinterpret_cast<const float4 *>(lse2 + c0 + c);
                        tc_wait_ld();
                        if (t * KT > s.ctx - KT && j >= 0) {
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const int32_t k = (r0 + c0 + c) / a.group;
                                if (j > 63 || r0 + c0 + c >= s.rows || !((sh.tree[k] >> j) & 1)) {
                                    e[c] = INFINITY;
                                    x[c] = 0;   // whatever the key holds
                                }
                            }
                        }
                        // rows that add nothing, behind the last or without an lse:
                        // infinite keys would make their scores NaN
                        if (c0 + 16 > rows || without) {
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                if (e[c] == INFINITY) x[c] = 0;
                        }
                        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 16; ++c) part[c & 3] += exp2_fast(fmaf(__uint_as_float(x[c]), a.c, -e[c]));
                        add += (part[0] + part[1]) + (part[2] + part[3]);
                    }
                    if (valid) mine[(t - s.t0) * KT] += add;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&sh.s_empty[wg]);
                        bar_arrive(&sh.slots_empty[job % kMaskRing]);
                    }
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.q_empty[qb]);
            }
            // the two warpgroups' sums, in order; all leave together when one gave up
            ok = !sums_barrier_or(!ok);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int x = i * 256 + static_cast<int>(threadIdx.x);
                const int64_t pos = static_cast<int64_t>(s.t0) * KT + x;
                if (x < (s.t1 - s.t0) * KT && pos < s.n && pos < p.width) w[pos] = held[i] + (sums[x] + sums[kSpan * KT + x]);
            }
            sums_barrier_or(false);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 256);
    if (threadIdx.x == 0 && sh.abort) atomicOr(a.status, kStatusCopyLost);
}

template <bool BF16, int DP, int NQ>
cudaError_t launch_shape(const WeightParams &p, int sms, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(weights_kernel<BF16, DP, NQ>, Shape<DP, NQ>::kSmem, allowed);
    if (e != cudaSuccess) return e;
    return launch_pdl(weights_kernel<BF16, DP, NQ>, dim3(static_cast<unsigned>(sms)), Shape<DP, NQ>::kThreads, Shape<DP, NQ>::kSmem,
                      stream, 1, p);
}

// By the rows of a head, all accepted (how many are is not known here).
template <bool BF16>
cudaError_t launch_weights(const WeightParams &p, int sms, cudaStream_t s) {
    const bool few = p.a.next_n * p.a.group <= 32;
    if (p.a.dim <= 64) return few ? launch_shape<BF16, 64, 32>(p, sms, s) : launch_shape<BF16, 64, 128>(p, sms, s);
    if (p.a.dim <= 128) return few ? launch_shape<BF16, 128, 32>(p, sms, s) : launch_shape<BF16, 128, 128>(p, sms, s);
    return few ? launch_shape<BF16, 256, 32>(p, sms, s) : launch_shape<BF16, 256, 64>(p, sms, s);
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" int gbtopk_cache_weights(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride,
                                    int64_t q_head_stride, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                    const void *k_cache, int64_t k_slot_stride, int64_t k_head_stride, int64_t num_slots,
                                    const float *lse, const int32_t *page_table, int64_t pt_cols, int64_t pt_row_stride,
                                    int32_t page_size, const int32_t *seq_lens, int32_t next_n, const int64_t *tree_mask,
                                    const int64_t *accept_mask, float scale, float *weights, int32_t weight_heads,
                                    int64_t width, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (next_n < 1 || num_rows % next_n != 0 || width < 0) return GBTOPK_EINVAL;
    if (weight_heads != 1 && weight_heads != kv_heads) return GBTOPK_EINVAL;
    if (next_n > GBTOPK_MAX_NEXT_N || width > INT32_MAX || num_slots > INT32_MAX) return GBTOPK_EUNSUPPORTED;
    WeightParams p{};
    AttnParams &a = p.a;
    if ((rc = check_pages(page_table, pt_cols, pt_row_stride, page_size, num_slots, num_rows / next_n, &a.pages)) != GBTOPK_OK)
        return rc;
    if (num_rows == 0 || width == 0) return GBTOPK_OK;
    if (!seq_lens || !lse || !weights) return GBTOPK_EINVAL;
    if ((rc = check_rows(q, q_row_stride, q_head_stride, true)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(k_cache, k_slot_stride, k_head_stride, num_slots > 0)) != GBTOPK_OK) return rc;
    if (!aligned_to(lse, 4) || !aligned_to(weights, 16) || !aligned_to(seq_lens, 4) || !aligned_to(tree_mask, 8) ||
        !aligned_to(accept_mask, 8))
        return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < kWsHeaderBytes) return GBTOPK_EWORKSPACE;
    a.q = q;
    a.q_row = q_row_stride;
    a.q_head = q_head_stride;
    a.k = k_cache;
    a.k_slot = k_slot_stride;
    a.k_head = k_head_stride;
    a.seq_lens = seq_lens;
    a.tree_mask = tree_mask;
    a.requests = static_cast<int32_t>(num_rows / next_n);
    a.next_n = next_n;
    a.q_heads = q_heads;
    a.kv_heads = kv_heads;
    a.group = q_heads / kv_heads;
    a.dim = head_dim;
    a.row_tiles = 1;
    a.request_units = weight_heads;
    a.c = fmaxf(fabsf(scale) * kLog2e, FLT_MIN);
    a.negative = scale < 0.f;
    a.status = static_cast<uint32_t *>(workspace);
    a.wait_cycles = wait_cycles();
    a.pages.spare = static_cast<const int32_t *>(workspace);
    p.accept_mask = accept_mask;
    p.lse = lse;
    p.weights = weights;
    p.weight_heads = weight_heads;
    p.width = width;
    const int sms = device_sms();
    if (sms == 0) return GBTOPK_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return (dtype == GBTOPK_BF16 ? launch_weights<true>(p, sms, s) : launch_weights<false>(p, sms, s)) == cudaSuccess
               ? GBTOPK_OK
               : GBTOPK_ECUDA;
}
