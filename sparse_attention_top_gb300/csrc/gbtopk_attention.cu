// Attention of drafted tokens over a paged cache (gbtopk_tree_attention) and
// over selected slots (gbtopk_selected_attention).
//
// The rows that share a cached head - next_n tokens x the query heads of the
// group - are the rows of one matrix tile, so each cached key and value is
// copied once for all of them; above 256 rows (128 above dimension 128) once
// for each row tile of as many.  Per tile of KT cached positions:
//     S = Q K^T (tensor core, 32-bit accumulator in tensor memory),
//     P = 2^(c S - m), the reference m (about the running maximum) and the
//         sum l in registers,
//     O += P V (P from tensor memory, O stays there),
// O being rescaled only when a tile's maximum rises more than 8 (base 2) over
// m: P then stays below 2^8, in fp16 kernels below 2^15 (see kLift), which the
// type holds.  P is rounded to the inputs' type for the product (each
// probability is off by up to 2^-8 of itself in bf16 and 2^-11 in fp16, as the
// output is by its own rounding; the sum l is of the unrounded values); S, m, l
// and O are 32 bits.  The work of a call is the list of all (request, kv head,
// row tile, position tile); block c of a grid of one block per SM takes the
// c-th share of equal cost of that list whatever the lengths are, and a unit
// (request, head, row tile) that spans blocks leaves partial O, m, l in the
// workspace for combine_kernel.
//
// A block: W warpgroups of softmax (one row a thread), a warpgroup one warp of
// which issues the matrix products and whose others look up the cache slots of
// the tiles to come, a warpgroup that copies keys and values from those slots
// (cp.async, 16 bytes a lane, any page size and stride) into a ring of tiles.
// Copies run ahead of the products by the whole ring.
//
// Bound by the cache's bytes up to some 100 rows a head, above by the softmax
// and the products, which wait for one another: a tile's value product for all
// of its P, the key product after next for that.  Measured on one GB300 (copy
// rate 6.78 TB/s, bf16 products 1884 TFLOP/s), the kernels alone: 64 requests x
// 4 drafts over 1..8192 positions, 8 heads of 128, fp16, 170 us = 6.34 TB/s; of
// 256, 331 us = 6.51 TB/s; 2 requests x 8 over 163840 positions in pages of
// one, 8 heads of 64, 135 us = 4.96 TB/s (128-byte rows at random), of 256,
// 426 us = 6.30 TB/s; 16 requests x 64 drafts, 512 rows a head of 128, 105 us =
// 972 TFLOP/s (14 us of it the join), of 256, 276 us = 742 TFLOP/s (four row
// tiles, each of which copies the cache); 64 rows x 2048 selected entries of two
// heads, 29 us = 4.5 TB/s; one request of 1027 positions, 11.6 us.
#include <cfloat>
#include <cmath>

#include "gbtopk_paged.cuh"

namespace gbtopk {
namespace {

constexpr int kMaxGrid = 160;       // blocks of the attention kernel (workspace bound)
constexpr int kMaskRing = 8;        // tiles whose slots and validity bits are looked up ahead
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

// DP: head dimension rounded up to 64, 128 or 256.  W: softmax warpgroups.
// ROWS: query rows of a unit.  With two warpgroups and up to 128 rows both
// have the same rows and take the position tiles in turn (kSplit), each with
// an O of its own, joined at the unit's end; with 256 each has 128 of them.
// (A warp needs about 1000 to 2000 cycles for the softmax of a tile of 128
// columns, whose copies take 2800 at dimension 128 and 1400 at 64.)  A tile
// of 32 query rows leaves a stage more to the ring; the product reads 128
// rows all the same, the ring's bytes around them, whose results no one
// reads.  The second warpgroup's products then start 32 rows early, so that
// its rows lie in the tensor memory of its second warp: each of the two warps
// that have rows, and the one that issues products, has an SM quarter to
// itself.
template <int DP, int W, int ROWS>
struct Shape {
    static constexpr bool kSplit = W == 2 && ROWS <= 128;
    static constexpr int KT = DP == 256 ? 64 : 128;         // positions a tile
    static constexpr int kRows = ROWS;
    static constexpr int kJobs = kSplit ? 1 : W;            // products (jobs) a tile
    static constexpr int kShift = ROWS == 32 ? 32 : 0;      // tensor memory rows before the second warpgroup's
    static constexpr int kThreads = 128 * W + 256;
    static constexpr int kStageBytes = KT * DP * 2;
    static constexpr int kQBytes = kRows * DP * 2;
    static constexpr int kQBufs = ROWS == 32 ? 2 : 1;       // units whose queries are held
    static constexpr int kJoinCols = ROWS == 32 ? 32 : 16;  // columns of O that the warpgroups exchange at a time
    static constexpr int kJoin = kSplit ? (2 * ROWS * (kJoinCols + 1) * 4 + 127) / 128 * 128 : 0;
    static constexpr int kFixed = 7168;                     // barriers, slots and masks, scan scratch
    static constexpr int kFit = (static_cast<int>(kMaxSmemBytes) - 1024 - kFixed - kJoin - kQBufs * kQBytes) / kStageBytes;
    static constexpr int kStages = kFit < 12 ? kFit : 12;
    static constexpr size_t kSmem = 1024 + kFixed + kJoin + kQBufs * kQBytes + static_cast<size_t>(kStages) * kStageBytes;
    static constexpr uint32_t kS = 0, kO = 2 * KT;          // tensor memory columns
    static_assert(kO + W * DP <= 512, "tensor memory");
    static_assert(kStages >= 4 && kStages / 2 + 1 <= kMaskRing, "ring");   // copies never wait for slots behind the softmax
    static_assert(kSplit || ROWS == 128 * W, "rows");
};

struct Shared {
    uint64_t full[12], empty[12];   // ring stages: K and V of a tile alternate
    uint64_t slots_full[kMaskRing], slots_empty[kMaskRing];   // slots and validity bits of a tile
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2];             // S of a job is in tensor memory
    uint64_t p_full[2];             // P of a job is
    uint64_t pv_done[2];            // O holds the job's product
    uint64_t drain;
    int32_t slots[kMaskRing][128];  // cache slot of each position, -1 where there is none
    uint32_t mask[kMaskRing][4];    // positions with a slot, as bits
    uint64_t odd[kMaskRing];        // a tile's drafts left out of the value product (see clean_values)
    float2 ml[2][128];              // (m, l) of the two warpgroups' rows
    ScanScratch scan;
    uint32_t tmem;
    uint32_t abort;
};
static_assert(sizeof(Shared) <= 7168, "shared block");

// Barrier of the two softmax warps that share rows; true for both when `v`
// is for one.
__device__ __forceinline__ bool pair_barrier_or(int id, bool v) {
    uint32_t any;
    __syncwarp();
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(v)), "r"(id)
        : "memory");
    return any != 0;
}

// Drafted tokens whose values hold an infinity or a NaN: the product P V
// would carry 0 x inf into the rows that do not see them.  Their rows of the
// tile (drafts are `first` up to `end`) are set to zero and marked as bits, and the
// softmax warps add them at the unit's end to the rows that do.  By the warp
// that issues the products, in a call of its own: 2 % of the time of a batch of
// four drafts a request, 3 % of trees of 64 (inlined there 25 %, in the softmax
// warps, whose registers are all in use, 7 to 12 %, where the slots are looked
// up 10 %).  Only kernels for several tokens a request have it.
template <bool BF16, int DP, int KT>
__device__ __noinline__ void clean_values(uint8_t *tile, int32_t first, int32_t end, int32_t dim, uint64_t *marks) {
    constexpr int kLanes = DP / 8;   // of a row
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    const int lane = threadIdx.x & 31, c = lane % kLanes;
    const int32_t from = first < 0 ? 0 : first, to = end < KT ? end : KT;
    uint64_t odd = 0;
#pragma unroll 4
    for (int32_t r = from + lane / kLanes; r < to; r += 32 / kLanes) {
        if (c >= dim / 8) continue;
        const uint4 x = *reinterpret_cast<const uint4 *>(tile + tile_offset(KT, r, c));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((w[i] & kExp) == kExp || (w[i] >> 16 & kExp) == kExp) odd |= 1ull << (r - from);
    }
    odd = static_cast<uint64_t>(__reduce_or_sync(~0u, static_cast<uint32_t>(odd >> 32))) << 32 |
          __reduce_or_sync(~0u, static_cast<uint32_t>(odd));
    for (uint64_t left = odd; left; left &= left - 1) {
        const int32_t r = from + __ffsll(static_cast<long long>(left)) - 1;
        if (lane < kLanes) *reinterpret_cast<uint4 *>(tile + tile_offset(KT, r, lane)) = make_uint4(0, 0, 0, 0);
    }
    fence_async_reads();
    if (lane == 0) *marks = odd << (from - first);
    __threadfence_block();
    __syncwarp();
}

// 2^(c q.k - m) of one row and one position.
template <bool BF16>
__device__ __forceinline__ float row_prob(const AttnParams &p, const uint4 *q, const uint4 *k, float m) {
    float s = 0.f;
#pragma unroll 1
    for (int c = 0; c < p.dim / 8; ++c) {
        const uint4 a = fetch(q + c), b = fetch(k + c);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
        for (int i = 0; i < 4; ++i) {
            const float2 f = Half2<BF16>::up(x[i]), g = Half2<BF16>::up(y[i]);
            s = fmaf(f.x, g.x, fmaf(f.y, g.y, s));
        }
    }
    return exp2f((p.negative ? -s : s) * p.c - m);
}

template <bool BF16, int DP, int W, int ROWS, bool DRAFTS>
__global__ void __launch_bounds__(Shape<DP, W, ROWS>::kThreads, 1) attention_kernel(const __grid_constant__ AttnParams p) {
    using Sh = Shape<DP, W, ROWS>;
    constexpr bool SPLIT = Sh::kSplit;
    constexpr int KT = Sh::KT;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    float *join = reinterpret_cast<float *>(smem + Sh::kQBufs * Sh::kQBytes + Sh::kStages * Sh::kStageBytes);   // [2][kRows][kJoinCols + 1]
    Shared &sh = *reinterpret_cast<Shared *>(reinterpret_cast<uint8_t *>(join) + Sh::kJoin);
    // stage 0, the queries, the other stages (the products of kShift read
    // around the queries)
    const uint32_t ring = smem_addr(smem), q_smem = ring + Sh::kStageBytes;
    auto stage_at = [&](uint32_t s) { return ring + s * Sh::kStageBytes + (s ? Sh::kQBufs * Sh::kQBytes : 0); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kRoleWarp = 4 * W, kMmaWarp = kRoleWarp + 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            bar_init(&sh.full[i], 128);
            bar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kMaskRing; ++i) {
            bar_init(&sh.slots_full[i], 1);
            bar_init(&sh.slots_empty[i], 4 * Sh::kJobs);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.q_full[i], 128);
            bar_init(&sh.q_empty[i], 1);
            bar_init(&sh.s_full[i], 1);
            bar_init(&sh.p_full[i], 4);
            bar_init(&sh.pv_done[i], 1);
        }
        bar_init(&sh.drain, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) tmem_alloc(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_release();

    const Share share = block_share<KT, Sh::kThreads>(p, &sh.scan);
    const Waits abort{&sh.abort, p.wait_cycles};
    const uint32_t tmem = sh.tmem;
    Walk<KT> walk(p, share);
    const int32_t rows = p.next_n * p.group;   // of a (request, kv head)
    const int32_t chunks = (p.dim + 15) / 16 * 2, loaded = p.dim / 8;

    if (warp >= kRoleWarp + 4) {
        // ------------------------------------------------ copies
        const int w = warp - kRoleWarp - 4;
        const uint8_t *kb = static_cast<const uint8_t *>(p.k), *vb = static_cast<const uint8_t *>(p.v);
        const int64_t k_bytes = p.k_slot * 2, v_bytes = p.v_slot * 2;
        uint32_t unit = 0, g = 0, tile = 0;   // counters of units, ring stages and tiles
        uint32_t stage = 0, lap = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next()) {
            const Unit u = walk.u;
            if (u.span.n == 0) continue;   // nothing to see: the rows' zeros need no products
            const int32_t h = u.hm / p.row_tiles, r0 = (u.hm - h * p.row_tiles) * Sh::kRows;
            // the unit's queries
            const uint32_t qb = unit % Sh::kQBufs;
            if (unit >= Sh::kQBufs) ok = __all_sync(~0u, bar_wait(&sh.q_empty[qb], (unit / Sh::kQBufs - 1) & 1, abort));
            if (!ok) break;
            constexpr int kRowChunks = DP / 8 < 32 ? DP / 8 : 32, kStep = 128 / kRowChunks;   // lanes a row, rows a step
            for (int32_t r = (w * 32 + lane) / kRowChunks; r < Sh::kRows && r0 + r < rows; r += kStep) {
                const int32_t c = lane % kRowChunks, t = (r0 + r) / p.group, gq = r0 + r - t * p.group;
                const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                                     2 * ((static_cast<int64_t>(u.b) * p.next_n + t) * p.q_row + (h * p.group + gq) * p.q_head);
                if (c < chunks) copy16(q_smem + qb * Sh::kQBytes + tile_offset(Sh::kRows, r, c), c < loaded ? src + c * 16 : src, c < loaded ? 16u : 0u);
            }
            bar_arrive_copies(&sh.q_full[qb]);
            ++unit;
            for (int32_t t = u.t0; t < u.t1; ++t, ++tile) {
                ok = __all_sync(~0u, bar_wait(&sh.slots_full[tile % kMaskRing], (tile / kMaskRing) & 1, abort));
                if (!ok) break;
                const int32_t slot = reinterpret_cast<volatile int32_t *>(sh.slots[tile % kMaskRing])[w * (KT / 4) + (lane & (KT / 4 - 1))];
                for (int kv = 0; kv < 2; ++kv, ++g) {
                    if (g >= Sh::kStages) ok = __all_sync(~0u, bar_wait(&sh.empty[stage], (lap - 1) & 1, abort));
                    if (!ok) break;
                    copy_tile<DP, KT>(stage_at(stage), (kv ? vb + 2 * h * p.v_head : kb + 2 * h * p.k_head),
                                      kv ? v_bytes : k_bytes, slot, chunks, loaded, w, lane);
                    bar_arrive_copies(&sh.full[stage]);
                    if (++stage == Sh::kStages) {
                        stage = 0;
                        ++lap;
                    }
                }
                if (!ok) break;
            }
        }
        copies_land();
    } else if (warp >= kRoleWarp) {
        // ------------------------------------------------ matrix products
        if (warp == kMmaWarp) {   // all lanes alike, see elect_lane
            const bool lead = elect_lane();
            constexpr uint32_t kPanel = KT * 128;
            const uint32_t qk_desc = mma_desc(BF16, 128, KT, false, p.negative != 0);
            const uint32_t n_out = (p.dim + 15) / 16 * 16;
            const uint32_t pv_desc = mma_desc(BF16, 128, n_out, true, false);
            const int ksteps = chunks / 2;
            uint32_t unit = 0, job0 = 0, gi = 0;   // gi: the unit's first tile since the start
            bool ok = true;
            // stage and parity of ring item i
            auto wait_item = [&](uint32_t i) { return __all_sync(~0u, bar_wait(&sh.full[i % Sh::kStages], (i / Sh::kStages) & 1, abort)); };
            // (broadcasts: values known to be warp-uniform need no move to
            // uniform registers for every product)
            for (; __any_sync(~0u, walk.more()) && ok; walk.next()) {
                if (__any_sync(~0u, walk.u.span.n == 0)) continue;
                const uint32_t nt = __shfl_sync(~0u, static_cast<uint32_t>(walk.u.t1 - walk.u.t0), 0), jobs = nt * Sh::kJobs;
                // the first job that reaches the drafts
                const int32_t before = walk.u.span.ctx / KT - walk.u.t0;
                const uint32_t drafts = __shfl_sync(~0u, before > 0 && walk.u.span.ctx > 0 ? static_cast<uint32_t>(before) * Sh::kJobs : 0u, 0);
                const uint32_t qb = unit % Sh::kQBufs;
                ok = __all_sync(~0u, bar_wait(&sh.q_full[qb], (unit / Sh::kQBufs) & 1, abort));
                if (!ok) break;
                auto issue_qk = [&](uint32_t j) {
                    const uint32_t item = 2 * (gi + j / Sh::kJobs), s = item % Sh::kStages, sb = (job0 + j) & 1;
                    if (!wait_item(item)) return false;
                    fence_async_reads();
                    tc_fence_after();
                    const uint32_t qa = q_smem + qb * Sh::kQBytes + (Sh::kJobs == 2 ? (j & 1) * 128 * 128 : 0) - sb * Sh::kShift * 128, ka = stage_at(s);
                    if (lead) {   // unrolled: one thread issues, and its instructions bound the products' rate
#pragma unroll
                        for (int kk = 0; kk < DP / 16; ++kk)
                            if (kk < ksteps)
                                mma_ss(tmem + Sh::kS + sb * KT,
                                       smem_desc(qa + (kk >> 2) * (Sh::kRows * 128) + (kk & 3) * 32, 16, 1024),
                                       smem_desc(ka + (kk >> 2) * kPanel + (kk & 3) * 32, 16, 1024), qk_desc, kk > 0);
                        tc_commit(&sh.s_full[sb]);
                        if (Sh::kJobs == 1 || (j & 1)) tc_commit(&sh.empty[s]);
                        if (j + 1 == jobs) tc_commit(&sh.q_empty[qb]);
                    }
                    __syncwarp();
                    return true;
                };
                for (uint32_t j = 0; j < 2 && j < jobs && ok; ++j) ok = issue_qk(j);
                for (uint32_t j = 0; j < jobs && ok; ++j) {
                    const uint32_t job = job0 + j, sb = job & 1;
                    const uint32_t item = 2 * (gi + j / Sh::kJobs) + 1, s = item % Sh::kStages;
                    ok = wait_item(item);
                    if (!ok) break;
                    if constexpr (DRAFTS) {
                        if (j >= drafts && (Sh::kJobs == 1 || !(j & 1))) {
                            const int32_t at = (walk.u.t0 + static_cast<int32_t>(j / Sh::kJobs)) * KT;
                            clean_values<BF16, DP, KT>(smem + (stage_at(s) - ring), walk.u.span.ctx - at, walk.u.span.n - at, p.dim,
                                                       &sh.odd[(gi + j / Sh::kJobs) % kMaskRing]);
                        }
                    }
                    ok = __all_sync(~0u, bar_wait(&sh.p_full[sb], (job >> 1) & 1, abort));
                    if (!ok) break;
                    fence_async_reads();
                    tc_fence_after();
                    const uint32_t va = stage_at(s);
                    if (lead) {
#pragma unroll
                        for (int kk = 0; kk < KT / 16; ++kk)
                            mma_ts(tmem + Sh::kO + (W == 2 ? sb * DP : 0), tmem + Sh::kS + sb * KT + kk * 8,
                                   smem_desc(va + kk * 2048, kPanel, 1024), pv_desc, j >= W || kk > 0);
                        tc_commit(&sh.pv_done[sb]);
                        if (Sh::kJobs == 1 || (j & 1)) tc_commit(&sh.empty[s]);
                    }
                    __syncwarp();
                    if (j + 2 < jobs) ok = issue_qk(j + 2);
                }
                job0 += jobs;
                gi += nt;
                ++unit;
            }
            // every product is done before the block gives its memory up
            if (lead) tc_commit(&sh.drain);
            __syncwarp();
            if (!bar_wait(&sh.drain, 0, abort)) {
                const long long t0 = clock64();
                while (!bar_try(&sh.drain, 0) && clock64() - t0 < kWaitCycles) {
                }
            }
        }
        else {
            // -------------------------------------------- slots of the tiles to come
            // Three warps take the tiles in turn, up to kMaskRing tiles ahead of
            // the softmax: the page-table reads (DRAM latency where pages are
            // small) are then behind neither the copies nor one another.
            const int turn = warp == kRoleWarp + 3 ? 2 : warp - kRoleWarp;
            int32_t last_b = -1;
            uint64_t seen = ~0ull;   // drafted tokens that some row of the request sees
            uint32_t tile = 0;
            bool ok = true;
            for (; walk.more() && ok; walk.next()) {
                const Unit u = walk.u;
                if (u.span.n == 0) continue;
                if (u.b != last_b && p.seq_lens && p.tree_mask) {
                    const int64_t *tm = p.tree_mask + static_cast<int64_t>(u.b) * p.next_n;
                    uint64_t m = lane < p.next_n ? static_cast<uint64_t>(fetch(tm + lane)) : 0;
                    if (lane + 32 < p.next_n) m |= static_cast<uint64_t>(fetch(tm + lane + 32));
                    seen = static_cast<uint64_t>(__reduce_or_sync(~0u, static_cast<uint32_t>(m >> 32))) << 32 |
                           __reduce_or_sync(~0u, static_cast<uint32_t>(m));
                }
                last_b = u.b;
                for (int32_t t = u.t0; t < u.t1; ++t, ++tile) {
                    if (tile % 3 != static_cast<uint32_t>(turn)) continue;
                    const uint32_t r = tile % kMaskRing;
                    Paging::Place at[KT / 32];
#pragma unroll
                    for (int k = 0; k < KT / 32; ++k) {
                        const int32_t pos = t * KT + k * 32 + lane;
                        const bool is = pos < u.span.n && (pos < u.span.ctx || ((seen >> (pos - u.span.ctx)) & 1));
                        at[k] = p.seq_lens ? p.pages.place(u.b, pos, is) : p.pages.listed(p.indices + u.b * p.idx_row + pos, is);
                    }
                    if (tile >= kMaskRing) ok = __all_sync(~0u, bar_wait(&sh.slots_empty[r], (tile / kMaskRing - 1) & 1, abort));
                    if (!ok) break;
#pragma unroll
                    for (int k = 0; k < KT / 32; ++k) {
                        const int32_t slot = static_cast<int32_t>(p.pages.slot(at[k]));
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
        // ------------------------------------------------ softmax, output
        const int wg = warp >> 2, row0 = (warp & 3) * 32 - wg * Sh::kShift, row = row0 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // the warp's tensor memory lanes
        const uint32_t t_o = tmem + lanes + Sh::kO + wg * DP;
        const int row_wg = SPLIT ? 0 : wg * 128;   // the warpgroup's first row of a unit
        uint32_t job = Sh::kJobs == 2 ? wg : 0, tile = 0;
        bool ok = true;
        for (; walk.more() && ok; walk.next()) {
            const Unit u = walk.u;
            const int32_t h = u.hm / p.row_tiles, mt = u.hm - h * p.row_tiles;
            const int32_t rho = mt * Sh::kRows + row_wg + row;
            const bool mine = row >= 0 && rho < rows;
            const int32_t t = rho / p.group, gq = rho - t * p.group;
            const int64_t r = static_cast<int64_t>(u.b) * p.next_n + t;
            const bool active = row0 >= 0 && mt * Sh::kRows + row_wg + row0 < rows;   // any row of the warp
            if (u.span.n == 0) {
                if (threadIdx.x < 2) p.unit_ends[2 * (static_cast<int64_t>(u.b) * p.request_units + u.hm) + threadIdx.x] = static_cast<int32_t>(blockIdx.x);
                if (mine && !(SPLIT && wg == 1)) {
                    const int64_t at = r * p.q_heads + h * p.group + gq;
                    for (int c = 0; c < p.dim; c += 8)
                        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + 2 * (at * p.dim + c)) = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[at] = -INFINITY;
                }
                continue;
            }
            uint64_t tree = 0;
            if (mine && p.seq_lens) tree = p.tree_mask ? static_cast<uint64_t>(fetch(p.tree_mask + r)) : (~0ull >> (63 - t));
            float m = -INFINITY, l = 0.f;
            uint32_t last = ~0u;   // the unit's latest job of this warpgroup
            for (int32_t i = u.t0; i < u.t1; ++i, ++tile, job += Sh::kJobs) {
                const uint32_t sb = job & 1, ph = (job >> 1) & 1;
                if (SPLIT && sb != static_cast<uint32_t>(wg)) continue;
                ok = __all_sync(~0u, bar_wait(&sh.slots_full[tile % kMaskRing], (tile / kMaskRing) & 1, abort) &&
                                         bar_wait(&sh.s_full[sb], ph, abort));
                if (!ok) break;
                if (active) {
                    tc_fence_after();
                    const uint32_t t_s = tmem + lanes + Sh::kS + sb * KT;
                    // Half of the tile's scores are held at a time, so that 128
                    // registers do for every role: the upper half is read for its
                    // maximum, then the lower half, whose P goes over its own
                    // columns, then the upper half again.
                    constexpr int kHalf = KT / 2;
                    uint32_t x[kHalf];
                    // bits of the positions this row sees; all of them as a rule
                    uint32_t bits[KT / 32];
                    bool whole = true;
#pragma unroll
                    for (int c = 0; c < KT / 32; ++c) {
                        bits[c] = reinterpret_cast<volatile uint32_t *>(sh.mask[tile % kMaskRing])[c];
                        whole &= bits[c] == ~0u;
                    }
                    if (i * KT > u.span.ctx - KT) {   // (KT more could pass 31 bits)
                        whole = false;
#pragma unroll
                        for (int c = 0; c < KT / 32; ++c) {
                            const int32_t j0 = i * KT + c * 32 - u.span.ctx;   // drafted token of the word's bit 0
                            uint32_t see = 0;
                            if (j0 <= -32) see = ~0u;
                            else if (j0 < 0) see = static_cast<uint32_t>(tree << -j0) | ((1u << -j0) - 1);
                            else if (j0 < 64) see = static_cast<uint32_t>(tree >> j0);
                            bits[c] &= see;
                        }
                    }
                    auto load_half = [&](int half) {
#pragma unroll
                        for (int c = 0; c < kHalf; c += 32) tmem_load32(t_s + half * kHalf + c, x + c);
                        tc_wait_ld();
                        if (!whole) {
#pragma unroll
                            for (int c = 0; c < kHalf; ++c)
                                if (!((bits[(half * kHalf + c) / 32] >> (c & 31)) & 1)) x[c] = 0xff800000u;
                        }
                    };
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto max_half = [&]() {
#pragma unroll
                        for (int c = 0; c < kHalf; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(x[c]));
                    };
                    load_half(1);
                    max_half();
                    load_half(0);
                    max_half();
                    const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.c;
                    bool move = best > m + (kRescale + kLift<BF16>);   // also from -inf
                    if constexpr (!BF16) move |= best < m + (kLift<BF16> - kRescale) && best >= -FLT_MAX;
                    if (__any_sync(~0u, move)) {
                        float f = 1.f;
                        if constexpr (BF16) {
                            f = move && l > 0.f ? exp2_fast(m - best) : 1.f;
                            if (move) {
                                l *= f;
                                m = best;
                            }
                        } else if (move && !(l > 0.f)) {
                            m = best - kLift<BF16>;
                        } else if (move) {
                            // a whole number k lower; m - k is rounded where it is the larger
                            const float k = rintf(m + kLift<BF16> - best), to = m - k;
                            const float g = exp2_whole(k) * exp2_fast(m - (to + k));
                            if (k < 0.f || l * g <= kMostSum) {
                                f = g;
                                l *= f;
                                m = to;
                            }
                        }
                        if (__any_sync(~0u, f != 1.f)) {
                            // O is complete up to the row's last job
                            ok = __all_sync(~0u, bar_wait(&sh.pv_done[last & 1], (last >> 1) & 1, abort));
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < DP; c += 16) {
                                uint32_t o[16];
                                tmem_load16(t_o + c, o);
                                tc_wait_ld();
#pragma unroll
                                for (int d = 0; d < 16; ++d) o[d] = __float_as_uint(__uint_as_float(o[d]) * f);
                                tmem_store16(t_o + c, o);
                            }
                        }
                    }
                    const float mm = m == -INFINITY ? 0.f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    auto exp_half = [&](int half) {
#pragma unroll
                        for (int c0 = 0; c0 < kHalf; c0 += 32) {
                            uint32_t y[16];
#pragma unroll
                            for (int c = 0; c < 32; c += 2) {
                                const float a = exp2_fast(fmaf(__uint_as_float(x[c0 + c]), p.c, -mm));
                                const float b = exp2_fast(fmaf(__uint_as_float(x[c0 + c + 1]), p.c, -mm));
                                sum[c & 2] += a;
                                sum[(c & 2) + 1] += b;
                                y[c / 2] = Half2<BF16>::down(a, b);
                            }
                            tmem_store16(t_s + (half * kHalf + c0) / 2, y);
                        }
                    };
                    exp_half(0);
                    load_half(1);
                    exp_half(1);
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc_wait_st();
                    tc_fence_before();
                }
                last = job;
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&sh.p_full[sb]);
                    bar_arrive(&sh.slots_empty[tile % kMaskRing]);
                }
            }
            if (ok && last != ~0u) ok = __all_sync(~0u, bar_wait(&sh.pv_done[last & 1], (last >> 1) & 1, abort));
            if (!SPLIT && !ok) break;
            if (threadIdx.x == 0 && ok) {   // the blocks that share the unit
                int32_t *ends = p.unit_ends + 2 * (static_cast<int64_t>(u.b) * p.request_units + u.hm);
                if (u.t0 == 0) ends[0] = static_cast<int32_t>(blockIdx.x);
                if (u.t1 == u.tiles) ends[1] = static_cast<int32_t>(blockIdx.x);
            }
            __syncwarp();
            if (!active) {
                if (!ok) break;
                continue;
            }
            if (DRAFTS && ok && (u.t1 - 1) * KT > u.span.ctx - KT) {
                // Odd drafts of this warpgroup's tiles (they are in the last
                // two), the same for the warp's rows: added where a row sees them.
                uint64_t odd = 0;
                for (uint32_t back = 1; back <= 2; ++back)
                    if (u.t1 - u.t0 >= static_cast<int32_t>(back) && (u.t1 - static_cast<int32_t>(back)) * KT > u.span.ctx - KT &&
                        !(SPLIT && ((tile - back) & 1) != static_cast<uint32_t>(wg)))
                        odd |= reinterpret_cast<volatile uint64_t *>(sh.odd)[(tile - back) % kMaskRing];
                if (odd != 0) tc_fence_after();
#pragma unroll 1
                for (; odd; odd &= odd - 1) {
                    const int j = __ffsll(static_cast<long long>(odd)) - 1;
                    const int64_t slot = p.pages.slot(u.b, u.span.ctx + j);
                    const uint8_t *k = static_cast<const uint8_t *>(p.k) + 2 * (slot * p.k_slot + h * p.k_head);
                    const uint8_t *q = static_cast<const uint8_t *>(p.q) + 2 * (r * p.q_row + (h * p.group + gq) * p.q_head);
                    const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.v) + 2 * (slot * p.v_slot + h * p.v_head));
                    const bool sees = mine && ((tree >> j) & 1);
                    const float pr = sees ? row_prob<BF16>(p, reinterpret_cast<const uint4 *>(q), reinterpret_cast<const uint4 *>(k), m) : 0.f;
                    __syncwarp();
#pragma unroll 1
                    for (int c = 0; c < p.dim; c += 16) {
                        uint32_t o[16];
                        tmem_load16(t_o + c, o);
                        tc_wait_ld();
                        const uint4 x = fetch(v + c / 8), y = c + 8 < p.dim ? fetch(v + c / 8 + 1) : x;
                        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int d = 0; d < 8; ++d) {
                            const float2 f = Half2<BF16>::up(w[d]);
                            if (sees) {
                                o[2 * d] = __float_as_uint(fmaf(pr, f.x, __uint_as_float(o[2 * d])));
                                o[2 * d + 1] = __float_as_uint(fmaf(pr, f.y, __uint_as_float(o[2 * d + 1])));
                            }
                        }
                        __syncwarp();
                        tmem_store16(t_o + c, o);
                        tc_wait_st();
                    }
                }
            }
            const int pair = 1 + row0 / 32;   // barrier of the two warps that have these rows
            float f_own = 1.f, f_other = 0.f;   // SPLIT: factors of the two O
            if constexpr (SPLIT) {
                sh.ml[wg][row] = make_float2(m, l);
                ok = !pair_barrier_or(pair, !ok);   // both leave when one gave up
                if (!ok) break;
                const float2 other = sh.ml[1 - wg][row];
                const float top = fmaxf(m, other.x);
                // (an O without a job holds what an earlier unit left there)
                f_own = l == 0.f ? 0.f : exp2_between<BF16>(m, top);   // (a NaN score leaves l NaN)
                f_other = other.y == 0.f ? 0.f : exp2_between<BF16>(other.x, top);
                l = l * f_own + other.y * f_other;
                m = top;
            }
            tc_fence_after();
            const bool whole = u.t0 == 0 && u.t1 == u.tiles;
            const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (u.t0 > 0 ? 0 : 1);
            const int32_t part_row = row_wg + row;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int64_t q_at = r * p.q_heads + h * p.group + gq;
            auto put = [&](int c0, auto &o) {   // columns of the row, eight or more
                constexpr int N = sizeof(o) / 4;
                if (whole) {
                    uint8_t *dst = static_cast<uint8_t *>(p.out) + 2 * (q_at * p.dim + c0);
#pragma unroll
                    for (int c = 0; c < N; c += 8) {
                        if (c0 + c >= p.dim) break;
                        uint32_t y[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            y[d] = Half2<BF16>::down(__uint_as_float(o[c + 2 * d]) * inv, __uint_as_float(o[c + 2 * d + 1]) * inv);
                        *reinterpret_cast<uint4 *>(dst + 2 * c) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                } else {
                    // column by column: a warp's rows are 128 consecutive bytes
                    float *dst = p.part_o + (part * DP + c0) * Sh::kRows + part_row;
#pragma unroll
                    for (int c = 0; c < N; ++c) dst[c * Sh::kRows] = __uint_as_float(o[c]);
                }
            };
            if constexpr (SPLIT) {
                // Each warpgroup puts half of the columns out, the other's part
                // of them through shared memory, a piece at a time.
                constexpr int N = Sh::kJoinCols, kStride = N + 1;
                float *give = join + (wg * Sh::kRows + row) * kStride;
                const float *take = join + ((1 - wg) * Sh::kRows + row) * kStride;
                auto load = [&](int c0, uint32_t *o) {
                    if constexpr (N == 32) tmem_load32(t_o + c0, o);
                    else tmem_load16(t_o + c0, o);
                    tc_wait_ld();
                };
                for (int c0 = 0; c0 < DP / 2; c0 += N) {
                    const int mine0 = wg * (DP / 2) + c0, other0 = (1 - wg) * (DP / 2) + c0;
                    uint32_t o[N];
                    load(other0, o);
#pragma unroll
                    for (int c = 0; c < N; ++c) give[c] = __uint_as_float(o[c]);
                    load(mine0, o);
                    pair_barrier_or(pair, false);
#pragma unroll
                    for (int c = 0; c < N; ++c) {
                        const float x = f_own > 0.f ? __uint_as_float(o[c]) * f_own : 0.f, y = f_other > 0.f ? take[c] * f_other : 0.f;
                        o[c] = __float_as_uint(x + y);
                    }
                    pair_barrier_or(pair, false);
                    if (mine && mine0 < p.dim) put(mine0, o);
                    __syncwarp();
                }
            } else {
                for (int c0 = 0; c0 < p.dim; c0 += 32) {
                    uint32_t o[32];
                    tmem_load32(t_o + c0, o);
                    tc_wait_ld();
                    if (mine) put(c0, o);
                    __syncwarp();
                }
            }
            if (mine && !(SPLIT && wg == 1)) {
                if (!whole) p.part_ml[part * Sh::kRows + part_row] = make_float2(m, l);
                else if (p.lse) p.lse[q_at] = row_lse<BF16>(m, l);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free(tmem, 512);
    if (threadIdx.x == 0 && sh.abort) atomicOr(p.status, kStatusCopyLost);
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

int dim_class(int32_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

size_t partial_rows(int32_t dim) { return static_cast<size_t>(2 * kMaxGrid) * (dim > 128 ? 128 : 256); }
size_t unit_bytes(int64_t num_rows, int32_t q_heads) {   // a unit has a row or more
    return (static_cast<size_t>(num_rows) * q_heads * 8 + 255) / 256 * 256;
}

template <bool BF16, int DP, int W, int ROWS>
cudaError_t launch_shape(AttnParams p, uint8_t *ws, int sms, cudaStream_t stream) {
    using Sh = Shape<DP, W, ROWS>;
    const int64_t rows = static_cast<int64_t>(p.next_n) * p.group;
    p.row_tiles = static_cast<int32_t>((rows + Sh::kRows - 1) / Sh::kRows);
    p.request_units = p.kv_heads * p.row_tiles;
    p.unit_ends = reinterpret_cast<int32_t *>(ws + kWsHeaderBytes);
    p.part_ml = reinterpret_cast<float2 *>(ws + kWsHeaderBytes + unit_bytes(static_cast<int64_t>(p.requests) * p.next_n, p.q_heads));
    p.part_o = reinterpret_cast<float *>(p.part_ml + partial_rows(p.dim));
    // (a single token is seen by all of its request's rows)
    const int grid = sms < kMaxGrid ? sms : kMaxGrid;
    auto launch = [&](auto kernel, std::atomic<uint64_t> &allowed) {
        const cudaError_t e = allow_smem(kernel, Sh::kSmem, allowed);
        return e != cudaSuccess ? e : launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), Sh::kThreads, Sh::kSmem, stream, 1, p);
    };
    static std::atomic<uint64_t> allowed[2];
    const cudaError_t e = p.next_n > 1 ? launch(attention_kernel<BF16, DP, W, ROWS, true>, allowed[1])
                                       : launch(attention_kernel<BF16, DP, W, ROWS, false>, allowed[0]);
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(p.requests) * p.request_units;
    // no unit spans blocks where none has more than one tile
    const int64_t longest = p.seq_lens ? p.pages.cols * p.pages.page.d : p.top_k;
    if (longest <= Sh::KT) return cudaSuccess;
    const int64_t each = rows < Sh::kRows ? rows : Sh::kRows;
    dim3 blocks(static_cast<unsigned>(units), static_cast<unsigned>((each + kCombineRows - 1) / kCombineRows));
    blocks.z = DP / 16;
    if (units * blocks.y * blocks.z <= sms)
        return launch_pdl(combine_kernel<BF16, DP, 4, 16, 4>, blocks, kCombineThreads, 0, stream, 1, p, Sh::kRows);
    blocks.z = DP / 64;
    if (units * blocks.y * blocks.z <= sms)
        return launch_pdl(combine_kernel<BF16, DP, 4, 16, 1>, blocks, kCombineThreads, 0, stream, 1, p, Sh::kRows);
    blocks.z = 1;
    if (DP == 128 && units * blocks.y <= sms)
        return launch_pdl(combine_kernel<BF16, DP, DP / 16, DP == 128 ? 8 : 4, 1>, blocks, kCombineThreads, 0, stream, 1, p, Sh::kRows);
    return launch_pdl(combine_kernel<BF16, DP, DP / 16, 4, 1>, blocks, kCombineThreads, 0, stream, 1, p, Sh::kRows);
}

// By the rows of a head: up to 32, up to 128 (both warpgroups on them), more
// (each its row tile; they share each copied tile, and one's softmax runs
// beside the other's products).  Above dimension 128 tensor memory has room
// for one O.
template <bool BF16, int DP>
cudaError_t launch_dim(const AttnParams &p, uint8_t *ws, int sms, cudaStream_t s) {
    if constexpr (DP == 256) {
        return launch_shape<BF16, DP, 1, 128>(p, ws, sms, s);
    } else {
        const int64_t rows = static_cast<int64_t>(p.next_n) * p.group;
        if (rows <= 32) return launch_shape<BF16, DP, 2, 32>(p, ws, sms, s);
        if (rows <= 128) return launch_shape<BF16, DP, 2, 128>(p, ws, sms, s);
        return launch_shape<BF16, DP, 2, 256>(p, ws, sms, s);
    }
}

template <bool BF16>
cudaError_t launch_attention(const AttnParams &p, uint8_t *ws, int sms, cudaStream_t s) {
    switch (dim_class(p.dim)) {
        case 64: return launch_dim<BF16, 64>(p, ws, sms, s);
        case 128: return launch_dim<BF16, 128>(p, ws, sms, s);
        default: return launch_dim<BF16, 256>(p, ws, sms, s);
    }
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
    if (num_slots > INT32_MAX) return GBTOPK_EUNSUPPORTED;
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
    p.requests = static_cast<int32_t>(num_rows / p.next_n);
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.dim = head_dim;
    p.c = fmaxf(fabsf(scale) * kLog2e, FLT_MIN);   // a scale of 0 stays a product that ignores no mask
    p.negative = scale < 0.f;
    p.out = out;
    p.lse = lse;
    p.status = static_cast<uint32_t *>(workspace);
    p.wait_cycles = wait_cycles();
    p.pages.spare = static_cast<const int32_t *>(workspace);
    const int sms = device_sms();
    if (sms == 0) return GBTOPK_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    return (dtype == GBTOPK_BF16 ? launch_attention<true>(p, ws, sms, s) : launch_attention<false>(p, ws, sms, s)) ==
                   cudaSuccess
               ? GBTOPK_OK
               : GBTOPK_ECUDA;
}

}  // namespace

extern "C" {

size_t gbtopk_attention_workspace_bytes(int64_t num_rows, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (check_heads(GBTOPK_BF16, num_rows, q_heads, kv_heads, head_dim) != GBTOPK_OK) return 0;
    return kWsHeaderBytes + unit_bytes(num_rows, q_heads) + partial_rows(head_dim) * (8 + 4 * static_cast<size_t>(dim_class(head_dim)));
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
    if (!aligned_to(seq_lens, 4) || !aligned_to(tree_mask, 8)) return GBTOPK_EALIGN;
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
    if (!aligned_to(indices, 4)) return GBTOPK_EALIGN;
    AttnParams p{};
    p.pages.num_slots = num_slots;
    p.pages.page.init(1);
    p.indices = indices;
    p.top_k = static_cast<int32_t>(top_k);
    p.idx_row = idx_row_stride;
    p.next_n = 1;
    return attend(p, dtype, q, num_rows, q_row_stride, q_head_stride, q_heads, kv_heads, head_dim, k_cache, k_slot_stride,
                  k_head_stride, v_cache, v_slot_stride, v_head_stride, scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
