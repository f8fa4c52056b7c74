// Causal attention over whole prompts: packed sequences, grouped heads
// (gbtopk_prompt_attention).
//
// A unit is a sequence's next 256 query rows of one kv head (128 above dimension
// 128): tokens x the query heads of a group, as many of them as a power of two
// that divides the group has room for, so that a copied tile of keys and values
// serves all of them and a unit is short in tokens, which keeps what the
// diagonal wastes small.  Per tile of KT keys and each half of 128 rows:
//     S = Q K^T,   P = 2^(c S - m),   O += P V,
// with m, the sums and the rescaling of O as in gbtopk_attention.cu.  The halves
// take turns on the tensor cores: while one's softmax runs, the other's
// products do.  S and P of a half share tensor memory, so its next scores follow
// its value product, in issue order.
//
// Units are sorted by their number of key tiles (a counting sort by one block,
// in front of the kernel, 4.8 us) and dealt out to the persistent blocks in snake
// order, longest first: equal shares without a counter that blocks would race for
// (16 prompts 229 us a call, shortest first 256; one of 10007 tokens 605, 672).
//
// A block: two warpgroups of softmax and output (a row a thread), one warp that
// issues products, one that has tiles copied by tensor maps, one that cleans the
// value tiles that some row sees only in part: rows behind the sequence are
// zeroed, and rows with an infinity or NaN too (0 x inf would reach rows that do
// not see them); the softmax warps add the latter to the rows that do, at the
// unit's end.
//
// Measured a call, 32 over 8 heads of 128, bf16: one prompt of 10007 tokens 604 us
// (the kernel alone 584), 1358 TFLOP/s (72% of the burst rate; the products' own
// issue would take 547 us); 16 prompts up to 2048 tokens 228 us; 2 chunks up to 2048
// tokens over 16384 keys of 64, 32 over 4 heads, 443 us: at 64 columns a product's
// issue costs as much as at 128, 375 us of them.  Bound by the tensor pipe, and where units are short by their
// starts and ends and the diagonal's masked halves.
#include <cfloat>
#include <cmath>

#include "gbtopk_join.cuh"
#include "gbtopk_tma.cuh"

namespace gbtopk {
namespace {

// References up to which a score's product and its difference from the reference are
// one operation.  The difference of the largest is then what the product's rounding
// left off, up to 2^-24 of it: next to nothing here, and from 2^31 on a power beyond
// 32 bits.  Tiles with a row beyond it take products and differences one by one, in a
// loop of their own.  (All tiles so: 16 prompts 229 -> 237 us, the long one 607 -> 642.)
constexpr float kFused = 0x1p20f;
constexpr int kOddUnits = 8, kOddTiles = 4;   // units and their tiles whose marks are kept
constexpr int kBuckets = 2048;

struct PromptParams {
    CUtensorMap q_map, k_map, v_map;
    const void *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;   // elements
    const int32_t *cu_q, *cu_k;
    int64_t rows, keys;
    int32_t seqs, q_heads, kv_heads, group, dim;
    int32_t pack, shift;          // query heads of a unit: 1 << shift
    int32_t heads;                // units of a token tile
    float c;
    int32_t negative;
    void *out;
    float *lse;
    uint32_t *status;
    int64_t wait_cycles;
    int32_t *count;               // token tiles of the call
    int2 *list;                   // (sequence, token tile), longest first
    int32_t room;                 // its entries (offsets that are not ascending could ask for more)
};

struct Sequence {
    int32_t q0, rows, k0, keys;
};

__device__ __forceinline__ Sequence sequence(const PromptParams &p, int32_t i) {
    auto clamp = [](int64_t x, int64_t lo, int64_t hi) { return static_cast<int32_t>(x < lo ? lo : x > hi ? hi : x); };
    Sequence s;
    s.q0 = clamp(fetch(p.cu_q + i), 0, p.rows);
    s.rows = clamp(fetch(p.cu_q + i + 1), s.q0, p.rows) - s.q0;
    s.k0 = clamp(fetch(p.cu_k + i), 0, p.keys);
    s.keys = clamp(fetch(p.cu_k + i + 1), s.k0, p.keys) - s.k0;
    return s;
}

// Key tiles that the tokens before `end` of a sequence see.
template <int KT>
__device__ __forceinline__ int32_t key_tiles(const Sequence &s, int32_t end) {
    const int32_t seen = s.keys - s.rows + (end < s.rows ? end : s.rows);
    return seen > 0 ? (seen - 1) / KT + 1 : 0;
}

// Lists the token tiles, longest first (in buckets of key tiles).
template <int KT, int ROWS>
__global__ void __launch_bounds__(1024) order_kernel(const __grid_constant__ PromptParams p) {
    __shared__ int32_t at[kBuckets];
    __shared__ int32_t warps[32];
    __shared__ int32_t most;
    pdl_wait();
    pdl_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tokens = ROWS >> p.shift;
    for (int i = threadIdx.x; i < kBuckets; i += 1024) at[i] = 0;
    if (threadIdx.x == 0) most = 1;
    __syncthreads();
    int32_t mine = 1;
    for (int32_t i = threadIdx.x; i < p.seqs; i += 1024) {
        const Sequence s = sequence(p, i);
        const int32_t n = key_tiles<KT>(s, s.rows);
        mine = n > mine ? n : mine;
    }
    atomicMax(&most, mine);
    __syncthreads();
    const int32_t per = most / kBuckets + 1;
    for (int pass = 0; pass < 2; ++pass) {
        for (int32_t i = warp; i < p.seqs; i += 32) {
            const Sequence s = sequence(p, i);
            const int32_t tiles = (s.rows + tokens - 1) / tokens;
            for (int32_t t = lane; t < tiles; t += 32) {
                const int64_t end = (static_cast<int64_t>(t) + 1) * tokens;
                const int32_t b = kBuckets - 1 - key_tiles<KT>(s, end < s.rows ? static_cast<int32_t>(end) : s.rows) / per;
                const int32_t n = atomicAdd(&at[b], 1);
                if (pass && static_cast<uint32_t>(n) < static_cast<uint32_t>(p.room)) p.list[n] = make_int2(i, t);
            }
        }
        __syncthreads();
        if (pass) break;
        // counts to first places, two buckets a thread
        const int32_t a = at[2 * threadIdx.x], b = at[2 * threadIdx.x + 1];
        int32_t inc = a + b;
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) warps[warp] = inc;
        __syncthreads();
        int32_t before = 0, all = 0;
        for (int w = 0; w < 32; ++w) {
            before += w < warp ? warps[w] : 0;
            all += warps[w];
        }
        at[2 * threadIdx.x] = before + inc - a - b;
        at[2 * threadIdx.x + 1] = before + inc - b;
        // (counts as unsigned: offsets that are not ascending can ask for more than int32 holds)
        if (threadIdx.x == 0) *p.count = static_cast<uint32_t>(all) < static_cast<uint32_t>(p.room) ? all : p.room;
        __syncthreads();
    }
}

// DP: head dimension rounded up to 64, 128 or 256.  W: row tiles of a unit.
template <int DP>
struct Prompt {
    static constexpr int W = DP == 256 ? 1 : 2;
    static constexpr int KT = DP == 256 ? 64 : 128;
    static constexpr int kRows = 128 * W;
    static constexpr int kPanels = DP / 64;
    static constexpr int kThreads = 128 * W + 128;
    static constexpr uint32_t kQBytes = kRows * DP * 2, kStageBytes = KT * DP * 2;
    static constexpr int kFit = static_cast<int>((kMaxSmemBytes - 1024 - 2048 - kQBytes) / kStageBytes);
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr size_t kSmem = 1024 + 2048 + kQBytes + kStages * kStageBytes;
    static constexpr uint32_t kS = 0, kO = 2 * KT;      // tensor memory columns
    static_assert(kO + W * DP <= 512 && kStages >= 4, "tensor memory, ring");
    // a unit's tiles that are not whole: its tokens' and one more
    static_assert((kRows + KT - 1) / KT + 1 <= kOddTiles && kStages / 2 + 2 <= kOddUnits, "marks");
};

struct PromptShared {
    uint64_t full[10], empty[10];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t clean[10];              // a stage's value tile has been cleaned
    uint64_t seen[10];               // the cleaning warp has done with a stage
    uint64_t drain;
    uint32_t odd[kOddUnits][kOddTiles][4];   // rows of value tiles that were set to zero and have a value
    uint32_t any_odd[kOddUnits];
    uint32_t tmem;
    uint32_t abort;
};
static_assert(sizeof(PromptShared) <= 2048, "shared block");

// The units of block blockIdx.x, in order.
template <int DP>
struct Deal {
    const PromptParams &p;
    int64_t total, round = -1;
    Sequence s;
    int32_t token, head, kv;       // first token of the unit, its first query head, its kv head
    int32_t tiles, whole;          // key tiles, those that every row sees whole
    bool here = false;
    __device__ explicit Deal(const PromptParams &p) : p(p), total(static_cast<int64_t>(fetch(p.count)) * p.heads) { next(); }
    __device__ __forceinline__ void next() {
        using Sh = Prompt<DP>;
        const int64_t g = gridDim.x, b = blockIdx.x;
        here = false;
        while (!here && ++round * g < total) {
            const int64_t u = round * g + (round & 1 ? g - 1 - b : b);
            if (u >= total) continue;
            here = true;
            const int32_t x = static_cast<int32_t>(u / p.heads), hs = static_cast<int32_t>(u - static_cast<int64_t>(x) * p.heads);
            const int2 e = p.list[x];
            s = sequence(p, e.x);
            const int32_t sub = p.group >> p.shift, tokens = Sh::kRows >> p.shift;
            kv = hs / sub;
            head = kv * p.group + ((hs - kv * sub) << p.shift);
            token = e.y * tokens;
            tiles = key_tiles<Sh::KT>(s, s.rows - token < tokens ? s.rows : token + tokens);
            const int32_t all = s.keys - s.rows + token + 1;    // keys that the first token sees
            whole = all > 0 ? all / Sh::KT : 0;
            if (whole > tiles) whole = tiles;
        }
    }
};

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Waits &w) { return __all_sync(~0u, bar_wait(bar, parity, w)); }

__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Rows from `first` on of a value tile: those behind `end` are zeroed, those
// before it that hold an infinity or NaN zeroed and marked.
template <bool BF16, int DP, int KT>
__device__ __forceinline__ bool clean_tile(uint8_t *tile, int32_t first, int32_t end, int32_t dim, volatile uint32_t *marks) {
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    constexpr int kLanes = DP / 8;   // of a row
    const int lane = threadIdx.x & 31, c = lane % kLanes;
    bool any = false;
    for (int w = 0; w < KT / 32; ++w) {
        uint32_t odd = 0;
        for (int r = w * 32 + lane / kLanes; r < w * 32 + 32; r += 32 / kLanes) {
            if (r < first) continue;
            uint4 *at = reinterpret_cast<uint4 *>(tile + tile_offset(KT, r, c));
            const uint4 x = *at;
            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) bad |= (v[i] & kExp) == kExp || (v[i] >> 16 & kExp) == kExp;
            if (r >= end) *at = make_uint4(0, 0, 0, 0);
            else if (bad) odd |= 1u << (r & 31);
        }
        odd = __reduce_or_sync(~0u, odd);
        for (uint32_t left = odd; left; left &= left - 1) {
            const int r = w * 32 + __ffs(left) - 1;
            if (lane < kLanes) *reinterpret_cast<uint4 *>(tile + tile_offset(KT, r, lane)) = make_uint4(0, 0, 0, 0);
        }
        if (lane == 0) marks[w] = odd;
        any |= odd != 0;
    }
    return any;
}

template <bool BF16, int DP>
__global__ void __launch_bounds__(Prompt<DP>::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    using Sh = Prompt<DP>;
    constexpr int W = Sh::W, KT = Sh::KT;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    const uint32_t q_smem = smem_addr(smem), ring = q_smem + Sh::kQBytes;
    PromptShared &sh = *reinterpret_cast<PromptShared *>(smem + Sh::kQBytes + Sh::kStages * Sh::kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kIssue = 4 * W, kCopy = kIssue + 1, kClean = kIssue + 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Sh::kStages; ++i) {
            bar_init(&sh.full[i], 1);
            bar_init(&sh.empty[i], 1);
            bar_init(&sh.seen[i], 1);
            bar_init(&sh.clean[i], 1);
        }
        bar_init(&sh.q_full, 1);
        bar_init(&sh.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.s_full[i], 1);
            bar_init(&sh.p_full[i], 4);
            bar_init(&sh.pv_done[i], 1);
        }
        bar_init(&sh.drain, 1);
        for (int i = 0; i < kOddUnits; ++i) sh.any_odd[i] = 0;
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssue) tmem_alloc(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_release();

    const Waits abort{&sh.abort, p.wait_cycles};
    const uint32_t tmem = sh.tmem;
    Deal<DP> deal(p);
    bool ok = true;

    if (warp >= kIssue) {
        if (warp == kCopy) {
            // ------------------------------------------------ copies
            const bool lead = elect_lane();
            uint32_t unit = 0, stage = 0, lap = 0;
            for (; deal.here && ok; deal.next()) {
                if (deal.tiles == 0) continue;
                if (unit > 0) ok = warp_wait(&sh.q_empty, (unit - 1) & 1, abort);
                if (!ok) break;
                if (lead) {
                    bar_expect(&sh.q_full, Sh::kQBytes);
                    for (int w = 0; w < W; ++w)
                        for (int n = 0; n < Sh::kPanels; ++n)
                            copy_box(q_smem + (w * Sh::kPanels + n) * 128 * 128, &p.q_map, n * 64, deal.head,
                                     deal.s.q0 + deal.token + w * (128 >> p.shift), &sh.q_full);
                }
                ++unit;
                for (int32_t t = 0; t < deal.tiles && ok; ++t) {
                    for (int kv = 0; kv < 2; ++kv) {
                        if (lap > 0) ok = warp_wait(&sh.empty[stage], (lap - 1) & 1, abort) && warp_wait(&sh.seen[stage], (lap - 1) & 1, abort);
                        if (!ok) break;
                        if (lead) {
                            bar_expect(&sh.full[stage], Sh::kStageBytes);
                            for (int n = 0; n < Sh::kPanels; ++n)
                                copy_box(ring + stage * Sh::kStageBytes + n * KT * 128, kv ? &p.v_map : &p.k_map, n * 64, deal.kv,
                                         deal.s.k0 + t * KT, &sh.full[stage]);
                        }
                        __syncwarp();
                        if (++stage == Sh::kStages) {
                            stage = 0;
                            ++lap;
                        }
                    }
                }
            }
            // the block does not end before its copies have
            const long long t0 = clock64();
            const uint32_t n = lap * Sh::kStages + stage;     // items begun
            for (uint32_t i = n > Sh::kStages ? n - Sh::kStages : 0; i < n; ++i)
                while (!bar_try(&sh.full[i % Sh::kStages], (i / Sh::kStages) & 1) && clock64() - t0 < kWaitCycles) {
                }
            while (unit > 0 && !bar_try(&sh.q_full, (unit - 1) & 1) && clock64() - t0 < kWaitCycles) {
            }
            __syncwarp();
        } else if (warp == kIssue) {
            // ------------------------------------------------ matrix products (all lanes alike, see elect_lane)
            const bool lead = elect_lane();
            const uint32_t qk_desc = mma_desc(BF16, 128, KT, false, p.negative != 0);
            const uint32_t pv_desc = mma_desc(BF16, 128, (p.dim + 15) / 16 * 16, true, false);
            const int ksteps = (p.dim + 15) / 16;
            uint32_t unit = 0, job0 = 0, gi = 0, cleaned = 0;   // gi: the unit's first tile since the start; parities of the stages' cleaning
            auto wait_item = [&](uint32_t i) { return warp_wait(&sh.full[i % Sh::kStages], (i / Sh::kStages) & 1, abort); };
            for (; __any_sync(~0u, deal.here) && ok; deal.next()) {
                const uint32_t nt = __shfl_sync(~0u, static_cast<uint32_t>(deal.tiles), 0), jobs = nt * W;
                const uint32_t whole = __shfl_sync(~0u, static_cast<uint32_t>(deal.whole), 0);
                if (nt == 0) continue;
                ok = warp_wait(&sh.q_full, unit & 1, abort);
                if (!ok) break;
                auto issue_qk = [&](uint32_t j) {
                    const uint32_t item = 2 * (gi + j / W), s = item % Sh::kStages, sb = (job0 + j) & 1;
                    if (!wait_item(item)) return false;
                    tc_fence_after();
                    const uint64_t qa = smem_desc(q_smem + (W == 2 ? sb * 128 * DP * 2 : 0), 16, 1024), ka = smem_desc(ring + s * Sh::kStageBytes, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk)
                        if (kk < ksteps)
                            mma_ss_if(lead, tmem + Sh::kS + sb * KT, qa + (kk >> 2) * 1024 + (kk & 3) * 2, ka + (kk >> 2) * (KT * 8) + (kk & 3) * 2, qk_desc, kk > 0);
                    if (lead) {
                        tc_commit(&sh.s_full[sb]);
                        if (W == 1 || (j & 1)) tc_commit(&sh.empty[s]);
                        if (j + 1 == jobs) tc_commit(&sh.q_empty);
                    }
                    __syncwarp();
                    return true;
                };
                for (uint32_t j = 0; j < 2 && j < jobs && ok; ++j) ok = issue_qk(j);
                for (uint32_t j = 0; j < jobs && ok; ++j) {
                    const uint32_t job = job0 + j, sb = job & 1, item = 2 * (gi + j / W) + 1, s = item % Sh::kStages;
                    ok = wait_item(item);
                    if (ok && j / W >= whole && (W == 1 || !(j & 1))) {
                        ok = warp_wait(&sh.clean[s], (cleaned >> s) & 1, abort);
                        cleaned ^= 1u << s;
                    }
                    ok = ok && warp_wait(&sh.p_full[sb], (job >> 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t va = smem_desc(ring + s * Sh::kStageBytes, KT * 128, 1024);
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        mma_ts_if(lead, tmem + Sh::kO + (W == 2 ? sb * DP : 0), tmem + Sh::kS + sb * KT + kk * 8, va + kk * 128, pv_desc, j >= W || kk > 0);
                    if (lead) {
                        tc_commit(&sh.pv_done[sb]);
                        if (W == 1 || (j & 1)) tc_commit(&sh.empty[s]);
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
            __syncwarp();
        } else if (warp == kClean) {
            // ------------------------------------------------ value tiles that are not whole
            uint32_t unit = 0, gi = 0;
            for (; deal.here && ok; deal.next()) {
                if (deal.tiles == 0) continue;
                const uint32_t u = unit % kOddUnits;
                bool any = false;
                // (every item is waited for in turn, and none copied over one that this warp has not
                // seen: a parity tells two laps of a stage apart, not three.  By arrivals at `empty`
                // in place of `seen` the long prompt took 611 us for 604)
                for (int32_t t = 0; t < deal.tiles; ++t) {
                    const uint32_t item = 2 * (gi + t) + 1, s = item % Sh::kStages;
                    ok = warp_wait(&sh.full[(item - 1) % Sh::kStages], ((item - 1) / Sh::kStages) & 1, abort);
                    if (ok && lane == 0) bar_arrive(&sh.seen[(item - 1) % Sh::kStages]);
                    ok = ok && warp_wait(&sh.full[s], (item / Sh::kStages) & 1, abort);
                    if (!ok) break;
                    if (t < deal.whole) {
                        if (lane == 0) bar_arrive(&sh.seen[s]);
                        continue;
                    }
                    const int32_t first = deal.s.keys - deal.s.rows + deal.token + 1 - t * KT;    // the first that not every row sees
                    any |= clean_tile<BF16, DP, KT>(smem + Sh::kQBytes + s * Sh::kStageBytes, first, deal.s.keys - t * KT, p.dim, sh.odd[u][t - deal.whole]);
                    if (lane == 0) reinterpret_cast<volatile uint32_t *>(sh.any_odd)[u] = any;
                    fence_async_reads();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&sh.clean[s]);
                        bar_arrive(&sh.seen[s]);
                    }
                }
                gi += deal.tiles;
                ++unit;
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------ softmax, output
        const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // the warp's tensor memory lanes
        const uint32_t t_o = tmem + lanes + Sh::kO + wg * DP;
        uint32_t job = W == 2 ? wg : 0, unit = 0;
        for (; deal.here && ok; deal.next()) {
            const int32_t t = deal.token + wg * (128 >> p.shift) + (row >> p.shift);      // the row's token
            const bool mine = t < deal.s.rows;
            const int32_t last = deal.s.keys - deal.s.rows + (mine ? t : deal.s.rows - 1);   // the last key that it sees
            const int64_t q_at = (static_cast<int64_t>(deal.s.q0) + t) * p.q_heads + deal.head + (row & (p.pack - 1));
            if (deal.tiles == 0) {
                if (mine) {
                    for (int c = 0; c < p.dim; c += 8)
                        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + 2 * (q_at * p.dim + c)) = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[q_at] = -INFINITY;
                }
                continue;
            }
            float m = -INFINITY, l = 0.f;
            uint32_t before = ~0u;   // the unit's latest job of this warpgroup
            bool far = false;        // some row's reference is beyond kFused
            for (int32_t i = 0; i < deal.tiles; ++i, job += W) {
                const uint32_t sb = job & 1;
                ok = warp_wait(&sh.s_full[sb], (job >> 1) & 1, abort);
                if (!ok) break;
                tc_fence_after();
                const uint32_t t_s = tmem + lanes + Sh::kS + sb * KT;
                uint32_t x[KT];
#pragma unroll
                for (int c = 0; c < KT; c += 32) tmem_load32(t_s + c, x + c);
                tc_wait_ld();
                if (i >= deal.whole) {
                    const int32_t seen = last - i * KT;    // the last column that the row sees
#pragma unroll
                    for (int c = 0; c < KT; ++c)
                        if (c > seen) x[c] = 0xff800000u;
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < KT; ++c) top[c & 3] = fmaxf(top[c & 3], __uint_as_float(x[c]));
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
                        const float k = rintf(m + kLift<BF16> - best);
                        float to = m - k, g = exp2_whole(k) * exp2_fast(m - (to + k));
                        if (fabsf(best) > kFused) {      // (whose own steps are whole numbers or nearly)
                            to = best - kLift<BF16>;
                            g = exp2_fast(m - to);
                        }
                        if (to > m || l * g <= kMostSum) {
                            f = g;
                            l *= f;
                            m = to;
                        }
                    }
                    if constexpr (DP == 64) far = __any_sync(~0u, fabsf(m) > kFused && m != -INFINITY);
                    if (__any_sync(~0u, f != 1.f)) {
                        // O is complete up to the row's last job
                        ok = warp_wait(&sh.pv_done[before & 1], (before >> 1) & 1, abort);
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
                float2 sum[2] = {};
                // (at dimension 64 a vote a tile costs more than the flag does: 2 chunks over 16384
                // keys 460 us, with the flag 443, without either 429; else less: one of 10007 tokens
                // 606, 614, 607)
                if (DP == 64 ? far : __any_sync(~0u, fabsf(mm) > kFused)) {
#pragma unroll 1
                    for (int c0 = 0; c0 < KT; c0 += 16) {
                        uint32_t z[16], y[8];
                        tmem_load16(t_s + c0, z);
                        tc_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; c += 2) {
                            const int32_t seen = i < deal.whole ? KT : last - i * KT - c0;
                            const float a = c > seen ? 0.f : exp2_fast(__fmul_rn(__uint_as_float(z[c]), p.c) - mm);
                            const float b = c + 1 > seen ? 0.f : exp2_fast(__fmul_rn(__uint_as_float(z[c + 1]), p.c) - mm);
                            add2(sum[c / 2 & 1], a, b);
                            y[c / 2] = Half2<BF16>::down(a, b);
                        }
                        tmem_store8(t_s + c0 / 2, y);      // (over scores that have been read)
                    }
                } else {
#pragma unroll
                    for (int c0 = 0; c0 < KT; c0 += 32) {
                        uint32_t y[16];
#pragma unroll
                        for (int c = 0; c < 32; c += 2) {
                            const float2 e = fma2(__uint_as_float(x[c0 + c]), __uint_as_float(x[c0 + c + 1]), p.c, -mm);
                            const float a = exp2_fast(e.x), b = exp2_fast(e.y);
                            add2(sum[c / 2 & 1], a, b);
                            y[c / 2] = Half2<BF16>::down(a, b);
                        }
                        tmem_store16(t_s + c0 / 2, y);
                    }
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tc_wait_st();
                tc_fence_before();
                before = job;
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.p_full[sb]);
            }
            if (ok) ok = warp_wait(&sh.pv_done[before & 1], (before >> 1) & 1, abort);
            if (!ok) break;
            tc_fence_after();
            if (deal.whole < deal.tiles && reinterpret_cast<volatile uint32_t *>(sh.any_odd)[unit % kOddUnits]) {
                // odd values, added where a row sees them
                const uint8_t *q = static_cast<const uint8_t *>(p.q) + 2 * ((static_cast<int64_t>(deal.s.q0) + (mine ? t : 0)) * p.q_row +
                                                                            (deal.head + (row & (p.pack - 1))) * p.q_head);
#pragma unroll 1
                for (int n = 0; n < (deal.tiles - deal.whole) * (KT / 32); ++n) {
                    const int32_t tile = n / (KT / 32), word = n - tile * (KT / 32);
                    uint32_t odd = reinterpret_cast<volatile uint32_t *>(sh.odd[unit % kOddUnits][tile])[word];
#pragma unroll 1
                    for (; odd; odd &= odd - 1) {
                        const int32_t j = (deal.whole + tile) * KT + word * 32 + __ffs(static_cast<int>(odd)) - 1;
                        const int64_t key = static_cast<int64_t>(deal.s.k0) + j;
                        const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.k) + 2 * (key * p.k_row + deal.kv * p.k_head));
                        const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.v) + 2 * (key * p.v_row + deal.kv * p.v_head));
                        const bool sees = mine && j <= last;
                        float s = 0.f;
#pragma unroll 1
                        for (int c = 0; sees && c < p.dim / 8; ++c) {
                            const uint4 a = fetch(reinterpret_cast<const uint4 *>(q) + c), b = fetch(k + c);
                            const uint32_t f[4] = {a.x, a.y, a.z, a.w}, g[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int d = 0; d < 4; ++d) {
                                const float2 qq = Half2<BF16>::up(f[d]), kk = Half2<BF16>::up(g[d]);
                                s = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, s));
                            }
                        }
                        // (no larger than the softmax lets it be: s is another sum than its, of other roundings)
                        const float pr = sees ? exp2_fast(fminf(__fmul_rn(p.negative ? -s : s, p.c) - m, kRescale + kLift<BF16>)) : 0.f;
                        __syncwarp();
#pragma unroll 1
                        for (int c = 0; c < p.dim; c += 16) {
                            uint32_t o[16];
                            tmem_load16(t_o + c, o);
                            tc_wait_ld();
                            const uint4 a = fetch(v + c / 8), b = c + 8 < p.dim ? fetch(v + c / 8 + 1) : a;
                            const uint32_t f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int d = 0; d < 8; ++d) {
                                const float2 g = Half2<BF16>::up(f[d]);
                                if (sees) {
                                    o[2 * d] = __float_as_uint(fmaf(pr, g.x, __uint_as_float(o[2 * d])));
                                    o[2 * d + 1] = __float_as_uint(fmaf(pr, g.y, __uint_as_float(o[2 * d + 1])));
                                }
                            }
                            __syncwarp();
                            tmem_store16(t_o + c, o);
                            tc_wait_st();
                        }
                    }
                }
            }
            ++unit;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint8_t *dst = static_cast<uint8_t *>(p.out) + 2 * q_at * p.dim;
#pragma unroll 1
            for (int c0 = 0; c0 < p.dim; c0 += 32) {
                uint32_t o[32];
                tmem_load32(t_o + c0, o);
                tc_wait_ld();
                if (mine) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        if (c0 + c >= p.dim) break;
                        uint32_t y[4];
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            y[d] = Half2<BF16>::down(__uint_as_float(o[c + 2 * d]) * inv, __uint_as_float(o[c + 2 * d + 1]) * inv);
                        *reinterpret_cast<uint4 *>(dst + 2 * (c0 + c)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                __syncwarp();
            }
            if (mine && p.lse) p.lse[q_at] = row_lse<BF16>(m, l);
            tc_fence_before();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssue) tmem_free(tmem, 512);
    if (threadIdx.x == 0 && sh.abort) atomicOr(p.status, kStatusCopyLost);
}

template <bool BF16, int DP>
int launch_prompt(const PromptParams &p, int sms, cudaStream_t s) {
    using Sh = Prompt<DP>;
    static std::atomic<uint64_t> allowed;
    auto kernel = prompt_kernel<BF16, DP>;
    cudaError_t e = allow_smem(kernel, Sh::kSmem, allowed);
    if (e == cudaSuccess) e = launch_pdl(order_kernel<Sh::KT, Sh::kRows>, dim3(1), 1024, 0, s, 1, p);
    if (e == cudaSuccess) e = launch_pdl(kernel, dim3(static_cast<unsigned>(sms)), Sh::kThreads, Sh::kSmem, s, 1, p);
    return e == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}

template <bool BF16>
int launch_prompt(const PromptParams &p, int sms, cudaStream_t s) {
    if (p.dim <= 64) return launch_prompt<BF16, 64>(p, sms, s);
    if (p.dim <= 128) return launch_prompt<BF16, 128>(p, sms, s);
    return launch_prompt<BF16, 256>(p, sms, s);
}

// Query heads of a unit: the largest power of two up to 128 that divides the group
// (groups of 4, 16 prompts: 229 us a call, a head a unit 330; one of 10007 tokens 605, 668).
int log2_pack(int32_t group) {
    int shift = 0;
    while (shift < 7 && group % (2 << shift) == 0) ++shift;
    return shift;
}

// Token tiles of a call, at most.
size_t token_tiles(int64_t rows, int64_t seqs, int32_t group, int32_t dim) {
    return static_cast<size_t>(rows / ((dim > 128 ? 128 : 256) >> log2_pack(group)) + seqs);
}

// Strides of a dimension of one entry may be anything: a map wants some.
bool head_map(CUtensorMap *map, const void *base, int32_t dim, int32_t heads, int64_t rows, int64_t head, int64_t row, uint32_t box_heads,
              uint32_t box_rows) {
    const int64_t h = heads > 1 ? head : dim, r = rows > 1 ? row : dim;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(h) * 2, static_cast<cuuint64_t>(r) * 2};
    const cuuint32_t box[3] = {64, box_heads, box_rows};
    return tensor_map(map, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" {

size_t gbtopk_prompt_workspace_bytes(int64_t num_rows, int32_t num_seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
    if (check_heads(GBTOPK_BF16, num_rows, q_heads, kv_heads, head_dim) != GBTOPK_OK || num_seqs < 0) return 0;
    return kWsHeaderBytes + 256 + token_tiles(num_rows, num_seqs, q_heads / kv_heads, head_dim) * sizeof(int2);
}

int gbtopk_prompt_attention(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                            int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *k, int64_t k_row_stride,
                            int64_t k_head_stride, const void *v, int64_t v_row_stride, int64_t v_head_stride, int64_t num_keys,
                            const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int32_t num_seqs, float scale, void *out,
                            float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (num_keys < 0 || num_seqs < 0) return GBTOPK_EINVAL;
    if (num_keys > INT32_MAX - 1024 || num_rows > INT32_MAX - 1024) return GBTOPK_EUNSUPPORTED;
    if ((rc = check_rows(q, q_row_stride, q_head_stride, num_rows > 0)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(k, k_row_stride, k_head_stride, num_keys > 0)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(v, v_row_stride, v_head_stride, num_keys > 0)) != GBTOPK_OK) return rc;
    if (num_rows == 0 || num_seqs == 0) return GBTOPK_OK;
    // (rows that lie over one another have no tensor map)
    auto over = [&](int64_t rows, int64_t row, int32_t heads, int64_t head) { return (rows > 1 && row == 0) || (heads > 1 && head == 0); };
    if (over(num_rows, q_row_stride, q_heads, q_head_stride) || over(num_keys, k_row_stride, kv_heads, k_head_stride) ||
        over(num_keys, v_row_stride, kv_heads, v_head_stride))
        return GBTOPK_EUNSUPPORTED;
    if (!cu_seqlens_q || !out) return GBTOPK_EINVAL;
    if (!aligned_to(cu_seqlens_q, 4) || !aligned_to(cu_seqlens_k, 4) || !aligned_to(out, 16) || !aligned_to(lse, 4)) return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) ||
        workspace_bytes < gbtopk_prompt_workspace_bytes(num_rows, num_seqs, q_heads, kv_heads, head_dim))
        return GBTOPK_EWORKSPACE;
    PromptParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_row = q_row_stride;
    p.q_head = q_head_stride;
    p.k_row = k_row_stride;
    p.k_head = k_head_stride;
    p.v_row = v_row_stride;
    p.v_head = v_head_stride;
    p.cu_q = cu_seqlens_q;
    p.cu_k = cu_seqlens_k ? cu_seqlens_k : cu_seqlens_q;
    p.rows = num_rows;
    p.keys = num_keys;
    p.seqs = num_seqs;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.dim = head_dim;
    p.shift = log2_pack(p.group);
    p.pack = 1 << p.shift;
    p.heads = q_heads >> p.shift;
    p.c = fmaxf(fabsf(scale) * kLog2e, FLT_MIN);   // a scale of 0 stays a product that ignores no mask
    p.negative = scale < 0.f;
    p.out = out;
    p.lse = lse;
    p.status = static_cast<uint32_t *>(workspace);
    p.wait_cycles = wait_cycles();
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.count = reinterpret_cast<int32_t *>(ws + kWsHeaderBytes);
    p.list = reinterpret_cast<int2 *>(ws + kWsHeaderBytes + 256);
    const size_t room = token_tiles(num_rows, num_seqs, p.group, head_dim);
    p.room = static_cast<int32_t>(room < INT32_MAX ? room : INT32_MAX);
    // (without keys nothing is copied: any map does)
    const uint32_t kt = head_dim > 128 ? 64 : 128;
    const bool keys = num_keys > 0;
    if (!head_map(&p.q_map, q, head_dim, q_heads, num_rows, q_head_stride, q_row_stride, p.pack, 128 >> p.shift) ||
        !head_map(&p.k_map, keys ? k : q, head_dim, keys ? kv_heads : 1, keys ? num_keys : 1, k_head_stride, k_row_stride, 1, kt) ||
        !head_map(&p.v_map, keys ? v : q, head_dim, keys ? kv_heads : 1, keys ? num_keys : 1, v_head_stride, v_row_stride, 1, kt))
        return GBTOPK_ECUDA;
    const int sms = device_sms();
    if (sms == 0) return GBTOPK_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dtype == GBTOPK_BF16 ? launch_prompt<true>(p, sms, s) : launch_prompt<false>(p, sms, s);
}

}  // extern "C"
