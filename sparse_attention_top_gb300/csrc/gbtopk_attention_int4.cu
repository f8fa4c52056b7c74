// Attention of drafted tokens over a paged 4-bit cache
// (gbtopk_tree_attention_int4) and over selected slots of one
// (gbtopk_selected_attention_int4).
//
// Per tile of 128 cached positions, with the rows that share a cached head
// (next_n tokens x the query heads of the group) as columns:
//     S^T = K Q^T      (positions x rows; K from tensor memory),
//     P^T = 2^(c S^T - m),
//     O^T += V^T P^T   (head dimension x rows; V from shared memory),
// O^T being rescaled only when a score rises more than 8 (base 2) over its
// row's reference m.  A product costs by its columns, so a few rows cost few
// cycles, and one thread has one position: its key goes from its codes to its
// lane of tensor memory without touching shared memory again, and neither
// maximum nor sum of a row crosses threads except where m moves and at the
// unit's end.
//
// Keys and values are exact in bf16 (3 bits of code x 4 bits of scale), for fp16
// inputs too.  An fp16 query is the sum of two bf16 numbers (11 bits are 8 + 3),
// each a column of its own, and so is its probability (16 bits of it); S and O
// are the sums of the two columns.  So fp16 needs no scaling against its
// range, and its probabilities are more exact than fp16's own.  With bf16
// inputs each probability is rounded to bf16 (2^-8 of itself) for its product,
// as the 16-bit kernels' are.  S, m, l and O are 32 bits.
//
// A block, one an SM: four warps of softmax and output, four that turn the codes
// of keys into tensor memory, four that turn those of values into a
// shared-memory tile, seven that look up slots and have the rows copied into a
// ring (each a tile in turn; a lane gathers four rows by a tensor map), one that
// issues products.  Shares, units and the join are those of gbtopk_attention.cu,
// but that a gang of blocks takes the units of one request (its heads and row
// tiles) over the same positions at once: a 128-byte line of the cache holds parts
// of two heads' rows, which are then read from memory together.
//
// Measured: 64 requests x 4 drafts, 1..8192 positions of 8 heads of 128, fp16: 132
// us, the 300 MB of the cache read once (45 us at the copy rate); 4 requests x 8
// drafts over 131072 positions of 4 heads, 64 rows a head, bf16: 224 us (45).  Bound by the roles'
// own instructions: a tile of 128 positions takes about 2400 cycles, in which the
// ALU pipes are busy for 1100, the values' decoding, the issue of products and the
// softmax each for most of it.
#include <cfloat>
#include <cmath>
#include <numeric>
#include <type_traits>

#include "gbtopk_int4.cuh"
#include "gbtopk_join.cuh"
#include "gbtopk_tma.cuh"

namespace gbtopk {
namespace {

constexpr int kTile = 128;          // positions a tile
constexpr int kThreads4 = 640;
constexpr int kMaxStages = 12;
constexpr int kMasks = 16;          // tiles whose validity bits are kept: the ring's and the two that are decoded
constexpr float kRise = 8.f;        // rise of a score over its row's reference (base 2) that moves it
constexpr float kFar = FLT_MAX;     // a score's distance from a reference that is not there: above kRise for every number
constexpr int kKeyWarp = 4, kValueWarp = 8, kCopyWarp = 12, kCopyWarps = 7, kIssueWarp = 19;
static_assert(kMaxStages <= 2 * kCopyWarps, "two stages a copy warp at most");

struct Int4Params {
    CUtensorMap rows;               // the cache: a line of `row` bytes every pitch
    AttnParams a;                   // k_slot, k_head: strides in pitches
    int32_t codes, row, four;       // bytes of a row's codes, of a row, of four rows in shared memory
    int32_t gang, units;            // blocks side by side; units of a request
    int32_t stages, q_bufs;
    uint32_t q_off, p_off, ring_off, stage_bytes, shared_off;   // shared memory
    float k_mul, v_mul;             // c and the values' unit, times 2^15
};

struct Shared4 {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t q_full[2], q_empty[2];
    uint64_t key_full[2], s_full[2], p_full[2], v_full[2], v_free[2], pv_done[2];
    uint64_t drain;
    uint32_t mask[kMasks][4];       // positions of a tile with a slot: bit b of word w is position 4 b + w
    uint64_t tree[64];              // tree masks of the unit's rows
    int64_t row_at[64];             // (row, head) of the output, -1: none
    float4 less_m[16];              // rows' references, negated; kFar: none yet
    float4 scale[16];               // factors of a move, of the output
    float part[4][64];              // a warp's maxima or sums
    ScanScratch scan;
    uint32_t tmem;
    uint32_t abort;
};

__device__ __forceinline__ void tmem_load8(uint32_t addr, uint32_t *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(addr)
                 : "memory");
}

// A wait of the whole warp.  (A try sleeps for longer than most waits take: a look at
// the clock behind each costs nothing, 64 x 4 drafts 132.4 us, behind 256 of them 134.9.)
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const Waits &w) { return __all_sync(~0u, bar_wait(bar, parity, w)); }

// Barrier of the softmax warps.
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool v) {
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(v))
        : "memory");
    return any != 0;
}

// A number as an integer of the same order (a NaN as the least), and back.
__device__ __forceinline__ int32_t order_of(float x) {
    const int32_t b = __float_as_int(x);
    return x == x ? b ^ ((b >> 31) & 0x7fffffff) : INT32_MIN;
}
__device__ __forceinline__ float of_order(int32_t b) {
    return b == INT32_MIN ? -INFINITY : __int_as_float(b ^ ((b >> 31) & 0x7fffffff));
}

// 32 elements (two blocks, their scales the bytes of `two`) times 2^-15, as bf16.
__device__ __forceinline__ void decode32(const uint4 &c, uint32_t two, uint32_t *out) {
    const uint32_t s = int4_scales2(__byte_perm(two, 0, 0x4140)), s0 = __byte_perm(s, 0, 0x1010), s1 = __byte_perm(s, 0, 0x3232);
    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        out[4 * w] = mul_bf16x2(int4_pair<0>(word[w]), w < 2 ? s0 : s1);
        out[4 * w + 1] = mul_bf16x2(int4_pair<1>(word[w]), w < 2 ? s0 : s1);
        out[4 * w + 2] = mul_bf16x2(int4_pair<2>(word[w]), w < 2 ? s0 : s1);
        out[4 * w + 3] = mul_bf16x2(int4_pair<3>(word[w]), w < 2 ? s0 : s1);
    }
}

__device__ __forceinline__ void put16(uint32_t addr, const uint32_t *v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Columns of a product: R rows, two each with fp16; 16 at least.
template <bool F16, int R>
constexpr int kCols = F16 ? 2 * R : R < 16 ? 16 : R;

// R: query rows of a unit.  WIDE: head dimensions above 128.
template <bool F16, int R, bool WIDE>
__global__ void __launch_bounds__(kThreads4, 1) attention_int4_kernel(const __grid_constant__ Int4Params pp) {
    const AttnParams &p = pp.a;
    constexpr int N = kCols<F16, R>;
    constexpr int CH = R < 16 ? 8 : 16;             // rows at a time
    constexpr int kBlocks = WIDE ? 2 : 1;           // blocks of 128 of the head dimension
    constexpr uint32_t kKeyCols = WIDE ? 128 : 64;  // tensor memory columns of a tile's keys
    constexpr uint32_t kS = 0, kK = 2 * N, kO = kK + 2 * kKeyCols;
    constexpr uint32_t kValueBytes = kTile * 256, kProbBytes = kTile * 128;
    static_assert(kO + kBlocks * N <= 512 && N <= 64, "tensor memory, one panel of probabilities");
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Shared4 &sh = *reinterpret_cast<Shared4 *>(smem + pp.shared_off);
    float *less_m = reinterpret_cast<float *>(sh.less_m), *scale = reinterpret_cast<float *>(sh.scale);
    const uint32_t base = smem_addr(smem), v_smem = base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < pp.stages; ++i) {
            bar_init(&sh.full[i], 1);
            bar_init(&sh.empty[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.q_full[i], kCopyWarps);
            bar_init(&sh.q_empty[i], 1);
            bar_init(&sh.key_full[i], 4);
            bar_init(&sh.s_full[i], 1);
            bar_init(&sh.p_full[i], 4);
            bar_init(&sh.v_full[i], 4);
            bar_init(&sh.v_free[i], 1);
            bar_init(&sh.pv_done[i], 1);
        }
        bar_init(&sh.drain, 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssueWarp) tmem_alloc(&sh.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_release();

    const int gang = static_cast<int>(blockIdx.x) / pp.gang, member = static_cast<int>(blockIdx.x) - gang * pp.gang;
    const int gangs = static_cast<int>(gridDim.x) / pp.gang;
    const int block = member * gangs + gang;       // the blocks of a unit one behind another
    const Share share = block_share<kTile, kThreads4>(p, &sh.scan, gang, gangs);
    const Waits abort{&sh.abort, p.wait_cycles};
    const uint32_t tmem = sh.tmem;
    Walk<kTile> walk(p, share);
    const int32_t rows = p.next_n * p.group;   // of a (request, kv head)
    bool ok = true;

    // The softmax warps hold a sum and a score a row: 160 registers a thread for
    // them (184 with 64 rows) and 80 (72) for the other four warpgroups are 480
    // (472) of the launch's 480.
    if (warp < kKeyWarp) {
        if constexpr (R > 32) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    } else {
        if constexpr (R > 32) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    }

    if (warp < kKeyWarp) {
        // ------------------------------------------------ softmax, output
        const int at = warp * 32 + lane;                               // position of the tile, and lane of O
        const uint32_t lanes = static_cast<uint32_t>(warp) << 21;      // the warp's tensor memory lanes
        uint32_t job = 0;
        float l[R];
        for (; walk.more() && ok; walk.next()) {
            Unit u = walk.u;
            u.hm = u.hm * pp.gang + member;
            const int32_t h = u.hm / p.row_tiles, r0 = (u.hm - h * p.row_tiles) * R;
            const int32_t here = rows - r0 < R ? rows - r0 : R;
            if (at < R) {
                const int32_t t = (r0 + at) / p.group, gq = r0 + at - t * p.group;
                const int64_t r = static_cast<int64_t>(u.b) * p.next_n + t;
                sh.row_at[at] = at < here ? r * p.q_heads + h * p.group + gq : -1;
                sh.tree[at] = at >= here || !p.seq_lens ? 0 : p.tree_mask ? static_cast<uint64_t>(fetch(p.tree_mask + r)) : ~0ull >> (63 - t);
                less_m[at] = at < here ? kFar : 0.f;
            }
            if (at == 0) {   // the blocks that share the unit
                int32_t *ends = p.unit_ends + 2 * (static_cast<int64_t>(u.b) * pp.units + u.hm);
                if (u.t0 == 0) ends[0] = block;
                if (u.t1 == u.tiles) ends[1] = block;
            }
            softmax_sync();
            if (u.span.n == 0) {   // nothing to see
                for (int32_t r = 0; r < here; ++r)
                    for (int32_t d = at; d < p.dim; d += 128) static_cast<uint16_t *>(p.out)[sh.row_at[r] * p.dim + d] = 0;
                if (p.lse && at < here) p.lse[sh.row_at[at]] = -INFINITY;
                softmax_sync();
                continue;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) l[r] = 0.f;
            const uint32_t job0 = job;
            for (int32_t i = u.t0; i < u.t1; ++i, ++job) {
                const uint32_t sb = job & 1, ph = (job >> 1) & 1;
                ok = wait(&sh.s_full[sb], ph, abort);
                tc_fence_after();
                const uint32_t t_s = tmem + lanes + kS + sb * N;
                const bool is = (reinterpret_cast<volatile uint32_t *>(sh.mask[job % kMasks])[at & 3] >> (at >> 2)) & 1;
                using Rows = std::conditional_t<(R > 32), uint64_t, uint32_t>;
                constexpr Rows kEvery = ~static_cast<Rows>(0);
                Rows sees = is ? kEvery : 0;     // rows that see the thread's position
                if (i * kTile > u.span.ctx - kTile) {
                    const int32_t draft = i * kTile + at - u.span.ctx;
                    if (is && draft >= 0) {
                        sees = 0;
#pragma unroll 1
                        for (int r = 0; r < here; ++r) sees |= static_cast<Rows>(draft < 64 ? (sh.tree[r] >> draft) & 1 : 0) << r;
                    }
                }
                const bool all = __all_sync(~0u, sees == kEvery);
                // Scores of the thread's position less their rows' references, base 2.  The
                // product is rounded before the difference, as the reference was: fused, the
                // difference of the largest would be what its rounding left off, up to 2^-24 of
                // it, and a power beyond 32 bits from 2^31 on.  (Sums one at a time: a packed
                // product and a packed sum do get fused.  64 x 4 drafts 134 -> 135 us, 64 rows a
                // head over 131072 positions 224 -> 226.)
                float d[R];
                auto scores = [&]() {
#pragma unroll
                    for (int c = 0; c < R; c += CH) {
                        if (c >= here) break;
                        uint32_t x[16], y[16];
                        if constexpr (!F16 && CH == 8) tmem_load8(t_s, x);
                        else tmem_load16(t_s + c, x);      // (eight rows of fp16: both halves)
                        if constexpr (F16 && CH == 16) tmem_load16(t_s + R + c, y);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < CH; k += 4) {
                            const float4 m = sh.less_m[(c + k) / 4];
                            const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                            for (int j = 0; j < 4; j += 2) {
                                float2 v = make_float2(__uint_as_float(x[k + j]), __uint_as_float(x[k + j + 1]));
                                if constexpr (F16 && CH == 8) add2(v, __uint_as_float(x[(k + j + 8) & 15]), __uint_as_float(x[(k + j + 9) & 15]));
                                if constexpr (F16 && CH == 16) add2(v, __uint_as_float(y[k + j]), __uint_as_float(y[k + j + 1]));
                                v = mul2(v.x, v.y, pp.k_mul);
                                v = make_float2(__fadd_rn(v.x, mm[j]), __fadd_rn(v.y, mm[j + 1]));
                                d[c + k + j] = v.x;
                                d[c + k + j + 1] = v.y;
                            }
                        }
                        if (!all) {
#pragma unroll
                            for (int k = 0; k < CH; ++k)
                                if (!((sees >> (c + k)) & 1)) d[c + k] = -INFINITY;
                        }
                    }
                };
                scores();
                float over = -INFINITY;
#pragma unroll
                for (int c = 0; c < R; c += CH) {
                    if (c >= here) break;
#pragma unroll
                    for (int k = 0; k < CH; ++k) over = fmaxf(over, d[c + k]);   // (a NaN is no maximum)
                }
                if (softmax_any(over > kRise || !ok)) {
                    // ---- some row's reference moves, or a wait ran out
                    if (*reinterpret_cast<volatile uint32_t *>(&sh.abort)) ok = false;
                    // O is complete up to the last job
                    if (ok && job != job0) ok = wait(&sh.pv_done[(job - 1) & 1], ((job - 1) >> 1) & 1, abort);
                    if (softmax_any(!ok)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // (the new reference is a score itself, no sum of differences)
                    const float before = at < R ? less_m[at] : 0.f;
                    if (at < R) less_m[at] = 0.f;
                    softmax_sync();
                    scores();
#pragma unroll
                    for (int c = 0; c < R; c += CH) {
                        if (c >= here) break;
#pragma unroll
                        for (int k = 0; k < CH; ++k) {
                            const float best = of_order(__reduce_max_sync(~0u, order_of(d[c + k])));
                            if (lane == 0) sh.part[warp][c + k] = best;
                        }
                    }
                    softmax_sync();
                    if (at < R) {
                        float f = 1.f, now = before;
                        if (at < here) {
                            const float best = fmaxf(fmaxf(sh.part[0][at], sh.part[1][at]), fmaxf(sh.part[2][at], sh.part[3][at]));
                            if (best + before > kRise) {
                                now = -best;
                                if (before != kFar) f = exp2_fast(now - before);
                            }
                        }
                        less_m[at] = now;
                        scale[at] = f;
                    }
                    softmax_sync();
#pragma unroll
                    for (int r = 0; r < R; ++r) l[r] *= scale[r];
                    if (job != job0) {
#pragma unroll 1
                        for (int c = 0; c < kBlocks * N; c += 16) {
                            uint32_t o[16];
                            tmem_load16(tmem + lanes + kO + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * scale[(c + k) % R]);
                            tmem_store16(tmem + lanes + kO + c, o);
                        }
                        tc_wait_st();
                    }
                    scores();
                }
                // P^T of the tile before last has been read
                if (job >= 2) ok = wait(&sh.pv_done[sb], ph ^ 1, abort);
                const uint32_t p_row = base + pp.p_off + sb * kProbBytes + at * 128, swizzle = (at & 7) << 4;
#pragma unroll
                for (int c = 0; c < R; c += 8) {
                    if (c >= here) break;
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float a = exp2_fast(d[c + k]), b = exp2_fast(d[c + k + 1]);
                        l[c + k] += a;
                        l[c + k + 1] += b;
                        hi[k / 2] = Half2<true>::down(a, b);
                        if constexpr (F16) {
                            const float2 f = Half2<true>::up(hi[k / 2]);
                            lo[k / 2] = Half2<true>::down(a - f.x, b - f.y);
                        }
                    }
                    put16(p_row + ((c * 2) ^ swizzle), hi);
                    if constexpr (F16) put16(p_row + (((R + c) * 2) ^ swizzle), lo);
                }
                fence_async_reads();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.p_full[sb]);
            }
            if (ok) ok = wait(&sh.pv_done[(job - 1) & 1], ((job - 1) >> 1) & 1, abort);
            if (softmax_any(!ok)) {
                ok = false;
                break;
            }
            // ---- the unit's output: sums over the positions, then a thread a dimension
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float s = l[r];
                for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
                if (lane == 0) sh.part[warp][r] = s;
            }
            softmax_sync();
            const bool whole = u.t0 == 0 && u.t1 == u.tiles;
            const int64_t part = 2ll * block + (u.t0 > 0 ? 0 : 1);
            if (at < R) {
                const float s = (sh.part[0][at] + sh.part[1][at]) + (sh.part[2][at] + sh.part[3][at]);
                const float m = less_m[at] == kFar ? -INFINITY : -less_m[at];
                scale[at] = whole ? (s == 0.f ? 0.f : pp.v_mul / s) : pp.v_mul;
                if (at < here) {
                    if (!whole) p.part_ml[part * R + at] = make_float2(m, s);
                    else if (p.lse) p.lse[sh.row_at[at]] = row_lse<true>(m, s);
                }
            }
            softmax_sync();
            tc_fence_after();
            const int dp = WIDE ? 256 : p.dim <= 64 ? 64 : 128;
#pragma unroll 1
            for (int b = 0; b < kBlocks; ++b) {
                const int d = b * 128 + at;
#pragma unroll 1
                for (int c = 0; c < here; c += 8) {
                    uint32_t o[8], y[8];
                    float x[8];
                    tmem_load8(tmem + lanes + kO + b * N + c, o);
                    if constexpr (F16) tmem_load8(tmem + lanes + kO + b * N + R + c, y);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = (__uint_as_float(o[k]) + (F16 ? __uint_as_float(y[k]) : 0.f)) * scale[c + k];
                    if (whole) {
                        if (d < p.dim) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (c + k < here)
                                    static_cast<uint16_t *>(p.out)[sh.row_at[c + k] * p.dim + d] = static_cast<uint16_t>(Half2<!F16>::down(x[k], 0.f));
                        }
                    } else if (d < dp) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + (part * dp + d) * R + c);
                        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            softmax_sync();   // (the next unit writes what this one's output reads)
        }
    } else if (warp < kValueWarp) {
        // ------------------------------------------------ keys to tensor memory
        const int w = warp - kKeyWarp, at = w * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(w) << 21;
        uint32_t job = 0, stage = 0, lap = 0;
        for (; walk.more() && ok; walk.next()) {
            if (walk.u.span.n == 0) continue;
            for (int32_t i = walk.u.t0; i < walk.u.t1; ++i, ++job) {
                // (the tile before last has been multiplied)
                ok = wait(&sh.full[stage], lap & 1, abort) && (job < 2 || wait(&sh.s_full[job & 1], ((job >> 1) & 1) ^ 1, abort));
                if (!ok) break;
                tc_fence_after();
                const uint8_t *row = smem + pp.ring_off + stage * pp.stage_bytes + (at >> 2) * pp.four + (at & 3) * pp.row;
                const uint32_t dst = tmem + lanes + kK + (job & 1) * kKeyCols;
                // (the next codes are loaded before the store, which holds later loads back)
                const uint8_t *scales = row + 2 * pp.codes;
                uint4 c = *reinterpret_cast<const uint4 *>(row);
                uint32_t two = *reinterpret_cast<const uint16_t *>(scales);
#pragma unroll 1
                for (int b = 0; b * 32 < p.dim; ++b) {
                    uint32_t y[16];
                    decode32(c, two, y);
                    c = *reinterpret_cast<const uint4 *>(row + b * 16 + 16);   // (behind the last: the row's other bytes)
                    two = *reinterpret_cast<const uint16_t *>(scales + b * 2 + 2);
                    tmem_store16(dst + b * 16, y);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&sh.key_full[job & 1]);
                    bar_arrive(&sh.empty[stage]);
                }
                if (++stage == static_cast<uint32_t>(pp.stages)) {
                    stage = 0;
                    ++lap;
                }
            }
        }
    } else if (warp < kCopyWarp) {
        // ------------------------------------------------ values to shared memory
        const int at = (warp - kValueWarp) * 32 + lane;
        uint32_t item = 0, stage = 0, lap = 0;
        for (; walk.more() && ok; walk.next()) {
            if (walk.u.span.n == 0) continue;
            for (int32_t i = walk.u.t0; i < walk.u.t1; ++i) {
                ok = wait(&sh.full[stage], lap & 1, abort);
                if (!ok) break;
                const uint8_t *row = smem + pp.ring_off + stage * pp.stage_bytes + (at >> 2) * pp.four + (at & 3) * pp.row;
                const uint8_t *scales = row + 2 * pp.codes + (WIDE ? 16 : 8);
                row += pp.codes;
                uint4 c = *reinterpret_cast<const uint4 *>(row);
                uint32_t two = *reinterpret_cast<const uint16_t *>(scales);
                for (int b = 0; b * 32 < p.dim; ++item) {   // items of 128 dimensions
                    if (item >= 2) ok = wait(&sh.v_free[item & 1], ((item >> 1) & 1) ^ 1, abort);
                    if (!ok) break;
                    uint32_t to = v_smem + (item & 1) * kValueBytes + at * 128, turn = (at & 7) << 4;
                    const int end = b + 4;
#pragma unroll 1
                    for (; b < end && b * 32 < p.dim; ++b) {
                        uint32_t y[16];
                        decode32(c, two, y);
                        c = *reinterpret_cast<const uint4 *>(row + b * 16 + 16);   // (behind the last: the row's scales)
                        two = *reinterpret_cast<const uint16_t *>(scales + b * 2 + 2);
#pragma unroll
                        for (int k = 0; k < 4; ++k) put16(to + (turn ^ (k * 16)), y + 4 * k);
                        turn ^= 64;
                        to += b & 1 ? kTile * 128 : 0;
                    }
                    fence_async_reads();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&sh.v_full[item & 1]);
                }
                if (!ok) break;
                if (lane == 0) bar_arrive(&sh.empty[stage]);
                if (++stage == static_cast<uint32_t>(pp.stages)) {
                    stage = 0;
                    ++lap;
                }
            }
        }
    } else if (warp != kIssueWarp) {
        // ------------------------------------------------ slots and copies, the warps in turn; queries
        // A stage is one warp's, so that the parities that a warp waits for, of its
        // stage emptied and in the end of its last copy there, are never two phases
        // behind.
        const uint32_t turn = warp - kCopyWarp, turns = pp.stages < kCopyWarps ? pp.stages : kCopyWarps;
        int32_t last_b = -1;
        uint64_t seen = ~0ull;   // drafted tokens that some row of the request sees
        uint32_t stage = 0, lap = 0, tile = 0, unit = 0, flying = 0, odd_lap = 0;   // stages that the warp has copied to, their parity
        for (; walk.more() && ok; walk.next()) {
            Unit u = walk.u;
            u.hm = u.hm * pp.gang + member;
            if (u.span.n == 0) continue;
            if (u.b != last_b && p.seq_lens && p.tree_mask) {
                const int64_t *tm = p.tree_mask + static_cast<int64_t>(u.b) * p.next_n;
                uint64_t m = lane < p.next_n ? static_cast<uint64_t>(fetch(tm + lane)) : 0;
                if (lane + 32 < p.next_n) m |= static_cast<uint64_t>(fetch(tm + lane + 32));
                seen = static_cast<uint64_t>(__reduce_or_sync(~0u, static_cast<uint32_t>(m >> 32))) << 32 |
                       __reduce_or_sync(~0u, static_cast<uint32_t>(m));
            }
            last_b = u.b;
            const int64_t head = (u.hm / p.row_tiles) * p.k_head;
            // some tiles before the unit's queries, so that copies start (no more than
            // there are stages: theirs are the last unit's, whose queries are there)
            const int32_t q_at = u.t1 - u.t0 < static_cast<int32_t>(turns) ? u.t1 : u.t0 + static_cast<int32_t>(turns);
            for (int32_t t = u.t0; ok; ++t) {
                if (t == q_at) {
                    const int32_t h = u.hm / p.row_tiles, r0 = (u.hm - h * p.row_tiles) * R;
                    const int32_t here = rows - r0 < R ? rows - r0 : R, padded = (here + CH - 1) / CH * CH, lanes8 = p.dim / 8;
                    const uint32_t qb = pp.q_bufs == 2 ? unit & 1 : 0, qph = pp.q_bufs == 2 ? unit >> 1 : unit;
                    if (qph > 0) ok = wait(&sh.q_empty[qb], (qph - 1) & 1, abort);
                    if (!ok) break;
                    const uint32_t q_tile = base + pp.q_off + qb * (N * (WIDE ? 512 : 256));
#pragma unroll 2
                    for (int32_t k = turn * 32 + lane; k < padded * lanes8; k += kCopyWarps * 32) {
                        const int32_t r = k / lanes8, c = k - r * lanes8, tok = (r0 + r) / p.group, gq = r0 + r - tok * p.group;
                        const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                                             2 * ((static_cast<int64_t>(u.b) * p.next_n + tok) * p.q_row + (h * p.group + gq) * p.q_head);
                        const uint4 v = r < here ? fetch(reinterpret_cast<const uint4 *>(src) + c) : make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                        if constexpr (F16) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 f = Half2<false>::up(x[j]);
                                hi[j] = Half2<true>::down(f.x, f.y);
                                const float2 g = Half2<true>::up(hi[j]);
                                // (an infinity is whole)
                                lo[j] = Half2<true>::down(isinf(f.x) ? 0.f : f.x - g.x, isinf(f.y) ? 0.f : f.y - g.y);
                            }
                            put16(q_tile + tile_offset(N, r, c), hi);
                            put16(q_tile + tile_offset(N, R + r, c), lo);
                        } else {
                            put16(q_tile + tile_offset(N, r, c), x);
                        }
                    }
                    fence_async_reads();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&sh.q_full[qb]);
                    ++unit;
                }
                if (t >= u.t1) break;
                const uint32_t n = tile++;
                if (stage == turn || stage == turn + turns) {   // (fewer stages than twice the warps)
                    Paging::Place place[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int32_t pos = t * kTile + lane * 4 + k;
                        const bool is = pos < u.span.n && (pos < u.span.ctx || ((seen >> (pos - u.span.ctx)) & 1));
                        place[k] = p.seq_lens ? p.pages.place(u.b, pos, is) : p.pages.listed(p.indices + u.b * p.idx_row + pos, is);
                    }
                    if (lap > 0) ok = wait(&sh.empty[stage], (lap - 1) & 1, abort);
                    if (!ok) break;
                    int32_t row[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t slot = p.pages.slot(place[k]);
                        const uint32_t bits = __ballot_sync(~0u, slot >= 0);
                        if (lane == 0) sh.mask[n % kMasks][k] = bits;
                        // (a position without a slot gets the first one's row: its probability is 0)
                        row[k] = static_cast<int32_t>((slot < 0 ? 0 : slot) * p.k_slot + head);
                    }
                    if (lane == 0) bar_expect(&sh.full[stage], kTile * pp.row);
                    __syncwarp();
                    gather_rows4(base + pp.ring_off + stage * pp.stage_bytes + lane * pp.four, &pp.rows, make_int4(row[0], row[1], row[2], row[3]),
                                 &sh.full[stage]);
                    flying |= 1u << stage;
                    if (lap & 1) odd_lap |= 1u << stage;
                    else odd_lap &= ~(1u << stage);
                }
                if (++stage == static_cast<uint32_t>(pp.stages)) {
                    stage = 0;
                    ++lap;
                }
            }
        }
        // the block does not end before its copies have
        const long long t0 = clock64();
        for (int i = 0; i < pp.stages; ++i)
            while (((flying >> i) & 1) && !bar_try(&sh.full[i], (odd_lap >> i) & 1) && clock64() - t0 < kWaitCycles) {
            }
    } else {
        // ------------------------------------------------ matrix products (all lanes alike, see elect_lane)
        const bool lead = elect_lane();
        const uint32_t s_desc = mma_desc(true, 128, N, false, p.negative != 0);
        const uint32_t o_desc = mma_desc(true, 128, N, true, false) | 1u << 15;   // A transposed too
        const int ksteps = p.dim / 16;
        const uint32_t q_bytes = N * (WIDE ? 512 : 256);
        // (broadcasts: values known to be warp-uniform)
        const uint32_t t_issue = __shfl_sync(~0u, tmem, 0), base_u = __shfl_sync(~0u, base, 0);
        uint32_t unit = 0, job0 = 0, item = 0;
        for (; __any_sync(~0u, walk.more()) && ok; walk.next()) {
            if (__any_sync(~0u, walk.u.span.n == 0)) continue;
            const uint32_t jobs = __shfl_sync(~0u, static_cast<uint32_t>(walk.u.t1 - walk.u.t0), 0);
            const uint32_t qb = pp.q_bufs == 2 ? unit & 1 : 0, qph = pp.q_bufs == 2 ? unit >> 1 : unit;
            ok = wait(&sh.q_full[qb], qph & 1, abort);
            // scores run two jobs ahead of outputs
            for (uint32_t ahead = 0; ahead < jobs + 2 && ok; ++ahead) {
                if (ahead >= 2) {
                    const uint32_t j = ahead - 2, job = job0 + j, sb = job & 1;
#pragma unroll 1
                    for (int mb = 0; mb < kBlocks; ++mb, ++item) {
                        ok = wait(&sh.v_full[item & 1], (item >> 1) & 1, abort) && wait(&sh.p_full[sb], (job >> 1) & 1, abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t va = smem_desc(base_u + (item & 1) * kValueBytes, kTile * 128, 1024);
                        const uint64_t pa = smem_desc(base_u + pp.p_off + sb * kProbBytes, kTile * 128, 1024);
#pragma unroll 2
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma_ss_if(lead, t_issue + kO + mb * N, va + kk * 128, pa + kk * 128, o_desc, j > 0 || kk > 0);
                        if (lead) {
                            tc_commit(&sh.v_free[item & 1]);
                            if (mb + 1 == kBlocks) tc_commit(&sh.pv_done[sb]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                if (ahead < jobs) {
                    const uint32_t job = job0 + ahead, sb = job & 1;
                    ok = wait(&sh.key_full[sb], (job >> 1) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t qa = smem_desc(base_u + pp.q_off + qb * q_bytes, 16, 1024);
                    const uint32_t ka = t_issue + kK + sb * kKeyCols;
#pragma unroll 2
                    for (int kk = 0; kk < ksteps; ++kk)
                        mma_ts_if(lead, t_issue + kS + sb * N, ka + kk * 8, qa + (kk >> 2) * (N * 8) + (kk & 3) * 2, s_desc, kk > 0);
                    if (lead) {
                        tc_commit(&sh.s_full[sb]);
                        if (ahead + 1 == jobs) tc_commit(&sh.q_empty[qb]);
                    }
                    __syncwarp();
                }
            }
            job0 += jobs;
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
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssueWarp) tmem_free(tmem, 512);
    if (threadIdx.x == 0 && sh.abort) atomicOr(p.status, kStatusCopyLost);
}

template <bool F16, int R, bool WIDE>
cudaError_t launch_rows(Int4Params pp, uint8_t *ws, int sms, cudaStream_t stream) {
    AttnParams &p = pp.a;
    const int64_t rows = static_cast<int64_t>(p.next_n) * p.group;
    p.row_tiles = static_cast<int32_t>((rows + R - 1) / R);
    const int grid = sms < kMaxGrid ? sms : kMaxGrid;
    // a gang: as many units as divide a request's and leave at most 7 blocks over
    // (64 requests, 8 heads: 135 us, by single blocks 145 and 516 MB for 300)
    pp.units = p.kv_heads * p.row_tiles;
    for (pp.gang = pp.units < 8 ? pp.units : 8; pp.units % pp.gang != 0 || pp.gang > grid; --pp.gang) {
    }
    p.request_units = pp.units / pp.gang;
    place_parts(p, ws);
    pp.codes = int4_codes(p.dim);
    pp.row = int4_row(p.dim);
    pp.four = (4 * pp.row + 127) / 128 * 128;
    // values (two tiles of 128 x 128), probabilities, queries, the ring
    constexpr uint32_t kQ = kCols<F16, R> * (WIDE ? 512 : 256);
    constexpr uint32_t most = kMaxSmemBytes - 1024 - (sizeof(Shared4) + 15) / 16 * 16;
    pp.p_off = 2 * kTile * 256;
    pp.q_off = pp.p_off + 2 * kTile * 128;
    pp.q_bufs = kQ > 16384 ? 1 : 2;
    pp.ring_off = pp.q_off + pp.q_bufs * kQ;
    pp.stage_bytes = kTile / 4 * pp.four;
    const uint32_t fit = (most - pp.ring_off) / pp.stage_bytes;
    pp.stages = static_cast<int32_t>(fit < kMaxStages ? fit : kMaxStages);
    if (pp.stages < 1) return cudaErrorInvalidValue;
    pp.shared_off = pp.ring_off + pp.stages * pp.stage_bytes;
    const size_t bytes = 1024 + pp.shared_off + sizeof(Shared4);
    static std::atomic<uint64_t> allowed;
    auto kernel = attention_int4_kernel<F16, R, WIDE>;
    cudaError_t e = allow_smem(kernel, kMaxSmemBytes, allowed);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid / pp.gang * pp.gang)), kThreads4, bytes, stream, 1, pp);
    if (e != cudaSuccess) return e;
    p.request_units = pp.units;
    if constexpr (WIDE) return launch_join<!F16, 256>(p, R, kTile, sms, stream);
    else return p.dim <= 64 ? launch_join<!F16, 64>(p, R, kTile, sms, stream) : launch_join<!F16, 128>(p, R, kTile, sms, stream);
}

// By the rows of a head: 8, 16, 32, and 64 where they are a column each and one
// block of the head dimension.  Fewer rows are less work a tile (one request of
// 4 rows a head: 22.4 us a call, as 16 rows 23.3; 16 rows 30.6 us, as 32 36.7);
// more rows are more units, each of which decodes the cache (4 requests x 8 drafts
// over 131072 positions, 64 rows a head: 223 us, by two units of 32 263).
template <bool F16>
cudaError_t launch_int4(const Int4Params &pp, uint8_t *ws, int sms, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(pp.a.next_n) * pp.a.group;
    if (pp.a.dim > 128) return rows <= 16 ? launch_rows<F16, 16, true>(pp, ws, sms, s) : launch_rows<F16, 32, true>(pp, ws, sms, s);
    if (rows <= 8) return launch_rows<F16, 8, false>(pp, ws, sms, s);
    if (rows <= 16) return launch_rows<F16, 16, false>(pp, ws, sms, s);
    if constexpr (!F16)
        if (rows > 32) return launch_rows<F16, 64, false>(pp, ws, sms, s);
    return launch_rows<F16, 32, false>(pp, ws, sms, s);
}

int attend_int4(Int4Params &pp, int dtype, const void *q, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *cache, int64_t slot_stride, int64_t head_stride,
                float k_scale, float v_scale, float scale, void *out, float *lse, void *workspace, size_t workspace_bytes,
                void *stream) {
    AttnParams &p = pp.a;
    int rc;
    if ((rc = check_rows(q, q_row_stride, q_head_stride, true)) != GBTOPK_OK) return rc;
    if ((rc = check_int4(cache, slot_stride, head_stride, p.pages.num_slots, head_dim)) != GBTOPK_OK) return rc;
    if (!int4_unit(k_scale) || !int4_unit(v_scale)) return GBTOPK_EINVAL;
    // what a product of queries and keys' codes is multiplied by; a scale of 0 stays a product that ignores no mask
    pp.k_mul = fmaxf(fabsf(scale) * (kLog2e * k_scale * kInt4Lift), FLT_MIN);
    if (pp.k_mul > FLT_MAX) return GBTOPK_EUNSUPPORTED;
    if (!out) return GBTOPK_EINVAL;
    if (!aligned_to(out, 16) || !aligned_to(lse, 4)) return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) ||
        workspace_bytes < gbtopk_attention_workspace_bytes(num_rows, q_heads, kv_heads, head_dim))
        return GBTOPK_EWORKSPACE;
    p.q = q;
    p.q_row = q_row_stride;
    p.q_head = q_head_stride;
    // A map of lines at one pitch that holds every row: the strides' greatest
    // common divisor (an empty cache: one line of the workspace, never read as a row).
    const int64_t slots = p.pages.num_slots, row = int4_row(head_dim);
    const int64_t heads_at = kv_heads > 1 ? head_stride : 0, slots_at = slots > 1 ? slot_stride : 0;
    int64_t pitch = std::gcd(heads_at, slots_at);
    if (pitch == 0) pitch = row;
    if (pitch < row) return GBTOPK_EUNSUPPORTED;
    const int64_t lines = slots > 0 ? ((slots - 1) * slots_at + (kv_heads - 1) * heads_at) / pitch + 1 : 1;
    if (lines > INT32_MAX || pitch >= 1ll << 40) return GBTOPK_EUNSUPPORTED;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row / 2), static_cast<cuuint64_t>(lines)}, strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(row / 2), 1};
    if (!tensor_map(&pp.rows, slots > 0 ? cache : workspace, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE)) return GBTOPK_ECUDA;
    p.k_slot = slots_at / pitch;
    p.k_head = slots > 0 ? heads_at / pitch : 0;
    p.requests = static_cast<int32_t>(num_rows / p.next_n);
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.dim = head_dim;
    pp.v_mul = v_scale * kInt4Lift;
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
    return (dtype == GBTOPK_F16 ? launch_int4<true>(pp, ws, sms, s) : launch_int4<false>(pp, ws, sms, s)) == cudaSuccess
               ? GBTOPK_OK
               : GBTOPK_ECUDA;
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" {

int gbtopk_tree_attention_int4(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                               int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *cache, int64_t slot_stride,
                               int64_t head_stride, int64_t num_slots, float k_scale, float v_scale, const int32_t *page_table,
                               int64_t pt_cols, int64_t pt_row_stride, int32_t page_size, const int32_t *seq_lens, int32_t next_n,
                               const int64_t *tree_mask, float scale, void *out, float *lse, void *workspace,
                               size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (next_n < 1 || num_rows % next_n != 0) return GBTOPK_EINVAL;
    if (next_n > GBTOPK_MAX_NEXT_N || head_dim % 16 != 0) return GBTOPK_EUNSUPPORTED;
    Int4Params pp{};
    AttnParams &p = pp.a;
    if ((rc = check_pages(page_table, pt_cols, pt_row_stride, page_size, num_slots, num_rows / next_n, &p.pages)) != GBTOPK_OK)
        return rc;
    if (num_rows == 0) return GBTOPK_OK;
    if (!seq_lens) return GBTOPK_EINVAL;
    if (!aligned_to(seq_lens, 4) || !aligned_to(tree_mask, 8)) return GBTOPK_EALIGN;
    p.seq_lens = seq_lens;
    p.next_n = next_n;
    p.tree_mask = tree_mask;
    return attend_int4(pp, dtype, q, num_rows, q_row_stride, q_head_stride, q_heads, kv_heads, head_dim, cache, slot_stride,
                       head_stride, k_scale, v_scale, scale, out, lse, workspace, workspace_bytes, stream);
}

int gbtopk_selected_attention_int4(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride, int64_t q_head_stride,
                                   int32_t q_heads, int32_t kv_heads, int32_t head_dim, const void *cache, int64_t slot_stride,
                                   int64_t head_stride, int64_t num_slots, float k_scale, float v_scale, const int32_t *indices,
                                   int64_t top_k, int64_t idx_row_stride, float scale, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream) {
    int rc = check_heads(dtype, num_rows, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (head_dim % 16 != 0) return GBTOPK_EUNSUPPORTED;
    if (top_k < 0 || num_slots < 0 || (num_rows > 1 && idx_row_stride < top_k)) return GBTOPK_EINVAL;
    if (top_k > INT32_MAX / 2) return GBTOPK_EUNSUPPORTED;
    if (num_rows == 0) return GBTOPK_OK;
    if (top_k > 0 && !indices) return GBTOPK_EINVAL;
    if (!aligned_to(indices, 4)) return GBTOPK_EALIGN;
    Int4Params pp{};
    AttnParams &p = pp.a;
    p.pages.num_slots = num_slots;
    p.pages.page.init(1);
    p.indices = indices;
    p.top_k = static_cast<int32_t>(top_k);
    p.idx_row = idx_row_stride;
    p.next_n = 1;
    return attend_int4(pp, dtype, q, num_rows, q_row_stride, q_head_stride, q_heads, kv_heads, head_dim, cache, slot_stride,
                       head_stride, k_scale, v_scale, scale, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
