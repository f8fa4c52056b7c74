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
// inputs each probability is rounded to bf16 (2^-9 of itself) for its product,
// as the 16-bit kernels' are.  S, m, l and O are 32 bits.
//
// A block, one an SM: four warps of softmax and output, four that turn the codes
// of keys into tensor memory, four that turn those of values into a
// shared-memory tile, four that copy the cached rows (cp.async, 16 bytes a
// lane) into a ring, one that issues products, three that look up slots and
// fetch queries.  Shares, units and the join are those of gbtopk_attention.cu.
#include <cfloat>
#include <cmath>

#include "gbtopk_int4.cuh"
#include "gbtopk_join.cuh"

namespace gbtopk {
namespace {

constexpr int kTile = 128;          // positions a tile
constexpr int kThreads4 = 640;
constexpr int kSlotRing = 8;        // tiles whose slots are looked up ahead
constexpr int kMaxStages = 12;
constexpr float kRise = 8.f;        // rise of a score over its row's reference (base 2) that moves it
constexpr int kKeyWarp = 4, kValueWarp = 8, kCopyWarp = 12, kIssueWarp = 16;

struct Int4Params {
    AttnParams a;                   // k, k_slot, k_head: the rows, strides in bytes
    int32_t codes, row, stride;     // bytes of a row's codes, of a row, of a row in shared memory
    int32_t stages, q_bufs;
    uint32_t q_off, p_off, ring_off, stage_bytes, shared_off;   // shared memory
    float k_mul, v_mul;             // c and the values' unit, times 2^15
};

struct Shared4 {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t slots_full[kSlotRing], slots_empty[kSlotRing];
    uint64_t q_full[2], q_empty[2];
    uint64_t key_full[2], s_full[2], p_full[2], v_full[2], v_free[2], pv_done[2];
    uint64_t drain;
    int32_t slots[kSlotRing][kTile];
    uint64_t tree[64];              // tree masks of the unit's rows
    int64_t row_at[64];             // (row, head) of the output, -1: none
    float m[64], scale[64];         // references; factors of a move, of the output
    float part[4][64];              // a warp's maxima or sums
    ScanScratch scan;
    uint32_t tmem;
    uint32_t abort;
};

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

// The block of sixteen elements whose codes are c0, c1 and whose scale (times
// 2^118, twice) is s, times 2^-15.
__device__ __forceinline__ void decode16(uint32_t c0, uint32_t c1, uint32_t s, uint32_t *out) {
    out[0] = mul_bf16x2(int4_pair<0>(c0), s);
    out[1] = mul_bf16x2(int4_pair<1>(c0), s);
    out[2] = mul_bf16x2(int4_pair<2>(c0), s);
    out[3] = mul_bf16x2(int4_pair<3>(c0), s);
    out[4] = mul_bf16x2(int4_pair<0>(c1), s);
    out[5] = mul_bf16x2(int4_pair<1>(c1), s);
    out[6] = mul_bf16x2(int4_pair<2>(c1), s);
    out[7] = mul_bf16x2(int4_pair<3>(c1), s);
}

// R: query rows of a unit.  WIDE: head dimensions above 128.
template <bool F16, int R, bool WIDE>
__global__ void __launch_bounds__(kThreads4, 1) attention_int4_kernel(const __grid_constant__ Int4Params pp) {
    const AttnParams &p = pp.a;
    constexpr int N = F16 ? 2 * R : R;              // columns of a product
    constexpr int kBlocks = WIDE ? 2 : 1;           // blocks of 128 of the head dimension
    constexpr uint32_t kKeyCols = WIDE ? 128 : 64;  // tensor memory columns of a tile's keys
    constexpr uint32_t kS = 0, kK = 2 * N, kO = kK + 2 * kKeyCols;
    constexpr uint32_t kValueBytes = kTile * 256, kProbBytes = kTile * 128 * (N > 64 ? 2 : 1);
    static_assert(kO + kBlocks * N <= 512, "tensor memory");
    extern __shared__ uint8_t raw[];
    uint8_t *smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Shared4 &sh = *reinterpret_cast<Shared4 *>(smem + pp.shared_off);
    const uint32_t base = smem_addr(smem), v_smem = base;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < pp.stages; ++i) {
            bar_init(&sh.full[i], 128);
            bar_init(&sh.empty[i], 8);
        }
        for (int i = 0; i < kSlotRing; ++i) {
            bar_init(&sh.slots_full[i], 1);
            bar_init(&sh.slots_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&sh.q_full[i], 3);
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

    const Share share = block_share<kTile, kThreads4>(p, &sh.scan);
    const Waits abort{&sh.abort, p.wait_cycles};
    const uint32_t tmem = sh.tmem;
    Walk<kTile> walk(p, share);
    const int32_t rows = p.next_n * p.group;   // of a (request, kv head)
    bool ok = true;

    if (warp < kKeyWarp) {
        // ------------------------------------------------ softmax, output
        const int at = warp * 32 + lane;                               // position of the tile, and lane of O
        const uint32_t lanes = static_cast<uint32_t>(warp) << 21;      // the warp's tensor memory lanes
        uint32_t job = 0;
        float l[R];
        for (; walk.more() && ok; walk.next()) {
            const Unit u = walk.u;
            const int32_t h = u.hm / p.row_tiles, r0 = (u.hm - h * p.row_tiles) * R;
            const int32_t here = rows - r0 < R ? rows - r0 : R;
            if (at < R) {
                const int32_t t = (r0 + at) / p.group, gq = r0 + at - t * p.group;
                const int64_t r = static_cast<int64_t>(u.b) * p.next_n + t;
                sh.row_at[at] = at < here ? r * p.q_heads + h * p.group + gq : -1;
                sh.tree[at] = at >= here || !p.seq_lens ? 0 : p.tree_mask ? static_cast<uint64_t>(fetch(p.tree_mask + r)) : ~0ull >> (63 - t);
                sh.m[at] = -INFINITY;
            }
            if (at == 0) {   // the blocks that share the unit
                int32_t *ends = p.unit_ends + 2 * (static_cast<int64_t>(u.b) * p.request_units + u.hm);
                if (u.t0 == 0) ends[0] = static_cast<int32_t>(blockIdx.x);
                if (u.t1 == u.tiles) ends[1] = static_cast<int32_t>(blockIdx.x);
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
                ok = __all_sync(~0u, bar_wait(&sh.slots_full[job % kSlotRing], (job / kSlotRing) & 1, abort) &&
                                         bar_wait(&sh.s_full[sb], ph, abort));
                // (the warps leave together: they meet at barriers)
                if (softmax_any(!ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t t_s = tmem + lanes + kS + sb * N;
                const bool is = reinterpret_cast<volatile int32_t *>(sh.slots[job % kSlotRing])[at] >= 0;
                const bool drafts = i * kTile > u.span.ctx - kTile;          // the tile has drafted tokens
                const int32_t draft = i * kTile + at - u.span.ctx;
                // 16 rows' scores of the thread's position, base 2
                auto scores = [&](int c, float *t) {
                    uint32_t x[16];
                    tmem_load16(t_s + c, x);
                    if constexpr (F16) {
                        uint32_t y[16];
                        tmem_load16(t_s + R + c, y);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) t[k] = (__uint_as_float(x[k]) + __uint_as_float(y[k])) * pp.k_mul;
                    } else {
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) t[k] = __uint_as_float(x[k]) * pp.k_mul;
                    }
                    if (!is) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) t[k] = -INFINITY;
                    } else if (drafts && draft >= 0) {
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (draft > 63 || !((sh.tree[c + k] >> draft) & 1)) t[k] = -INFINITY;
                    }
                };
                float over = -INFINITY;
#pragma unroll
                for (int c = 0; c < R; c += 16) {
                    if (c >= here) break;
                    float t[16];
                    scores(c, t);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float rise = t[k] - sh.m[c + k];
                        if (c + k < here) over = fmaxf(over, rise);   // (a NaN is no maximum)
                    }
                }
                if (softmax_any(over > kRise)) {
                    // ---- some row's reference moves
#pragma unroll
                    for (int c = 0; c < R; c += 16) {
                        if (c >= here) break;
                        float t[16];
                        scores(c, t);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int32_t best = __reduce_max_sync(~0u, order_of(t[k]));
                            if (lane == 0) sh.part[warp][c + k] = of_order(best);
                        }
                    }
                    softmax_sync();
                    if (at < R) {
                        float f = 1.f;
                        if (at < here) {
                            const float best = fmaxf(fmaxf(sh.part[0][at], sh.part[1][at]), fmaxf(sh.part[2][at], sh.part[3][at]));
                            const float m = sh.m[at];
                            if (best - m > kRise) {
                                f = m == -INFINITY ? 0.f : exp2_fast(m - best);
                                sh.m[at] = best;
                            }
                        }
                        sh.scale[at] = f;
                    }
                    softmax_sync();
#pragma unroll
                    for (int r = 0; r < R; ++r) l[r] *= sh.scale[r];
                    if (job != job0) {
                        // O is complete up to the last job
                        ok = __all_sync(~0u, bar_wait(&sh.pv_done[(job - 1) & 1], ((job - 1) >> 1) & 1, abort));
                        if (softmax_any(!ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < kBlocks * N; c += 16) {
                            uint32_t o[16];
                            tmem_load16(tmem + lanes + kO + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sh.scale[(c + k) % R]);
                            tmem_store16(tmem + lanes + kO + c, o);
                        }
                        tc_wait_st();
                    }
                }
                // P^T of the tile before last has been read
                if (job >= 2) ok = __all_sync(~0u, bar_wait(&sh.pv_done[sb], ph ^ 1, abort));
                const uint32_t p_tile = pp.p_off + sb * kProbBytes;
#pragma unroll
                for (int c = 0; c < R; c += 16) {
                    if (c >= here) break;
                    float t[16];
                    scores(c, t);
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float e[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float m = sh.m[c + k + j];
                            e[j] = exp2_fast(t[k + j] - (m == -INFINITY ? 0.f : m));
                            l[c + k + j] += e[j];
                        }
                        hi[k / 2] = Half2<true>::down(e[0], e[1]);
                        if constexpr (F16) {
                            const float2 f = Half2<true>::up(hi[k / 2]);
                            lo[k / 2] = Half2<true>::down(e[0] - f.x, e[1] - f.y);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        *reinterpret_cast<uint4 *>(smem + p_tile + tile_offset(kTile, at, c / 8 + k)) =
                            make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                        if constexpr (F16)
                            *reinterpret_cast<uint4 *>(smem + p_tile + tile_offset(kTile, at, (R + c) / 8 + k)) =
                                make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                    }
                }
                fence_async_reads();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(&sh.p_full[sb]);
                    bar_arrive(&sh.slots_empty[job % kSlotRing]);
                }
            }
            if (ok && job != job0) ok = __all_sync(~0u, bar_wait(&sh.pv_done[(job - 1) & 1], ((job - 1) >> 1) & 1, abort));
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
            const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (u.t0 > 0 ? 0 : 1);
            if (at < R) {
                const float s = (sh.part[0][at] + sh.part[1][at]) + (sh.part[2][at] + sh.part[3][at]);
                sh.scale[at] = whole ? (s == 0.f ? 0.f : pp.v_mul / s) : pp.v_mul;
                if (at < here) {
                    if (!whole) p.part_ml[part * R + at] = make_float2(sh.m[at], s);
                    else if (p.lse) p.lse[sh.row_at[at]] = row_lse<true>(sh.m[at], s);
                }
            }
            softmax_sync();
            tc_fence_after();
#pragma unroll 1
            for (int b = 0; b < kBlocks; ++b) {
                const int d = b * 128 + at;
#pragma unroll 1
                for (int c = 0; c < here; c += 16) {
                    uint32_t o[16];
                    float x[16];
                    tmem_load16(tmem + lanes + kO + b * N + c, o);
                    if constexpr (F16) {
                        uint32_t y[16];
                        tmem_load16(tmem + lanes + kO + b * N + R + c, y);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] = (__uint_as_float(o[k]) + __uint_as_float(y[k])) * sh.scale[c + k];
                    } else {
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(o[k]) * sh.scale[c + k];
                    }
                    if (whole) {
                        if (d < p.dim) {
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (c + k < here) {
                                    const uint32_t y = Half2<!F16>::down(x[k], 0.f);
                                    static_cast<uint16_t *>(p.out)[sh.row_at[c + k] * p.dim + d] = static_cast<uint16_t>(y);
                                }
                        }
                    } else if (d < (WIDE ? 256 : p.dim <= 64 ? 64 : 128)) {
                        float4 *dst = reinterpret_cast<float4 *>(p.part_o + (part * (WIDE ? 256 : p.dim <= 64 ? 64 : 128) + d) * R + c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
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
                ok = __all_sync(~0u, bar_wait(&sh.full[stage], lap & 1, abort));
                if (!ok) break;
                const uint8_t *row = smem + pp.ring_off + stage * pp.stage_bytes + at * pp.stride;
                const uint4 s0 = *reinterpret_cast<const uint4 *>(row + 2 * pp.codes);
                uint32_t s[8];   // scales of blocks 0, 2 | 1, 3 | 4, 6 | 5, 7 | ...
                int4_scales4(s0.x, s);
                int4_scales4(s0.y, s + 2);
                if constexpr (WIDE) {
                    int4_scales4(s0.z, s + 4);
                    int4_scales4(s0.w, s + 6);
                }
                // the tile before last has been multiplied
                if (job >= 2) ok = __all_sync(~0u, bar_wait(&sh.s_full[job & 1], ((job >> 1) & 1) ^ 1, abort));
                if (!ok) break;
                tc_fence_after();
                const uint32_t dst = tmem + lanes + kK + (job & 1) * kKeyCols;
#pragma unroll
                for (int b = 0; b < (WIDE ? 16 : 8); b += 2) {
                    if (b * 16 >= p.dim) break;
                    const uint4 c = *reinterpret_cast<const uint4 *>(row + b * 8);
                    uint32_t y[16];
                    const int sel = b & 2 ? 0x3232 : 0x1010, q = b / 4 * 2;
                    decode16(c.x, c.y, __byte_perm(s[q], 0, sel), y);
                    decode16(c.z, c.w, __byte_perm(s[q + 1], 0, sel), y + 8);
                    tmem_store16(dst + b * 8, y);
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
            for (int32_t i = walk.u.t0; i < walk.u.t1 && ok; ++i) {
                ok = __all_sync(~0u, bar_wait(&sh.full[stage], lap & 1, abort));
                if (!ok) break;
                const uint8_t *row = smem + pp.ring_off + stage * pp.stage_bytes + at * pp.stride;
                const uint8_t *from = row + 2 * pp.codes + (WIDE ? 16 : 8);
                for (int mb = 0; mb < kBlocks; ++mb, ++item) {
                    uint32_t s[4];
                    const uint2 s0 = *reinterpret_cast<const uint2 *>(from + mb * 8);
                    int4_scales4(s0.x, s);
                    int4_scales4(s0.y, s + 2);
                    if (item >= 2) ok = __all_sync(~0u, bar_wait(&sh.v_free[item & 1], ((item >> 1) & 1) ^ 1, abort));
                    if (!ok) break;
                    uint8_t *dst = smem + (item & 1) * kValueBytes;
#pragma unroll
                    for (int b = 0; b < 8; b += 2) {
                        if (mb * 128 + b * 16 >= p.dim) break;
                        const uint4 c = *reinterpret_cast<const uint4 *>(row + pp.codes + mb * 64 + b * 8);
                        uint32_t y[16];
                        const int sel = b & 2 ? 0x3232 : 0x1010, q = b / 4 * 2;
                        decode16(c.x, c.y, __byte_perm(s[q], 0, sel), y);
                        decode16(c.z, c.w, __byte_perm(s[q + 1], 0, sel), y + 8);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4 *>(dst + tile_offset(kTile, at, 2 * b + k)) =
                                make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                    }
                    fence_async_reads();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&sh.v_full[item & 1]);
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.empty[stage]);
                if (++stage == static_cast<uint32_t>(pp.stages)) {
                    stage = 0;
                    ++lap;
                }
            }
        }
    } else if (warp < kIssueWarp) {
        // ------------------------------------------------ copies
        const int tid = (warp - kCopyWarp) * 32 + lane;
        const uint8_t *cache = static_cast<const uint8_t *>(p.k);
        const int32_t chunks = pp.row / 16;
        uint32_t stage = 0, lap = 0, tile = 0;
        for (; walk.more() && ok; walk.next()) {
            if (walk.u.span.n == 0) continue;
            const int32_t h = walk.u.hm / p.row_tiles;
            const uint8_t *head = cache + h * p.k_head;
            for (int32_t i = walk.u.t0; i < walk.u.t1; ++i, ++tile) {
                ok = __all_sync(~0u, bar_wait(&sh.slots_full[tile % kSlotRing], (tile / kSlotRing) & 1, abort));
                if (ok && lap) ok = __all_sync(~0u, bar_wait(&sh.empty[stage], (lap - 1) & 1, abort));
                if (!ok) break;
                const volatile int32_t *slots = sh.slots[tile % kSlotRing];
                const uint32_t dst = base + pp.ring_off + stage * pp.stage_bytes;
                // lane groups walk a row's chunks: (row, chunk) of tid, then 128 chunks on
                int32_t r = tid / chunks, c = tid - r * chunks;
                const int32_t dr = 128 / chunks, dc = 128 - dr * chunks;
#pragma unroll 4
                for (int k = 0; k < chunks; ++k) {
                    const int32_t slot = slots[r];
                    copy16(dst + r * pp.stride + c * 16, head + static_cast<int64_t>(slot < 0 ? 0 : slot) * p.k_slot + c * 16, slot < 0 ? 0u : 16u);
                    r += dr;
                    c += dc;
                    if (c >= chunks) {
                        c -= chunks;
                        ++r;
                    }
                }
                bar_arrive_copies(&sh.full[stage]);
                if (++stage == static_cast<uint32_t>(pp.stages)) {
                    stage = 0;
                    ++lap;
                }
            }
        }
        copies_land();
    } else if (warp == kIssueWarp) {
        // ------------------------------------------------ matrix products (all lanes alike, see elect_lane)
        const bool lead = elect_lane();
        const uint32_t s_desc = mma_desc(true, 128, N, false, p.negative != 0);
        const uint32_t o_desc = mma_desc(true, 128, N, true, false) | 1u << 15;   // A transposed too
        const int ksteps = p.dim / 16;
        const uint32_t q_bytes = N * (WIDE ? 512 : 256);
        uint32_t unit = 0, job0 = 0, item = 0;
        for (; __any_sync(~0u, walk.more()) && ok; walk.next()) {
            if (__any_sync(~0u, walk.u.span.n == 0)) continue;
            const uint32_t jobs = __shfl_sync(~0u, static_cast<uint32_t>(walk.u.t1 - walk.u.t0), 0);
            const uint32_t qb = pp.q_bufs == 2 ? unit & 1 : 0, qph = pp.q_bufs == 2 ? unit >> 1 : unit;
            ok = __all_sync(~0u, bar_wait(&sh.q_full[qb], qph & 1, abort));
            if (!ok) break;
            auto issue_s = [&](uint32_t j) {
                const uint32_t job = job0 + j, sb = job & 1;
                if (!__all_sync(~0u, bar_wait(&sh.key_full[sb], (job >> 1) & 1, abort))) return false;
                tc_fence_after();
                const uint32_t qa = base + pp.q_off + qb * q_bytes, ka = tmem + kK + sb * kKeyCols;
                if (lead) {
#pragma unroll
                    for (int kk = 0; kk < (WIDE ? 16 : 8); ++kk)
                        if (kk < ksteps)
                            mma_ts(tmem + kS + sb * N, ka + kk * 8, smem_desc(qa + (kk >> 2) * (N * 128) + (kk & 3) * 32, 16, 1024), s_desc, kk > 0);
                    tc_commit(&sh.s_full[sb]);
                    if (j + 1 == jobs) tc_commit(&sh.q_empty[qb]);
                }
                __syncwarp();
                return true;
            };
            for (uint32_t j = 0; j < 2 && j < jobs && ok; ++j) ok = issue_s(j);
            for (uint32_t j = 0; j < jobs && ok; ++j) {
                const uint32_t job = job0 + j, sb = job & 1;
                for (int mb = 0; mb < kBlocks; ++mb, ++item) {
                    ok = __all_sync(~0u, bar_wait(&sh.v_full[item & 1], (item >> 1) & 1, abort) &&
                                             bar_wait(&sh.p_full[sb], (job >> 1) & 1, abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t va = v_smem + (item & 1) * kValueBytes, pa = base + pp.p_off + sb * kProbBytes;
                    if (lead) {
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            mma_ss(tmem + kO + mb * N, smem_desc(va + kk * 2048, kTile * 128, 1024),
                                   smem_desc(pa + kk * 2048, kTile * 128, 1024), o_desc, j > 0 || kk > 0);
                        tc_commit(&sh.v_free[item & 1]);
                        if (mb + 1 == kBlocks) tc_commit(&sh.pv_done[sb]);
                    }
                    __syncwarp();
                }
                if (ok && j + 2 < jobs) ok = issue_s(j + 2);
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
    } else {
        // ------------------------------------------------ queries, slots of the tiles to come
        const int turn = warp - kIssueWarp - 1, tid = turn * 32 + lane;
        int32_t last_b = -1;
        uint64_t seen = ~0ull;   // drafted tokens that some row of the request sees
        uint32_t tile = 0, unit = 0;
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
            auto look_up = [&](int32_t t) {
                const uint32_t r = tile % kSlotRing;
                Paging::Place place[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int32_t pos = t * kTile + k * 32 + lane;
                    const bool is = pos < u.span.n && (pos < u.span.ctx || ((seen >> (pos - u.span.ctx)) & 1));
                    place[k] = p.seq_lens ? p.pages.place(u.b, pos, is) : p.pages.listed(p.indices + u.b * p.idx_row + pos, is);
                }
                if (tile >= kSlotRing && !__all_sync(~0u, bar_wait(&sh.slots_empty[r], (tile / kSlotRing - 1) & 1, abort))) return false;
#pragma unroll
                for (int k = 0; k < 4; ++k) sh.slots[r][k * 32 + lane] = static_cast<int32_t>(p.pages.slot(place[k]));
                __syncwarp();
                if (lane == 0) bar_arrive(&sh.slots_full[r]);
                return true;
            };
            // the warp's first tile of the unit goes before the queries, so that copies start
            int32_t t = u.t0;
            for (; t < u.t1 && t < u.t0 + 3 && ok; ++t, ++tile)
                if (tile % 3 == static_cast<uint32_t>(turn)) ok = look_up(t);
            if (!ok) break;
            const int32_t h = u.hm / p.row_tiles, r0 = (u.hm - h * p.row_tiles) * R;
            const int32_t here = rows - r0 < R ? rows - r0 : R, lanes8 = p.dim / 8;
            const uint32_t qb = pp.q_bufs == 2 ? unit & 1 : 0, qph = pp.q_bufs == 2 ? unit >> 1 : unit;
            if (qph > 0) ok = __all_sync(~0u, bar_wait(&sh.q_empty[qb], (qph - 1) & 1, abort));
            if (!ok) break;
            uint8_t *q_tile = smem + pp.q_off + qb * (N * (WIDE ? 512 : 256));
#pragma unroll 4
            for (int32_t k = tid; k < here * lanes8; k += 96) {
                const int32_t r = k / lanes8, c = k - r * lanes8, tok = (r0 + r) / p.group, gq = r0 + r - tok * p.group;
                const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                                     2 * ((static_cast<int64_t>(u.b) * p.next_n + tok) * p.q_row + (h * p.group + gq) * p.q_head);
                const uint4 v = fetch(reinterpret_cast<const uint4 *>(src) + c);
                if constexpr (F16) {
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = Half2<false>::up(x[j]);
                        hi[j] = Half2<true>::down(f.x, f.y);
                        const float2 g = Half2<true>::up(hi[j]);
                        // (an infinity is whole)
                        lo[j] = Half2<true>::down(isinf(f.x) ? 0.f : f.x - g.x, isinf(f.y) ? 0.f : f.y - g.y);
                    }
                    *reinterpret_cast<uint4 *>(q_tile + tile_offset(N, r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(q_tile + tile_offset(N, R + r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                } else {
                    *reinterpret_cast<uint4 *>(q_tile + tile_offset(N, r, c)) = v;
                }
            }
            fence_async_reads();
            __syncwarp();
            if (lane == 0) bar_arrive(&sh.q_full[qb]);
            ++unit;
            for (; t < u.t1 && ok; ++t, ++tile)
                if (tile % 3 == static_cast<uint32_t>(turn)) ok = look_up(t);
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
    constexpr int N = F16 ? 2 * R : R;
    const int64_t rows = static_cast<int64_t>(p.next_n) * p.group;
    p.row_tiles = static_cast<int32_t>((rows + R - 1) / R);
    p.request_units = p.kv_heads * p.row_tiles;
    place_parts(p, ws);
    pp.codes = int4_codes(p.dim);
    pp.row = int4_row(p.dim);
    pp.stride = pp.row | 16;       // an odd number of 16-byte pieces: neighbouring rows in other banks
    // values (two tiles of 128 x 128), probabilities, queries, the ring
    constexpr uint32_t kQ = N * (WIDE ? 512 : 256);
    const uint32_t most = kMaxSmemBytes - 1024 - (sizeof(Shared4) + 15) / 16 * 16;
    pp.p_off = 2 * kTile * 256;
    pp.q_off = pp.p_off + 2 * kTile * 128 * (N > 64 ? 2 : 1);
    pp.q_bufs = kQ > 16384 ? 1 : 2;
    pp.ring_off = pp.q_off + pp.q_bufs * kQ;
    pp.stage_bytes = kTile * pp.stride;
    const uint32_t fit = (most - pp.ring_off) / pp.stage_bytes;
    pp.stages = static_cast<int32_t>(fit < kMaxStages ? fit : kMaxStages);
    if (pp.stages > kSlotRing - 1) pp.stages = kSlotRing - 1;   // (copies wait for a stage, never for slots behind it)
    if (pp.stages < 1) return cudaErrorInvalidValue;
    pp.shared_off = pp.ring_off + pp.stages * pp.stage_bytes;
    const size_t bytes = 1024 + pp.shared_off + sizeof(Shared4);
    static std::atomic<uint64_t> allowed;
    auto kernel = attention_int4_kernel<F16, R, WIDE>;
    cudaError_t e = allow_smem(kernel, kMaxSmemBytes, allowed);
    if (e != cudaSuccess) return e;
    const int grid = sms < kMaxGrid ? sms : kMaxGrid;
    e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kThreads4, bytes, stream, 1, pp);
    if (e != cudaSuccess) return e;
    if constexpr (WIDE) return launch_join<!F16, 256>(p, R, kTile, sms, stream);
    else return p.dim <= 64 ? launch_join<!F16, 64>(p, R, kTile, sms, stream) : launch_join<!F16, 128>(p, R, kTile, sms, stream);
}

// By the rows of a head: 16, 32, 64 (above dimension 128 tensor memory has room
// for 32).  More rows are more units, each of which decodes the cache.
template <bool F16>
cudaError_t launch_int4(const Int4Params &pp, uint8_t *ws, int sms, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(pp.a.next_n) * pp.a.group;
    if (pp.a.dim > 128) return rows <= 16 ? launch_rows<F16, 16, true>(pp, ws, sms, s) : launch_rows<F16, 32, true>(pp, ws, sms, s);
    if (rows <= 16) return launch_rows<F16, 16, false>(pp, ws, sms, s);
    if (rows <= 32) return launch_rows<F16, 32, false>(pp, ws, sms, s);
    return launch_rows<F16, 64, false>(pp, ws, sms, s);
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
    if (!out) return GBTOPK_EINVAL;
    if (!aligned_to(out, 16) || !aligned_to(lse, 4)) return GBTOPK_EALIGN;
    if (!workspace || !aligned_to(workspace, 256) ||
        workspace_bytes < gbtopk_attention_workspace_bytes(num_rows, q_heads, kv_heads, head_dim))
        return GBTOPK_EWORKSPACE;
    p.q = q;
    p.q_row = q_row_stride;
    p.q_head = q_head_stride;
    p.k = cache;
    p.k_slot = slot_stride;
    p.k_head = head_stride;
    p.requests = static_cast<int32_t>(num_rows / p.next_n);
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.dim = head_dim;
    pp.k_mul = fmaxf(fabsf(scale) * kLog2e * k_scale * kInt4Lift, FLT_MIN);   // a scale of 0 stays a product that ignores no mask
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
