// PTX wrappers for the tensor-core kernels (sm_103a): mbarriers with bounded
// waits, 16-byte asynchronous copies into swizzled tiles, tcgen05 matrix
// products with tensor-memory accumulators.  Not part of the ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace gbtopk {

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------- mbarriers

__device__ __forceinline__ void bar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Arrives once every cp.async that the thread has issued so far has landed
// (the barrier's count includes this arrival).
__device__ __forceinline__ void bar_arrive_copies(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool bar_try(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// About a second of SM cycles: no wait of these kernels takes a thousandth
// of it, so a wait that reaches it has lost its partner.
constexpr long long kWaitCycles = 2000000000ll;

// A block's waits: `given_up` is set by the first that runs out, after `limit`
// cycles.
struct Waits {
    volatile uint32_t *given_up;
    long long limit;
};

// Waits for the phase of `parity` to complete.  False when the wait gave up
// or another one of the block did: the caller leaves its loop.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, const Waits &w) {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
        if (*w.given_up) return false;
        if (clock64() - t0 > w.limit) {
            *w.given_up = 1;
            return false;
        }
    }
    return true;
}

// ---------------------------------------------------------------- copies

// 16 bytes to shared memory, or 16 zero bytes when `bytes` is 0 (nothing is
// read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copies_land() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Orders shared memory written by ordinary stores and cp.async (seen through
// a barrier) before the tensor core's reads of it.
__device__ __forceinline__ void fence_async_reads() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Byte offset of 16-byte chunk c of row r in a tile of `rows` rows: panels of
// 64 16-bit elements (128 bytes) a row, the chunks of each eight rows XORed
// with the row number (the 128-byte swizzle of the matrix descriptors).
__device__ __forceinline__ uint32_t tile_offset(uint32_t rows, uint32_t r, uint32_t c) {
    return (c >> 3) * rows * 128 + r * 128 + (((c ^ r) & 7) << 4);
}

// --------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t *where, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(where)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The barrier's one arrival when every matrix product issued so far is done.
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets in 16-byte units, version 1.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
    return static_cast<uint64_t>((addr & 0x3ffff) >> 4) | static_cast<uint64_t>(lead >> 4) << 16 |
           static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: 16-bit A and B of one type, 32-bit accumulator.
__device__ __forceinline__ uint32_t mma_desc(bool bf16, uint32_t m, uint32_t n, bool b_transposed, bool negate) {
    return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (negate ? 1u << 13 : 0u) | (b_transposed ? 1u << 16 : 0u) |
           (n >> 3) << 17 | (m >> 4) << 24;
}

// One lane of the (converged) warp.  The warp that issues products runs its
// loop with all lanes on equal values and puts only the instructions
// themselves under this: their descriptors go through warp-uniform registers,
// and in a branch of one lane the compiler may take another lane's stale copy.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// D (tensor memory) = A B, + D when `add`; A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// The same with A in tensor memory: lane = row, two elements of K a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// The same issued by the lane with `lead` of a converged warp: a predicate in
// place of a branch, in which every descriptor is moved to uniform registers
// again (with packed sums, a long prompt's attention 648 -> 613 us a call).
__device__ __forceinline__ void mma_ss_if(bool lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(lead))
        : "memory");
}
__device__ __forceinline__ void mma_ts_if(bool lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(lead))
        : "memory");
}

// 32 columns of the warp's 32 lanes, one lane a thread.  The values are there
// after tc_wait_ld.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// Two products and sums, two products, two sums, as one instruction.
__device__ __forceinline__ float2 fma2(float x, float y, float k, float n) {   // k x + n, k y + n
    float2 r;
    asm("{\n .reg .b64 v, k, n;\n mov.b64 v, {%2, %3};\n mov.b64 k, {%4, %4};\n mov.b64 n, {%5, %5};\n"
        " fma.rn.f32x2 v, v, k, n;\n mov.b64 {%0, %1}, v;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x), "f"(y), "f"(k), "f"(n));
    return r;
}
__device__ __forceinline__ float2 mul2(float x, float y, float k) {   // k x, k y, rounded
    float2 r;
    asm("{\n .reg .b64 v, k;\n mov.b64 v, {%2, %3};\n mov.b64 k, {%4, %4};\n mul.rn.f32x2 v, v, k;\n mov.b64 {%0, %1}, v;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x), "f"(y), "f"(k));
    return r;
}
__device__ __forceinline__ void add2(float2 &s, float x, float y) {
    asm("{\n .reg .b64 v, s;\n mov.b64 v, {%2, %3};\n mov.b64 s, {%0, %1};\n add.rn.f32x2 s, s, v;\n mov.b64 {%0, %1}, s;\n}"
        : "+f"(s.x), "+f"(s.y)
        : "f"(x), "f"(y));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace gbtopk
