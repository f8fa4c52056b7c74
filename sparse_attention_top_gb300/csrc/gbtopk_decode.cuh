// Shared by the decode-step kernels (gbtopk_attention.cu, gbtopk_cache.cu,
// gbtopk_verify.cu): the paged cache's address arithmetic, 16-bit element
// conversions, launch helpers and argument checks.  Not part of the ABI.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "gbtopk.h"
#include "gbtopk_internal.h"

namespace gbtopk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Unsigned division by a launch-constant divisor: q = (x * mul) >> (32 +
// shift) for 0 <= x < 2^31, with mul = ceil(2^(32+shift) / d) and shift =
// ceil(log2 d) - 1 (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994): the rounding of mul adds less than x / 2^31
// of 1/d, so the quotient is exact.  d = 1 uses mul = 0 (the identity).
struct FastDiv {
    uint32_t d, mul, shift;
    __host__ void init(uint32_t divisor) {
        d = divisor;
        mul = 0;
        shift = 0;
        if (divisor > 1) {
            uint32_t l = 0;
            while ((1ull << l) < divisor) ++l;
            shift = l - 1;
            mul = static_cast<uint32_t>(((1ull << (32 + shift)) + divisor - 1) / divisor);
        }
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const {
        return mul ? __umulhi(x, mul) >> shift : x;
    }
};

// An ordinary load of data that the stream's previous kernel may have
// written: it stays behind pdl_wait, which a load of constant data need not.
template <typename T>
__device__ __forceinline__ T fetch(const T *p) {
    return *p;
}

// The page table of a batch of requests over one cache.
struct Paging {
    const int32_t *table;
    const int32_t *spare;   // any readable word
    int64_t cols, row_stride;
    int64_t num_slots;
    FastDiv page;

    // Page id and offset in it of a position.  The id's load is in flight
    // until slot() looks at it: it is unconditional (from
    // `spare` where there is no position),
    // because a load that is merged with a constant is waited for at once.
    struct Place {
        int32_t id;
        uint32_t rest;
        bool is;
    };
    __device__ __forceinline__ Place place(int64_t i, int32_t p, bool is) const {
        const uint32_t c = page.div(static_cast<uint32_t>(p));
        is = is && p >= 0 && static_cast<int64_t>(c) < cols;
        return listed(table + i * row_stride + c, is, static_cast<uint32_t>(p) - c * page.d);
    }
    __device__ __forceinline__ Place listed(const int32_t *at, bool is, uint32_t rest = 0) const {
        return Place{fetch(is ? at : spare), rest, is};
    }
    // The cache slot, or -1 where there is none.
    __device__ __forceinline__ int64_t slot(const Place &at) const {
        const int64_t s = static_cast<int64_t>(at.id) * page.d + at.rest;
        return at.is && at.id >= 0 && s < num_slots ? s : -1;
    }
    __device__ __forceinline__ int64_t slot(int64_t i, int32_t p) const { return slot(place(i, p, true)); }
};

template <bool BF16>
struct Half2 {
    using T = __nv_bfloat16;
    __device__ __forceinline__ static float2 up(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    __device__ __forceinline__ static uint32_t down(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

template <>
struct Half2<false> {
    using T = __half;
    __device__ __forceinline__ static float2 up(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    __device__ __forceinline__ static uint32_t down(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// SMs of the current device (0: the runtime refused), asked once a device.
inline int device_sms() {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
    return sms;
}

// Lets the kernel use up to `bytes` of dynamic shared memory, once a device.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (r == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return r;
}

// Launch as a programmatic dependent of the stream's previous kernel: the
// launch overlaps its tail, and the kernel waits (pdl_wait) before it reads
// anything.
template <typename... A, typename... B>
cudaError_t launch_pdl(void (*kernel)(A...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                       int cluster, B... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool multiple_of(int64_t v, int64_t a) { return v % a == 0; }

inline int check_heads(int dtype, int64_t num_rows, int32_t q_heads, int32_t kv_heads, int32_t dim) {
    if (dtype != GBTOPK_F32 && dtype != GBTOPK_BF16 && dtype != GBTOPK_F16) return GBTOPK_EINVAL;
    if (num_rows < 0 || q_heads < 1 || kv_heads < 1 || dim < 1 || q_heads % kv_heads != 0) return GBTOPK_EINVAL;
    if (dtype == GBTOPK_F32 || dim > GBTOPK_MAX_HEAD_DIM || dim % 8 != 0) return GBTOPK_EUNSUPPORTED;
    if (num_rows > INT32_MAX || q_heads > 65535) return GBTOPK_EUNSUPPORTED;
    return GBTOPK_OK;
}

// Rows of 16-bit elements read in 16-byte pieces; `any`: there are some.
inline int check_rows(const void *base, int64_t a, int64_t b, bool any) {
    if (any && !base) return GBTOPK_EINVAL;
    if (a < 0 || b < 0) return GBTOPK_EINVAL;
    if (!aligned_to(base, 16) || !multiple_of(a, 8) || !multiple_of(b, 8)) return GBTOPK_EALIGN;
    return GBTOPK_OK;
}

inline int check_pages(const int32_t *table, int64_t cols, int64_t stride, int32_t page, int64_t num_slots,
                int64_t requests, Paging *out) {
    if (page < 1 || page > (1 << 30) || cols < 0 || num_slots < 0 || (requests > 1 && stride < cols)) return GBTOPK_EINVAL;
    if (requests > 0 && cols > 0 && !table) return GBTOPK_EINVAL;
    if (!aligned_to(table, 4)) return GBTOPK_EALIGN;
    if (cols > INT32_MAX / page) cols = INT32_MAX / page;  // positions are 31-bit numbers
    out->table = table;
    out->cols = cols;
    out->row_stride = stride;
    out->num_slots = num_slots;
    out->page.init(static_cast<uint32_t>(page));
    return GBTOPK_OK;
}

}  // namespace gbtopk
