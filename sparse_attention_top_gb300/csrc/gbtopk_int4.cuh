// Rows of a 4-bit cache (include/gbtopk.h states the format): sizes, and the
// two steps that every reader takes.  Not part of the ABI.
#pragma once

#include <cmath>

#include <cuda_bf16.h>

#include "gbtopk_decode.cuh"

namespace gbtopk {

// Bytes of a row's areas: codes of the keys, as many of the values, scales of
// the keys, as many of the values.
__host__ __device__ constexpr int int4_codes(int dim) { return (dim + 31) / 32 * 16; }
__host__ __device__ constexpr int int4_scales(int dim) { return dim <= 128 ? 8 : 16; }
__host__ __device__ constexpr int int4_row(int dim) { return 2 * (int4_codes(dim) + int4_scales(dim)); }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Codes 2j and 2j + 1 of a word of eight: a rotation and a mask leave sign and
// magnitude where bf16 has its sign and its last three bits, which is the
// subnormal number code * 2^-133.  A multiplication by the block's scale times
// 2^118 gives code * scale * 2^-15, which bf16 holds exactly (3 + 4 bits); the
// 2^15 is the caller's.  So a pair of elements costs three instructions and no
// conversion.
constexpr float kInt4Lift = 32768.f;
template <int J>
__device__ __forceinline__ uint32_t int4_pair(uint32_t word) {
    return (J ? __funnelshift_r(word, word, 4 * J) : word) & 0x80078007u;
}

// Two scales, the bytes 0 and 2 of `bytes`, times 2^118 as bf16.  A byte's low
// seven bits, moved to bf16's exponent and mantissa, are the scale times 2^-120
// (its subnormals are bf16's); 2^238 is more than one factor holds.
__device__ __forceinline__ uint32_t int4_scales2(uint32_t bytes) {
    constexpr uint32_t k119 = (119u + 127u) << 7, kTwice = k119 << 16 | k119;
    return mul_bf16x2(mul_bf16x2((bytes & 0x007f007fu) << 4, kTwice), kTwice);
}

// (a power of two: codes times scales stay exact)
inline bool int4_unit(float s) {
    int e;
    return std::isfinite(s) && s > 0.f && std::frexp(s, &e) == 0.5f && e > -60 && e <= 61;
}

// Rows of a 4-bit cache, read and written in 16-byte pieces.
inline int check_int4(const void *base, int64_t slot_stride, int64_t head_stride, int64_t num_slots, int32_t dim) {
    if (num_slots < 0 || slot_stride < 0 || head_stride < 0) return GBTOPK_EINVAL;
    if (num_slots > 0 && !base) return GBTOPK_EINVAL;
    if (dim % 16 != 0 || num_slots > INT32_MAX) return GBTOPK_EUNSUPPORTED;
    if (!aligned_to(base, 16) || !multiple_of(slot_stride, 16) || !multiple_of(head_stride, 16)) return GBTOPK_EALIGN;
    return GBTOPK_OK;
}

}  // namespace gbtopk
