// Norms and rotation of queries and keys with the cache write in the same pass
// (gbtopk_rotate_and_cache, gbtopk_rotate_and_cache_int4), and a 4-bit cache
// read back (gbtopk_cache_read_int4).
//
// A token's q, k and v rows are read once, 16 bytes a lane and a group of lanes
// a head row, and written once:
//     y = x rsqrt(mean x^2 + eps) w,   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin).
// The angle of pair i is position * inv_freq[i]; its turns are reduced in 64
// bits (32 lose the angles of far positions), once a token for all of its
// heads, and their sine and cosine are 32 bits.  A lane's partner in the
// rotation is another lane of its group, whose inputs come by shuffle.
//
// 4-bit rows: blocks of sixteen elements are two lanes' eight each.  Codes and
// scales are those of the formula's real numbers, not of their 32-bit
// approximations: an element whose 32-bit value lies nearer to a border between
// two codes (or two scales) than its error, some 2 in 100,000, makes its warp
// compute the row once more in 64 bits.  So a cache does not depend on the
// order of sums, and two builds agree bit for bit.
//
// Bound by the bytes read and written.
#include <cfloat>
#include <cmath>

#include "gbtopk_int4.cuh"

namespace gbtopk {
namespace {

constexpr int kRowThreads = 256;
constexpr int kInFlight = 3;   // head rows that a lane group has in flight

struct RotateParams {
    const void *x[3];                 // q, k, v
    int64_t x_row[3], x_head[3];      // strides in elements
    const void *w[2];                 // norm weights of q and k, or null
    const int32_t *positions, *slots;
    const float *inv_freq;
    void *q_out, *k_cache, *v_cache;  // (4-bit rows: k_cache)
    int64_t qo_row, qo_head, k_slot, k_head, v_slot, v_head;   // elements (4-bit rows: bytes)
    int64_t num_slots;
    int32_t q_heads, kv_heads, dim, half;   // half: rotated pairs
    int32_t steps;                    // row groups of a block
    float eps, inv_unit[2];
};

template <bool BF16>
__device__ __forceinline__ void load_weights(const void *w, bool wide, int32_t at, float *f) {
    if (wide) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at + 4);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(w) + 2 * at);
        const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = Half2<BF16>::up(v[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}

// A scale (in units) of a block whose largest magnitude is `top` units: top / 7
// to four significant bits and at least 2^-9 steps, ties to even, at most 448.
// *near: how near top lies to the border, in top's units.
__device__ __forceinline__ float block_scale(float top, float *near) {
    const float t = top * (1.f / 7.f);
    int e = static_cast<int>(__float_as_uint(t) >> 23) - 127;
    e = e < -6 ? -6 : e > 9 ? 9 : e;
    const float step = __int_as_float((e - 3 + 127) << 23), per = __int_as_float((3 - e + 127) << 23);
    const float low = floorf(t * per), off = top * per - 7.f * (low + 0.5f);   // exact: 7 (low + 1/2) has 8 bits
    *near = fabsf(off) * step;
    const bool up = off > 0.f || (off == 0.f && (static_cast<int>(low) & 1));
    return fminf((low + (up ? 1.f : 0.f)) * step, 448.f);
}

__device__ __forceinline__ uint32_t scale_byte(float s) {   // of a number that has one
    if (s < 0x1p-6f) return static_cast<uint32_t>(s * 512.f);
    return (__float_as_uint(s) >> 20) - (120u << 3);
}

__device__ __forceinline__ uint32_t put_code(int i, int code) {   // element i of a word of eight
    const int j = i / 2;
    const uint32_t mag = static_cast<uint32_t>(code < 0 ? -code : code), sign = code < 0;
    return i & 1 ? mag << (4 * j + 16) | sign << ((4 * j + 31) & 31) : mag << (4 * j) | sign << (4 * j + 15);
}

struct Row {
    uint32_t raw[4];       // the lane's eight elements
    int32_t at;            // the first one's index
    bool there;            // the lane has elements
};

// The lane's eight elements of the normalised and rotated row in 64 bits, one
// row a group of LP lanes; every lane of the warp takes part.
template <bool BF16, int LP, bool PAIRS>
__device__ __noinline__ void turned_wide(const RotateParams &p, const Row &row, const void *w, bool w_wide, double position, double *y) {
    const int lane = threadIdx.x & (LP - 1);
    double sum = 0;
    float x[8], f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = Half2<BF16>::up(row.raw[i]);
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
        sum += static_cast<double>(t.x) * t.x + static_cast<double>(t.y) * t.y;
    }
    for (int o = LP / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    const double r = w ? 1.0 / sqrt(sum / p.dim + static_cast<double>(p.eps)) : 1.0;
    if (w && row.there) load_weights<BF16>(w, w_wide, row.at, f);
    for (int i = 0; i < 8; ++i) y[i] = w && row.there ? x[i] * r * f[i] : x[i] * r;
    auto turn = [&](int32_t k, double *c, double *s) {
        const double a = position * (static_cast<double>(p.inv_freq[k]) * 0.15915494309189533577);
        sincospi(2 * (a - rint(a)), s, c);
    };
    const int32_t rotary = 2 * p.half;
    if constexpr (PAIRS) {
        if (!row.there || row.at >= rotary) return;
        for (int i = 0; i < 8; i += 2) {
            double c, s;
            turn((row.at + i) / 2, &c, &s);
            const double a = y[i], b = y[i + 1];
            y[i] = a * c - b * s;
            y[i + 1] = b * c + a * s;
        }
    } else {
        const bool in = row.there && row.at < rotary, second = row.at >= p.half;
        const int from = in ? (second ? lane - p.half / 8 : lane + p.half / 8) : lane;
        for (int i = 0; i < 8; ++i) {
            const double other = __shfl_sync(~0u, y[i], from, LP);
            if (!in) continue;
            double c, s;
            turn(row.at - (second ? p.half : 0) + i, &c, &s);
            y[i] = second ? y[i] * c + other * s : y[i] * c - other * s;
        }
    }
}

// Codes of the lane's elements (a block's other eight are the lane's
// neighbour's) and the block's scale byte, from numbers in 64 bits.
__device__ __noinline__ uint32_t encode_wide(const double *y, double inv_unit, uint32_t *byte) {
    double top = 0;
    for (int i = 0; i < 8; ++i) top = fmax(top, fabs(y[i] * inv_unit));
    top = fmax(top, __shfl_xor_sync(~0u, top, 1));
    double t = top / 7;
    t = t > 448 ? 448 : t;
    int e = static_cast<int>(static_cast<unsigned long long>(__double_as_longlong(t)) >> 52) - 1023;
    e = e < -6 ? -6 : e;
    const double step = __longlong_as_double(static_cast<long long>(e - 3 + 1023) << 52);
    double s = rint(t / step) * step;
    s = s > 448 ? 448 : s;
    *byte = scale_byte(static_cast<float>(s));
    uint32_t word = 0;
    for (int i = 0; i < 8; ++i) {
        double c = s > 0 ? rint(y[i] * inv_unit / s) : 0;
        c = c > 7 ? 7 : c < -7 ? -7 : c == c ? c : 0;
        word |= put_code(i, static_cast<int>(c));
    }
    return word;
}

// The same from 32-bit numbers with errors up to err[i]; *doubt where an error
// could have changed a code or the scale.
__device__ __forceinline__ uint32_t encode(const float *y, const float *err, float inv_unit, uint32_t *byte, bool *doubt) {
    float top = 0.f, off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        top = fmaxf(top, fabsf(y[i] * inv_unit));   // (a NaN is no maximum)
        off = fmaxf(off, err[i] * inv_unit);
    }
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
    off = fmaxf(off, __shfl_xor_sync(~0u, off, 1));
    float near;
    const float s = block_scale(fminf(top, 4096.f), &near);   // (saturated from 7 * 464 on)
    bool odd = off > 0.f && near <= off;
    *byte = scale_byte(s);
    const float per = s > 0.f ? 1.f / s : 0.f, half = 0.5f * s;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = y[i] * inv_unit;
        float c = rintf(fminf(fmaxf(x * per, -8.f), 8.f));
        if (!(x == x)) c = 0.f;
        const float rest = fmaf(-c, s, x), far = fabsf(rest);   // exact where the nearest code is not beyond 8
        const bool tie = far == half && (static_cast<int>(c) & 1);
        if (fabsf(c) < 8.f && s > 0.f && (far > half || tie)) c += rest > 0.f ? 1.f : -1.f;
        odd |= err[i] > 0.f && fabsf(far - half) <= err[i] * inv_unit;
        c = fminf(fmaxf(c, -7.f), 7.f);
        word |= put_code(i, static_cast<int>(c));
    }
    *doubt = odd;
    return word;
}

// Grid (tokens, chunks of a token's head rows): rows q heads, k heads, v heads.
template <bool BF16, int LP, bool PAIRS, bool INT4>
__global__ void __launch_bounds__(kRowThreads) rotate_kernel(const __grid_constant__ RotateParams p, int w_wide) {
    constexpr int kRows = kRowThreads / LP;   // a step
    __shared__ float2 turn[128];           // cosine and sine of the token's angles
    pdl_wait();
    pdl_release();
    const int64_t token = blockIdx.x;
    const int lane = threadIdx.x & (LP - 1), group = threadIdx.x / LP;
    const int32_t rows = p.q_heads + 2 * p.kv_heads;
    const int32_t first = static_cast<int32_t>(blockIdx.y) * p.steps;
    const int32_t slot = p.slots[token];
    const bool kept = slot >= 0 && slot < p.num_slots;
    const int32_t at = lane * 8;
    const bool there = at < p.dim;
    const int32_t position = p.half ? p.positions[token] : 0;
    bool turned = false;
    for (int32_t s0 = 0; s0 < p.steps; s0 += kInFlight) {
        Row row[kInFlight];
        int32_t head[kInFlight];
        int kind[kInFlight];                  // q, k, v, or -1
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            int32_t h = s0 + u < p.steps ? (first + s0 + u) * kRows + group : rows;
            kind[u] = h >= rows ? -1 : h < p.q_heads ? 0 : h < p.q_heads + p.kv_heads ? 1 : 2;
            if (kind[u] > 0) h -= p.q_heads + (kind[u] - 1) * p.kv_heads;
            head[u] = h;
            if (kind[u] > 0 && !kept) kind[u] = -1;
            row[u].at = at;
            row[u].there = there && kind[u] >= 0;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row[u].there) {
                const uint8_t *base = static_cast<const uint8_t *>(kind[u] == 0 ? p.x[0] : kind[u] == 1 ? p.x[1] : p.x[2]);
                const int64_t sr = kind[u] == 0 ? p.x_row[0] : kind[u] == 1 ? p.x_row[1] : p.x_row[2];
                const int64_t sh = kind[u] == 0 ? p.x_head[0] : kind[u] == 1 ? p.x_head[1] : p.x_head[2];
                v = *reinterpret_cast<const uint4 *>(base + 2 * (token * sr + h * sh + at));
            }
            row[u].raw[0] = v.x; row[u].raw[1] = v.y; row[u].raw[2] = v.z; row[u].raw[3] = v.w;
        }
        if (!turned && p.half) {           // while the rows are in flight
            for (int k = threadIdx.x; k < p.half; k += kRowThreads) {
                const double a = static_cast<double>(position) * (static_cast<double>(p.inv_freq[k]) * 0.15915494309189533577);
                float s, c;
                sincospif(2.f * static_cast<float>(a - rint(a)), &s, &c);
                turn[k] = make_float2(c, s);
            }
            __syncthreads();
            turned = true;
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (__all_sync(~0u, kind[u] < 0)) continue;
            const void *w = kind[u] == 0 ? p.w[0] : kind[u] == 1 ? p.w[1] : nullptr;
            const bool rotates = kind[u] == 0 || kind[u] == 1;
            float y[8], err[8];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 t = Half2<BF16>::up(row[u].raw[i]);
                y[2 * i] = t.x;
                y[2 * i + 1] = t.y;
                sum = fmaf(t.x, t.x, fmaf(t.y, t.y, sum));
            }
            for (int o = LP / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            const float r = rsqrtf(sum / static_cast<float>(p.dim) + p.eps);
            if (w && row[u].there) {
                float f[8];
                load_weights<BF16>(w, w_wide != 0, at, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= r * f[i];
            }
            // Relative errors, in units of 2^-24: the sum 14, halved by the
            // root, rsqrtf 4, the products 3; cosine and sine 2 ulp and the
            // turns' rounding, 2 pi / 2, of 1.  2^-19 of the terms is twice that.
#pragma unroll
            for (int i = 0; i < 8; ++i) err[i] = w ? fabsf(y[i]) * 0x1p-19f : 0.f;
            const int32_t rotary = 2 * p.half;
            if constexpr (PAIRS) {
                if (rotates && there && at < rotary) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float2 cs = turn[(at + i) / 2];
                        const float a = y[i], b = y[i + 1];
                        y[i] = a * cs.x - b * cs.y;
                        y[i + 1] = b * cs.x + a * cs.y;
                        if constexpr (INT4) err[i] = err[i + 1] = (fabsf(a) + fabsf(b)) * 0x1p-19f;
                    }
                }
            } else {
                const bool in = rotates && there && at < rotary, second = at >= p.half;
                const int from = in ? (second ? lane - p.half / 8 : lane + p.half / 8) : lane;
                const int32_t k0 = in ? at - (second ? p.half : 0) : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float other = __shfl_sync(~0u, y[i], from, LP);
                    if (!in) continue;
                    const float2 cs = turn[k0 + i];
                    if constexpr (INT4) err[i] = (fabsf(y[i]) + fabsf(other)) * 0x1p-19f;
                    y[i] = second ? y[i] * cs.x + other * cs.y : y[i] * cs.x - other * cs.y;
                }
            }
            if (!INT4 || __any_sync(~0u, kind[u] == 0)) {
                if (row[u].there && !(INT4 && kind[u] > 0)) {
                    uint4 v;
                    v.x = Half2<BF16>::down(y[0], y[1]);
                    v.y = Half2<BF16>::down(y[2], y[3]);
                    v.z = Half2<BF16>::down(y[4], y[5]);
                    v.w = Half2<BF16>::down(y[6], y[7]);
                    if (kind[u] == 2) v = make_uint4(row[u].raw[0], row[u].raw[1], row[u].raw[2], row[u].raw[3]);
                    uint8_t *dst = kind[u] == 0 ? static_cast<uint8_t *>(p.q_out) + 2 * (token * p.qo_row + head[u] * p.qo_head)
                                   : kind[u] == 1 ? static_cast<uint8_t *>(p.k_cache) + 2 * (slot * p.k_slot + head[u] * p.k_head)
                                                  : static_cast<uint8_t *>(p.v_cache) + 2 * (slot * p.v_slot + head[u] * p.v_head);
                    *reinterpret_cast<uint4 *>(dst + 2 * at) = v;
                }
            }
            if constexpr (INT4) {
                if (__all_sync(~0u, kind[u] <= 0)) continue;
                const float inv_unit = kind[u] == 2 ? p.inv_unit[1] : p.inv_unit[0];
                uint32_t byte;
                bool doubt;
                uint32_t word = encode(y, err, inv_unit, &byte, &doubt);
                if (__any_sync(~0u, doubt && row[u].there && kind[u] == 1)) {
                    double wide[8];
                    turned_wide<BF16, LP, PAIRS>(p, row[u], kind[u] == 1 ? p.w[1] : nullptr, w_wide != 0, position, wide);
                    uint32_t b;
                    const uint32_t again = encode_wide(wide, inv_unit, &b);
                    if (kind[u] == 1) {
                        word = again;
                        byte = b;
                    }
                }
                if (row[u].there && kind[u] > 0) {
                    uint8_t *dst = static_cast<uint8_t *>(p.k_cache) + slot * p.k_slot + head[u] * p.k_head;
                    const int c = int4_codes(p.dim), part = kind[u] - 1;
                    *reinterpret_cast<uint32_t *>(dst + part * c + at / 2) = word;
                    if (!(lane & 1)) dst[2 * c + part * int4_scales(p.dim) + at / 16] = static_cast<uint8_t>(byte);
                }
            }
        }
    }
}

// ------------------------------------------------------------- reading back

struct ReadParams {
    const uint8_t *cache;
    int64_t slot_stride, head_stride, num_slots, n;   // bytes; n: listed slots
    const int32_t *slots;
    void *out[2];
    float unit[2];           // times 2^15
    int32_t kv_heads, dim;
    FastDiv words, heads;    // words of a row's codes, heads
};

// A thread a word of codes: four bytes in, sixteen out, neighbours of
// neighbours; grid (pieces of the listed rows, keys and values).
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int kEach = 4;
    pdl_wait();
    pdl_release();
    const int part = blockIdx.y;
    const int c = int4_codes(p.dim), sb = 2 * c + part * int4_scales(p.dim);
    const int64_t total = p.n * p.kv_heads * (p.dim / 8);
    const int64_t base = static_cast<int64_t>(blockIdx.x) * (kRowThreads * kEach) + threadIdx.x;
    uint32_t word[kEach], byte[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int64_t i = base + u * kRowThreads;
        word[u] = byte[u] = 0;
        if (i >= total) continue;
        // (whole numbers below 2^31: the launch splits longer lists)
        const uint32_t row = p.words.div(static_cast<uint32_t>(i)), w = static_cast<uint32_t>(i) - row * p.words.d;
        const uint32_t at = p.heads.div(row), h = row - at * p.heads.d;
        const int32_t slot = p.slots[at];
        if (slot < 0 || slot >= p.num_slots) continue;
        const uint8_t *src = p.cache + slot * p.slot_stride + h * p.head_stride;
        word[u] = *reinterpret_cast<const uint32_t *>(src + part * c + 4 * w);
        byte[u] = src[sb + w / 2];
    }
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int64_t i = base + u * kRowThreads;
        if (i >= total) continue;
        const uint32_t scale = __byte_perm(int4_scales2(byte[u]), 0, 0x1010);
        const uint32_t pair[4] = {int4_pair<0>(word[u]), int4_pair<1>(word[u]), int4_pair<2>(word[u]), int4_pair<3>(word[u])};
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = Half2<true>::up(mul_bf16x2(pair[j], scale));
            out[j] = Half2<BF16>::down(f.x * p.unit[part], f.y * p.unit[part]);
        }
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out[part]) + 16 * i) = make_uint4(out[0], out[1], out[2], out[3]);
    }
}

template <bool BF16, int LP, bool PAIRS>
cudaError_t launch_rotate(RotateParams p, int64_t tokens, bool int4, int w_wide, int sms, cudaStream_t s) {
    const int32_t rows = p.q_heads + 2 * p.kv_heads, per = kRowThreads / LP, steps = (rows + per - 1) / per;
    // A block a token; where that leaves SMs idle, a block a step of its rows
    // (each works the token's angles out again).
    const int32_t chunks = tokens < 2ll * sms ? steps : 1;
    p.steps = chunks == 1 ? steps : 1;
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(chunks));
    return int4 ? launch_pdl(rotate_kernel<BF16, LP, PAIRS, true>, grid, kRowThreads, 0, s, 1, p, w_wide)
                : launch_pdl(rotate_kernel<BF16, LP, PAIRS, false>, grid, kRowThreads, 0, s, 1, p, w_wide);
}

template <bool BF16, bool PAIRS>
cudaError_t launch_lanes(const RotateParams &p, int64_t tokens, bool int4, int w_wide, int sms, cudaStream_t s) {
    if (p.dim <= 64) return launch_rotate<BF16, 8, PAIRS>(p, tokens, int4, w_wide, sms, s);
    if (p.dim <= 128) return launch_rotate<BF16, 16, PAIRS>(p, tokens, int4, w_wide, sms, s);
    return launch_rotate<BF16, 32, PAIRS>(p, tokens, int4, w_wide, sms, s);
}

int rotate(RotateParams &p, int dtype, int64_t tokens, int weight_dtype, int interleaved, bool int4, void *stream) {
    int rc;
    if (tokens > 0 && !p.slots) return GBTOPK_EINVAL;
    if (p.half > 0 && (!p.positions || !p.inv_freq) && tokens > 0) return GBTOPK_EINVAL;
    if (!(p.eps >= 0.f)) return GBTOPK_EINVAL;
    if (2 * static_cast<int64_t>(p.half) > p.dim || p.half < 0) return GBTOPK_EINVAL;
    if (p.half % 8 != 0) return GBTOPK_EUNSUPPORTED;   // pairs of whole lanes
    if (weight_dtype != GBTOPK_F32 && weight_dtype != dtype) return GBTOPK_EUNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if ((rc = check_rows(p.x[i], p.x_row[i], p.x_head[i], tokens > 0)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(p.q_out, p.qo_row, p.qo_head, tokens > 0)) != GBTOPK_OK) return rc;
    if (!aligned_to(p.positions, 4) || !aligned_to(p.slots, 4) || !aligned_to(p.inv_freq, 4) || !aligned_to(p.w[0], 16) ||
        !aligned_to(p.w[1], 16))
        return GBTOPK_EALIGN;
    if (tokens == 0) return GBTOPK_OK;
    const int sms = device_sms();
    if (sms == 0) return GBTOPK_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int wide = weight_dtype == GBTOPK_F32;
    cudaError_t e;
    if (dtype == GBTOPK_BF16)
        e = interleaved ? launch_lanes<true, true>(p, tokens, int4, wide, sms, s) : launch_lanes<true, false>(p, tokens, int4, wide, sms, s);
    else
        e = interleaved ? launch_lanes<false, true>(p, tokens, int4, wide, sms, s) : launch_lanes<false, false>(p, tokens, int4, wide, sms, s);
    return e == cudaSuccess ? GBTOPK_OK : GBTOPK_ECUDA;
}

RotateParams fill(const void *q, int64_t q_row, int64_t q_head, const void *k, int64_t k_row, int64_t k_head, const void *v,
                  int64_t v_row, int64_t v_head, int32_t q_heads, int32_t kv_heads, int32_t dim, const int32_t *positions,
                  const float *inv_freq, int32_t half, const void *wq, const void *wk, float eps, void *q_out, int64_t qo_row,
                  int64_t qo_head, const int32_t *slots, int64_t num_slots) {
    RotateParams p{};
    p.x[0] = q; p.x[1] = k; p.x[2] = v;
    p.x_row[0] = q_row; p.x_row[1] = k_row; p.x_row[2] = v_row;
    p.x_head[0] = q_head; p.x_head[1] = k_head; p.x_head[2] = v_head;
    p.w[0] = wq; p.w[1] = wk;
    p.positions = positions;
    p.slots = slots;
    p.inv_freq = inv_freq;
    p.q_out = q_out;
    p.qo_row = qo_row;
    p.qo_head = qo_head;
    p.num_slots = num_slots;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.dim = dim;
    p.half = half;
    p.eps = eps;
    return p;
}

}  // namespace
}  // namespace gbtopk

using namespace gbtopk;

extern "C" {

int gbtopk_rotate_and_cache(const void *q, int dtype, int64_t num_tokens, int64_t q_row_stride, int64_t q_head_stride,
                            const void *k, int64_t k_row_stride, int64_t k_head_stride, const void *v, int64_t v_row_stride,
                            int64_t v_head_stride, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                            const int32_t *positions, const float *inv_freq, int32_t num_freqs, int interleaved,
                            const void *q_weight, const void *k_weight, int weight_dtype, float eps, void *q_out,
                            int64_t q_out_row_stride, int64_t q_out_head_stride, const int32_t *slots, void *k_cache,
                            int64_t k_slot_stride, int64_t k_cache_head_stride, void *v_cache, int64_t v_slot_stride,
                            int64_t v_cache_head_stride, int64_t num_slots, void *stream) {
    int rc = check_heads(dtype, num_tokens, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if (num_slots < 0) return GBTOPK_EINVAL;
    if (num_slots > INT32_MAX) return GBTOPK_EUNSUPPORTED;
    RotateParams p = fill(q, q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, q_heads,
                          kv_heads, head_dim, positions, inv_freq, num_freqs, q_weight, k_weight, eps, q_out, q_out_row_stride,
                          q_out_head_stride, slots, num_slots);
    if ((rc = check_rows(k_cache, k_slot_stride, k_cache_head_stride, num_slots > 0)) != GBTOPK_OK) return rc;
    if ((rc = check_rows(v_cache, v_slot_stride, v_cache_head_stride, num_slots > 0)) != GBTOPK_OK) return rc;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k_slot = k_slot_stride;
    p.k_head = k_cache_head_stride;
    p.v_slot = v_slot_stride;
    p.v_head = v_cache_head_stride;
    return rotate(p, dtype, num_tokens, weight_dtype, interleaved, false, stream);
}

int gbtopk_rotate_and_cache_int4(const void *q, int dtype, int64_t num_tokens, int64_t q_row_stride, int64_t q_head_stride,
                                 const void *k, int64_t k_row_stride, int64_t k_head_stride, const void *v,
                                 int64_t v_row_stride, int64_t v_head_stride, int32_t q_heads, int32_t kv_heads,
                                 int32_t head_dim, const int32_t *positions, const float *inv_freq, int32_t num_freqs,
                                 int interleaved, const void *q_weight, const void *k_weight, int weight_dtype, float eps,
                                 void *q_out, int64_t q_out_row_stride, int64_t q_out_head_stride, const int32_t *slots,
                                 void *cache, int64_t slot_stride, int64_t head_stride, int64_t num_slots, float k_scale,
                                 float v_scale, void *stream) {
    int rc = check_heads(dtype, num_tokens, q_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if ((rc = check_int4(cache, slot_stride, head_stride, num_slots, head_dim)) != GBTOPK_OK) return rc;
    if (!int4_unit(k_scale) || !int4_unit(v_scale)) return GBTOPK_EINVAL;
    RotateParams p = fill(q, q_row_stride, q_head_stride, k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, q_heads,
                          kv_heads, head_dim, positions, inv_freq, num_freqs, q_weight, k_weight, eps, q_out, q_out_row_stride,
                          q_out_head_stride, slots, num_slots);
    p.k_cache = cache;
    p.k_slot = slot_stride;
    p.k_head = head_stride;
    p.inv_unit[0] = 1.f / k_scale;
    p.inv_unit[1] = 1.f / v_scale;
    return rotate(p, dtype, num_tokens, weight_dtype, interleaved, true, stream);
}

int64_t gbtopk_int4_row_bytes(int32_t head_dim) {
    return head_dim >= 16 && head_dim <= GBTOPK_MAX_HEAD_DIM && head_dim % 16 == 0 ? int4_row(head_dim) : 0;
}

int gbtopk_cache_read_int4(const void *cache, int64_t slot_stride, int64_t head_stride, int64_t num_slots, int32_t kv_heads,
                           int32_t head_dim, const int32_t *slots, int64_t n, float k_scale, float v_scale, int dtype,
                           void *k_out, void *v_out, void *stream) {
    int rc = check_heads(dtype, 0, kv_heads, kv_heads, head_dim);
    if (rc != GBTOPK_OK) return rc;
    if ((rc = check_int4(cache, slot_stride, head_stride, num_slots, head_dim)) != GBTOPK_OK) return rc;
    if (n < 0 || !int4_unit(k_scale) || !int4_unit(v_scale)) return GBTOPK_EINVAL;
    if (n > INT32_MAX) return GBTOPK_EUNSUPPORTED;
    if (n == 0) return GBTOPK_OK;
    if (!slots || !k_out || !v_out) return GBTOPK_EINVAL;
    if (!aligned_to(slots, 4) || !aligned_to(k_out, 16) || !aligned_to(v_out, 16)) return GBTOPK_EALIGN;
    ReadParams p{};
    p.cache = static_cast<const uint8_t *>(cache);
    p.slot_stride = slot_stride;
    p.head_stride = head_stride;
    p.num_slots = num_slots;
    p.unit[0] = k_scale * kInt4Lift;
    p.unit[1] = v_scale * kInt4Lift;
    p.kv_heads = kv_heads;
    p.dim = head_dim;
    p.words.init(static_cast<uint32_t>(head_dim / 8));
    p.heads.init(static_cast<uint32_t>(kv_heads));
    // slots a launch whose words are counted in 31 bits
    const int64_t each = static_cast<int64_t>(kv_heads) * (head_dim / 8), most = (INT32_MAX - 4 * kRowThreads) / each;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (int64_t from = 0; from < n; from += most) {
        p.n = n - from < most ? n - from : most;
        p.slots = slots + from;
        p.out[0] = static_cast<uint8_t *>(k_out) + from * each * 16;
        p.out[1] = static_cast<uint8_t *>(v_out) + from * each * 16;
        const dim3 grid(static_cast<unsigned>((p.n * each + 4 * kRowThreads - 1) / (4 * kRowThreads)), 2);
        const cudaError_t e = dtype == GBTOPK_BF16 ? launch_pdl(read_kernel<true>, grid, kRowThreads, 0, s, 1, p)
                                                   : launch_pdl(read_kernel<false>, grid, kRowThreads, 0, s, 1, p);
        if (e != cudaSuccess) return GBTOPK_ECUDA;
    }
    return GBTOPK_OK;
}

}  // extern "C"
