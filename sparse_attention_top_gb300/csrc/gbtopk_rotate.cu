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
// two codes (or two scales) than its error, a few in 100,000, makes its warp
// compute the row once more in 64 bits.  So a cache does not depend on the
// order of sums, and two builds agree bit for bit.
//
// Bound by the bytes read and written: 16,001 tokens of 32 + 2 x 8 heads of 128
// move 393 MB in 77 us (75% of the copy rate; the angles, worked out in 64 bits
// once a token, and short rows take the rest).  Into 4 bits the codes bind: 8,192
// tokens of such heads 102 us on the GPU, of which the bytes are 26 and the rows
// in doubt 23; 32,769 slots read back 36 us (25), a word and a scale byte a thread
// and so two loads for 16 bytes out.
#include <cfloat>
#include <cmath>

#include "gbtopk_int4.cuh"

namespace gbtopk {
namespace {

constexpr int kRowThreads = 256;
constexpr int kMostTokens = 8;   // of a block

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
    int64_t num_tokens;
    int32_t tokens, groups;           // of a block
    FastDiv by_half;
    float eps, inv_dim, unit[2], inv_unit[2];
    double inv_dim_wide;
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

// Element i of a word of eight: a whole number of at most 7 in magnitude.
__device__ __forceinline__ uint32_t put_code(int i, float code) {
    const int j = i / 2, m = i & 1 ? 4 * j + 16 : 4 * j, s = i & 1 ? (4 * j + 31) & 31 : 4 * j + 15;
    const uint32_t mag = __float_as_uint(fabsf(code) + 0x1p23f) & 7u, sign = __float_as_uint(code + 0.f) >> 31;   // (-0 is 0)
    return mag << m | sign << s;
}

struct Row {
    uint32_t raw[4];       // the lane's eight elements
    int32_t at;            // the first one's index
    bool there;            // the lane has elements
};

// Sine and cosine of 2 pi x for |x| <= 1/2, off by less than 1e-13: the quarter
// turn nearest to x by its symmetries, the rest, at most pi / 4, by its Taylor
// series up to the 15th power.
__device__ __forceinline__ void turn_wide(double x, double *sine, double *cosine) {
    const double quarter = rint(4 * x), r = (x - 0.25 * quarter) * 6.283185307179586477, z = r * r;
    double s = -1.0 / 1307674368000.0, c = -1.0 / 87178291200.0;
    s = fma(s, z, 1.0 / 6227020800.0);
    c = fma(c, z, 1.0 / 479001600.0);
    s = fma(s, z, -1.0 / 39916800.0);
    c = fma(c, z, -1.0 / 3628800.0);
    s = fma(s, z, 1.0 / 362880.0);
    c = fma(c, z, 1.0 / 40320.0);
    s = fma(s, z, -1.0 / 5040.0);
    c = fma(c, z, -1.0 / 720.0);
    s = fma(s, z, 1.0 / 120.0);
    c = fma(c, z, 1.0 / 24.0);
    s = fma(s, z, -1.0 / 6.0);
    c = fma(c, z, -0.5);
    s = fma(s * z, r, r);
    c = fma(c, z, 1.0);
    const int q = static_cast<int>(quarter) & 3;
    *sine = q == 0 ? s : q == 1 ? c : q == 2 ? -s : -c;
    *cosine = q == 0 ? c : q == 1 ? -s : q == 2 ? -c : s;
}

// Mean squares of 2^-96 .. 2^120 (a NaN is neither) are those whose root 32 bits
// take: no square that counts, and no sum of 256 of them, is beyond their range.
// Other rows' norms are computed in 64 bits (the test costs a long prompt 1.2 of 77 us).
__device__ __forceinline__ bool far_mean(float mean) {
    constexpr uint32_t kLeast = (127u - 96u) << 23, kMost = (127u + 120u) << 23;
    return __float_as_uint(mean) - kLeast >= kMost - kLeast;
}

// A row's mean square and eps in 64 bits, in every lane of its group.
template <int LP>
__device__ __forceinline__ double mean_wide(const RotateParams &p, const float *x) {
    double sum = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) sum = fma(static_cast<double>(x[i]), static_cast<double>(x[i]), sum);
#pragma unroll 1
    for (int o = LP / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    return fma(sum, p.inv_dim_wide, static_cast<double>(p.eps));
}

// 1 / sqrt(v) of a number that 32 bits may not hold: v = m 4^h with 1 <= m < 4, and
// two steps of Newton's method from 22 bits of m's root.
__device__ __noinline__ double root_far(double v) {
    if (!(v > 0 && v <= DBL_MAX)) return rsqrtf(static_cast<float>(v));      // of 0, infinity, NaN
    const int h = (static_cast<int>(static_cast<unsigned long long>(__double_as_longlong(v)) >> 52) - 1023) >> 1;
    const double m = v * __longlong_as_double(static_cast<long long>(1023 - 2 * h) << 52);
    double r = rsqrtf(static_cast<float>(m));
    r = r * fma(-0.5 * m * r, r, 1.5);
    r = r * fma(-0.5 * m * r, r, 1.5);
    return r * __longlong_as_double(static_cast<long long>(1023 - h) << 52);
}

// The lane's eight elements of a query or a 16-bit key once more, where 32 bits do
// not hold the row's mean square.  One row a group of LP lanes; every lane of the
// warp takes part.
template <bool BF16, int LP, bool PAIRS>
__device__ __noinline__ uint4 norm_again(const RotateParams &p, const Row &row, const void *w, bool w_wide, const float2 *turn) {
    const int lane = threadIdx.x & (LP - 1);
    const bool in = row.there && row.at < 2 * p.half, second = !PAIRS && row.at >= p.half;
    const int from = in && !PAIRS ? (second ? lane - p.half / 8 : lane + p.half / 8) : lane;
    float x[8], f[8] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = Half2<BF16>::up(row.raw[i]);
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
    }
    const double r = root_far(mean_wide<LP>(p, x));
    if (row.there) load_weights<BF16>(w, w_wide, row.at, f);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(static_cast<double>(x[i]) * r * f[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = PAIRS ? x[i ^ 1] : __shfl_sync(~0u, x[i], from, LP);
        y[i] = x[i];
        if (in) {
            const float2 cs = turn[PAIRS ? i / 2 : i];
            y[i] = fmaf((PAIRS ? i & 1 : second) ? other : -other, cs.y, x[i] * cs.x);
        }
    }
    return make_uint4(Half2<BF16>::down(y[0], y[1]), Half2<BF16>::down(y[2], y[3]), Half2<BF16>::down(y[4], y[5]), Half2<BF16>::down(y[6], y[7]));
}

// The lane's eight codes and the block's scale once more, where 32 bits leave a
// doubt: word and *byte as stored, in which the elements in doubt (all eight where
// the scale is) are replaced by those of 64 bits.  One row a group of LP lanes;
// every lane of the warp takes part.  Rare (a few in 100,000 elements) and by one
// warp alone at its end, whose time is mostly that of cold instructions (without
// the doubts 2000 tokens would take 33 us, not 50): loops that are not unrolled,
// no division.  An element's angle and rotation are taken in 64 bits only where 32
// bits, with a bound eight times as wide as the one that raised the doubt, find it
// near a border (2000 tokens 50 us a call, all eight elements 53).
template <bool BF16, int LP, bool PAIRS>
__device__ __noinline__ uint32_t encode_again(const RotateParams &p, const Row &row, const void *w, bool w_wide, int32_t position,
                                              const float2 *turn, uint32_t word, uint32_t *byte) {
    const int lane = threadIdx.x & (LP - 1);
    const bool in = row.there && row.at < 2 * p.half, second = !PAIRS && row.at >= p.half;
    const int from = in && !PAIRS ? (second ? lane - p.half / 8 : lane + p.half / 8) : lane;
    float x[8], f[8] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = Half2<BF16>::up(row.raw[i]);
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
    }
    double r = 1;
    bool far = false;
    if (w) {
        const double v = mean_wide<LP>(p, x);
        const float low = static_cast<float>(v) * 0.5f, high = static_cast<float>(v) * 2.f;
        far = far_mean(low) || far_mean(high);      // (32 bits may have found it on the other side)
        r = rsqrtf(static_cast<float>(v));      // two steps of Newton's method from 22 bits
        r = r * fma(-0.5 * v * r, r, 1.5);
        r = r * fma(-0.5 * v * r, r, 1.5);
        if (far) r = root_far(v);
        if (row.there) load_weights<BF16>(w, w_wide, row.at, f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.f;
    }
    // ---- in 32 bits: which elements, and is it the scale
    const float inv_unit = p.inv_unit[0];
    float z[8], terms[8], most = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i] * (static_cast<float>(r) * f[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float other = PAIRS ? x[i ^ 1] * (static_cast<float>(r) * f[i ^ 1]) : __shfl_sync(~0u, x[i] * (static_cast<float>(r) * f[i]), from, LP);
        terms[i] = fabsf(z[i]);
        if (in) {
            const float2 cs = turn[PAIRS ? i / 2 : i];
            terms[i] += fabsf(other);
            z[i] = fmaf((PAIRS ? i & 1 : second) ? other : -other, cs.y, z[i] * cs.x);
        }
        most = fmaxf(most, terms[i]);
        top = fmaxf(top, fabsf(z[i]));
    }
    most = fmaxf(most, __shfl_xor_sync(~0u, most, 1)) * inv_unit;
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1)) * inv_unit;
    float near;
    const float small = block_scale(fminf(top, 4096.f), &near), small_per = small > 0.f ? inv_unit / small : 0.f;
    const bool wide = far || near <= most * 0x1p-17f;     // (all of a far row)
    uint32_t need = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = z[i] * small_per;
        if (wide || fabsf(fabsf(t - rintf(t)) - 0.5f) <= terms[i] * small_per * 0x1p-17f) need |= 1u << i;
    }
    // ---- in 64 bits, an element of every lane where one has it in doubt
    const int32_t k0 = !in ? 0 : PAIRS ? row.at / 2 : row.at - (second ? p.half : 0);
    const uint32_t any = __reduce_or_sync(~0u, need);
    double y[8], tops = 0;
#pragma unroll 1
    for (uint32_t left = any; left; left &= left - 1) {
        const int i = __ffs(static_cast<int>(left)) - 1;
        const double mine = static_cast<double>(x[i]) * r * f[i];
        double v = mine;
        if (p.half) {
            const float ox = PAIRS ? x[i ^ 1] : __shfl_sync(~0u, x[i], from, LP), of = PAIRS ? f[i ^ 1] : __shfl_sync(~0u, f[i], from, LP);
            const double a = position * (static_cast<double>(p.inv_freq[k0 + (PAIRS ? i / 2 : i)]) * 0.15915494309189533577);
            double sine, cosine;
            turn_wide(a - rint(a), &sine, &cosine);
            const double other = static_cast<double>(ox) * r * of;
            if (in) v = fma(mine, cosine, (PAIRS ? i & 1 : second) ? other * sine : -(other * sine));
        }
        y[i] = v * inv_unit;
        tops = fmax(tops, fabs(y[i]));
    }
    double scale = small;
    if (__any_sync(~0u, wide)) {      // (then every element has been taken)
        tops = fmax(tops, __shfl_xor_sync(~0u, tops, 1));
        // as block_scale
        tops = fmin(tops, 4096.0);
        int e = static_cast<int>(static_cast<unsigned long long>(__double_as_longlong(tops * (1.0 / 7.0))) >> 52) - 1023;
        e = e < -6 ? -6 : e;
        const double step = __longlong_as_double(static_cast<long long>(e - 3 + 1023) << 52), steps = __longlong_as_double(static_cast<long long>(3 - e + 1023) << 52);
        const double low = floor(tops * (1.0 / 7.0) * steps), off = tops * steps - 7 * (low + 0.5);
        const bool up = off > 0 || (off == 0 && (static_cast<int>(low) & 1));
        if (wide) {
            scale = fmin((low + (up ? 1 : 0)) * step, 448.0);
            *byte = scale_byte(static_cast<float>(scale));
            if (scale == 0) word = need = 0;
        }
    }
    double per = scale > 0 ? 1.f / static_cast<float>(scale) : 0.f;
    per = per * fma(-scale, per, 2.0);
#pragma unroll 1
    for (uint32_t left = any; left; left &= left - 1) {
        const int i = __ffs(static_cast<int>(left)) - 1;
        double c = rint(y[i] * per);
        const double rest = fma(-c, scale, y[i]);
        if (fabs(rest) == 0.5 * scale) c = 2 * rint(0.5 * (c + copysign(0.5, rest)));
        c = c > 7 ? 7 : c < -7 ? -7 : c == c ? c : 0;
        if ((need >> i) & 1) word = (word & ~put_code(i, -7.f)) | put_code(i, static_cast<float>(c));
    }
    return word;
}

// The same from 32-bit numbers, keys with errors of at most err[i]; *doubt where
// an error could have changed a code or the scale.
template <bool KEYS>
__device__ __forceinline__ uint32_t encode(float *y, const float *err, float unit, float inv_unit, bool wild, uint32_t *byte, bool *doubt) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));   // (a NaN is no maximum)
    top = fmaxf(top, __shfl_xor_sync(~0u, top, 1)) * inv_unit;
    // A NaN is stored as 0.  What lies beyond the largest scale's range comes back
    // to where its code is the largest all the same: its quotient could be infinite,
    // and the correction then a NaN without the number's sign.
    if (__any_sync(~0u, wild || top > 4096.f)) {
        const float most = 4096.f * unit;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] == y[i] ? fminf(fmaxf(y[i], -most), most) : 0.f;
    }
    float near;
    const float steps = block_scale(fminf(top, 4096.f), &near);   // (saturated from 7 * 464 on)
    *byte = scale_byte(steps);
    const float s = steps * unit, per = s > 0.f ? 1.f / s : 0.f;
    constexpr float kWhole = 0x1.8p23f;    // a sum with it is rounded to a whole number
    float border = 1.f, most = 0.f;        // the least of distances from a border less errors, in codes
    float mag[8];
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // The quotient with its one correction is exact on borders (shown for all
        // scales and codes), and away from them by more than it is off: the
        // 16-bit types' own numbers have at most 11 bits, keys their err.
        float t = y[i] * per;
        t = fmaf(fmaf(-t, s, y[i]), per, t);
        const float c = (t + kWhole) - kWhole;
        if constexpr (KEYS) {
            border = fminf(border, err[i] > 0.f ? fmaf(-err[i], per, fabsf(fabsf(t - c) - 0.5f)) : 1.f);
            most = fmaxf(most, err[i]);
        }
        mag[i] = fminf(fabsf(c), 7.f);
        const int j = i / 2, at = i & 1 ? (4 * j + 31) & 31 : 4 * j + 15;
        word |= (__float_as_uint(c) & 0x80000000u) >> (31 - at);
    }
    const float even = fmaf(fmaf(fmaf(mag[6], 16.f, mag[4]), 16.f, mag[2]), 16.f, mag[0]);
    const float odd = fmaf(fmaf(fmaf(mag[7], 16.f, mag[5]), 16.f, mag[3]), 16.f, mag[1]);
    word |= __byte_perm(__float_as_uint(even + 0x1p23f), __float_as_uint(odd + 0x1p23f), 0x5410);
    if constexpr (KEYS) {
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
        *doubt = border <= 0.f || (most > 0.f && near <= most * inv_unit);
    }
    return s > 0.f ? word : 0u;
}

// A block has p.tokens tokens, and of each the head-row groups blockIdx.y *
// p.groups on.  A group is a warp's rows at a time (32 / LP heads of q, of k or
// of v): a warp has one kind of work, whose addresses and weights it keeps while
// it goes through the tokens, four rows in flight.  (With the heads inside and
// the tokens outside, 16,001 tokens of 32 over 8 heads took 94 us, most of it
// address arithmetic.)
template <bool BF16, int LP, bool PAIRS, bool INT4>
__global__ void __launch_bounds__(kRowThreads, 4) rotate_kernel(const __grid_constant__ RotateParams p, int w_wide) {
    constexpr int kRows = 32 / LP;         // of a group
    constexpr int kAhead = 4;
    extern __shared__ float2 turns[];      // [tokens][half]: cosine and sine
    __shared__ int32_t slots[kMostTokens];
    pdl_wait();
    pdl_release();
    const int64_t token0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
    const int32_t tokens = static_cast<int32_t>(p.num_tokens - token0 < p.tokens ? p.num_tokens - token0 : p.tokens);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & (LP - 1), sub = (threadIdx.x & 31) / LP;
    const int32_t gq = (p.q_heads + kRows - 1) / kRows, gk = (p.kv_heads + kRows - 1) / kRows;
    const int32_t at = lane * 8, rotary = 2 * p.half;
    const int32_t end = gq + 2 * gk < (static_cast<int32_t>(blockIdx.y) + 1) * p.groups ? gq + 2 * gk : (static_cast<int32_t>(blockIdx.y) + 1) * p.groups;
    if (static_cast<int32_t>(threadIdx.x) < tokens) slots[threadIdx.x] = p.slots[token0 + threadIdx.x];
    bool bad = false;      // some angle is a NaN
    for (int k = threadIdx.x; k < tokens * p.half; k += kRowThreads) {
        const int32_t t = static_cast<int32_t>(p.by_half.div(static_cast<uint32_t>(k)));
        const double a = static_cast<double>(p.positions[token0 + t]) * (static_cast<double>(p.inv_freq[k - t * p.half]) * 0.15915494309189533577);
        float s, c;
        const double rest = a - rint(a);
        const float near = static_cast<float>(rest), off = static_cast<float>(rest - near) * 6.2831853f;
        sincospif(2.f * near, &s, &c);
        turns[k] = make_float2(fmaf(-s, off, c), fmaf(c, off, s));     // (what the 32-bit turns leave out)
        if constexpr (INT4) bad |= !(fabsf(near) <= 0.5f);
    }
    if constexpr (INT4) bad = __syncthreads_or(bad);
    else __syncthreads();
    // the lane's partner in the rotation, its angles, the sign of its sine
    const bool in = at < rotary, second = !PAIRS && at >= p.half;
    const int from = in ? (second ? lane - p.half / 8 : lane + p.half / 8) : lane;
    const float2 *mine = turns + (!in ? 0 : PAIRS ? at / 2 : at - (second ? p.half : 0));

    for (int32_t g = static_cast<int32_t>(blockIdx.y) * p.groups + warp; g < end; g += kRowThreads / 32) {
        const int kind = g < gq ? 0 : g < gq + gk ? 1 : 2;
        const int32_t head = (g - (kind == 0 ? 0 : gq + (kind - 1) * gk)) * kRows + sub;
        const bool there = at < p.dim && head < (kind == 0 ? p.q_heads : p.kv_heads);
        const uint8_t *src = static_cast<const uint8_t *>(p.x[kind]) + 2 * (token0 * p.x_row[kind] + (there ? head * p.x_head[kind] + at : 0));
        const int64_t step = 2 * p.x_row[kind];
        // (16-bit caches: rows of k or v; 4-bit ones: bytes of the row)
        uint8_t *dst;
        int64_t dst_step;
        if (kind == 0) {
            dst = static_cast<uint8_t *>(p.q_out) + 2 * (token0 * p.qo_row + head * p.qo_head + at);
            dst_step = 2 * p.qo_row;
        } else if (INT4) {
            dst = static_cast<uint8_t *>(p.k_cache) + head * p.k_head + (kind - 1) * int4_codes(p.dim) + at / 2;
            dst_step = p.k_slot;
        } else {
            dst = static_cast<uint8_t *>(kind == 1 ? p.k_cache : p.v_cache) + 2 * (head * (kind == 1 ? p.k_head : p.v_head) + at);
            dst_step = 2 * (kind == 1 ? p.k_slot : p.v_slot);
        }
        const void *w = kind < 2 ? p.w[kind] : nullptr;
        float f[8];
        bool wild = bad;          // some weight or angle is a NaN: some of the keys may be
        if (w && there) {
            load_weights<BF16>(w, w_wide != 0, at, f);
            if constexpr (INT4) {
#pragma unroll
                for (int j = 0; j < 8; ++j) wild |= f[j] != f[j];
            }
        }
        uint32_t again = 0;       // tokens whose row of this lane needs 64 bits
        for (int32_t t0 = 0; t0 < tokens; t0 += kAhead) {
            uint4 raw[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                raw[u] = there && t0 + u < tokens ? *reinterpret_cast<const uint4 *>(src + (t0 + u) * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t t = t0 + u;
                if (t >= tokens) break;
                const int32_t slot = kind > 0 ? slots[t] : t;
                if (kind > 0 && (slot < 0 || slot >= p.num_slots)) continue;
                uint8_t *to = dst + slot * dst_step;
                if (kind == 2 && !INT4) {      // as they are
                    if (there) *reinterpret_cast<uint4 *>(to) = raw[u];
                    continue;
                }
                const uint32_t v[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
                float y[8], pair[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 z = Half2<BF16>::up(v[j]);
                    y[2 * j] = z.x;
                    y[2 * j + 1] = z.y;
                    pair[j] = fmaf(z.x, z.x, z.y * z.y);
                }
                float sum = (pair[0] + pair[1]) + (pair[2] + pair[3]);
                bool far = false;
                if (w) {
                    for (int o = LP / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                    const float mean = fmaf(sum, p.inv_dim, p.eps);
                    far = far_mean(mean);
                    if (far) again |= 1u << t;
                    float r = rsqrtf(mean);
                    if (INT4 && kind == 1) r = fmaf(0.5f * r, fmaf(-mean * r, r, 1.f), r);    // (a step of Newton's method)
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= r * f[j];
                }
                // Relative errors of a key, in units of 2^-24: the sum 9, its mean 2, both
                // halved by the root; the refined root 2, the products 2; sine and cosine
                // 2; the rotation 2.  2^-20 of an element's terms is more than all of it.
                float err[8];
                if constexpr (INT4) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) err[j] = w ? fabsf(y[j]) * 0x1p-20f : 0.f;
                }
                if (kind < 2 && rotary) {
                    const float2 *turn = mine + t * p.half;
                    if constexpr (PAIRS) {
                        if (in) {
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                const float2 cs = turn[j / 2];
                                const float a = y[j], b = y[j + 1];
                                y[j] = a * cs.x - b * cs.y;
                                y[j + 1] = b * cs.x + a * cs.y;
                                if constexpr (INT4) err[j] = err[j + 1] = (fabsf(a) + fabsf(b)) * 0x1p-20f;
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float other = __shfl_sync(~0u, y[j], from, LP);
                            const float2 cs = turn[j];
                            if constexpr (INT4) err[j] = in ? (fabsf(y[j]) + fabsf(other)) * 0x1p-20f : err[j];
                            y[j] = in ? fmaf(second ? other : -other, cs.y, y[j] * cs.x) : y[j];
                        }
                    }
                }
                if (!INT4 || kind == 0) {
                    if (there && !far)      // (q may be q_out: its row is read again)
                        *reinterpret_cast<uint4 *>(to) = make_uint4(Half2<BF16>::down(y[0], y[1]), Half2<BF16>::down(y[2], y[3]),
                                                                    Half2<BF16>::down(y[4], y[5]), Half2<BF16>::down(y[6], y[7]));
                } else if constexpr (INT4) {
                    uint32_t byte;
                    bool doubt = false;
                    const bool odd = wild || !(sum < INFINITY);
                    const float unit = p.unit[kind - 1], inv_unit = p.inv_unit[kind - 1];
                    const uint32_t word = kind == 1 ? encode<true>(y, err, unit, inv_unit, odd, &byte, &doubt)
                                                    : encode<false>(y, err, unit, inv_unit, odd, &byte, &doubt);
                    if (there) {
                        *reinterpret_cast<uint32_t *>(to) = word;
                        // (the scales lie behind both codes)
                        if (!(lane & 1))
                            to[(3 - kind) * int4_codes(p.dim) - at / 2 + (kind - 1) * int4_scales(p.dim) + at / 16] = static_cast<uint8_t>(byte);
                    }
                    if (doubt && there) again |= 1u << t;
                }
            }
        }
        // (behind the loop, whose registers it would take)
#pragma unroll 1
        for (uint32_t left = __reduce_or_sync(~0u, there ? again : 0); left; left &= left - 1) {
            const int32_t t = __ffs(static_cast<int>(left)) - 1;
            Row row;
            row.at = at;
            row.there = there;
            const uint4 v = there ? *reinterpret_cast<const uint4 *>(src + t * step) : make_uint4(0, 0, 0, 0);
            row.raw[0] = v.x;
            row.raw[1] = v.y;
            row.raw[2] = v.z;
            row.raw[3] = v.w;
            const float2 *turn = mine + t * p.half;
            if constexpr (INT4) {
                if (kind > 0) {      // (keys: only they have doubts)
                    uint8_t *to = dst + slots[t] * dst_step, *to_scale = to + 2 * int4_codes(p.dim) - at / 2 + at / 16;
                    uint32_t byte = there ? *to_scale : 0;
                    const uint32_t word = encode_again<BF16, LP, PAIRS>(p, row, w, w_wide != 0, p.half ? p.positions[token0 + t] : 0, turn,
                                                                        there ? *reinterpret_cast<uint32_t *>(to) : 0, &byte);
                    if (there) {
                        *reinterpret_cast<uint32_t *>(to) = word;
                        if (!(lane & 1)) *to_scale = static_cast<uint8_t>(byte);
                    }
                    continue;
                }
            }
            const uint4 y = norm_again<BF16, LP, PAIRS>(p, row, w, w_wide != 0, turn);
            if (there && ((again >> t) & 1)) *reinterpret_cast<uint4 *>(dst + (kind > 0 ? slots[t] : t) * dst_step) = y;
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
    const int32_t per = 32 / LP, warps = kRowThreads / 32;
    const int32_t groups = (p.q_heads + per - 1) / per + 2 * ((p.kv_heads + per - 1) / per);
    // As many tokens a block as leave every SM four blocks (16,001 tokens: 78 us, a
    // token a block 152; 8,192 into 4 bits and read back 143, 164); a token's groups
    // spread over blocks (each of which works its angles out again) where even two
    // blocks a SM are not there (256 tokens 18.6 us a call, in one block each 20.8).
    p.num_tokens = tokens;
    const int64_t fair = tokens / (4ll * sms);
    p.tokens = fair >= kMostTokens ? kMostTokens : fair > 1 ? static_cast<int32_t>(fair) : 1;
    p.groups = tokens < 2ll * sms && groups > warps ? warps : groups;
    p.by_half.init(static_cast<uint32_t>(p.half > 0 ? p.half : 1));
    const dim3 grid(static_cast<unsigned>((tokens + p.tokens - 1) / p.tokens), static_cast<unsigned>((groups + p.groups - 1) / p.groups));
    const size_t bytes = static_cast<size_t>(p.tokens) * p.half * sizeof(float2);
    return int4 ? launch_pdl(rotate_kernel<BF16, LP, PAIRS, true>, grid, kRowThreads, bytes, s, 1, p, w_wide)
                : launch_pdl(rotate_kernel<BF16, LP, PAIRS, false>, grid, kRowThreads, bytes, s, 1, p, w_wide);
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
    p.inv_dim = 1.f / static_cast<float>(dim > 0 ? dim : 1);
    p.inv_dim_wide = 1.0 / (dim > 0 ? dim : 1);
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
    p.unit[0] = k_scale;
    p.unit[1] = v_scale;
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
