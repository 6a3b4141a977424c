// Pieces that the attention kernels over 512-value rows share (not part of the C ABI).
#pragma once

#include "operators.h"

namespace fp4idx {

constexpr int kD = 512;
constexpr int kTile = 64;        // entries per step
constexpr int kRow = kD + 16;    // LDS row of a query or an output in 16-bit values (the pad spreads rows over the banks)
constexpr int kPRow = kTile + 8;
constexpr int kQRow = 32;
constexpr float kNone = -3.0e38f;  // reference of a head that has met no entry
constexpr float kRoom = 7.0f;   // the reference lies this far below the largest logit (base 2) when it is set
constexpr float kMost = 15.0f;   // and a logit at most this far above it: probabilities up to 2^15
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __fp16 hv4 __attribute__((vector_size(8)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) hv4 lds_hv4;

__device__ __forceinline__ float ninf() { return -__builtin_inff(); }

// exchanges inside a wavefront without LDS: a value moved by a data-parallel-primitive pattern, and the two lanes
// that lie 16 or 32 apart joined
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max(s[0], s[1]);
}
__device__ __forceinline__ uint32_t max32(uint32_t v) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(s[0], s[1]);
}
// over the four lane groups of a column
__device__ __forceinline__ float group_max(float v) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float group_sum(float v) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ROWS query rows, one after another from `at` on (those past the first `left` as zeros): read by WAVES wavefronts, a row
// per wavefront and step, 8 values per lane; then into LDS as scaled fp16, and per head the factor that turns a dot product
// of theirs into s2.
template <int ROWS, int WAVES = 4>
struct QueryRows {
    uint4 raw[ROWS / WAVES];
};
template <int ROWS, int WAVES = 4>
__device__ __forceinline__ void load_query(const uint16_t* at, int left, QueryRows<ROWS, WAVES>& q) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < ROWS / WAVES; ++i) {
        const int h = w * (ROWS / WAVES) + i, hc = h < left ? h : left - 1;
        q.raw[i] = *reinterpret_cast<const uint4*>(at + hc * kD + lane * 8);
    }
}
template <int ROWS, int WAVES = 4>
__device__ __forceinline__ void stage_query(float scale, int left, QueryRows<ROWS, WAVES>& q, _Float16* lds, float2* factor) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < ROWS / WAVES; ++i) {
        const int row = w * (ROWS / WAVES) + i;
        const uint32_t keep = row < left ? 0xffffffffu : 0u;
        const uint32_t v[4] = {q.raw[i].x & keep, q.raw[i].y & keep, q.raw[i].z & keep, q.raw[i].w & keep};
        us2 two = {0, 0};  // the largest magnitude of each half
#pragma unroll
        for (int c = 0; c < 4; ++c) two = __builtin_elementwise_max(two, __builtin_bit_cast(us2, v[c] & 0x7fff7fffu));
        uint32_t m = max((uint32_t)two[0], (uint32_t)two[1]);
        m = max(m, dpp<0xB1>(m));   // quad_perm [1,0,3,2]
        m = max(m, dpp<0x4E>(m));   // quad_perm [2,3,0,1]
        m = max(m, dpp<0x141>(m));  // row_half_mirror
        m = max(m, dpp<0x140>(m));  // row_mirror
        m = max16(m);
        m = max32(m);
        // 2^(14 - exponent of the largest), a power of two kept inside the normal range. A row that is not finite
        // becomes NaN throughout: an infinity's products may all be -inf, as if nothing had been attended to.
        int e = (int)(m >> 7);
        const bool finite = e < 255;
        e = e < 15 ? 15 : (e > 254 ? 254 : e);
        const float mul = finite ? __uint_as_float((uint32_t)(127 + 141 - e) << 23) : __builtin_nanf("");
        h8 o;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            o[2 * c] = (_Float16)(__uint_as_float(v[c] << 16) * mul);
            o[2 * c + 1] = (_Float16)(__uint_as_float(v[c] & 0xffff0000u) * mul);
        }
        *reinterpret_cast<h8*>(lds + row * kRow + lane * 8) = o;
        // (above zero or below it: a masked entry's product is an infinity of the other sign)
        const float f = scale * kLog2e * __uint_as_float((uint32_t)(e - 14) << 23);
        factor[row] = float2{fabsf(f) < 0x1p-126f ? 0x1p-126f : f, -kNone};
    }
}

// (host) time until the last of n1 blocks of t1 and then n2 of t2 <= t1 ends, each taken by the first of `places` that is free.
inline float time_of(int64_t places, int64_t n1, float t1, int64_t n2, float t2) {
    const int64_t rest = n1 % places;
    const float before = (float)(n1 / places) * t1;
    if (n2 == 0) return before + (rest ? t1 : 0.0f);
    if (rest == 0) return before + (float)((n2 + places - 1) / places) * t2;
    // `rest` places end their long block at t1; the others take short ones from the start
    for (int64_t j = 0;; ++j) {
        const float end = t1 + (float)j * t2;
        const int64_t k = (int64_t)(end / t2);
        if (k * (places - rest) + j * rest < n2) continue;
        const float sooner = (float)k * t2;  // the other places' last one ends before these places' j-th
        const bool enough = j > 0 && sooner >= t1 && k * (places - rest) + (j - 1) * rest >= n2;
        return before + (enough ? sooner : end);
    }
}

}  // namespace fp4idx
