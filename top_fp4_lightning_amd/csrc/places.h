// Where the entries of a cache lie, and the rotary angle of a position: shared by the kernels that write, read and
// attend to cache rows at places of their own (not part of the C ABI).
#pragma once

#include "operators.h"

namespace fp4idx {

// p / d for 0 <= p < 2^30 as a product: with d <= 2^b < 2 d, mul = floor(2^(31+b) / d) + 1 is below 2^32 and exceeds
// 2^(31+b) / d by at most 1, so 2 p mul / 2^(32+b) exceeds p / d by at most p / 2^(31+b) < 1 / (2 d): the floors agree.
inline Division division_by(int64_t d) {
    Division v{0, 0, 0};
    if (d <= 0) return v;  // none: every quotient is 0
    int b = 0;
    while (((int64_t)1 << b) < d) ++b;
    v.by = (uint32_t)d;
    v.mul = (uint32_t)(((uint64_t)1 << (31 + b)) / (uint64_t)d + 1);
    v.shift = b;
    return v;
}
__device__ __forceinline__ uint32_t divided(const Division& d, uint32_t p) { return __umulhi(2 * p, d.mul) >> d.shift; }

// the place of an entry below max_n
__device__ __forceinline__ uint32_t place_of(const Places& a, uint32_t p) { return p - divided(a.ring, p) * a.ring.by; }

// The cache row of entry `at` (any value) of row s of the page table, or from `base` on; -1 where it has none.
__device__ __forceinline__ int64_t row_at(const Places& a, int64_t s, int64_t base, int64_t at) {
    if (at < 0 || at >= a.max_n) return -1;
    const uint32_t p = place_of(a, (uint32_t)at);
    int64_t row;
    if (a.pages) {
        if (s < 0 || s >= a.nseq) return -1;
        const uint32_t column = divided(a.page, p);
        const int32_t page = a.pages[s * a.pages_stride + column];
        if (page < 0) return -1;
        row = (int64_t)page * a.page.by + (p - column * a.page.by);
    } else {
        row = (int64_t)((uint64_t)base + p);  // (a base near the type's ends wraps below 0)
    }
    return row >= 0 && row < a.rows ? row : -1;
}

// pos * freq / 2 pi without its whole turns, in 64 bits: freq / 2 pi with what its rounding leaves, and the product
// with pos without one
__device__ __forceinline__ double turns_of(int64_t pos, double freq) {
    constexpr double kInv2Pi = 0x1.45f306dc9c883p-3, kInv2PiLow = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double p = (double)pos, per = freq * kInv2Pi, low = fma(freq, kInv2Pi, -per) + freq * kInv2PiLow;
    return fma(p, per, -rint(p * per)) + p * low;
}

// sin and cos of t turns, |t| at most about 1/2, to 2^-49: t's quarter turns taken off, then the Taylor series to the 15th
// and 14th power of an angle of at most pi / 4 (the next terms are below 2^-53 and 2^-49)
__device__ __forceinline__ void sincos_turns(double t, double& s, double& c) {
    const double k = rint(4.0 * t), x = fma(k, -0.25, t) * 6.283185307179586477, z = x * x;
    double p = -1.0 / 1307674368000.0, q = -1.0 / 87178291200.0;  // 1 / 15!, 1 / 14!
    p = fma(p, z, 1.0 / 6227020800.0), q = fma(q, z, 1.0 / 479001600.0);
    p = fma(p, z, -1.0 / 39916800.0), q = fma(q, z, -1.0 / 3628800.0);
    p = fma(p, z, 1.0 / 362880.0), q = fma(q, z, 1.0 / 40320.0);
    p = fma(p, z, -1.0 / 5040.0), q = fma(q, z, -1.0 / 720.0);
    p = fma(p, z, 1.0 / 120.0), q = fma(q, z, 1.0 / 24.0);
    p = fma(p, z, -1.0 / 6.0), q = fma(q, z, -0.5);
    const double sx = fma(p * z, x, x), cx = fma(q, z, 1.0);
    const int n = (int)k;  // quarter turns
    s = n & 1 ? cx : sx;
    c = n & 1 ? sx : cx;
    if (n & 2) s = -s;
    if ((n + 1) & 2) c = -c;
}

// The same in fp32, to 2^-23: the series to the 9th and 10th power (the next terms are below 2^-26)
__device__ __forceinline__ void sincos_turns(float t, float& s, float& c) {
    const float k = rintf(4.0f * t), x = fmaf(k, -0.25f, t) * 6.283185307f, z = x * x;
    float p = fmaf(1.0f / 362880.0f, z, -1.0f / 5040.0f), q = fmaf(-1.0f / 3628800.0f, z, 1.0f / 40320.0f);
    p = fmaf(p, z, 1.0f / 120.0f), q = fmaf(q, z, -1.0f / 720.0f);
    p = fmaf(p, z, -1.0f / 6.0f), q = fmaf(q, z, 1.0f / 24.0f);
    q = fmaf(q, z, -0.5f);
    const float sx = fmaf(p * z, x, x), cx = fmaf(q, z, 1.0f);
    const int n = (int)k;  // quarter turns
    s = n & 1 ? cx : sx;
    c = n & 1 ? sx : cx;
    s = __uint_as_float(__float_as_uint(s) ^ ((uint32_t)n << 30 & 0x80000000u));
    c = __uint_as_float(__float_as_uint(c) ^ ((uint32_t)(n + 1) << 30 & 0x80000000u));
}

}  // namespace fp4idx
