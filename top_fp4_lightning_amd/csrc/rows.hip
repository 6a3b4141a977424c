// Rows written to and read from their places in a cache.
//
// Writing: y = x, normalised (x gamma / sqrt(mean x^2 + eps)), turned by its position, then quantised in the cache's
// format and stored in the row of its entry. One pass: a lane holds 16 values, a row of 512 takes 32 lanes, a key of 128
// eight; a rotated pair is a lane's (its angle, sine and cosine, both values).
//
// Which code a value gets turns on the side of a border it lies on, so everything up to that is in 64 bits, and what is
// compared in fp32 is a value cut to 20 bits behind the leading one, the last of them set where something was cut off
// (rounded to odd). It lies on the same side as the exact one of every number of fewer bits, and a border has at most 7.
//
// Reading: the stored values (a code times a scale is exact in fp32 and bf16), turned in fp32, rounded once.
//
// Under the tracer, writing takes 18 us for 32770 fp32 rows of the main KV, turned (76 MB at 4.3 TB/s), 13 for 16384 bf16 rows
// of local positions, normalised and turned, 18 for 65537 keys: vector instructions fill two thirds to nine tenths of the time,
// 24, 32 and 58 a value, a third of a key's for its pairs' sines and cosines. A fifth block on a compute unit changes nothing.
// Reading them takes 12, 7 and 6 us. One row 3.2 and 1.9 us: launch, three loads one behind the other.
#include "../../include/fp4idx.h"
#include <type_traits>

#include "lanes.h"
#include "places.h"

namespace fp4idx {
namespace {

template <int FMT>
struct Format;
template <>
struct Format<IDX_ROWS_MAIN> {
    static constexpr int kDim = 512, kGroup = 16;
};
template <>
struct Format<IDX_ROWS_LOCAL> {
    static constexpr int kDim = 512, kGroup = 32;
};
template <>
struct Format<IDX_ROWS_KEY> {
    static constexpr int kDim = 128, kGroup = 32;
};

__device__ __forceinline__ float bf16f(uint32_t h) { return __uint_as_float(h << 16); }

// A 64-bit value as fp32, rounded to odd behind 20 bits: its high word with the last bit set for what lies behind, the
// exponent moved (the largest and smallest numbers where fp32 has none)
__device__ __forceinline__ float to_odd(double y) {
    const uint64_t b = (uint64_t)__double_as_longlong(y);
    const uint32_t hi = (uint32_t)(b >> 32), lo = (uint32_t)b;
    uint32_t h = (hi & 0x7fffffffu) | min(lo, 1u);
    h = min(max(h, (896u << 20) + min(h, 1u)), (1151u << 20) - 1u);
    return __uint_as_float(((h - (896u << 20)) << 3) | (hi & 0x80000000u));
}
__device__ __forceinline__ float to_odd(float y) {
    const uint32_t b = __float_as_uint(y);
    return __uint_as_float((b | ((b & 7u) + 7u)) & 0xfffffff8u);
}

// The same where a value below fp32's smallest may become zero, and one above its largest an infinity
__device__ __forceinline__ float to_odd_local(double y) {
    const uint64_t b = (uint64_t)__double_as_longlong(y);
    const uint32_t hi = (uint32_t)(b >> 32) | min((uint32_t)b, 1u);
    return (float)__longlong_as_double((long long)((uint64_t)hi << 32));
}
template <int FMT, typename T>
__device__ __forceinline__ float odd(T y) {
    if constexpr (FMT == IDX_ROWS_LOCAL && sizeof(T) == 8)
        return to_odd_local(y);
    else
        return to_odd(y);
}

__device__ __forceinline__ bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// 16 values of a row of x from the place `at` on, as they lie: 8 words of bf16 or 16 of fp32, whole pieces or one by one
struct Raw {
    uint32_t w[16];
};
template <bool F32>
__device__ __forceinline__ void load16(const RowsArgs& a, int64_t row, int at, Raw& r) {
    const int64_t place = row * a.stride + at;
    if (a.wide) {
        const uint4* x = reinterpret_cast<const uint4*>((const uint8_t*)a.x + place * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32 ? 4 : 2); ++i) {
            const uint4 u = x[i];
            r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
        }
    } else if (F32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) r.w[i] = ((const uint32_t*)a.x)[place + i];
    } else {
        const uint16_t* x = (const uint16_t*)a.x + place;
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = x[2 * i] | (uint32_t)x[2 * i + 1] << 16;
    }
}
template <bool F32>
__device__ __forceinline__ void values16(const Raw& r, float (&f)[16]) {
    if (F32) {
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[2 * i] = __uint_as_float(r.w[i] << 16);
            f[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    }
}

// value of an E4M3 byte below 0x7f
__device__ __forceinline__ float e4m3_of(uint32_t b) {
    const uint32_t e = b >> 3, m = b & 7u;
    return e == 0 ? (float)m * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}
// Smallest E4M3 byte whose value s has 6 s >= a (a >= 0); 0x7e (448) at most. A sixth of a, less 2^-22 of it, is rounded up
// to three bits behind the leading one (steps of 2^-9 below 2^-6): that is the byte or the one before it.
__device__ __forceinline__ uint32_t e4m3_scale_for(float a) {
    const float t = a * (0x1.555554p-3f * (1.0f - 0x1p-22f));
    const uint32_t b = t < 0x1p-6f ? (uint32_t)ceilf(t * 512.0f) : (__float_as_uint(t) - (120u << 23) + 0xfffffu) >> 20;
    const uint32_t c = min(b, 0x7eu);
    return min(c + (6.0f * e4m3_of(c) < a ? 1u : 0u), 0x7eu);
}

// E2M1 codes of 8 values of at most 6 in magnitude; zero has no sign
__device__ __forceinline__ uint32_t e2m1_codes(const float* q) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[0], q[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[2], q[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[4], q[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, q[6], q[7], 1.0f, 3);
    const uint32_t some = ((w & 0x77777777u) + 0x77777777u) & 0x88888888u;
    return w & (some | 0x77777777u);
}

// smallest e in [lo, hi] with 7/4 2^(e + B) >= a or 3/2 2^(e + B) >= a: 448 = 1.75 2^8, 6 = 1.5 2^2
__device__ __forceinline__ int scale_exponent(float a, float most, int bits, int lo, int hi) {
    int E;
    const float m = frexpf(a, &E);  // a = m 2^E, 0.5 <= m < 1
    int e = E - bits + (m > most ? 1 : 0);
    e = a == 0.0f ? lo : e;
    return e < lo ? lo : (e > hi ? hi : e);
}

template <int FMT, bool F32, bool NORM>
__global__ __launch_bounds__(256) void write_rows_kernel(const RowsArgs a) {
    typedef Format<FMT> F;
    constexpr int kLanes = F::kDim / 16, kRows = 256 / kLanes;  // of a row; of a block
    constexpr bool kKey = FMT == IDX_ROWS_KEY;
    typedef std::conditional_t<kKey, double, float> Part;  // keys go on in 64 bits
    // The turned part on its way to the lanes of pairs and back: value e at e + kPad (e / 16), so that lanes' sixteens and
    // rows lie in different banks (without, 65537 keys took 20.9 us).
    constexpr int kPad = kKey ? 2 : 4, kWidth = F::kDim + kLanes * kPad + (kKey ? 2 : 0);
    __shared__ __align__(16) Part s_part[kRows][kWidth];
    const auto part = [](int e) { return e + (e >> 4) * kPad; };
    const int li = threadIdx.x % kLanes, r = threadIdx.x / kLanes;
    const int64_t t = (int64_t)blockIdx.x * kRows + r;
    const bool live = t < a.tokens;
    const int64_t tc = live ? t : a.tokens - 1;
    const int rot = a.turn.rot, pairs = a.turn.freq ? rot / 2 : 0, offset = a.turn.offset;
    Raw raw;
    load16<F32>(a, tc, 16 * li, raw);
    const int64_t at = a.at[tc], keep = a.keep ? a.keep[tc] : 0;
    constexpr int kAhead = kKey ? 4 : 1;  // pairs of a lane whose frequencies are read ahead
    double freq[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) freq[i] = li + i * kLanes < pairs ? a.turn.freq[li + i * kLanes] : 0.0;
    uint4 signs{};
    if constexpr (kKey) signs = reinterpret_cast<const uint4*>(a.signs)[li];
    int64_t row = row_at(a.places, a.places.seq ? a.places.seq[tc] : tc, a.places.base ? a.places.base[tc] : 0, at);
    if (!live || keep < 0) row = -1;
    // this lane's values among the turned ones: first .. last - 1
    const int first = pairs ? max(offset - 16 * li, 0) : 16, last = pairs ? min(offset + rot - 16 * li, 16) : 16;
    float f[16];
    values16<F32>(raw, f);

    double by = 1.0;
    float gamma[16];
    if (NORM) {
        if (a.gamma && aligned16(a.gamma)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 u = reinterpret_cast<const float4*>(a.gamma + 16 * li)[i];
                gamma[4 * i] = u.x, gamma[4 * i + 1] = u.y, gamma[4 * i + 2] = u.z, gamma[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) gamma[i] = a.gamma ? a.gamma[16 * li + i] : 1.0f;
        }
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            sum = fma((double)f[i], (double)f[i], sum);
            if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
        }
        // (the values are widened again below, not kept in 64 bits: registers)
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+v"(f[i]));
        sum += xor_lane<1>(sum, li);
        sum += xor_lane<2>(sum, li);
        sum += xor_lane<4>(sum, li);
        if constexpr (kLanes == 32) {
            sum += xor_lane<8>(sum, li);
            sum += xor_lane<16>(sum, li);
        }
        // 1 / sqrt by the instruction's approximation (2^-23 or better) and two of Newton's steps
        const double mean = fmax(fma(sum, 1.0 / F::kDim, a.eps), 0x1p-1020);
        by = __builtin_amdgcn_rsq(mean);
#pragma unroll
        for (int i = 0; i < 2; ++i) by = fma(by * 0.5, fma(-mean * by, by, 1.0), by);
    }
    const auto normal = [&](int i) {
        return (double)f[i] * by * (double)gamma[i];
    };
    double y[kKey ? 16 : 1];
    if constexpr (kKey) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = NORM ? normal(i) : (double)f[i];
    }
    if (pairs) {
        if (first < last) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if constexpr (kKey)
                    s_part[r][(16 + kPad) * li + i] = y[i];
                else
                    s_part[r][(16 + kPad) * li + i] = f[i];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (a row is one wavefront's)
        __builtin_amdgcn_wave_barrier();
        const int64_t pos = a.turn.pos ? a.turn.pos[tc] : at;
        const auto turned = [&](int p, double per) {
            double s, c;
            sincos_turns(turns_of(pos, per), s, c);
            if (a.turn.mscale != 1.0) s *= a.turn.mscale, c *= a.turn.mscale;
            const int i0 = offset + (a.turn.half ? p : 2 * p), i1 = i0 + (a.turn.half ? pairs : 1);
            Part& at0 = s_part[r][part(i0)];
            Part& at1 = s_part[r][part(i1)];
            double x0 = at0, x1 = at1;
            if (NORM && !kKey) {
                x0 *= by, x1 *= by;
                if (a.gamma) x0 *= (double)a.gamma[i0], x1 *= (double)a.gamma[i1];
            }
            const double y0 = x0 * c - x1 * s, y1 = x1 * c + x0 * s;
            if constexpr (kKey)
                at0 = y0, at1 = y1;
            else
                at0 = odd<FMT>(y0), at1 = odd<FMT>(y1);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (li + i * kLanes < pairs) turned(li + i * kLanes, freq[i]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll 1
        for (int p = li + kAhead * kLanes; p < pairs; p += kLanes) turned(p, a.turn.freq[p]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }

    int place = li;  // which sixteen of the row this lane holds in the end
    if constexpr (kKey) {
        if (first == 0 && last == 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = s_part[r][(16 + kPad) * li + i];
        } else if (first < last) {
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = i >= first && i < last ? s_part[r][(16 + kPad) * li + i] : y[i];
        }
        // the signs, the transform in 64 bits, then fl32(S) fl32(2^-3.5) in fp32
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t word = i < 4 ? signs.x : i < 8 ? signs.y : i < 12 ? signs.z : signs.w;
            const uint64_t minus = (uint64_t)((word << (24 - 8 * (i & 3))) & 0x80000000u) << 32;
            y[i] = __longlong_as_double((long long)((uint64_t)__double_as_longlong(y[i]) ^ minus));
        }
#pragma unroll
        for (int b = 1; b < 16; b <<= 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (!(i & b)) {
                    const double p = y[i], q = y[i | b];
                    y[i] = p + q;
                    y[i | b] = p - q;
                }
            }
        }
        // Over the eight lanes by exchanges with l ^ 1, l ^ 2 and l ^ 7 (a mirror, one instruction; l ^ 4 takes three). As a
        // basis they are as good: with l = a 1 + b 2 + c 7, a = l0 + l2, b = l1 + l2, c = l2, the sums over a, b and c leave
        // in lane l the sixteen of index L with L0 = a, L1 = b, L0 + L1 + L2 = c: L2 = l0 + l1 + l2 (all modulo 2).
        const int l0 = li & 1, l1 = li >> 1 & 1, l2 = li >> 2;
        const auto stage = [&](double other, double mine, int upper) { return fma(mine, upper ? -1.0 : 1.0, other); };
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = stage(xor_lane<1>(y[i], li), y[i], l0 ^ l2);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = stage(xor_lane<2>(y[i], li), y[i], l1 ^ l2);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = stage(mirror8(y[i]), y[i], l2);
        place = (l0 ^ l2) | (l1 ^ l2) << 1 | (l0 ^ l1 ^ l2) << 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = (float)y[i] * 0x1.6a09e6p-4f;  // fl32(2^-3.5)
    } else {
        if (NORM) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                f[i] = odd<FMT>(normal(i));
                if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // (few 64-bit values at a time: registers)
            }
        } else if (F32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = odd<FMT>(f[i]);
        }
        if (first == 0 && last == 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = s_part[r][(16 + kPad) * li + i];
        } else if (first < last) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = i >= first && i < last ? s_part[r][(16 + kPad) * li + i] : f[i];
        }
    }

    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(f[i]));
    // (a key's other half of a group is in lane l ^ 6: of l ^ 2 and l ^ 4, L0 alone changes)
    if constexpr (kKey) top = fmaxf(top, mirror8f(xor_lanef<1>(top, li)));
    if constexpr (FMT == IDX_ROWS_LOCAL) top = fmaxf(top, xor_lanef<1>(top, li));
    constexpr int kGroupLanes = F::kGroup / 16, kScales = F::kDim / F::kGroup;
    uint32_t scale;
    if constexpr (FMT == IDX_ROWS_LOCAL) {
        const int e = scale_exponent(fminf(top, 0x1.fffffep127f), 0.875f, 9, IDX_LOCAL_MIN_EXP, IDX_LOCAL_MAX_EXP);
        scale = (uint32_t)(e + 127);
        const float by_e = __uint_as_float((uint32_t)(127 - e) << 23);
        // (a value that leaves fp32's normal range on the way lies far below half of the smallest code)
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = __builtin_amdgcn_fmed3f(f[i] * by_e, -448.0f, 448.0f);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
            b = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], b, true);
            const uint32_t some = (((uint32_t)b & 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u;
            w[i] = (uint32_t)b & (some | 0x7f7f7f7fu);  // zero has no sign
        }
        if (row >= 0) *reinterpret_cast<uint4*>(a.codes + row * 512 + 16 * li) = uint4{w[0], w[1], w[2], w[3]};
    } else {
        float q[16];
        if constexpr (FMT == IDX_ROWS_MAIN) {
            scale = e4m3_scale_for(top);
            const float s = e4m3_of(scale), inv = s > 0.0f ? 1.0f / s : 0.0f;
            // Quotients by a product with 1 / s, off by 2^-23 of themselves at most, then rounded to 21 bits behind
            // the leading one: on a border where the value is on it (half a step there is 1.14 2^-23), and on the
            // value's side of it where it is not (it lies 2^-21 off at least, a border's neighbours are 2^-22 off
            // at most).
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = __builtin_amdgcn_fmed3f(f[i] * inv, -6.0f, 6.0f);
                q[i] = __uint_as_float((__float_as_uint(x) + 2u) & 0xfffffffcu);
            }
        } else {
            const int e = scale_exponent(top, 0.75f, 3, -127, 127);
            scale = (uint32_t)(e + 127);
#pragma unroll
            for (int i = 0; i < 16; ++i) q[i] = ldexpf(f[i], -e);
        }
        const uint2 words{e2m1_codes(q), e2m1_codes(q + 8)};
        if (row >= 0) *reinterpret_cast<uint2*>(a.codes + row * (F::kDim / 2) + 8 * place) = words;
    }
    if (row >= 0 && place % kGroupLanes == 0) a.scales[row * kScales + place / kGroupLanes] = (uint8_t)scale;
}

constexpr int kReadAngles = 256;  // a wavefront's table

// kReads: rows of a lane, their reads in flight together
template <int FMT, int kReads>
__global__ __launch_bounds__(256) void read_rows_kernel(const RowsArgs a) {
    typedef Format<FMT> F;
    constexpr bool kKey = FMT == IDX_ROWS_KEY;
    constexpr int kLanes = F::kDim / 8, kSide = 64 / kLanes;  // of a row; rows side by side in a wavefront
    constexpr int kGroupLanes = F::kGroup / 8, kScales = F::kDim / F::kGroup;
    __shared__ __align__(16) float2 s_cs[kKey ? 1 : 4][kReadAngles];
    __shared__ __align__(16) float s_y[kKey ? 1 : 4][F::kDim];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, li = lane % kLanes;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + w) * (kSide * kReads) + lane / kLanes;
    if (t0 - lane / kLanes >= a.tokens) return;  // the whole wavefront (no barrier below)
    int64_t at[kReads], row[kReads];
#pragma unroll
    for (int k = 0; k < kReads; ++k) at[k] = a.at[min(t0 + k * kSide, a.tokens - 1)];
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
        const int64_t t = min(t0 + k * kSide, a.tokens - 1);
        row[k] = row_at(a.places, a.places.seq ? a.places.seq[t] : t, a.places.base ? a.places.base[t] : 0, at[k]);
    }
    uint2 code[kReads];
    uint32_t sb[kReads];
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
        code[k] = uint2{0, 0};
        sb[k] = 0;
        if (row[k] >= 0) {
            sb[k] = a.scales[row[k] * kScales + li / kGroupLanes];
            if constexpr (FMT == IDX_ROWS_LOCAL)
                code[k] = *reinterpret_cast<const uint2*>(a.codes + row[k] * 512 + 8 * li);
            else
                code[k].x = reinterpret_cast<const uint32_t*>(a.codes + row[k] * (F::kDim / 2))[li];
        }
    }
    const int rot = a.turn.rot, pairs = !kKey && a.turn.freq ? rot / 2 : 0, offset = a.turn.offset;
    const float m = (float)a.turn.mscale;
    const auto angle = [&](int64_t t, int64_t entry, int p) {
        float s, c;
        sincos_turns((float)turns_of(a.turn.pos ? a.turn.pos[t] : entry, a.turn.freq[p]), s, c);
        return float2{c * m, (a.turn.inverse ? -s : s) * m};
    };
    // angles of all the rows at once where they are few
    const bool all = kReads * pairs <= kReadAngles;
    if (pairs && all) {
        // i / pairs as a product: i below 256, the factor above 2^16 / pairs by at most 1
        const uint32_t by = (1u << 16) / (uint32_t)pairs + 1;
        for (uint32_t i = lane; i < (uint32_t)(kReads * pairs); i += 64) {
            const uint32_t k = i * by >> 16;
            const int64_t t = min(t0 + k, a.tokens - 1);
            s_cs[kKey ? 0 : w][i] = angle(t, a.at[t], (int)(i - k * pairs));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
        const int64_t t = t0 + k * kSide;
        float y[8];
        if constexpr (FMT == IDX_ROWS_LOCAL) {
            const float s = ldexpf(1.0f, (int)sb[k] - 127);
            const uint32_t ws[2] = {code[k].x, code[k].y};
            typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f2 u = __builtin_amdgcn_cvt_pk_f32_fp8((int)ws[i], false), v = __builtin_amdgcn_cvt_pk_f32_fp8((int)ws[i], true);
                y[4 * i] = u[0] * s, y[4 * i + 1] = u[1] * s, y[4 * i + 2] = v[0] * s, y[4 * i + 3] = v[1] * s;
            }
        } else {
            float s;
            if constexpr (FMT == IDX_ROWS_MAIN)
                s = sb[k] & 0x80u ? -e4m3_of(sb[k] & 0x7fu) : e4m3_of(sb[k]);
            else
                s = ldexpf(1.0f, (int)sb[k] - 127);
            typedef float f2 __attribute__((ext_vector_type(2)));
            const f2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k].x, 1.0f, 0),
                             __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k].x, 1.0f, 1),
                             __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k].x, 1.0f, 2),
                             __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code[k].x, 1.0f, 3)};
#pragma unroll
            for (int i = 0; i < 4; ++i) y[2 * i] = v[i][0] * s, y[2 * i + 1] = v[i][1] * s;
        }
        if (row[k] < 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        }
        if constexpr (!kKey) {
            if (pairs) {
                const float2* cs = s_cs[w] + (all ? k * pairs : 0);
                const bool apart = a.turn.half || (offset & 1);  // a pair's values lie with two lanes
                if (!all || apart) {
                    if (!all) {
                        for (int p = lane; p < pairs; p += 64) s_cs[w][p] = angle(min(t, a.tokens - 1), at[k], p);
                    }
                    *reinterpret_cast<float4*>(s_y[w] + 8 * li) = float4{y[0], y[1], y[2], y[3]};
                    *reinterpret_cast<float4*>(s_y[w] + 8 * li + 4) = float4{y[4], y[5], y[6], y[7]};
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
                const int j0 = 8 * li - offset;
                if (j0 > -8 && j0 < rot) {
                    if (!apart && !((offset | rot) & 7)) {  // whole lanes
                        const float4 z[2] = {reinterpret_cast<const float4*>(cs)[j0 >> 2],
                                             reinterpret_cast<const float4*>(cs)[(j0 >> 2) + 1]};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float c = i & 1 ? z[i >> 1].z : z[i >> 1].x, d = i & 1 ? z[i >> 1].w : z[i >> 1].y;
                            const float x0 = y[2 * i], x1 = y[2 * i + 1];
                            y[2 * i] = x0 * c - x1 * d;
                            y[2 * i + 1] = x1 * c + x0 * d;
                        }
                    } else if (!apart) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = j0 + 2 * i;
                            if (j < 0 || j >= rot) continue;
                            const float2 z = cs[j >> 1];
                            const float x0 = y[2 * i], x1 = y[2 * i + 1];
                            y[2 * i] = x0 * z.x - x1 * z.y;
                            y[2 * i + 1] = x1 * z.x + x0 * z.y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int j = j0 + i;
                            if (j < 0 || j >= rot) continue;
                            const bool second = a.turn.half ? j >= pairs : j & 1;
                            const float2 z = cs[a.turn.half ? (second ? j - pairs : j) : j >> 1];
                            const float x = s_y[w][offset + (a.turn.half ? (second ? j - pairs : j + pairs) : j ^ 1)];
                            y[i] = second ? y[i] * z.x + x * z.y : y[i] * z.x - x * z.y;
                        }
                    }
                }
                if (!all || apart) {  // before the next row's
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
            }
        }
        if (t >= a.tokens) continue;
        if (a.f32) {
            float* o = (float*)a.out + t * a.stride + 8 * li;
            if (a.wide) {
                reinterpret_cast<float4*>(o)[0] = float4{y[0], y[1], y[2], y[3]};
                reinterpret_cast<float4*>(o)[1] = float4{y[4], y[5], y[6], y[7]};
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = y[i];
            }
        } else {
            uint16_t* o = (uint16_t*)a.out + t * a.stride + 8 * li;
            const uint4 v{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7])};
            if (a.wide) {
                *reinterpret_cast<uint4*>(o) = v;
            } else {
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = (uint16_t)(x[i >> 1] >> (16 * (i & 1)));
            }
        }
    }
}

template <int FMT>
void start_write(const RowsArgs& a, hipStream_t stream) {
    constexpr int kRows = 256 * 16 / Format<FMT>::kDim;
    const dim3 grid((unsigned)((a.tokens + kRows - 1) / kRows));
    if (a.f32 && a.norm)
        hipLaunchKernelGGL((write_rows_kernel<FMT, true, true>), grid, dim3(256), 0, stream, a);
    else if (a.f32)
        hipLaunchKernelGGL((write_rows_kernel<FMT, true, false>), grid, dim3(256), 0, stream, a);
    else if (a.norm)
        hipLaunchKernelGGL((write_rows_kernel<FMT, false, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((write_rows_kernel<FMT, false, false>), grid, dim3(256), 0, stream, a);
}

}  // namespace

hipError_t launch_write_rows(const RowsArgs& a, hipStream_t stream) {
    if (a.format == IDX_ROWS_MAIN)
        start_write<IDX_ROWS_MAIN>(a, stream);
    else if (a.format == IDX_ROWS_LOCAL)
        start_write<IDX_ROWS_LOCAL>(a, stream);
    else
        start_write<IDX_ROWS_KEY>(a, stream);
    return hipGetLastError();
}

hipError_t launch_read_rows(const RowsArgs& a, hipStream_t stream) {
    // Two rows a lane where the wavefronts fill the card four times: 32768 rows of the main KV, turned, replayed 15.3 us with one,
    // 13.1 with two, 14.5 with four; 65536 26.5, 21.9, 22.4; 8192 rows of local positions in fp32 7.05, 7.25, 7.35.
    const int64_t lanes = a.tokens * (a.format == IDX_ROWS_KEY ? kDim : 512) / 8;
    if (lanes >= (int64_t)4 * 64 * 4096) {
        const dim3 grid((unsigned)((lanes + 511) / 512));
        if (a.format == IDX_ROWS_KEY)
            hipLaunchKernelGGL((read_rows_kernel<IDX_ROWS_KEY, 2>), grid, dim3(256), 0, stream, a);
        else if (a.format == IDX_ROWS_MAIN)
            hipLaunchKernelGGL((read_rows_kernel<IDX_ROWS_MAIN, 2>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((read_rows_kernel<IDX_ROWS_LOCAL, 2>), grid, dim3(256), 0, stream, a);
    } else {
        const dim3 grid((unsigned)((lanes + 255) / 256));
        if (a.format == IDX_ROWS_KEY)
            hipLaunchKernelGGL((read_rows_kernel<IDX_ROWS_KEY, 1>), grid, dim3(256), 0, stream, a);
        else if (a.format == IDX_ROWS_MAIN)
            hipLaunchKernelGGL((read_rows_kernel<IDX_ROWS_MAIN, 1>), grid, dim3(256), 0, stream, a);
        else
            hipLaunchKernelGGL((read_rows_kernel<IDX_ROWS_LOCAL, 1>), grid, dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace fp4idx
