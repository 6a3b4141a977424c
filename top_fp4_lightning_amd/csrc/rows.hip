// Rows written to and read from their places in a cache.
//
// Writing: y = x, normalised (x gamma / sqrt(mean x^2 + eps)), turned by its position, then quantised in the cache's
// format and stored in the row of its entry. One pass: a lane holds 8 values, a row of 512 takes a wavefront, a key of
// 128 sixteen lanes. A rotated pair is a lane's: its angle, sine and cosine, both values.
//
// Which code a value gets turns on the side of a border it lies on, so everything up to that is in 64 bits, and what is
// compared in fp32 is a value cut to 20 bits behind the leading one, the last of them set where something was cut off
// (rounded to odd). It lies on the same side as the exact one of every number of fewer bits, and a border has at most 7.
//
// Reading: the stored values (a code times a scale is exact in fp32 and bf16), turned in fp32, rounded once.
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
    static constexpr int kDim = 512, kGroup = 16, kLanes = 64;
};
template <>
struct Format<IDX_ROWS_LOCAL> {
    static constexpr int kDim = 512, kGroup = 32, kLanes = 64;
};
template <>
struct Format<IDX_ROWS_KEY> {
    static constexpr int kDim = 128, kGroup = 32, kLanes = 16;
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

// values of a row of x (8 of lane li), whole pieces or one by one
__device__ __forceinline__ void load8(const RowsArgs& a, int64_t row, int li, float (&f)[8]) {
    if (a.f32) {
        const float* x = (const float*)a.x + row * a.stride + 8 * li;
        if (a.wide) {
            const float4 u = reinterpret_cast<const float4*>(x)[0], v = reinterpret_cast<const float4*>(x)[1];
            f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = x[i];
        }
    } else {
        const uint16_t* x = (const uint16_t*)a.x + row * a.stride + 8 * li;
        if (a.wide) {
            const uint4 u = *reinterpret_cast<const uint4*>(x);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16f(w[i] & 0xffffu);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = bf16f(x[i]);
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

// E2M1 codes of 8 values of at most 6 in magnitude, or cut to it; zero has no sign
__device__ __forceinline__ uint32_t e2m1_codes(const float (&q)[8]) {
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

template <int FMT>
__global__ __launch_bounds__(256) void write_rows_kernel(const RowsArgs a) {
    typedef Format<FMT> F;
    constexpr int kRows = 256 / F::kLanes;  // of a block
    constexpr bool kKey = FMT == IDX_ROWS_KEY;
    typedef std::conditional_t<kKey, double, float> Part;  // a turned value: keys go on in 64 bits
    __shared__ __align__(16) float s_x[kRows][F::kDim];
    __shared__ __align__(16) Part s_y[kRows][F::kDim];
    const int li = threadIdx.x % F::kLanes, r = threadIdx.x / F::kLanes;
    const int64_t t = (int64_t)blockIdx.x * kRows + r;
    const bool live = t < a.tokens;
    const int64_t tc = live ? t : a.tokens - 1;
    float f[8];
    load8(a, tc, li, f);
    const int64_t at = a.at[tc];
    int64_t row = row_at(a.places, a.places.seq ? a.places.seq[tc] : tc, a.places.base ? a.places.base[tc] : 0, at);
    if (!live) row = -1;

    double by = 1.0;
    if (a.norm) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)f[i], (double)f[i], sum);
        sum += xor_lane<1>(sum, li);
        sum += xor_lane<2>(sum, li);
        sum += xor_lane<4>(sum, li);
        sum += xor_lane<8>(sum, li);
        if constexpr (F::kLanes == 64) {
            sum += xor_lane<16>(sum, li);
            sum += xor_lane<32>(sum, li);
        }
        by = 1.0 / sqrt(sum / F::kDim + a.eps);
    }
    const auto normal = [&](float x, int i) {
        double y = (double)x * by;
        if (a.gamma) y *= (double)a.gamma[i];
        return y;
    };
    if (a.turn.freq) {
        const int rot = a.turn.rot, pairs = rot / 2, offset = a.turn.offset;
        const int64_t pos = a.turn.pos ? a.turn.pos[tc] : at;
        *reinterpret_cast<float4*>(s_x[r] + 8 * li) = float4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<float4*>(s_x[r] + 8 * li + 4) = float4{f[4], f[5], f[6], f[7]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // (a row is one wavefront's)
        __builtin_amdgcn_wave_barrier();
        for (int p = li; p < pairs; p += F::kLanes) {
            double s, c;
            sincos_turns(turns_of(pos, a.turn.freq[p]), s, c);
            s *= a.turn.mscale, c *= a.turn.mscale;
            const int i0 = offset + (a.turn.half ? p : 2 * p), i1 = i0 + (a.turn.half ? pairs : 1);
            double x0 = s_x[r][i0], x1 = s_x[r][i1];
            if (a.norm) x0 = normal((float)x0, i0), x1 = normal((float)x1, i1);
            const double y0 = x0 * c - x1 * s, y1 = x1 * c + x0 * s;
            if constexpr (kKey) {
                s_y[r][i0] = y0, s_y[r][i1] = y1;
            } else {
                s_y[r][i0] = to_odd(y0), s_y[r][i1] = to_odd(y1);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // this lane's values among the turned ones: first .. last - 1
    const int first = a.turn.freq ? max(a.turn.offset - 8 * li, 0) : 8;
    const int last = a.turn.freq ? min(a.turn.offset + a.turn.rot - 8 * li, 8) : 8;

    if constexpr (kKey) {
        double y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = a.norm ? normal(f[i], 8 * li + i) : (double)f[i];
        if (first < last) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = i >= first && i < last ? s_y[r][8 * li + i] : y[i];
        }
        // the signs, the transform in 64 bits, then fl32(S) fl32(2^-3.5) in fp32
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = a.signs[8 * li + i] < 0 ? -y[i] : y[i];
#pragma unroll
        for (int b = 1; b < 8; b <<= 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!(i & b)) {
                    const double p = y[i], q = y[i | b];
                    y[i] = p + q;
                    y[i | b] = p - q;
                }
            }
        }
        const auto stage = [&](double other, double mine, bool upper) { return upper ? other - mine : mine + other; };
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = stage(xor_lane<1>(y[i], li), y[i], li & 1);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = stage(xor_lane<2>(y[i], li), y[i], li & 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = stage(xor_lane<4>(y[i], li), y[i], li & 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = stage(xor_lane<8>(y[i], li), y[i], li & 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)y[i] * 0x1.6a09e6p-4f;  // fl32(2^-3.5)
    } else {
        if (a.norm) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = to_odd(normal(f[i], 8 * li + i));
        } else if (a.f32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = to_odd(f[i]);
        }
        if (first < last) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = i >= first && i < last ? s_y[r][8 * li + i] : f[i];
        }
    }

    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
    top = fmaxf(top, xor_lanef<1>(top, li));
    if constexpr (F::kGroup == 32) top = fmaxf(top, xor_lanef<2>(top, li));
    constexpr int kGroupLanes = F::kGroup / 8, kScales = F::kDim / F::kGroup;
    uint32_t scale;
    if constexpr (FMT == IDX_ROWS_LOCAL) {
        const int e = scale_exponent(top, 0.875f, 9, IDX_LOCAL_MIN_EXP, IDX_LOCAL_MAX_EXP);
        scale = (uint32_t)(e + 127);
        const float by_e = __uint_as_float((uint32_t)(127 - e) << 23);
        float v[8];
        // (a value that leaves fp32's normal range on the way lies far below half of the smallest code)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(f[i] * by_e, -448.0f), 448.0f);
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
            b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], b, true);
            const uint32_t some = (((uint32_t)b & 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u;
            w[i] = (uint32_t)b & (some | 0x7f7f7f7fu);  // zero has no sign
        }
        if (row >= 0) *reinterpret_cast<uint2*>(a.codes + row * 512 + 8 * li) = uint2{w[0], w[1]};
    } else {
        float q[8];
        if constexpr (FMT == IDX_ROWS_MAIN) {
            scale = e4m3_scale_for(top);
            const float s = e4m3_of(scale), inv = s > 0.0f ? 1.0f / s : 0.0f;
            // Quotients by a product with 1 / s, off by 2^-23 of themselves at most, then rounded to 21 bits behind the
            // leading one: on a border where the value is on it (half a step there is 1.14 2^-23), and on the value's
            // side of it where it is not (it lies 2^-21 off at least, a border's neighbours are 2^-22 off at most).
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = fminf(fmaxf(f[i] * inv, -6.0f), 6.0f);
                q[i] = __uint_as_float((__float_as_uint(x) + 2u) & 0xfffffffcu);
            }
        } else {
            const int e = scale_exponent(top, 0.75f, 3, -127, 127);
            scale = (uint32_t)(e + 127);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = ldexpf(f[i], -e);
        }
        const uint32_t word = e2m1_codes(q);
        if (row >= 0) reinterpret_cast<uint32_t*>(a.codes + row * (F::kDim / 2))[li] = word;
    }
    if (row >= 0 && li % kGroupLanes == 0) a.scales[row * kScales + li / kGroupLanes] = (uint8_t)scale;
}

// E2M1 nibble -> value
__device__ __forceinline__ float e2m1_value(uint32_t n) {
    const uint32_t m = n & 7u;
    const uint32_t bits = m >= 2 ? ((((m >> 1) + 126u) << 23) | ((m & 1u) << 22)) : (m == 1 ? 0x3f000000u : 0u);
    return __uint_as_float(bits | ((n & 8u) << 28));
}

template <int FMT>
__global__ __launch_bounds__(256) void read_rows_kernel(const RowsArgs a) {
    typedef Format<FMT> F;
    constexpr int kRows = 256 / F::kLanes;
    constexpr int kGroupLanes = F::kGroup / 8, kScales = F::kDim / F::kGroup;
    __shared__ float2 s_cs[kRows][F::kDim / 2];
    __shared__ float s_y[kRows][F::kDim];
    const int li = threadIdx.x % F::kLanes, r = threadIdx.x / F::kLanes;
    const int64_t t = (int64_t)blockIdx.x * kRows + r;
    const bool live = t < a.tokens;
    const int64_t tc = live ? t : a.tokens - 1;
    const int64_t at = a.at[tc];
    const int64_t row = row_at(a.places, a.places.seq ? a.places.seq[tc] : tc, a.places.base ? a.places.base[tc] : 0, at);
    float y[8] = {};
    if (row >= 0) {
        const uint32_t sb = a.scales[row * kScales + li / kGroupLanes];
        if constexpr (FMT == IDX_ROWS_LOCAL) {
            const uint2 w = *reinterpret_cast<const uint2*>(a.codes + row * 512 + 8 * li);
            const float s = ldexpf(1.0f, (int)sb - 127);
            const uint32_t ws[2] = {w.x, w.y};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = ws[i >> 2] >> (8 * (i & 3));
                const float m = e4m3_of(b & 0x7fu);
                y[i] = (b & 0x80u ? -m : m) * s;
            }
        } else {
            const uint32_t w = reinterpret_cast<const uint32_t*>(a.codes + row * (F::kDim / 2))[li];
            float s;
            if constexpr (FMT == IDX_ROWS_MAIN)
                s = sb & 0x80u ? -e4m3_of(sb & 0x7fu) : e4m3_of(sb);
            else
                s = ldexpf(1.0f, (int)sb - 127);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = e2m1_value(w >> (4 * i)) * s;
        }
    }
    if (a.turn.freq) {
        const int rot = a.turn.rot, pairs = rot / 2, offset = a.turn.offset;
        const int64_t pos = a.turn.pos ? a.turn.pos[tc] : at;
        const float m = (float)a.turn.mscale;
        for (int p = li; p < pairs; p += F::kLanes) {
            float s, c;
            sincospif(2.0f * (float)turns_of(pos, a.turn.freq[p]), &s, &c);
            s_cs[r][p] = float2{c * m, (a.turn.inverse ? -s : s) * m};
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s_y[r][8 * li + i] = y[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = 8 * li + i - offset;
            if (j < 0 || j >= rot) continue;
            const bool second = a.turn.half ? j >= pairs : j & 1;
            const int pair = a.turn.half ? (second ? j - pairs : j) : j >> 1;
            const int other = a.turn.half ? (second ? j - pairs : j + pairs) : j ^ 1;
            const float2 cs = s_cs[r][pair];
            const float z = s_y[r][offset + other];
            y[i] = second ? y[i] * cs.x + z * cs.y : y[i] * cs.x - z * cs.y;
        }
    }
    if (!live) return;
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
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

template <int FMT, typename K>
hipError_t launch(K kernel, const RowsArgs& a, hipStream_t stream) {
    constexpr int kRows = 256 / Format<FMT>::kLanes;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.tokens + kRows - 1) / kRows)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_write_rows(const RowsArgs& a, hipStream_t stream) {
    if (a.format == IDX_ROWS_MAIN) return launch<IDX_ROWS_MAIN>(write_rows_kernel<IDX_ROWS_MAIN>, a, stream);
    if (a.format == IDX_ROWS_LOCAL) return launch<IDX_ROWS_LOCAL>(write_rows_kernel<IDX_ROWS_LOCAL>, a, stream);
    return launch<IDX_ROWS_KEY>(write_rows_kernel<IDX_ROWS_KEY>, a, stream);
}

hipError_t launch_read_rows(const RowsArgs& a, hipStream_t stream) {
    if (a.format == IDX_ROWS_MAIN) return launch<IDX_ROWS_MAIN>(read_rows_kernel<IDX_ROWS_MAIN>, a, stream);
    if (a.format == IDX_ROWS_LOCAL) return launch<IDX_ROWS_LOCAL>(read_rows_kernel<IDX_ROWS_LOCAL>, a, stream);
    return launch<IDX_ROWS_KEY>(read_rows_kernel<IDX_ROWS_KEY>, a, stream);
}

}  // namespace fp4idx
