// Rows written to and read from their places in a cache.
//
// Writing: y = x, normalised (x gamma / sqrt(mean x^2 + eps)), turned by its position, then quantised in the cache's
// format and stored in the row of its entry. One pass: a lane holds 8 values, a row of 512 takes a wavefront, a key of
// 128 sixteen lanes.
//
// Which code a value gets turns on the side of a border it lies on, so everything up to that is in 64 bits, and what is
// compared in fp32 is rounded to odd: cut, with the last bit set where something was cut off. Such a value lies on the
// same side of every number of fewer bits as the exact one, and a border has at most 8.
//
// Reading: the stored values (a code times a scale is exact in fp32 and bf16), turned in fp32, rounded once.
#include "../../include/fp4idx.h"
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

// fp32 of a 64-bit value, rounded to odd
__device__ __forceinline__ float to_odd(double y) {
    const float f = (float)y;
    const double d = (double)f;
    uint32_t b = __float_as_uint(f);
    if (d != y && !(b & 1u)) b += fabs(d) < fabs(y) ? 1u : 0xffffffffu;
    return __uint_as_float(b);
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

// smallest E4M3 byte whose value s has 6 s >= a (a >= 0); 0x7e (448) at most
__device__ __forceinline__ float e4m3_of(uint32_t b) {
    const uint32_t e = b >> 3, m = b & 7u;
    return e == 0 ? (float)m * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
}
__device__ __forceinline__ uint32_t e4m3_scale_for(float a) {
    uint32_t lo = 0, hi = 0x7e;
#pragma unroll
    for (int it = 0; it < 7; ++it) {
        const uint32_t mid = (lo + hi) >> 1;
        if (6.0f * e4m3_of(mid) >= a)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo < 0x7e ? lo : 0x7e;
}

// E2M1 code of x for scale s > 0: the number of middles below |x|, a tie to the even code
__device__ __forceinline__ uint32_t e2m1_code(float x, float s) {
    const float a = fabsf(x);
    uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) +
                 (a >= 3.5f * s) + (a > 5.0f * s);
    return (c != 0 && __float_as_uint(x) >> 31) ? (c | 8u) : c;
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
    constexpr int kPairs = F::kDim / 2;
    __shared__ double2 s_cs[kRows][kPairs];
    __shared__ double s_y[kRows][F::kDim];
    const int li = threadIdx.x % F::kLanes, r = threadIdx.x / F::kLanes;
    const int64_t t = (int64_t)blockIdx.x * kRows + r;
    const bool live = t < a.tokens;
    const int64_t tc = live ? t : a.tokens - 1;
    float f[8];
    load8(a, tc, li, f);
    const int64_t at = a.at[tc];
    int64_t row = row_at(a.places, a.places.seq ? a.places.seq[tc] : tc, a.places.base ? a.places.base[tc] : 0, at);
    if (!live) row = -1;

    const bool turn = a.turn.freq != nullptr;
    double y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (double)f[i];
    if (a.norm) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma(y[i], y[i], sum);
        sum += xor_lane<1>(sum, li);
        sum += xor_lane<2>(sum, li);
        sum += xor_lane<4>(sum, li);
        sum += xor_lane<8>(sum, li);
        if constexpr (F::kLanes == 64) {
            sum += xor_lane<16>(sum, li);
            sum += xor_lane<32>(sum, li);
        }
        const double by = 1.0 / sqrt(sum / F::kDim + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= by;
        if (a.gamma) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= (double)a.gamma[8 * li + i];
        }
    }
    if (turn) {
        const int rot = a.turn.rot, pairs = rot / 2, offset = a.turn.offset;
        const int64_t pos = a.turn.pos ? a.turn.pos[tc] : at;
        for (int p = li; p < pairs; p += F::kLanes) {
            double s, c;
            sincospi(2.0 * turns_of(pos, a.turn.freq[p]), &s, &c);
            s_cs[r][p] = double2{c * a.turn.mscale, (a.turn.inverse ? -s : s) * a.turn.mscale};
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
            const double2 cs = s_cs[r][pair];
            const double z = s_y[r][offset + other];
            y[i] = second ? y[i] * cs.x + z * cs.y : y[i] * cs.x - z * cs.y;
        }
    }

    if constexpr (FMT == IDX_ROWS_KEY) {
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
    } else if (a.norm || turn) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = to_odd(y[i]);
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
        float v[8];
        // (a value that leaves fp32's range on the way lies far above 448 or far below half of the smallest code)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(ldexpf(f[i], -e), -448.0f), 448.0f);
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
        float s = 0.0f;
        uint32_t word = 0;
        if constexpr (FMT == IDX_ROWS_MAIN) {
            scale = e4m3_scale_for(top);
            s = e4m3_of(scale);
            if (s > 0.0f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) word |= e2m1_code(f[i], s) << (4 * i);
            }
        } else {
            const int e = scale_exponent(top, 0.75f, 3, -127, 127);
            scale = (uint32_t)(e + 127);
#pragma unroll
            for (int i = 0; i < 8; ++i) word |= e2m1_code(ldexpf(f[i], -e), 1.0f) << (4 * i);
        }
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
