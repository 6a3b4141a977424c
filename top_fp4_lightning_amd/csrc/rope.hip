// Rotary positions: pair i of a row's rotated part turns by the angle pos * freq_i,
//   y0 = m (x0 cos - x1 sin),  y1 = m (x1 cos + x0 sin);  inverse (the gradient): the angle negated.
// Pairs are (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved").
//
// Angles of far positions need more than 32 bits (at position 2^20 an fp32 product is off by up to
// 0.06 rad): turns = pos * freq / 2 pi in fp64, its whole part taken off exactly, then sin and cos of
// the remainder in fp32. They are computed once per token, in LDS, and used by all heads.
//
// The kernel is a copy: one read and one write of every value (the rotated part only, in place). A
// lane moves 16, 8 or 4 bytes at a time as sizes and addresses allow, else one value or pair, of four rows at a time
// (131 us with one). Bound by HBM: 4096 x 64 x 512 bf16 values take 102 us, 5.3 TB/s; one token of 32 heads 2.6 us.
// Writing past the last-level cache gave 82 us for that call by itself, but the call that reads the result lost more
// (chained with it 225 against 201 us; at 32 MB 38 against 27).
#include "operators.h"

namespace fp4idx {
namespace {

constexpr int kRopeLds = 4096;  // (cos, sin) pairs per block: 32 KB
constexpr int kRows = 4;        // rows of a lane in flight
constexpr double kInv2Pi = 0x1.45f306dc9c883p-3, kInv2PiLow = -0x1.6b01ec5417056p-57;  // 1 / 2 pi

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ uint16_t from_f(float v) { return (uint16_t)bf16_pair(v, 0.0f); }
template <> __device__ __forceinline__ float from_f(float v) { return v; }

// V values moved as one access
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// (cos, sin) of a block's tokens into LDS. Whole block.
__device__ __forceinline__ void angles(const RopeArgs& a, int64_t tok0, int toks, float2* cs) {
    const int pairs = a.rot / 2;
    for (int i = threadIdx.x; i < toks * pairs; i += 256) {
        const int tk = i / pairs, pr = i - tk * pairs;
        // freq / 2 pi with what its rounding leaves, and the product with pos without one: at 2^31 each is 2^-22 rad
        const double pos = (double)a.pos[tok0 + tk], freq = a.freq[pr];
        const double per = freq * kInv2Pi, per_low = fma(freq, kInv2Pi, -per) + freq * kInv2PiLow;
        const double turns = fma(pos, per, -rint(pos * per)) + pos * per_low;
        float s, c;
        sincospif(2.0f * (float)turns, &s, &c);
        cs[i] = float2{c * a.mscale, (a.inverse ? -s : s) * a.mscale};
    }
    __syncthreads();
}

// A block takes `tokens_per_block` tokens; a row (token, head) takes `lanes` lanes (a power of two).
// items of a row: first the rotated ones (V values of each half of a pair, or of whole pairs), then those that pass
// through, by P (none in place).
template <typename T, int V, int P, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a, int tokens_per_block, int lanes_log2,
                                                   int rot_items, int items) {
    __shared__ float2 s_cs[kRopeLds];
    const int64_t tok0 = (int64_t)blockIdx.x * tokens_per_block;
    const int toks = (int)min((int64_t)tokens_per_block, a.tokens - tok0);
    const int pairs = a.rot / 2;
    angles(a, tok0, toks, s_cs);

    const int lanes = 1 << lanes_log2;
    const int at = threadIdx.x & (lanes - 1);
    const int step = 256 >> lanes_log2;  // rows per pass of the block
    const int step_tok = step / a.heads, step_head = step - step_tok * a.heads;
    const T* xs = (const T*)a.x;
    T* ys = (T*)a.out;
    typedef Vec<T, V> W;
    typedef Vec<T, P> WP;
    for (int it = at; it < items; it += lanes) {
        // what the item reads and writes of a row: one vector, or two (n1 apart)
        const bool turns = it < rot_items;
        constexpr int kPairs = HALF ? V : (V > 1 ? V / 2 : 1);  // of an item
        int i0 = (it - rot_items) * P;
        if (turns)
            i0 = a.offset + it * (HALF ? V : 2 * kPairs);
        else if (i0 >= a.offset)
            i0 += a.rot;
        const int i1 = i0 + (HALF ? pairs : V);
        constexpr bool kTwo = HALF || V == 1;
        int tk = (int)(threadIdx.x >> lanes_log2) / a.heads;
        int h = (int)(threadIdx.x >> lanes_log2) - tk * a.heads;
        while (tk < toks) {
            // kRows rows at a time, their reads ahead of the first use
            W v[kRows][kTwo ? 2 : 1];
            WP through[V == P ? 1 : kRows];
            int64_t to[kRows];
            int tok[kRows];
            int n = 0;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                tok[r] = tk;
                if (tk < toks) {
                    const T* x = xs + (tok0 + tk) * a.x_token + h * a.x_head;
                    to[r] = (tok0 + tk) * a.out_token + h * a.out_head;
                    if constexpr (V == P) {
                        v[r][0] = *reinterpret_cast<const W*>(x + i0);
                    } else {
                        if (turns)
                            v[r][0] = *reinterpret_cast<const W*>(x + i0);
                        else
                            through[r] = *reinterpret_cast<const WP*>(x + i0);
                    }
                    if (kTwo && turns) v[r][kTwo ? 1 : 0] = *reinterpret_cast<const W*>(x + i1);
                    n = r + 1;
                    tk += step_tok;
                    h += step_head;
                    if (h >= a.heads) {
                        h -= a.heads;
                        ++tk;
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (r >= n) continue;
                if (turns) {
                    const float2* cs = s_cs + tok[r] * pairs + it * kPairs;
                    T* e = reinterpret_cast<T*>(v[r]);
#pragma unroll
                    for (int k = 0; k < kPairs; ++k) {
                        const float2 z = cs[k];
                        T& e0 = e[HALF ? k : 2 * k];
                        T& e1 = e[HALF ? V + k : 2 * k + 1];
                        const float x0 = to_f<T>(e0), x1 = to_f<T>(e1);
                        e0 = from_f<T>(x0 * z.x - x1 * z.y);
                        e1 = from_f<T>(x1 * z.x + x0 * z.y);
                    }
                }
                if constexpr (V != P) {
                    if (!turns) {
                        *reinterpret_cast<WP*>(ys + to[r] + i0) = through[r];
                        continue;
                    }
                }
                *reinterpret_cast<W*>(ys + to[r] + i0) = v[r][0];
                if (kTwo && turns) *reinterpret_cast<W*>(ys + to[r] + i1) = v[r][kTwo ? 1 : 0];
            }
        }
    }
}

// Halves, rows of at most 64 vectors: every lane reads and writes one vector of the row and has the other half's from
// the lane that holds it (4096 x 64 x 512 bf16 values, 64 rotated: 143 us with two reads and writes by the lanes of
// one half, 117 us so).
template <typename T, int V>
__global__ __launch_bounds__(256) void rope_halves_kernel(const RopeArgs a, int tokens_per_block, int lanes_log2,
                                                          int items) {
    __shared__ float2 s_cs[kRopeLds];
    const int64_t tok0 = (int64_t)blockIdx.x * tokens_per_block;
    const int toks = (int)min((int64_t)tokens_per_block, a.tokens - tok0);
    const int pairs = a.rot / 2;
    angles(a, tok0, toks, s_cs);

    typedef Vec<T, V> W;
    constexpr int kWords = sizeof(W) / 4;
    const int lanes = 1 << lanes_log2;
    const int at = threadIdx.x & (lanes - 1);
    if (at >= items) return;
    const int step = 256 >> lanes_log2;  // rows per pass of the block
    const int step_tok = step / a.heads, step_head = step - step_tok * a.heads;
    const bool in_place = a.out == a.x;
    const int i0 = (in_place ? a.offset : 0) + at * V, rel = i0 - a.offset;
    const bool turns = rel >= 0 && rel < a.rot, second = rel >= pairs;
    const int pair = second ? rel - pairs : rel;
    const int other = ((int)threadIdx.x & 63) + (turns ? (second ? -pairs / V : pairs / V) : 0);
    const T* xs = (const T*)a.x + i0;
    T* ys = (T*)a.out + i0;
    int tk = (int)(threadIdx.x >> lanes_log2) / a.heads;
    int h = (int)(threadIdx.x >> lanes_log2) - tk * a.heads;
    while (tk < toks) {
        W v[kRows];
        int64_t to[kRows];
        int tok[kRows];
        int n = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            tok[r] = tk;
            if (tk < toks) {
                v[r] = *reinterpret_cast<const W*>(xs + (tok0 + tk) * a.x_token + h * a.x_head);
                to[r] = (tok0 + tk) * a.out_token + h * a.out_head;
                n = r + 1;
                tk += step_tok;
                h += step_head;
                if (h >= a.heads) {
                    h -= a.heads;
                    ++tk;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (r >= n) continue;
            // (the other lane has the same row: it is here, too)
            uint32_t words[kWords];
            __builtin_memcpy(words, &v[r], sizeof(W));
#pragma unroll
            for (int k = 0; k < kWords; ++k) words[k] = __shfl(words[k], other);
            if (turns) {
                W o;
                __builtin_memcpy(&o, words, sizeof(W));
                const float2* cs = s_cs + tok[r] * pairs + pair;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float2 z = cs[k];
                    const float x = to_f<T>(v[r].v[k]), y = to_f<T>(o.v[k]);
                    v[r].v[k] = from_f<T>(x * z.x + (second ? y : -y) * z.y);
                }
            }
            *reinterpret_cast<W*>(ys + to[r]) = v[r];
        }
    }
}

template <typename T, int V, int P>
void launch_rope_as(const RopeArgs& a, hipStream_t stream) {
    const bool in_place = a.out == a.x;
    const int rot_items = a.rot / 2 / (a.half ? V : (V > 1 ? V / 2 : 1));
    const int items = rot_items + (in_place ? 0 : (a.dim - a.rot) / P);
    int lanes_log2 = 0;
    while (lanes_log2 < 6 && (1 << lanes_log2) < items) ++lanes_log2;
    // about 16 passes of the block over its rows (64 KB of bf16), fewer while that leaves the 256
    // compute units short of blocks; what the table of angles holds at most
    const int64_t rows_per_block = 16 * (256 >> lanes_log2);
    int64_t tpb = rows_per_block / a.heads;
    const int64_t most = kRopeLds / (a.rot / 2);
    const int64_t spread = (a.tokens + 1023) / 1024;
    tpb = tpb < spread ? tpb : spread;
    tpb = tpb < most ? tpb : most;
    tpb = tpb < 1 ? 1 : tpb;
    const dim3 grid((unsigned)((a.tokens + tpb - 1) / tpb));
    if constexpr (V == P && V > 1) {
        const int whole = (in_place ? a.rot : a.dim) / V;
        if (a.half && whole <= 64) {
            // (as many lanes as before or twice)
            lanes_log2 = 0;
            while ((1 << lanes_log2) < whole) ++lanes_log2;
            hipLaunchKernelGGL((rope_halves_kernel<T, V>), grid, dim3(256), 0, stream, a, (int)tpb, lanes_log2, whole);
            return;
        }
    }
    if (a.half)
        hipLaunchKernelGGL((rope_kernel<T, V, P, true>), grid, dim3(256), 0, stream, a, (int)tpb, lanes_log2, rot_items,
                           items);
    else
        hipLaunchKernelGGL((rope_kernel<T, V, P, false>), grid, dim3(256), 0, stream, a, (int)tpb, lanes_log2, rot_items,
                           items);
}

template <typename T>
void launch_rope_of(const RopeArgs& a, hipStream_t stream) {
    // how many values an access can have: sizes and addresses are multiples of it (19636 x 16 x 130 bf16 values by 4
    // bytes 57 us, by one value 98)
    constexpr int kMost = 16 / sizeof(T);
    const auto width = [&](int64_t sizes) {
        const uint64_t all = (uint64_t)sizes | ((uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.out) / sizeof(T);
        int v = kMost;
        while (v > 1 && all % v) v /= 2;
        return v;
    };
    const int64_t strides = (a.tokens > 1 ? a.x_token | a.out_token : 0) | (a.heads > 1 ? a.x_head | a.out_head : 0);
    const int rotated = width(strides | a.offset | (a.half ? a.rot / 2 : a.rot));
    const int through = width(strides | a.offset | a.rot | a.dim);
    const int v = rotated < through ? rotated : through;
    if (v == kMost) return launch_rope_as<T, kMost, kMost>(a, stream);
    if (v == kMost / 2) return launch_rope_as<T, kMost / 2, kMost / 2>(a, stream);
    if constexpr (kMost > 4) {
        if (v == kMost / 4) return launch_rope_as<T, kMost / 4, kMost / 4>(a, stream);
    }
    // halves of an odd length: the rest two at a time (47558 x 3 x 96 fp32 values with one pair: 55 -> 32 us)
    if (through > 1) return launch_rope_as<T, 1, 2>(a, stream);
    launch_rope_as<T, 1, 1>(a, stream);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, hipStream_t stream) {
    if (a.f32)
        launch_rope_of<float>(a, stream);
    else
        launch_rope_of<uint16_t>(a, stream);
    return hipGetLastError();
}

}  // namespace fp4idx
