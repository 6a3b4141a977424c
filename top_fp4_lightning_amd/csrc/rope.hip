// Rotary positions: pair i of a row's rotated part turns by the angle pos * freq_i,
//   y0 = m (x0 cos - x1 sin),  y1 = m (x1 cos + x0 sin);  inverse (the gradient): the angle negated.
// Pairs are (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved").
//
// Angles of far positions need more than 32 bits (at position 2^20 an fp32 product is off by up to
// 0.06 rad): turns = pos * freq / 2 pi in fp64, its whole part taken off exactly, then sin and cos of
// the remainder in fp32. They are computed once per token, in LDS, and used by all heads.
//
// The kernel is a copy: one read and one write of every value (the rotated part only, in place). A
// lane moves 16 bytes at a time where sizes and addresses allow it, else one value or pair, of four rows at a time
// (131 us with one). Bound by HBM: 4096 x 64 x 512 bf16 values take 100 us, 5.4 TB/s; one token of 32 heads 2.8 us.
// Writing past the last-level cache gave 82 us for that call by itself, but the call that reads the result lost more
// (chained with it 225 against 201 us; at 32 MB 38 against 27).
#include "operators.h"

namespace fp4idx {
namespace {

constexpr int kRopeLds = 4096;  // (cos, sin) pairs per block: 32 KB
constexpr int kRows = 4;        // rows of a lane in flight

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

// A block takes `tokens_per_block` tokens; a row (token, head) takes `lanes` lanes (a power of two).
// items of a row: first the rotated ones (a vector of each half of a pair, or a vector of whole pairs),
// then the vectors that pass through (none in place).
template <typename T, int V, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(const RopeArgs a, int tokens_per_block, int lanes_log2,
                                                   int rot_items, int items) {
    __shared__ float2 s_cs[kRopeLds];
    const int64_t tok0 = (int64_t)blockIdx.x * tokens_per_block;
    const int toks = (int)min((int64_t)tokens_per_block, a.tokens - tok0);
    const int pairs = a.rot / 2;
    for (int i = threadIdx.x; i < toks * pairs; i += 256) {
        const int tk = i / pairs, pr = i - tk * pairs;
        double turns = (double)a.pos[tok0 + tk] * (a.freq[pr] * 0.15915494309189533577);
        turns -= rint(turns);
        float s, c;
        sincospif(2.0f * (float)turns, &s, &c);
        s_cs[i] = float2{c * a.mscale, (a.inverse ? -s : s) * a.mscale};
    }
    __syncthreads();

    const int lanes = 1 << lanes_log2;
    const int at = threadIdx.x & (lanes - 1);
    const int step = 256 >> lanes_log2;  // rows per pass of the block
    const int step_tok = step / a.heads, step_head = step - step_tok * a.heads;
    const T* xs = (const T*)a.x;
    T* ys = (T*)a.out;
    typedef Vec<T, V> W;
    for (int it = at; it < items; it += lanes) {
        // what the item reads and writes of a row: one vector, or two (n1 apart)
        const bool turns = it < rot_items;
        constexpr int P = HALF ? V : (V > 1 ? V / 2 : 1);  // pairs of an item
        int i0 = (it - rot_items) * V;
        if (turns)
            i0 = a.offset + it * (HALF ? V : 2 * P);
        else if (i0 >= a.offset)
            i0 += a.rot;
        const int i1 = i0 + (HALF ? pairs : V);
        constexpr bool kTwo = HALF || V == 1;
        int tk = (int)(threadIdx.x >> lanes_log2) / a.heads;
        int h = (int)(threadIdx.x >> lanes_log2) - tk * a.heads;
        while (tk < toks) {
            // kRows rows at a time, their reads ahead of the first use
            W v[kRows][kTwo ? 2 : 1];
            int64_t to[kRows];
            int tok[kRows];
            int n = 0;
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                tok[r] = tk;
                if (tk < toks) {
                    const T* x = xs + (tok0 + tk) * a.x_token + h * a.x_head;
                    to[r] = (tok0 + tk) * a.out_token + h * a.out_head;
                    v[r][0] = *reinterpret_cast<const W*>(x + i0);
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
                    const float2* cs = s_cs + tok[r] * pairs + it * P;
                    T* e = reinterpret_cast<T*>(v[r]);
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const float2 z = cs[k];
                        T& e0 = e[HALF ? k : 2 * k];
                        T& e1 = e[HALF ? V + k : 2 * k + 1];
                        const float x0 = to_f<T>(e0), x1 = to_f<T>(e1);
                        e0 = from_f<T>(x0 * z.x - x1 * z.y);
                        e1 = from_f<T>(x1 * z.x + x0 * z.y);
                    }
                }
                *reinterpret_cast<W*>(ys + to[r] + i0) = v[r][0];
                if (kTwo && turns) *reinterpret_cast<W*>(ys + to[r] + i1) = v[r][kTwo ? 1 : 0];
            }
        }
    }
}

template <typename T, int V>
void launch_rope_as(const RopeArgs& a, hipStream_t stream) {
    const bool in_place = a.out == a.x;
    const int rot_items = a.rot / 2 / (a.half ? V : (V > 1 ? V / 2 : 1));
    const int items = rot_items + (in_place ? 0 : (a.dim - a.rot) / V);
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
    if (a.half)
        hipLaunchKernelGGL((rope_kernel<T, V, true>), grid, dim3(256), 0, stream, a, (int)tpb, lanes_log2, rot_items,
                           items);
    else
        hipLaunchKernelGGL((rope_kernel<T, V, false>), grid, dim3(256), 0, stream, a, (int)tpb, lanes_log2, rot_items,
                           items);
}

template <typename T>
void launch_rope_of(const RopeArgs& a, hipStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int64_t strides = a.x_token | a.x_head | a.out_token | a.out_head | a.dim | a.offset |
                            (a.half ? a.rot / 2 : a.rot);
    const bool wide = strides % V == 0 && ((uintptr_t)a.x | (uintptr_t)a.out) % 16 == 0;
    if (wide)
        launch_rope_as<T, V>(a, stream);
    else
        launch_rope_as<T, 1>(a, stream);
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
