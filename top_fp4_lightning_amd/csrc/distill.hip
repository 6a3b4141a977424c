// Distillation of score rows from a teacher's top logits: the divergence
//   L = sum_i p_i (log p_i - log q_{x_i}),  p = softmax(t / T) over the teacher's entries,
//   q = softmax(s / T) over the row's visible positions with a score above -inf,
// and its gradient dL/ds = (q - p) / T.
//
// Both directions are one pass over the row: the forward reads it (running maximum and sum per
// thread, base 2), the gradient reads it and writes as much, with the teacher's probabilities of a piece
// of the row laid out in LDS before the piece is streamed. They are bound by HBM: 4096 whole rows of 32768 scores
// (0.54 GB, moved three times) take 103 us forward and 294 us with the gradient (5.5 TB/s over both; a copy reaches 4.8).
// Few rows are cut into pieces of at least 4096 scores, so that the compute units have about four blocks each, and joined
// by a second launch
// (8 rows of 2^20: 7 and 5 us, the gradient 13).
#include <type_traits>

#include "operators.h"

namespace fp4idx {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kThreads = 256;
constexpr int kPiece = 4096;       // values whose teacher probabilities are in LDS at a time
constexpr int kPerThread = kMaxK / kThreads;

typedef float f4u __attribute__((ext_vector_type(4), aligned(4)));  // rows start at any fp32 address

__device__ __forceinline__ float ninf() { return -__builtin_inff(); }

// sum = l * exp(m / T). m is a value of the row itself and differences are taken before the factor
// c = log2(e) / T: values near the type's lowest would overflow with it.
struct MaxSum {
    float m, l;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float r = m == ninf() ? 0.0f : m;
    return MaxSum{m, a.l * __builtin_amdgcn_exp2f((a.m - r) * c) + b.l * __builtin_amdgcn_exp2f((b.m - r) * c)};
}
// (G: threads of the block, 256 or one wavefront)
template <int G>
__device__ __forceinline__ MaxSum block_join(MaxSum v, float c, MaxSum* lds) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = join(v, MaxSum{__shfl_xor(v.m, d), __shfl_xor(v.l, d)}, c);
    if (G == 64) return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return join(join(lds[0], lds[1], c), join(lds[2], lds[3], c), c);
}
template <int G>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    if (G == 64) return v;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__device__ __forceinline__ int32_t visible(const DistillArgs& a, int64_t t) {
    const int32_t n = a.n_vis[t];
    return n < 0 ? 0 : (n > a.max_n ? (int32_t)a.max_n : n);
}

// natural log of a sum
__device__ __forceinline__ double log_of(MaxSum v, float inv_temp) {
    return v.l == 0.0f ? -__builtin_inf() : (double)v.m * inv_temp + log((double)v.l);
}

// A thread's share of the row's teacher entries, asked for before the row's own sum is known: three dependent
// reads (position, score, logit) would otherwise stand at the end of every row.
struct Teacher {
    int32_t p[kPerThread];                 // positions, -1: not an entry
    float tl[kPerThread], sl[kPerThread];  // logits, the row's scores there
};
template <int G>
__device__ __forceinline__ void load_teacher(const DistillArgs& a, int64_t t, Teacher& e) {
    const int32_t n = visible(a, t);
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int i = k * G + (int)threadIdx.x;
        const int32_t p = i < a.k ? a.t_idx[t * a.t_stride + i] : -1;
        e.tl[k] = i < a.k ? a.t_logit[t * a.t_stride + i] : ninf();
        e.p[k] = p < n ? p : -1;
    }
}
__device__ __forceinline__ void load_scores(const float* __restrict__ s, Teacher& e) {
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
        if (e.p[k] >= 0) e.sl[k] = s[e.p[k]];
}

// The sum over s[i0 .. i1), this thread's share. With teacher entries (i0 = 0, the whole row), their scores are taken
// on the way, from a copy of each piece in LDS: read by themselves they would cost a line each (4096 rows of up to
// 32768 scores with 512 entries: 0.72 GB of reads in place of 0.49).
template <int G, bool TAKE>
__device__ __forceinline__ MaxSum row_part(const float* __restrict__ s, int32_t i0, int32_t i1, float c, Teacher* e,
                                           float* piece) {
    constexpr int kPart = 16 * G;
    MaxSum v{ninf(), 0.0f};
    for (int32_t p0 = i0; p0 < i1; p0 += kPart) {
        const int32_t i = p0 + (int32_t)threadIdx.x * 4;
        f4u x[4];
        if (p0 + kPart <= i1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const f4u*>(s + i + k * G * 4);
        } else {
            // the row's end; what is past it adds nothing
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int32_t ik = i + k * G * 4;
                if (ik + 4 <= i1) {
                    x[k] = *reinterpret_cast<const f4u*>(s + ik);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[k][j] = ik + j < i1 ? s[ik + j] : ninf();
                }
            }
        }
        if constexpr (TAKE) {
            if (p0) __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k) *reinterpret_cast<v4f*>(piece + (threadIdx.x + k * G) * 4) = x[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kPerThread; ++k)
                if (e->p[k] >= p0 && e->p[k] < p0 + kPart) e->sl[k] = piece[e->p[k] - p0];
        }
        float top = ninf();
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fmaxf(x[k][0], x[k][1]), fmaxf(x[k][2], x[k][3])));
        const float m = fmaxf(v.m, top);
        const float r = m == ninf() ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += __builtin_amdgcn_exp2f((x[k][j] - r) * c);
        v.l = v.l * __builtin_amdgcn_exp2f((v.m - r) * c) + sum;
        v.m = m;
    }
    return v;
}

// the row's end: the teacher's sum and the loss. Whole block.
template <int G>
__device__ __forceinline__ void finish_row(const DistillArgs& a, int64_t t, Teacher& e, MaxSum row,
                                           MaxSum* lds_ms, double* lds_d) {
    const float c = a.inv_temp * kLog2e;
    MaxSum v{ninf(), 0.0f};
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        if (e.p[k] < 0 || e.sl[k] == ninf()) e.tl[k] = ninf();
        if (e.tl[k] != ninf()) v = join(v, MaxSum{e.tl[k], 1.0f}, c);
    }
    v = block_join<G>(v, c, lds_ms);
    // differences to the largest first: a logarithm near the type's lowest value would swallow the sum's
    const double tlog = log((double)v.l), log_sum = log((double)row.l);
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
        if (e.tl[k] != ninf()) {
            const double d = ((double)e.tl[k] - v.m) * a.inv_temp - tlog;
            sum += (double)expf((float)d) * (d - (((double)e.sl[k] - row.m) * a.inv_temp - log_sum));
        }
    sum = block_sum<G>(sum, lds_d);
    if (threadIdx.x == 0) {
        a.loss[t] = (float)sum;
        a.lse[t] = (float)log_of(row, a.inv_temp);
        a.t_lse[t] = (float)log_of(v, a.inv_temp);
    }
}

// a block for every row
template <int G>
__global__ __launch_bounds__(G) void distill_kernel(const DistillArgs a) {
    __shared__ MaxSum s_ms[4];
    __shared__ double s_d[4];
    __shared__ __align__(16) float s_piece[16 * G];
    const int64_t t = blockIdx.x;
    const float c = a.inv_temp * kLog2e;
    Teacher e;
    load_teacher<G>(a, t, e);
    const MaxSum v = row_part<G, true>(a.scores + t * a.score_stride, 0, visible(a, t), c, &e, s_piece);
    finish_row<G>(a, t, e, block_join<G>(v, c, s_ms), s_ms, s_d);
}

// few rows: a block for a piece of one, whose (max, sum) it writes
__global__ __launch_bounds__(kThreads) void distill_piece_kernel(const DistillArgs a, int pieces) {
    __shared__ MaxSum s_ms[4];
    const int64_t t = blockIdx.x / pieces;
    const int piece = (int)(blockIdx.x % pieces);
    const int32_t n = visible(a, t);
    const int32_t per = ((n + pieces - 1) / pieces + 3) & ~3;
    const int32_t i0 = (int32_t)min((int64_t)piece * per, (int64_t)n);
    const int32_t i1 = (int32_t)min((int64_t)i0 + per, (int64_t)n);
    const float c = a.inv_temp * kLog2e;
    const float* s = a.scores + t * a.score_stride;
    const MaxSum v = block_join<kThreads>(row_part<kThreads, false>(s, i0, i1, c, nullptr, nullptr), c, s_ms);
    if (threadIdx.x == 0) reinterpret_cast<MaxSum*>(a.ws)[blockIdx.x] = v;
}

__global__ __launch_bounds__(kThreads) void distill_join_kernel(const DistillArgs a, int pieces) {
    __shared__ MaxSum s_ms[4];
    __shared__ double s_d[4];
    const int64_t t = blockIdx.x;
    const float c = a.inv_temp * kLog2e;
    Teacher e;
    load_teacher<kThreads>(a, t, e);
    load_scores(a.scores + t * a.score_stride, e);
    MaxSum v{ninf(), 0.0f};
    for (int i = threadIdx.x; i < pieces; i += kThreads)
        v = join(v, reinterpret_cast<const MaxSum*>(a.ws)[t * pieces + i], c);
    v = block_join<kThreads>(v, c, s_ms);
    finish_row<kThreads>(a, t, e, v, s_ms, s_d);
}

__device__ __forceinline__ float softmax_of(float x, float inv_temp, float lse) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(x, inv_temp, -lse) * kLog2e);
}

// From this size of a logarithm on, a row's gradient takes its sums again, as (largest, sum): half a step of fp32 at
// the logarithm is 2^-15 of every q and p below it and 1 at 2^24 (a row of equal scores at the type's lowest value would
// get q = 1 for each). What that costs, against rows about zero: 4096 rows of 32768 scores 215 -> 288 us, 64 of 131072
// 16 -> 121, 8 of 2^20 15 -> 860.
constexpr float kFar = 1024.0f;

// Gradient: a block takes a range of whole pieces of one row. The last rows come first: after the forward the last-level
// cache holds those. PAST: the gradient is written past that cache, which leaves it to the scores. A far row is one
// block's: in place, another's writes would be in the sums.
template <bool PAST>
__global__ __launch_bounds__(kThreads) void distill_bwd_kernel(const DistillArgs a, int blocks_per_row) {
    __shared__ float s_p[kPiece];
    __shared__ MaxSum s_ms[4];
    const int64_t t = a.nq - 1 - (int64_t)(blockIdx.x / blocks_per_row);
    const int part = (int)(blockIdx.x % blocks_per_row);
    const int32_t n = visible(a, t);
    const int32_t pieces = (n + kPiece - 1) / kPiece;
    const float tlse = a.t_lse[t];
    const float lse = a.lse[t];
    const bool far = tlse != ninf() && (fabsf(lse) >= kFar || fabsf(tlse) >= kFar);
    const int32_t per = far ? pieces : (pieces + blocks_per_row - 1) / blocks_per_row;
    const int32_t p0 = min(part * per, pieces), p1 = min(p0 + per, pieces);
    if (p0 >= p1) return;
    const float* s = a.scores + t * a.score_stride;
    float* d = a.dscores + t * a.d_stride;
    const float gain = tlse == ninf() ? 0.0f : a.dloss[t] * a.inv_temp;
    if (tlse == ninf()) {  // no teacher entry: no gradient
        for (int32_t i = p0 * kPiece + (int32_t)threadIdx.x; i < min(p1 * kPiece, n); i += kThreads) d[i] = 0.0f;
        return;
    }
    // A position given several times sums in one order in every run: each wavefront has 512 consecutive slots, and
    // the wavefronts add theirs one after the other (one turn up to 512 slots).
    const int wave = (int)(threadIdx.x >> 6), turns = (a.k + kMaxK / 4 - 1) / (kMaxK / 4);
    int32_t at[kPerThread];
    float p[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int i = (wave * kPerThread + k) * 64 + (int)(threadIdx.x & 63);
        at[k] = -1;
        p[k] = ninf();
        if (i < a.k) {
            at[k] = a.t_idx[t * a.t_stride + i];
            p[k] = a.t_logit[t * a.t_stride + i];
        }
        if (!far) p[k] = p[k] == ninf() ? 0.0f : softmax_of(p[k], a.inv_temp, tlse);
    }
    const float c = a.inv_temp * kLog2e;
    float row_m = 0.0f, row_inv = 0.0f;
    if (far) {
        const MaxSum row = block_join<kThreads>(row_part<kThreads, false>(s, 0, n, c, nullptr, nullptr), c, s_ms);
        row_m = row.m;
        row_inv = 1.0f / row.l;
        MaxSum v{ninf(), 0.0f};
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
            if (at[k] < 0 || at[k] >= n || s[at[k]] == ninf()) p[k] = ninf();
            if (p[k] != ninf()) v = join(v, MaxSum{p[k], 1.0f}, c);
        }
        v = block_join<kThreads>(v, c, s_ms);
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) p[k] = __builtin_amdgcn_exp2f((p[k] - v.m) * c) / v.l;
    }
    const auto q_of = [&](auto is_far, float x) {
        if constexpr (decltype(is_far)::value) return __builtin_amdgcn_exp2f((x - row_m) * c) * row_inv;
        else return softmax_of(x, a.inv_temp, lse);
    };
    const auto stream_piece = [&](auto is_far, int32_t i0, int32_t i1) {
        for (int32_t i = i0 + (int32_t)threadIdx.x * 4; i < i1; i += kThreads * 4) {
            const v4f pv = *reinterpret_cast<const v4f*>(s_p + (i - i0));
            if (i + 4 <= i1) {
                const f4u x = *reinterpret_cast<const f4u*>(s + i);
                f4u y;
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = x[j] == ninf() ? 0.0f : gain * (q_of(is_far, x[j]) - pv[j]);
                if constexpr (PAST)
                    __builtin_nontemporal_store(y, reinterpret_cast<f4u*>(d + i));
                else
                    *reinterpret_cast<f4u*>(d + i) = y;
            } else {
                for (int j = 0; i + j < i1; ++j) {
                    const float x = s[i + j];
                    d[i + j] = x == ninf() ? 0.0f : gain * (q_of(is_far, x) - pv[j]);
                }
            }
        }
    };
    for (int32_t pc = p0; pc < p1; ++pc) {
        const int32_t i0 = pc * kPiece, i1 = min(i0 + kPiece, n);
        for (int i = threadIdx.x * 4; i < kPiece; i += kThreads * 4) *reinterpret_cast<v4f*>(s_p + i) = v4f{};
        for (int turn = 0; turn < turns; ++turn) {
            __syncthreads();
            if (wave != turn) continue;
#pragma unroll
            for (int k = 0; k < kPerThread; ++k)
                if (at[k] >= i0 && at[k] < i1) atomicAdd(s_p + (at[k] - i0), p[k]);
        }
        __syncthreads();
        if (far)
            stream_piece(std::true_type{}, i0, i1);
        else
            stream_piece(std::false_type{}, i0, i1);
        __syncthreads();
    }
}

}  // namespace

// Blocks per row: one while the rows alone give every compute unit four blocks, else enough for that
// with at least 4096 values each.
int distill_pieces(int32_t nq, int64_t max_n) {
    if (nq <= 0 || nq >= 1024) return 1;
    const int64_t want = (1024 + nq - 1) / nq, most = (max_n + kPiece - 1) / kPiece;
    return (int)(want < most ? want : (most < 1 ? 1 : most));
}

// For any number of rows up to nq and any length up to max_n: r ceil(1024 / r) pieces are below 1024 + r, of fewer than
// 1024 rows (more are whole).
size_t distill_workspace_bytes(int32_t nq, int64_t max_n) {
    const int64_t most = (max_n + kPiece - 1) / kPiece;
    if (nq <= 0 || most <= 1) return 16;
    const int64_t all = nq * most, few = 1023 + (nq < 1023 ? nq : 1023);
    return (size_t)(all < few ? all : few) * sizeof(MaxSum);
}

hipError_t launch_distill(const DistillArgs& a, hipStream_t stream) {
    const int pieces = distill_pieces(a.nq, a.max_n);
    if (pieces == 1) {
        // Many short rows: a wavefront each, which has no barriers to wait at (4096 rows of 500 scores 21 -> 12 us, of
        // 16000 49 -> 48, 20000 of 2000 91 -> 46; 1024 rows 11 -> 12).
        if (a.nq >= 2048 && a.max_n <= 16384 && a.k <= 64 * kPerThread)
            hipLaunchKernelGGL(distill_kernel<64>, dim3((unsigned)a.nq), dim3(64), 0, stream, a);
        else
            hipLaunchKernelGGL(distill_kernel<kThreads>, dim3((unsigned)a.nq), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(distill_piece_kernel, dim3((unsigned)a.nq * pieces), dim3(kThreads), 0, stream, a, pieces);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL(distill_join_kernel, dim3((unsigned)a.nq), dim3(kThreads), 0, stream, a, pieces);
    return hipGetLastError();
}

hipError_t launch_distill_bwd(const DistillArgs& a, hipStream_t stream) {
    const int pieces = distill_pieces(a.nq, a.max_n);
    // Past the 256 MB cache from 128 MB of scores on. Both directions and a read of the gradient, us (past / not): 1024 x
    // 32768 100 / 102, 2048 206 / 225, 4096 395 / 416; 256 (32 MB) 43 / 40.
    const dim3 grid((unsigned)a.nq * pieces);
    if ((int64_t)a.nq * a.max_n >= (int64_t)1 << 25)
        hipLaunchKernelGGL(distill_bwd_kernel<true>, grid, dim3(kThreads), 0, stream, a, pieces);
    else
        hipLaunchKernelGGL(distill_bwd_kernel<false>, grid, dim3(kThreads), 0, stream, a, pieces);
    return hipGetLastError();
}

}  // namespace fp4idx
