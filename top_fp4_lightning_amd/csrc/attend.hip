// Core attention over the FP4 main-KV cache (rows of 512 values, E2M1 codes with an E4M3 scale per
// 16), for chunks of new tokens and for single ones: over everything a query sees, or over its
// selected positions.
//
//   s_{h,i} = scale * q_h . kv_i,  p = softmax_i(s_h),  o_h = sum_i p_{h,i} kv_i   (one row is key and value)
//
// One pass over the entries with a running maximum M and sum l per head (base 2: s2 = s * log2 e).
// A block of four wavefronts takes 32 heads of one query and 64 entries at a time: wavefront w
// multiplies entries 16w .. 16w+15 with all 32 heads, then values 128w .. 128w+127 of all 64 entries
// with the probabilities.
//
// Arithmetic. An E2M1 code times an E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688]: exact in fp16. A query row is multiplied by the power of two that brings its largest
// value to [2^14, 2^15); its bf16 values are then exact in fp16 down to 2^-28 of the row's largest
// (below that they lose bits worth less than 2^-39 of it). Products and sums are fp32 in the matrix
// units. Probabilities enter the second product as fp16 values in (0, 2^14] (11 bits; the offset keeps
// them normal numbers down to 2^-28 of the largest).
#include "operators.h"

namespace fp4idx {
namespace {

constexpr int kD = 512;
constexpr int kTile = 64;        // entries per step
constexpr int kHeadTile = 32;    // heads per block
constexpr int kRow = kD + 16;    // LDS row of a tile in fp16 values (the pad spreads rows over the banks)
constexpr int kPRow = kTile + 8;
constexpr float kPBits = 14.0f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __fp16 hv4 __attribute__((vector_size(8)));
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) hv4 lds_hv4;

__device__ __forceinline__ float ninf() { return -__builtin_inff(); }

// The entries of one query and where their rows lie.
struct Entries {
    int32_t visible;    // n_vis clamped to 0 .. max_n
    int32_t n;          // the same, 0 where no position has a row
    int32_t first;      // range form: the first position
    int32_t count;      // entries: list slots, or positions first .. first + count - 1
    const int32_t* list;
    const int32_t* pages;
    int64_t base;
};

__device__ __forceinline__ Entries entries_of(const AttendArgs& a, int64_t t) {
    Entries e;
    int64_t n = a.n_vis[t];
    n = n < 0 ? 0 : (n > a.max_n ? a.max_n : n);
    e.visible = (int32_t)n;
    e.base = 0;
    e.pages = nullptr;
    if (a.pages) {
        const int64_t s = a.seq ? (int64_t)a.seq[t] : t;
        if (s < 0 || s >= a.nseq) n = 0;
        else e.pages = a.pages + s * a.pages_stride;
    } else {
        e.base = a.kv_base[t];
        if (e.base <= -a.max_n || e.base >= a.rows) n = 0;  // no position lies in the cache
    }
    if (a.rows == 0) n = 0;
    e.n = (int32_t)n;
    e.list = a.idx ? a.idx + t * a.idx_stride : nullptr;
    e.first = (!a.idx && a.window > 0 && n > a.window) ? (int32_t)(n - a.window) : 0;
    e.count = a.idx ? (n > 0 ? a.k : 0) : (int32_t)n - e.first;
    return e;
}

// cache row of entry i, or -1 (past the end, a position that is not visible, a row outside the cache)
__device__ __forceinline__ int32_t row_of(const AttendArgs& a, const Entries& e, int i) {
    if (i >= e.count) return -1;
    const int32_t p = e.list ? e.list[i] : e.first + i;
    if (p < 0 || p >= e.n) return -1;
    int64_t r;
    if (e.pages) {
        const uint32_t pg = (uint32_t)p / (uint32_t)a.page_size;
        const int64_t page = e.pages[pg];
        if (page < 0) return -1;
        r = page * a.page_size + (p - (int32_t)(pg * (uint32_t)a.page_size));
    } else {
        r = e.base + p;
    }
    return (r >= 0 && r < a.rows) ? (int32_t)r : -1;
}

// One lane's share of a cache row: lane group g (of 4) holds, for j = 0 .. 3, values 128j + 32g ..
// 128j + 32g + 31: sixteen code bytes and two scales. The four groups read 64 consecutive bytes.
struct RowPart {
    uint4 code[4];
    uint32_t scale[4];
};

__device__ __forceinline__ void load_row(const AttendArgs& a, int32_t row, int g, RowPart& r) {
    const int64_t at = row < 0 ? 0 : row;
    const uint8_t* c = a.codes + at * 256 + g * 16;
    const uint8_t* s = a.scales + at * 32 + g * 2;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        r.code[j] = *reinterpret_cast<const uint4*>(c + 64 * j);
        r.scale[j] = *reinterpret_cast<const uint16_t*>(s + 8 * j);
    }
    // a row that is not there counts as zeros (codes are always finite)
    if (row < 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r.scale[j] = 0;
    }
}

// values 8u .. 8u+7 of chunk j as fp16 (exact)
__device__ __forceinline__ h8 values8(const RowPart& r, int j, int u) {
    const uint32_t w = u == 0 ? r.code[j].x : u == 1 ? r.code[j].y : u == 2 ? r.code[j].z : r.code[j].w;
    const h2 sp = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)r.scale[j], 1.0f, false);
    const _Float16 s1 = u < 2 ? sp[0] : sp[1];
    const h2 s = {s1, s1};
    const h2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
    const h2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
    const h2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
    const h2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
    return h8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// 32 query rows (heads h0 .. h0+31, rows past the last head as zeros) into LDS as scaled fp16, and
// per head the factor that turns a dot product of theirs into s2: 8 rows per wavefront, a row per
// step, 8 values per lane.
__device__ __forceinline__ void stage_query(const AttendArgs& a, int64_t t, int h0, _Float16* lds, float* factor) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    uint4 raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int h = h0 + w * 8 + i;
        raw[i] = uint4{0, 0, 0, 0};
        if (h < a.heads) raw[i] = *reinterpret_cast<const uint4*>(a.q + (t * a.heads + h) * kD + lane * 8);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t hi = v[c] & 0x7fff0000u, lo = (v[c] << 16) & 0x7fff0000u;
            m = max(m, max(hi, lo));
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
        // 2^(14 - exponent of the largest), a power of two kept inside the normal range
        int e = (int)(m >> 23);
        e = e < 15 ? 15 : (e > 254 ? 254 : e);
        const float mul = __uint_as_float((uint32_t)(127 + 141 - e) << 23);
        h8 o;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            o[2 * c] = (_Float16)(__uint_as_float(v[c] << 16) * mul);
            o[2 * c + 1] = (_Float16)(__uint_as_float(v[c] & 0xffff0000u) * mul);
        }
        *reinterpret_cast<h8*>(lds + (w * 8 + i) * kRow + lane * 8) = o;
        if (lane == 0) factor[w * 8 + i] = a.scale * kLog2e * __uint_as_float((uint32_t)(e - 14) << 23);
    }
}

// block -> (query and part, head tile): the head tiles of one query run on one XCD (blocks b and
// b + 8 do), so the second reads the rows from that XCD's L2
__device__ __forceinline__ bool unit_of(uint32_t b, uint32_t units, uint32_t tiles, uint32_t& unit, uint32_t& tile) {
    const uint32_t per = 8 * tiles;
    unit = b / per * 8 + (b & 7);
    tile = b % per / 8;
    return unit < units;
}

// Registers per lane: 128 of the queries, 64 of the outputs.
__global__ __launch_bounds__(256, 2) void attend_kernel(const AttendArgs a, int splits) {
    __shared__ __align__(16) _Float16 s_kv[kTile * kRow];
    __shared__ __align__(16) _Float16 s_p[kHeadTile * kPRow];
    __shared__ __align__(16) float s_m[kHeadTile][4];
    __shared__ __align__(16) float s_l[kHeadTile][4];
    __shared__ float s_factor[kHeadTile];

    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    const uint32_t head_tiles = (a.heads + kHeadTile - 1) / kHeadTile;
    uint32_t unit, tile;
    if (!unit_of(blockIdx.x, (uint32_t)a.nq * splits, head_tiles, unit, tile)) return;
    const int64_t t = unit / splits;
    const int part = (int)(unit % splits);
    const int h0 = (int)tile * kHeadTile;
    const Entries e = entries_of(a, t);
    const int steps_all = (e.count + kTile - 1) / kTile;
    const int per = (steps_all + splits - 1) / splits;
    const int step0 = part * per;
    const int step1 = min(step0 + per, steps_all);

    RowPart kv;
    int32_t row = -1, row_next = -1;
    if (step0 < step1) {
        row = row_of(a, e, step0 * kTile + w * 16 + c);
        load_row(a, row, g, kv);
        row_next = row_of(a, e, (step0 + 1) * kTile + w * 16 + c);
    }

    stage_query(a, t, h0, s_kv, s_factor);
    __syncthreads();
    h8 q[2][16];
    float f[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        f[hf] = s_factor[hf * 16 + c];
#pragma unroll
        for (int x = 0; x < 16; ++x)
            q[hf][x] = *reinterpret_cast<const h8*>(s_kv + (hf * 16 + c) * kRow + (x >> 2) * 128 + g * 32 + (x & 3) * 8);
    }
    v4f o[2][8] = {};
    float M[2] = {ninf(), ninf()};   // maximum (an integer) that all four wavefronts know
    float m[2] = {ninf(), ninf()};   // reference of this wavefront's sum
    float l[2] = {0.0f, 0.0f};       // this lane's part of it

    for (int step = step0; step < step1; ++step) {
        __syncthreads();  // the last step's reads of s_kv, s_p and s_m are done
        v4f s[2] = {};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const h8 v = values8(kv, j, u);
                s[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, q[0][j * 4 + u], s[0], 0, 0, 0);
                s[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, q[1][j * 4 + u], s[1], 0, 0, 0);
                *reinterpret_cast<h8*>(s_kv + (w * 16 + c) * kRow + j * 128 + g * 32 + u * 8) = v;
            }
        }
        const uint32_t seen = (uint32_t)__ballot(row >= 0) >> (g * 4);
        // the next step's rows travel while this one is finished
        row = row_next;
        if (step + 1 < step1) {
            load_row(a, row, g, kv);
            row_next = row_of(a, e, (step + 2) * kTile + w * 16 + c);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            float x[4];
            float top = ninf();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = (seen >> i) & 1 ? s[hf][i] * f[hf] : ninf();
                top = fmaxf(top, x[i]);
            }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float mn = fmaxf(M[hf], ceilf(top));
            const float ref = mn == ninf() ? 0.0f : mn - kPBits;
            float sum = 0.0f;
            h4 p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ex = __builtin_amdgcn_exp2f(x[i] - ref);
                sum += ex;
                p[i] = (_Float16)ex;
            }
            l[hf] = l[hf] * (m[hf] == ninf() ? 0.0f : __builtin_amdgcn_exp2f(m[hf] - mn)) + sum;
            m[hf] = mn;
            *reinterpret_cast<h4*>(s_p + (hf * 16 + c) * kPRow + w * 16 + g * 4) = p;
            if (g == 0) s_m[hf * 16 + c][w] = mn;
        }
        __syncthreads();
        // bring the four wavefronts' probabilities to one maximum: powers of two, exact
        h8 p[2][2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const v4f mv = *reinterpret_cast<const v4f*>(s_m[hf * 16 + c]);
            const float mx = fmaxf(fmaxf(mv[0], mv[1]), fmaxf(mv[2], mv[3]));
            const float shift = mx == ninf() ? 0.0f : mx;
            const float alpha = __builtin_amdgcn_exp2f(M[hf] - shift);  // 0 before the first maximum (o is 0 then)
            M[hf] = mx;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const float mw = g < 2 ? mv[2 * ks] : mv[2 * ks + 1];
                const _Float16 r = (_Float16)__builtin_amdgcn_exp2f(mw - shift);
                p[hf][ks] = *reinterpret_cast<const h8*>(s_p + (hf * 16 + c) * kPRow + ks * 32 + g * 8) * r;
            }
            if (__any(alpha != 1.0f)) {
#pragma unroll
                for (int d = 0; d < 8; ++d) o[hf][d] *= alpha;
            }
        }
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                // a transposed read: lane group g gets entries 32 ks + 8 g .. + 7 of value 16 d + c
                _Float16* at = s_kv + (ks * 32 + g * 8 + (c >> 2)) * kRow + w * 128 + d * 16 + (c & 3) * 4;
                const hv4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)at);
                const hv4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(at + 4 * kRow));
                h8 v;
                __builtin_memcpy(&v, &lo, 8);
                __builtin_memcpy((char*)&v + 8, &hi, 8);
                o[0][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[0][ks], o[0][d], 0, 0, 0);
                o[1][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[1][ks], o[1][d], 0, 0, 0);
            }
        }
    }

    // the sum over the four lane groups and the four wavefronts, each relative to its own maximum
    __syncthreads();
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        float x = l[hf];
        x += __shfl_xor(x, 16);
        x += __shfl_xor(x, 32);
        if (g == 0) {
            s_l[hf * 16 + c][w] = x;
            s_m[hf * 16 + c][w] = m[hf];
        }
    }
    __syncthreads();
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int hl = hf * 16 + c;
        const v4f mv = *reinterpret_cast<const v4f*>(s_m[hl]);
        const v4f lv = *reinterpret_cast<const v4f*>(s_l[hl]);
        float L = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) L += mv[i] == ninf() ? 0.0f : lv[i] * __builtin_amdgcn_exp2f(mv[i] - M[hf]);
        const int h = h0 + hl;
        if (splits > 1) {
            const int64_t r = (int64_t)(unit * head_tiles + tile) * kHeadTile + hl;
            float* po = a.part_o + r * kD + w * 128 + g * 4;
#pragma unroll
            for (int d = 0; d < 8; ++d) *reinterpret_cast<v4f*>(po + d * 16) = o[hf][d];
            if (w == 0 && g == 0) {
                a.part_ml[2 * r] = M[hf];
                a.part_ml[2 * r + 1] = L;
            }
        } else if (h < a.heads) {
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            uint16_t* po = a.out + (t * a.heads + h) * kD + w * 128 + g * 4;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const v4f y = o[hf][d] * inv;
                *reinterpret_cast<uint2*>(po + d * 16) = uint2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
            }
            if (a.lse && w == 0 && g == 0)
                a.lse[t * a.heads + h] = L == 0.0f ? ninf() : (M[hf] + __builtin_amdgcn_logf(L) - kPBits) * kLn2;
        }
    }
}

// join of the parts of one (query, head): 128 threads, 4 values each
__global__ __launch_bounds__(128) void attend_join_kernel(const AttendArgs a, int splits) {
    const int64_t t = blockIdx.x / a.heads;
    const int h = (int)(blockIdx.x % a.heads);
    const int head_tiles = (a.heads + kHeadTile - 1) / kHeadTile;
    const int64_t first = ((t * splits) * head_tiles + h / kHeadTile) * kHeadTile + h % kHeadTile;
    const int64_t step = (int64_t)head_tiles * kHeadTile;
    float M = ninf();
    for (int i = 0; i < splits; ++i) M = fmaxf(M, a.part_ml[2 * (first + i * step)]);
    const float ref = M == ninf() ? 0.0f : M;
    float L = 0.0f;
    v4f o = {};
    for (int i = 0; i < splits; ++i) {
        const int64_t r = first + i * step;
        const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * r] - ref);
        L += f * a.part_ml[2 * r + 1];
        o += f * *reinterpret_cast<const v4f*>(a.part_o + r * kD + threadIdx.x * 4);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    o *= inv;
    *reinterpret_cast<uint2*>(a.out + (int64_t)blockIdx.x * kD + threadIdx.x * 4) =
        uint2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    if (a.lse && threadIdx.x == 0)
        a.lse[blockIdx.x] = L == 0.0f ? ninf() : (M + __builtin_amdgcn_logf(L) - kPBits) * kLn2;
}

// The attention's probability of every entry, mean over the heads, from the saved lse:
//   w_i = 1/H sum_h exp(s_{h,i} - lse_h).
// The first product alone; entries are independent, so a query's entries spread over blocks freely.
// Heads beyond 32 are further rounds over the same entries, added by the lane that wrote them.
__global__ __launch_bounds__(256, 2) void attend_weights_kernel(const AttendArgs a, const float* __restrict__ lse,
                                                                float* __restrict__ weights, int64_t w_stride,
                                                                int splits) {
    __shared__ __align__(16) _Float16 s_q[kHeadTile * kRow];
    __shared__ float s_factor[kHeadTile];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    const int64_t t = blockIdx.x / splits;
    const int part = (int)(blockIdx.x % splits);
    const Entries e = entries_of(a, t);
    // a list's slots are all written; of a range, the visible positions
    const int slots = a.idx ? a.k : e.visible;
    const int steps_all = (slots + kTile - 1) / kTile;
    const int per = (steps_all + splits - 1) / splits;
    const int step0 = part * per;
    const int step1 = min(step0 + per, steps_all);
    if (step0 >= step1) return;
    float* out = weights + t * w_stride;
    if (e.count == 0) {  // no row is read (the cache may hold none)
        for (int i = step0 * kTile + (int)threadIdx.x; i < min(step1 * kTile, slots); i += 256) out[i] = 0.0f;
        return;
    }
    const float mean = 1.0f / (float)a.heads;

    for (int h0 = 0; h0 < a.heads; h0 += kHeadTile) {
        __syncthreads();
        stage_query(a, t, h0, s_q, s_factor);
        __syncthreads();
        h8 q[2][16];
        float f[2][4], off[2][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int hl = hf * 16 + g * 4 + i;
                f[hf][i] = s_factor[hl];
                // a head that is not there, or that saw nothing, adds nothing
                float y = h0 + hl < a.heads ? lse[t * a.heads + h0 + hl] : ninf();
                off[hf][i] = y == ninf() ? __builtin_inff() : y * kLog2e;
            }
#pragma unroll
            for (int x = 0; x < 16; ++x)
                q[hf][x] =
                    *reinterpret_cast<const h8*>(s_q + (hf * 16 + c) * kRow + (x >> 2) * 128 + g * 32 + (x & 3) * 8);
        }
        for (int step = step0; step < step1; ++step) {
            const int i = step * kTile + w * 16 + c;
            const int32_t row = row_of(a, e, i);
            RowPart kv;
            load_row(a, row, g, kv);
            v4f s[2] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const h8 v = values8(kv, j, u);
                    s[0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[0][j * 4 + u], v, s[0], 0, 0, 0);
                    s[1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[1][j * 4 + u], v, s[1], 0, 0, 0);
                }
            }
            float sum = 0.0f;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sum += __builtin_amdgcn_exp2f(__builtin_fmaf(s[hf][k], f[hf][k], -off[hf][k]));
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (g == 0 && i < slots) {
                const float x = row >= 0 ? sum * mean : 0.0f;
                out[i] = h0 ? out[i] + x : x;
            }
        }
    }
}

}  // namespace

// Parts per query: enough blocks for two on each of the 256 compute units, at least one step of 64
// entries each.
int attend_splits(int32_t nq, int32_t heads, int64_t entries) {
    if (nq <= 0 || heads <= 0 || entries <= 0) return 1;
    const int64_t blocks = (int64_t)nq * ((heads + kHeadTile - 1) / kHeadTile);
    const int64_t steps = (entries + kTile - 1) / kTile;
    const int64_t want = (512 + blocks - 1) / blocks;
    return (int)(want < steps ? want : steps);
}

size_t attend_workspace_bytes(int32_t nq, int32_t heads, int64_t entries) {
    const int64_t splits = attend_splits(nq, heads, entries);
    if (splits <= 1) return 16;
    const size_t rows = (size_t)nq * splits * ((heads + kHeadTile - 1) / kHeadTile) * kHeadTile;
    return rows * (kD + 2) * sizeof(float);
}

hipError_t launch_attend(AttendArgs a, void* ws, hipStream_t stream) {
    const int64_t entries = a.idx ? a.k : (a.window > 0 && a.window < a.max_n ? a.window : a.max_n);
    const int splits = attend_splits(a.nq, a.heads, entries);
    const uint32_t head_tiles = (a.heads + kHeadTile - 1) / kHeadTile;
    if (splits > 1) {
        const size_t rows = (size_t)a.nq * splits * head_tiles * kHeadTile;
        a.part_o = (float*)ws;
        a.part_ml = a.part_o + rows * kD;
    }
    const uint32_t units = (uint32_t)a.nq * splits;
    hipLaunchKernelGGL(attend_kernel, dim3((units + 7) / 8 * 8 * head_tiles), dim3(256), 0, stream, a, splits);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || splits <= 1) return err;
    hipLaunchKernelGGL(attend_join_kernel, dim3((uint32_t)a.nq * a.heads), dim3(128), 0, stream, a, splits);
    return hipGetLastError();
}

hipError_t launch_attend_weights(const AttendArgs& a, const float* lse, float* weights, int64_t w_stride,
                                 hipStream_t stream) {
    const int64_t entries = a.idx ? a.k : a.max_n;
    if (entries == 0) return hipSuccess;
    const int splits = attend_splits(a.nq, kHeadTile, entries);
    hipLaunchKernelGGL(attend_weights_kernel, dim3((uint32_t)a.nq * splits), dim3(256), 0, stream, a, lse, weights,
                       w_stride, splits);
    return hipGetLastError();
}

}  // namespace fp4idx
