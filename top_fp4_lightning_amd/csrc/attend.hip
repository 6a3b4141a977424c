// Core attention over the FP4 main-KV cache (rows of 512 values, E2M1 codes with an E4M3 scale per
// 16), for chunks of new tokens and for single ones: over everything a query sees, or over its
// selected positions.
//
//   s_{h,i} = scale * q_h . kv_i,  p = softmax_i(s_h),  o_h = sum_i p_{h,i} kv_i   (one row is key and value)
//
// One pass over the entries with a running maximum M and sum l per head (base 2: s2 = s * log2 e).
// A block of four wavefronts takes 16, 32 or 64 heads of one query and 64 entries per step. Wavefront w
// reads the rows of entries 16w .. 16w+15 straight into registers, widens them to fp16 there, multiplies
// them with all heads of the block and leaves them in LDS; after a barrier it multiplies values
// 128w .. 128w+127 of all 64 entries with the probabilities. So every row is widened once, and read from
// LDS once (transposed). Queries and outputs stay in registers: at 64 heads 256 + 128 of a lane's 512.
//
// Arithmetic. An E2M1 code times an E4M3 scale has at most 6 significant bits and lies in
// [2^-10, 2688]: exact in fp16. A query row is multiplied by the power of two that brings its largest
// value to [2^14, 2^15); its bf16 values are then exact in fp16 down to 2^-28 of the row's largest
// (below that they lose bits worth less than 2^-39 of it). Products and sums are fp32 in the matrix
// units. Probabilities enter the second product as fp16 values (11 bits) up to 2^15, the largest so far of a
// head above 2^6: values down to 2^-20 of it are normal numbers, and what rounds to zero is below 2^-31 of it.
//
// What bounds it. Per step and wavefront at 64 heads: 2048 cycles of matrix instructions (64 of 16x16x32, 32 of
// 32x32x16) and about 290 others, in 1.65 us. The matrix units are busy 46% of the time (counters, 514 queries): one
// wavefront per SIMD issues everything in order, since queries and outputs fill its registers, and what it waits for
// adds up, none of it large: 16-byte LDS writes (52 cycles for the four wavefronts' one), transposed reads, the
// barrier and the probabilities between the two products. Leaving any one of these out saved 1 to 14%.
// Measured at 64 heads, in sessions that differ: 4096 queries over 512 listed rows 373 to 401 us (0.69 to 0.74 PFLOP/s; a
// block's query, first rows and output take 11 of its 24 us), 514 over about 14600 rows 903 to 973 us (0.99 to 1.06), 8 over
// about 115000 rows 142 us (0.85).
// Measured and not taken: rows kept as codes in LDS and widened twice (a step 20% slower), eight wavefronts of 256
// registers (spills, three times slower), two blocks of 32 heads per compute unit (equal), blocks that take
// several queries (+10%), the probabilities under the next step's first product (+5%), stores past the cache (equal).
#include <type_traits>

#include "operators.h"

namespace fp4idx {
namespace {

constexpr int kD = 512;
constexpr int kTile = 64;        // entries per step
constexpr int kRow = kD + 16;    // LDS row of a query or an output in 16-bit values (the pad spreads rows over the banks)
constexpr int kPRow = kTile + 8;
constexpr int kQRow = 32;
constexpr int kMostParts = 256;         // of a query's entries
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

// An entry's row is found in three stages, so that a kernel can keep the loads of each in flight: its position, its
// page, its row. No branches: an entry that is not there (past the end, not visible, outside the cache) reads
// a place that is and becomes row -1. Only for queries with entries.
template <bool LIST>
__device__ __forceinline__ int32_t position_of(const Entries& e, int i, int end) {
    const int32_t p = LIST ? e.list[min(i, end - 1)] : e.first + i;
    return i < end ? p : -1;
}
__device__ __forceinline__ uint32_t page_index(const AttendArgs& a, uint32_t p) {
    return __umulhi(2 * p, a.page_mul) >> a.page_shift;
}
template <bool PAGED>
__device__ __forceinline__ int32_t page_of(const AttendArgs& a, const Entries& e, int32_t p) {
    if (!PAGED) return 0;
    return e.pages[page_index(a, (uint32_t)p < (uint32_t)e.n ? (uint32_t)p : 0u)];
}
template <bool PAGED>
__device__ __forceinline__ int32_t row_of(const AttendArgs& a, const Entries& e, int32_t p, int32_t page) {
    bool there = (uint32_t)p < (uint32_t)e.n;
    uint32_t r;
    if (PAGED) {
        const uint32_t in_page = (uint32_t)p - page_index(a, (uint32_t)p) * (uint32_t)a.page_size;
        const uint64_t at = (uint64_t)(uint32_t)page * (uint32_t)a.page_size + in_page;
        there &= page >= 0 && at < (uint64_t)a.rows;
        r = (uint32_t)at;
    } else {
        // the base lies in (-2^30, rows) and p in [0, 2^30): a sum below zero wraps above any row
        r = (uint32_t)e.base + (uint32_t)p;
        there &= r < (uint32_t)a.rows;
    }
    return there ? (int32_t)r : -1;
}

// One lane's share of a cache row: lane group g (of 4) holds values 128g .. 128g + 127, 64 code bytes (read 16 at a
// time) and eight scales. (The products take the values in any order that queries and rows share. A read of 16 bytes
// by every lane touches 64 places and holds the address unit for as many cycles; with 32 values of each 128 per
// lane group, the scales took four reads and the address unit bounded the weights' kernel.)
typedef uint32_t u32_by2 __attribute__((aligned(2)));  // scales lie at any even address
struct RowPart {
    uint4 code[4];
    uint32_t scale[2];
};

// chunk j of a row and the scales; a row that is not there counts as zeros (codes are always finite)
__device__ __forceinline__ void load_chunk(const AttendArgs& a, int32_t row, int g, int j, RowPart& r) {
    const int64_t at = row < 0 ? 0 : row;
    r.code[j] = *reinterpret_cast<const uint4*>(a.codes + at * 256 + g * 64 + 16 * j);
}
__device__ __forceinline__ void load_scales(const AttendArgs& a, int32_t row, int g, uint32_t (&scale)[2]) {
    const u32_by2* at = reinterpret_cast<const u32_by2*>(a.scales + (int64_t)(row < 0 ? 0 : row) * 32 + g * 8);
    scale[0] = at[0];
    scale[1] = at[1];
}

// values 8x .. 8x + 7 of the part as fp16 (exact); there: the row is in the cache
__device__ __forceinline__ h8 values8(const RowPart& r, int x, bool there) {
    const uint4 c = r.code[x >> 2];
    const uint32_t w = (x & 3) == 0 ? c.x : (x & 3) == 1 ? c.y : (x & 3) == 2 ? c.z : c.w;
    const int e = there ? (int)r.scale[x >> 3] : 0;
    const h2 sp = (x >> 2) & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(e, 1.0f, true)
                               : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(e, 1.0f, false);
    const _Float16 s1 = (x & 2) == 0 ? sp[0] : sp[1];
    const h2 s = {s1, s1};
    const h2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * s;
    const h2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * s;
    const h2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * s;
    const h2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * s;
    return h8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

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

// ROWS query rows (heads h0 .. , rows past the last head as zeros): read, a row per wavefront and step, 8 values per
// lane; then into LDS as scaled fp16, and per head the factor that turns a dot product of theirs into s2.
template <int ROWS>
struct QueryRows {
    uint4 raw[ROWS / 4];
};
template <int ROWS>
__device__ __forceinline__ void load_query(const AttendArgs& a, int64_t t, int h0, QueryRows<ROWS>& q) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < ROWS / 4; ++i) {
        const int h = h0 + w * (ROWS / 4) + i, hc = h < a.heads ? h : a.heads - 1;
        q.raw[i] = *reinterpret_cast<const uint4*>(a.q + (t * a.heads + hc) * kD + lane * 8);
    }
}
template <int ROWS>
__device__ __forceinline__ void stage_query(const AttendArgs& a, int h0, QueryRows<ROWS>& q, _Float16* lds,
                                            float2* factor) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < ROWS / 4; ++i) {
        const int row = w * (ROWS / 4) + i;
        const uint32_t keep = h0 + row < a.heads ? 0xffffffffu : 0u;
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
        const float f = a.scale * kLog2e * __uint_as_float((uint32_t)(e - 14) << 23);
        factor[row] = float2{fabsf(f) < 0x1p-126f ? 0x1p-126f : f, -kNone};
    }
}

// How a call's queries are cut: those below `whole` into `parts` parts of their entries, the others into one more, so
// that units (a part of a query each) come in whole rounds over the compute units; the longer ones come first. 514
// queries over 16384 rows, in one session: 1005 us in 3 parts each (6.02 rounds), 924 us in 2 or 3 (1280 units).
struct Place {
    uint32_t t, part, parts;
};
struct Cut {
    int nh;  // head sixteens of a block
    uint32_t parts, whole;
    __host__ __device__ uint32_t units(uint32_t nq) const { return nq * parts + (nq - whole); }
    __device__ uint32_t parts_of(uint32_t t) const { return parts + (t >= whole); }
    __device__ uint32_t first_of(uint32_t t) const { return t * parts + (t >= whole ? t - whole : 0); }
    __device__ Place place(uint32_t unit) const {
        const uint32_t longer = whole * parts, by = parts + (unit >= longer), rest = unit >= longer ? unit - longer : unit;
        return Place{(unit >= longer ? whole : 0) + rest / by, rest % by, by};
    }
};

// block -> (query and part, head tile): the head tiles of one query run on one XCD (blocks b and
// b + 8 do), so the second reads the rows from that XCD's L2
__device__ __forceinline__ bool unit_of(uint32_t b, uint32_t units, uint32_t tiles, uint32_t& unit, uint32_t& tile) {
    const uint32_t per = 8 * tiles;
    unit = b / per * 8 + (b & 7);
    tile = b % per / 8;
    return unit < units;
}

// Blocks of 16 heads come in pairs on a compute unit: half its registers each, and one step's rows in LDS, so the two
// products of a block take turns and the blocks cover each other's waits. 8000 queries of one head over 64 rows: 163 ->
// 87 us, 8000 of 16 heads over 512 rows 424 -> 274; one block by itself is as fast either way.
template <int NH>
constexpr bool kPair = NH == 1;

// NH: heads of a block in sixteens
template <int NH>
struct Shared {
    _Float16 kv[(kPair<NH> ? 1 : 2) * kTile * kD];  // a step's or two steps' rows; queries and outputs on their ways
    _Float16 p[2][NH * 16 * kPRow];
    float m[NH * 16][4];
    float l[NH * 16][4];
    int over[2][4];
    float2 fr[NH * 16];                // per head: the factor of stage_query, and minus R
    _Float16 q[NH * 16 * kQRow];       // the queries' last fragment (the registers hold 15 of 16)
};

// What a wavefront holds of the next steps. Loads in flight: the rows of the next step, the page of the one after,
// the position of the one after that.
struct Feed {
    RowPart kv;
    uint32_t scale1[2];      // one step on
    int32_t row;             // of the step whose rows kv holds
    int32_t pos1, page1;     // one step on
    int32_t pos2;            // two steps on
};

template <int NH, bool LIST, bool PAGED>
__global__ __launch_bounds__(256, kPair<NH> ? 2 : 1) void attend_kernel(const AttendArgs a, Cut cut) {
    __shared__ __align__(16) Shared<NH> sh;
    constexpr int kHeads = NH * 16;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    const uint32_t head_tiles = (a.heads + kHeads - 1) / kHeads;
    uint32_t unit, tile;
    if (!unit_of(blockIdx.x, cut.units((uint32_t)a.nq), head_tiles, unit, tile)) return;
    const Place at_cut = cut.place(unit);
    const int64_t t = at_cut.t;
    const int part = (int)at_cut.part, splits = (int)at_cut.parts;
    const int h0 = (int)tile * kHeads;
    const Entries e = entries_of(a, t);
    const int steps_all = (e.count + kTile - 1) / kTile;
    const int per = (steps_all + splits - 1) / splits;
    const int step0 = part * per;
    const int steps = min(per, steps_all - step0);  // may be 0 or less
    const int end = steps > 0 ? min((step0 + steps) * kTile, e.count) : 0;
    const int i0 = step0 * kTile + w * 16 + c;      // this lane's entry of the first step

    QueryRows<kHeads> qr;
    load_query<kHeads>(a, t, h0, qr);
    Feed fd;
    if (steps > 0) {
        const int32_t p = position_of<LIST>(e, i0, end);
        fd.pos1 = position_of<LIST>(e, i0 + kTile, end);
        fd.pos2 = position_of<LIST>(e, i0 + 2 * kTile, end);
        const int32_t page = page_of<PAGED>(a, e, p);
        fd.page1 = page_of<PAGED>(a, e, fd.pos1);
        fd.row = row_of<PAGED>(a, e, p, page);
#pragma unroll
        for (int j = 0; j < 4; ++j) load_chunk(a, fd.row, g, j, fd.kv);
        load_scales(a, fd.row, g, fd.kv.scale);
    }
    stage_query<kHeads>(a, h0, qr, sh.kv, sh.fr);
    __syncthreads();
    h8 q[NH][15];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        const _Float16* at = sh.kv + (n * 16 + c) * kRow + g * 128;
#pragma unroll
        for (int x = 0; x < 15; ++x) q[n][x] = *reinterpret_cast<const h8*>(at + x * 8);
        const h8 ql = *reinterpret_cast<const h8*>(at + 15 * 8);
        if (w == 0) *reinterpret_cast<h8*>(sh.q + (n * 16 + c) * kQRow + g * 8) = ql;
        // in the accumulation half of the register file: matrix operands only
#pragma unroll
        for (int x = 0; x < 15; ++x) asm volatile("" : "+a"(q[n][x]));
    }
    __syncthreads();  // before kv takes rows
    // The second product is 32 heads wide where the block has as many: half the instructions of 16, of twice the time
    // (each holds back the wavefront's next ones as long as two others).
    constexpr bool kWide = NH > 1;
    constexpr int kOh = kWide ? NH / 2 : 1, kOv = kWide ? 4 : 8;  // output tiles: heads, values
    typedef std::conditional_t<kWide, v16f, v4f> Out;
    Out o[kOh][kOv] = {};
    const int oc = kWide ? lane & 31 : c;          // this lane's head of an output tile
    const int og = kWide ? lane >> 5 : g;          // and which fours of its values
    v4f s[NH];
    float l[NH];         // this lane's part of the sum of 2^(s2 - R)
    float sum[NH];       // and of the step whose probabilities were formed last
#pragma unroll
    for (int n = 0; n < NH; ++n) l[n] = 0.0f;

    // A row of a step is 1024 bytes, and its 16-byte pieces are exchanged within each 128: piece p lies at
    // p ^ (2 (row % 4) + row / 4 % 2). Eight rows' same pieces (a write), and four rows' same pairs of pieces (a
    // transposed read), then lie in different banks. Addresses of other pieces, of rows 4 on and of the other buffer
    // differ from these in single bits.
    const int at_in = (w * 16 + c) * kD + g * 128 + ((c & 3) * 2 + ((c >> 2) & 1)) * 8;
    const int first = kWide ? (g & 1) * 2 + ((c >> 1) & 1) : (c >> 1) & 1;  // piece
    const int at_out = (og * 8 + (c >> 2)) * kD + w * 128 + (first ^ ((c >> 2) * 2)) * 8 + (c & 1) * 4;
    // Probabilities 2^(s2 - R) of sixteen heads' products s into p[step & 1]; true if a logit lies too far above R.
    const auto probabilities = [&](int n, float2 fr, int step) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __builtin_fmaf(s[n][i], fr.x, fr.y);
        h4 x;
        sum[n] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float ex = __builtin_amdgcn_exp2f(y[i]);
            sum[n] += ex;
            x[i] = (_Float16)ex;
        }
        *reinterpret_cast<h4*>(sh.p[step & 1] + (n * 16 + c) * kPRow + w * 16 + g * 4) = x;
        return fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) > kMost;
    };
    // R is set kRoom below the largest logit at hand. Where one comes to lie more than kMost above R (seldom after the
    // first step), the four wavefronts agree on a new R and bring outputs and sums to it (powers of two, exact), and
    // the step's probabilities are formed again.
    const auto new_reference = [&](const float2 (&fr)[NH], float (&r)[NH]) {
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            float top = ninf();
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[n][i] * fr[n].x);
            top = group_max(top);
            if (g == 0) sh.m[n * 16 + c][w] = top + fr[n].y > kMost ? ceilf(top) - kRoom : -fr[n].y;
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const v4f mv = *reinterpret_cast<const v4f*>(sh.m[n * 16 + c]);
            r[n] = fmaxf(fmaxf(mv[0], mv[1]), fmaxf(mv[2], mv[3]));
        }
    };
    const auto rebase = [&](int step) {
        float2 fr[NH];
        float r[NH], was[kOh];
#pragma unroll
        for (int n = 0; n < NH; ++n) fr[n] = sh.fr[n * 16 + c];
#pragma unroll
        for (int n = 0; n < kOh; ++n) was[n] = sh.fr[n * 32 + oc].y;
        new_reference(fr, r);
#pragma unroll
        for (int n = 0; n < NH; ++n) l[n] *= __builtin_amdgcn_exp2f(-fr[n].y - r[n]);  // 0 at a head's first entry
#pragma unroll
        for (int n = 0; n < kOh; ++n) {
            const v4f mv = *reinterpret_cast<const v4f*>(sh.m[n * 32 + oc]);
            const float alpha = __builtin_amdgcn_exp2f(-was[n] - fmaxf(fmaxf(mv[0], mv[1]), fmaxf(mv[2], mv[3])));
#pragma unroll
            for (int d = 0; d < kOv; ++d) o[n][d] *= alpha;
        }
        if (w == 0 && g == 0) {  // (every wavefront has read the old ones)
#pragma unroll
            for (int n = 0; n < NH; ++n) sh.fr[n * 16 + c].y = -r[n];
        }
#pragma unroll
        for (int n = 0; n < NH; ++n) probabilities(n, float2{fr[n].x, -r[n]}, step);
        __syncthreads();
    };

    // Turn i of the pipe, after a barrier: the first product of step i + 1 and the second product of step i, then the
    // probabilities of step i + 1 under the rest of the second product. Widening, exponentials, LDS and loads run
    // under the matrix instructions: one takes 16 cycles, four times another instruction.
    const auto turn = [&](auto pv, auto qk, auto first_step, int i) {
        constexpr bool kPv = decltype(pv)::value, kQk = decltype(qk)::value, kFirst = decltype(first_step)::value;
        const int buf = i & 1;
        const int in = at_in ^ (kPair<NH> || buf ? 0 : kTile * kD);
        const int out = at_out ^ (!kPair<NH> && buf ? kTile * kD : 0);
        const _Float16* prob = sh.p[buf] + oc * kPRow + og * 8;
        // a transposed read of unit y's eight entries (below) of this lane's value
        const auto rows8 = [&](int y) {
            int lo, hi, at;
            if constexpr (kWide) {
                lo = out ^ ((y & 1) * 32), hi = out ^ ((y & 1) * 32 + 4 * kD + 8);
                at = (y >> 2) * 16 * kD + ((y >> 1) & 1) * 64;
            } else {
                lo = out ^ ((y & 3) * 16), hi = out ^ ((y & 3) * 16 + 4 * kD + 8);
                at = (y >> 3) * 32 * kD + ((y >> 2) & 1) * 64;
            }
            const hv4 l4 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(sh.kv + lo + at));
            const hv4 h4 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(sh.kv + hi + at));
            h8 v;
            __builtin_memcpy(&v, &l4, 8);
            __builtin_memcpy((char*)&v + 8, &h4, 8);
            return v;
        };
        h8 k, v[4], p[kOh], ql[NH];
        int4 ov{0, 0, 0, 0};
        if constexpr (kPv) {
            ov = *reinterpret_cast<const int4*>(sh.over[buf]);
#pragma unroll
            for (int n = 0; n < kOh; ++n) p[n] = *reinterpret_cast<const h8*>(prob + n * 32 * kPRow);
            v[0] = rows8(0);
        }
        const bool there = fd.row >= 0;
        int32_t row1 = -1;
        if constexpr (kQk) {
            row1 = row_of<PAGED>(a, e, fd.pos1, fd.page1);
            fd.pos1 = fd.pos2;
            fd.page1 = page_of<PAGED>(a, e, fd.pos2);
            fd.pos2 = position_of<LIST>(e, i0 + (i + 4) * kTile, end);
            k = values8(fd.kv, 0, there);
        }
        if constexpr (kPv) {
            if (__builtin_amdgcn_readfirstlane(ov.x | ov.y | ov.z | ov.w)) {
                rebase(i);
#pragma unroll
                for (int n = 0; n < kOh; ++n) p[n] = *reinterpret_cast<const h8*>(prob + n * 32 * kPRow);
            }
#pragma unroll
            for (int n = 0; n < NH; ++n) l[n] += sum[n];
        }
        // y-th unit of the second product: entries 32 (y / 8) .. + 31 of values 16 (y % 8) .. + 15, or, wide, entries
        // 16 (y / 4) .. + 15 of values 32 (y % 4) .. + 31
        const auto unit = [&](int y) {
            // operands are read one unit ahead, three where units follow each other closely
            const auto ahead = [](int u) { return u < 0 ? 0 : u + 1 + (u >= 4) + (u >= 6); };
#pragma unroll
            for (int r = 1; r < 16; ++r)
                if (r > ahead(y - 1) && r <= ahead(y)) v[r & 3] = rows8(r);
#pragma unroll
            for (int n = 0; n < kOh; ++n) {
                if constexpr (kWide) {
                    o[n][y & 3] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[y & 3], p[n], o[n][y & 3], 0, 0, 0);
                    if ((y & 3) == 3 && y < 15)
                        p[n] = *reinterpret_cast<const h8*>(prob + n * 32 * kPRow + ((y >> 2) + 1) * 16);
                } else {
                    o[n][y & 7] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[y & 3], p[n], o[n][y & 7], 0, 0, 0);
                    if (y == 7) p[n] = *reinterpret_cast<const h8*>(prob + 32);
                }
            }
        };
        if constexpr (kQk) {
#pragma unroll
            for (int n = 0; n < NH; ++n) s[n] = v4f{};
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            if constexpr (kPv) {
                if (!kQk || (x & 1)) unit(kQk ? x >> 1 : x);
            }
            if constexpr (kQk) {
                const h8 kx = k;
                *reinterpret_cast<h8*>(sh.kv + (in ^ ((x & 7) * 8)) + (x >> 3) * 64) = kx;
                if (x < 15) k = values8(fd.kv, x + 1, there);
                if (x == 3) load_scales(a, row1, g, fd.scale1);
                if ((x & 3) == 3) load_chunk(a, row1, g, x >> 2, fd.kv);
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    if (x == 14) ql[n] = *reinterpret_cast<const h8*>(sh.q + (n * 16 + c) * kQRow + g * 8);
                    s[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kx, x < 15 ? q[n][x < 15 ? x : 0] : ql[n], s[n], 0, 0, 0);
                }
            }
#pragma unroll
            for (int y = 0; y < NH * kQk + kOh * (kPv && (x & 1)); ++y) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kQk) {
            const uint64_t all = __ballot(there);
            float2 fr[NH];
#pragma unroll
            for (int n = 0; n < NH; ++n) fr[n] = sh.fr[n * 16 + c];
            if (all != ~0ull) {
                const uint32_t seen = (uint32_t)all >> (g * 4);
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    const float hole = fr[n].x < 0.0f ? __builtin_inff() : ninf();
#pragma unroll
                    for (int y = 0; y < 4; ++y) s[n][y] = (seen >> y) & 1 ? s[n][y] : hole;
                }
            }
            fd.row = row1;
            fd.kv.scale[0] = fd.scale1[0];
            fd.kv.scale[1] = fd.scale1[1];
            bool over = false;
            if constexpr (kFirst) {
                // the first step sets R
                float r[NH];
                new_reference(fr, r);
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    fr[n].y = -r[n];
                    if (w == 0 && g == 0) sh.fr[n * 16 + c].y = -r[n];
                }
            }
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                if constexpr (kPv) {
#pragma unroll
                    for (int y = 8 + n * 8 / NH; y < 8 + (n + 1) * 8 / NH; ++y) unit(y);
                }
                over |= probabilities(n, fr[n], i + 1);
                if constexpr (kPv) {
#pragma unroll
                    for (int y = 0; y < 8 * kOh / NH; ++y) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x2, 3 * NH / kOh, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            const int mine = __any(over);
            sh.over[buf ^ 1][w] = mine;
            __syncthreads();
        }
    };

    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (steps > 0) {
        turn(no, yes, yes, -1);
        if constexpr (kPair<NH>) {
            for (int i = 0; i + 1 < steps; ++i) {
                turn(yes, no, no, i);
                __syncthreads();  // before the next step's rows take the place
                turn(no, yes, no, i);
            }
        } else {
            for (int i = 0; i + 1 < steps; ++i) turn(yes, yes, no, i);
        }
        turn(yes, no, no, steps - 1);
    }

    // the sum over the four lane groups and the four wavefronts
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        const float x = group_sum(l[n]);
        if (g == 0) sh.l[n * 16 + c][w] = x;
    }
    __syncthreads();
    _Float16* rows = sh.kv;  // (bf16) the block's output rows, to be written whole
#pragma unroll
    for (int n = 0; n < kOh; ++n) {
        const int hl = n * 32 + oc;
        const v4f lv = *reinterpret_cast<const v4f*>(sh.l[hl]);
        const float L = (lv[0] + lv[1]) + (lv[2] + lv[3]);
        const int h = h0 + hl;
        // four values of tile d lie at 16 d + 4 g, or, wide, at 32 (d / 4) + 8 (d % 4) + 4 og
        const auto four = [&](int d) {
            if constexpr (kWide) {
                const Out& x = o[n][d >> 2];
                const int i = (d & 3) * 4;
                return v4f{x[i], x[i + 1], x[i + 2], x[i + 3]};
            } else {
                return o[n][d];
            }
        };
        const auto at_four = [&](int d) { return kWide ? (d >> 2) * 32 + (d & 3) * 8 + og * 4 : d * 16 + og * 4; };
        constexpr int kFours = kWide ? 16 : 8;
        if (splits > 1) {
            if (h >= a.heads) continue;
            const int64_t r = (int64_t)unit * a.heads + h;
            float* po = a.part_o + r * kD + w * 128;
#pragma unroll
            for (int d = 0; d < kFours; ++d) *reinterpret_cast<v4f*>(po + at_four(d)) = four(d);
            if (w == 0 && og == 0) {
                a.part_ml[2 * r] = -sh.fr[hl].y;
                a.part_ml[2 * r + 1] = L;
            }
        } else {
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            _Float16* po = rows + hl * kRow + w * 128;
#pragma unroll
            for (int d = 0; d < kFours; ++d) {
                const v4f y = four(d) * inv;
                *reinterpret_cast<uint2*>(po + at_four(d)) = uint2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
            }
            if (a.lse && h < a.heads && w == 0 && og == 0)
                a.lse[t * a.heads + h] = L == 0.0f ? ninf() : (__builtin_amdgcn_logf(L) - sh.fr[hl].y) * kLn2;
        }
    }
    if (splits > 1) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NH * 4; ++i) {
        const int hl = w * NH * 4 + i;
        if (h0 + hl < a.heads)
            *reinterpret_cast<uint4*>(a.out + (t * a.heads + h0 + hl) * kD + lane * 8) =
                *reinterpret_cast<const uint4*>(rows + hl * kRow + lane * 8);
    }
}

// Join of the parts of one (query, head): o = sum 2^(R_i - R) o_i over sum 2^(R_i - R) l_i. 128 threads take 4 values
// each; with many parts, G groups of them take every G-th.
template <int G>
__global__ __launch_bounds__(128 * G) void attend_join_kernel(const AttendArgs a, Cut cut, int t0) {
    __shared__ float s_f[kMostParts];
    __shared__ float2 s_wave[2 * G];
    __shared__ __align__(16) v4f s_o[G > 1 ? (G - 1) * 128 : 1];
    const uint32_t t = t0 + blockIdx.x / a.heads;
    const int h = (int)(blockIdx.x % a.heads), splits = (int)cut.parts_of(t);
    const int64_t first = (int64_t)cut.first_of(t) * a.heads + h;
    const int64_t pair = (int64_t)t * a.heads + h;
    const int64_t step = a.heads;
    // references and sums: a part per thread
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    constexpr int kPer = (kMostParts + 128 * G - 1) / (128 * G);
    float2 mine[kPer];
    float R = kNone;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = k * 128 * G + (int)threadIdx.x;
        mine[k] = i < splits ? ml[first + i * step] : float2{kNone, 0.0f};
        R = fmaxf(R, mine[k].x);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) R = fmaxf(R, __shfl_xor(R, d));
    if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6].x = R;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2 * G; ++k) R = fmaxf(R, s_wave[k].x);
    float L = 0.0f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = k * 128 * G + (int)threadIdx.x;
        const float f = __builtin_amdgcn_exp2f(mine[k].x - R);
        if (i < splits) s_f[i] = f;
        L += f * mine[k].y;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) L += __shfl_xor(L, d);
    if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6].y = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int k = 0; k < 2 * G; ++k) L += s_wave[k].y;

    const int grp = threadIdx.x >> 7, at = threadIdx.x & 127;
    const float* po = a.part_o + first * kD + at * 4;
    v4f o = {};
    int i = grp;
    for (; i + 7 * G < splits; i += 8 * G) {  // eight loads in flight
        v4f v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const v4f*>(po + (int64_t)(i + k * G) * step * kD);
#pragma unroll
        for (int k = 0; k < 8; ++k) o += s_f[i + k * G] * v[k];
    }
#pragma unroll 4
    for (; i < splits; i += G) o += s_f[i] * *reinterpret_cast<const v4f*>(po + (int64_t)i * step * kD);
    if constexpr (G > 1) {
        if (grp) s_o[(grp - 1) * 128 + at] = o;
        __syncthreads();
        if (grp) return;
#pragma unroll
        for (int k = 0; k < G - 1; ++k) o += s_o[k * 128 + at];
    }
    o *= L == 0.0f ? 0.0f : 1.0f / L;
    *reinterpret_cast<uint2*>(a.out + pair * kD + at * 4) = uint2{bf16_pair(o[0], o[1]), bf16_pair(o[2], o[3])};
    if (a.lse && at == 0) a.lse[pair] = L == 0.0f ? ninf() : (R + __builtin_amdgcn_logf(L)) * kLn2;
}

// The attention's probability of every entry, mean over the heads, from the saved lse:
//   w_i = 1/H sum_h exp(s_{h,i} - lse_h).
// The first product alone, with heads as rows: a lane's column is one entry, whose terms it adds up over the heads.
// Each wavefront takes 16 entries per step by itself (no barrier); the exponentials of a step run under the matrix
// instructions of the next. Heads beyond the block's 16 NH are further rounds over the same entries, added by the lane
// that wrote them. 1021 queries of 64 heads over about 3600 rows: 213 us (1.0 PFLOP/s), 0.8 us a step, of which the
// matrix instructions are 0.43; without reading the rows 0.68.
template <int NH, bool LIST, bool PAGED>
__global__ __launch_bounds__(256, 1) void attend_weights_kernel(const AttendArgs a, const float* __restrict__ lse,
                                                                float* __restrict__ weights, int64_t w_stride,
                                                                int splits) {
    constexpr int kHeads = 16 * NH;
    __shared__ __align__(16) _Float16 s_q[kHeads * kRow];
    __shared__ float2 s_factor[kHeads];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    const int64_t t = blockIdx.x / splits;
    const int part = (int)(blockIdx.x % splits);
    const Entries e = entries_of(a, t);
    // a list's slots are all written; of a range, the visible positions
    const int slots = LIST ? a.k : e.visible;
    const int steps_all = (slots + kTile - 1) / kTile;
    const int per = (steps_all + splits - 1) / splits;
    const int step0 = part * per;
    const int steps = min(per, steps_all - step0);
    if (steps <= 0) return;
    float* out = weights + t * w_stride;
    const int end = min((step0 + steps) * kTile, slots);
    if (e.count == 0) {  // no row is read (the cache may hold none)
        for (int i = step0 * kTile + (int)threadIdx.x; i < end; i += 256) out[i] = 0.0f;
        return;
    }
    const int i0 = step0 * kTile + w * 16 + c;  // this lane's entry of the first step
    const float mean = 1.0f / (float)a.heads;

    for (int h0 = 0; h0 < a.heads; h0 += kHeads) {
        QueryRows<kHeads> qr;
        load_query<kHeads>(a, t, h0, qr);
        Feed fd;
        {
            const int32_t p = position_of<LIST>(e, i0, end);
            fd.pos1 = position_of<LIST>(e, i0 + kTile, end);
            fd.pos2 = position_of<LIST>(e, i0 + 2 * kTile, end);
            const int32_t page = page_of<PAGED>(a, e, p);
            fd.page1 = page_of<PAGED>(a, e, fd.pos1);
            fd.row = row_of<PAGED>(a, e, p, page);
#pragma unroll
            for (int j = 0; j < 4; ++j) load_chunk(a, fd.row, g, j, fd.kv);
            load_scales(a, fd.row, g, fd.kv.scale);
        }
        if (h0) __syncthreads();
        stage_query<kHeads>(a, h0, qr, s_q, s_factor);
        __syncthreads();
        h8 q[NH][16];
        float f[NH][4], off[NH][4];
#pragma unroll
        for (int n = 0; n < NH; ++n) {
#pragma unroll
            for (int x = 0; x < 16; ++x)
                q[n][x] = *reinterpret_cast<const h8*>(s_q + (n * 16 + c) * kRow + g * 128 + x * 8);
#pragma unroll
            for (int x = 0; x < 16; ++x) asm volatile("" : "+a"(q[n][x]));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int hl = n * 16 + g * 4 + i, h = min(h0 + hl, a.heads - 1);
                f[n][i] = s_factor[hl].x;
                // a head that is not there, or that saw nothing, adds nothing
                const float y = h0 + hl < a.heads ? lse[t * a.heads + h] : ninf();
                off[n][i] = y == ninf() ? ninf() : -y * kLog2e;
            }
        }
        v4f s[NH], last[NH];  // products of the step at hand and of the one before, whose row was last_row
        int32_t last_row;
        const auto store = [&](int i, float sum) {
            sum = group_sum(sum);
            if (g == 0 && i < end) {
                const float x = last_row >= 0 ? sum * mean : 0.0f;
                out[i] = h0 ? out[i] + x : x;
            }
        };
        const auto turn = [&](auto first, int step) {
            constexpr bool kFirst = decltype(first)::value;
            const bool there = fd.row >= 0;
            const int32_t row1 = row_of<PAGED>(a, e, fd.pos1, fd.page1);
            fd.pos1 = fd.pos2;
            fd.page1 = page_of<PAGED>(a, e, fd.pos2);
            fd.pos2 = position_of<LIST>(e, i0 + (step + 3) * kTile, end);
            float sum = 0.0f;
            h8 k = values8(fd.kv, 0, there);
#pragma unroll
            for (int n = 0; n < NH; ++n) s[n] = v4f{};
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const h8 kx = k;
                if (x < 15) k = values8(fd.kv, x + 1, there);
                if (x == 3) load_scales(a, row1, g, fd.scale1);
                if ((x & 3) == 3) load_chunk(a, row1, g, x >> 2, fd.kv);
                if (!kFirst && x < 4 * NH)
                    sum += __builtin_amdgcn_exp2f(__builtin_fmaf(last[x >> 2][x & 3], f[x >> 2][x & 3], off[x >> 2][x & 3]));
#pragma unroll
                for (int n = 0; n < NH; ++n) {
                    s[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[n][x], kx, s[n], 0, 0, 0);
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (!kFirst) store(i0 + (step - 1) * kTile, sum);
#pragma unroll
            for (int n = 0; n < NH; ++n) last[n] = s[n];
            last_row = fd.row;
            fd.row = row1;
            fd.kv.scale[0] = fd.scale1[0];
            fd.kv.scale[1] = fd.scale1[1];
        };
        turn(std::true_type{}, 0);
        for (int step = 1; step < steps; ++step) turn(std::false_type{}, step);
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < NH; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += __builtin_amdgcn_exp2f(__builtin_fmaf(last[n][i], f[n][i], off[n][i]));
        store(i0 + (steps - 1) * kTile, sum);
    }
}

}  // namespace

namespace {

// Time until the last of n1 blocks of t1 and then n2 of t2 <= t1 ends, each taken by the first of `places` that is free.
float time_of(int64_t places, int64_t n1, float t1, int64_t n2, float t2) {
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
// How a call is cut: head sixteens of a block and parts of a query's entries, by the time that the 256 compute
// units (a block each, or two of 16 heads) would take. Large head tiles widen a row for more heads, small ones and
// parts give blocks and even rounds. Measured per step of 64 entries and per block apart from its steps, in
// microseconds: 1.65 and 10.5 at 64 heads, 1.2 and 6 at 32, 1.6 and 5 for the pairs at 16 (2048 queries over 64 .. 4096
// rows); with at most one block for every compute unit 1.65 and 13, 1.16 and 9, 1.2 and 7 (256 queries); a join 4, and its
// parts at 4 TB/s. Where a query is cut at all, every unit's output and sums lie in the workspace, which has room for
// `room` units.
Cut best_cut(int32_t nq, int32_t heads, int64_t entries, uint64_t room) {
    static constexpr struct {
        int nh, places;
        float step, block, step_alone, block_alone;
    } kTiles[] = {{4, 256, 1.65f, 10.5f, 1.65f, 13.0f}, {2, 256, 1.2f, 6.0f, 1.16f, 9.0f}, {1, 512, 1.6f, 5.0f, 1.2f, 7.0f}};
    const int64_t steps = entries > kTile ? (entries + kTile - 1) / kTile : 1;
    Cut best{1, 1, (uint32_t)nq};
    float least = 0.0f;
    for (const auto& t : kTiles) {
        if (t.nh > 1 && heads <= 8 * t.nh) continue;  // half of the tile would be empty
        const int64_t tiles = (heads + 16 * t.nh - 1) / (16 * t.nh);
        const auto consider = [&](int64_t parts, int64_t whole) {
            const int64_t n1 = whole * parts, n2 = (nq - whole) * (parts + 1), joined = parts > 1 ? n1 + n2 : n2;
            if (n1 + n2 > nq && (uint64_t)(n1 + n2) > room) return;
            const bool alone = (n1 + n2) * tiles <= 256;
            const float step = alone ? t.step_alone : t.step, block = alone ? t.block_alone : t.block;
            const auto one = [&](int64_t n) { return (float)((steps + n - 1) / n) * step + block; };
            const float time = time_of(t.places, n1 * tiles, one(parts), n2 * tiles, one(parts + 1)) +
                               (joined ? 4.0f + 1e-3f * (float)heads * (float)joined : 0.0f);
            if (least == 0.0f || time < least) {
                least = time;
                best = Cut{t.nh, (uint32_t)parts, (uint32_t)whole};
            }
        };
        for (int64_t s = 1; s <= steps && s <= kMostParts; ++s) {
            if (s > 1 && nq * tiles * s > 8 * t.places + nq * tiles) break;  // rounds are even enough
            consider(s, nq);
        }
        for (int64_t rounds = 1; rounds <= 8; ++rounds) {  // units for whole rounds
            const int64_t units = rounds * t.places / tiles, parts = units / nq;
            if (parts >= 1 && parts < steps && parts < kMostParts && units % nq) consider(parts, nq * (parts + 1) - units);
        }
    }
    return best;
}

// The same for the sizes asked for last: the next call mostly has the same (a search takes up to some ten
// microseconds). The best cut in some room is also the best in less that it fits into.
Cut cut_of(int32_t nq, int32_t heads, int64_t entries, uint64_t room) {
    thread_local int64_t of[3] = {0, 0, 0};
    thread_local uint64_t in = 0;
    thread_local Cut cut{};
    const auto fits = [&] { return cut.units((uint32_t)nq) == (uint32_t)nq || cut.units((uint32_t)nq) <= room; };
    if (of[0] != nq || of[1] != heads || of[2] != entries || in < room || !fits()) {
        cut = best_cut(nq, heads, entries, room);
        of[0] = nq;
        of[1] = heads;
        of[2] = entries;
        in = room;
    }
    return cut;
}
constexpr size_t unit_bytes(int32_t heads) { return (size_t)heads * (kD + 2) * sizeof(float); }

// Parts of a query's entries in the weights' kernel, in the same way. Measured per step and per block apart from its
// steps, in microseconds: 0.8 and 7.5 at 64 heads, 0.55 and 3.2 at 32, 0.5 and 2.6 at 16 (1024 queries over 64 .. 4096
// rows).
int best_parts(int32_t nq, int32_t heads, int64_t steps) {
    const float step = heads > 32 ? 0.8f : heads > 16 ? 0.55f : 0.5f, block = heads > 32 ? 7.5f : heads > 16 ? 3.2f : 2.6f;
    int best = 1;
    float least = 0.0f;
    for (int64_t s = 1; s <= steps; ++s) {
        if (s > 1 && nq * s > 8 * 256 + nq) break;  // rounds are even enough
        const float time = (float)((nq * s + 255) / 256) * ((float)((steps + s - 1) / s) * step + block);
        if (least == 0.0f || time < least) {
            least = time;
            best = (int)s;
        }
    }
    return best;
}
int weights_parts(int32_t nq, int32_t heads, int64_t steps) {
    thread_local int64_t of[3] = {0, 0, 0};
    thread_local int parts = 1;
    if (of[0] != nq || of[1] != heads || of[2] != steps) {
        parts = best_parts(nq, heads, steps);
        of[0] = nq;
        of[1] = heads;
        of[2] = steps;
    }
    return parts;
}

// p / page_size for 0 <= p < 2^30 as a product: with d <= 2^b < 2 d, mul = floor(2^(31+b) / d) + 1 is below 2^32 and exceeds
// 2^(31+b) / d by at most 1, so 2 p mul / 2^(32+b) exceeds p / d by at most p / 2^(31+b) < 1 / (2 d): the floors agree.
void set_page_division(AttendArgs& a) {
    if (!a.pages) return;
    int b = 0;
    while (((int64_t)1 << b) < a.page_size) ++b;
    a.page_mul = (uint32_t)(((uint64_t)1 << (31 + b)) / (uint64_t)a.page_size + 1);
    a.page_shift = b;
}

// the kernel of the call's entries: listed or a range, paged or contiguous
template <typename F>
void by_entries(const AttendArgs& a, F&& launch) {
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (a.idx)
        a.pages ? launch(yes, yes) : launch(yes, no);
    else
        a.pages ? launch(no, yes) : launch(no, no);
}

template <int NH>
void launch_attend_as(const AttendArgs& a, const Cut& cut, hipStream_t stream) {
    const uint32_t units = cut.units((uint32_t)a.nq), head_tiles = (a.heads + 16 * NH - 1) / (16 * NH);
    by_entries(a, [&](auto list, auto paged) {
        hipLaunchKernelGGL((attend_kernel<NH, decltype(list)::value, decltype(paged)::value>),
                           dim3((units + 7) / 8 * 8 * head_tiles), dim3(256), 0, stream, a, cut);
    });
}

}  // namespace

size_t attend_workspace_bytes(int32_t nq, int32_t heads, int64_t entries) {
    if (nq <= 0 || entries <= 0) return 16;
    const size_t units = cut_of(nq, heads, entries, UINT64_MAX).units((uint32_t)nq);
    return units == (size_t)nq ? 16 : units * unit_bytes(heads);
}

hipError_t launch_attend(AttendArgs a, void* ws, size_t ws_bytes, hipStream_t stream) {
    const int64_t entries = a.idx ? a.k : (a.window > 0 && a.window < a.max_n ? a.window : a.max_n);
    const Cut cut = cut_of(a.nq, a.heads, entries, ws_bytes / unit_bytes(a.heads));
    set_page_division(a);
    const uint32_t units = cut.units((uint32_t)a.nq);
    if (units > (uint32_t)a.nq) {
        a.part_o = (float*)ws;
        a.part_ml = a.part_o + (size_t)units * a.heads * kD;
    }
    if (cut.nh == 4)
        launch_attend_as<4>(a, cut, stream);
    else if (cut.nh == 2)
        launch_attend_as<2>(a, cut, stream);
    else
        launch_attend_as<1>(a, cut, stream);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || units == (uint32_t)a.nq) return err;
    // queries in one part are done
    const int t0 = cut.parts > 1 ? 0 : (int)cut.whole;
    // (four groups: 17 -> 8 us for 512 pairs of 32 parts; one: 35 us for 33000 pairs of 3, bound by HBM)
    const dim3 pairs((uint32_t)(a.nq - t0) * a.heads);
    if (cut.parts >= 8)
        hipLaunchKernelGGL(attend_join_kernel<4>, pairs, dim3(512), 0, stream, a, cut, t0);
    else
        hipLaunchKernelGGL(attend_join_kernel<1>, pairs, dim3(128), 0, stream, a, cut, t0);
    return hipGetLastError();
}

hipError_t launch_attend_weights(AttendArgs a, const float* lse, float* weights, int64_t w_stride,
                                 hipStream_t stream) {
    const int64_t entries = a.idx ? a.k : a.max_n;
    if (entries == 0) return hipSuccess;
    set_page_division(a);
    const int splits = weights_parts(a.nq, a.heads, (entries + kTile - 1) / kTile);
    by_entries(a, [&](auto list, auto paged) {
        constexpr bool L = decltype(list)::value, P = decltype(paged)::value;
        const dim3 grid((uint32_t)a.nq * splits);
        if (a.heads > 32)
            hipLaunchKernelGGL((attend_weights_kernel<4, L, P>), grid, dim3(256), 0, stream, a, lse, weights, w_stride,
                               splits);
        else if (a.heads > 16)
            hipLaunchKernelGGL((attend_weights_kernel<2, L, P>), grid, dim3(256), 0, stream, a, lse, weights, w_stride,
                               splits);
        else
            hipLaunchKernelGGL((attend_weights_kernel<1, L, P>), grid, dim3(256), 0, stream, a, lse, weights, w_stride,
                               splits);
    });
    return hipGetLastError();
}

}  // namespace fp4idx
