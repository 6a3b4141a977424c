// Attention over the FP8 cache of local positions (rows of 512 values, E4M3 codes with a power of two per 32): each
// query's last `window` entries or all it sees, joined with another part of the same softmax (the selection's), and the
// result turned back to the query's frame.
//
//   s_p = scale * q . kv_p,  l = log sum e^{s_p},  o = sum e^{s_p - l} kv_p
//   with another part (o', l'):  L = log(e^l + e^{l'}),  out = e^{l - L} o + e^{l' - L} o'
//
// Three kernels. Long ranges, and whatever the others do not take: a block of four wavefronts takes 16, 32 or 64 rows, a row
// being one head of one query; rows of consecutive queries of a sequence share the cache rows they see, so that few heads
// fill a block too, and which entries a row sees is masked where the block's queries differ. 64 entries a step: wavefront w
// reads those 16w .. 16w + 15 straight into registers, widens them to fp16, multiplies them with the block's rows and leaves
// them in LDS; after a barrier it multiplies values 128w .. 128w + 127 of all 64 entries with the probabilities. Two blocks of
// 16 rows on a compute unit cover each other's waits; larger ones have it to themselves. Windows of queries that follow each
// other, and single queries of at most 128 entries, have kernels of their own below. A run's entries are split where its rows
// do not fill the card, and the parts joined by another launch.
//
// 64 heads: 514 queries over 16384 entries in pages 1.03 to 1.07 ms (0.9 PFLOP/s of the 1.36 that a large product reaches:
// one wavefront per SIMD, whose issue and waits leave the matrix units busy half of the time); 24 queries over about 57400
// 218 us (0.83 PFLOP/s: 84 steps of about 2 us a block, and 33 MB of parts, written and read); 4096 over windows of 128,
// joined, 183 us (805 MB at 4.4 TB/s, nine tenths of a copy's rate).
//
// Arithmetic. A stored value is an fp16 number; queries are scaled by a power of two per row and exact down to 2^-28 of
// the row's largest; products and sums are fp32. Probabilities enter the second product in 11 bits, against a reference
// 7 below the largest logit that moves when one comes to lie 15 above it (both base 2). The join and the rotation are
// fp32, rounded once.
#include <algorithm>
#include <string.h>
#include <type_traits>

#include "attend_common.h"
#include "places.h"

namespace fp4idx {
namespace {

constexpr int kMostParts = 64;  // of a run's entries (a lane each when they are joined)
constexpr int kShares = 64;     // runs (a lane each) whose blocks are shared out on the device,
constexpr int kShareGroup = 8;  // and queries of one

// what a block's rows see
struct Span {
    int32_t first;  // the first entry that a row sees
    int32_t count;  // up to the last one
    bool mixed;     // not every row sees the same
    int32_t each;   // above 0: the queries' windows lie far apart and are gone through one by one, `each` places for each
};

// entries lo .. hi - 1 that a query sees
__device__ __forceinline__ int2 seen_by(const LocalArgs& a, int64_t t) {
    int64_t n = a.n_vis[t];
    n = n < 0 ? 0 : (n > a.places.max_n ? a.places.max_n : n);
    const int64_t lo = a.window > 0 && n > a.window ? n - a.window : 0;
    return int2{(int32_t)lo, (int32_t)n};
}

// One lane's share of a cache row: lane group g (of 4) holds values 128g .. 128g + 127 and their four scales. (Reading 64
// bytes of a row by four neighbouring lanes, and exchanging the pieces between them, would free the address unit, but the 64
// more instructions of a step cost more: 514 queries over 16384 entries 1248 -> 1356 us.)
struct LocalPart {
    uint4 code[8];
    uint32_t scale;
};
__device__ __forceinline__ void load_piece(const LocalArgs& a, int32_t row, int g, int j, LocalPart& r) {
    r.code[j] = *reinterpret_cast<const uint4*>(a.codes + (int64_t)max(row, 0) * kD + g * 128 + 16 * j);
}
__device__ __forceinline__ uint32_t load_scale(const LocalArgs& a, int32_t row, int g) {
    return *reinterpret_cast<const uint32_t*>(a.scales + (int64_t)max(row, 0) * 16 + g * 4);
}
// values 8x .. 8x + 7 of the part as fp16 (exact)
__device__ __forceinline__ h8 local_values8(const LocalPart& r, int x) {
    const uint4 c = r.code[x >> 1];
    const uint32_t w0 = x & 1 ? c.z : c.x, w1 = x & 1 ? c.w : c.y;
    const float s = __uint_as_float((r.scale >> (8 * (x >> 2)) & 0xffu) << 23);
    const h2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, s, false);
    const h2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, s, true);
    const h2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, s, false);
    const h2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, s, true);
    return h8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// How a call is cut: blocks (tiles) of 16 nh rows of a run's heads x queries, the first `whole` tiles of a run over `parts`
// parts of its entries, the others over one more, so that blocks come in whole rounds over the compute units; or, with
// `queries` above 0, blocks of the window kernel over so many queries; or, with `one` above 0, blocks of one query and so many
// times 16 heads. With `shared` the blocks are shared out on the device, by what the runs see (see share_of).
struct LocalCut {
    int nh;
    uint32_t parts, tiles, whole;
    int queries, one;
    bool shared;
    __host__ __device__ uint32_t of_run() const { return tiles * (parts + 1) - whole; }
    __host__ __device__ uint32_t slots() const { return parts + (whole < tiles); }  // of a row's parts
    __device__ uint32_t parts_of(uint32_t tile) const { return parts + (tile >= whole); }
};

// Weights of a row's sums o and of its other part, and the joined logarithm: L = sum 2^(s2 - R).
struct Weights {
    float mine, other, lse;
};
__device__ __forceinline__ Weights join_weights(const LocalArgs& a, float l2, float R, float L) {
    Weights w{L == 0.0f ? 0.0f : 1.0f / L, 0.0f, L == 0.0f ? ninf() : (__builtin_amdgcn_logf(L) + R) * kLn2};
    if (a.other) {
        const float top = fmaxf(w.lse, l2);
        if (top > ninf()) {
            const float e1 = __builtin_amdgcn_exp2f((w.lse - top) * kLog2e), e2 = __builtin_amdgcn_exp2f((l2 - top) * kLog2e);
            const float inv = 1.0f / (e1 + e2);
            w.mine *= e1 * inv;
            w.other = e2 * inv;
            w.lse = top + __builtin_amdgcn_logf(e1 + e2) * kLn2;
        }
    }
    return w;
}
// values 8 lane .. + 7 of the other part added (what lies in one of no weight has no effect)
__device__ __forceinline__ void add_other(const uint4& u, float weight, float (&v)[8]) {
    if (weight == 0.0f) return;
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = fmaf(weight, __uint_as_float(x[i] << 16), v[2 * i]);
        v[2 * i + 1] = fmaf(weight, __uint_as_float(x[i] & 0xffff0000u), v[2 * i + 1]);
    }
}
// (cos, sin) of a pair, times the factor
__device__ __forceinline__ float2 angle_of(const LocalArgs& a, int64_t t, int pair) {
    float s, c;
    sincos_turns((float)turns_of(a.turn.pos[t], a.turn.freq[pair]), s, c);
    const float m = (float)a.turn.mscale;
    return float2{c * m, (a.turn.inverse ? -s : s) * m};
}
// A row's values 8 lane .. + 7, turned by angles cs; row: LDS of its 512 values for pairs that lanes do not hold together
__device__ __forceinline__ void turn_row(const LocalArgs& a, const float2* cs, float* row, float (&v)[8]) {
    const int lane = threadIdx.x & 63, rot = a.turn.rot, pairs = rot / 2, j0 = 8 * lane - a.turn.offset;
    if (!a.turn.half && !((a.turn.offset | rot) & 7)) {  // whole lanes
        if (j0 < 0 || j0 >= rot) return;
        const v4f z[2] = {reinterpret_cast<const v4f*>(cs)[j0 >> 2], reinterpret_cast<const v4f*>(cs)[(j0 >> 2) + 1]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = z[i >> 1][(i & 1) * 2], s = z[i >> 1][(i & 1) * 2 + 1];
            const float x0 = v[2 * i], x1 = v[2 * i + 1];
            v[2 * i] = x0 * c - x1 * s;
            v[2 * i + 1] = x1 * c + x0 * s;
        }
        return;
    }
    *reinterpret_cast<v4f*>(row + 8 * lane) = v4f{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<v4f*>(row + 8 * lane + 4) = v4f{v[4], v[5], v[6], v[7]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = j0 + i;
        if (j < 0 || j >= rot) continue;
        const bool second = a.turn.half ? j >= pairs : j & 1;
        const float2 z = cs[a.turn.half ? (second ? j - pairs : j) : j >> 1];
        const float x = row[a.turn.offset + (a.turn.half ? (second ? j - pairs : j + pairs) : j ^ 1)];
        v[i] = second ? v[i] * z.x + x * z.y : v[i] * z.x - x * z.y;
    }
}
__device__ __forceinline__ void store_row(const LocalArgs& a, int64_t pair, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(a.out + pair * kD + 8 * (threadIdx.x & 63)) =
        uint4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
}

// The sum over a wavefront
__device__ __forceinline__ int wave_sum(int v) {
    v += (int)dpp<0xB1>((uint32_t)v);   // quad_perm [1,0,3,2]
    v += (int)dpp<0x4E>((uint32_t)v);   // quad_perm [2,3,0,1]
    v += (int)dpp<0x141>((uint32_t)v);  // row_half_mirror
    v += (int)dpp<0x140>((uint32_t)v);  // row_mirror
    const auto s = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
    v = (int)(s[0] + s[1]);
    const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    return __builtin_amdgcn_readfirstlane((int)(r[0] + r[1]));
}
// Blocks for runs of different lengths (at most 64, a lane each): parts of as few steps as the blocks suffice for, so that
// the blocks end together; every run has one at least. A lane gets its run's first block and number of parts.
__device__ __forceinline__ int2 share_of(const LocalArgs& a, int tiles, int blocks) {
    const int lane = threadIdx.x & 63, runs = a.nq / a.group;
    int n = 0;
#pragma unroll
    for (int j = 0; j < kShareGroup; ++j)
        n = max(n, seen_by(a, (int64_t)min(lane, runs - 1) * a.group + min(j, a.group - 1)).y);
    if (lane >= runs) n = 0;
    const int steps = (n + kTile - 1) / kTile, all = wave_sum(steps);
    int most = steps;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = max(most, __shfl_xor(most, d));
    const auto parts_at = [&](int per) { return lane < runs ? max((steps + per - 1) / per, 1) : 0; };
    // The smallest number of steps whose parts the blocks suffice for lies in low .. high: a part has at most that many, and
    // parts come to at most all / steps + runs.
    const int64_t total = (int64_t)all * tiles;
    int low = max(max((int)((total + blocks - 1) / blocks), (most + kMostParts - 1) / kMostParts), 1), high = max(most, low);
    if (blocks > runs * tiles) high = max((int)min((int64_t)high, total / (blocks - runs * tiles) + 1), low);
    while (low < high) {
        const int per = (low + high) / 2;
        if (wave_sum(parts_at(per)) * tiles <= blocks)
            high = per;
        else
            low = per + 1;
    }
    const int parts = parts_at(low);
    int first = parts * tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int before = __shfl_up(first, d);
        if (lane >= d) first += before;
    }
    return int2{first - parts * tiles, parts};
}

// NH: rows of a block in sixteens. Blocks of 16 rows come in pairs on a compute unit, half its registers each and one
// step's rows in LDS: the two products of a block take turns, and the blocks cover each other's waits. The others have it
// to themselves, and two steps' rows. (Pairs of 32 rows spill registers: 3.4 ms for 514 queries over 16384 entries.)
template <int NH>
constexpr bool kLocalPair = NH == 1;

template <int NH>
struct LocalShared {
    static constexpr bool PAIR = kLocalPair<NH>;
    _Float16 kv[(PAIR ? 1 : 2) * kTile * kD];  // rows; queries and outputs on their ways
    _Float16 p[2][NH * 16 * kPRow];
    float m[NH * 16][4];
    float l[NH * 16][4];
    int over[2][4];
    float2 fr[NH * 16];           // per row: the factor of stage_query, and minus R
    int2 sees[NH * 16];           // per row: the entries it sees, from the span's first on
    _Float16 q[NH * 16 * kQRow];  // the queries' last fragment (the registers hold 15 of 16)
};

// Of a window's entries, perhaps in a ring, or of all visible ones, these in blocks shared out on the device or not. (Template
// arguments: a branch inside a turn of the pipe costs the blocks of 64 rows a sixth, and the few more values that the shared
// blocks keep cost the others a twentieth, in spilled registers.)
enum Entries { kAll, kShared, kWindow };
template <int NH, bool PAGED, Entries ENTRIES>
__global__ __launch_bounds__(256, kLocalPair<NH> ? 2 : 1) void attend_local_kernel(const LocalArgs a, const LocalCut cut, uint32_t units) {
    __shared__ __align__(16) LocalShared<NH> sh;
    constexpr bool PAIR = kLocalPair<NH>, WINDOW = ENTRIES == kWindow;
    constexpr int kRows = NH * 16;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    uint32_t run32, tile, part, parts, unit_of = 0;
    if constexpr (ENTRIES == kShared) {
        const uint32_t share = (units + 7) / 8, unit = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
        if ((blockIdx.x >> 3) >= share || unit >= units) return;
        const int2 own = share_of(a, (int)cut.tiles, (int)units);
        if (unit == 0 && w == 0 && lane < a.nq / a.group) a.shares[lane] = own;
        run32 = (uint32_t)__builtin_popcountll(__ballot(own.y > 0 && own.x <= (int)unit)) - 1;
        const uint32_t v = unit - (uint32_t)__builtin_amdgcn_readlane(own.x, (int)run32);
        parts = (uint32_t)__builtin_amdgcn_readlane(own.y, (int)run32);
        tile = v % cut.tiles, part = v / cut.tiles;
        if (part >= parts) return;  // behind the last run's
        unit_of = unit;
    } else if (cut.whole == cut.tiles) {
        // blocks b, b + 8, .. run on one XCD: it takes neighbouring units, those of a run's part, which read the same entries
        const uint32_t share = (units + 7) / 8, unit = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
        if ((blockIdx.x >> 3) >= share || unit >= units) return;
        tile = unit % cut.tiles, part = unit / cut.tiles % cut.parts, run32 = unit / cut.tiles / cut.parts;
    } else {
        // the longer ones of all runs first
        const uint32_t longer = cut.whole * cut.parts, shorter = cut.tiles - cut.whole, first = units / cut.of_run() * longer;
        if (blockIdx.x >= units) return;
        if (blockIdx.x < first) {
            run32 = blockIdx.x / longer;
            tile = blockIdx.x % longer % cut.whole, part = blockIdx.x % longer / cut.whole;
        } else {
            const uint32_t v = blockIdx.x - first, of_run = shorter * (cut.parts + 1);
            run32 = v / of_run;
            tile = cut.whole + v % of_run % shorter, part = v % of_run / shorter;
        }
    }
    if constexpr (ENTRIES != kShared) parts = cut.parts_of(tile);
    const int64_t run = run32;
    const int r0 = (int)tile * kRows, left = a.group * a.heads - r0;  // rows of the run from r0 on
    const int64_t t0 = run * a.group;                                 // the run's first query
    const int64_t pair0 = t0 * a.heads + r0;                          // the block's first row

    QueryRows<kRows> qr;
    load_query<kRows>(a.q + pair0 * kD, left, qr);

    // the entries that the block's rows see
    const int ta = r0 / a.heads, tb = (min(r0 + kRows, a.group * a.heads) - 1) / a.heads;
    Span sp;
    int2 mine;
    if (ta == tb) {
        mine = seen_by(a, t0 + ta);
        sp = Span{mine.x, mine.y - mine.x, false, 0};
    } else {
        const int row = min(r0 + (lane & (kRows - 1)), a.group * a.heads - 1);
        mine = seen_by(a, t0 + row / a.heads);
        const bool none = mine.y <= mine.x;
        int lo = none ? INT32_MAX : mine.x, hi = none ? 0 : mine.y;
        int lo_most = none ? INT32_MAX : mine.x, hi_least = none ? 0 : mine.y;
#pragma unroll
        for (int d = 1; d < kRows; d <<= 1) {
            lo = min(lo, __shfl_xor(lo, d));
            hi = max(hi, __shfl_xor(hi, d));
            lo_most = max(lo_most, __shfl_xor(lo_most, d));
            hi_least = min(hi_least, __shfl_xor(hi_least, d));
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
        hi = __builtin_amdgcn_readfirstlane(hi);
        sp = Span{lo, hi - lo, __builtin_amdgcn_readfirstlane((int)(lo != lo_most || hi != hi_least)) != 0, 0};
        if (hi == 0) sp = Span{0, 0, false, 0};
        const int64_t each = (a.window + kTile - 1) / kTile * kTile;
        if (WINDOW && each * (tb - ta + 1) < sp.count) {
            sp.each = (int32_t)each;
            sp.count = (int32_t)each * (tb - ta + 1);
        }
    }
    if (w == 0 && lane < kRows) sh.sees[lane] = int2{mine.x - sp.first, mine.y - sp.first};
    if (WINDOW && sp.each) __syncthreads();
    // where they lie
    int64_t base = 0;
    const int32_t* pages = nullptr;
    if (PAGED) {
        const int64_t s = a.places.seq ? (int64_t)a.places.seq[run * a.seq_stride] : run;
        if (s < 0 || s >= a.places.nseq)
            sp.count = 0;
        else
            pages = a.places.pages + s * a.places.pages_stride;
    } else if (a.places.base) {
        base = a.places.base[run];
        if (base <= -a.places.max_n || base >= a.places.rows) sp.count = 0;  // no entry lies in the cache
    }
    if (a.places.rows == 0) sp.count = 0;
    const int steps_all = (sp.count + kTile - 1) / kTile;
    const int per = (steps_all + (int)parts - 1) / (int)parts;
    const int step0 = (int)part * per;
    const int steps = min(per, steps_all - step0);  // may be 0 or less
    const int end = steps > 0 ? min((step0 + steps) * kTile, sp.count) : 0;
    const int i0 = step0 * kTile + w * 16 + c;      // this lane's entry of the first step

    // an entry's row in three stages, so that the loads of each are in flight: its place, its page, its row
    const auto row_in_block = [&](int query) { return max((ta + query) * a.heads - r0, 0); };
    const auto place = [&](int i) {
        if (!WINDOW) return i < end ? i : -1;
        int p = sp.first + i;
        bool there = i < end;
        if (sp.each) {
            const int query = min(i, end - 1) / sp.each;
            const int2 see = sh.sees[row_in_block(query)];
            there &= i - query * sp.each < see.y - see.x;
            p = sp.first + see.x + i - query * sp.each;
        }
        return there ? (int)place_of(a.places, (uint32_t)p) : -1;
    };
    const auto page = [&](int p) { return PAGED ? pages[divided(a.places.page, (uint32_t)max(p, 0))] : 0; };
    const auto row_of = [&](int p, int32_t pg) {
        uint32_t r;
        bool there = p >= 0;
        if (PAGED) {
            const uint32_t in_page = (uint32_t)p - divided(a.places.page, (uint32_t)max(p, 0)) * a.places.page.by;
            const uint64_t at = (uint64_t)(uint32_t)pg * a.places.page.by + in_page;
            there &= pg >= 0 && at < (uint64_t)a.places.rows;
            r = (uint32_t)at;
        } else {
            // the base lies in (-2^30, rows) and p in [0, 2^30): a sum below zero wraps above any row
            r = (uint32_t)base + (uint32_t)p;
            there &= r < (uint32_t)a.places.rows;
        }
        return there ? (int32_t)r : -1;
    };

    LocalPart kv;
    uint32_t scale1 = 0;
    int32_t row = -1;
    int place1 = -1, place2 = -1;
    int32_t page1 = 0;
    if (steps > 0) {
        const int p = place(i0);
        place1 = place(i0 + kTile);
        place2 = place(i0 + 2 * kTile);
        const int32_t pg = page(p);
        page1 = page(place1);
        row = row_of(p, pg);
#pragma unroll
        for (int j = 0; j < 8; ++j) load_piece(a, row, g, j, kv);
        kv.scale = load_scale(a, row, g);
    }
    // angles of the result, while the rows are on their way: one a thread, where they are so few
    const int queries = tb - ta + 1, pairs = parts == 1 && a.turn.freq ? a.turn.rot / 2 : 0;
    const bool early = queries * pairs <= 256;
    float2 angle{};
    if (early && (int)threadIdx.x < queries * pairs)
        angle = angle_of(a, t0 + ta + (int)threadIdx.x / pairs, (int)threadIdx.x % pairs);
    stage_query<kRows>(a.scale, left, qr, sh.kv, sh.fr);
    __syncthreads();
    h8 q[NH][15];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
        const _Float16* at = sh.kv + (n * 16 + c) * kRow + g * 128;
#pragma unroll
        for (int x = 0; x < 15; ++x) q[n][x] = *reinterpret_cast<const h8*>(at + x * 8);
        const h8 ql = *reinterpret_cast<const h8*>(at + 15 * 8);
        if (w == 0) *reinterpret_cast<h8*>(sh.q + (n * 16 + c) * kQRow + g * 8) = ql;
        if constexpr (!PAIR) {
            // in the accumulation half of the register file: matrix operands only
#pragma unroll
            for (int x = 0; x < 15; ++x) asm volatile("" : "+a"(q[n][x]));
        }
    }
    __syncthreads();  // before kv takes rows

    // The second product is 32 rows wide where the block has as many.
    constexpr bool kWide = NH > 1;
    constexpr int kOh = kWide ? NH / 2 : 1, kOv = kWide ? 4 : 8;  // output tiles: rows, values
    typedef std::conditional_t<kWide, v16f, v4f> Out;
    Out o[kOh][kOv] = {};
    const int oc = kWide ? lane & 31 : c;    // this lane's row of an output tile
    const int og = kWide ? lane >> 5 : g;    // and which fours of its values
    v4f s[NH];
    float l[NH], sum[NH];  // this lane's part of the sum of 2^(s2 - R), and of the step formed last
#pragma unroll
    for (int n = 0; n < NH; ++n) l[n] = sum[n] = 0.0f;

    // A row of a step is 1024 bytes, and its 16-byte pieces are exchanged within each 128: piece p lies at
    // p ^ (2 (row % 4) + row / 4 % 2). Eight rows' same pieces (a write), and four rows' same pairs of pieces (a
    // transposed read), then lie in different banks.
    const int at_in = (w * 16 + c) * kD + g * 128 + ((c & 3) * 2 + ((c >> 2) & 1)) * 8;
    const int first = kWide ? (g & 1) * 2 + ((c >> 1) & 1) : (c >> 1) & 1;  // piece
    const int at_out = (og * 8 + (c >> 2)) * kD + w * 128 + (first ^ ((c >> 2) * 2)) * 8 + (c & 1) * 4;

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
        for (int n = 0; n < NH; ++n) l[n] *= __builtin_amdgcn_exp2f(-fr[n].y - r[n]);  // 0 at a row's first entry
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

    // The logits of step i at entries that a row does not see; seen: which of this lane's four have a row; at: where the
    // step's rows lie.
    const auto mask_step = [&](int i, uint32_t seen, const float2 (&fr)[NH], int at_rows) {
        const int e = (step0 + i) * kTile + w * 16 + g * 4;
        const int query = WINDOW && sp.each ? (step0 + i) * kTile / sp.each : 0;  // of the step, where they go one by one
        bool odd = false;
#pragma unroll
        for (int n = 0; n < NH; ++n) {
            const float hole = fr[n].x < 0.0f ? __builtin_inff() : ninf();
            int2 see = sh.sees[n * 16 + c];
            if (WINDOW && sp.each) see = (r0 + n * 16 + c) / a.heads == ta + query ? int2{INT32_MIN, INT32_MAX} : int2{0, 0};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const bool mine = ((seen >> y) & 1) && e + y >= see.x && e + y < see.y;
                odd |= !mine && !(fabsf(s[n][y]) < __builtin_inff());
                s[n][y] = mine ? s[n][y] : hole;
            }
        }
        // A row that holds NaN codes, and that is not there (what was read is another) or that some of the block's queries
        // do not see: for the second product it is zeros (those that see it have a NaN probability). A query's own NaN or
        // infinity looks the same; then nothing is found here.
        if (__any(odd)) {
#pragma unroll 1
            for (int j = 0; j < 16; ++j) {
                h8* at = reinterpret_cast<h8*>(sh.kv + at_rows + (w * 16 + j) * kD + lane * 8);
                const h8 v = *at;
                bool bad = false;
#pragma unroll
                for (int y = 0; y < 8; ++y) bad |= !(fabsf((float)v[y]) < __builtin_inff());
                if (__any(bad)) *at = h8{};
            }
        }
    };

    // Turn i of the pipe, after a barrier: the first product of step i + 1 (its rows widened, multiplied, left in LDS) and
    // the second product of step i, then the probabilities of step i + 1 under the rest of the second product. Widening,
    // exponentials, LDS and loads run under the matrix instructions.
    const auto turn = [&](auto pv, auto qk, auto first_step, int i) {
        constexpr bool kPv = decltype(pv)::value, kQk = decltype(qk)::value, kFirst = decltype(first_step)::value;
        const int buf = i & 1;
        const int in = at_in ^ (PAIR || buf ? 0 : kTile * kD);
        const int out = at_out ^ (!PAIR && buf ? kTile * kD : 0);
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
        const bool there = row >= 0;
        const uint64_t all = __ballot(there);
        int32_t row1 = -1;
        if constexpr (kQk) {
            row1 = row_of(place1, page1);
            place1 = place2;
            page1 = page(place2);
            place2 = place(i0 + (i + 4) * kTile);
            k = local_values8(kv, 0);
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
                if (x < 15) k = local_values8(kv, x + 1);
                if (x == 3) scale1 = load_scale(a, row1, g);
                if (x & 1) load_piece(a, row1, g, x >> 1, kv);
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
            row = row1;
            kv.scale = scale1;
            float2 fr[NH];
#pragma unroll
            for (int n = 0; n < NH; ++n) fr[n] = sh.fr[n * 16 + c];
            if (all != ~0ull || sp.mixed) mask_step(i + 1, (uint32_t)all >> (g * 4), fr, in - at_in);
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
            const int any = __any(over);
            sh.over[buf ^ 1][w] = any;
            __syncthreads();
        }
    };

    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (steps > 0) {
        turn(no, yes, yes, -1);
        if constexpr (PAIR) {
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
    // The block's outputs in fp32 through LDS (piece p of a row, 4 values, at p ^ row % 32), to be written whole
    float* rows = reinterpret_cast<float*>(sh.kv);
#pragma unroll
    for (int n = 0; n < kOh; ++n) {
        const int hl = n * 32 + oc;
        // four values of tile d lie at 16 d + 4 g, or, wide, at 32 (d / 4) + 8 (d % 4) + 4 og
        constexpr int kFours = kWide ? 16 : 8;
#pragma unroll
        for (int d = 0; d < kFours; ++d) {
            v4f x;
            if constexpr (kWide) {
                const Out& u = o[n][d >> 2];
                const int i = (d & 3) * 4;
                x = v4f{u[i], u[i + 1], u[i + 2], u[i + 3]};
            } else {
                x = o[n][d];
            }
            const int at = w * 128 + (kWide ? (d >> 2) * 32 + (d & 3) * 8 + og * 4 : d * 16 + og * 4);
            *reinterpret_cast<v4f*>(rows + hl * kD + (((at >> 2) ^ (hl & 31)) << 2)) = x;
        }
    }
    // angles of the block's queries, as many at a time as fit where the probabilities were
    float2* cs = reinterpret_cast<float2*>(sh.p);
    const bool finish = parts == 1;
    const int batch = early ? queries : pairs ? min(queries, (int)(sizeof(sh.p) / sizeof(float2)) / pairs) : queries;
    for (int first_query = 0; first_query < queries; first_query += batch) {
        const int some = min(batch, queries - first_query);
        if (early) {
            if ((int)threadIdx.x < queries * pairs) cs[threadIdx.x] = angle;
        } else {
            for (int i = threadIdx.x; i < some * pairs; i += 256)
                cs[i] = angle_of(a, t0 + ta + first_query + i / pairs, i % pairs);
        }
        __syncthreads();
        const int begin = max((ta + first_query) * a.heads - r0, 0);
        const int stop = min((ta + first_query + some) * a.heads - r0, min(kRows, left));
        // four rows at a time, the other part's on their way together
        for (int h0 = begin + ((w - begin) & 3); h0 < stop; h0 += 16) {
            uint4 u[4] = {};
            float l2[4] = {};
            if (finish && a.other) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (h0 + 4 * k >= stop) break;
                    u[k] = *reinterpret_cast<const uint4*>(a.other + (pair0 + h0 + 4 * k) * kD + 8 * lane);
                    l2[k] = a.other_lse[pair0 + h0 + 4 * k];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int hl = h0 + 4 * k;
                if (hl >= stop) break;
                const v4f lv = *reinterpret_cast<const v4f*>(sh.l[hl]);
                const float L = (lv[0] + lv[1]) + (lv[2] + lv[3]), R = -sh.fr[hl].y;
                float* row = rows + hl * kD;
                const v4f x = *reinterpret_cast<const v4f*>(row + (((2 * lane) ^ (hl & 31)) << 2));
                const v4f y = *reinterpret_cast<const v4f*>(row + (((2 * lane + 1) ^ (hl & 31)) << 2));
                const int64_t pair = pair0 + hl;
                if (!finish) {
                    const int64_t at = ENTRIES == kShared ? (int64_t)unit_of * kRows + hl : pair * cut.slots() + part;
                    *reinterpret_cast<v4f*>(a.part_o + at * kD + 8 * lane) = x;
                    *reinterpret_cast<v4f*>(a.part_o + at * kD + 8 * lane + 4) = y;
                    if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = float2{R, L};
                    continue;
                }
                const Weights wt = join_weights(a, l2[k], R, L);
                float v[8] = {x[0] * wt.mine, x[1] * wt.mine, x[2] * wt.mine, x[3] * wt.mine,
                              y[0] * wt.mine, y[1] * wt.mine, y[2] * wt.mine, y[3] * wt.mine};
                add_other(u[k], wt.other, v);
                if (pairs) turn_row(a, cs + (queries == 1 ? 0 : (r0 + hl) / a.heads - ta - first_query) * pairs, row, v);
                store_row(a, pair, v);
                if (a.lse && lane == 0) a.lse[pair] = wt.lse;
            }
        }
        if (first_query + batch < queries) __syncthreads();  // before the next angles
    }
}

// The parts of a row, joined by G wavefronts that take every G-th (o = sum 2^(R_i - R) o_i over sum 2^(R_i - R) l_i), then
// as above.
template <int G>
__global__ __launch_bounds__(256) void local_join_kernel(const LocalArgs a, const LocalCut cut) {
    constexpr int kRows = 4 / G;  // of a block
    __shared__ __align__(16) float s_o[4][kD];
    __shared__ __align__(16) float2 s_cs[kRows][kD / 2];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, own = w / G, take = w % G;
    const int64_t all = (int64_t)a.nq * a.heads, at_row = (int64_t)blockIdx.x * kRows + own;
    const bool live = at_row < all;
    const int64_t pair = live ? at_row : all - 1, of_run = (int64_t)a.group * a.heads;
    const int rows = 16 * cut.nh, in_run = (int)(pair % of_run), tile = in_run / rows;
    int parts = (int)cut.parts_of(tile);
    int64_t slot = pair * cut.slots(), next = 1;  // the row's first part, and the next one from it
    if (cut.shared) {
        const int2 own = a.shares[pair / of_run];
        parts = own.y;
        slot = (int64_t)(own.x + tile) * rows + in_run % rows, next = (int64_t)cut.tiles * rows;
    }
    float2 ml{kNone, 0.0f};
    if (lane < parts) ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (slot + lane * next));
    uint4 u{};
    float l2 = 0.0f;
    if (take == 0 && a.other) {
        u = *reinterpret_cast<const uint4*>(a.other + pair * kD + 8 * lane);
        l2 = a.other_lse[pair];
    }
    if (a.turn.freq) {
        for (int i = take * 64 + lane; i < a.turn.rot / 2; i += 64 * G) s_cs[own][i] = angle_of(a, pair / a.heads, i);
    }
    float R = ml.x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) R = fmaxf(R, __shfl_xor(R, d));
    const float f = __builtin_amdgcn_exp2f(ml.x - R);
    float L = f * ml.y;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) L += __shfl_xor(L, d);
    const float* po = a.part_o + slot * kD + 8 * lane;
    v4f x{}, y{};
#pragma unroll 4
    for (int i = take; i < parts; i += G) {
        const float fi = __shfl(f, i);
        x += fi * reinterpret_cast<const v4f*>(po + i * next * kD)[0];
        y += fi * reinterpret_cast<const v4f*>(po + i * next * kD)[1];
    }
    if constexpr (G > 1) {
        *reinterpret_cast<v4f*>(s_o[w] + 8 * lane) = x;
        *reinterpret_cast<v4f*>(s_o[w] + 8 * lane + 4) = y;
    }
    __syncthreads();
    if (take || !live || parts == 1) return;  // (a row in one part is done)
    if constexpr (G > 1) {
#pragma unroll
        for (int k = 1; k < G; ++k) {
            x += *reinterpret_cast<const v4f*>(s_o[w + k] + 8 * lane);
            y += *reinterpret_cast<const v4f*>(s_o[w + k] + 8 * lane + 4);
        }
    }
    const Weights wt = join_weights(a, l2, R, L);
    float v[8] = {x[0] * wt.mine, x[1] * wt.mine, x[2] * wt.mine, x[3] * wt.mine,
                  y[0] * wt.mine, y[1] * wt.mine, y[2] * wt.mine, y[3] * wt.mine};
    add_other(u, wt.other, v);
    if (a.turn.freq) turn_row(a, s_cs[own], s_o[w], v);
    store_row(a, pair, v);
    if (a.lse && lane == 0) a.lse[pair] = wt.lse;
}

// ---- windows of queries that follow each other ----
// Consecutive queries of a sequence see nearly the same window, so a block takes as many of them as fit: their entries are
// widened into LDS once, and then its wavefronts take 16 rows at a time, each by itself (no barrier): the products with all
// entries, an exact softmax, the second product with the probabilities where the first left them, half of the values at a
// time, and the result. The order in which a product adds up its entries is free, so the probabilities of two tiles of 16
// entries are the second product's operand as they lie, and the values' transposed reads go by that order. 4096 queries of 64
// heads over 128 entries, joined and turned: 183 us (573 by the kernel above, which widens every query's entries again),
// 805 MB at 4.4 TB/s.
constexpr int kWinTiles = 9;                   // of 16 entries
constexpr int kWinKeys = 16 * kWinTiles;       // 144 rows of 1 KB
constexpr int kWinWaves = 8;
constexpr int kWinCuts = 2;                    // of the values, for the second product
constexpr int kWinAngles = 1536;
constexpr int kWinQueries = 64;                // at most, a lane each

struct WindowShared {
    _Float16 kv[kWinKeys * kD];  // a row's 16-byte piece p lies at p ^ win_swap(row)
    float2 cs[kWinAngles];
    int2 sees[kWinQueries];
    uint32_t absent[5], bad[5];  // a bit for each entry: no row, NaN codes
};
// Rows of a transposed read (4) and of an ordinary one (16) exchanged so that they lie in different banks.
__device__ __forceinline__ int win_swap(int row) { return (row & 3) * 2 + ((row >> 2) & 1) * 8 + ((row >> 3) & 1); }

// this lane's eight values of finish64
__device__ __forceinline__ int of_64(int g) { return (g & 1) * 16 + (g & 2) * 4; }
// Values `from` .. + 63 of a row, in four tiles o of 16 where a lane has four of each (4 g ..), joined with the other part's
// u, turned and written. Lane groups exchange halves of two tiles: eight values in a row each, of 32 by 32 two at a time.
__device__ __forceinline__ void finish64(const LocalArgs& a, int64_t pair, bool live, int from, const v4f* o, const uint4* u,
                                         const Weights& wt, const float2* cs) {
    const int mine8 = of_64((threadIdx.x & 63) >> 4), at = from + mine8, pairs = a.turn.freq ? a.turn.rot / 2 : 0;
    const int turn_at = a.turn.freq ? a.turn.offset : kD;
    float v[2][8];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const v4f x = o[2 * b], z = o[2 * b + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const auto sw = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[i]), __float_as_uint(z[i]), false, false);
            v[b][i] = __uint_as_float(sw[0]) * wt.mine;
            v[b][4 + i] = __uint_as_float(sw[1]) * wt.mine;
        }
        const uint32_t x2[4] = {u[b].x, u[b].y, u[b].z, u[b].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[b][2 * i] = fmaf(wt.other, __uint_as_float(x2[i] << 16), v[b][2 * i]);
            v[b][2 * i + 1] = fmaf(wt.other, __uint_as_float(x2[i] & 0xffff0000u), v[b][2 * i + 1]);
        }
    }
    const int from_turn = from - turn_at;  // of the block's first value
    if (from_turn > -64 && from_turn < 2 * pairs) {
        if (a.turn.half) {  // 64 values at a multiple of 64
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 z = cs[mine8 + i];
                const float x0 = v[0][i], x1 = v[1][i];
                v[0][i] = x0 * z.x - x1 * z.y;
                v[1][i] = x1 * z.x + x0 * z.y;
            }
        } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = at + 32 * b + 2 * i - turn_at;
                    if (j < 0 || j >= 2 * pairs) continue;
                    const float2 z = cs[j >> 1];
                    const float x0 = v[b][2 * i], x1 = v[b][2 * i + 1];
                    v[b][2 * i] = x0 * z.x - x1 * z.y;
                    v[b][2 * i + 1] = x1 * z.x + x0 * z.y;
                }
            }
        }
    }
    if (live) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
            *reinterpret_cast<uint4*>(a.out + pair * kD + at + 32 * b) =
                uint4{bf16_pair(v[b][0], v[b][1]), bf16_pair(v[b][2], v[b][3]), bf16_pair(v[b][4], v[b][5]),
                      bf16_pair(v[b][6], v[b][7])};
    }
}

__global__ __launch_bounds__(64 * kWinWaves) void attend_window_kernel(const LocalArgs a, int queries, uint32_t per_run,
                                                                       uint32_t units) {
    __shared__ __align__(16) WindowShared sh;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    const uint32_t share = (units + 7) / 8, unit = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= share || unit >= units) return;
    const int64_t run = unit / per_run;
    const int q0 = (int)(unit % per_run) * queries, some = min(queries, a.group - q0);
    const int64_t t0 = run * a.group + q0;
    int64_t base = 0, s = 0;
    bool cached = a.places.rows > 0;
    if (a.places.pages) {
        s = a.places.seq ? (int64_t)a.places.seq[run * a.seq_stride] : run;
        cached &= s >= 0 && s < a.places.nseq;
    } else if (a.places.base) {
        base = a.places.base[run];
    }
    const int2 mine = lane < some ? seen_by(a, t0 + lane) : int2{0, 0};
    const bool none = mine.y <= mine.x || !cached;
    const int pairs = a.turn.freq ? a.turn.rot / 2 : 0;

    // As many queries at a time as see kWinKeys entries together: all of them, unless their lengths do not follow each
    // other.
    for (int begin = 0; begin < some;) {
        int lo = INT32_MAX, hi = 0, stop = begin;
        {
            const bool there = lane >= begin && !none;
            int l = there ? mine.x : INT32_MAX, h = there ? mine.y : 0;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                l = min(l, __shfl_xor(l, d));
                h = max(h, __shfl_xor(h, d));
            }
            lo = __builtin_amdgcn_readfirstlane(l);
            hi = __builtin_amdgcn_readfirstlane(h);
        }
        if (hi == 0 || hi - lo <= kWinKeys) {
            stop = some;
        } else {
            lo = INT32_MAX, hi = 0;
            for (; stop < some; ++stop) {
                const int l = __builtin_amdgcn_readlane(none ? INT32_MAX : mine.x, stop);
                const int h = __builtin_amdgcn_readlane(none ? 0 : mine.y, stop);
                const int l2 = min(lo, l), h2 = max(hi, h);
                if (h2 > 0 && h2 - l2 > kWinKeys) break;
                lo = l2, hi = h2;
            }
        }
        const int first = hi ? lo : 0, count = hi ? hi - lo : 0;
        if (threadIdx.x < 5) sh.absent[threadIdx.x] = sh.bad[threadIdx.x] = 0;
        if (w == 0) sh.sees[lane] = none ? int2{0, 0} : int2{mine.x - first, mine.y - first};
        __syncthreads();

        // the entries: 16 values a lane, two rows a wavefront
        constexpr int kReads = (kWinKeys + 2 * kWinWaves - 1) / (2 * kWinWaves);
        {
            const int part = lane & 31;
            int64_t row[kReads];
            uint4 code[kReads];
            uint32_t scale[kReads];
#pragma unroll
            for (int i = 0; i < kReads; ++i) {
                const int e = (i * kWinWaves + w) * 2 + (lane >> 5);
                row[i] = e < count ? row_at(a.places, s, base, (int64_t)first + e) : -1;
            }
#pragma unroll
            for (int i = 0; i < kReads; ++i) {
                code[i] = uint4{0, 0, 0, 0};
                scale[i] = 0;
                if (row[i] >= 0) {
                    code[i] = *reinterpret_cast<const uint4*>(a.codes + row[i] * kD + 16 * part);
                    scale[i] = a.scales[row[i] * 16 + (part >> 1)];
                }
            }
            for (int i = threadIdx.x; i < (stop - begin) * pairs; i += 64 * kWinWaves)
                sh.cs[i] = angle_of(a, t0 + begin + i / pairs, i % pairs);
#pragma unroll
            for (int i = 0; i < kReads; ++i) {
                const int e = (i * kWinWaves + w) * 2 + (lane >> 5);
                if (kWinKeys % (2 * kWinWaves) && (i * kWinWaves + w) * 2 >= kWinKeys) continue;
                const float by = __uint_as_float(scale[i] << 23);
                const uint32_t word[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
                h8 v[2];
                bool odd = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const h2 x = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word[j], by, false);
                    const h2 y = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word[j], by, true);
                    v[j >> 1][(j & 1) * 4] = x[0], v[j >> 1][(j & 1) * 4 + 1] = x[1];
                    v[j >> 1][(j & 1) * 4 + 2] = y[0], v[j >> 1][(j & 1) * 4 + 3] = y[1];
                    odd |= !(fabsf((float)x[0]) < __builtin_inff()) | !(fabsf((float)x[1]) < __builtin_inff()) |
                           !(fabsf((float)y[0]) < __builtin_inff()) | !(fabsf((float)y[1]) < __builtin_inff());
                }
                const uint64_t odd_lanes = __ballot(odd);
                const bool bad = (uint32_t)(lane >> 5 ? odd_lanes >> 32 : odd_lanes) != 0;
                if (bad) v[0] = v[1] = h8{};
                if (part == 0 && e < count) {
                    if (row[i] < 0) atomicOr(&sh.absent[e >> 5], 1u << (e & 31));
                    if (bad) atomicOr(&sh.bad[e >> 5], 1u << (e & 31));
                }
                _Float16* at = sh.kv + e * kD;
                *reinterpret_cast<h8*>(at + ((2 * part) ^ win_swap(e)) * 8) = v[0];
                *reinterpret_cast<h8*>(at + ((2 * part + 1) ^ win_swap(e)) * 8) = v[1];
            }
        }
        __syncthreads();
        uint32_t flags = 0;
#pragma unroll
        for (int i = 0; i < 5; ++i) flags |= sh.absent[i] | sh.bad[i];
        flags = __builtin_amdgcn_readfirstlane(flags);

        const int rows = (stop - begin) * a.heads;
        const int64_t pair0 = (t0 + begin) * a.heads;
        for (int tile = w; tile * 16 < rows; tile += kWinWaves) {
            const int r = min(tile * 16 + c, rows - 1), query = r / a.heads;
            const bool live = tile * 16 + c < rows;
            const int64_t pair = pair0 + r;
            // the rows' queries, as scaled fp16 (as stage_query)
            h8 q[16];
            float fr;
            {
                uint4 raw[16];
                const uint16_t* at = a.q + pair * kD + 8 * g;
#pragma unroll
                for (int x = 0; x < 16; ++x) raw[x] = *reinterpret_cast<const uint4*>(at + 32 * x);
                us2 two = {0, 0};
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    two = __builtin_elementwise_max(two, __builtin_bit_cast(us2, raw[x].x & 0x7fff7fffu));
                    two = __builtin_elementwise_max(two, __builtin_bit_cast(us2, raw[x].y & 0x7fff7fffu));
                    two = __builtin_elementwise_max(two, __builtin_bit_cast(us2, raw[x].z & 0x7fff7fffu));
                    two = __builtin_elementwise_max(two, __builtin_bit_cast(us2, raw[x].w & 0x7fff7fffu));
                }
                const uint32_t m = max32(max16(max((uint32_t)two[0], (uint32_t)two[1])));
                int e = (int)(m >> 7);
                const bool finite = e < 255;
                e = e < 15 ? 15 : (e > 254 ? 254 : e);
                const float mul = finite ? __uint_as_float((uint32_t)(127 + 141 - e) << 23) : __builtin_nanf("");
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const uint32_t v[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        q[x][2 * y] = (_Float16)(__uint_as_float(v[y] << 16) * mul);
                        q[x][2 * y + 1] = (_Float16)(__uint_as_float(v[y] & 0xffff0000u) * mul);
                    }
                    if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                }
                fr = a.scale * kLog2e * __uint_as_float((uint32_t)(e - 14) << 23);
            }
            const int2 see = sh.sees[begin + query];
            // the tiles of entries that any of the rows sees, and those that all see whole
            int from = see.y > see.x ? see.x : INT32_MAX, to = see.y > see.x ? see.y : 0, low = see.x, high = see.y;
            from = min(from, (int)dpp<0xB1>(from)), to = max(to, (int)dpp<0xB1>(to));  // quad_perm [1,0,3,2]
            low = max(low, (int)dpp<0xB1>(low)), high = min(high, (int)dpp<0xB1>(high));
            from = min(from, (int)dpp<0x4E>(from)), to = max(to, (int)dpp<0x4E>(to));  // quad_perm [2,3,0,1]
            low = max(low, (int)dpp<0x4E>(low)), high = min(high, (int)dpp<0x4E>(high));
            from = min(from, (int)dpp<0x141>(from)), to = max(to, (int)dpp<0x141>(to));  // row_half_mirror
            low = max(low, (int)dpp<0x141>(low)), high = min(high, (int)dpp<0x141>(high));
            from = min(from, (int)dpp<0x140>(from)), to = max(to, (int)dpp<0x140>(to));  // row_mirror
            low = max(low, (int)dpp<0x140>(low)), high = min(high, (int)dpp<0x140>(high));
            from = __builtin_amdgcn_readfirstlane(from) / 16;
            to = (__builtin_amdgcn_readfirstlane(to) + 15) / 16;
            low = __builtin_amdgcn_readfirstlane(low);
            high = __builtin_amdgcn_readfirstlane(high);

            v4f y[kWinTiles];
            // (the lane's place in the first entries' rows; the exchange of pieces makes the others differ in single bits)
            int at_key = c * kD + (g ^ win_swap(c)) * 8;
            asm volatile("" : "+v"(at_key));  // not kept for all of them over the rows
#pragma unroll
            for (int k3 = 0; k3 < kWinTiles; k3 += 3) {
                v4f d[3] = {};
                if (k3 + 3 > from && k3 < to) {
                    const _Float16* at = sh.kv + k3 * 16 * kD;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const _Float16* piece = at + (at_key ^ ((x & 3) * 32)) + (x >> 2) * 128;
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const h8 v = *reinterpret_cast<const h8*>(piece + k * 16 * kD);
                            d[k] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, q[x], d[k], 0, 0, 0);
                        }
                        if (x % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                    }
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const int e = (k3 + k) * 16;
                    y[k3 + k] = d[k] * fr;
                    if (e < low || e + 16 > high) {  // some rows see only some of them
                        const uint32_t place = (uint32_t)(e + 4 * g - see.x), seen = (uint32_t)max(see.y - see.x, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[k3 + k][i] = place + i < seen ? y[k3 + k][i] : ninf();
                    }
                }
            }
            if (flags) {
#pragma unroll
                for (int k = 0; k < kWinTiles; ++k) {
                    const int e = k * 16 + 4 * g;
                    const uint32_t absent = sh.absent[e >> 5] >> (e & 31), bad = sh.bad[e >> 5] >> (e & 31);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if ((absent >> i) & 1) y[k][i] = ninf();
                        if (((bad >> i) & 1) && e + i >= see.x && e + i < see.y) y[k][i] = __builtin_nanf("");
                    }
                }
            }
            float top = ninf();
#pragma unroll
            for (int k = 0; k < kWinTiles; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, y[k][i]);
            }
            top = group_max(top);
            // probabilities up to 2^15: those down to 2^-29 of the largest are normal fp16 numbers
            const float R = top > ninf() ? ceilf(top) - 15.0f : 0.0f;
            float L = 0.0f;
            h8 p[(kWinTiles + 1) / 2];
#pragma unroll
            for (int k = 0; k < kWinTiles; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float ex = __builtin_amdgcn_exp2f(y[k][i] - R);
                    L += ex;
                    p[k / 2][(k & 1) * 4 + i] = (_Float16)ex;
                }
            }
            L = group_sum(L);
            __builtin_amdgcn_sched_barrier(0);
            const Weights wt = join_weights(a, a.other ? a.other_lse[pair] : 0.0f, R, L);
            if (a.lse && g == 0 && live) a.lse[pair] = wt.lse;

            // lane (c, g) reads four values' piece of entry 4g + c / 4 of a tile; it gets value c of four entries
            const int entry = 4 * g + (c >> 2);
            int at_value = entry * kD + (((c & 3) >> 1) ^ win_swap(entry)) * 8 + (c & 1) * 4;
            asm volatile("" : "+v"(at_value));
            const float2* cs = sh.cs + query * pairs;
#pragma unroll 1
            for (int half = 0; half < kWinCuts; ++half) {
                constexpr int kTwos = 8 / kWinCuts, kValues = kD / kWinCuts;  // blocks of 64 values
                v4f o[4 * kTwos] = {};
                const int mine8 = of_64(g);
                uint4 u[2 * kTwos] = {};
                if (wt.other != 0.0f) {  // (what lies in a part of no weight has no effect)
#pragma unroll
                    for (int b = 0; b < 2 * kTwos; ++b)
                        u[b] = *reinterpret_cast<const uint4*>(a.other + pair * kD + half * kValues + 32 * b + mine8);
                }
#pragma unroll
                for (int k = 0; k < kWinTiles; k += 2) {
                    if (k + 2 <= from || k >= to) continue;
#pragma unroll
                    for (int d = 0; d < 4 * kTwos; ++d) {
                        const _Float16* at = sh.kv + half * kValues + k * 16 * kD + (at_value ^ ((d & 7) * 16)) + (d >> 3) * 128;
                        const hv4 l4 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)at);
                        if (k + 1 < kWinTiles) {
                            const hv4 h4v = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(at + 16 * kD));
                            h8 v;
                            __builtin_memcpy(&v, &l4, 8);
                            __builtin_memcpy((char*)&v + 8, &h4v, 8);
                            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p[k / 2], o[d], 0, 0, 0);
                        } else {
                            h4 v;
                            __builtin_memcpy(&v, &l4, 8);
                            const h4 last = {p[k / 2][0], p[k / 2][1], p[k / 2][2], p[k / 2][3]};
                            o[d] = __builtin_amdgcn_mfma_f32_16x16x16f16(v, last, o[d], 0, 0, 0);
                        }
                        if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int two = 0; two < kTwos; ++two) {
                    finish64(a, pair, live, half * kValues + two * 64, o + 4 * two, u + 2 * two, wt, cs);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        begin = stop;
        if (begin < some) __syncthreads();  // before other entries take the place
    }
}

// ---- one query, few entries ----
// One query that sees at most 128 entries, a decode step's window: eight wavefronts read and widen 16 entries each and keep
// them in registers and LDS. Then 16 heads at a time: each wavefront multiplies its entries with them and leaves the
// probabilities in LDS, against a reference of its own; behind a barrier each multiplies 64 values of all the entries with
// the probabilities, brought to the largest of the references (powers of two), and finishes them. A wavefront reads two
// whole rows at once: of 16 rows a piece each, its lanes' addresses alone take 64 cycles (128 rows 1.7 us). One query of 64
// heads over 128 entries, joined and turned: 7.6 us in four blocks, 10.25 by the kernel above, in two steps of 64 entries.
// What bounds it is one wavefront's way through: five loads one behind the other, LDS, two barriers.
// Each 16 heads more of a block take 3 us, most of it vector instructions.
constexpr int kOneKeys = 128;
struct OneShared {
    _Float16 kv[kOneKeys * kD];  // a row's first half holds its codes before
    _Float16 q[16 * kRow];
    _Float16 p[8][16][16];  // by wavefront, head and entry
    float m[16][8], l[16][8];
    float2 fr[16];
    float2 cs[kD / 2];
};

__global__ __launch_bounds__(512) void attend_one_kernel(const LocalArgs a, int tiles, uint32_t per_query, uint32_t units) {
    __shared__ __align__(16) OneShared sh;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    const uint32_t share = (units + 7) / 8, unit = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= share || unit >= units) return;
    const int64_t t = unit / per_query, run = t / a.group;
    const int first = (int)(unit % per_query) * tiles * 16, stop = min(first + tiles * 16, a.heads);

    QueryRows<16, 8> qr;
    load_query<16, 8>(a.q + (t * a.heads + first) * kD, stop - first, qr);
    const int2 see = seen_by(a, t);
    const int count = see.y - see.x;
    int32_t row = -1;  // of entry 16 w + c
    if (16 * w + c < count && a.places.rows > 0)
        row = (int32_t)row_at(a.places, a.places.seq ? (int64_t)a.places.seq[run * a.seq_stride] : run, a.places.base ? a.places.base[run] : 0,
                              (int64_t)see.x + 16 * w + c);
    // two rows at a time, whole
    uint4 code[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int even = __builtin_amdgcn_readlane(row, 2 * i), odd = __builtin_amdgcn_readlane(row, 2 * i + 1);
        const int r = lane < 32 ? even : odd;
        code[i] = uint4{0, 0, 0, 0};
        if (r >= 0) code[i] = *reinterpret_cast<const uint4*>(a.codes + (int64_t)r * kD + 16 * (lane & 31));
    }
    LocalPart kv;
    kv.scale = row >= 0 ? load_scale(a, row, g) : 0;
    const uint32_t seen = (uint32_t)__ballot(row >= 0) >> (4 * g);
    uint4 u[2] = {};
    float l2 = 0.0f;
    const auto load_other = [&](int head) {
        if (!a.other) return;
        const int64_t pair = t * a.heads + min(head + c, stop - 1);
        l2 = a.other_lse[pair];
#pragma unroll
        for (int b = 0; b < 2; ++b) u[b] = *reinterpret_cast<const uint4*>(a.other + pair * kD + 64 * w + 32 * b + of_64(g));
    };
    load_other(first);
    if (a.turn.freq && (int)threadIdx.x < a.turn.rot / 2) sh.cs[threadIdx.x] = angle_of(a, t, threadIdx.x);
    stage_query<16, 8>(a.scale, stop - first, qr, sh.q, sh.fr);
    // A row's codes through its place in LDS, from two rows a wavefront to this lane's part of one (piece p of entry e at
    // p ^ e: sixteen entries' same pieces, and a row's, in different banks)
    uint4* raw = reinterpret_cast<uint4*>(sh.kv) + 16 * w * 64;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = 2 * i + (lane >> 5);
        raw[e * 64 + ((lane & 31) ^ e)] = code[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < 8; ++j) kv.code[j] = raw[c * 64 + ((8 * g + j) ^ c)];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    h8 keys[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
        keys[x] = local_values8(kv, x);
        *reinterpret_cast<h8*>(sh.kv + (16 * w + c) * kD + ((16 * g + x) ^ win_swap(c)) * 8) = keys[x];
    }

    for (int head = first;;) {
        const int left = min(stop - head, 16);
        const int64_t pair = t * a.heads + head + min(c, left - 1);
        __syncthreads();  // the queries are there; the tile before is done with the probabilities
        v4f s[2] = {};
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const h8 q = *reinterpret_cast<const h8*>(sh.q + c * kRow + g * 128 + x * 8);
            s[x & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(keys[x], q, s[x & 1], 0, 0, 0);
        }
        const bool more = head + 16 < stop;
        if (more) load_query<16, 8>(a.q + (t * a.heads + head + 16) * kD, stop - head - 16, qr);
        {
            const float fr = sh.fr[c].x;
            float y[4], top = ninf(), l = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = seen >> i & 1 ? (s[0][i] + s[1][i]) * fr : ninf();
                top = fmaxf(top, y[i]);
            }
            top = group_max(top);
            const float R = top > ninf() ? ceilf(top) - 15.0f : 0.0f;  // probabilities as the window kernel's
            h4 p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float ex = __builtin_amdgcn_exp2f(y[i] - R);
                l += ex;
                p[i] = (_Float16)ex;
            }
            l = group_sum(l);
            *reinterpret_cast<h4*>(&sh.p[w][c][4 * g]) = p;
            if (g == 0) sh.m[c][w] = top > ninf() ? R : kNone, sh.l[c][w] = l;
        }
        // other_lse may be lse, which the first wavefront writes behind the barrier: every wavefront's read of it ends before
        // (a barrier waits for LDS alone; the wait that the join has right behind it stands here instead)
        asm volatile("" : "+v"(l2));
        __syncthreads();

        // The wavefronts' references below the largest (none: far enough below). Their probabilities are brought to it in
        // fp16, rounded where they leave its normal numbers: below 2^-28 of the largest.
        int down[8];
        float R = kNone, L = 0.0f;
        {
            const v4f m[2] = {*reinterpret_cast<const v4f*>(sh.m[c]), *reinterpret_cast<const v4f*>(sh.m[c] + 4)};
            const v4f l[2] = {*reinterpret_cast<const v4f*>(sh.l[c]), *reinterpret_cast<const v4f*>(sh.l[c] + 4)};
#pragma unroll
            for (int k = 0; k < 8; ++k) R = fmaxf(R, m[k >> 2][k & 3]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float d = fmaxf(m[k >> 2][k & 3] - R, -128.0f);
                down[k] = (int)d;
                L = fmaf(l[k >> 2][k & 3], __builtin_amdgcn_exp2f(d), L);
            }
        }
        const Weights wt = join_weights(a, l2, R, L);
        if (wt.other == 0.0f) u[0] = u[1] = uint4{0, 0, 0, 0};  // (what lies in a part of no weight has no effect)
        // the values' transposed reads go by the order in which the probabilities lie (as in the window kernel)
        const int entry = 4 * g + (c >> 2);
        const int at_value = entry * kD + (((c & 3) >> 1) ^ win_swap(entry)) * 8 + (c & 1) * 4;
        v4f o[4] = {};
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            if (16 * k >= count) continue;
            h8 p;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const h4 x = *reinterpret_cast<const h4*>(&sh.p[k + half][c][4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) p[4 * half + i] = __builtin_ldexpf16(x[i], down[k + half]);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int tile = 4 * w + d;
                const _Float16* at = sh.kv + k * 16 * kD + (at_value ^ ((tile & 7) * 16)) + (tile >> 3) * 128;
                const hv4 low = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)at);
                const hv4 high = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(at + 16 * kD));
                h8 v;
                __builtin_memcpy(&v, &low, 8);
                __builtin_memcpy((char*)&v + 8, &high, 8);
                o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p, o[d], 0, 0, 0);
            }
        }
        if (more) stage_query<16, 8>(a.scale, stop - head - 16, qr, sh.q, sh.fr);
        finish64(a, pair, c < left, 64 * w, o, u, wt, sh.cs);
        if (a.lse && w == 0 && lane < left) a.lse[pair] = wt.lse;
        if (!more) break;
        head += 16;
        load_other(head);
    }
}

// whether the pairs of a rotation lie as finish64 takes them
bool turned_by_64(const LocalArgs& a) {
    return !a.turn.freq || (a.turn.half ? a.turn.rot == 64 && a.turn.offset % 64 == 0 : a.turn.offset % 2 == 0);
}
// The most queries that a block of the window kernel takes; 0: the call is not for it.
int window_queries(const LocalArgs& a) {
    if (a.window <= 0 || a.window > kWinKeys || !turned_by_64(a)) return 0;
    int64_t most = std::min<int64_t>({kWinKeys - a.window + 1, kWinQueries, a.group});
    if (a.turn.freq) most = std::min<int64_t>(most, kWinAngles / (a.turn.rot / 2));
    return (int)most;
}
// whether the kernel of one query and few entries can take the call
bool one_query(const LocalArgs& a) {
    const int64_t entries = a.window > 0 ? std::min(a.window, a.places.max_n) : a.places.max_n;
    return entries <= kOneKeys && (a.group == 1 || a.heads % 16 == 0) && turned_by_64(a);
}

constexpr int64_t up(int64_t x, int64_t by) { return (x + by - 1) / by; }
size_t part_bytes(int64_t rows) { return (size_t)rows * (kD + 2) * sizeof(float); }

// The cut that takes the least time on 256 compute units, by what was measured (microseconds): a block of 16, 32 or 64 rows
// kLocalTiles' apart from its steps and for each step of 64 entries (1 .. 1024 queries of 1 .. 128 heads over 1000 .. 65536
// entries); a join 4, and its parts at 4 TB/s; a block of the window kernel 17, and 14.5 for each 128 rows (9 for a
// last 64); one of one query 3.6, 3.5 for each 16 heads, and 2 shared by the blocks that read the same entries (16 .. 2048
// queries of 16 .. 128 heads; 64 heads over 128 entries: 64 queries 8.6 us and 11.1 without, 256 21.0 and 27.2, 1024 78 and
// 110). `most`: parts that the workspace has room for. most_queries: window_queries(). one: one_query().
constexpr struct {
    int nh, places;
    float step, block, step_alone, block_alone;
} kLocalTiles[] = {{4, 256, 1.8f, 24.0f, 1.8f, 24.0f}, {2, 256, 1.3f, 13.0f, 1.3f, 13.0f}, {1, 512, 2.5f, 9.0f, 1.9f, 7.3f}};

LocalCut best_local_cut(int64_t runs, int64_t group, int64_t heads, int64_t entries, int64_t most, int most_queries, bool one) {
    LocalCut best{1, 1, (uint32_t)up(group * heads, 16), (uint32_t)up(group * heads, 16), 0, 0, false};
    float least = 0.0f;
    const auto consider = [&](float time, const LocalCut& cut) {
        if (least == 0.0f || time < least) least = time, best = cut;
    };
    for (const auto& t : kLocalTiles) {
        const int64_t rows = 16 * t.nh;
        if (t.nh > 1 && group * heads <= 8 * t.nh) continue;  // half of the tile would be empty
        const int64_t tiles = up(group * heads, rows), steps = std::max<int64_t>(up(entries, kTile), 1);
        // the first `whole` tiles of a run in `parts` parts, the others in one more
        const auto in_parts = [&](int64_t parts, int64_t whole) {
            const LocalCut cut{t.nh, (uint32_t)parts, (uint32_t)tiles, (uint32_t)whole, 0, 0, false};
            if (parts < 1 || cut.slots() > kMostParts || (cut.slots() > 1 && (cut.slots() > most || cut.slots() > steps))) return;
            const int64_t n1 = runs * whole * parts, n2 = runs * (tiles - whole) * (parts + 1);
            const bool alone = n1 + n2 <= 256;
            const auto one = [&](int64_t n) {
                return (float)up(steps, n) * (alone ? t.step_alone : t.step) + (alone ? t.block_alone : t.block);
            };
            consider(time_of(t.places, n1, one(parts), n2, n2 ? one(parts + 1) : 0.0f) +
                         (cut.slots() > 1 ? 6.0f + 5e-4f * (float)((n1 + n2) * rows) : 0.0f),
                     cut);
        };
        for (int parts = 1; parts <= 8; ++parts) in_parts(parts, tiles);
        for (int parts = 12; parts <= 64; parts += parts >= 32 ? 16 : parts >= 16 ? 8 : 4) in_parts(parts, tiles);
        for (int rounds = 1; rounds <= 8; ++rounds) {  // whole rounds, as nearly as runs alike allow
            const int64_t of_run = rounds * t.places / runs, parts = of_run / tiles;
            if (parts >= 1) in_parts(parts, tiles * (parts + 1) - of_run);
        }
    }
    for (int queries = 1; queries <= most_queries; ++queries) {
        const int64_t tiles = up(queries * heads, 16), last = tiles % 8;
        const float rows = 14.5f * (float)(tiles / 8) + (last == 0 ? 0.0f : last <= 4 ? 9.0f : 14.5f);
        consider((float)up(runs * up(group, queries), 256) * (17.0f + rows), LocalCut{0, 1, 0, 0, queries, 0, false});
    }
    const int64_t all = up(heads, 16);
    for (int tiles = 1; one && tiles <= all; ++tiles) {
        const int64_t blocks = up(all, tiles);
        consider((float)up(runs * group * blocks, 256) * (3.6f + 3.5f * (float)tiles + 2.0f / (float)blocks),
                 LocalCut{0, 1, 0, 0, 0, tiles, false});
    }
    return best;
}

// The same for the sizes asked for last: the next call mostly has the same.
LocalCut local_cut(int64_t runs, int64_t group, int64_t heads, int64_t entries, int64_t most, int most_queries, bool one) {
    thread_local int64_t of[7] = {0, 0, 0, 0, 0, 0, 0};
    thread_local LocalCut cut{};
    const int64_t now[7] = {runs, group, heads, entries, most, most_queries, one};
    if (memcmp(of, now, sizeof(of))) {
        cut = best_local_cut(runs, group, heads, entries, most, most_queries, one);
        memcpy(of, now, sizeof(of));
    }
    return cut;
}

}  // namespace

size_t local_workspace_bytes(int32_t nq, int32_t heads, int64_t entries) {
    if (nq <= 0 || entries <= 0) return 16;
    // (how the queries come in runs is not known here: as one, whose tiles are the fewest and parts the most)
    const LocalCut cut = best_local_cut(1, nq, heads, entries, kMostParts, 0, false);
    return cut.slots() == 1 ? 16 : cut.slots() * part_bytes((int64_t)nq * heads);
}

hipError_t launch_attend_local(LocalArgs a, void* ws, size_t ws_bytes, hipStream_t stream) {
    const int64_t rows = (int64_t)a.nq * a.heads, runs = a.nq / a.group;
    int64_t entries = a.places.max_n;
    if (a.window > 0) entries = std::min(entries, a.window + std::min<int64_t>(a.group, 16) - 1);
    const int64_t room = std::min<int64_t>(kMostParts, ws_bytes / part_bytes(rows));
    LocalCut cut = local_cut(runs, a.group, a.heads, entries, std::max<int64_t>(room, 1), window_queries(a),
                             one_query(a));
    if (cut.one) {
        const uint32_t per_query = (uint32_t)up(up(a.heads, 16), cut.one), units = (uint32_t)a.nq * per_query;
        hipLaunchKernelGGL(attend_one_kernel, dim3((units + 7) / 8 * 8), dim3(512), 0, stream, a, cut.one, per_query, units);
        return hipGetLastError();
    }
    if (cut.queries) {
        const uint32_t per_run = (uint32_t)up(a.group, cut.queries), units = (uint32_t)runs * per_run;
        hipLaunchKernelGGL(attend_window_kernel, dim3((units + 7) / 8 * 8), dim3(64 * kWinWaves), 0, stream, a, cut.queries,
                           per_run, units);
        return hipGetLastError();
    }
    uint32_t slots = cut.slots(), units = (uint32_t)runs * cut.of_run();
    if (slots > 1) {
        a.part_o = (float*)ws;
        a.part_ml = a.part_o + (size_t)slots * rows * kD;
    }
    // As many blocks for all runs together, in whole rounds: where blocks have eight steps or more (16, of 16 rows). 8 runs of
    // 3 queries of 64 heads over up to 65537 entries: of lengths alike 241 -> 225 us, spread evenly 179 -> 113, one long and
    // seven short 169 -> 60; 8 runs of one query over 4096, two steps a block: 22 -> 26.
    const int64_t places = cut.nh == 1 ? 512 : 256, blocks = up(units, places) * places;
    if (slots > 1 && a.window == 0 && runs > 1 && runs <= kShares && a.group <= kShareGroup &&
        runs * cut.tiles * up(entries, kTile) >= (cut.nh == 1 ? 16 : 8) * blocks &&
        kShares * sizeof(int2) + part_bytes(blocks * 16 * cut.nh) <= ws_bytes) {
        cut.shared = true;
        units = (uint32_t)blocks;
        a.shares = (int2*)ws;
        a.part_o = (float*)(a.shares + kShares);
        a.part_ml = a.part_o + (size_t)blocks * 16 * cut.nh * kD;
    }
    const auto start = [&](auto nh) {
        constexpr int kNh = decltype(nh)::value;
        const dim3 grid((units + 7) / 8 * 8);
        const auto go = [&](auto entries) {
            constexpr Entries kEntries = decltype(entries)::value;
            if (a.places.pages)
                hipLaunchKernelGGL((attend_local_kernel<kNh, true, kEntries>), grid, dim3(256), 0, stream, a, cut, units);
            else
                hipLaunchKernelGGL((attend_local_kernel<kNh, false, kEntries>), grid, dim3(256), 0, stream, a, cut, units);
        };
        if (a.window > 0)
            go(std::integral_constant<Entries, kWindow>{});
        else if (cut.shared)
            go(std::integral_constant<Entries, kShared>{});
        else
            go(std::integral_constant<Entries, kAll>{});
    };
    if (cut.nh == 1)
        start(std::integral_constant<int, 1>{});
    else if (cut.nh == 2)
        start(std::integral_constant<int, 2>{});
    else
        start(std::integral_constant<int, 4>{});
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || slots == 1) return err;
    if (slots > 4 || cut.shared)
        hipLaunchKernelGGL(local_join_kernel<4>, dim3((unsigned)rows), dim3(256), 0, stream, a, cut);
    else
        hipLaunchKernelGGL(local_join_kernel<1>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, cut);
    return hipGetLastError();
}

}  // namespace fp4idx
