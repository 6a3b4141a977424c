// Attention over the FP8 cache of local positions (rows of 512 values, E4M3 codes with a power of two per 32): each
// query's last `window` entries or all it sees, joined with another part of the same softmax (the selection's), and the
// result turned back to the query's frame.
//
//   s_p = scale * q . kv_p,  l = log sum e^{s_p},  o = sum e^{s_p - l} kv_p
//   with another part (o', l'):  L = log(e^l + e^{l'}),  out = e^{l - L} o + e^{l' - L} o'
//
// A block of four wavefronts takes 16 or 32 rows, a row being one head of one query: rows of consecutive queries of a
// sequence share the cache rows they see, so that few heads fill a block too; which entries a row sees is masked where
// the block's queries differ. 64 entries a step: wavefront w reads those 16w .. 16w + 15 straight into registers, widens
// them to fp16, multiplies them with the block's rows and leaves them in LDS; after a barrier it multiplies values
// 128w .. 128w + 127 of all 64 entries with the probabilities. Two blocks on a compute unit cover each other's waits.
//
// Arithmetic. A stored value is an fp16 number; queries are scaled by a power of two per row and exact down to 2^-28 of
// the row's largest; products and sums are fp32. Probabilities enter the second product in 11 bits, against a reference
// 7 below the largest logit that moves when one comes to lie 15 above it (both base 2). The join and the rotation are
// fp32, rounded once.
#include <algorithm>
#include <type_traits>

#include "attend_common.h"
#include "places.h"

namespace fp4idx {
namespace {

constexpr int kMostParts = 64;  // of a run's entries

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

// One lane's share of a cache row: lane group g (of 4) holds values 128g .. 128g + 127 and their four scales.
struct LocalPart {
    uint4 code[8];
    uint32_t scale;
};
__device__ __forceinline__ void load_piece(const LocalArgs& a, int64_t row, int g, int j, LocalPart& r) {
    r.code[j] = *reinterpret_cast<const uint4*>(a.codes + (row < 0 ? 0 : row) * kD + g * 128 + 16 * j);
}
__device__ __forceinline__ uint32_t load_scale(const LocalArgs& a, int64_t row, int g) {
    return *reinterpret_cast<const uint32_t*>(a.scales + (row < 0 ? 0 : row) * 16 + g * 4);
}
// values 8x .. 8x + 7 of the part as fp16 (exact); keep: all ones, or zero for a row that is not there
__device__ __forceinline__ h8 local_values8(const LocalPart& r, int x, uint32_t keep) {
    const uint4 c = r.code[x >> 1];
    const uint32_t w0 = (x & 1 ? c.z : c.x) & keep, w1 = (x & 1 ? c.w : c.y) & keep;
    const float s = __uint_as_float((r.scale >> (8 * (x >> 2)) & 0xffu) << 23);
    const h2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, s, false);
    const h2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, s, true);
    const h2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, s, false);
    const h2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, s, true);
    return h8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// How a call is cut: blocks take `rows` rows (16 or 32) of a run's heads x queries, and one of `parts` parts of the
// entries.
struct LocalCut {
    int nh;
    uint32_t parts, tiles;  // tiles of a run
};

// Weights of a row's sums o and of its other part, and the joined logarithm: L = sum 2^(s2 - R).
struct Weights {
    float mine, other, lse;
};
__device__ __forceinline__ Weights join_weights(const LocalArgs& a, int64_t pair, float R, float L) {
    Weights w{L == 0.0f ? 0.0f : 1.0f / L, 0.0f, L == 0.0f ? ninf() : (__builtin_amdgcn_logf(L) + R) * kLn2};
    if (a.other) {
        const float l2 = a.other_lse[pair], top = fmaxf(w.lse, l2);
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
    sincospif(2.0f * (float)turns_of(a.turn.pos[t], a.turn.freq[pair]), &s, &c);
    const float m = (float)a.turn.mscale;
    return float2{c * m, (a.turn.inverse ? -s : s) * m};
}
// A row's values 8 lane .. + 7, turned by angles cs; row: LDS of its 512 values for pairs that lanes do not hold together
__device__ __forceinline__ void turn_row(const LocalArgs& a, const float2* cs, float* row, float (&v)[8]) {
    const int lane = threadIdx.x & 63, rot = a.turn.rot, pairs = rot / 2, j0 = 8 * lane - a.turn.offset;
    if (!a.turn.half && !(a.turn.offset & 1)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (j0 + 2 * i < 0 || j0 + 2 * i >= rot) continue;
            const float2 z = cs[(j0 >> 1) + i];
            const float x0 = v[2 * i], x1 = v[2 * i + 1];
            v[2 * i] = x0 * z.x - x1 * z.y;
            v[2 * i + 1] = x1 * z.x + x0 * z.y;
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

// NH: rows of a block in sixteens
template <int NH>
struct LocalShared {
    _Float16 kv[kTile * kD];  // a step's rows; queries and outputs on their ways
    _Float16 p[2][NH * 16 * kPRow];
    float m[NH * 16][4];
    float l[NH * 16][4];
    int over[2][4];
    float2 fr[NH * 16];           // per row: the factor of stage_query, and minus R
    int2 sees[NH * 16];           // per row: the entries it sees, from the span's first on
    _Float16 q[NH * 16 * kQRow];  // the queries' last fragment (the registers hold 15 of 16)
};

template <int NH, bool PAGED>
__global__ __launch_bounds__(256, 2) void attend_local_kernel(const LocalArgs a, const LocalCut cut, uint32_t units) {
    __shared__ __align__(16) LocalShared<NH> sh;
    constexpr int kRows = NH * 16;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int g = lane >> 4, c = lane & 15;
    // blocks b, b + 8, .. run on one XCD: it takes neighbouring units, whose rows lie together
    const uint32_t share = (units + 7) / 8, unit = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= share || unit >= units) return;
    const uint32_t tile = unit % cut.tiles, part = unit / cut.tiles % cut.parts;
    const int64_t run = unit / cut.tiles / cut.parts;
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
        if (a.window > 0 && each * (tb - ta + 1) < sp.count) {
            sp.each = (int32_t)each;
            sp.count = (int32_t)each * (tb - ta + 1);
        }
    }
    if (w == 0 && lane < kRows) sh.sees[lane] = int2{mine.x - sp.first, mine.y - sp.first};
    if (sp.each) __syncthreads();
    // where they lie
    int64_t base = 0;
    const int32_t* pages = nullptr;
    if (PAGED) {
        const int64_t s = a.places.seq ? (int64_t)a.places.seq[run] : run;
        if (s < 0 || s >= a.places.nseq)
            sp.count = 0;
        else
            pages = a.places.pages + s * a.places.pages_stride;
    } else if (a.places.base) {
        base = a.places.base[run];
    }
    if (a.places.rows == 0) sp.count = 0;
    const int steps_all = (sp.count + kTile - 1) / kTile;
    const int per = (steps_all + (int)cut.parts - 1) / (int)cut.parts;
    const int step0 = (int)part * per;
    const int steps = min(per, steps_all - step0);  // may be 0 or less
    const int end = steps > 0 ? min((step0 + steps) * kTile, sp.count) : 0;
    const int i0 = step0 * kTile + w * 16 + c;      // this lane's entry of the first step

    // an entry's row in three stages, so that the loads of each are in flight: its place, its page, its row
    const auto row_in_block = [&](int query) { return max((ta + query) * a.heads - r0, 0); };
    const auto place = [&](int i) {
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
        int64_t r;
        if (PAGED) {
            const uint32_t in_page = (uint32_t)p - divided(a.places.page, (uint32_t)max(p, 0)) * a.places.page.by;
            r = pg < 0 ? -1 : (int64_t)pg * a.places.page.by + in_page;
        } else {
            r = (int64_t)((uint64_t)base + (uint32_t)p);
        }
        return p >= 0 && r >= 0 && r < a.places.rows ? r : (int64_t)-1;
    };

    LocalPart kv;
    uint32_t scale1 = 0;
    int64_t row = -1;
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

    // The first product of step i: rows widened, multiplied, left in LDS; then their probabilities.
    const auto first_product = [&](int i, auto first_step) {
        constexpr bool kFirst = decltype(first_step)::value;
        const uint32_t keep = row >= 0 ? ~0u : 0u;
        const bool there = row >= 0;
        const int64_t row1 = row_of(place1, page1);
        place1 = place2;
        page1 = page(place2);
        place2 = place(i0 + (i + 3) * kTile);
        h8 k = local_values8(kv, 0, keep), ql[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n) s[n] = v4f{};
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const h8 kx = k;
            *reinterpret_cast<h8*>(sh.kv + (at_in ^ ((x & 7) * 8)) + (x >> 3) * 64) = kx;
            if (x < 15) k = local_values8(kv, x + 1, keep);
            if (x == 3) scale1 = load_scale(a, row1, g);
            if (x & 1) load_piece(a, row1, g, x >> 1, kv);
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                if (x == 14) ql[n] = *reinterpret_cast<const h8*>(sh.q + (n * 16 + c) * kQRow + g * 8);
                s[n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kx, x < 15 ? q[n][x < 15 ? x : 0] : ql[n], s[n], 0, 0, 0);
            }
        }
        row = row1;
        kv.scale = scale1;
        float2 fr[NH];
#pragma unroll
        for (int n = 0; n < NH; ++n) fr[n] = sh.fr[n * 16 + c];
        const uint64_t all = __ballot(there);
        if (all != ~0ull || sp.mixed) {
            const uint32_t seen = (uint32_t)all >> (g * 4);
            const int e = (step0 + i) * kTile + w * 16 + g * 4;
            bool odd = false;
            const int query = sp.each ? (step0 + i) * kTile / sp.each : 0;  // of the step, where they go one by one
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                const float hole = fr[n].x < 0.0f ? __builtin_inff() : ninf();
                int2 see = sh.sees[n * 16 + c];
                if (sp.each) see = (r0 + n * 16 + c) / a.heads == ta + query ? int2{INT32_MIN, INT32_MAX} : int2{0, 0};
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const bool mine = ((seen >> y) & 1) && e + y >= see.x && e + y < see.y;
                    odd |= !mine && !(fabsf(s[n][y]) < __builtin_inff());
                    s[n][y] = mine ? s[n][y] : hole;
                }
            }
            // A row that holds NaN codes and that some of the block's queries do not see: for the second product it is
            // zeros (those that see it have a NaN probability). A query's own NaN or infinity looks the same; then
            // nothing is found here.
            if (__any(odd)) {
#pragma unroll 1
                for (int j = 0; j < 16; ++j) {
                    h8* at = reinterpret_cast<h8*>(sh.kv + (w * 16 + j) * kD + lane * 8);
                    const h8 v = *at;
                    bool bad = false;
#pragma unroll
                    for (int y = 0; y < 8; ++y) bad |= !(fabsf((float)v[y]) < __builtin_inff());
                    if (__any(bad)) *at = h8{};
                }
            }
        }
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
        for (int n = 0; n < NH; ++n) over |= probabilities(n, fr[n], i);
        const int any = __any(over);
        sh.over[i & 1][w] = any;
        __syncthreads();
    };
    const auto second_product = [&](int i) {
        const int4 ov = *reinterpret_cast<const int4*>(sh.over[i & 1]);
        if (__builtin_amdgcn_readfirstlane(ov.x | ov.y | ov.z | ov.w)) rebase(i);
#pragma unroll
        for (int n = 0; n < NH; ++n) l[n] += sum[n];
        const _Float16* prob = sh.p[i & 1] + oc * kPRow + og * 8;
        // a transposed read of unit y's eight entries of this lane's value
        const auto rows8 = [&](int y) {
            int lo, hi, at;
            if constexpr (kWide) {
                lo = at_out ^ ((y & 1) * 32), hi = at_out ^ ((y & 1) * 32 + 4 * kD + 8);
                at = (y >> 2) * 16 * kD + ((y >> 1) & 1) * 64;
            } else {
                lo = at_out ^ ((y & 3) * 16), hi = at_out ^ ((y & 3) * 16 + 4 * kD + 8);
                at = (y >> 3) * 32 * kD + ((y >> 2) & 1) * 64;
            }
            const hv4 l4 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(sh.kv + lo + at));
            const hv4 h4 = __builtin_amdgcn_ds_read_tr16_b64_v4f16((lds_hv4*)(sh.kv + hi + at));
            h8 v;
            __builtin_memcpy(&v, &l4, 8);
            __builtin_memcpy((char*)&v + 8, &h4, 8);
            return v;
        };
#pragma unroll
        for (int y = 0; y < 16; ++y) {
            const h8 v = rows8(y);
#pragma unroll
            for (int n = 0; n < kOh; ++n) {
                if constexpr (kWide) {
                    const h8 p = *reinterpret_cast<const h8*>(prob + n * 32 * kPRow + (y >> 2) * 16);
                    o[n][y & 3] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p, o[n][y & 3], 0, 0, 0);
                } else {
                    const h8 p = *reinterpret_cast<const h8*>(prob + (y >> 3) * 32);
                    o[n][y & 7] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, p, o[n][y & 7], 0, 0, 0);
                }
            }
        }
    };

    if (steps > 0) {
        first_product(0, std::true_type{});
        for (int i = 0; i + 1 < steps; ++i) {
            second_product(i);
            __syncthreads();  // before the next step's rows take the place
            first_product(i + 1, std::false_type{});
        }
        second_product(steps - 1);
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
    const bool finish = cut.parts == 1;
    const int pairs = finish && a.turn.freq ? a.turn.rot / 2 : 0;
    const int queries = tb - ta + 1, batch = pairs ? min(queries, (int)(sizeof(sh.p) / sizeof(float2)) / pairs) : queries;
    for (int first_query = 0; first_query < queries; first_query += batch) {
        const int some = min(batch, queries - first_query);
        for (int i = threadIdx.x; i < some * pairs; i += 256)
            cs[i] = angle_of(a, t0 + ta + first_query + i / pairs, i % pairs);
        __syncthreads();
        const int begin = max((ta + first_query) * a.heads - r0, 0);
        const int stop = min((ta + first_query + some) * a.heads - r0, min(kRows, left));
#pragma unroll 2
        for (int hl = begin + ((w - begin) & 3); hl < stop; hl += 4) {
            const v4f lv = *reinterpret_cast<const v4f*>(sh.l[hl]);
            const float L = (lv[0] + lv[1]) + (lv[2] + lv[3]), R = -sh.fr[hl].y;
            float* row = rows + hl * kD;
            const v4f x = *reinterpret_cast<const v4f*>(row + (((2 * lane) ^ (hl & 31)) << 2));
            const v4f y = *reinterpret_cast<const v4f*>(row + (((2 * lane + 1) ^ (hl & 31)) << 2));
            const int64_t pair = pair0 + hl;
            if (!finish) {
                const int64_t at = pair * cut.parts + part;
                *reinterpret_cast<v4f*>(a.part_o + at * kD + 8 * lane) = x;
                *reinterpret_cast<v4f*>(a.part_o + at * kD + 8 * lane + 4) = y;
                if (lane == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * at) = float2{R, L};
                continue;
            }
            uint4 u{};
            if (a.other) u = *reinterpret_cast<const uint4*>(a.other + pair * kD + 8 * lane);
            const Weights wt = join_weights(a, pair, R, L);
            float v[8] = {x[0] * wt.mine, x[1] * wt.mine, x[2] * wt.mine, x[3] * wt.mine,
                          y[0] * wt.mine, y[1] * wt.mine, y[2] * wt.mine, y[3] * wt.mine};
            add_other(u, wt.other, v);
            if (pairs) turn_row(a, cs + ((r0 + hl) / a.heads - ta - first_query) * pairs, row, v);
            store_row(a, pair, v);
            if (a.lse && lane == 0) a.lse[pair] = wt.lse;
        }
        if (first_query + batch < queries) __syncthreads();  // before the next angles
    }
}

// The parts of a row, a wavefront each: o = sum 2^(R_i - R) o_i over sum 2^(R_i - R) l_i, then as above.
__global__ __launch_bounds__(256) void local_join_kernel(const LocalArgs a, int parts) {
    __shared__ __align__(16) float s_o[4][kD];
    __shared__ float2 s_cs[4][kD / 2];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t pair = (int64_t)blockIdx.x * 4 + w;
    if (pair >= (int64_t)a.nq * a.heads) return;  // (no barrier below)
    float2 ml{kNone, 0.0f};
    if (lane < parts) ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * (pair * parts + lane));
    float R = ml.x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) R = fmaxf(R, __shfl_xor(R, d));
    const float f = __builtin_amdgcn_exp2f(ml.x - R);
    float L = f * ml.y;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) L += __shfl_xor(L, d);
    const float* po = a.part_o + pair * parts * kD + 8 * lane;
    v4f x{}, y{};
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float fi = __shfl(f, i);
        x += fi * reinterpret_cast<const v4f*>(po + (int64_t)i * kD)[0];
        y += fi * reinterpret_cast<const v4f*>(po + (int64_t)i * kD)[1];
    }
    uint4 u{};
    if (a.other) u = *reinterpret_cast<const uint4*>(a.other + pair * kD + 8 * lane);
    const Weights wt = join_weights(a, pair, R, L);
    float v[8] = {x[0] * wt.mine, x[1] * wt.mine, x[2] * wt.mine, x[3] * wt.mine,
                  y[0] * wt.mine, y[1] * wt.mine, y[2] * wt.mine, y[3] * wt.mine};
    add_other(u, wt.other, v);
    if (a.turn.freq) {
        for (int i = lane; i < a.turn.rot / 2; i += 64) s_cs[w][i] = angle_of(a, pair / a.heads, i);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        turn_row(a, s_cs[w], s_o[w], v);
    }
    store_row(a, pair, v);
    if (a.lse && lane == 0) a.lse[pair] = wt.lse;
}

// Parts of a run's entries: two blocks for each of the 256 compute units, with two steps each at least.
int64_t parts_for(int64_t blocks, int64_t entries) {
    const int64_t steps = (entries + kTile - 1) / kTile;
    return std::max<int64_t>(1, std::min<int64_t>({(int64_t)kMostParts, 512 / std::max<int64_t>(blocks, 1), steps / 2}));
}
size_t part_bytes(int64_t rows) { return (size_t)rows * (kD + 2) * sizeof(float); }

}  // namespace

size_t local_workspace_bytes(int32_t nq, int32_t heads, int64_t entries) {
    if (nq <= 0 || entries <= 0) return 16;
    const int64_t rows = (int64_t)nq * heads, parts = parts_for((rows + 31) / 32, entries);
    return parts == 1 ? 16 : parts * part_bytes(rows);
}

hipError_t launch_attend_local(LocalArgs a, void* ws, size_t ws_bytes, hipStream_t stream) {
    const int64_t rows = (int64_t)a.nq * a.heads, runs = a.nq / a.group, run_rows = (int64_t)a.group * a.heads;
    int64_t entries = a.places.max_n;
    if (a.window > 0) entries = std::min(entries, a.window + std::min<int64_t>(a.group, 31));
    LocalCut cut;
    cut.nh = run_rows > 16 ? 2 : 1;
    cut.tiles = (uint32_t)((run_rows + 16 * cut.nh - 1) / (16 * cut.nh));
    const int64_t blocks = runs * cut.tiles;
    cut.parts = (uint32_t)std::max<int64_t>(1, std::min<int64_t>(parts_for(blocks, entries), ws_bytes / part_bytes(rows)));
    if (cut.parts > 1) {
        a.part_o = (float*)ws;
        a.part_ml = a.part_o + (size_t)cut.parts * rows * kD;
    }
    const uint32_t units = (uint32_t)(blocks * cut.parts);
    const dim3 grid((units + 7) / 8 * 8);
    if (cut.nh == 2) {
        if (a.places.pages)
            hipLaunchKernelGGL((attend_local_kernel<2, true>), grid, dim3(256), 0, stream, a, cut, units);
        else
            hipLaunchKernelGGL((attend_local_kernel<2, false>), grid, dim3(256), 0, stream, a, cut, units);
    } else {
        if (a.places.pages)
            hipLaunchKernelGGL((attend_local_kernel<1, true>), grid, dim3(256), 0, stream, a, cut, units);
        else
            hipLaunchKernelGGL((attend_local_kernel<1, false>), grid, dim3(256), 0, stream, a, cut, units);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || cut.parts == 1) return err;
    hipLaunchKernelGGL(local_join_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a, (int)cut.parts);
    return hipGetLastError();
}

}  // namespace fp4idx
