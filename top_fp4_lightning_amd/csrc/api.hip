// C-ABI entry points of libfp4idx: host-side validation, then asynchronous launches.
// Every check runs before the first HIP call, so argument errors never touch the device.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <mutex>
#include <string>

#include "../../include/fp4idx.h"
#include "operators.h"
#include "places.h"

using namespace fp4idx;

// ---- scratch of idx_build_pool_noalloc, for callers that cannot allocate ----
// The selection workspace lives in this file-scope device array: one copy on every GPU the
// library runs on, held until the process ends, shared by every call on that GPU (calls that
// overlap on one GPU race). On the host, `scratch` is only a stand-in for the device symbol and is
// never passed to a kernel or a copy: its device address is resolved once per device with
// hipGetSymbolAddress and kept in g_scratch.
constexpr size_t kScratchBytes = (size_t)80 << 20;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

namespace {

thread_local std::string g_last_error;

idx_status fail(idx_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return st;
}

idx_status ok() {
    g_last_error.clear();
    return IDX_OK;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

idx_status hip_status(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(IDX_EHIP, "%s: HIP launch failed: %s", what, hipGetErrorString(e));
    return ok();
}

#define REQUIRE(cond, st, ...)                   \
    do {                                          \
        if (!(cond)) return fail(st, __VA_ARGS__); \
    } while (0)

constexpr int64_t kMaxRows = (int64_t)1 << 36;
constexpr int64_t kMaxN = (int64_t)1 << 30;
constexpr int32_t kMaxQueries = 65535;  // grid y dimension
constexpr int32_t kMaxAttendHeads = 128;
constexpr int32_t kMaxAttendList = 1 << 24;
constexpr int64_t kMaxRopeTokens = (1 << 24) - 1;  // a block of 256 threads for each: below 2^32
constexpr int64_t kMaxPoolScoreN = (int64_t)1 << 28;  // a score row read through a pool: below 2^30 bytes

size_t ws_bytes_for(int32_t op, int32_t nq, int64_t max_n, int32_t k) {
    if (nq < 0 || max_n < 0 || max_n > kMaxN || k < 1 || k > kMaxK) return 0;
    if (op == IDX_OP_ATTEND) return k > kMaxAttendHeads ? 0 : attend_workspace_bytes(nq, k, max_n);
    if (op == IDX_OP_ATTEND_LOCAL) return k > kMaxAttendHeads ? 0 : local_workspace_bytes(nq, k, max_n);
    if (op == IDX_OP_DISTILL) return distill_workspace_bytes(nq, max_n);
    if (op == IDX_OP_BUILD_POOL) return select_workspace_bytes(nq, (max_n + kBlock - 1) / kBlock, k);
    if (op == IDX_OP_TOPK) return select_workspace_bytes(nq, max_n, k);
    return 0;
}


// Validation shared by the two pool entry points; fills the selection arguments (all but the
// workspace).
idx_status pool_args(const char* fn, const float* block_max, int64_t bm_stride, const int32_t* n_vis, int32_t nq,
                     int64_t max_n, int32_t topk_blocks, int32_t block, int32_t* pool_blocks, int64_t pool_stride,
                     int32_t* pool_count, bool pin, SelectArgs& a) {
    REQUIRE(block == kBlock, IDX_EUNSUPPORTED, "%s: block=%d (only 8 is implemented)", fn, block);
    REQUIRE(topk_blocks >= 1 && topk_blocks <= kMaxK, IDX_EUNSUPPORTED, "%s: topk_blocks=%d out of [1, 2048]", fn,
            topk_blocks);
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "%s: nq=%d out of [0, 65535]", fn, nq);
    REQUIRE(max_n >= 0 && max_n <= kMaxN, IDX_EINVAL, "%s: max_n=%lld out of [0, 2^30]", fn, (long long)max_n);
    if (nq == 0) return ok();
    REQUIRE(block_max && n_vis && pool_blocks && pool_count, IDX_EINVAL, "%s: null pointer", fn);
    REQUIRE(bm_stride >= (max_n + kBlock - 1) / kBlock, IDX_EINVAL, "%s: bm_stride < ceil(max_n/8)", fn);
    REQUIRE(pool_stride >= topk_blocks, IDX_EINVAL, "%s: pool_stride=%lld < topk_blocks=%d", fn,
            (long long)pool_stride, topk_blocks);
    REQUIRE(aligned(block_max, 4) && aligned(n_vis, 4) && aligned(pool_blocks, 4) && aligned(pool_count, 4),
            IDX_EALIGN, "%s: misaligned pointer", fn);
    a.vals = block_max;
    a.stride = bm_stride;
    a.nv = n_vis;
    a.nq = nq;
    a.max_n = max_n;
    a.k = topk_blocks;
    a.pool_mode = true;
    a.pin = pin;
    a.out_idx = pool_blocks;
    a.out_stride = pool_stride;
    a.out_count = pool_count;
    a.pad_to = topk_blocks;
    return ok();
}

// Validation shared by the attention entry points; fills the arguments common to them.
idx_status attend_args(const char* fn, const uint16_t* q, int32_t nq, int32_t heads, const uint8_t* codes,
                       const uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                       int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq, const int32_t* n_vis,
                       int64_t max_n, int64_t window, const int32_t* idx, int64_t idx_stride, int32_t k, float scale,
                       AttendArgs& a) {
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "%s: nq=%d out of [0, 65535]", fn, nq);
    REQUIRE(heads >= 1 && heads <= kMaxAttendHeads, IDX_EUNSUPPORTED, "%s: heads=%d out of [1, 128]", fn, heads);
    REQUIRE(max_n >= 0 && max_n <= kMaxN, IDX_EUNSUPPORTED, "%s: max_n=%lld out of [0, 2^30]", fn, (long long)max_n);
    REQUIRE(rows >= 0 && rows <= INT32_MAX, IDX_EUNSUPPORTED, "%s: rows=%lld out of [0, 2^31 - 1]", fn,
            (long long)rows);
    REQUIRE(window >= 0 && !(window && idx), IDX_EINVAL, "%s: window=%lld must be >= 0, and 0 with a list", fn,
            (long long)window);
    REQUIRE(isfinite(scale), IDX_EINVAL, "%s: scale is not finite", fn);
    if (idx) {
        REQUIRE(k >= 0 && k <= kMaxAttendList, IDX_EUNSUPPORTED, "%s: k=%d out of [0, 2^24]", fn, k);
        REQUIRE(idx_stride >= k, IDX_EINVAL, "%s: idx_stride=%lld < k=%d", fn, (long long)idx_stride, k);
    }
    if (nq == 0) return ok();
    REQUIRE(q && n_vis && (rows == 0 || (codes && scales)), IDX_EINVAL, "%s: null pointer", fn);
    REQUIRE((kv_base != nullptr) != (pages != nullptr), IDX_EINVAL, "%s: give either kv_base or pages", fn);
    if (pages) {
        REQUIRE(page_size >= 1, IDX_EINVAL, "%s: page_size=%d must be >= 1", fn, page_size);
        REQUIRE(pages_stride >= (max_n + page_size - 1) / page_size, IDX_EINVAL,
                "%s: pages_stride=%lld < ceil(max_n / page_size)", fn, (long long)pages_stride);
        REQUIRE(nseq >= 1 && (seq || nseq >= nq), IDX_EINVAL,
                "%s: nseq=%d page rows; without seq, query t uses row t of nq=%d", fn, nseq, nq);
    }
    REQUIRE(aligned(q, 16) && aligned(codes, 16) && aligned(scales, 2) && aligned(kv_base, 8) && aligned(pages, 4) &&
                aligned(seq, 4) && aligned(n_vis, 4) && aligned(idx, 4),
            IDX_EALIGN, "%s: misaligned pointer", fn);
    a = AttendArgs{q, nq, heads, codes, scales, rows, kv_base, pages, pages_stride, nseq, page_size, seq, n_vis,
                   max_n, window, idx, idx_stride, idx ? k : 0, scale, nullptr, nullptr, 0, 0, nullptr, nullptr};
    return ok();
}

// Validation shared by the two directions of the distillation
idx_status distill_args(const char* fn, const float* scores, int64_t score_stride, const int32_t* n_vis, int32_t nq,
                        int64_t max_n, const int32_t* t_idx, const float* t_logit, int64_t t_stride, int32_t k,
                        float inv_temp, DistillArgs& a) {
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "%s: nq=%d out of [0, 65535]", fn, nq);
    REQUIRE(max_n >= 0 && max_n <= kMaxN, IDX_EUNSUPPORTED, "%s: max_n=%lld out of [0, 2^30]", fn, (long long)max_n);
    REQUIRE(k >= 0 && k <= kMaxK, IDX_EUNSUPPORTED, "%s: k=%d out of [0, 2048]", fn, k);
    REQUIRE(isfinite(inv_temp) && inv_temp > 0.0f, IDX_EINVAL, "%s: inv_temp must be finite and above 0", fn);
    if (nq == 0) return ok();
    REQUIRE(n_vis && (max_n == 0 || scores) && (k == 0 || (t_idx && t_logit)), IDX_EINVAL, "%s: null pointer", fn);
    REQUIRE(score_stride >= max_n, IDX_EINVAL, "%s: score_stride=%lld < max_n=%lld", fn, (long long)score_stride,
            (long long)max_n);
    REQUIRE(t_stride >= k, IDX_EINVAL, "%s: t_stride=%lld < k=%d", fn, (long long)t_stride, k);
    REQUIRE(aligned(scores, 4) && aligned(n_vis, 4) && aligned(t_idx, 4) && aligned(t_logit, 4), IDX_EALIGN,
            "%s: misaligned pointer", fn);
    a.scores = scores;
    a.score_stride = score_stride;
    a.n_vis = n_vis;
    a.nq = nq;
    a.max_n = max_n;
    a.t_idx = t_idx;
    a.t_logit = t_logit;
    a.t_stride = t_stride;
    a.k = k;
    a.inv_temp = inv_temp;
    return ok();
}

// Validation of where a cache's entries lie (n: how many kv_base and seq name)
idx_status places_args(const char* fn, int64_t rows, const int64_t* kv_base, const int32_t* pages, int64_t pages_stride,
                       int32_t nseq, int32_t page_size, const int32_t* seq, int64_t n, int64_t max_n, int64_t ring,
                       Places& a) {
    REQUIRE(rows >= 0 && rows <= kMaxRows, IDX_EUNSUPPORTED, "%s: rows=%lld out of [0, 2^36]", fn, (long long)rows);
    REQUIRE(max_n >= 0 && max_n <= kMaxN, IDX_EUNSUPPORTED, "%s: max_n=%lld out of [0, 2^30]", fn, (long long)max_n);
    REQUIRE(ring >= 0 && ring <= kMaxN, IDX_EUNSUPPORTED, "%s: ring=%lld out of [0, 2^30]", fn, (long long)ring);
    REQUIRE(!(kv_base && pages), IDX_EINVAL, "%s: give either kv_base or pages", fn);
    if (pages) {
        const int64_t most = ring && ring < max_n ? ring : max_n;
        REQUIRE(page_size >= 1, IDX_EINVAL, "%s: page_size=%d must be >= 1", fn, page_size);
        REQUIRE(pages_stride >= (most + page_size - 1) / page_size, IDX_EINVAL,
                "%s: pages_stride=%lld < ceil(%lld / page_size)", fn, (long long)pages_stride, (long long)most);
        REQUIRE(nseq >= 1 && (seq || nseq >= n), IDX_EINVAL, "%s: nseq=%d page rows; without seq, %lld are used", fn,
                nseq, (long long)n);
    }
    REQUIRE(aligned(kv_base, 8) && aligned(pages, 4) && aligned(seq, 4), IDX_EALIGN, "%s: misaligned pointer", fn);
    a = Places{rows, kv_base, pages, pages_stride, nseq, seq, division_by(pages ? page_size : 0), division_by(ring), max_n};
    return ok();
}

// Validation of a rotation of rows of `dim` values (freq NULL: none)
idx_status turn_args(const char* fn, int32_t dim, const int64_t* pos, const double* freq, int32_t rot, int32_t offset,
                     int32_t layout, double mscale, int32_t inverse, Turn& a) {
    a = Turn{nullptr, nullptr, 0, 0, false, false, 1.0};
    if (!freq) return ok();
    REQUIRE(layout == IDX_ROPE_HALF || layout == IDX_ROPE_INTERLEAVED, IDX_EUNSUPPORTED, "%s: layout=%d", fn, layout);
    REQUIRE(rot >= 2 && rot <= dim && rot % 2 == 0 && offset >= 0 && offset <= dim - rot, IDX_EINVAL,
            "%s: rot=%d must be even, 2 or more, and lie in the row: offset=%d, dim=%d", fn, rot, offset, dim);
    REQUIRE(isfinite(mscale), IDX_EINVAL, "%s: mscale is not finite", fn);
    REQUIRE(aligned(pos, 8) && aligned(freq, 8), IDX_EALIGN, "%s: misaligned pointer", fn);
    a = Turn{pos, freq, rot, offset, layout == IDX_ROPE_HALF, inverse != 0, mscale};
    return ok();
}

// Validation shared by the two calls on rows at places; x: the rows written or read into
idx_status rows_args(const char* fn, int32_t format, const void* x, int32_t dtype, int64_t tokens, int64_t stride,
                     const uint8_t* codes, const uint8_t* scales, const int64_t* at, RowsArgs& a) {
    REQUIRE(format >= IDX_ROWS_MAIN && format <= IDX_ROWS_KEY, IDX_EUNSUPPORTED, "%s: format=%d", fn, format);
    REQUIRE(dtype == IDX_BF16 || dtype == IDX_F32, IDX_EUNSUPPORTED, "%s: dtype=%d", fn, dtype);
    REQUIRE(tokens >= 0 && tokens <= kMaxRopeTokens, IDX_EUNSUPPORTED, "%s: tokens=%lld out of [0, 2^24 - 1]", fn,
            (long long)tokens);
    if (tokens == 0) return ok();
    const size_t size = dtype == IDX_F32 ? 4 : 2;
    REQUIRE(x && at && (a.places.rows == 0 || (codes && scales)), IDX_EINVAL, "%s: null pointer", fn);
    REQUIRE(aligned(x, size) && aligned(codes, format == IDX_ROWS_LOCAL ? 8 : 4) && aligned(at, 8), IDX_EALIGN,
            "%s: misaligned pointer", fn);
    a.format = format;
    a.f32 = dtype == IDX_F32;
    a.wide = aligned(x, 16) && (stride * (int64_t)size) % 16 == 0;
    a.tokens = tokens;
    a.stride = stride;
    a.at = at;
    a.codes = const_cast<uint8_t*>(codes);
    a.scales = const_cast<uint8_t*>(scales);
    return ok();
}
constexpr int32_t row_dim(int32_t format) { return format == IDX_ROWS_KEY ? kDim : 512; }

// idx_write_rows, tokens left out where keep is below 0 (null: none)
idx_status write_rows(const char* fn, int32_t format, const void* x, int32_t dtype, int64_t tokens, int64_t x_stride,
                      int32_t norm, const float* gamma, double eps, const int64_t* pos, const double* freq, int32_t rot,
                      int32_t offset, int32_t layout, double mscale, const int8_t* signs, uint8_t* codes, uint8_t* scales,
                      int64_t rows, const int64_t* kv_base, const int32_t* pages, int64_t pages_stride, int32_t nseq,
                      int32_t page_size, const int32_t* seq, const int64_t* at, int64_t max_n, int64_t ring,
                      const int64_t* keep, void* stream) {
    RowsArgs a{};
    idx_status st = places_args(fn, rows, kv_base, pages, pages_stride, nseq, page_size, seq, tokens, max_n, ring, a.places);
    if (st == IDX_OK) st = rows_args(fn, format, x, dtype, tokens, x_stride, codes, scales, at, a);
    if (st == IDX_OK) st = turn_args(fn, row_dim(format), pos, freq, rot, offset, layout, mscale, 0, a.turn);
    if (st != IDX_OK) return st;
    REQUIRE(!norm || (isfinite(eps) && eps > 0.0), IDX_EINVAL, "%s: eps must be finite and above 0", fn);
    REQUIRE(x_stride >= 0, IDX_EINVAL, "%s: x_stride=%lld is negative", fn, (long long)x_stride);
    if (tokens == 0 || rows == 0) return ok();
    REQUIRE(format != IDX_ROWS_KEY || signs, IDX_EINVAL, "%s: keys need signs", fn);
    REQUIRE(aligned(codes, 16) && aligned(gamma, 4) && aligned(keep, 8) && (format != IDX_ROWS_KEY || aligned(signs, 16)),
            IDX_EALIGN, "%s: codes and signs must be 16-byte aligned, keep 8-byte, gamma 4-byte", fn);
    a.x = x;
    a.norm = norm != 0;
    a.gamma = gamma;
    a.eps = eps;
    a.signs = signs;
    a.keep = keep;
    return hip_status(launch_write_rows(a, (hipStream_t)stream), fn);
}

// idx_attend_local, run i's sequence seq_stride numbers behind the one before
idx_status attend_local(const char* fn, const uint16_t* q, int32_t nq, int32_t heads, int32_t group, const uint8_t* codes,
                        const uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                        int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq, int64_t seq_stride,
                        const int32_t* n_vis, int64_t max_n, int64_t window, int64_t ring, float scale,
                        const uint16_t* other, const float* other_lse, const int64_t* pos, const double* freq,
                        int32_t rot, int32_t offset, int32_t layout, double mscale, uint16_t* out, float* lse,
                        void* ws, size_t ws_bytes, void* stream) {
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "%s: nq=%d out of [0, 65535]", fn, nq);
    REQUIRE(heads >= 1 && heads <= kMaxAttendHeads, IDX_EUNSUPPORTED, "%s: heads=%d out of [1, 128]", fn, heads);
    REQUIRE(group >= 1 && nq % group == 0, IDX_EINVAL, "%s: group=%d must divide nq=%d", fn, group, nq);
    LocalArgs a{};
    idx_status st = places_args(fn, rows, kv_base, pages, pages_stride, nseq, page_size, seq, nq / group, max_n, ring,
                                a.places);
    if (st == IDX_OK) st = turn_args(fn, row_dim(IDX_ROWS_LOCAL), pos, freq, rot, offset, layout, mscale, 1, a.turn);
    if (st != IDX_OK) return st;
    REQUIRE(rows <= INT32_MAX, IDX_EUNSUPPORTED, "%s: rows=%lld out of [0, 2^31 - 1]", fn, (long long)rows);
    REQUIRE(window >= 0, IDX_EINVAL, "%s: window=%lld is negative", fn, (long long)window);
    REQUIRE(!ring || (window >= 1 && window <= ring - (group - 1)), IDX_EINVAL,
            "%s: ring=%lld must hold window=%lld + group - 1=%d entries", fn, (long long)ring, (long long)window, group - 1);
    REQUIRE(isfinite(scale), IDX_EINVAL, "%s: scale is not finite", fn);
    REQUIRE(seq_stride >= 0, IDX_EINVAL, "%s: seq_stride=%lld is negative", fn, (long long)seq_stride);
    REQUIRE((other != nullptr) == (other_lse != nullptr), IDX_EINVAL, "%s: other and other_lse go together", fn);
    if (nq == 0) return ok();
    REQUIRE(q && n_vis && out && (rows == 0 || (codes && scales)) && (!freq || pos), IDX_EINVAL, "%s: null pointer", fn);
    REQUIRE(kv_base || pages, IDX_EINVAL, "%s: give either kv_base or pages", fn);
    REQUIRE(ws && ws_bytes >= 16, IDX_EWORKSPACE, "%s: workspace %zu bytes, need at least 16", fn, ws_bytes);
    REQUIRE(aligned(q, 16) && aligned(codes, 16) && aligned(scales, 4) && aligned(n_vis, 4) && aligned(other, 16) &&
                aligned(other_lse, 4) && aligned(out, 16) && aligned(lse, 4) && aligned(ws, 16),
            IDX_EALIGN, "%s: misaligned pointer", fn);
    a.q = q;
    a.nq = nq;
    a.heads = heads;
    a.group = group;
    a.codes = codes;
    a.scales = scales;
    a.seq_stride = seq_stride;
    a.n_vis = n_vis;
    a.window = window < kMaxN ? window : kMaxN;  // (no range is longer, and the kernel's sums with it fit)
    a.scale = scale;
    a.other = other;
    a.other_lse = other_lse;
    a.out = out;
    a.lse = lse;
    return hip_status(launch_attend_local(a, ws, ws_bytes, (hipStream_t)stream), fn);
}

constexpr int kMaxDevices = 64;
struct DeviceScratch {
    void* ptr;             // device address of this device's `scratch`
    int32_t rows_cleared;  // per-row counters [0, rows_cleared) known to be zero
};
std::mutex g_scratch_mu;
DeviceScratch g_scratch[kMaxDevices];

__global__ void clear_bytes_kernel(uint8_t* p, size_t bytes) {
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < bytes; i += (size_t)gridDim.x * blockDim.x)
        p[i] = 0;
}

// This device's scratch address; on first use and whenever a call needs the counters of more rows
// than any call before it, those counters are cleared on `stream` (a fill kernel, no memset) before
// the call's own kernels. Every selection call restores the counters it uses to zero.
idx_status device_scratch(int32_t nq, hipStream_t stream, void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(IDX_EHIP, "idx_build_pool_noalloc: hipGetDevice: %s", hipGetErrorString(e));
    REQUIRE(dev >= 0 && dev < kMaxDevices, IDX_EUNSUPPORTED, "idx_build_pool_noalloc: device %d above %d", dev,
            kMaxDevices - 1);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    DeviceScratch& ds = g_scratch[dev];
    if (!ds.ptr) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p)
            return fail(IDX_EHIP, "idx_build_pool_noalloc: hipGetSymbolAddress(scratch): %s", hipGetErrorString(e));
        ds.ptr = p;
        ds.rows_cleared = 0;
    }
    if (nq > ds.rows_cleared) {
        const size_t from = select_counter_bytes(ds.rows_cleared), to = select_counter_bytes(nq);
        const size_t bytes = to - from;
        const unsigned blocks = (unsigned)((bytes + 255) / 256 < 1024 ? (bytes + 255) / 256 : 1024);
        hipLaunchKernelGGL(clear_bytes_kernel, dim3(blocks), dim3(256), 0, stream, (uint8_t*)ds.ptr + from, bytes);
        e = hipGetLastError();
        if (e != hipSuccess) return fail(IDX_EHIP, "idx_build_pool_noalloc: clear: %s", hipGetErrorString(e));
        ds.rows_cleared = nq;
    }
    *out = ds.ptr;
    return ok();
}

}  // namespace

extern "C" {

int32_t idx_abi_version(void) { return IDX_ABI_VERSION; }

const char* idx_last_error(void) { return g_last_error.c_str(); }

size_t idx_workspace_size(int32_t op, int32_t nq, int64_t max_n, int32_t k) {
    return ws_bytes_for(op, nq, max_n, k);
}

idx_status idx_quantize_q(const uint16_t* x_bf16, int64_t rows, const int8_t* signs, uint8_t* codes,
                          uint8_t* scales, void* stream) {
    REQUIRE(rows >= 0 && rows <= kMaxRows, IDX_EINVAL, "idx_quantize_q: rows=%lld out of [0, 2^36]", (long long)rows);
    if (rows == 0) return ok();
    REQUIRE(x_bf16 && signs && codes && scales, IDX_EINVAL, "idx_quantize_q: null pointer");
    REQUIRE(aligned(x_bf16, 16) && aligned(codes, 16) && aligned(signs, 16) && aligned(scales, 4), IDX_EALIGN,
            "idx_quantize_q: x, codes and signs must be 16-byte aligned, scales 4-byte aligned");
    return hip_status(launch_quantize(x_bf16, rows, signs, codes, scales, (hipStream_t)stream), "idx_quantize_q");
}

idx_status idx_score_full(const uint8_t* k_codes, const uint8_t* k_scales, const int64_t* k_base,
                          const int32_t* n_vis, int32_t nq, int32_t group, int64_t max_n, const uint8_t* q_codes,
                          const uint8_t* q_scales, const float* w, float* scores, int64_t score_stride,
                          float* block_max, int64_t bm_stride, float* head_dots, void* stream) {
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "idx_score_full: nq=%d out of [0, 65535]", nq);
    REQUIRE(max_n >= 0 && max_n <= kMaxScanKeys, IDX_EUNSUPPORTED, "idx_score_full: max_n=%lld out of [0, 2^24]",
            (long long)max_n);
    REQUIRE(group >= 1 && (nq == 0 || nq % group == 0), IDX_EINVAL, "idx_score_full: group=%d must divide nq=%d",
            group, nq);
    REQUIRE(scores || block_max || head_dots, IDX_EINVAL, "idx_score_full: no output requested");
    if (nq == 0 || max_n == 0) return ok();
    REQUIRE(k_codes && k_scales && k_base && n_vis && q_codes && q_scales && w, IDX_EINVAL,
            "idx_score_full: null input pointer");
    REQUIRE(aligned(k_codes, 16) && aligned(q_codes, 16) && aligned(k_scales, 4) && aligned(q_scales, 4) &&
                aligned(w, 4) && aligned(k_base, 8) && aligned(n_vis, 4),
            IDX_EALIGN, "idx_score_full: misaligned input pointer");
    if (scores || head_dots)
        REQUIRE(score_stride >= max_n, IDX_EINVAL, "idx_score_full: score_stride=%lld < max_n=%lld",
                (long long)score_stride, (long long)max_n);
    if (block_max)
        REQUIRE(bm_stride >= (max_n + kBlock - 1) / kBlock, IDX_EINVAL,
                "idx_score_full: bm_stride=%lld < ceil(max_n/8)", (long long)bm_stride);
    REQUIRE((!scores || aligned(scores, 4)) && (!block_max || aligned(block_max, 4)) &&
                (!head_dots || aligned(head_dots, 4)),
            IDX_EALIGN, "idx_score_full: misaligned output pointer");
    ScoreArgs a{k_codes, k_scales, k_base, n_vis, nq, group, max_n, q_codes, q_scales, w,
                scores, score_stride, block_max, bm_stride, head_dots};
    return hip_status(launch_score_full(a, (hipStream_t)stream), "idx_score_full");
}

idx_status idx_build_pool(const float* block_max, int64_t bm_stride, const int32_t* n_vis, int32_t nq,
                          int64_t max_n, int32_t topk_blocks, int32_t block, int32_t* pool_blocks,
                          int64_t pool_stride, int32_t* pool_count, void* ws, size_t ws_bytes, void* stream) {
    SelectArgs a{};
    const idx_status st = pool_args("idx_build_pool", block_max, bm_stride, n_vis, nq, max_n, topk_blocks, block,
                                    pool_blocks, pool_stride, pool_count, true, a);
    if (st != IDX_OK || nq == 0) return st;
    const size_t need = ws_bytes_for(IDX_OP_BUILD_POOL, nq, max_n, topk_blocks);
    REQUIRE(ws && ws_bytes >= need, IDX_EWORKSPACE, "idx_build_pool: workspace %zu bytes, need %zu", ws_bytes, need);
    REQUIRE(aligned(ws, 16), IDX_EALIGN, "idx_build_pool: misaligned workspace");
    a.ws = ws;
    return hip_status(launch_select(a, (hipStream_t)stream), "idx_build_pool");
}

idx_status idx_build_pool_noalloc(const float* block_max, int64_t bm_stride, const int32_t* n_vis, int32_t nq,
                                  int64_t max_n, int32_t topk_blocks, int32_t block, int32_t* pool_blocks,
                                  int64_t pool_stride, int32_t* pool_count, void* stream) {
    SelectArgs a{};
    const idx_status st = pool_args("idx_build_pool_noalloc", block_max, bm_stride, n_vis, nq, max_n, topk_blocks,
                                    block, pool_blocks, pool_stride, pool_count, true, a);
    if (st != IDX_OK || nq == 0) return st;
    const size_t need = ws_bytes_for(IDX_OP_BUILD_POOL, nq, max_n, topk_blocks);
    REQUIRE(need <= kScratchBytes, IDX_EUNSUPPORTED,
            "idx_build_pool_noalloc: nq=%d rows of max_n=%lld positions need %zu bytes of scratch, above the "
            "library's fixed %zu",
            nq, (long long)max_n, need, kScratchBytes);
    void* ptr = nullptr;
    const idx_status sst = device_scratch(nq, (hipStream_t)stream, &ptr);
    if (sst != IDX_OK) return sst;
    a.ws = ptr;
    return hip_status(launch_select(a, (hipStream_t)stream), "idx_build_pool_noalloc");
}

idx_status idx_top_blocks(const float* block_max, int64_t bm_stride, const int32_t* n_vis, int32_t nq, int64_t max_n,
                          int32_t k, int32_t block, int32_t* blocks, int64_t blocks_stride, int32_t* count, void* ws,
                          size_t ws_bytes, void* stream) {
    SelectArgs a{};
    const idx_status st = pool_args("idx_top_blocks", block_max, bm_stride, n_vis, nq, max_n, k, block, blocks,
                                    blocks_stride, count, false, a);
    if (st != IDX_OK || nq == 0) return st;
    const size_t need = ws_bytes_for(IDX_OP_BUILD_POOL, nq, max_n, k);
    REQUIRE(ws && ws_bytes >= need, IDX_EWORKSPACE, "idx_top_blocks: workspace %zu bytes, need %zu", ws_bytes, need);
    REQUIRE(aligned(ws, 16), IDX_EALIGN, "idx_top_blocks: misaligned workspace");
    a.ws = ws;
    return hip_status(launch_select(a, (hipStream_t)stream), "idx_top_blocks");
}

idx_status idx_score_pool_gather(const uint8_t* k_codes, const uint8_t* k_scales, const int64_t* k_base,
                                 const int32_t* n_vis, int32_t nq, const int32_t* blocks, int64_t blocks_stride,
                                 const int32_t* block_count, int32_t max_blocks, int32_t block,
                                 const uint8_t* q_codes, const uint8_t* q_scales, const float* w, float* scores,
                                 int64_t score_stride, float* head_dots, void* stream) {
    REQUIRE(block == kBlock, IDX_EUNSUPPORTED, "idx_score_pool_gather: block=%d (only 8 is implemented)", block);
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "idx_score_pool_gather: nq=%d out of [0, 65535]", nq);
    REQUIRE(max_blocks >= 0 && max_blocks <= (1 << 20), IDX_EINVAL,
            "idx_score_pool_gather: max_blocks=%d out of [0, 2^20]", max_blocks);
    if (nq == 0 || max_blocks == 0) return ok();
    REQUIRE(k_codes && k_scales && k_base && n_vis && blocks && block_count && q_codes && q_scales && w && scores,
            IDX_EINVAL, "idx_score_pool_gather: null pointer");
    REQUIRE(blocks_stride >= max_blocks, IDX_EINVAL, "idx_score_pool_gather: blocks_stride < max_blocks");
    REQUIRE(score_stride >= (int64_t)max_blocks * kBlock, IDX_EINVAL,
            "idx_score_pool_gather: score_stride < 8 * max_blocks");
    REQUIRE(aligned(k_codes, 16) && aligned(q_codes, 16) && aligned(k_scales, 4) && aligned(q_scales, 4) &&
                aligned(w, 4) && aligned(k_base, 8) && aligned(n_vis, 4) && aligned(blocks, 4) &&
                aligned(block_count, 4) && aligned(scores, 4) && (!head_dots || aligned(head_dots, 4)),
            IDX_EALIGN, "idx_score_pool_gather: misaligned pointer");
    GatherArgs a{k_codes, k_scales, k_base, n_vis, nq, blocks, blocks_stride, block_count, max_blocks,
                 q_codes, q_scales, w, scores, score_stride, head_dots};
    return hip_status(launch_score_gather(a, (hipStream_t)stream), "idx_score_pool_gather");
}

idx_status idx_topk(const float* scores, int64_t score_stride, const int32_t* n_valid, int32_t nq, int64_t max_n,
                    int32_t k, const int32_t* blocks, int64_t blocks_stride, int32_t block, int32_t* out_idx,
                    int64_t out_stride, float* out_val, void* ws, size_t ws_bytes, void* stream) {
    REQUIRE(k >= 1 && k <= kMaxK, IDX_EUNSUPPORTED, "idx_topk: k=%d out of [1, 2048]", k);
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "idx_topk: nq=%d out of [0, 65535]", nq);
    REQUIRE(max_n >= 0 && max_n <= kMaxN, IDX_EINVAL, "idx_topk: max_n=%lld out of [0, 2^30]", (long long)max_n);
    if (blocks) REQUIRE(block == kBlock, IDX_EUNSUPPORTED, "idx_topk: block=%d (only 8 is implemented)", block);
    if (nq == 0) return ok();
    REQUIRE(scores && out_idx, IDX_EINVAL, "idx_topk: null pointer");
    REQUIRE(score_stride >= max_n, IDX_EINVAL, "idx_topk: score_stride < max_n");
    REQUIRE(out_stride >= k, IDX_EINVAL, "idx_topk: out_stride < k");
    if (blocks)
        REQUIRE(blocks_stride >= (max_n + kBlock - 1) / kBlock, IDX_EINVAL, "idx_topk: blocks_stride < ceil(max_n/8)");
    const size_t need = ws_bytes_for(IDX_OP_TOPK, nq, max_n, k);
    REQUIRE(ws && ws_bytes >= need, IDX_EWORKSPACE, "idx_topk: workspace %zu bytes, need %zu", ws_bytes, need);
    REQUIRE(aligned(ws, 16) && aligned(scores, 4) && aligned(out_idx, 4) && (!out_val || aligned(out_val, 4)) &&
                (!n_valid || aligned(n_valid, 4)) && (!blocks || aligned(blocks, 4)),
            IDX_EALIGN, "idx_topk: misaligned pointer");
    SelectArgs a{};
    a.vals = scores;
    a.stride = score_stride;
    a.nv = n_valid;
    a.nq = nq;
    a.max_n = max_n;
    a.k = k;
    a.pool_mode = false;
    a.map = blocks;
    a.map_stride = blocks_stride;
    a.out_idx = out_idx;
    a.out_stride = out_stride;
    a.out_val = out_val;
    a.out_count = nullptr;
    a.pad_to = k;
    a.ws = ws;
    return hip_status(launch_select(a, (hipStream_t)stream), "idx_topk");
}

idx_status idx_topk_pool(const float* scores, int64_t score_stride, const int32_t* n_vis, int32_t nq, int64_t max_n,
                         const int32_t* pool_blocks, int64_t pool_stride, const int32_t* pool_count,
                         int32_t max_blocks, int32_t group, int32_t block, int32_t k, int32_t* out_idx,
                         int64_t out_stride, float* out_val, void* stream) {
    REQUIRE(k >= 1 && k <= kMaxK, IDX_EUNSUPPORTED, "idx_topk_pool: k=%d out of [1, 2048]", k);
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "idx_topk_pool: nq=%d out of [0, 65535]", nq);
    REQUIRE(max_n >= 0 && max_n <= kMaxPoolScoreN, IDX_EUNSUPPORTED, "idx_topk_pool: max_n=%lld out of [0, 2^28]",
            (long long)max_n);
    REQUIRE(block == kBlock, IDX_EUNSUPPORTED, "idx_topk_pool: block=%d (only 8 is implemented)", block);
    REQUIRE(max_blocks >= 0 && max_blocks <= kMaxK, IDX_EUNSUPPORTED, "idx_topk_pool: max_blocks=%d out of [0, 2048]",
            max_blocks);
    REQUIRE(group >= 1 && (nq == 0 || nq % group == 0), IDX_EINVAL, "idx_topk_pool: group=%d must divide nq=%d",
            group, nq);
    if (nq == 0) return ok();
    REQUIRE(scores && n_vis && pool_blocks && pool_count && out_idx, IDX_EINVAL, "idx_topk_pool: null pointer");
    REQUIRE(score_stride >= max_n, IDX_EINVAL, "idx_topk_pool: score_stride=%lld < max_n=%lld",
            (long long)score_stride, (long long)max_n);
    REQUIRE(pool_stride >= max_blocks, IDX_EINVAL, "idx_topk_pool: pool_stride=%lld < max_blocks=%d",
            (long long)pool_stride, max_blocks);
    REQUIRE(out_stride >= k, IDX_EINVAL, "idx_topk_pool: out_stride < k");
    REQUIRE(aligned(scores, 4) && aligned(n_vis, 4) && aligned(pool_blocks, 4) && aligned(pool_count, 4) &&
                aligned(out_idx, 4) && (!out_val || aligned(out_val, 4)),
            IDX_EALIGN, "idx_topk_pool: pointers must be 4-byte aligned");
    SelectArgs a{};
    a.vals = scores;
    a.stride = score_stride;
    a.nv = n_vis;
    a.nq = nq;
    a.max_n = max_n;
    a.k = k;
    a.pool_mode = false;
    a.map = pool_blocks;
    a.map_stride = pool_stride;
    a.map_values = true;
    a.map_count = pool_count;
    a.map_group = group;
    a.map_width = max_blocks;
    a.out_idx = out_idx;
    a.out_stride = out_stride;
    a.out_val = out_val;
    a.out_count = nullptr;
    a.pad_to = k;
    a.ws = nullptr;
    return hip_status(launch_select(a, (hipStream_t)stream), "idx_topk_pool");
}

idx_status idx_quantize_kv(const uint16_t* x_bf16, int64_t rows, uint8_t* codes, uint8_t* scales, void* stream) {
    REQUIRE(rows >= 0 && rows <= (int64_t)1 << 31, IDX_EINVAL, "idx_quantize_kv: rows=%lld out of [0, 2^31]",
            (long long)rows);
    if (rows == 0) return ok();
    REQUIRE(x_bf16 && codes && scales, IDX_EINVAL, "idx_quantize_kv: null pointer");
    REQUIRE(aligned(x_bf16, 16) && aligned(codes, 4) && aligned(scales, 1), IDX_EALIGN,
            "idx_quantize_kv: x must be 16-byte aligned, codes 4-byte aligned");
    return hip_status(launch_quantize_kv(x_bf16, rows, codes, scales, (hipStream_t)stream), "idx_quantize_kv");
}

idx_status idx_gather_kv(const uint8_t* codes, const uint8_t* scales, const int64_t* kv_base, const int32_t* n_vis,
                         int32_t nq, const int32_t* idx, int64_t idx_stride, int32_t k, uint16_t* out,
                         void* stream) {
    REQUIRE(nq >= 0 && k >= 0, IDX_EINVAL, "idx_gather_kv: nq=%d, k=%d must be >= 0", nq, k);
    REQUIRE(nq <= kMaxQueries, IDX_EUNSUPPORTED, "idx_gather_kv: nq=%d above 65535", nq);
    REQUIRE((int64_t)nq * k <= (int64_t)1 << 31, IDX_EUNSUPPORTED, "idx_gather_kv: nq * k above 2^31");
    if (nq == 0 || k == 0) return ok();
    REQUIRE(codes && scales && kv_base && n_vis && idx && out, IDX_EINVAL, "idx_gather_kv: null pointer");
    REQUIRE(idx_stride >= k, IDX_EINVAL, "idx_gather_kv: idx_stride=%lld < k=%d", (long long)idx_stride, k);
    REQUIRE(aligned(codes, 4) && aligned(kv_base, 8) && aligned(n_vis, 4) && aligned(idx, 4) && aligned(out, 16),
            IDX_EALIGN, "idx_gather_kv: codes, n_vis and idx must be 4-byte, kv_base 8-byte, out 16-byte aligned");
    return hip_status(launch_gather_kv(codes, scales, kv_base, n_vis, nq, idx, idx_stride, k, out, (hipStream_t)stream),
                      "idx_gather_kv");
}

idx_status idx_mask_pool(float* scores, int64_t score_stride, const int32_t* n_vis, int32_t nq, int64_t max_n,
                         const int32_t* pool_blocks, int64_t pool_stride, const int32_t* pool_count, int32_t group,
                         int32_t block, void* stream) {
    REQUIRE(nq >= 0 && nq <= kMaxQueries, IDX_EUNSUPPORTED, "idx_mask_pool: nq=%d out of [0, 65535]", nq);
    REQUIRE(max_n >= 0 && max_n <= kMaxN, IDX_EUNSUPPORTED, "idx_mask_pool: max_n=%lld out of [0, 2^30]",
            (long long)max_n);
    REQUIRE(block == kBlock, IDX_EUNSUPPORTED, "idx_mask_pool: block=%d (only %d)", block, kBlock);
    REQUIRE(group >= 1 && (nq == 0 || nq % group == 0), IDX_EINVAL, "idx_mask_pool: group=%d must divide nq=%d",
            group, nq);
    if (nq == 0 || max_n == 0) return ok();
    REQUIRE(scores && n_vis && pool_blocks && pool_count, IDX_EINVAL, "idx_mask_pool: null pointer");
    REQUIRE(score_stride >= max_n, IDX_EINVAL, "idx_mask_pool: score_stride=%lld < max_n", (long long)score_stride);
    REQUIRE(pool_stride >= 0, IDX_EINVAL, "idx_mask_pool: negative pool_stride");
    REQUIRE(aligned(scores, 4) && aligned(n_vis, 4) && aligned(pool_blocks, 4) && aligned(pool_count, 4), IDX_EALIGN,
            "idx_mask_pool: pointers must be 4-byte aligned");
    return hip_status(launch_mask_pool(scores, score_stride, n_vis, nq, max_n, pool_blocks, pool_stride, pool_count,
                                       group, (hipStream_t)stream),
                      "idx_mask_pool");
}

idx_status idx_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, double original, double fast,
                          double slow, double* freq, float* mscale) {
    REQUIRE(rot >= 2 && rot <= IDX_MAX_ROT && rot % 2 == 0, IDX_EINVAL,
            "idx_rope_freqs: rot=%d must be even, 2 .. 8192", rot);
    REQUIRE(freq && mscale, IDX_EINVAL, "idx_rope_freqs: null pointer");
    REQUIRE(isfinite(base) && base > 1.0, IDX_EINVAL, "idx_rope_freqs: base must be finite and above 1");
    REQUIRE(scaling >= IDX_ROPE_PLAIN && scaling <= IDX_ROPE_YARN, IDX_EUNSUPPORTED, "idx_rope_freqs: scaling=%d",
            scaling);
    REQUIRE(scaling == IDX_ROPE_PLAIN || (isfinite(factor) && factor >= 1.0), IDX_EINVAL,
            "idx_rope_freqs: factor must be finite and at least 1");
    REQUIRE(scaling != IDX_ROPE_NTK || rot > 2, IDX_EINVAL, "idx_rope_freqs: the changed base needs rot > 2");
    REQUIRE(scaling != IDX_ROPE_YARN || (isfinite(original) && original > 0.0 && isfinite(fast) && isfinite(slow) &&
                                         fast > slow),
            IDX_EINVAL, "idx_rope_freqs: needs original > 0 and fast > slow");
    if (scaling == IDX_ROPE_NTK) base *= pow(factor, (double)rot / (rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * i / rot);
        if (scaling == IDX_ROPE_LINEAR) f /= factor;
        if (scaling == IDX_ROPE_YARN) {
            const double turns = original * f / (2.0 * M_PI);
            const double keep = fmin(fmax((turns - slow) / (fast - slow), 0.0), 1.0);
            f = f * keep + f / factor * (1.0 - keep);
        }
        freq[i] = f;
    }
    *mscale = scaling == IDX_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
    return ok();
}

idx_status idx_rope(const void* x, int32_t dtype, int64_t tokens, int32_t heads, int32_t dim, int64_t x_token,
                    int64_t x_head, const int64_t* pos, const double* freq, int32_t rot, int32_t offset,
                    int32_t layout, float mscale, int32_t inverse, void* out, int64_t out_token, int64_t out_head,
                    void* stream) {
    REQUIRE(dtype == IDX_BF16 || dtype == IDX_F32, IDX_EUNSUPPORTED, "idx_rope: dtype=%d", dtype);
    REQUIRE(layout == IDX_ROPE_HALF || layout == IDX_ROPE_INTERLEAVED, IDX_EUNSUPPORTED, "idx_rope: layout=%d",
            layout);
    REQUIRE(tokens >= 0 && tokens <= kMaxRopeTokens, IDX_EUNSUPPORTED, "idx_rope: tokens=%lld out of [0, 2^24 - 1]",
            (long long)tokens);
    REQUIRE(heads >= 1 && heads <= 65535, IDX_EUNSUPPORTED, "idx_rope: heads=%d out of [1, 65535]", heads);
    REQUIRE(dim >= 2 && dim <= (1 << 20), IDX_EUNSUPPORTED, "idx_rope: dim=%d out of [2, 2^20]", dim);
    REQUIRE(rot >= 2 && rot <= IDX_MAX_ROT && rot % 2 == 0 && offset >= 0 && offset <= dim - rot, IDX_EINVAL,
            "idx_rope: rot=%d must be even, 2 .. 8192, and lie in the row: offset=%d, dim=%d", rot, offset, dim);
    REQUIRE(isfinite(mscale), IDX_EINVAL, "idx_rope: mscale is not finite");
    if (tokens == 0) return ok();
    REQUIRE(x && pos && freq && out, IDX_EINVAL, "idx_rope: null pointer");
    REQUIRE(x_token >= 0 && x_head >= 0, IDX_EINVAL, "idx_rope: strides must be >= 0");
    // rows dim apart, and one axis of out inside a step of the other
    REQUIRE((tokens == 1 || out_token >= dim) && (heads == 1 || out_head >= dim) &&
                (tokens == 1 || heads == 1 || (out_token - dim) / (heads - 1) >= out_head ||
                 (out_head - dim) / (tokens - 1) >= out_token),
            IDX_EINVAL, "idx_rope: rows of out overlap: strides %lld and %lld", (long long)out_token,
            (long long)out_head);
    REQUIRE(out != x || ((tokens == 1 || x_token == out_token) && (heads == 1 || x_head == out_head)), IDX_EINVAL,
            "idx_rope: in place, the strides must agree");
    const size_t size = dtype == IDX_BF16 ? 2 : 4;
    REQUIRE(aligned(x, size) && aligned(out, size) && aligned(pos, 8) && aligned(freq, 8), IDX_EALIGN,
            "idx_rope: misaligned pointer");
    const RopeArgs a{x, dtype == IDX_F32, tokens, heads, dim, x_token, x_head, pos, freq, rot, offset,
                     layout == IDX_ROPE_HALF, inverse != 0, mscale, out, out_token, out_head};
    return hip_status(launch_rope(a, (hipStream_t)stream), "idx_rope");
}

idx_status idx_attend(const uint16_t* q, int32_t nq, int32_t heads, const uint8_t* codes, const uint8_t* scales,
                      int64_t rows, const int64_t* kv_base, const int32_t* pages, int64_t pages_stride, int32_t nseq,
                      int32_t page_size, const int32_t* seq, const int32_t* n_vis, int64_t max_n, int64_t window,
                      const int32_t* idx, int64_t idx_stride, int32_t k, float scale, uint16_t* out, float* lse,
                      void* ws, size_t ws_bytes, void* stream) {
    AttendArgs a{};
    const idx_status st = attend_args("idx_attend", q, nq, heads, codes, scales, rows, kv_base, pages, pages_stride,
                                      nseq, page_size, seq, n_vis, max_n, window, idx, idx_stride, k, scale, a);
    if (st != IDX_OK || nq == 0) return st;
    REQUIRE(out, IDX_EINVAL, "idx_attend: null pointer");
    REQUIRE(aligned(out, 16) && aligned(lse, 4), IDX_EALIGN, "idx_attend: misaligned pointer");
    REQUIRE(ws && ws_bytes >= 16, IDX_EWORKSPACE, "idx_attend: workspace %zu bytes, need at least 16", ws_bytes);
    REQUIRE(aligned(ws, 16), IDX_EALIGN, "idx_attend: misaligned workspace");
    a.out = out;
    a.lse = lse;
    return hip_status(launch_attend(a, ws, ws_bytes, (hipStream_t)stream), "idx_attend");
}

idx_status idx_attend_weights(const uint16_t* q, int32_t nq, int32_t heads, const uint8_t* codes,
                              const uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                              int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq,
                              const int32_t* n_vis, int64_t max_n, const int32_t* idx, int64_t idx_stride, int32_t k,
                              float scale, const float* lse, float* weights, int64_t w_stride, void* stream) {
    AttendArgs a{};
    const idx_status st = attend_args("idx_attend_weights", q, nq, heads, codes, scales, rows, kv_base, pages,
                                      pages_stride, nseq, page_size, seq, n_vis, max_n, 0, idx, idx_stride, k, scale, a);
    if (st != IDX_OK || nq == 0) return st;
    const int64_t width = idx ? k : max_n;
    if (width == 0) return ok();
    REQUIRE(lse && weights, IDX_EINVAL, "idx_attend_weights: null pointer");
    REQUIRE(w_stride >= width, IDX_EINVAL, "idx_attend_weights: w_stride=%lld < %lld", (long long)w_stride,
            (long long)width);
    REQUIRE(aligned(lse, 4) && aligned(weights, 4), IDX_EALIGN, "idx_attend_weights: misaligned pointer");
    return hip_status(launch_attend_weights(a, lse, weights, w_stride, (hipStream_t)stream), "idx_attend_weights");
}

idx_status idx_distill(const float* scores, int64_t score_stride, const int32_t* n_vis, int32_t nq, int64_t max_n,
                       const int32_t* t_idx, const float* t_logit, int64_t t_stride, int32_t k, float inv_temp,
                       float* loss, float* lse, float* t_lse, void* ws, size_t ws_bytes, void* stream) {
    DistillArgs a{};
    const idx_status st = distill_args("idx_distill", scores, score_stride, n_vis, nq, max_n, t_idx, t_logit, t_stride,
                                       k, inv_temp, a);
    if (st != IDX_OK || nq == 0) return st;
    REQUIRE(loss && lse && t_lse, IDX_EINVAL, "idx_distill: null pointer");
    REQUIRE(aligned(loss, 4) && aligned(lse, 4) && aligned(t_lse, 4), IDX_EALIGN, "idx_distill: misaligned pointer");
    const size_t need = distill_workspace_bytes(nq, max_n);
    REQUIRE(ws && ws_bytes >= need, IDX_EWORKSPACE, "idx_distill: workspace %zu bytes, need %zu", ws_bytes, need);
    REQUIRE(aligned(ws, 16), IDX_EALIGN, "idx_distill: misaligned workspace");
    a.loss = loss;
    a.lse = lse;
    a.t_lse = t_lse;
    a.ws = ws;
    return hip_status(launch_distill(a, (hipStream_t)stream), "idx_distill");
}

idx_status idx_distill_bwd(const float* scores, int64_t score_stride, const int32_t* n_vis, int32_t nq, int64_t max_n,
                           const int32_t* t_idx, const float* t_logit, int64_t t_stride, int32_t k, float inv_temp,
                           const float* lse, const float* t_lse, const float* dloss, float* dscores, int64_t d_stride,
                           void* stream) {
    DistillArgs a{};
    const idx_status st = distill_args("idx_distill_bwd", scores, score_stride, n_vis, nq, max_n, t_idx, t_logit,
                                       t_stride, k, inv_temp, a);
    if (st != IDX_OK || nq == 0 || max_n == 0) return st;
    REQUIRE(lse && t_lse && dloss && dscores, IDX_EINVAL, "idx_distill_bwd: null pointer");
    REQUIRE(d_stride >= max_n, IDX_EINVAL, "idx_distill_bwd: d_stride=%lld < max_n", (long long)d_stride);
    REQUIRE(dscores != scores || d_stride == score_stride, IDX_EINVAL, "idx_distill_bwd: in place, the strides must agree");
    REQUIRE(aligned(lse, 4) && aligned(t_lse, 4) && aligned(dloss, 4) && aligned(dscores, 4), IDX_EALIGN,
            "idx_distill_bwd: misaligned pointer");
    a.lse = const_cast<float*>(lse);
    a.t_lse = const_cast<float*>(t_lse);
    a.dloss = dloss;
    a.dscores = dscores;
    a.d_stride = d_stride;
    return hip_status(launch_distill_bwd(a, (hipStream_t)stream), "idx_distill_bwd");
}

idx_status idx_write_rows(int32_t format, const void* x, int32_t dtype, int64_t tokens, int64_t x_stride, int32_t norm,
                          const float* gamma, double eps, const int64_t* pos, const double* freq, int32_t rot,
                          int32_t offset, int32_t layout, double mscale, const int8_t* signs, uint8_t* codes,
                          uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                          int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq, const int64_t* at,
                          int64_t max_n, int64_t ring, void* stream) {
    return write_rows("idx_write_rows", format, x, dtype, tokens, x_stride, norm, gamma, eps, pos, freq, rot, offset, layout,
                      mscale, signs, codes, scales, rows, kv_base, pages, pages_stride, nseq, page_size, seq, at, max_n, ring,
                      nullptr, stream);
}

idx_status idx_write_rows_kept(int32_t format, const void* x, int32_t dtype, int64_t tokens, int64_t x_stride, int32_t norm,
                               const float* gamma, double eps, const int64_t* pos, const double* freq, int32_t rot,
                               int32_t offset, int32_t layout, double mscale, const int8_t* signs, uint8_t* codes,
                               uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                               int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq, const int64_t* at,
                               int64_t max_n, int64_t ring, const int64_t* keep, void* stream) {
    return write_rows("idx_write_rows_kept", format, x, dtype, tokens, x_stride, norm, gamma, eps, pos, freq, rot, offset,
                      layout, mscale, signs, codes, scales, rows, kv_base, pages, pages_stride, nseq, page_size, seq, at,
                      max_n, ring, keep, stream);
}

idx_status idx_read_rows(int32_t format, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                         const int64_t* kv_base, const int32_t* pages, int64_t pages_stride, int32_t nseq,
                         int32_t page_size, const int32_t* seq, const int64_t* at, int64_t max_n, int64_t ring,
                         int64_t tokens, const int64_t* pos, const double* freq, int32_t rot, int32_t offset,
                         int32_t layout, double mscale, int32_t inverse, void* out, int32_t dtype, int64_t out_stride,
                         void* stream) {
    const char* fn = "idx_read_rows";
    RowsArgs a{};
    idx_status st = places_args(fn, rows, kv_base, pages, pages_stride, nseq, page_size, seq, tokens, max_n, ring, a.places);
    if (st == IDX_OK) st = rows_args(fn, format, out, dtype, tokens, out_stride, codes, scales, at, a);
    if (st == IDX_OK) st = turn_args(fn, row_dim(format), pos, freq, rot, offset, layout, mscale, inverse, a.turn);
    if (st != IDX_OK) return st;
    REQUIRE(!freq || format != IDX_ROWS_KEY, IDX_EINVAL, "%s: keys are stored transformed and cannot be turned", fn);
    REQUIRE(out_stride >= row_dim(format), IDX_EINVAL, "%s: out_stride=%lld < %d", fn, (long long)out_stride,
            row_dim(format));
    if (tokens == 0) return ok();
    a.out = out;
    return hip_status(launch_read_rows(a, (hipStream_t)stream), fn);
}

idx_status idx_attend_local(const uint16_t* q, int32_t nq, int32_t heads, int32_t group, const uint8_t* codes,
                            const uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                            int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq,
                            const int32_t* n_vis, int64_t max_n, int64_t window, int64_t ring, float scale,
                            const uint16_t* other, const float* other_lse, const int64_t* pos, const double* freq,
                            int32_t rot, int32_t offset, int32_t layout, double mscale, uint16_t* out, float* lse,
                            void* ws, size_t ws_bytes, void* stream) {
    return attend_local("idx_attend_local", q, nq, heads, group, codes, scales, rows, kv_base, pages, pages_stride, nseq,
                        page_size, seq, 1, n_vis, max_n, window, ring, scale, other, other_lse, pos, freq, rot, offset,
                        layout, mscale, out, lse, ws, ws_bytes, stream);
}

idx_status idx_attend_local_strided(const uint16_t* q, int32_t nq, int32_t heads, int32_t group, const uint8_t* codes,
                                    const uint8_t* scales, int64_t rows, const int64_t* kv_base, const int32_t* pages,
                                    int64_t pages_stride, int32_t nseq, int32_t page_size, const int32_t* seq,
                                    int64_t seq_stride, const int32_t* n_vis, int64_t max_n, int64_t window, int64_t ring,
                                    float scale, const uint16_t* other, const float* other_lse, const int64_t* pos,
                                    const double* freq, int32_t rot, int32_t offset, int32_t layout, double mscale,
                                    uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
    return attend_local("idx_attend_local_strided", q, nq, heads, group, codes, scales, rows, kv_base, pages, pages_stride,
                        nseq, page_size, seq, seq_stride, n_vis, max_n, window, ring, scale, other, other_lse, pos, freq, rot,
                        offset, layout, mscale, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
