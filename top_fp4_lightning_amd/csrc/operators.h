// Internal declarations of the operators beside the indexer: rotary positions, core attention over the
// main-KV cache, distillation of score rows, cache rows at places of their own (not part of the C ABI).
#pragma once

#include "internal.h"

namespace fp4idx {

// two fp32 values as a pair of bf16 bit patterns, round to nearest even
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 v = {(__bf16)lo, (__bf16)hi};
    uint32_t r;
    __builtin_memcpy(&r, &v, 4);
    return r;
}

// core attention over the main-KV cache
struct AttendArgs {
    const uint16_t* q;      // bf16 [nq][heads][512]
    int32_t nq;
    int32_t heads;
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t rows;           // cache rows; a row outside is as a position that is not visible
    const int64_t* kv_base; // contiguous form: position p of query t is row kv_base[t] + p
    const int32_t* pages;   // paged form: row pages[seq[t]][p / page_size] * page_size + p % page_size
    int64_t pages_stride;
    int32_t nseq;
    int32_t page_size;
    const int32_t* seq;     // may be null (query t is of sequence t)
    const int32_t* n_vis;
    int64_t max_n;
    int64_t window;         // range form: the last `window` visible positions; 0 is all
    const int32_t* idx;     // list form: positions, or null
    int64_t idx_stride;
    int32_t k;
    float scale;
    uint16_t* out;          // bf16 [nq][heads][512]
    float* lse;             // [nq][heads] or null
    uint32_t page_mul;      // set by the launch: p / page_size = (p * page_mul >> 32) >> page_shift
    int32_t page_shift;
    float* part_o;
    float* part_ml;
};
// the bytes of the fastest cut of such a call; a launch in fewer cuts into what fits. entries: list slots, or the most
// positions a query attends to
size_t attend_workspace_bytes(int32_t nq, int32_t heads, int64_t entries);
hipError_t launch_attend(AttendArgs a, void* ws, size_t ws_bytes, hipStream_t stream);
hipError_t launch_attend_weights(AttendArgs a, const float* lse, float* weights, int64_t w_stride,
                                 hipStream_t stream);

// rotary positions
struct RopeArgs {
    const void* x;          // [tokens][heads][dim], element strides x_token, x_head
    bool f32;               // else bf16
    int64_t tokens;
    int32_t heads;
    int32_t dim;
    int64_t x_token, x_head;
    const int64_t* pos;
    const double* freq;     // [rot / 2], radians per position
    int32_t rot;            // even; values offset .. offset + rot - 1 of a row
    int32_t offset;
    bool half;              // pairs (i, i + rot / 2), else (2i, 2i + 1)
    bool inverse;
    float mscale;
    void* out;              // may be x (with its strides)
    int64_t out_token, out_head;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t stream);

// distillation of score rows
struct DistillArgs {
    const float* scores;
    int64_t score_stride;
    const int32_t* n_vis;
    int32_t nq;
    int64_t max_n;
    const int32_t* t_idx;
    const float* t_logit;
    int64_t t_stride;
    int32_t k;
    float inv_temp;
    float* loss;            // forward: written
    float* lse;             // forward: written; gradient: read
    float* t_lse;
    const float* dloss;     // gradient
    float* dscores;
    int64_t d_stride;
    void* ws;
};
size_t distill_workspace_bytes(int32_t nq, int64_t max_n);
hipError_t launch_distill(const DistillArgs& a, hipStream_t stream);
hipError_t launch_distill_bwd(const DistillArgs& a, hipStream_t stream);

// cache rows at places of their own
struct Division {  // by a number known to the host (places.h), 0: none
    uint32_t by, mul;
    int32_t shift;
};
struct Places {
    int64_t rows;           // cache rows; an entry whose row is outside is not there
    const int64_t* base;    // contiguous form: entry p lies in row base + p
    const int32_t* pages;   // paged form: row pages[s][p / page] * page + p % page
    int64_t pages_stride;
    int32_t nseq;
    const int32_t* seq;
    Division page, ring;    // ring: entry p takes the place of entry p % ring
    int64_t max_n;          // entries 0 .. max_n - 1
};
struct Turn {
    const int64_t* pos;     // null with freq: the entry's number
    const double* freq;     // null: none
    int32_t rot;
    int32_t offset;
    bool half;
    bool inverse;
    double mscale;
};
struct RowsArgs {
    int32_t format;
    bool f32;               // x, out: else bf16
    bool wide;              // x, out: rows of whole, aligned 16-byte pieces
    int64_t tokens;
    Places places;
    const int64_t* at;      // [tokens]
    Turn turn;
    uint8_t* codes;
    uint8_t* scales;
    const void* x;          // write: rows, stride elements apart
    bool norm;
    const float* gamma;     // may be null
    double eps;
    const int8_t* signs;    // keys
    const int64_t* keep;    // write: below 0 where a token is left out; may be null
    void* out;              // read
    int64_t stride;         // of x or out
};
// attention over the cache of local positions, joined with another part
struct LocalArgs {
    const uint16_t* q;      // bf16 [nq][heads][512]
    int32_t nq;
    int32_t heads;
    int32_t group;          // consecutive queries of one sequence
    const uint8_t* codes;
    const uint8_t* scales;
    Places places;          // base and seq by run of `group` queries,
    int64_t seq_stride;     // run i's sequence at seq[i * seq_stride]
    const int32_t* n_vis;
    int64_t window;         // the last `window` visible entries; 0 is all
    float scale;
    const uint16_t* other;  // bf16 [nq][heads][512] or null: another part of the softmax, normalised by itself
    const float* other_lse; // [nq][heads]
    Turn turn;              // of the result
    uint16_t* out;
    float* lse;             // or null
    float* part_o;          // set by the launch
    float* part_ml;
    int2* shares;
};
size_t local_workspace_bytes(int32_t nq, int32_t heads, int64_t entries);
hipError_t launch_attend_local(LocalArgs a, void* ws, size_t ws_bytes, hipStream_t stream);
hipError_t launch_write_rows(const RowsArgs& a, hipStream_t stream);
hipError_t launch_read_rows(const RowsArgs& a, hipStream_t stream);

}  // namespace fp4idx
