// Launchers of the operators around the quantised products (moe_rows.hip, moe_route.hip, gated.hip, norm.hip).
#pragma once

#include "glowq_internal.h"

namespace glowq {

// Above this many bytes a tensor does not stay in the L2 caches (8 x 4 MB) for its next reader.
constexpr int64_t kStreamBytes = (int64_t)32 << 20;

constexpr int kMoeMaxTopK = 64;  // choices per token: one lane of a wavefront each

// Routing lists.  n pairs (T top_k), buckets 0 .. n_exp - 1 for the experts and n_exp for pairs
// without one.  Up to kSortOnePairs pairs one workgroup does everything; above, n_blocks
// workgroups of `chunk` pairs count into part [n_blocks][n_exp + 1] and place in a second launch.
constexpr int kSortThreads = 1024;
constexpr int64_t kSortOnePairs = 8192;
constexpr int64_t kSortMaxBlocks = 256;
struct SortArgs {
    const int32_t* ids;
    int32_t n, top_k, n_exp;
    int32_t n_blocks, chunk;
    int32_t* part;
    int32_t* offsets;    // [n_exp + 1]
    int32_t* row_token;  // [n]
    int32_t* pair_row;   // [n]
    int32_t* err;
};
hipError_t launch_moe_sort(const SortArgs& a, hipStream_t stream);

struct RowsArgs {
    const void* x;             // dispatch: [T][d]; combine: rows [n_rows][d]; gradient: dy [T][d]
    const void* rows;          // combine gradient: rows [n_rows][d]
    const void* add;           // combine: [T][d] or nullptr
    const int32_t* row_token;  // [n_rows]
    const int32_t* pair_row;   // [T][top_k]
    const float* w;            // [T][top_k] or nullptr (ones)
    void* out;                 // dispatch: rows; combine: y; gradient: d_rows
    float* dw;                 // gradient: [T][top_k]
    int32_t T, top_k, n_rows;
    int64_t d;
    int32_t dtype;             // GLOWQ_DTYPE_*
    int32_t whole;             // gradient: rows that no pair takes are zeroed
    int32_t* err;
};
hipError_t launch_moe_dispatch(const RowsArgs& a, hipStream_t stream);
hipError_t launch_moe_combine(const RowsArgs& a, hipStream_t stream);
hipError_t launch_moe_combine_backward(const RowsArgs& a, hipStream_t stream);

// Router (moe_route.hip).
struct RouteArgs {
    const void* logits;   // [T][n_exp]
    const float* bias;    // [n_exp] or nullptr
    int32_t T, n_exp, top_k;
    int32_t score;        // GLOWQ_SCORE_*
    int32_t n_group, keep_groups, group_best;
    int32_t renorm;
    float scale;
    int32_t* ids;         // [T][top_k]
    float* w;             // [T][top_k]; gradient: d_weights
    void* out;            // gradient: d_logits [T][n_exp]
    int32_t* err;
};
hipError_t launch_moe_route(const RouteArgs& a, int32_t dtype, hipStream_t stream);
hipError_t launch_moe_route_backward(const RouteArgs& a, int32_t dtype, hipStream_t stream);

// Layer norm (norm.hip).
constexpr int64_t kNormMaxD = 16384;  // a row in its threads' registers
constexpr int kNormParts = 256;       // workgroups of a gradient launch, each with sums [2][d] of its own
struct NormArgs {
    const void *x, *w, *b, *dy;  // w, b may be nullptr
    int32_t T, d;
    float eps;
    void* out;            // y; gradient: dx
    float *mean, *rstd;   // [T]
    float *dw, *db;       // [d], fp32
    float* part;          // [kNormParts][2][d], nullptr where neither dw nor db is wanted
};
hipError_t launch_layer_norm(const NormArgs& a, int32_t dtype, hipStream_t stream);
hipError_t launch_layer_norm_backward(const NormArgs& a, int32_t dtype, hipStream_t stream);

hipError_t launch_swiglu(const void* gate, const void* up, int64_t n, int32_t dtype, void* h, hipStream_t stream);
hipError_t launch_swiglu_backward(const void* dh, const void* gate, const void* up, int64_t n, int32_t dtype,
                                  void* dgate, void* dup, hipStream_t stream);

}  // namespace glowq
