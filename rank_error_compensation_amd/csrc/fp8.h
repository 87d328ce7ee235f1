// The block-scaled 8-bit floating-point products (fp8.hip): layout constants, arguments and launchers.
#pragma once

#include "glowq_internal.h"

namespace glowq {

constexpr int kFmtFp8 = 5;           // GLOWQ_FMT_FP8_BLOCK
constexpr int kFp8Block = 2048;      // bytes of one 16-row x 128-input weight block
constexpr int kFp8Waves = 8;         // wavefronts that split the input groups of a small tile
constexpr int64_t kFp8MaxD = 16384;  // inputs

// Bytes of one module's scales (fp32 [ceil(n_out / 128)][k_in / 128]), whole 64 bytes.
inline size_t fp8_sz_bytes(int64_t n_out, int64_t k_in) {
    return (size_t)ceil_div(ceil_div(n_out, 128) * (k_in / kGroup) * 4, 64) * 64u;
}
// Row stride of the activation scales [T][gp]: whole 16 bytes.
inline int64_t fp8_scale_stride(int64_t d) { return ceil_div(d / kGroup, 4) * 4; }

// Codes and scales of the tokens and, for r > 0, the projection, one launch.
struct Fp8PrepArgs {
    const _Float16* x;  // [T][d]
    const _Float16* b;  // [r][d]
    int32_t T, d, r, rp;
    int32_t range, ks;  // inputs per K range of the projection, ranges
    int32_t gp;
    uint8_t* xq;        // [T][d]
    float* xs;          // [T][gp]
    float* part;        // [ks][T][rp], nullptr for one range rounded directly
    _Float16* R;        // [T][rp]
};

struct Fp8Module {
    const uint8_t* q;    // device layout (of expert 0)
    const float* sz;
    const _Float16* a;   // [n_out][r], nullptr where not corrected
    _Float16* y;         // [T or n_rows][n_out]
    int64_t q_step, sz_step, a_step;  // from one expert to the next: bytes, values, values
    int32_t n_out, n_tiles16;
    int32_t block_begin;  // first row block of this module in the launch's numbering
};

struct Fp8Args {
    int32_t T, d, G, gp;
    int32_t n_mod;
    const uint8_t* xq;
    const float* xs;
    int32_t r, rp;
    const void* R;        // r_ranges fp32 K ranges [.][r_rows][rp], or fp16 [r_rows][rp] where r_ranges is 0
    int32_t r_ranges, r_rows;
    int32_t tt, rr;       // 16-token and 16-row tiles per workgroup; rr >= 8: the large tiles
    int32_t kh;           // teams of wavefronts in a workgroup that split its input groups (large tiles)
    int32_t ks, gk;       // K ranges over workgroups, input groups per range (large tiles)
    float* part;          // the K ranges' fp32 tiles
    int32_t row_blocks;   // of all modules
    int32_t m_blocks;     // token blocks
    // experts (offsets != nullptr): rows listed by expert
    const int32_t* row_token;  // [n_rows] or nullptr
    const int32_t* offsets;    // [n_exp + 1]
    int32_t n_exp, n_rows;
    int32_t r_by_token;   // R's row is the row's token (else the row itself)
    int32_t* err;
    Fp8Module mod[kMaxModules];
};

hipError_t launch_repack_fp8(const uint8_t* codes, const float* scales, int64_t n_out, int64_t k_in, uint8_t* q, float* sz,
                             int32_t* flag, hipStream_t stream);
// experts (may be nullptr): the projection by each expert's own B, over row_blocks blocks of 16 tt rows at most.
hipError_t launch_fp8_prep(const Fp8PrepArgs& a, int tt, int nj, bool join, const struct Fp8Args* experts, int64_t row_blocks,
                           hipStream_t stream);
// Large tiles by Fp8Args::tt x rr: 8 x 16 and 8 x 8 on four wavefronts, 4 x 8 on two, times kh teams.
// items: an upper bound of the launch's work tiles.  p: the preparation of the same call, whose projection ranges a launch
// with K ranges joins.
hipError_t launch_fp8(const Fp8Args& a, const Fp8PrepArgs& p, int64_t items, hipStream_t stream);

}  // namespace glowq
