// The 8-bit integer group forward (w8a8.hip): layout constants and launchers.
#pragma once

#include "glowq_internal.h"

namespace glowq {

constexpr int kFmtInt8 = 4;        // GLOWQ_FMT_INT8_CHANNEL
constexpr int kW8Block = 2048;     // bytes of one 16-row x 128-input weight block
constexpr int kW8Waves = 8;        // wavefronts that split the input groups of a small tile
// Tiles by ForwardArgs::tile_tt x tile_rr (16-token and 16-row tiles per workgroup): 8 x 16 and 8 x 8 on four
// wavefronts, 4 x 8 on two, times ForwardArgs::dec_ks teams; rr = 1, 2 is the small form, whose wavefronts split the
// input groups.
constexpr int64_t kW8MaxD = 16384; // a token's row in the quantiser's registers; int32 sums exact

// Launch shape of a call.
struct W8Shape {
    int tt, rr;      // 16-token tiles and 16-row tiles per workgroup
    int kh;          // teams of wavefronts in a workgroup that split its input groups (tiles)
    int ks, gk;      // K ranges over workgroups, input groups per range
};

hipError_t launch_repack_w8(const int8_t* codes, const float* scales, int64_t n_out, int64_t k_in, uint8_t* q, float* sz,
                            int32_t* flag, hipStream_t stream);
// Token codes and scales and, for r > 0, the projection, one launch.  For the small form and for
// unsplit tiles of several teams (one round of workgroups, each of which reads few of them) the K ranges'
// fp32 sums [ks][T][rp] stay in `part` for the product to add (a launch of 4 us less: 2 x 11008 <- 4096 at T = 64,
// 32 us, 33.5 with it); for the other tiles they are joined into the fp16 R [T][rp] by a second launch (written
// directly with one range).
struct PrepPlan {
    int tt, nj;     // 16-token tiles and 16-column tiles of R per workgroup
    int range, ks;  // inputs per K range, ranges
};
PrepPlan w8a8_prep_plan(int64_t T, int64_t d, int32_t r, bool small);
struct PrepArgs {
    const _Float16* x;  // [T][d]
    const _Float16* b;  // [r][d]
    int32_t T, d, r, rp;
    int32_t range, ks;
    int8_t* xq;
    float* xscale;
    float* part;   // [ks][T][rp], nullptr for one range rounded directly
    _Float16* R;
};
// join: add the projection's ranges here (false where launch_w8a8 does, in a call whose K is split)
hipError_t launch_w8a8_prep(const PrepArgs& a, const PrepPlan& p, bool join, hipStream_t stream);
hipError_t launch_w8a8(const ForwardArgs& a, const PrepArgs& p, hipStream_t stream);

}  // namespace glowq
