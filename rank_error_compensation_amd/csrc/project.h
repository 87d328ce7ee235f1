// The projection R = X B^T as the 8-bit group forwards form it beside the token codes (w8a8.hip, fp8.hip): K ranges
// over workgroups, their fp32 sums joined by whoever comes next.  A: PrepArgs or Fp8PrepArgs (x, b, T, d, r, rp, ks, part, R).
#pragma once

#include "glowq_internal.h"

namespace glowq {

namespace {

constexpr int kPrepThreads = 512;
constexpr int kPrepWaves = kPrepThreads / 64;

// Where the inputs of TT rows of the result lie, as the rows themselves do.
template <int TT>
struct RowsInOrder {
    const _Float16* x;
    int d;
    __device__ __forceinline__ void operator()(const int (&t)[TT], const _Float16* (&at)[TT]) const {
#pragma unroll
        for (int i = 0; i < TT; ++i) at[i] = x + (size_t)t[i] * d;
    }
};

// Sums of R over the 32-input steps [s_begin, s_end) for 16 TT rows from t0 on (t_end at most) and 16 NJ rank columns: the
// wavefronts take steps in turn (U in flight) and add their tiles through LDS in wavefront order.
// part != nullptr: fp32 sums of this range to part [.][rp]; else one rounding to fp16 into R.
// Columns r .. r_pad - 1 are zero.
// rows(t, at): where the inputs of the rows t lie.
// RUNS: a wavefront takes U steps in a row (whole lines of X and B, and the wavefronts together spread over the memory
// channels: rows are often a multiple of their stride apart), else every kPrepWaves-th.
template <int TT, int NJ, bool RUNS, class A, class Row>
__device__ void project_tile(const A& a, const _Float16* b, const Row& rows, int t0, int t_end, int jb, int s_begin, int s_end,
                             float* part, f4* red) {
    constexpr int U = TT * NJ == 1 ? 8 : (TT * NJ <= 8 ? 4 : 2), N = TT * NJ;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int kofs = 8 * (lane >> 4), d = a.d, r = a.r, rp = a.rp;
    const _Float16 *xr[TT], *br[NJ];
    {
        int t[TT];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) t[tt] = min(t0 + 16 * tt + (lane & 15), t_end - 1);
        rows(t, xr);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) xr[tt] += kofs;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) br[j] = b + (size_t)min(16 * (NJ * jb + j) + (lane & 15), r - 1) * d + kofs;
    f4 acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
    constexpr int kApart = RUNS ? 1 : kPrepWaves;
    for (int s0 = s_begin + wave * (RUNS ? U : 1); s0 < s_end; s0 += U * kPrepWaves) {
        h8 xv[U][TT], bv[U][NJ];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = 32 * min(s0 + u * kApart, s_end - 1);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) xv[u][tt] = load_h8(xr[tt] + k);
#pragma unroll
            for (int j = 0; j < NJ; ++j) bv[u][j] = load_h8(br[j] + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u * kApart < s_end) {
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) acc[tt * NJ + j] = mfma16(xv[u][tt], bv[u][j], acc[tt * NJ + j]);
            }
    }
    // the upper half's tiles into the lower half, then wavefront i < N sums tile i (half the LDS of one
    // step: the token workgroups of the same launch need the room to run side by side)
    constexpr int H = kPrepWaves / 2;
    if (wave >= H) {
#pragma unroll
        for (int i = 0; i < N; ++i) red[((wave - H) * N + i) * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (wave < H) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f4* own = red + (wave * N + i) * 64 + lane;
            *own = acc[i] + *own;
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; n += kPrepWaves) {
        const int tile = n + wave;
        if (tile >= N) return;
        f4 v = red[tile * 64 + lane];
#pragma unroll
        for (int w = 1; w < H; ++w) v += red[(w * N + tile) * 64 + lane];
        const int col = 16 * (NJ * jb + tile % NJ) + (lane & 15);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = t0 + 16 * (tile / NJ) + 4 * (lane >> 4) + i;
            const float o = col < r ? v[i] : 0.f;
            if (t < t_end && col < rp) {
                if (part != nullptr) part[(size_t)t * rp + col] = o;
                else a.R[(size_t)t * rp + col] = (_Float16)o;
            }
        }
    }
}

// R = the K ranges' sums added in order, rounded once to fp16; four values from value 4 i.  A few MB out of
// the caches (T = 2048, r = 64, 4 ranges: 2.1 MB, 4.9 us): bound by its launch.
template <class A>
__device__ __forceinline__ void join_ranges(const A& a, size_t i) {
    const size_t n = (size_t)a.T * a.rp / 4;
    if (i >= n) return;
    const f4* p = reinterpret_cast<const f4*>(a.part) + i;
    f4 v = p[0];
#pragma unroll 4
    for (int k = 1; k < a.ks; ++k) v += p[(size_t)k * n];
    const h2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
    reinterpret_cast<u2*>(a.R)[i] = u2{as_u32(lo), as_u32(hi)};
}

}  // namespace

}  // namespace glowq
