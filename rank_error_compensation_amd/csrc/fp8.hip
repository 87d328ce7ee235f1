// Products on 8-bit floating-point weights (e4m3) with one fp32 scale for each block of 128 rows x 128 inputs, as a group
// forward and over the experts of a mixture, on the gfx950 matrix cores; the low-rank correction on the fp16 activations.
//
//   per token t and group g of 128 inputs, fp32:  s[t, g] = max |x| / 448,  c = e4m3(x (448 / max |x|)), ties to even
//   y_i[t, o] = sum_g s[t, g] S_i[o / 128, g] sum_{k in g} c[t, k] q_i[o, k] + R[t] . A_i[o],   R = X B^T
//
// One v_mfma_f32_16x16x128_f8f6f4 step is one group of 16 rows and 16 tokens, and the group's sum is scaled once, in
// fp32, as it is added.  Inside the step the matrix core brings eight products at a time to the exponent 2^e of the
// largest and drops what lies below 2^(e - 13); the sixteen sums of eight meet in fp32.  On activations and weights that
// are spread like normal numbers sums move by 3e-5 of their norm, rounded results by 1.1e-4, which leaves their distance from
// the exact ones at that of the rounding to fp16 (2.0e-4).  An input in every eight that is 300 times the others
// leaves them 2.2e-4 from the exact ones; where those inputs' products cancel over each group, the rest is 2.5e-2 of its norm off,
// as much as the rounding to codes moves it (2.6e-2).  fp32 throughout would cost the step at half the rate (16x16x32).
// A group with an infinity or a NaN has scale NaN: the token's results are NaN.
//
// Weight layout: NT x G blocks of 2048 bytes, block (rt, g) at (rt G + g) 2048 holding rows 16 rt .. + 15 and
// inputs 128 g .. + 127 as two 1024-byte halves: half m, lane l (16 bytes at 1024 m + 16 l) is row 16 rt + l % 16, inputs
// 128 g + 64 m + 16 (l / 16) .. + 15.  A lane's 32 bytes of the step's operand are its pieces of both halves; the
// activation operand takes the same inputs in the same places, so the order of inputs inside the step does not matter.
// Rows >= n_out are zero.  Codes of the activations lie in their natural order [T][d], scales [T][G rounded up to 4].
//
// Launches: codes, scales and the projection (with K ranges a launch more that adds them, where the product does not), then
// the product, in pieces whose wavefronts share the input groups (few tokens: one round of loads each) or in tiles; with K
// ranges of the tiles a last launch joins those.  r = 64, kernels alone (shortest and mean of 53 warm runs: the clock falls while
// the large products run) / the call from the host, us:
//   T = 1, 4096 + 2 x 1024 <- 4096         4.3, 4.9 + 6.1, 7.2 / 16.8 (two launches from the host; 25 MB of weights)
//   T = 77, 4096 <- 14336                  6.8, 8.1 + 17.8, 19.1 + 7.0, 7.2 / 33.6 (eight ranges: 59 MB of weights, 17 MB of sums)
//   T = 2048, 2 x 11008 <- 4096            14.2, 15.8 + 4.0, 5.1 + 174, 187 / 199 (the tile 2.15 and 2.0 PFLOP/s, the library's
//                                          product alone 2.25)
//   T = 1, 4 of 60 experts 2048 -> 2 x 1408    4.3, 4.9 + 6.3, 7.3 / 17.3
//   T = 4095, 60 experts, 4 choices        38, 45 + 147, 160 / 190 (a B each; 1.2 PFLOP/s: a fifth of the tiles' token rows
//                                          are empty, and 2 x 1408 rows are computed as 2 x 1536)
#include <algorithm>
#include <type_traits>

#include "fp8.h"
#include "project.h"

namespace glowq {

typedef int32_t i8v __attribute__((ext_vector_type(8)));

namespace {

// The two 16-byte pieces of an operand, as the eight registers that the matrix core reads.
__device__ __forceinline__ i8v load_operand(const void* p0, const void* p1) {
    typedef int32_t i4v __attribute__((ext_vector_type(4)));
    return __builtin_shufflevector(*static_cast<const i4v*>(p0), *static_cast<const i4v*>(p1), 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f4 mfma_fp8(const i8v& w, const i8v& x) {
    // scale operands of zero: the form without block scales
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// --------------------------------------------------------------------- load step
// One workgroup per (128-input group, row tile): 128 threads, each one lane's 16 bytes.  NaN codes (0x7F, 0xFF) are reported.
__global__ __launch_bounds__(128) void repack_fp8_kernel(const uint8_t* __restrict__ codes, int64_t n_out, int64_t k_in, int groups,
                                                         uint8_t* __restrict__ q, int32_t* __restrict__ flag) {
    const int64_t blk = blockIdx.x;  // rt G + g
    const int64_t rt = blk / groups, g = blk - rt * groups;
    const int m = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t row = 16 * rt + (l & 15);
    u4 v = {0u, 0u, 0u, 0u};
    if (row < n_out) v = *reinterpret_cast<const u4*>(codes + row * k_in + 128 * g + 64 * m + 16 * (l >> 4));
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) bad |= ((v[i / 4] >> (8 * (i % 4))) & 0x7Fu) == 0x7Fu;
    if (bad) __hip_atomic_store(flag, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *reinterpret_cast<u4*>(q + blk * kFp8Block + 1024 * m + 16 * l) = v;
}

__global__ __launch_bounds__(256) void repack_fp8_scales_kernel(const float* __restrict__ scales, int64_t n, int64_t n_pad,
                                                                float* __restrict__ sz, int32_t* __restrict__ flag) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n_pad) return;
    const float s = i < n ? scales[i] : 0.f;
    if (!(fabsf(s) < INFINITY)) __hip_atomic_store(flag, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sz[i] = s;
}

// --------------------------------------------------------------------- token codes and projection
// Eight inputs of one group by each thread, a group by 16 threads, U groups in turn with all their loads in flight.  The
// workgroups of the projection come first in the same launch: both read X, neither needs the other.
template <int U>
__device__ __forceinline__ void quant_groups(const Fp8PrepArgs& a, int64_t block) {
    const int per = a.d / 8;
    const int64_t first = block * (U * kPrepThreads) + threadIdx.x, chunks = (int64_t)a.T * per;
    h8 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t chunk = first + u * kPrepThreads;
        v[u] = chunk < chunks ? load_h8(a.x + 8 * chunk) : h8{0, 0, 0, 0, 0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t chunk = first + u * kPrepThreads;
        if (chunk >= chunks) return;  // whole groups of 16 threads: T d is a multiple of 128
        const int64_t t = chunk / per;
        const int c = (int)(chunk - t * per);
        const u4 bits = __builtin_bit_cast(u4, v[u]) & 0x7FFF7FFFu;
        uint32_t top = 0;  // as fp16 bits: infinities and NaN order above every number
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(bits[e] & 0xFFFFu, bits[e] >> 16));
#define GLOWQ_ROR(N) top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x120 + N, 0xf, 0xf, false))
        GLOWQ_ROR(8);
        GLOWQ_ROR(4);
        GLOWQ_ROR(2);
        GLOWQ_ROR(1);
#undef GLOWQ_ROR
        const float amax = (float)__builtin_bit_cast(_Float16, (uint16_t)top);
        const bool finite = top < 0x7C00u;
        const float scale = finite ? amax / 448.0f : __builtin_nanf("");  // IEEE divisions
        const float inv = finite && top > 0 ? 448.0f / amax : 0.f;
        // |x inv| <= 448 (1 + 2^-23): rounds to 448 at most, no saturation needed
        uint32_t w[2] = {0u, 0u};
        if (finite) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int p = __builtin_amdgcn_cvt_pk_fp8_f32((float)v[u][4 * j] * inv, (float)v[u][4 * j + 1] * inv, 0, false);
                p = __builtin_amdgcn_cvt_pk_fp8_f32((float)v[u][4 * j + 2] * inv, (float)v[u][4 * j + 3] * inv, p, true);
                w[j] = (uint32_t)p;
            }
        }
        *reinterpret_cast<u2*>(a.xq + 8 * chunk) = u2{w[0], w[1]};
        const int g = c >> 4;
        if ((c & 15) == 0) a.xs[t * a.gp + g] = scale;
        // zeros up to the stride
        if (g == a.d / kGroup - 1 && (c & 15) > 0 && g + (c & 15) < a.gp) a.xs[t * a.gp + g + (c & 15)] = 0.f;
    }
}

template <int TT, int NJ, int U>
__global__ __launch_bounds__(kPrepThreads) void fp8_prep_kernel(const Fp8PrepArgs a, int proj_blocks) {
    __shared__ f4 red[kPrepWaves / 2 * TT * NJ * 64];
    const int blk = blockIdx.x;
    if (blk >= proj_blocks) {
        quant_groups<U>(a, blk - proj_blocks);
        return;
    }
    const int cols = (a.rp / 16 + NJ - 1) / NJ;
    const int k = blk % a.ks, rest = blk / a.ks, jb = rest % cols, tb = rest / cols;
    const int per = a.range / 32;
    project_tile<TT, NJ, true>(a, a.b, RowsInOrder<TT>{a.x, a.d}, 16 * TT * tb, a.T, jb, k * per, min((k + 1) * per, a.d / 32),
                         a.part != nullptr ? a.part + (size_t)k * a.T * a.rp : nullptr, red);
}

__global__ __launch_bounds__(256) void fp8_join_kernel(const Fp8PrepArgs a) {
    join_ranges(a, (size_t)blockIdx.x * 256 + threadIdx.x);
}

// --------------------------------------------------------------------- work tiles
// What a workgroup computes: token rows j0 .. j1 - 1 (at most a block of them) on row block rb of all modules.
struct Work {
    int e;        // expert (0 without)
    int rb;
    int j0, j1;   // rows of the outputs
};

// Item of the launch with experts, in the order (expert, one of row_blocks, block of its rows).  Every wavefront finds its
// own, four experts a lane.  Offsets out of order or range are clamped and reported by the first workgroup.  spread: XCD x
// (workgroups b with b % 8 == x) takes a run of consecutive items, so that an expert's row block stays in one L2.
__device__ __forceinline__ bool expert_work(const Fp8Args& a, int rows_per_block, int row_blocks, int item, bool spread, Work& w) {
    const int lane = threadIdx.x & 63;
    int o[5], lo[4], hi[4], nb[4], sum = 0;
#pragma unroll
    for (int q = 0; q < 5; ++q) o[q] = a.offsets[min(4 * lane + q, a.n_exp)];  // past the last expert: no rows
    bool bad = (lane == 0 && o[0] != 0) || (4 * lane + 4 >= a.n_exp && o[4] != a.n_rows);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        bad |= o[q] < 0 || o[q + 1] > a.n_rows || o[q + 1] < o[q];
        lo[q] = min(max(o[q], 0), a.n_rows);
        hi[q] = min(max(o[q + 1], lo[q]), a.n_rows);
        nb[q] = 4 * lane + q < a.n_exp ? (hi[q] - lo[q] + rows_per_block - 1) / rows_per_block : 0;
        sum += nb[q];
    }
    if (bad && blockIdx.x == 0) __hip_atomic_fetch_or(a.err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    int upto = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int n = __shfl_up(upto, off, 64);
        if (lane >= off) upto += n;
    }
    if (spread) {
        const int total = __builtin_amdgcn_readlane(upto, 63) * row_blocks, run = (total + 7) >> 3;
        if ((item >> 3) >= run) return false;
        item = (item & 7) * run + (item >> 3);
    }
    int at = (upto - sum) * row_blocks, e = 0, blocks = 1, first = 0, l = 0, h = 0;
    bool hit = false;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int end = at + nb[q] * row_blocks;
        if (item >= at && item < end) hit = true, e = 4 * lane + q, blocks = nb[q], first = at, l = lo[q], h = hi[q];
        at = end;
    }
    const uint64_t who = __ballot(hit);
    if (who == 0) return false;
    const int src = __ffsll((unsigned long long)who) - 1;
    blocks = __builtin_amdgcn_readlane(blocks, src);
    first = __builtin_amdgcn_readlane(first, src);
    l = __builtin_amdgcn_readlane(l, src);
    h = __builtin_amdgcn_readlane(h, src);
    w.e = __builtin_amdgcn_readlane(e, src);
    const int local = item - first;
    w.rb = local / blocks;
    w.j0 = l + (local - w.rb * blocks) * rows_per_block;
    w.j1 = min(w.j0 + rows_per_block, h);
    return true;
}

__device__ __forceinline__ int fp8_module_of(const Fp8Args& a, int rb) {
    int i = 0;
#pragma unroll
    for (int k = 1; k < kMaxModules; ++k) i += (k < a.n_mod && rb >= a.mod[k].block_begin) ? 1 : 0;
    return __builtin_amdgcn_readfirstlane(i);
}

// Tokens of N output rows: themselves, or where the list says; one out of range is clamped and reported.  The N entries
// are requested together.
template <bool EXPERTS, int N>
__device__ __forceinline__ void tokens_of(const Fp8Args& a, const int (&j)[N], int (&t)[N]) {
    if (!EXPERTS || a.row_token == nullptr) {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = j[i];
        return;
    }
    int listed[N];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < N; ++i) listed[i] = a.row_token[j[i]];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = min(max(listed[i], 0), a.T - 1);
        bad |= t[i] != listed[i];
    }
    if (bad) __hip_atomic_fetch_or(a.err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Codes and scales of the tokens and, in the first workgroups, the projection of every expert's rows by its own B: R's row j
// is that of output row j.
template <int TT, int NJ, int U>
__global__ __launch_bounds__(kPrepThreads) void fp8_prep_experts_kernel(const Fp8PrepArgs p, const Fp8Args a, int proj_blocks) {
    __shared__ f4 red[kPrepWaves / 2 * TT * NJ * 64];
    const int blk = blockIdx.x;
    if (blk >= proj_blocks) {
        quant_groups<U>(p, blk - proj_blocks);
        return;
    }
    const int k = blk % p.ks, cols = (p.rp / 16 + NJ - 1) / NJ;
    Work w;
    if (!expert_work(a, 16 * TT, cols, blk / p.ks, p.ks == 1, w)) return;
    const int per = p.range / 32;
    auto rows = [&](const int (&j)[TT], const _Float16* (&at)[TT]) {
        int t[TT];
        tokens_of<true>(a, j, t);
#pragma unroll
        for (int i = 0; i < TT; ++i) at[i] = p.x + (size_t)t[i] * p.d;
    };
    project_tile<TT, NJ, true>(p, p.b + (size_t)w.e * p.r * p.d, rows, w.j0, w.j1, w.rb, k * per, min((k + 1) * per, p.d / 32),
                         p.part != nullptr ? p.part + (size_t)k * a.n_rows * p.rp : nullptr, red);
}

// Four consecutive rows of output row j, rounded to fp16.
__device__ __forceinline__ void store_rows(const Fp8Module& M, int j, int row0, const f4& v) {
    _Float16* y = M.y + (size_t)j * M.n_out;
    if ((M.n_out & 3) == 0 && row0 + 3 < M.n_out) {
        const h2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
        *reinterpret_cast<u2*>(y + row0) = u2{as_u32(lo), as_u32(hi)};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + i < M.n_out) y[row0 + i] = (_Float16)v[i];
    }
}

// Eight columns of R from column c on, row ri, as fp16.
__device__ __forceinline__ h8 r_columns(const Fp8Args& a, int ri, int c) {
    if (a.r_ranges == 0) return load_h8(static_cast<const _Float16*>(a.R) + (size_t)ri * a.rp + c);
    const float* p = static_cast<const float*>(a.R) + (size_t)ri * a.rp + c;
    f4 lo = *reinterpret_cast<const f4*>(p), hi = *reinterpret_cast<const f4*>(p + 4);
    for (int k = 1; k < a.r_ranges; ++k) {
        p += (size_t)a.r_rows * a.rp;
        lo += *reinterpret_cast<const f4*>(p);
        hi += *reinterpret_cast<const f4*>(p + 4);
    }
    h8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = (_Float16)lo[i];
        v[4 + i] = (_Float16)hi[i];
    }
    return v;
}

// --------------------------------------------------------------------- product, small form
// 16 TT tokens x 16 RR rows per workgroup; its wavefronts take the input groups in turn (group g to wavefront
// g % kFp8Waves), operands straight from memory, and add their scaled sums through LDS in order.  Wavefront w then finishes
// tile w (w < TT RR): correction steps, one rounding to fp16.
template <int TT, int RR, bool EXPERTS>
__global__ __launch_bounds__(64 * kFp8Waves) void fp8_split_kernel(const Fp8Args args) {
    constexpr int NW = kFp8Waves, NT = TT * RR;
    static_assert(NT <= NW, "one tile per wavefront at the end");
    __shared__ f4 red[NW][NT][64];
    Work wk;
    if constexpr (EXPERTS) {
        if (!expert_work(args, 16 * TT, args.row_blocks, blockIdx.x, false, wk)) return;
    } else {
        wk.e = 0;
        wk.rb = blockIdx.x / args.m_blocks;
        wk.j0 = (blockIdx.x % args.m_blocks) * 16 * TT;
        wk.j1 = min(wk.j0 + 16 * TT, args.T);
    }
    const Fp8Module& M = args.mod[fp8_module_of(args, wk.rb)];
    const int rt0 = (wk.rb - M.block_begin) * RR;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int d = args.d, G = args.G, nt16 = M.n_tiles16;
    const uint8_t* q = M.q + (EXPERTS ? (size_t)wk.e * M.q_step : 0);
    const float* sz = M.sz + (EXPERTS ? (size_t)wk.e * M.sz_step : 0);

    const uint8_t* qp[RR];
    const float* sp[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) {
        const int rt = min(rt0 + rr, nt16 - 1);
        qp[rr] = q + (size_t)rt * G * kFp8Block + lane * 16;
        sp[rr] = sz + (size_t)(rt >> 3) * G;
    }
    const uint8_t* xp[TT];
    const float* xsp[TT];
    int tok[TT], rows[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) rows[tt] = min(wk.j0 + 16 * tt + (lane & 15), wk.j1 - 1);  // past the block: its last row
    tokens_of<EXPERTS>(args, rows, tok);
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        xp[tt] = args.xq + (size_t)tok[tt] * d + 16 * (lane >> 4);
        xsp[tt] = args.xs + (size_t)tok[tt] * args.gp;
    }
    f4 acc[TT][RR];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = f4{0.f, 0.f, 0.f, 0.f};
    constexpr int U = 2;
    for (int g0 = wave; g0 < G; g0 += U * NW) {
        i8v w[U][RR], x[U][TT];
        float xs[U][TT], ws[U][RR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = min(g0 + u * NW, G - 1);
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                w[u][rr] = load_operand(qp[rr] + (size_t)g * kFp8Block, qp[rr] + (size_t)g * kFp8Block + 1024);
                ws[u][rr] = sp[rr][g];
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                x[u][tt] = load_operand(xp[tt] + (size_t)g * kGroup, xp[tt] + (size_t)g * kGroup + 64);
                xs[u][tt] = xsp[tt][g];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g0 + u * NW < G) {
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr) {
                        const f4 p = mfma_fp8(w[u][rr], x[u][tt]);
                        const float s = xs[u][tt] * ws[u][rr];
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[tt][rr][i] = fmaf(p[i], s, acc[tt][rr][i]);
                    }
            }
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) red[wave][tt * RR + rr][lane] = acc[tt][rr];
    __syncthreads();
    if (wave >= NT) return;
    const int rt = rt0 + wave % RR;
    if (rt >= nt16) return;
    f4 v = red[0][wave][lane];
#pragma unroll
    for (int k = 1; k < NW; ++k) v += red[k][wave][lane];
    const int j = wk.j0 + 16 * (wave / RR) + (lane & 15);
    const bool ok = j < wk.j1;
    if (args.r > 0) {
        const int r = args.r, arow = rt * 16 + (lane & 15);
        const _Float16* A = M.a + (EXPERTS ? (size_t)wk.e * M.a_step : 0);
        int at[1] = {ok ? j : wk.j0}, t[1];
        tokens_of<EXPERTS>(args, at, t);
        const int ri = EXPERTS && args.r_by_token ? t[0] : at[0];
        const h8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int kb = 0; kb < args.rp / 32; ++kb) {
            const int col = 32 * kb + 8 * (lane >> 4);
            const h8 av = (arow < M.n_out && col < r) ? load_h8(A + (size_t)arow * r + col) : zero8;
            v = mfma16(av, r_columns(args, ri, col), v);
        }
    }
    if (ok) store_rows(M, j, rt * 16 + 4 * (lane >> 4), v);
}

// --------------------------------------------------------------------- product, tiles
// 16 TT WM tokens x 64 WN rows per workgroup: WM x WN wavefronts, each 16 TT tokens x 4 row tiles.
// The token codes of an input group (128 bytes a token) go memory -> LDS by the load unit into a ring of four stages, two
// groups ahead, with one barrier for two groups; a wavefront's weight operands come straight into registers, WA groups
// ahead (with WM = 2 the two wavefronts that share rows find them in the L1 cache), so that LDS carries only the codes and
// scales.  A token's scales of four groups come as one 16-byte piece through LDS; the scale of the wavefront's 64 rows (one
// 128-row block) is a lane of a register.
// A group's sums leave the matrix core into four registers a tile and are added, scaled, while the next
// steps run: per step 4 additions to 32 cycles of matrix core, which two wavefronts a SIMD overlap.
// In a stage, row r keeps its 16-byte piece c at position c ^ f(r), f(r) = (r / 2) ^ ((r / 4 ^ r / 8) % 2).  LDS serves
// a 16-byte read 16 lanes at a time: rows 0-3 and 12-15 of one piece with rows 4-11 of its neighbour, then the others.
// Rows of one parity share a half of the banks, and f puts the eight of them at eight places: the operands' reads are free of
// conflicts.  Those that the counters show (0.19 of the access cycles) are 0.15 of the scales' reads, 4 bytes by each of 16 lanes,
// and 0.04 of the results' way out; without the scales' reads the call takes the same time.
// Groups past the workgroup's range repeat the last one with a scale of zero; token rows past the block repeat its last
// row and row tiles past the module its last tile, neither is stored.
//
// Where the tiles do not fill the GPU, KH such teams of WM x WN wavefronts share a workgroup: each takes a part of the
// input groups through a ring of its own, the sums meet in LDS, and a team finishes TT / KH of the token
// tiles.  With args.ks > 1 the input groups are split over workgroups too: each writes its fp32 tile to the
// workspace, and fp8_tile_join_kernel adds them in order and finishes.
//
// What bounds 128 x 256 tiles at T = 2048, 2 x 11008 <- 4096 (matrix cores busy 0.67 of the cycles): the loads'
// issue and return beside the matrix cores (the call, 198 us, without the codes' loads 180, without the weights' 142, without
// both 127; scaling costs nothing), and 2.7 tiles a slot.  256 x 256 on eight wavefronts took the same, 128 x 128 a fifth more.
typedef __attribute__((address_space(3))) void lds_void;
template <int I>
using ic = std::integral_constant<int, I>;

// Column of the launch (row block of a module and K range) and token block of a workgroup: XCD x (workgroups b with
// b % 8 == x) takes the columns x, x + 8, ..., eight token blocks at a time, so that a column's weights stay in one L2
// and its workgroups run together.
__device__ __forceinline__ bool tile_place(const Fp8Args& args, int block, int& mb, int& col) {
    const int cols = args.row_blocks * args.ks;
    const int xcd = block & 7, local = block >> 3;
    const int mine = (cols - xcd + 7) >> 3;  // columns of this XCD
    if (mine <= 0) return false;
    const int per = 8 * mine;
    const int ms = local / per, in = local - ms * per;
    const int width = min(8, args.m_blocks - 8 * ms);
    if (width <= 0) return false;
    const int c = in / width;
    if (c >= mine) return false;
    mb = 8 * ms + (in - c * width);
    col = xcd + 8 * c;
    return true;
}

enum : int { kFp8Plain = 0, kFp8Correct = 1, kFp8Split = 2 };  // what follows the sums

template <int WM, int WN, int TT, int KH, int MODE, bool EXPERTS>
__global__ __launch_bounds__(64 * WM * WN * KH, 2) void fp8_tile_kernel(const Fp8Args args, const Fp8PrepArgs prep,
                                                                       int join_blocks) {
    constexpr int RR = 4, NW = WM * WN, BM = 16 * TT * WM, SB = BM * 128;
    constexpr int NC = BM / 8 / NW;        // 1 KB code copies per wavefront and group
    constexpr int TE = TT / KH;            // token tiles that a wavefront finishes
    constexpr int NE = BM / 8 / (NW * KH); // copies per wavefront of a stage that all fill
    constexpr int WA = TT <= 4 ? 3 : 1;    // groups that the weights are ahead, as registers allow
    constexpr int WS = WA + 1;             // register slots of a group's weights
    static_assert(NC * 8 * NW == BM && NC % 2 == 0 && BM % 64 == 0 && NE > 0 && TE * KH == TT, "copies");
    __shared__ __attribute__((aligned(16))) uint8_t st0[KH * SB];
    __shared__ __attribute__((aligned(16))) uint8_t st1[KH * SB];
    __shared__ __attribute__((aligned(16))) uint8_t st2[KH * SB];
    __shared__ __attribute__((aligned(16))) uint8_t st3[KH * SB];
    // scales [token][4 groups] of a turn of the ring, for its first two groups and for its last two: an array is filled
    // while the other is read
    __shared__ __attribute__((aligned(16))) uint8_t sc0[KH * BM * 16];
    __shared__ __attribute__((aligned(16))) uint8_t sc1[KH * BM * 16];
    // With a K split the projection is only used by the launch after this one: the first workgroups (a
    // multiple of 8) join its ranges instead of a launch of their own
    if constexpr (MODE == kFp8Split) {
        if ((int)blockIdx.x < join_blocks) {
            join_ranges(prep, (size_t)blockIdx.x * (64 * NW * KH) + threadIdx.x);
            return;
        }
    }
    Work wk;
    int kr = 0, mb = 0;
    if constexpr (EXPERTS) {
        if (!expert_work(args, BM, args.row_blocks, blockIdx.x, true, wk)) return;
    } else {
        int col;
        if (!tile_place(args, (int)blockIdx.x - join_blocks, mb, col)) return;
        const int ks = MODE == kFp8Split ? args.ks : 1;
        wk.e = 0;
        wk.rb = col / ks;
        kr = col - wk.rb * ks;
        wk.j0 = mb * BM;
        wk.j1 = min(wk.j0 + BM, args.T);
    }
    const Fp8Module& M = args.mod[fp8_module_of(args, wk.rb)];
    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int kh = KH > 1 ? wave_all / NW : 0, wave = KH > 1 ? wave_all % NW : wave_all;  // team, wavefront of it
    const int wm = wave % WM, wn = wave / WM;
    const int d = args.d, NT = M.n_tiles16, n_out = M.n_out;
    const uint8_t* q = M.q + (EXPERTS ? (size_t)wk.e * M.q_step : 0);
    const int j0 = wk.j0, j1 = wk.j1, rt0 = (wk.rb - M.block_begin) * RR * WN + wn * RR;
    // groups of the workgroup, and the KH-th part of them, whole turns of the ring, that this team takes (the last may be
    // shorter, or none)
    const int n_all = min(args.gk, args.G - kr * args.gk), n_turn = ((n_all + KH - 1) / KH + 3) & ~3;
    const int g_begin = kr * args.gk + kh * n_turn, n_g = max(0, min(n_turn, n_all - kh * n_turn));
    const int g_last = min(g_begin + max(n_g, 1), args.G) - 1;
    // copy i of wave w fills rows 8 (NC w + i) .. + 7 of the stage; lane l lands at row + l / 8, position l % 8, which
    // holds the row's piece (l % 8) ^ f(row)
    // (the last entry: the token row whose scales the lane copies)
    uint32_t xoff[NC], soff;
    {
        int rows[NC + 1], tok[NC + 1];
#pragma unroll
        for (int i = 0; i < NC; ++i) rows[i] = min(j0 + 8 * (NC * wave + i) + (lane >> 3), j1 - 1);
        rows[NC] = min(j0 + 64 * (wave % (BM / 64)) + lane, j1 - 1);
        tokens_of<EXPERTS>(args, rows, tok);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int row = 8 * (NC * wave + i) + (lane >> 3);
            xoff[i] = (uint32_t)tok[i] * (uint32_t)d + 16 * (uint32_t)((lane & 7) ^ ((row >> 1) & 7) ^ (((row >> 2) ^ (row >> 3)) & 1));
        }
        soff = (uint32_t)tok[NC] * (uint32_t)args.gp * 4u;
    }
    const int lr = lane & 15, fr = (lr >> 1) ^ (((lr >> 2) ^ (lr >> 3)) & 1);
    const int rbase = (16 * TT * wm + lr) * 128;
    int rofs0 = rbase + 16 * ((lane >> 4) ^ fr), rofs1 = rbase + 16 * ((4 + (lane >> 4)) ^ fr);
    int sofs = (kh * BM + 16 * TT * wm + lr) * 16;
    uint32_t rts[RR];  // the wavefront's row tiles (scalar: weight addresses are scalar but for the lane's 16 bytes)
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) rts[rr] = (uint32_t)min(rt0 + rr, NT - 1);
    const uint32_t lofs = lane * 16;
    float wsc[2];  // scales of the wavefront's 128-row block, group g_begin + 64 i + lane
    {
        const float* sz = M.sz + (EXPERTS ? (size_t)wk.e * M.sz_step : 0) + (size_t)(rts[0] >> 3) * args.G;
#pragma unroll
        for (int i = 0; i < 2; ++i) wsc[i] = 64 * i + lane < n_g ? sz[g_begin + 64 * i + lane] : 0.f;
    }

    auto copy = [&](int v, uint8_t* stg, int i) {
        const uint8_t* base = args.xq + (size_t)min(g_begin + v, g_last) * kGroup;
        asm volatile("" : "+v"(xoff[i]));  // one register each: not widened to 64 bits in front of the loop
        __builtin_amdgcn_global_load_lds((const void*)(base + xoff[i]), (lds_void*)(stg + kh * SB + 8 * (NC * wave + i) * 128),
                                         16, 0, 0);
    };
    // scales of the groups v .. v + 3 (g_begin and v are multiples of 4; past the row's end the last four again)
    auto copy_scales = [&](int v, uint8_t* sc) {
        asm volatile("" : "+v"(soff));
        const uint8_t* base = reinterpret_cast<const uint8_t*>(args.xs) + (size_t)min(g_begin + v, args.gp - 4) * 4u;
        __builtin_amdgcn_global_load_lds((const void*)(base + soff),
                                         (lds_void*)(sc + (kh * BM + 64 * (wave % (BM / 64))) * 16), 16, 0, 0);
    };
    i8v w[WS][RR];
    auto wload = [&](int v, int slot, int rr) {
        const uint8_t* at = q + ((size_t)rts[rr] * args.G + min(g_begin + v, g_last)) * kFp8Block + lofs;
        w[slot][rr] = load_operand(at, at + 1024);
    };
    f4 acc[TT][RR];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = f4{0.f, 0.f, 0.f, 0.f};

    copy_scales(0, sc0);
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i) copy(i / NC, i < NC ? st0 : st1, i % NC);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < WA * RR; ++i) wload(i / RR, i / RR, i % RR);
    __builtin_amdgcn_sched_barrier(0);

    // Groups v and v + 1 in the stages S = v % 4 and S + 1.  At the barrier their copies have landed, and the scales.  The
    // copies of v + 2 and v + 3 go to stages whose last reads were before this barrier, and so do the scales (at S = 0
    // this turn's for its last two groups, at S = 2 the next turn's for its first two); operands go to slots whose last
    // steps were issued.  Loads are requested a few with each tile: a burst of
    // them fills the load unit's queue, and a wavefront that waits there issues no matrix-core steps either (2 x 11008 <- 4096
    // at T = 2048, the whole call: 200 us with them all at the start of a group, 190 so).
    // The waits count the loads behind the one that is due, so that none may move: the barriers keep the
    // order under any scheduling.
    // A tile's sums are added just before their registers take the next tile's, the last ones after the next barrier.
    f4 p[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) p[rr] = f4{0.f, 0.f, 0.f, 0.f};
    float last = 0.f;
    auto wait_for = [](auto Nc) {  // vmcnt(N)
        constexpr int N = decltype(Nc)::value;
        static_assert(N < 64, "vmcnt");
        __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
    };
    auto scale_of = [&](int v) {
        return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v < 64 ? wsc[0] : wsc[1]), v & 63));
    };
    auto step = [&](int v, auto Sc) {
        constexpr int S = decltype(Sc)::value;
        uint8_t* const st[4] = {st0, st1, st2, st3};
        asm volatile("" : "+v"(rofs0), "+v"(rofs1), "+v"(sofs));  // no addresses for every stage in front of the loop
        const uint8_t* sc = (S == 0 ? sc0 : sc1) + sofs;
        // WA == 1, tiles 0 .. 15: weights of v + 1 with the tiles 0 .. 3, copies with 4 .. 7, weights of v + 2 with 8 .. 11.
        // WA == 3, tiles 0 .. 7: copies with the tiles 0 .. 3, weights of v + 3 with 0 .. 3, of v + 4 with 4 .. 7.
        auto request = [&](auto Ic) {
            constexpr int I = decltype(Ic)::value, C0 = WA == 1 ? 4 : 0;
            if constexpr (I == C0) copy_scales(S == 0 ? v : v + 2, S == 0 ? sc1 : sc0);
            if constexpr (I >= C0 && I < C0 + 4) {
#pragma unroll
                for (int i = 2 * NC / 4 * (I - C0); i < 2 * NC / 4 * (I - C0 + 1); ++i)
                    copy(v + 2 + i / NC, st[(S + 2 + i / NC) & 3], i % NC);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (I < 4) wload(v + WA, (S + WA) % WS, I);
            else if constexpr (I >= TT && I < TT + 4) wload(v + 1 + WA, (S + 1 + WA) % WS, I - TT);
            __builtin_amdgcn_sched_barrier(0);
        };
        static_assert(RR == 4 && NC % 2 == 0, "requests with four tiles");
        wait_for(ic<WA == 1 ? 2 * RR : 2 + 2 * RR>{});  // the copies: behind them the weights of v, or of v + 2
        __builtin_amdgcn_s_barrier();
        if constexpr (WA == 1) wait_for(ic<0>{});       // the weights of v, the last that were requested
        __builtin_amdgcn_sched_barrier(0);
        const float sw[2] = {scale_of(v), scale_of(v + 1)};
        i8v x[2];
        float s[2];
        auto xread = [&](int i) {
            const uint8_t* at = st[S + i / TT] + kh * SB + (i % TT) * 2048;
            x[i % 2] = load_operand(at + rofs0, at + rofs1);
            s[i % 2] = *reinterpret_cast<const float*>(sc + (i % TT) * 256 + 4 * (S + i / TT));
        };
        xread(0);
        auto tile = [&](auto Ic) {
            constexpr int I = decltype(Ic)::value;
            if constexpr (I == TT) wait_for(ic<1 + 2 * NC + (WA == 1 ? 0 : 4 * RR)>{});  // the weights of v + 1
            request(Ic);
            if constexpr (I + 1 < 2 * TT) xread(I + 1);
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                f4& sum = acc[(I + TT - 1) % TT][rr];
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[e] = fmaf(p[rr][e], last, sum[e]);
                p[rr] = mfma_fp8(w[(S + I / TT) % WS][rr], x[I % 2]);
            }
            last = s[I % 2] * sw[I / TT];
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        tile(ic<0>{});
        tile(ic<1>{});
        tile(ic<2>{});
        tile(ic<3>{});
        tile(ic<4>{});
        tile(ic<5>{});
        tile(ic<6>{});
        tile(ic<7>{});
        if constexpr (TT == 8) {
            tile(ic<8>{});
            tile(ic<9>{});
            tile(ic<10>{});
            tile(ic<11>{});
            tile(ic<12>{});
            tile(ic<13>{});
            tile(ic<14>{});
            tile(ic<15>{});
        }
    };
    // whole turns of the ring; steps past the range only keep time
    for (int v = 0; v < n_turn; v += 4) {
        step(v, ic<0>{});
        step(v + 2, ic<2>{});
    }
#pragma unroll
    for (int rr = 0; rr < RR; ++rr)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[TT - 1][rr][e] = fmaf(p[rr][e], last, acc[TT - 1][rr][e]);
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no copy may land in LDS after this
    __syncthreads();
    // Team kh finishes token tiles TE kh .. + TE - 1: the others' sums of them come through LDS, past the
    // first SB bytes of the stages (those are R's).
    if constexpr (KH > 1) {
        constexpr int kPiece = TE * RR * 1024, kStage = (KH - 1) * SB / kPiece;
        static_assert(kStage * kPiece == (KH - 1) * SB && 4 * kStage == KH * NW * (KH - 1), "sums fill the stages");
        auto piece_at = [&](int to, int from) {
            const int at_ = (to * NW + wave) * (KH - 1) + (from - to + KH) % KH - 1, at = at_ / kStage;
            return (at == 0 ? st0 : (at == 1 ? st1 : (at == 2 ? st2 : st3))) + SB + (at_ % kStage) * kPiece + 16 * lane;
        };
#pragma unroll
        for (int to = 0; to < KH; ++to)
            if (to != kh) {
                uint8_t* dst = piece_at(to, kh);
#pragma unroll
                for (int i = 0; i < TE * RR; ++i) *reinterpret_cast<f4*>(dst + 1024 * i) = acc[to * TE + i / RR][i % RR];
            }
        f4 own[TE][RR];
#pragma unroll
        for (int to = 0; to < KH; ++to)
            if (to == kh) {
#pragma unroll
                for (int i = 0; i < TE * RR; ++i) own[i / RR][i % RR] = acc[to * TE + i / RR][i % RR];
            }
        __syncthreads();
        // added in the order of the teams, whichever finishes
#pragma unroll
        for (int i = 0; i < TE * RR; ++i) {
            f4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < KH; ++k)
                sum += k == kh ? own[i / RR][i % RR] : *reinterpret_cast<const f4*>(piece_at(kh, k) + 1024 * i);
            acc[i / RR][i % RR] = sum;
        }
    }
    if constexpr (MODE == kFp8Split) {
        f4* part = reinterpret_cast<f4*>(args.part) +
                   ((((size_t)mb * args.row_blocks + wk.rb) * args.ks + kr) * NW + wave) * (TT * RR * 64) + kh * (TE * RR * 64);
#pragma unroll
        for (int tt = 0; tt < TE; ++tt)
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) part[(tt * RR + rr) * 64 + lane] = acc[tt][rr];
        return;
    }
    const int te0 = TT * wm + TE * kh;  // first of the wavefront's token tiles
    // The correction: R's columns 64 j .. + 63 (128 bytes a token, as a group of codes) go to stage j (r <= 256), A's
    // operands to registers.  Rows of A past the module and token rows past the block repeat the last one
    // (their results are not stored); columns of A past r are taken as zero, R's are zero up to rp, a multiple of 64.
    if constexpr (MODE == kFp8Correct) {
        const int r = args.r, rp = args.rp;
        int rrow[NE];  // rows of R that the lane copies
        {
            int rows[NE], tok[NE], first = j0;
            asm volatile("" : "+s"(first));  // found again: the codes' rows are not kept over the loop (they spilled)
#pragma unroll
            for (int i = 0; i < NE; ++i) rows[i] = min(first + 8 * (NE * wave_all + i) + (lane >> 3), j1 - 1);
            tokens_of<EXPERTS>(args, rows, tok);
#pragma unroll
            for (int i = 0; i < NE; ++i) rrow[i] = EXPERTS && args.r_by_token ? tok[i] : rows[i];
        }
        auto rcopy = [&](int j, uint8_t* stg) {
            if (64 * j >= rp) return;
            // R as the K ranges' fp32 sums: added in order, rounded once to fp16 here (teams without a K split; the launchers
            // refuse it elsewhere)
            if constexpr (KH > 1) {
                if (args.r_ranges > 0) {
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        const int row = 8 * (NE * wave_all + i) + (lane >> 3), c = lane & 7;
                        *reinterpret_cast<h8*>(stg + row * 128 + 16 * (c ^ ((row >> 1) & 7) ^ (((row >> 2) ^ (row >> 3)) & 1))) =
                            r_columns(args, rrow[i], 64 * j + 8 * c);
                    }
                    return;
                }
            }
            const uint8_t* base = static_cast<const uint8_t*>(args.R) + 128 * j;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int row = 8 * (NE * wave_all + i) + (lane >> 3);
                const int piece = (lane & 7) ^ ((row >> 1) & 7) ^ (((row >> 2) ^ (row >> 3)) & 1);
                __builtin_amdgcn_global_load_lds((const void*)(base + (size_t)rrow[i] * rp * 2 + 16 * piece),
                                                 (lds_void*)(stg + 8 * (NE * wave_all + i) * 128), 16, 0, 0);
            }
        };
        const uint8_t* Ab = reinterpret_cast<const uint8_t*>(M.a + (EXPERTS ? (size_t)wk.e * M.a_step : 0)) + (size_t)rts[0] * 32 * r;
        rcopy(0, st0);
        rcopy(1, st1);
        rcopy(2, st2);
        rcopy(3, st3);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        int j = 0;
#pragma unroll 1
        do {
            const uint8_t* cur = j == 0 ? st0 : (j == 1 ? st1 : (j == 2 ? st2 : st3));
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int c = 64 * j + 32 * m + 8 * (lane >> 4);
                h8 av[RR];
#pragma unroll
                for (int rr = 0; rr < RR; ++rr) {
                    const uint32_t row = (uint32_t)min((rt0 + rr) * 16 + lr, n_out - 1) - rts[0] * 16;
                    const u4 bits = *reinterpret_cast<const u4*>(Ab + (row * (uint32_t)r + (uint32_t)min(c, r - 8)) * 2u);
                    av[rr] = __builtin_bit_cast(h8, c < r ? bits : u4{0u, 0u, 0u, 0u});
                }
#pragma unroll
                for (int tt = 0; tt < TE; ++tt) {
                    const h8 xv = *reinterpret_cast<const h8*>(cur + (m == 0 ? rofs0 : rofs1) + (TE * kh + tt) * 2048);
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = mfma16(av[rr], xv, acc[tt][rr]);
                }
            }
        } while (64 * ++j < rp);
    }
    // To memory through the wavefront's own part of the (finished) ring: [16 TE tokens][64 rows] fp16, a token's eight
    // 16-byte pieces p at p ^ (token % 8), then whole 128-byte lines.
    __syncthreads();
    constexpr int kPart = 16 * TE * 128, kPer = SB / kPart;
    static_assert(NW * KH * kPart <= 4 * SB && SB % kPart == 0, "a part per wavefront");
    const int sel = wave_all / kPer;
    uint8_t* out = (sel == 0 ? st0 : (sel == 1 ? st1 : (sel == 2 ? st2 : st3))) + (wave_all % kPer) * kPart;
#pragma unroll
    for (int tt = 0; tt < TE; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) {
            const f4 v = acc[tt][rr];
            const h2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
            const int p = 2 * rr + (lane >> 5);
            *reinterpret_cast<u2*>(out + (16 * tt + lr) * 128 + 16 * (p ^ (lane & 7)) + 8 * ((lane >> 4) & 1)) =
                u2{as_u32(lo), as_u32(hi)};
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int row0 = rt0 * 16 + 8 * (lane & 7);
    const bool vec = (n_out & 7) == 0 && row0 + 7 < n_out;
#pragma unroll 4
    for (int i = 0; i < 2 * TE; ++i) {
        const int tl = 8 * i + (lane >> 3), j = j0 + 16 * te0 + tl;
        const uint8_t* piece = out + tl * 128 + 16 * ((lane & 7) ^ (tl & 7));
        if (j >= j1) continue;
        _Float16* y = M.y + (size_t)j * n_out + row0;
        if (vec) *reinterpret_cast<h8*>(y) = *reinterpret_cast<const h8*>(piece);
        else {
#pragma unroll 1
            for (int e = 0; e < min(8, n_out - row0); ++e) y[e] = reinterpret_cast<const _Float16*>(piece)[e];
        }
    }
}

// Sums of the K ranges of one 16-token x 64-row piece per wavefront (pieces numbered as the tile kernel stores
// them), in order, correction, one rounding to fp16.
template <int WM, int WN, int TT>
__global__ __launch_bounds__(256) void fp8_tile_join_kernel(const Fp8Args args, int pieces) {
    constexpr int RR = 4, NW = WM * WN;
    const int lane = threadIdx.x & 63;
    const int piece = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (piece >= pieces) return;
    const int ks = args.ks, cols = args.row_blocks;
    const int tt = piece % TT, wave = piece / TT % NW, tile = piece / TT / NW;
    const int mb = tile / cols, rb = tile - mb * cols;
    const Fp8Module& M = args.mod[fp8_module_of(args, rb)];
    const int rt0 = (rb - M.block_begin) * RR * WN + (wave / WM) * RR;
    const int t = (mb * WM + wave % WM) * 16 * TT + 16 * tt + (lane & 15);
    if (rt0 >= M.n_tiles16) return;
    const bool ok = t < args.T;
    const f4* part = reinterpret_cast<const f4*>(args.part);
    f4 v[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) v[rr] = f4{0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < ks; ++k) {
        const f4* p = part + ((((size_t)tile * ks + k) * NW + wave) * TT + tt) * (RR * 64) + lane;
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) v[rr] += p[rr * 64];
    }
    if (args.r > 0) {
        const int r = args.r, rp = args.rp;
        const h8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int kb = 0; kb < rp / 32; ++kb) {
            const int c = 32 * kb + 8 * (lane >> 4);
            const h8 bv = load_h8(static_cast<const _Float16*>(args.R) + (size_t)(ok ? t : 0) * rp + c);
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                const int row = (rt0 + rr) * 16 + (lane & 15);
                const h8 av = (row < M.n_out && c < r) ? load_h8(M.a + (size_t)row * r + c) : zero8;
                v[rr] = mfma16(av, bv, v[rr]);
            }
        }
    }
    if (!ok) return;
#pragma unroll
    for (int rr = 0; rr < RR; ++rr)
        if (rt0 + rr < M.n_tiles16) store_rows(M, t, (rt0 + rr) * 16 + 4 * (lane >> 4), v[rr]);
}

}  // namespace

hipError_t launch_repack_fp8(const uint8_t* codes, const float* scales, int64_t n_out, int64_t k_in, uint8_t* q, float* sz,
                             int32_t* flag, hipStream_t stream) {
    const int64_t nt = ceil_div(n_out, 16), G = k_in / kGroup;
    hipLaunchKernelGGL(repack_fp8_kernel, dim3((unsigned)(nt * G)), dim3(128), 0, stream, codes, n_out, k_in, (int)G, q, flag);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = ceil_div(n_out, 128) * G, n_pad = (int64_t)fp8_sz_bytes(n_out, k_in) / 4;
    hipLaunchKernelGGL(repack_fp8_scales_kernel, dim3((unsigned)ceil_div(n_pad, 256)), dim3(256), 0, stream, scales, n, n_pad, sz,
                       flag);
    return hipGetLastError();
}

// Four groups of loads in flight per thread from here on, else one (the call on 128 rows, four and one: T = 8000, d = 4096,
// r = 64 72 and 75 us, T = 4096 58.7 and 59.5, T = 2048 33 and 33; r = 0, T = 2048 17.7 and 16.3).
constexpr int64_t kQuantWide = (int64_t)1 << 24;  // inputs

template <int TT, int NJ, int U>
static void launch_fp8_prep_n(const Fp8PrepArgs& a, const Fp8Args* experts, int64_t row_blocks, hipStream_t stream) {
    const int64_t cols = ceil_div(a.rp / 16, NJ);
    const int64_t proj = a.r > 0 ? (experts != nullptr ? 8 * ceil_div(row_blocks * cols, 8) : ceil_div(a.T, 16 * TT) * cols) * a.ks : 0;
    const dim3 grid((unsigned)(proj + ceil_div((int64_t)a.T * a.d / 8, U * kPrepThreads))), block(kPrepThreads);
    if (experts == nullptr) {
        if constexpr (TT <= 2) hipLaunchKernelGGL((fp8_prep_kernel<TT, NJ, U>), grid, block, 0, stream, a, (int)proj);
    } else if constexpr (TT > 1 || NJ == 1) {
        hipLaunchKernelGGL((fp8_prep_experts_kernel<TT, NJ, U>), grid, block, 0, stream, a, *experts, (int)proj);
    }
}

template <int TT, int NJ>
static void launch_fp8_prep_t(const Fp8PrepArgs& a, const Fp8Args* experts, int64_t row_blocks, hipStream_t stream) {
    if ((int64_t)a.T * a.d >= kQuantWide) launch_fp8_prep_n<TT, NJ, 4>(a, experts, row_blocks, stream);
    else launch_fp8_prep_n<TT, NJ, 1>(a, experts, row_blocks, stream);
}

hipError_t launch_fp8_prep(const Fp8PrepArgs& a, int tt, int nj, bool join, const Fp8Args* experts, int64_t row_blocks,
                           hipStream_t stream) {
    if (a.d % kGroup != 0) return hipErrorInvalidValue;
    if (experts != nullptr ? tt == 1 && nj == 4 : tt == 4) return hipErrorInvalidValue;
    if (tt == 4) launch_fp8_prep_t<4, 4>(a, experts, row_blocks, stream);
    else if (nj == 1) launch_fp8_prep_t<1, 1>(a, experts, row_blocks, stream);
    else if (tt == 1) launch_fp8_prep_t<1, 4>(a, experts, row_blocks, stream);
    else launch_fp8_prep_t<2, 4>(a, experts, row_blocks, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.r == 0 || a.part == nullptr || !join) return e;
    hipLaunchKernelGGL(fp8_join_kernel, dim3((unsigned)ceil_div((int64_t)a.T * a.rp / 4, 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <bool EXPERTS>
static hipError_t launch_fp8_split(const Fp8Args& a, int64_t items, hipStream_t stream) {
    const dim3 grid((unsigned)items), block(64 * kFp8Waves);
    switch (a.tt * 4 + a.rr) {
        case 4 + 1: hipLaunchKernelGGL((fp8_split_kernel<1, 1, EXPERTS>), grid, block, 0, stream, a); break;
        case 8 + 2: hipLaunchKernelGGL((fp8_split_kernel<2, 2, EXPERTS>), grid, block, 0, stream, a); break;
        case 16 + 2: hipLaunchKernelGGL((fp8_split_kernel<4, 2, EXPERTS>), grid, block, 0, stream, a); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

// Every XCD takes an eighth of the work, rounded up; workgroups without any return at once.
template <int WM, int WN, int TT>
static hipError_t launch_fp8_experts(const Fp8Args& a, const Fp8PrepArgs& p, int64_t items, hipStream_t stream) {
    if (a.r_ranges > 0) return hipErrorInvalidValue;  // projections come as R
    const dim3 grid((unsigned)(8 * ceil_div(items, 8))), block(64 * WM * WN);
    if (a.r > 0) hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, TT, 1, kFp8Correct, true>), grid, block, 0, stream, a, p, 0);
    else hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, TT, 1, kFp8Plain, true>), grid, block, 0, stream, a, p, 0);
    return hipGetLastError();
}

// SPLIT: the tile is used with K ranges; WHOLE: without.
template <int WM, int WN, int TT, int KH, bool SPLIT, bool WHOLE>
static hipError_t launch_fp8_tile(const Fp8Args& a, const Fp8PrepArgs& p, hipStream_t stream) {
    const int64_t join = a.ks > 1 && a.r > 0 && p.part != nullptr
                             ? ceil_div(ceil_div((int64_t)p.T * p.rp / 4, 64 * WM * WN * KH), 8) * 8 : 0;
    const int64_t grid = join + 8 * ceil_div((int64_t)a.row_blocks * a.ks, 8) * a.m_blocks;
    if (grid * 64 * WM * WN * KH > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
    if (a.r_ranges > 0 && (KH == 1 || a.ks > 1)) return hipErrorInvalidValue;  // the projection comes as R
    const dim3 g((unsigned)grid), block(64 * WM * WN * KH);
    if constexpr (SPLIT) {
        if (a.ks > 1) {
            hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, TT, KH, kFp8Split, false>), g, block, 0, stream, a, p, (int)join);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const int pieces = a.m_blocks * a.row_blocks * WM * WN * TT;
            hipLaunchKernelGGL((fp8_tile_join_kernel<WM, WN, TT>), dim3((unsigned)ceil_div(pieces, 4)), dim3(256), 0, stream, a,
                               pieces);
            return hipGetLastError();
        }
    }
    if constexpr (WHOLE) {
        if (a.ks > 1) return hipErrorInvalidValue;
        if (a.r > 0) hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, TT, KH, kFp8Correct, false>), g, block, 0, stream, a, p, 0);
        else hipLaunchKernelGGL((fp8_tile_kernel<WM, WN, TT, KH, kFp8Plain, false>), g, block, 0, stream, a, p, 0);
        return hipGetLastError();
    }
    return hipErrorInvalidValue;
}

hipError_t launch_fp8(const Fp8Args& a, const Fp8PrepArgs& p, int64_t items, hipStream_t stream) {
    if (a.offsets != nullptr) {
        if (a.rr == 16) return launch_fp8_experts<1, 4, 8>(a, p, items, stream);
        return launch_fp8_split<true>(a, items, stream);
    }
    if (a.rr == 16) return launch_fp8_tile<1, 4, 8, 1, false, true>(a, p, stream);
    if (a.rr == 8 && a.tt == 8)
        return a.kh == 2 ? launch_fp8_tile<2, 2, 4, 2, true, false>(a, p, stream) : launch_fp8_tile<2, 2, 4, 1, false, true>(a, p, stream);
    if (a.rr == 8) return launch_fp8_tile<1, 2, 4, 4, true, true>(a, p, stream);
    return launch_fp8_split<false>(a, items, stream);
}

}  // namespace glowq
