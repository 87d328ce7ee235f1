// Group forward on 8-bit integer weights and activations: one fp32 scale per output channel, one
// per token, the product on the gfx950 int8 matrix cores, the low-rank correction on the fp16
// activations (the 8-bit-activation rows of the GlowQ arXiv page, Tables 14 and 15, with 8-bit
// weights).
//
//   s_t = max_k |x[t, k]| / 127,  c[t, k] = clamp(round_half_even(x[t, k] / s_t), -127, 127)   (fp32)
//   y_i[t, o] = s_t s_i[o] sum_k c[t, k] q_i[o, k] + R[t] . A_i[o],   R = X B^T from the fp16 X
//
// |sum| <= 16384 x 127 x 128 < 2^31, so the int32 sums are exact in any order: K may be split over
// wavefronts and workgroups without changing a bit.  A token with an infinity or a NaN has scale
// NaN, and so a row of NaN.
//
// Weight layout: G x NT blocks of 2048 bytes, block (g, rt) at (g NT + rt) 2048 holding rows
// 16 rt .. + 15 and inputs 128 g .. + 127 as two 1024-byte operands of v_mfma_i32_16x16x64_i8:
// operand m, lane l (16 bytes at 1024 m + 16 l) is row 16 rt + l % 16, inputs 128 g + 64 m +
// 16 (l / 16) .. + 15.  Scales: 16 fp32 per row tile.  Rows >= n_out are zero.
// Activation codes lie in their natural order [T][d]; its 16-byte pieces are the other operand.
#include <algorithm>
#include <type_traits>

#include "glowq_internal.h"
#include "w8a8.h"

namespace glowq {

typedef int32_t i4v __attribute__((ext_vector_type(4)));

namespace {

__device__ __forceinline__ i4v mfma_i8(i4v a, i4v b, i4v c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Four consecutive rows of token t, rounded to fp16.
__device__ __forceinline__ void store_rows(const ModuleArgs& M, int t, int row0, const f4& v) {
    _Float16* yrow = M.y + (size_t)t * M.n_out;
    if ((M.n_out & 3) == 0 && row0 + 3 < M.n_out) {
        const h2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
        *reinterpret_cast<u2*>(yrow + row0) = u2{as_u32(lo), as_u32(hi)};
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row0 + i < M.n_out) yrow[row0 + i] = (_Float16)v[i];
    }
}

// --------------------------------------------------------------------- load step
// One workgroup per (128-input group, row tile): 128 threads, each one lane's 16 bytes.
__global__ __launch_bounds__(128) void repack_w8_kernel(const int8_t* __restrict__ codes, int64_t n_out, int64_t k_in,
                                                        int nt, uint8_t* __restrict__ q) {
    const int64_t blk = blockIdx.x;  // g nt + rt
    const int64_t g = blk / nt, rt = blk - g * nt;
    const int m = threadIdx.x >> 6, l = threadIdx.x & 63;
    const int64_t row = 16 * rt + (l & 15);
    u4 v = {0u, 0u, 0u, 0u};
    if (row < n_out) v = *reinterpret_cast<const u4*>(codes + row * k_in + 128 * g + 64 * m + 16 * (l >> 4));
    *reinterpret_cast<u4*>(q + blk * kW8Block + 1024 * m + 16 * l) = v;
}

__global__ __launch_bounds__(256) void repack_w8_scales_kernel(const float* __restrict__ scales, int64_t n_out, int64_t n_pad,
                                                               float* __restrict__ sz, int32_t* __restrict__ flag) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n_pad) return;
    const float s = i < n_out ? scales[i] : 0.f;
    if (!(fabsf(s) < INFINITY)) __hip_atomic_store(flag, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sz[i] = s;
}

// --------------------------------------------------------------------- token codes and projection
// One launch, two kinds of workgroups (both read X, neither needs the other): first those of the
// projection R = X B^T, then those of the scales and codes (512 / TPT tokens each, a token's row in
// registers between its maximum and its codes, so that X is read once for them).
// What bounds it: up to some 40 tokens the launch and one load's latency (d = 4096, r = 64: 4.9 us for one token,
// 6.4 us for 37); then memory (T = 2048: 16.8 MB of X and 8.9 MB of codes, scales and sums, 15.2 us; X again by the
// projection's workgroups, out of the caches).
constexpr int kPrepThreads = 512;
constexpr int kPrepWaves = kPrepThreads / 64;
constexpr int kPrepChunks = 8;  // 8-input chunks per thread at most
constexpr int kPrepMaxD = 16384;

// round_half_even(x / scale), the quotient the IEEE one, of eight values as bytes.  u = x (1 / scale)
// is within 127 (2^-23 + 2^-24) < 2^-15 of it, so both round alike unless u lies that close to a tie;
// only then (one value in 10^4) the eight are divided.  |x| <= amax keeps every code in -127 .. 127.
// Adding 1.5 2^23 rounds to a whole number whose low byte is the code.
__device__ __forceinline__ u2 codes_of(const h8& x, float scale, float inv) {
    constexpr float kWhole = 12582912.0f;
    uint32_t f[8];
    float near = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = fmaf((float)x[e], inv, kWhole);
        near = fmaxf(near, fabsf(fmaf((float)x[e], inv, -(v - kWhole))));
        f[e] = __builtin_bit_cast(uint32_t, v);
    }
    if (__builtin_expect(near > 0.5f - 0x1p-14f, 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __builtin_bit_cast(uint32_t, (float)x[e] / scale + kWhole);
    }
    u2 w;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(f[4 * j + 3], f[4 * j + 2], 0x0c0c0400),
                                     __builtin_amdgcn_perm(f[4 * j + 1], f[4 * j], 0x0c0c0400), 0x05040100);
    return w;
}

// kPrepThreads / TPT tokens from t0 on: each by TPT threads with C chunks of eight
// inputs (TPT C >= d / 8): the largest magnitude (as fp16 bits, so that infinities and NaN order above
// every number), the scale, the codes.
template <int TPT, int C>
__device__ void quant_tokens(const _Float16* __restrict__ x, int t0, int T, int d, int8_t* __restrict__ xq,
                             float* __restrict__ xscale, uint32_t* red) {
    const int tid = threadIdx.x, sub = tid & (TPT - 1), t = t0 + tid / TPT;
    const int n8 = t < T ? d / 8 : 0;
    const _Float16* row = x + (size_t)min(t, T - 1) * d;
    h8 v[C];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = sub + TPT * i;
        v[i] = c < n8 ? load_h8(row + 8 * c) : h8{0, 0, 0, 0, 0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const u4 bits = __builtin_bit_cast(u4, v[i]) & 0x7FFF7FFFu;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(bits[e] & 0xFFFFu, bits[e] >> 16));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if constexpr (TPT > 64) {
        if ((tid & 63) == 0) red[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPT / 64; ++w) top = max(top, red[tid / TPT * (TPT / 64) + w]);
    }
    const float amax = (float)__builtin_bit_cast(_Float16, (uint16_t)top);
    const bool finite = top < 0x7C00u;
    const float scale = finite ? amax / 127.0f : __builtin_nanf("");  // IEEE division
    if (sub == 0 && t < T) xscale[t] = scale;
    const bool some = finite && scale > 0.f;
    const float inv = some ? 1.0f / scale : 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = sub + TPT * i;
        if (c < n8)
            *reinterpret_cast<u2*>(xq + (size_t)t * d + 8 * (size_t)c) =
                some ? codes_of(v[i], scale, inv) : u2{0u, 0u};
    }
}

// Sums of R over the 32-input steps [s_begin, s_end) for 16 TT tokens and 16 NJ rank columns: the
// wavefronts take steps in turn (U in flight) and add their tiles through LDS in wavefront order.
// part != nullptr: fp32 sums of this range to part [T][rp]; else one rounding to fp16 into R.
// Columns r .. r_pad - 1 are zero.
template <int TT, int NJ>
__device__ void project_tile(const PrepArgs& a, int tb, int jb, int s_begin, int s_end, float* part, f4* red) {
    constexpr int U = TT * NJ == 1 ? 8 : 4, N = TT * NJ;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int kofs = 8 * (lane >> 4), T = a.T, d = a.d, r = a.r, rp = a.rp;
    const _Float16 *xr[TT], *br[NJ];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) xr[tt] = a.x + (size_t)min(16 * (TT * tb + tt) + (lane & 15), T - 1) * d + kofs;
#pragma unroll
    for (int j = 0; j < NJ; ++j) br[j] = a.b + (size_t)min(16 * (NJ * jb + j) + (lane & 15), r - 1) * d + kofs;
    f4 acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = f4{0.f, 0.f, 0.f, 0.f};
    for (int s0 = s_begin + wave; s0 < s_end; s0 += U * kPrepWaves) {
        h8 xv[U][TT], bv[U][NJ];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = 32 * min(s0 + u * kPrepWaves, s_end - 1);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) xv[u][tt] = load_h8(xr[tt] + k);
#pragma unroll
            for (int j = 0; j < NJ; ++j) bv[u][j] = load_h8(br[j] + k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + u * kPrepWaves < s_end) {
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
    if (wave >= N) return;
    f4 v = red[wave * 64 + lane];
#pragma unroll
    for (int w = 1; w < H; ++w) v += red[(w * N + wave) * 64 + lane];
    const int col = 16 * (NJ * jb + wave % NJ) + (lane & 15);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 16 * (TT * tb + wave / NJ) + 4 * (lane >> 4) + i;
        const float o = col < r ? v[i] : 0.f;
        if (t < T && col < rp) {
            if (part != nullptr) part[(size_t)t * rp + col] = o;
            else a.R[(size_t)t * rp + col] = (_Float16)o;
        }
    }
}

// TPT: threads per token of the code workgroups.
template <int TT, int NJ, int TPT>
__global__ __launch_bounds__(kPrepThreads) void prep_kernel(const PrepArgs a, int proj_blocks) {
    __shared__ f4 red[kPrepWaves / 2 * TT * NJ * 64];
    int blk = blockIdx.x;
    if (blk >= proj_blocks) {
        constexpr int C = (kPrepMaxD / 8 + TPT - 1) / TPT < kPrepChunks ? (kPrepMaxD / 8 + TPT - 1) / TPT : kPrepChunks;
        quant_tokens<TPT, C>(a.x, (blk - proj_blocks) * (kPrepThreads / TPT), a.T, a.d, a.xq, a.xscale,
                             reinterpret_cast<uint32_t*>(red));
        return;
    }
    const int cols = (a.rp / 16 + NJ - 1) / NJ;
    const int k = blk % a.ks, rest = blk / a.ks, jb = rest % cols, tb = rest / cols;
    const int per = a.range / 32;
    project_tile<TT, NJ>(a, tb, jb, k * per, min((k + 1) * per, a.d / 32),
                         a.part != nullptr ? a.part + (size_t)k * a.T * a.rp : nullptr, red);
}

// R = the K ranges' sums added in order, rounded once to fp16; four values from value 4 i.  A few MB out of
// the caches (T = 2048, r = 64, 4 ranges: 2.1 MB, 4.9 us): bound by its launch.
__device__ __forceinline__ void join_ranges(const PrepArgs& a, size_t i) {
    const size_t n = (size_t)a.T * a.rp / 4;
    if (i >= n) return;
    const f4* p = reinterpret_cast<const f4*>(a.part) + i;
    f4 v = p[0];
#pragma unroll 4
    for (int k = 1; k < a.ks; ++k) v += p[(size_t)k * n];
    const h2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
    reinterpret_cast<u2*>(a.R)[i] = u2{as_u32(lo), as_u32(hi)};
}

__global__ __launch_bounds__(256) void prep_join_kernel(const PrepArgs a) {
    join_ranges(a, (size_t)blockIdx.x * 256 + threadIdx.x);
}

// --------------------------------------------------------------------- product
// 16 TT tokens x 16 RR rows per workgroup; its NW wavefronts take the input groups in turn (group g
// to wavefront g % NW), operands straight from memory, and add their exact int32 tiles through LDS.
// Wavefront w then finishes tile w (w < TT RR): scales, correction steps, one rounding to fp16.
// Few tokens: the weights are the traffic and each call a few microseconds, so K is split inside the workgroup
// to have all its loads in flight at once; one row tile a workgroup up to 16 tokens, for workgroups enough.
// Bound by the latency of that one round of loads: one token, 4096 + 2 x 1024 rows <- 4096 (25 MB), warm in the
// caches 5.7 us, waits 0.84 of the wavefronts' time; 37 tokens, 2 x 1408 <- 2048 7.3 us.
template <int TT, int RR>
__global__ __launch_bounds__(64 * kW8Waves) void w8a8_split_kernel(const ForwardArgs args) {
    constexpr int NW = kW8Waves, NT = TT * RR;
    static_assert(NT <= NW, "one tile per wavefront at the end");
    __shared__ i4v red[NW][NT][64];
    const int mb = blockIdx.x % args.m_tiles, nbl = blockIdx.x / args.m_tiles;
    const ModuleArgs M = args.mod[module_of(args, nbl)];
    const int rt0 = (nbl - M.tile_begin) * RR, m0 = mb * 16 * TT;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int T = args.T, d = args.d, G = args.G;
    const i4v zero = {0, 0, 0, 0};

    const uint8_t* qp[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) qp[rr] = M.q + (size_t)min(rt0 + rr, M.n_tiles16 - 1) * kW8Block + lane * 16;
    const size_t qstride = (size_t)M.n_tiles16 * kW8Block;
    const int8_t* xp[TT];
    bool t_ok[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        const int t = m0 + 16 * tt + (lane & 15);
        t_ok[tt] = t < T;
        xp[tt] = args.xq + (size_t)(t_ok[tt] ? t : 0) * d + 16 * (lane >> 4);
    }
    i4v acc[TT][RR];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = zero;
    constexpr int U = 2;
    for (int g0 = wave; g0 < G; g0 += U * NW) {
        i4v w[U][RR][2], x[U][TT][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = min(g0 + u * NW, G - 1);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int rr = 0; rr < RR; ++rr)
                    w[u][rr][m] = *reinterpret_cast<const i4v*>(qp[rr] + (size_t)g * qstride + 1024 * m);
#pragma unroll
                for (int tt = 0; tt < TT; ++tt)
                    x[u][tt][m] = t_ok[tt] ? *reinterpret_cast<const i4v*>(xp[tt] + (size_t)g * kGroup + 64 * m) : zero;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g0 + u * NW < G) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = mfma_i8(w[u][rr][m], x[u][tt][m], acc[tt][rr]);
            }
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) red[wave][tt * RR + rr][lane] = acc[tt][rr];
    __syncthreads();
    if (wave >= NT) return;
    const int tt = wave / RR, rt = rt0 + wave % RR;
    if (rt >= M.n_tiles16) return;
    i4v sum = red[0][wave][lane];
#pragma unroll
    for (int k = 1; k < NW; ++k) sum += red[k][wave][lane];
    const int t = m0 + 16 * tt + (lane & 15);
    const bool ok = t < T;
    const float st = ok ? args.xscale[t] : 0.f;
    const int row0 = rt * 16 + 4 * (lane >> 4);
    const f4 sw = *reinterpret_cast<const f4*>(M.sz + (size_t)rt * 64 + 16 * (lane >> 4));
    f4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)sum[i] * sw[i] * st;
    if (args.r > 0 && M.a != nullptr) {
        // R as the K ranges' fp32 sums, added in order and rounded once to fp16 here (few tokens: a
        // launch that only joined them would take longer)
        const int r = args.r, rp = args.r_pad, kofs = 8 * (lane >> 4);
        const h8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
        const int arow = rt * 16 + (lane & 15);
        const float* R = static_cast<const float*>(args.R) + (size_t)min(t, T - 1) * rp;
        for (int kb = 0; kb < rp / 32; ++kb) {
            const int col = 32 * kb + kofs;
            const h8 av = (arow < M.n_out && col < r) ? load_h8(M.a + (size_t)arow * r + col) : zero8;
            f4 lo = *reinterpret_cast<const f4*>(R + col), hi = *reinterpret_cast<const f4*>(R + col + 4);
            for (int k = 1; k < args.n_proj; ++k) {
                const float* p = R + (size_t)k * T * rp + col;
                lo += *reinterpret_cast<const f4*>(p);
                hi += *reinterpret_cast<const f4*>(p + 4);
            }
            h8 bv;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bv[i] = (_Float16)lo[i];
                bv[4 + i] = (_Float16)hi[i];
            }
            v = mfma16(av, bv, v);
        }
    }
    if (ok) store_rows(M, t, row0, v);
}

// --------------------------------------------------------------------- large tiles
// 16 TT WM tokens x 64 WN rows per workgroup: WM x WN wavefronts, each 16 TT tokens x 4 row tiles.
// The token codes of an input group (128 bytes a token) go HBM/L2 -> LDS by the load unit into a ring
// of four stages; a wavefront's weight operands come straight into registers (the WM wavefronts that share
// rows find them in the L1 cache), so that LDS carries only the codes: a code byte read feeds 4 matrix-core
// steps.  Both are requested two or three groups ahead, but seldom stay in flight that long: where the paths
// around a team's last, shorter turn meet, the compiler cannot count the operand loads and waits for all of
// them, once in four groups with TT = 4, four times with TT = 8.
// In a stage, row r keeps its 16-byte piece c at position c ^ f(r), f(r) = (r % 8) ^ ((r / 8) % 2).  That is
// not free of bank conflicts: LDS serves a 16-byte read 16 lanes at a time, eight of one piece and eight of
// the next, and rows 12 to 15 of a piece meet rows 4 to 7 of the next one, rows 0 to 3 its rows 8 to 11 --
// two lanes a bank, conflicts for 0.47 to 0.49 of the access cycles.
// Tokens past T read token T - 1 and row tiles past the module its last tile; neither is stored.
//
// Where the tiles do not fill the GPU, KH such teams of WM x WN wavefronts share a workgroup: each takes a part
// of the input groups through a ring of its own, the exact int32 sums meet in LDS, and a team finishes
// TT / KH of the token tiles -- a full CU from one workgroup at a KH-th of the partial tiles that a split over
// workgroups writes.  With args.tile_ks > 1 the input groups are split over workgroups too: each writes its exact
// int32 tile to the workspace, and w8a8_join_kernel adds them and finishes.
//
// Measured (r = 64): 128 x 256, T = 2048, 2 x 11008 rows <- 4096: 175 to 193 us, 1.9 to 2.1 Pop/s of int8 (a plain
// int8 product of 8192^3 by the vendor's library: 2.07).  Matrix cores busy 0.47 of the time, operand returns from the
// L1/LDS path 0.70 (2.4 GB from the L2 caches, 13 TB/s; 0.40 GB from behind them).  Bound by the operands and the
// waits for them: a timing copy without the loads took 139 us of the 190, one without LDS reads too 131.  256 x 256
// on 4 or 8 wavefronts and 128 x 512 on 8 (half the weight traffic, one workgroup a CU) took 200 to 212 us.
// 128 x 128 with two teams in two K ranges, T = 512, 4096 rows <- 14336: 42 us, 1.4 Pop/s; unsplit, T = 128,
// 2 x 11008 <- 4096: 28 us (90 MB of weights from the last-level cache: 3.3 TB/s).  64 x 128 with four teams, T = 64,
// the same rows: 23 us (3.9 TB/s).
typedef __attribute__((address_space(3))) void lds_void;
template <int I>
using ic = std::integral_constant<int, I>;

// Column of the launch (row block of a module and K range) and token block of a workgroup: XCD x
// (workgroups b with b % 8 == x) takes the columns x, x + 8, ..., eight token blocks at a time, so
// that a column's weights stay in one L2 and its workgroups run together.
__device__ __forceinline__ bool w8_place(const ForwardArgs& args, int block, int& mb, int& col) {
    const int cols = args.n_tiles, MT = args.m_tiles;
    const int xcd = block & 7, local = block >> 3;
    const int mine = (cols - xcd + 7) >> 3;  // columns of this XCD
    if (mine <= 0) return false;
    const int per = 8 * mine;
    const int ms = local / per, in = local - ms * per;
    const int width = min(8, MT - 8 * ms);
    if (width <= 0) return false;
    const int c = in / width;
    if (c >= mine) return false;
    mb = 8 * ms + (in - c * width);
    col = xcd + 8 * c;
    return true;
}

enum : int { kW8Plain = 0, kW8Correct = 1, kW8Split = 2 };  // what follows the integer sums

template <int WM, int WN, int TT, int KH, int MODE>
__global__ __launch_bounds__(64 * WM * WN * KH, 2) void w8a8_tile_kernel(const ForwardArgs args, const PrepArgs prep,
                                                                        int join_blocks) {
    constexpr int RR = 4, NW = WM * WN, BM = 16 * TT * WM, SB = BM * 128;
    constexpr int NC = BM / 8 / NW;        // 1 KB code copies per wavefront and group
    constexpr int TE = TT / KH;            // token tiles that a wavefront finishes
    constexpr int NE = BM / 8 / (NW * KH); // copies per wavefront of a stage that all fill
    static_assert(NC * 8 * NW == BM && NC + 3 * RR < 63 && BM % 64 == 0 && NE > 0 && TE * KH == TT, "copies");
    __shared__ __attribute__((aligned(16))) uint8_t st0[KH * SB];
    __shared__ __attribute__((aligned(16))) uint8_t st1[KH * SB];
    __shared__ __attribute__((aligned(16))) uint8_t st2[KH * SB];
    __shared__ __attribute__((aligned(16))) uint8_t st3[KH * SB];
    __shared__ __attribute__((aligned(16))) float row_scale[NW * KH * 64];
    __shared__ __attribute__((aligned(16))) float tok_scale[BM];
    // With a K split the projection is only used by the launch after this one: the first workgroups (a
    // multiple of 8) join its ranges instead of a launch of their own
    if constexpr (MODE == kW8Split) {
        if ((int)blockIdx.x < join_blocks) {
            join_ranges(prep, (size_t)blockIdx.x * (64 * NW * KH) + threadIdx.x);
            return;
        }
    }
    int mb, col;
    if (!w8_place(args, (int)blockIdx.x - join_blocks, mb, col)) return;
    const int ks = MODE == kW8Split ? args.tile_ks : 1, nbl = col / ks, kr = col - nbl * ks;
    const ModuleArgs M = args.mod[module_of(args, nbl)];
    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int kh = KH > 1 ? wave_all / NW : 0, wave = KH > 1 ? wave_all % NW : wave_all;  // team, wavefront of it
    const int wm = wave % WM, wn = wave / WM;
    const int T = args.T, d = args.d, NT = M.n_tiles16;
    const int m0 = mb * BM, rt0 = (nbl - M.tile_begin) * RR * WN + wn * RR;
    // groups of the workgroup, and the KH-th part of them that this team takes (the last may be shorter, or none)
    const int n_all = min(args.dec_gk, args.G - kr * args.dec_gk), n_turn = (n_all + KH - 1) / KH;
    const int g_begin = kr * args.dec_gk + kh * n_turn, n_g = max(0, min(n_turn, n_all - kh * n_turn));
    const int g_last = min(g_begin + n_g, args.G) - 1;  // steps past the part repeat its last group
    // copy i of wave w fills rows 8 (NC w + i) .. + 7 of the stage; lane l lands at row + l / 8,
    // position l % 8, holding the row's piece (l % 8) ^ f(row)
    uint32_t xoff[NC];
    const uint32_t piece = 16 * ((lane & 7) ^ (lane >> 3));  // f(row) for even i; odd i flips bit 0
    static_assert(NC % 2 == 0, "row 8 (NC w + i) has parity i");
#pragma unroll
    for (int i = 0; i < NC; ++i)
        xoff[i] = (uint32_t)(min(m0 + 8 * (NC * wave + i) + (lane >> 3), T - 1) * d) + (piece ^ (16 * (i & 1)));
    const int fr = (lane & 7) ^ ((lane >> 3) & 1);
    const int rbase = (16 * TT * wm + (lane & 15)) * 128;
    const int rofs0 = rbase + 16 * ((lane >> 4) ^ fr), rofs1 = rbase + 16 * ((4 + (lane >> 4)) ^ fr);
    uint32_t rts[RR];  // the wavefront's row tiles (scalar: weight addresses are scalar but for the lane's 16 bytes)
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) rts[rr] = (uint32_t)min(rt0 + rr, NT - 1);
    const uint32_t lofs = lane * 16;

    auto copy = [&](int v, uint8_t* stg) {
        const int8_t* base = args.xq + (size_t)min(g_begin + v, g_last) * kGroup;
#pragma unroll
        for (int i = 0; i < NC; ++i)
            __builtin_amdgcn_global_load_lds((const void*)(base + xoff[i]), (lds_void*)(stg + kh * SB + 8 * (NC * wave + i) * 128),
                                             16, 0, 0);
    };
    // Operands requested: where registers allow (TT = 4), whole groups three ahead, group v in slot v % 4;
    // else halves, half h = 2 v + m in slot h % 4, three halves ahead.
    constexpr bool kDeep = TT <= 4;
    constexpr int kAhead = kDeep ? 3 : 2;  // groups the code copies are ahead
    i4v w[kDeep ? 8 : 4][RR];
    auto wload = [&](int v, int m, int slot) {
        const size_t g = (size_t)min(g_begin + v, g_last) * NT;
#pragma unroll
        for (int rr = 0; rr < RR; ++rr)
            w[slot][rr] = *reinterpret_cast<const i4v*>(M.q + (g + rts[rr]) * kW8Block + 1024 * m + lofs);
    };
    i4v acc[TT][RR];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = i4v{0, 0, 0, 0};

    {
        const uint32_t rt = (uint32_t)min(rt0 + (lane >> 4), NT - 1);
        __builtin_amdgcn_global_load_lds((const void*)(M.sz + (rt * 64 + (lane & 15) * 4)), (lds_void*)(row_scale + wave_all * 64),
                                         4, 0, 0);
        const int t0 = 64 * (wave_all % (BM / 64));
        __builtin_amdgcn_global_load_lds((const void*)(args.xscale + min(m0 + t0 + lane, T - 1)),
                                         (lds_void*)(tok_scale + t0), 4, 0, 0);
    }
    // The waits of the ring count the loads behind a copy, so that no operand load may move in front of one
    // (or a copy behind the operands of its group): the barriers keep the order under any scheduling.
    copy(0, st0);
    __builtin_amdgcn_sched_barrier(0);
    wload(0, 0, 0);
    wload(0, 1, 1);
    __builtin_amdgcn_sched_barrier(0);
    copy(1, st1);
    __builtin_amdgcn_sched_barrier(0);
    wload(1, 0, 2);
    if constexpr (kDeep) {
        wload(1, 1, 3);
        __builtin_amdgcn_sched_barrier(0);
        copy(2, st2);
        __builtin_amdgcn_sched_barrier(0);
        wload(2, 0, 4);
        wload(2, 1, 5);
    }
    __builtin_amdgcn_sched_barrier(0);

    // Group v in stage S = v % 4.  At the barrier its copies have landed: after them at most those of the
    // kAhead - 1 groups behind it and the operands in flight were issued.  The copies of v + kAhead go to a
    // stage whose last reads were before this barrier; operands go to slots whose last steps were issued.
    auto step = [&](int v, auto Sc) {
        constexpr int S = decltype(Sc)::value;
        constexpr int N = kDeep ? 2 * NC + 6 * RR : NC + 3 * RR;
        static_assert(N < 64, "vmcnt");
        uint8_t* const st[4] = {st0, st1, st2, st3};
        const uint8_t* cur = st[S] + kh * SB;
        uint8_t* nxt = st[(S + kAhead) & 3];
        __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N)
        __builtin_amdgcn_s_barrier();
        if constexpr (kDeep) {
            copy(v + 3, nxt);
            __builtin_amdgcn_sched_barrier(0);
            wload(v + 3, 0, (2 * S + 6) & 7);
            wload(v + 3, 1, (2 * S + 7) & 7);
            __builtin_amdgcn_sched_barrier(0);
            if (v >= n_g) return;
            i4v x[2][2];
            x[0][0] = *reinterpret_cast<const i4v*>(cur + rofs0);
            x[0][1] = *reinterpret_cast<const i4v*>(cur + rofs1);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                if (tt + 1 < TT) {
                    x[(tt + 1) & 1][0] = *reinterpret_cast<const i4v*>(cur + rofs0 + (tt + 1) * 2048);
                    x[(tt + 1) & 1][1] = *reinterpret_cast<const i4v*>(cur + rofs1 + (tt + 1) * 2048);
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = mfma_i8(w[2 * S + m][rr], x[tt & 1][m], acc[tt][rr]);
            }
            __builtin_amdgcn_sched_barrier(0);
            return;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            wload(v + 1 + m, 1 - m, (2 * S + m + 3) & 3);
            if (m == 0) {
                __builtin_amdgcn_sched_barrier(0);
                copy(v + 2, nxt);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (v >= n_g) continue;
            const int at = m == 0 ? rofs0 : rofs1;
            constexpr int D = 4;  // operand reads in flight: D - 1 ahead of the steps that take them
            i4v x[D];
#pragma unroll
            for (int tt = 0; tt < D - 1; ++tt) x[tt] = *reinterpret_cast<const i4v*>(cur + at + tt * 2048);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) {
                if (tt + D - 1 < TT) x[(tt + D - 1) % D] = *reinterpret_cast<const i4v*>(cur + at + (tt + D - 1) * 2048);
#pragma unroll
                for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = mfma_i8(w[(2 * S + m) & 3][rr], x[tt % D], acc[tt][rr]);
                __builtin_amdgcn_sched_barrier(0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // whole turns of the ring; steps past the range only keep time (a tail of its own made the
    // compiler move and spill accumulators)
    for (int v = 0; v < n_turn; v += 4) {
        step(v, ic<0>{});
        step(v + 1, ic<1>{});
        step(v + 2, ic<2>{});
        step(v + 3, ic<3>{});
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no copy may land in LDS after this
    __syncthreads();
    // Team kh finishes token tiles TE kh .. + TE - 1: the others' sums of them come through LDS, past the
    // first SB bytes of the stages (those are R's).
    if constexpr (KH > 1) {
        constexpr int kPiece = TE * RR * 1024, kStage = (KH - 1) * SB / kPiece;
        static_assert(kStage * kPiece == (KH - 1) * SB && 4 * kStage == KH * NW * (KH - 1), "sums fill the stages");
        auto piece_at = [&](int to, int from) {
            const int q = (to * NW + wave) * (KH - 1) + (from - to + KH) % KH - 1, at = q / kStage;
            return (at == 0 ? st0 : (at == 1 ? st1 : (at == 2 ? st2 : st3))) + SB + (q % kStage) * kPiece + 16 * lane;
        };
#pragma unroll
        for (int to = 0; to < KH; ++to)
            if (to != kh) {
                uint8_t* dst = piece_at(to, kh);
#pragma unroll
                for (int i = 0; i < TE * RR; ++i)
                    *reinterpret_cast<i4v*>(dst + 1024 * i) = acc[to * TE + i / RR][i % RR];
            }
#pragma unroll
        for (int to = 1; to < KH; ++to)
            if (to == kh) {
#pragma unroll
                for (int i = 0; i < TE * RR; ++i) acc[i / RR][i % RR] = acc[to * TE + i / RR][i % RR];
            }
        __syncthreads();
#pragma unroll
        for (int k = 1; k < KH; ++k) {
            const uint8_t* src = piece_at(kh, (kh + k) % KH);
#pragma unroll
            for (int i = 0; i < TE * RR; ++i) acc[i / RR][i % RR] += *reinterpret_cast<const i4v*>(src + 1024 * i);
        }
    }
    if constexpr (MODE == kW8Split) {
        i4v* part = reinterpret_cast<i4v*>(args.ypart) +
                    ((((size_t)mb * (args.n_tiles / ks) + nbl) * ks + kr) * NW + wave) * (TT * RR * 64) + kh * (TE * RR * 64);
#pragma unroll
        for (int tt = 0; tt < TE; ++tt)
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) part[(tt * RR + rr) * 64 + lane] = acc[tt][rr];
        return;
    }
    const int te0 = TT * wm + TE * kh;  // first of the wavefront's token tiles
    // The correction: R's columns 64 j .. + 63 (128 bytes a token, as a group of codes) go to stage j (r <= 256),
    // A's operands to registers, while the sums are scaled.  Rows of A past the module and tokens past T
    // repeat the last one (their results are not stored); columns of A past r are taken as zero, R's are
    // zero up to r_pad, here a multiple of 64.
    const int r = args.r, rp = args.r_pad;
    auto rcopy = [&](int j, uint8_t* stg) {
        if (64 * j >= rp) return;
        if constexpr (KH > 1) {  // R as the K ranges' fp32 sums: added in order, rounded once to fp16 here
            for (int i = threadIdx.x; i < BM * 8; i += 64 * NW * KH) {
                const int row = i >> 3, c = i & 7;
                const float* p = static_cast<const float*>(args.R) + (size_t)min(m0 + row, T - 1) * rp + (64 * j + 8 * c);
                f4 lo = *reinterpret_cast<const f4*>(p), hi = *reinterpret_cast<const f4*>(p + 4);
                for (int k = 1; k < args.n_proj; ++k) {
                    p += (size_t)T * rp;
                    lo += *reinterpret_cast<const f4*>(p);
                    hi += *reinterpret_cast<const f4*>(p + 4);
                }
                h8 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] = (_Float16)lo[e];
                    v[4 + e] = (_Float16)hi[e];
                }
                *reinterpret_cast<h8*>(stg + row * 128 + 16 * (c ^ (row & 7) ^ ((row >> 3) & 1))) = v;
            }
            return;
        }
        const uint8_t* base = reinterpret_cast<const uint8_t*>(args.R) + 128 * j;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int row = NE * wave_all + i;  // of eight tokens
            const uint32_t t = (uint32_t)min(m0 + 8 * row + (lane >> 3), T - 1);
            __builtin_amdgcn_global_load_lds((const void*)(base + (t * (uint32_t)rp * 2u + (piece ^ (16 * (row & 1))))),
                                             (lds_void*)(stg + 8 * row * 128), 16, 0, 0);
        }
    };
    const uint8_t* Ab = reinterpret_cast<const uint8_t*>(M.a) + (size_t)rts[0] * 32 * r;
    auto aload = [&](int j, int m) {  // into slot m
        const uint32_t c = (uint32_t)min(64 * j + 32 * m + 8 * (lane >> 4), r - 8);
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) {
            const uint32_t row = (uint32_t)min((rt0 + rr) * 16 + (lane & 15), M.n_out - 1) - rts[0] * 16;
            w[m][rr] = *reinterpret_cast<const i4v*>(Ab + (row * (uint32_t)r + c) * 2u);
        }
    };
    if constexpr (MODE == kW8Correct) {
        rcopy(0, st0);
        rcopy(1, st1);
        rcopy(2, st2);
        rcopy(3, st3);
        aload(0, 0);
        aload(0, 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    // The scaled sums take the integer sums' registers (as bits): the tile is all a wavefront can hold.
    // The empty asm keeps each product where it is written (it was sunk into the branches below, with
    // both forms of the tile live).
    {
        f4 sw[RR];
#pragma unroll
        for (int rr = 0; rr < RR; ++rr)
            sw[rr] = *reinterpret_cast<const f4*>(row_scale + wave_all * 64 + 16 * rr + 4 * (lane >> 4));
#pragma unroll
        for (int tt = 0; tt < TE; ++tt) {
            float st = tok_scale[16 * (te0 + tt) + (lane & 15)];
            asm volatile("" : "+v"(st));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                f4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)acc[tt][rr][i] * sw[rr][i] * st;
                asm volatile("" : "+v"(v));
                acc[tt][rr] = __builtin_bit_cast(i4v, v);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if constexpr (MODE == kW8Correct) {
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        int j = 0;
#pragma unroll 1
        do {
            const uint8_t* cur = j == 0 ? st0 : (j == 1 ? st1 : (j == 2 ? st2 : st3));
            if (j > 0) {
                aload(j, 0);
                aload(j, 1);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const bool in = 64 * j + 32 * m + 8 * (lane >> 4) < r;
                h8 av[RR];
#pragma unroll
                for (int rr = 0; rr < RR; ++rr) av[rr] = __builtin_bit_cast(h8, in ? w[m][rr] : i4v{0, 0, 0, 0});
#pragma unroll
                for (int tt = 0; tt < TE; ++tt) {
                    const h8 xv = *reinterpret_cast<const h8*>(cur + (m == 0 ? rofs0 : rofs1) + (TE * kh + tt) * 2048);
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr)
                        acc[tt][rr] = __builtin_bit_cast(i4v, mfma16(av[rr], xv, __builtin_bit_cast(f4, acc[tt][rr])));
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        } while (64 * ++j < rp);
    }
    // To memory through the wavefront's own part of the (finished) ring: [16 TT tokens][64 rows] fp16,
    // a token's eight 16-byte pieces p at p ^ (token % 8), then whole 128-byte lines.
    __syncthreads();
    constexpr int kPart = 16 * TE * 128, kPer = SB / kPart;
    static_assert(NW * KH * kPart <= 4 * SB && SB % kPart == 0, "a part per wavefront");
    const int sel = wave_all / kPer;
    uint8_t* out = (sel == 0 ? st0 : (sel == 1 ? st1 : (sel == 2 ? st2 : st3))) + (wave_all % kPer) * kPart;
#pragma unroll
    for (int tt = 0; tt < TE; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) {
            const f4 v = __builtin_bit_cast(f4, acc[tt][rr]);
            const h2 lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
            const int p = 2 * rr + (lane >> 5);
            *reinterpret_cast<u2*>(out + (16 * tt + (lane & 15)) * 128 + 16 * (p ^ (lane & 7)) + 8 * ((lane >> 4) & 1)) =
                u2{as_u32(lo), as_u32(hi)};
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int row0 = rt0 * 16 + 8 * (lane & 7);
    const bool vec = (M.n_out & 7) == 0 && row0 + 7 < M.n_out;
#pragma unroll 4
    for (int i = 0; i < 2 * TE; ++i) {
        const int tl = 8 * i + (lane >> 3), t = m0 + 16 * te0 + tl;
        const uint8_t* piece = out + tl * 128 + 16 * ((lane & 7) ^ (tl & 7));
        if (t >= T) continue;
        _Float16* y = M.y + (size_t)t * M.n_out + row0;
        if (vec) *reinterpret_cast<h8*>(y) = *reinterpret_cast<const h8*>(piece);
        else {
#pragma unroll 1
            for (int e = 0; e < min(8, M.n_out - row0); ++e) y[e] = reinterpret_cast<const _Float16*>(piece)[e];
        }
    }
}

// Sums of the K ranges of one 16-token x 64-row piece per wavefront (pieces numbered as the tile
// kernel stores them), scales, correction, one rounding to fp16.  Memory- and launch-bound: T = 512, 4096 rows, two
// ranges, 16.8 MB of sums and 4.2 MB of y: 9.7 us.
template <int WM, int WN, int TT>
__global__ __launch_bounds__(256) void w8a8_join_kernel(const ForwardArgs args, int pieces) {
    constexpr int RR = 4, NW = WM * WN;
    const int lane = threadIdx.x & 63;
    const int piece = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (piece >= pieces) return;
    const int ks = args.tile_ks, cols = args.n_tiles / ks;
    const int tt = piece % TT, wave = piece / TT % NW, tile = piece / TT / NW;
    const int mb = tile / cols, nbl = tile - mb * cols;
    const ModuleArgs M = args.mod[module_of(args, nbl)];
    const int rt0 = (nbl - M.tile_begin) * RR * WN + (wave / WM) * RR;
    const int t = (mb * WM + wave % WM) * 16 * TT + 16 * tt + (lane & 15);
    if (rt0 >= M.n_tiles16) return;
    const bool ok = t < args.T;
    const i4v* part = reinterpret_cast<const i4v*>(args.ypart);
    i4v sum[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) sum[rr] = i4v{0, 0, 0, 0};
    for (int k = 0; k < ks; ++k) {
        const i4v* p = part + ((((size_t)tile * ks + k) * NW + wave) * TT + tt) * (RR * 64) + lane;
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) sum[rr] += p[rr * 64];
    }
    const float st = ok ? args.xscale[t] : 0.f;
    f4 v[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) {
        const f4 sw = *reinterpret_cast<const f4*>(M.sz + (size_t)min(rt0 + rr, M.n_tiles16 - 1) * 64 + 16 * (lane >> 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[rr][i] = (float)sum[rr][i] * sw[i] * st;
    }
    if (args.r > 0 && M.a != nullptr) {
        const int r = args.r, rp = args.r_pad;
        const _Float16* R = reinterpret_cast<const _Float16*>(args.R);
        const h8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int kb = 0; kb < rp / 32; ++kb) {
            const int c = 32 * kb + 8 * (lane >> 4);
            const h8 bv = ok ? load_h8(R + (size_t)t * rp + c) : zero8;
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

hipError_t launch_repack_w8(const int8_t* codes, const float* scales, int64_t n_out, int64_t k_in, uint8_t* q, float* sz,
                            int32_t* flag, hipStream_t stream) {
    const int64_t nt = ceil_div(n_out, 16);
    hipLaunchKernelGGL(repack_w8_kernel, dim3((unsigned)(nt * (k_in / kGroup))), dim3(128), 0, stream, codes, n_out, k_in,
                       (int)nt, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(repack_w8_scales_kernel, dim3((unsigned)ceil_div(nt * 16, 256)), dim3(256), 0, stream, scales, n_out,
                       nt * 16, sz, flag);
    return hipGetLastError();
}

template <int TT, int NJ, int TPT>
static void launch_prep_n(const PrepArgs& a, hipStream_t stream) {
    const int64_t proj = a.r > 0 ? ceil_div(a.T, 16 * TT) * ceil_div(a.rp / 16, NJ) * a.ks : 0;
    const int64_t tokens = ceil_div(a.T, kPrepThreads / TPT);
    hipLaunchKernelGGL((prep_kernel<TT, NJ, TPT>), dim3((unsigned)(proj + tokens)), dim3(kPrepThreads), 0, stream, a,
                       (int)proj);
}

// Few tokens: a workgroup for each.  Many: as few threads per token as hold its row (64 values each).
template <int TT, int NJ>
static void launch_prep_t(const PrepArgs& a, hipStream_t stream) {
    if constexpr (NJ == 1) {
        launch_prep_n<TT, NJ, kPrepThreads>(a, stream);
    } else {
        if constexpr (TT == 1) {
            if (a.T <= 256) return launch_prep_n<TT, NJ, kPrepThreads>(a, stream);
        }
        if (a.d <= 64 * 64) launch_prep_n<TT, NJ, 64>(a, stream);
        else if (a.d <= 128 * 64) launch_prep_n<TT, NJ, 128>(a, stream);
        else launch_prep_n<TT, NJ, 256>(a, stream);
    }
}

PrepPlan w8a8_prep_plan(int64_t T, int64_t d, int32_t r, bool small) {
    PrepPlan p = {1, small ? 1 : 4, (int)d, 1};
    if (r == 0) return p;
    if (small) {  // one batch of loads per wavefront
        p.range = 32 * 8 * kPrepWaves;
    } else {
        // 32-token blocks halve the reads of B: where 16-token ones would read 24 MB of it or more (T / 16 blocks of d r
        // fp16 values) past the 128 tokens up to which a workgroup for each token's codes, which only the 16-token form
        // has, weighs more.  The call on 128 rows, 32- and 16-token blocks, r = 64: T = 300, d = 14336 31.8 us and 31.6;
        // T = 384, d = 8192 26.3 and 27.4; T = 768, d = 4096 26.0 and 26.9; T = 512, d = 14336 34.0 and 35.0, d = 4096
        // 24.7 and 23.6; T = 300, d = 8192 25.6 and 24.5.  r = 256: T = 300, d = 4096 28.7 and 31.9; T = 384, d = 14336
        // 47 and 61; T = 256, d = 4096 28.3 and 27.3; T = 128, d = 14336 37.1 and 35.2.  K ranges up to 256 workgroups
        // (one a CU, the codes' beside them; 384: 38 us at T = 512, d = 14336, 512: 36).
        p.tt = T > 128 && T * d * ceil_div((int64_t)r, 64) >= ((int64_t)3 << 20) ? 2 : 1;
        const int64_t blocks = ceil_div(T, 16 * p.tt) * ceil_div((int64_t)r, 64);
        const int64_t want = std::max<int64_t>(1, 256 / blocks);
        p.range = (int)std::max<int64_t>(32 * 4 * kPrepWaves, ceil_div(ceil_div(d, want), 32) * 32);
    }
    p.range = std::min<int>(p.range, (int)d);
    p.ks = (int)ceil_div(d, p.range);
    return p;
}

hipError_t launch_w8a8_prep(const PrepArgs& a, const PrepPlan& p, bool join, hipStream_t stream) {
    if (a.d % kGroup != 0 || a.d > kPrepMaxD) return hipErrorInvalidValue;
    if (p.nj == 1) launch_prep_t<1, 1>(a, stream);
    else if (p.tt == 1) launch_prep_t<1, 4>(a, stream);
    else launch_prep_t<2, 4>(a, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.r == 0 || p.nj == 1 || a.part == nullptr || !join) return e;
    hipLaunchKernelGGL(prep_join_kernel, dim3((unsigned)ceil_div((int64_t)a.T * a.rp / 4, 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

// SPLIT: the tile takes K ranges (128 x 128 with two teams and 64 x 128 do).
template <int WM, int WN, int TT, int KH, bool SPLIT>
static hipError_t launch_tile(const ForwardArgs& a, const PrepArgs& p, hipStream_t stream) {
    // every XCD takes ceil(columns / 8) columns of every token block; those it has not return at once
    const int64_t join = a.tile_ks > 1 && a.r > 0 && p.part != nullptr
                             ? ceil_div(ceil_div((int64_t)p.T * p.rp / 4, 64 * WM * WN * KH), 8) * 8 : 0;
    const int64_t grid = join + 8 * ceil_div(a.n_tiles, 8) * a.m_tiles;
    if (grid * 64 * WM * WN * KH > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 g((unsigned)grid), block(64 * WM * WN * KH);
    if constexpr (SPLIT) {
        if (a.tile_ks > 1) {
            hipLaunchKernelGGL((w8a8_tile_kernel<WM, WN, TT, KH, kW8Split>), g, block, 0, stream, a, p, (int)join);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
            const int pieces = a.m_tiles * (a.n_tiles / a.tile_ks) * WM * WN * TT;
            hipLaunchKernelGGL((w8a8_join_kernel<WM, WN, TT>), dim3((unsigned)ceil_div(pieces, 4)), dim3(256), 0, stream, a,
                               pieces);
            return hipGetLastError();
        }
    }
    if (a.tile_ks > 1) return hipErrorInvalidValue;
    if (a.r > 0) hipLaunchKernelGGL((w8a8_tile_kernel<WM, WN, TT, KH, kW8Correct>), g, block, 0, stream, a, p, (int)join);
    else hipLaunchKernelGGL((w8a8_tile_kernel<WM, WN, TT, KH, kW8Plain>), g, block, 0, stream, a, p, (int)join);
    return hipGetLastError();
}

hipError_t launch_w8a8(const ForwardArgs& a, const PrepArgs& p, hipStream_t stream) {
    if (a.tile_rr == 16) return launch_tile<1, 4, 8, 1, false>(a, p, stream);
    if (a.tile_rr == 8 && a.tile_tt == 8)
        return a.dec_ks == 2 ? launch_tile<2, 2, 4, 2, true>(a, p, stream) : launch_tile<2, 2, 4, 1, false>(a, p, stream);
    if (a.tile_rr == 8) return launch_tile<1, 2, 4, 4, true>(a, p, stream);
    const dim3 grid((unsigned)a.n_tiles), block(64 * kW8Waves);
    switch (a.tile_tt * 4 + a.tile_rr) {
        case 4 + 1: hipLaunchKernelGGL((w8a8_split_kernel<1, 1>), grid, block, 0, stream, a); break;
        case 8 + 2: hipLaunchKernelGGL((w8a8_split_kernel<2, 2>), grid, block, 0, stream, a); break;
        case 16 + 2: hipLaunchKernelGGL((w8a8_split_kernel<4, 2>), grid, block, 0, stream, a); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace glowq
