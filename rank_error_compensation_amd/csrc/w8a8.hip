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
//
// Code layout (workspace): [T][d], 16-byte pieces of the other operand in an order that suits LDS: of
// the eight pieces of token t's input group, piece c (inputs 16 c .. + 15) is at position c ^ f(t),
// f(t) = (t % 8) ^ ((t / 8) % 2).  A tile's rows then go to LDS as they lie in memory (the load unit
// takes 64 lanes of consecutive 16 bytes in 16 cycles, permuted ones in about 80: the 256 x 256 tile
// that permuted on the way took 269 us at 22016 x 4096, T = 2048), and the 16 rows of an operand read
// fall in distinct banks.
#include <type_traits>

#include "glowq_internal.h"
#include "w8a8.h"

namespace glowq {

typedef int32_t i4v __attribute__((ext_vector_type(4)));

namespace {

// f(t) of the code layout.
__device__ __forceinline__ int code_swizzle(int t) { return (t & 7) ^ ((t >> 3) & 1); }

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

// --------------------------------------------------------------------- token codes
constexpr int kQ8Threads = 256;
constexpr int kQ8Chunks = 4;  // 16-input chunks per thread: d <= 4 * 16 * 256 = 16384

// One workgroup per token: the largest magnitude (as fp16 bits, so that infinities and NaN order
// above every number), the scale, the codes.
__global__ __launch_bounds__(kQ8Threads) void quant_q8_kernel(const _Float16* __restrict__ x, int d, int8_t* __restrict__ xq,
                                                              float* __restrict__ xscale) {
    __shared__ uint32_t red[kQ8Threads / 64];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int n16 = d / 16;
    const _Float16* row = x + (size_t)t * d;
    h8 v[kQ8Chunks][2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kQ8Chunks; ++i) {
        const int c = tid + kQ8Threads * i;
        if (c < n16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[i][h] = load_h8(row + 16 * c + 8 * h);
                const u4 bits = __builtin_bit_cast(u4, v[i][h]) & 0x7FFF7FFFu;
#pragma unroll
                for (int e = 0; e < 4; ++e) top = max(top, max(bits[e] & 0xFFFFu, bits[e] >> 16));
            }
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = max(max(red[0], red[1]), max(red[2], red[3]));
    const float amax = (float)__builtin_bit_cast(_Float16, (uint16_t)top);
    const bool finite = top < 0x7C00u;
    const float scale = finite ? amax / 127.0f : __builtin_nanf("");  // IEEE division
    if (tid == 0) xscale[t] = scale;
    const bool some = finite && scale > 0.f;
#pragma unroll
    for (int i = 0; i < kQ8Chunks; ++i) {
        const int c = tid + kQ8Threads * i;
        if (c < n16) {
            u4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t word = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int e = 4 * j + b;
                    int code = 0;
                    if (some) {
                        const float rq = __builtin_rintf((float)v[i][e >> 3][e & 7] / scale);
                        code = (int)fminf(127.f, fmaxf(-127.f, rq));
                    }
                    word |= (uint32_t)(code & 0xFF) << (8 * b);
                }
                w[j] = word;
            }
            *reinterpret_cast<u4*>(xq + (size_t)t * d + 16 * (size_t)(c ^ code_swizzle(t))) = w;
        }
    }
}

// --------------------------------------------------------------------- product
// 16 TT tokens x 16 RR rows per workgroup; its NW wavefronts take the input groups in turn (group g
// to wavefront g % NW), operands straight from memory, and add their exact int32 tiles through LDS.
// Wavefront w then finishes tile w (w < TT RR): scales, correction steps, one rounding to fp16.
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
    int xofs[2];  // this lane's pieces of a group: f depends on the token's place in its 16-token tile alone
#pragma unroll
    for (int m = 0; m < 2; ++m) xofs[m] = 16 * ((4 * m + (lane >> 4)) ^ code_swizzle(lane & 15));
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
        const int t = m0 + 16 * tt + (lane & 15);
        t_ok[tt] = t < T;
        xp[tt] = args.xq + (size_t)(t_ok[tt] ? t : 0) * d;
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
                    x[u][tt][m] = t_ok[tt] ? *reinterpret_cast<const i4v*>(xp[tt] + (size_t)g * kGroup + xofs[m]) : zero;
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
        const int r = args.r, rp = args.r_pad, kofs = 8 * (lane >> 4);
        const _Float16* R = reinterpret_cast<const _Float16*>(args.R);
        const h8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
        const int arow = rt * 16 + (lane & 15);
        for (int kb = 0; kb < rp / 32; ++kb) {
            const int col = 32 * kb + kofs;
            const h8 av = (arow < M.n_out && col < r) ? load_h8(M.a + (size_t)arow * r + col) : zero8;
            const h8 bv = ok ? load_h8(R + (size_t)t * rp + col) : zero8;
            v = mfma16(av, bv, v);
        }
    }
    if (ok) store_rows(M, t, row0, v);
}

// --------------------------------------------------------------------- large tiles
// 16 TT WM tokens x 64 WN rows per workgroup: WM x WN wavefronts, each 16 TT tokens x 4 row tiles.
// The token codes of an input group (128 bytes a token) go HBM/L2 -> LDS by the load unit into a ring
// of four stages; a wavefront's weight operands come straight into registers, one group ahead (the WM
// wavefronts that share rows find them in the L1 cache), so that LDS carries only the codes: a code
// byte read feeds 4 matrix-core steps.
// Tokens past T read token T - 1 and row tiles past the module its last tile; neither is stored.
//
// With args.tile_ks > 1 the input groups are split over workgroups: each writes its exact int32
// tile to the workspace, and w8a8_join_kernel adds them and finishes.
typedef __attribute__((address_space(3))) void lds_void;
template <int I>
using ic = std::integral_constant<int, I>;

// Column of the launch (row block of a module and K range) and token block of a workgroup: XCD x
// (workgroups b with b % 8 == x) takes the columns x, x + 8, ..., eight token blocks at a time, so
// that a column's weights stay in one L2 and its workgroups run together.
__device__ __forceinline__ bool w8_place(const ForwardArgs& args, int& mb, int& col) {
    const int cols = args.n_tiles, MT = args.m_tiles;
    const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3;
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

template <int WM, int WN, int TT>
__global__ __launch_bounds__(64 * WM * WN, WM * WN <= 4 ? 2 : 1) void w8a8_tile_kernel(const ForwardArgs args) {
    constexpr int RR = 4, NW = WM * WN, BM = 16 * TT * WM, SB = BM * 128;
    constexpr int NC = BM / 8 / NW;  // 1 KB code copies per wavefront and group
    static_assert(NC * 8 * NW == BM && NC + 2 * RR < 64, "copies");
    __shared__ __attribute__((aligned(16))) uint8_t st0[SB];
    __shared__ __attribute__((aligned(16))) uint8_t st1[SB];
    __shared__ __attribute__((aligned(16))) uint8_t st2[SB];
    __shared__ __attribute__((aligned(16))) uint8_t st3[SB];
    int mb, col;
    if (!w8_place(args, mb, col)) return;
    const int ks = args.tile_ks, nbl = col / ks, kr = col - nbl * ks;
    const ModuleArgs M = args.mod[module_of(args, nbl)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int T = args.T, d = args.d, NT = M.n_tiles16;
    const int m0 = mb * BM, rt0 = (nbl - M.tile_begin) * RR * WN + wn * RR;
    const int g_begin = kr * args.dec_gk, g_end = min(g_begin + args.dec_gk, args.G);

    // code copy i of wave w fills rows 8 (NC w + i) .. + 7 of the stage, as they lie in memory
    uint32_t xoff[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
        xoff[i] = (uint32_t)(min(m0 + 8 * (NC * wave + i) + (lane >> 3), T - 1) * d + 16 * (lane & 7));
    const int fr = code_swizzle(lane & 15);
    const int rbase = (16 * TT * wm + (lane & 15)) * 128;
    const int rofs0 = rbase + 16 * ((lane >> 4) ^ fr), rofs1 = rbase + 16 * ((4 + (lane >> 4)) ^ fr);
    // row tiles are the wavefront's own, so weight addresses are scalar but for the lane's 16 bytes
    uint32_t rofs[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) rofs[rr] = (uint32_t)min(rt0 + rr, NT - 1);
    const uint32_t lofs = lane * 16;

    auto copy = [&](int g, uint8_t* stg) {
        const int8_t* xb = args.xq + (size_t)min(g, g_end - 1) * kGroup;
#pragma unroll
        for (int i = 0; i < NC; ++i)
            __builtin_amdgcn_global_load_lds((const void*)(xb + xoff[i]), (lds_void*)(stg + 8 * (NC * wave + i) * 128), 16, 0,
                                             0);
    };
    i4v w[2][RR][2];
    auto wload = [&](int g, int slot) {
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) {
            const uint8_t* qb = M.q + ((size_t)min(g, g_end - 1) * NT + rofs[rr]) * kW8Block;
#pragma unroll
            for (int m = 0; m < 2; ++m) w[slot][rr][m] = *reinterpret_cast<const i4v*>(qb + 1024 * m + lofs);
        }
    };
    i4v acc[TT][RR];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = i4v{0, 0, 0, 0};

    copy(g_begin, st0);
    wload(g_begin, 0);
    copy(g_begin + 1, st1);

    // group g in stage S = (g - g_begin) % 4, weights in slot S % 2.  At the barrier the copies of g and
    // the weights of g have landed: only the NC copies of g + 1, issued last, may be in flight.  Then
    // the weights of g + 1 and the copies of g + 2 are issued; their stage was last read in group g - 2.
    auto step = [&](int g, auto Sc) {
        constexpr int S = decltype(Sc)::value;
        uint8_t* cur = S == 0 ? st0 : (S == 1 ? st1 : (S == 2 ? st2 : st3));
        uint8_t* nxt = S == 0 ? st2 : (S == 1 ? st3 : (S == 2 ? st0 : st1));
        __builtin_amdgcn_s_waitcnt(0x0F70 | NC);  // vmcnt(NC)
        __builtin_amdgcn_s_barrier();
        wload(g + 1, (S + 1) & 1);
        __builtin_amdgcn_sched_barrier(0);
        copy(g + 2, nxt);
        __builtin_amdgcn_sched_barrier(0);
        if (g >= g_end) return;
        i4v x[2][2];
        x[0][0] = *reinterpret_cast<const i4v*>(cur + rofs0);
        x[0][1] = *reinterpret_cast<const i4v*>(cur + rofs1);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            if (tt + 1 < TT) {
                x[(tt + 1) & 1][0] = *reinterpret_cast<const i4v*>(cur + rofs0 + (tt + 1) * 2048);
                x[(tt + 1) & 1][1] = *reinterpret_cast<const i4v*>(cur + rofs1 + (tt + 1) * 2048);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int rr = 0; rr < RR; ++rr) acc[tt][rr] = mfma_i8(w[S & 1][rr][m], x[tt & 1][m], acc[tt][rr]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // whole turns of the ring; steps past the range only keep time (a tail of its own made the
    // compiler move and spill accumulators)
    for (int g = g_begin; g < g_end; g += 4) {
        step(g, ic<0>{});
        step(g + 1, ic<1>{});
        step(g + 2, ic<2>{});
        step(g + 3, ic<3>{});
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no copy may land in LDS after the workgroup ends

    if (ks > 1) {
        i4v* part = reinterpret_cast<i4v*>(args.ypart) + ((((size_t)mb * (args.n_tiles / ks) + nbl) * ks + kr) * NW + wave) * (TT * RR * 64);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) part[(tt * RR + rr) * 64 + lane] = acc[tt][rr];
        return;
    }
    // The scaled sums take the integer sums' registers (as bits): the tile is all a wavefront can hold.
    // The empty asm keeps each product where it is written (it was sunk into the branches below, with
    // both forms of the tile live), and gives each part its own addresses instead of kept ones.
    {
        const int tok0 = m0 + 16 * TT * wm + (lane & 15);
        f4 sw[RR];
        float st[TT];
#pragma unroll
        for (int rr = 0; rr < RR; ++rr)
            sw[rr] = *reinterpret_cast<const f4*>(M.sz + (size_t)min(rt0 + rr, NT - 1) * 64 + 16 * (lane >> 4));
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) st[tt] = args.xscale[min(tok0 + 16 * tt, T - 1)];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                f4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = (float)acc[tt][rr][i] * sw[rr][i] * st[tt];
                asm volatile("" : "+v"(v));
                acc[tt][rr] = __builtin_bit_cast(i4v, v);
            }
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (args.r > 0 && M.a != nullptr) {
        // rows past the module and tokens past T repeat the last one; their results are not stored.
        // Columns r .. r_pad - 1 of R are zero, and so must A's be
        int l = lane;
        asm volatile("" : "+v"(l));
        const int r = args.r, rp = args.r_pad, kofs = 8 * (l >> 4), row0 = min(rt0, NT - 1) * 16;
        const uint8_t* Rb = reinterpret_cast<const uint8_t*>(args.R);
        const uint8_t* Ab = reinterpret_cast<const uint8_t*>(M.a + (size_t)row0 * r);
        const h8 zero8 = {0, 0, 0, 0, 0, 0, 0, 0};
        uint32_t roff[TT], aoff[RR];
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
            roff[tt] = (uint32_t)(min(m0 + 16 * TT * wm + 16 * tt + (l & 15), T - 1) * rp) * 2u;
#pragma unroll
        for (int rr = 0; rr < RR; ++rr) aoff[rr] = (uint32_t)((min((rt0 + rr) * 16 + (l & 15), M.n_out - 1) - row0) * r) * 2u;
#pragma unroll 1
        for (int kb = 0; kb < rp / 32; ++kb) {
            const int c = 32 * kb + kofs;
            h8 av[RR], bv[TT];
#pragma unroll
            for (int rr = 0; rr < RR; ++rr) {
                const h8 v = load_h8(Ab + (aoff[rr] + 2u * (uint32_t)min(c, r - 8)));
                av[rr] = c < r ? v : zero8;
            }
#pragma unroll
            for (int tt = 0; tt < TT; ++tt) bv[tt] = load_h8(Rb + (roff[tt] + 2u * (uint32_t)c));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int rr = 0; rr < RR; ++rr)
                    acc[tt][rr] = __builtin_bit_cast(i4v, mfma16(av[rr], bv[tt], __builtin_bit_cast(f4, acc[tt][rr])));
        }
    }
    // To memory through the wavefront's own part of the (finished) ring: [16 TT tokens][64 rows] fp16,
    // a token's eight 16-byte pieces p at p ^ (token % 8), then whole 128-byte lines.
    __builtin_amdgcn_s_barrier();
    constexpr int kPart = 16 * TT * 128, kPer = SB / kPart;
    static_assert(NW * kPart <= 4 * SB && SB % kPart == 0, "a part per wavefront");
    const int sel = wave / kPer;
    uint8_t* out = (sel == 0 ? st0 : (sel == 1 ? st1 : (sel == 2 ? st2 : st3))) + (wave % kPer) * kPart;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
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
    for (int i = 0; i < 2 * TT; ++i) {
        const int tl = 8 * i + (lane >> 3), t = m0 + 16 * TT * wm + tl;
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
// kernel stores them), scales, correction, one rounding to fp16.
__global__ __launch_bounds__(256) void w8a8_join_kernel(const ForwardArgs args, int wm_n, int wn_n, int tt_n, int pieces) {
    constexpr int RR = 4;
    const int lane = threadIdx.x & 63;
    const int piece = (int)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (piece >= pieces) return;
    const int nw = wm_n * wn_n, ks = args.tile_ks, cols = args.n_tiles / ks;
    const int tt = piece % tt_n, wave = piece / tt_n % nw, tile = piece / tt_n / nw;
    const int mb = tile / cols, nbl = tile - mb * cols;
    const ModuleArgs M = args.mod[module_of(args, nbl)];
    const int rt0 = (nbl - M.tile_begin) * RR * wn_n + (wave / wm_n) * RR;
    const int t = (mb * wm_n + wave % wm_n) * 16 * tt_n + 16 * tt + (lane & 15);
    if (rt0 >= M.n_tiles16) return;
    const bool ok = t < args.T;
    const i4v* part = reinterpret_cast<const i4v*>(args.ypart);
    i4v sum[RR];
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) sum[rr] = i4v{0, 0, 0, 0};
    for (int k = 0; k < ks; ++k) {
        const i4v* p = part + ((((size_t)tile * ks + k) * nw + wave) * tt_n + tt) * (RR * 64) + lane;
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

hipError_t launch_quant_q8(const _Float16* x, int T, int d, int8_t* xq, float* xscale, hipStream_t stream) {
    if (d % kGroup != 0 || d > kQ8Chunks * 16 * kQ8Threads) return hipErrorInvalidValue;
    hipLaunchKernelGGL(quant_q8_kernel, dim3((unsigned)T), dim3(kQ8Threads), 0, stream, x, d, xq, xscale);
    return hipGetLastError();
}

template <int WM, int WN, int TT>
static hipError_t launch_tile(const ForwardArgs& a, hipStream_t stream) {
    // every XCD takes ceil(columns / 8) columns of every token block; those it has not return at once
    const int64_t grid = 8 * ceil_div(a.n_tiles, 8) * a.m_tiles;
    if (grid * 64 * WM * WN > (int64_t)UINT32_MAX) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((w8a8_tile_kernel<WM, WN, TT>), dim3((unsigned)grid), dim3(64 * WM * WN), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.tile_ks == 1) return e;
    const int pieces = a.m_tiles * (a.n_tiles / a.tile_ks) * WM * WN * TT;
    hipLaunchKernelGGL(w8a8_join_kernel, dim3((unsigned)ceil_div(pieces, 4)), dim3(256), 0, stream, a, WM, WN, TT, pieces);
    return hipGetLastError();
}

hipError_t launch_w8a8(const ForwardArgs& a, hipStream_t stream) {
    if (a.tile_rr == 16) return launch_tile<1, 4, 8>(a, stream);
    if (a.tile_rr == 8) return launch_tile<2, 2, 4>(a, stream);
    const dim3 grid((unsigned)a.n_tiles), block(64 * kW8Waves);
    switch (a.tile_tt * 4 + a.tile_rr) {
        case 4 + 1: hipLaunchKernelGGL((w8a8_split_kernel<1, 1>), grid, block, 0, stream, a); break;
        case 8 + 1: hipLaunchKernelGGL((w8a8_split_kernel<2, 1>), grid, block, 0, stream, a); break;
        case 8 + 2: hipLaunchKernelGGL((w8a8_split_kernel<2, 2>), grid, block, 0, stream, a); break;
        case 16 + 2: hipLaunchKernelGGL((w8a8_split_kernel<4, 2>), grid, block, 0, stream, a); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace glowq
