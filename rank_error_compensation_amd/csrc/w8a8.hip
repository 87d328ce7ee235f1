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
// 16 (l / 16) .. + 15.  Activation codes stay in their natural order [T][d], whose 16-byte pieces
// are the other operand.  Scales: 16 fp32 per row tile.  Rows >= n_out are zero.
#include "glowq_internal.h"
#include "w8a8.h"

namespace glowq {

typedef int32_t i4v __attribute__((ext_vector_type(4)));

namespace {

__device__ __forceinline__ i4v mfma_i8(i4v a, i4v b, i4v c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
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
            *reinterpret_cast<u4*>(xq + (size_t)t * d + 16 * (size_t)c) = w;
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
    if (!ok) return;
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

hipError_t launch_w8a8(const ForwardArgs& a, hipStream_t stream) {
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
