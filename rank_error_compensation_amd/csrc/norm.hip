// Layer norm over the last dimension and its gradients, rows [T][d]:
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),  xhat = (x - mean) rstd,  y = xhat w + b
//   with g = dy w:  dx = rstd (g - sum g / d - xhat sum g xhat / d),  dw = sum_t dy xhat,  db = sum_t dy
// A row stays in its threads' registers between the passes over it (the variance is taken around the mean,
// never as a difference of squares), so memory is moved once: 2 values per element, 3 for the gradients.
// Sums are fp32; every output is rounded once; the gradients of w and b stay fp32.
// Rows go to teams of TPR threads that hold V values each.  Workgroups take rows in turn: w and b, and in the
// gradient the column sums, stay in registers over all rows of a team.  The column sums of the workgroups meet in a
// second launch, in a fixed order: no atomics, so results do not depend on the order of execution.
// Bound by memory: 16383 x 4096 fp16 50 us (268 MB at 5.3 TB/s); its gradients at 16384 rows 85 + 2 us at their shortest, 90 + 4
// on average (403 MB at 4.7 and 4.5 TB/s; the call 88.5).  One row of 4096: 3.1 us, a load latency,
// two sums over the team and a store (11 us a call from the host); 515 x 2048 fp32 gradients 6.4 + 2.1 us.
#include <algorithm>

#include "glowq.h"
#include "layer.h"

namespace glowq {

namespace {

// 16 bytes of a row; a row starts at any multiple of its type's size
template <typename S>
struct Piece {
    static constexpr int N = 16 / sizeof(S);
    S v[N];
};
template <typename S>
struct Loose;
template <>
struct Loose<_Float16> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Loose<float> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};

template <typename S, bool NT>
__device__ __forceinline__ Piece<S> load_piece(const S* row, int col, int d) {
    if (col + Piece<S>::N <= d) {
        const typename Loose<S>::type* p = reinterpret_cast<const typename Loose<S>::type*>(row + col);
        const u4 bits = NT ? (u4)__builtin_nontemporal_load(p) : (u4)*p;
        return __builtin_bit_cast(Piece<S>, bits);
    }
    Piece<S> r;
#pragma unroll
    for (int k = 0; k < Piece<S>::N; ++k) r.v[k] = col + k < d ? row[col + k] : (S)0.f;
    return r;
}

template <typename S, bool NT>
__device__ __forceinline__ void store_piece(S* row, int col, int d, const Piece<S>& r) {
    if (col + Piece<S>::N <= d) {
        typename Loose<S>::type* p = reinterpret_cast<typename Loose<S>::type*>(row + col);
        if constexpr (NT) __builtin_nontemporal_store((typename Loose<S>::type)__builtin_bit_cast(u4, r), p);
        else *p = __builtin_bit_cast(u4, r);
        return;
    }
#pragma unroll
    for (int k = 0; k < Piece<S>::N; ++k)
        if (col + k < d) row[col + k] = r.v[k];
}

// Sums of M values over the TPR threads of each team; every thread of the workgroup calls it.  `slot`: LDS of this call alone
// until the second next call.
template <int TPR, int M>
__device__ __forceinline__ void team_sum(float (&v)[M], float* slot) {
#pragma unroll
    for (int off = (TPR < 64 ? TPR : 64) / 2; off > 0; off >>= 1)
#pragma unroll
        for (int m = 0; m < M; ++m) v[m] += __shfl_xor(v[m], off, 64);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int m = 0; m < M; ++m) slot[wave * M + m] = v[m];
        }
        __syncthreads();
        const int w0 = wave / W * W;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += slot[(w0 + w) * M + m];
            v[m] = s;
        }
    }
}

template <int TPR>
constexpr int norm_threads() {
    return TPR > 256 ? TPR : 256;
}

template <typename S, int TPR, int V, bool NT>
__global__ __launch_bounds__(norm_threads<TPR>()) void norm_kernel(const S* x, const S* __restrict__ w, const S* __restrict__ b,
                                                                   float eps, int T, int d, S* y, float* mean, float* rstd) {
    constexpr int N = Piece<S>::N, P = V / N, B = norm_threads<TPR>(), RG = B / TPR;
    __shared__ float slots[4][B / 64];
    const int sub = threadIdx.x % TPR, team = threadIdx.x / TPR;
    Piece<S> wv[P], bv[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int col = (p * TPR + sub) * N;
        if (w != nullptr) wv[p] = load_piece<S, false>(w, col, d);
        if (b != nullptr) bv[p] = load_piece<S, false>(b, col, d);
    }
    Piece<S> v[P];
    auto load = [&](int row, Piece<S>* to) {
        const S* r = x + (size_t)min(row, T - 1) * d;
#pragma unroll
        for (int p = 0; p < P; ++p) to[p] = load_piece<S, NT>(r, (p * TPR + sub) * N, d);
    };
    int turn = 0;
    load(blockIdx.x * RG + team, v);
    for (int row0 = blockIdx.x * RG; row0 < T; row0 += gridDim.x * RG, turn ^= 2) {
        const int row = row0 + team;
        Piece<S> next[P];
        if (row0 + (int)gridDim.x * RG < T) load(row + gridDim.x * RG, next);
        float s[1] = {0.f};
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < N; ++k) s[0] += (float)v[p].v[k];
        team_sum<TPR, 1>(s, slots[turn]);
        const float mu = s[0] / (float)d;
        s[0] = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float c = (float)v[p].v[k] - mu;
                if ((p * TPR + sub) * N + k < d) s[0] = fmaf(c, c, s[0]);
            }
        team_sum<TPR, 1>(s, slots[turn + 1]);
        const float rs = 1.0f / sqrtf(s[0] / (float)d + eps);
        if (row < T) {
            S* out = y + (size_t)row * d;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                Piece<S> o;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    float r = ((float)v[p].v[k] - mu) * rs;
                    if (w != nullptr) r *= (float)wv[p].v[k];
                    if (b != nullptr) r += (float)bv[p].v[k];
                    o.v[k] = (S)r;
                }
                store_piece<S, NT>(out, (p * TPR + sub) * N, d, o);
            }
            if (sub == 0) {
                if (mean != nullptr) mean[row] = mu;
                if (rstd != nullptr) rstd[row] = rs;
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = next[p];
    }
}

// Threads of a workgroup: 1024, or 512 where a thread holds more than 8 values (registers).
template <int V>
constexpr int back_threads() {
    return V <= 8 ? 1024 : 512;
}

// part [gridDim.x][2][d]: the workgroup's sums of dy xhat and dy, its teams' added in order.
template <typename S, int TPR, int V, bool NT>
__global__ __launch_bounds__(back_threads<V>()) void norm_backward_kernel(const S* dy, const S* x, const float* __restrict__ mean,
                                                                            const float* __restrict__ rstd,
                                                                            const S* __restrict__ w, int T, int d, S* dx,
                                                                            float* __restrict__ part) {
    constexpr int N = Piece<S>::N, P = V / N, B = back_threads<V>(), RG = B / TPR;
    __shared__ float slots[2][B / 64 * 2];
    __shared__ float cols[RG > 1 ? B * N : 1];
    const int sub = threadIdx.x % TPR, team = threadIdx.x / TPR;
    Piece<S> wv[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
        if (w != nullptr) wv[p] = load_piece<S, false>(w, (p * TPR + sub) * N, d);
    float aw[V], ab[V];
#pragma unroll
    for (int i = 0; i < V; ++i) aw[i] = ab[i] = 0.f;
    Piece<S> vx[P], vg[P];
    float mu, rs;
    auto load = [&](int row, Piece<S>* tx, Piece<S>* tg, float& m, float& r) {
        row = min(row, T - 1);
        const S *rx = x + (size_t)row * d, *rg = dy + (size_t)row * d;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            tx[p] = load_piece<S, NT>(rx, (p * TPR + sub) * N, d);
            tg[p] = load_piece<S, NT>(rg, (p * TPR + sub) * N, d);
        }
        m = mean[row];
        r = rstd[row];
    };
    constexpr bool kAhead = V <= 8;  // the next row requested before this one is used, as registers allow
    int turn = 0;
    if (kAhead) load(blockIdx.x * RG + team, vx, vg, mu, rs);
    for (int row0 = blockIdx.x * RG; row0 < T; row0 += gridDim.x * RG, turn ^= 1) {
        const int row = row0 + team;
        Piece<S> nx[P], ng[P];
        float nm = 0.f, nr = 0.f;
        if (!kAhead) load(row, vx, vg, mu, rs);
        else if (row0 + (int)gridDim.x * RG < T) load(row + gridDim.x * RG, nx, ng, nm, nr);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float xh = ((float)vx[p].v[k] - mu) * rs, dyv = (float)vg[p].v[k];
                const float g = w != nullptr ? dyv * (float)wv[p].v[k] : dyv;
                if ((p * TPR + sub) * N + k < d) {
                    s[0] += g;
                    s[1] = fmaf(g, xh, s[1]);
                    if (row < T) {
                        aw[p * N + k] = fmaf(dyv, xh, aw[p * N + k]);
                        ab[p * N + k] += dyv;
                    }
                }
            }
        team_sum<TPR, 2>(s, slots[turn]);
        const float c1 = s[0] / (float)d, c2 = s[1] / (float)d;
        if (row < T) {
            S* out = dx + (size_t)row * d;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                Piece<S> o;
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const float xh = ((float)vx[p].v[k] - mu) * rs, dyv = (float)vg[p].v[k];
                    const float g = w != nullptr ? dyv * (float)wv[p].v[k] : dyv;
                    o.v[k] = (S)(rs * (g - c1 - xh * c2));
                }
                store_piece<S, NT>(out, (p * TPR + sub) * N, d, o);
            }
        }
        if (kAhead) {
#pragma unroll
            for (int p = 0; p < P; ++p) vx[p] = nx[p], vg[p] = ng[p];
            mu = nm;
            rs = nr;
        }
    }
    if (part == nullptr) return;
    float* mine = part + (size_t)blockIdx.x * 2 * d;
    constexpr int C = TPR * N;  // columns of one piece of every thread of a team
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float* v = (which == 0 ? aw : ab) + p * N;
            if constexpr (RG == 1) {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if ((p * TPR + sub) * N + k < d) mine[(size_t)which * d + (p * TPR + sub) * N + k] = v[k];
            } else {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < N; ++k) cols[threadIdx.x * N + k] = v[k];
                __syncthreads();
                for (int c = threadIdx.x; c < C && p * C + c < d; c += B) {
                    float s = cols[c];
#pragma unroll 4
                    for (int t = 1; t < RG; ++t) s += cols[t * C + c];
                    mine[(size_t)which * d + p * C + c] = s;
                }
            }
        }
}

// dw and db: the workgroups' sums, 64 columns per workgroup, its 16 wavefronts' ranges added in order.
constexpr int kColumnWaves = 16;
__global__ __launch_bounds__(64 * kColumnWaves) void norm_columns_kernel(const float* __restrict__ part, int n, int d,
                                                                         float* __restrict__ dw, float* __restrict__ db) {
    __shared__ float red[kColumnWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + lane;  // of 2 d
    float s = 0.f;
    if (col < 2 * (int64_t)d) {
        const int per = (n + kColumnWaves - 1) / kColumnWaves, end = min(n, (wave + 1) * per);
#pragma unroll 8
        for (int i = wave * per; i < end; ++i) s += part[(size_t)i * 2 * d + col];
    }
    red[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || col >= 2 * (int64_t)d) return;
    for (int w = 1; w < kColumnWaves; ++w) s += red[w][lane];
    if (col < d) {
        if (dw != nullptr) dw[col] = s;
    } else if (db != nullptr) {
        db[col - d] = s;
    }
}

template <typename S, int TPR, int V>
hipError_t launch_norm_n(const NormArgs& a, hipStream_t stream) {
    constexpr int B = norm_threads<TPR>(), RG = B / TPR;
    const int64_t want = ceil_div(a.T, RG);
    const dim3 grid((unsigned)std::min<int64_t>(want, 2048)), block(B);
    const S *x = static_cast<const S*>(a.x), *w = static_cast<const S*>(a.w), *b = static_cast<const S*>(a.b);
    if ((int64_t)a.T * a.d * (int64_t)sizeof(S) > kStreamBytes)
        hipLaunchKernelGGL((norm_kernel<S, TPR, V, true>), grid, block, 0, stream, x, w, b, a.eps, a.T, a.d,
                           static_cast<S*>(a.out), a.mean, a.rstd);
    else
        hipLaunchKernelGGL((norm_kernel<S, TPR, V, false>), grid, block, 0, stream, x, w, b, a.eps, a.T, a.d,
                           static_cast<S*>(a.out), a.mean, a.rstd);
    return hipGetLastError();
}

template <typename S, int TPR, int V>
hipError_t launch_norm_backward_n(const NormArgs& a, hipStream_t stream) {
    constexpr int B = back_threads<V>(), RG = B / TPR;
    const int grid = (int)std::min<int64_t>(ceil_div(a.T, RG), kNormParts);
    const S *dy = static_cast<const S*>(a.dy), *x = static_cast<const S*>(a.x), *w = static_cast<const S*>(a.w);
    if ((int64_t)a.T * a.d * (int64_t)sizeof(S) > kStreamBytes)
        hipLaunchKernelGGL((norm_backward_kernel<S, TPR, V, true>), dim3(grid), dim3(B), 0, stream, dy, x, a.mean, a.rstd, w,
                           a.T, a.d, static_cast<S*>(a.out), a.part);
    else
        hipLaunchKernelGGL((norm_backward_kernel<S, TPR, V, false>), dim3(grid), dim3(B), 0, stream, dy, x, a.mean, a.rstd, w,
                           a.T, a.d, static_cast<S*>(a.out), a.part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.part == nullptr) return e;
    hipLaunchKernelGGL(norm_columns_kernel, dim3((unsigned)ceil_div(2 * (int64_t)a.d, 64)), dim3(64 * kColumnWaves), 0, stream,
                       a.part, grid, a.d, a.dw, a.db);
    return hipGetLastError();
}

// Teams just wide enough: idle threads cost as much as busy ones (2^24 values fp16, us: d = 128 16 threads x 8 values 15.5, 32 x
// 8 26.6; 512 64 x 8 15.6, 128 x 8 25; 2048 256 x 8 16.4, 512 x 8 25.4), while fewer values a thread cost little (1024: 64 x 16
// 15.6, 128 x 8 16.3; 4096: 256 x 16 16.7, 512 x 8 17.1, one row 3.4 and 3.1; 16384: 512 x 32 20.2, 1024 x 16 18.8, fp32 25.7
// and 26.8).  Between the powers of two a part of the threads is idle (the call, fp16, us: 512 17, 640 21.8, 768 18.9, 1024 17, 1280
// 22.3, 1536 19.5, 2048 17, 5120 24.9, 12288 31.4; fp32 26 to 31 but 38.7 at 12288).
template <typename S>
hipError_t launch_norm_t(const NormArgs& a, hipStream_t stream) {
    if (a.d <= 128) return launch_norm_n<S, 16, 8>(a, stream);
    if (a.d <= 256) return launch_norm_n<S, 16, 16>(a, stream);
    if (a.d <= 512) return launch_norm_n<S, 64, 8>(a, stream);
    if (a.d <= 1024) return launch_norm_n<S, 64, 16>(a, stream);
    if (a.d <= 2048) return launch_norm_n<S, 256, 8>(a, stream);
    if (a.d <= 4096) return launch_norm_n<S, 256, 16>(a, stream);
    if (a.d <= 8192) return launch_norm_n<S, 512, 16>(a, stream);
    return launch_norm_n<S, 512, 32>(a, stream);
}

// As above, at 8 values a thread, whose column sums leave room to request the next row ahead (2^24 values fp16, us: d = 256
// 32 x 8 23.6, 64 x 8 40; 4096 512 x 8 26.9, 256 x 16 28.5; 8192 1024 x 8 34.6, 512 x 16 36.4, fp32 47.6 and 51.9); above,
// 512 x 32 (16384: 51 us; 1024 threads x 16 spill: 60).  Between the powers of two, as above: 512 25, 640 39, 768 35, 1024 25.5,
// 1280 39, 1536 30, 2048 26, 5120 37, 12288 53; fp32 512 40, 640 55, 1024 42, 5120 49, 12288 64.
template <typename S>
hipError_t launch_norm_backward_t(const NormArgs& a, hipStream_t stream) {
    if (a.d <= 128) return launch_norm_backward_n<S, 16, 8>(a, stream);
    if (a.d <= 256) return launch_norm_backward_n<S, 32, 8>(a, stream);
    if (a.d <= 512) return launch_norm_backward_n<S, 64, 8>(a, stream);
    if (a.d <= 1024) return launch_norm_backward_n<S, 128, 8>(a, stream);
    if (a.d <= 2048) return launch_norm_backward_n<S, 256, 8>(a, stream);
    if (a.d <= 4096) return launch_norm_backward_n<S, 512, 8>(a, stream);
    if (a.d <= 8192) return launch_norm_backward_n<S, 1024, 8>(a, stream);
    return launch_norm_backward_n<S, 512, 32>(a, stream);
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, int32_t dtype, hipStream_t stream) {
    return dtype == GLOWQ_DTYPE_F16 ? launch_norm_t<_Float16>(a, stream) : launch_norm_t<float>(a, stream);
}

hipError_t launch_layer_norm_backward(const NormArgs& a, int32_t dtype, hipStream_t stream) {
    if (a.T == 0) {  // sums over no rows
        hipLaunchKernelGGL(norm_columns_kernel, dim3((unsigned)ceil_div(2 * (int64_t)a.d, 64)), dim3(64 * kColumnWaves), 0,
                           stream, a.part, 0, a.d, a.dw, a.db);
        return hipGetLastError();
    }
    return dtype == GLOWQ_DTYPE_F16 ? launch_norm_backward_t<_Float16>(a, stream) : launch_norm_backward_t<float>(a, stream);
}

}  // namespace glowq
