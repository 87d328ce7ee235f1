// The router of a mixture of experts: from a token's logits to the experts it takes and their weights, and the
// gradient back to the logits.
//
//   s = softmax(l) over the token's experts, or sigmoid(l); experts of logit -inf (or bias -inf) are out
//   order of choice: s_e + bias_e, or l_e without a bias; equal values: the lower expert first
//   groups: the n_group equal runs of experts rank by their best value, or by the sum of their two best s (+ bias);
//           only experts of the first keep_groups stay
//   w_j = scale s_j, or scale s_j / sum of the chosen s
//   renormalised softmax weights are the softmax over the chosen logits alone; for the gradient, with a_j = w_j / scale
//   and c = sum_j a_j dw_j:
//     softmax            dl_e = s_e scale (sum_{j: e_j = e} dw_j - sum_j dw_j s_{e_j})
//     softmax, renorm    dl_e = scale sum_{j: e_j = e} a_j (dw_j - c)               (no other expert has one)
//     sigmoid            dl_e = scale sum_{j: e_j = e} dw_j s_e (1 - s_e)
//     sigmoid, renorm    dl_e = scale sum_{j: e_j = e} a_j (dw_j - c) (1 - s_e)
//
// L lanes share a token.  Each sorts its E / L experts into a list of its best as it reads them, on 64-bit keys: the
// fp32 value widened (exactly, which leaves 29 bits), the expert in the low 8, so that one maximum finds value and
// lowest expert at once; then the best of the list heads leaves top_k times.  16 lanes serve up to 8 choices, 64 more.
// Decisions are those of exact arithmetic: logits are compared as they are.  Where scores decide (a bias, or
// groups by two scores) they are fp32 values within 2^-19 (1 + |value|) of the exact ones (exp and the quotient a few
// steps of 2^-24, a sum over E one step for each of its up to 20 additions in a row), so two values further apart
// than 2^-18 (1 + |value|) are in their exact order; a token with a closer pair at any place that matters is
// decided again in fp64.
#include <algorithm>
#include <type_traits>

#include "glowq.h"
#include "layer.h"

namespace glowq {

namespace {

constexpr int kRouteThreads = 256;
constexpr float kClose = 0x1p-18f;
constexpr double kOut = -1.7e308;  // key of an expert that is out; every value's key is above

// Rotation of the 16-lane row by N.
template <int N>
__device__ __forceinline__ float row_ror(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + N, 0xf, 0xf, false));
}
template <int N>
__device__ __forceinline__ double row_ror(double v) {
    const u2 b = __builtin_bit_cast(u2, v);
    const u2 r = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[0], 0x120 + N, 0xf, 0xf, false),
                  (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b[1], 0x120 + N, 0xf, 0xf, false)};
    return __builtin_bit_cast(double, r);
}

// Largest value, and sum, over the L lanes of a token; every lane gets the same bits (rotations add the same pairs).
template <int L, typename F>
__device__ __forceinline__ F lanes_max(F v) {
    v = fmax(v, row_ror<8>(v));
    v = fmax(v, row_ror<4>(v));
    v = fmax(v, row_ror<2>(v));
    v = fmax(v, row_ror<1>(v));
    if constexpr (L == 64) {
        v = fmax(v, __shfl_xor(v, 16, 64));
        v = fmax(v, __shfl_xor(v, 32, 64));
    }
    return v;
}
template <int L, typename F>
__device__ __forceinline__ F lanes_sum(F v) {
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    v += row_ror<1>(v);
    if constexpr (L == 64) {
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
    }
    return v;
}

// Bits of the token's lanes for which `on` holds.
template <int L>
__device__ __forceinline__ uint64_t lanes_with(bool on) {
    const uint64_t all = __ballot(on);
    if constexpr (L == 64) return all;
    return (all >> (threadIdx.x & 48)) & 0xFFFFu;
}

__device__ __forceinline__ void wave_sync() {  // LDS of one wavefront: written before, read after
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double key_of(float v, int e) {
    const double w = (double)(v + 0.f);  // -0 and 0 are equal
    const uint64_t bits = __builtin_bit_cast(uint64_t, w);
    return __builtin_bit_cast(double, bits | (uint64_t)(v < 0.f ? e : 255 - e));
}
__device__ __forceinline__ int key_expert(double k) {
    const int low = (int)(__builtin_bit_cast(uint64_t, k) & 255u);
    return k < 0.0 ? low : 255 - low;
}
__device__ __forceinline__ float key_value(double k) {
    return (float)__builtin_bit_cast(double, __builtin_bit_cast(uint64_t, k) & ~(uint64_t)255u);
}

template <typename F>
__device__ __forceinline__ F sigmoid_of(F l) {
    const F e = exp(-fabs(l)), q = (F)1 / ((F)1 + e);
    return l >= (F)0 ? q : e * q;
}

// Standings of the groups from the token's values `by` [E] in LDS (-inf: out): bit g of the answer is set where group g
// stays.  `near`: two groups are closer than fp32 scores tell apart.
template <int L, typename F>
__device__ uint32_t groups_that_stay(const F* by, const RouteArgs& a, int i, bool& near) {
    const int n = a.n_exp / a.n_group;
    F b1 = (F)-INFINITY, b2 = (F)-INFINITY;
    if (i < a.n_group)
        for (int q = 0; q < n; ++q) {
            const int at = q + i < n ? q + i : (q + i) % n;  // starts spread over the LDS banks
            const F v = by[i * n + at];
            b2 = fmax(b2, fmin(b1, v));
            b1 = fmax(b1, v);
        }
    const F stand = a.group_best == 2 && b2 > (F)-INFINITY ? b1 + b2 : b1;
    int rank = 0;
    bool close = false;
    for (int h = 0; h < a.n_group; ++h) {
        const F other = __shfl(stand, h, L);
        if (h == i) continue;
        rank += other > stand || (other == stand && h < i) ? 1 : 0;
        close |= fabs(other - stand) <= (F)kClose * ((F)1 + fabs(stand));  // (-inf from -inf: NaN, not close)
    }
    near = lanes_with<L>(close && i < a.n_group) != 0;
    return (uint32_t)lanes_with<L>(rank < a.keep_groups && i < a.n_group);
}

// Expert e's group stays.  e / n without a division: e < 256, 1 <= n <= 256.
__device__ __forceinline__ bool stays(uint32_t mask, int e, uint32_t inv) { return mask >> ((e * inv) >> 16) & 1u; }

// The choice of one token in fp64, by the definition: the lanes that hold it call it together.  v: its logits, lane i's
// expert j at e = i + L j.  Lane j < top_k gets the j-th expert.  At its end no lane reads `by` any more.
template <int L, int EPL>
__device__ __forceinline__ int choose_exact(const float (&v)[EPL], const RouteArgs& a, double* by, int i) {
    double s[EPL], u[EPL];
    double top = -INFINITY, sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) top = fmax(top, (double)v[j]);
    top = lanes_max<L>(top);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        s[j] = v[j] == -INFINITY ? 0.0 : (a.score == GLOWQ_SCORE_SIGMOID ? sigmoid_of((double)v[j]) : exp((double)v[j] - top));
        sum += s[j];
    }
    if (a.score == GLOWQ_SCORE_SOFTMAX) {
        sum = lanes_sum<L>(sum);
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = s[j] / sum;
    }
    uint32_t mask = ~0u, inv = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = i + L * j;
        if (a.bias != nullptr && e < a.n_exp) s[j] += (double)a.bias[e];
        if (v[j] == -INFINITY) s[j] = -INFINITY;
        u[j] = a.bias != nullptr ? s[j] : (double)v[j];
    }
    if (a.keep_groups < a.n_group) {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (i + L * j < a.n_exp) by[i + L * j] = a.group_best == 2 ? s[j] : u[j];
        wave_sync();
        bool near;
        mask = groups_that_stay<L>(by, a, i, near);
        wave_sync();
        inv = (65535u + (uint32_t)(a.n_exp / a.n_group)) / (uint32_t)(a.n_exp / a.n_group);
    }
    int mine = -1;
    for (int r = 0; r < a.top_k; ++r) {
        double best = -INFINITY;
        int at = 1 << 20;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {  // ascending experts: the first of equal values stays
            const int e = i + L * j;
            if (u[j] > best && (inv == 0 || stays(mask, e, inv))) best = u[j], at = e;
        }
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) {
            const double ob = __shfl_xor(best, off, L);
            const int oa = __shfl_xor(at, off, L);
            if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (i + L * j == at) u[j] = -INFINITY;
        if (i == r) mine = best == -INFINITY ? -1 : at;
    }
    return mine;
}

// SCORED: scores decide (a bias, or groups by two scores).
template <typename S, int L, int EPL, int KL, bool SCORED>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a) {
    constexpr int TB = kRouteThreads / L;
    __shared__ typename std::conditional<SCORED, double, float>::type by_all[TB][L * EPL];  // a token's values, fp32 or fp64
    const int i = threadIdx.x % L, slot = threadIdx.x / L;
    const int t = blockIdx.x * TB + slot;
    const bool live = t < a.T;
    const int E = a.n_exp, K = a.top_k;
    const S* row = static_cast<const S*>(a.logits) + (size_t)(live ? t : 0) * E;
    float v[EPL], b[EPL];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = i + L * j;
        v[j] = e < E ? (float)row[e] : -INFINITY;
        b[j] = SCORED && a.bias != nullptr && e < E ? a.bias[e] : 0.f;
        bad |= !(v[j] < INFINITY) || !(b[j] < INFINITY);  // NaN and +inf
    }
    bad = lanes_with<L>(bad) != 0;
    const bool groups = a.keep_groups < a.n_group;
    const bool softmax = a.score == GLOWQ_SCORE_SOFTMAX;
    float top = -INFINITY, sum = 1.f;
    if (softmax && (SCORED || !a.renorm)) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) top = fmaxf(top, v[j]);
        top = fmaxf(lanes_max<L>(top), -3e38f);  // a row without experts: no NaN
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) sum += __expf(v[j] - top);
        sum = lanes_sum<L>(sum);
    }
    uint32_t mask = ~0u, inv = 0;
    bool near = false;
    float u[EPL];
    if constexpr (SCORED) {
        const float rs = 1.f / sum;
        float* by = reinterpret_cast<float*>(by_all[slot]);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            float s;
            if (softmax) {
                s = __expf(v[j] - top) * rs;
            } else {
                const float x = __expf(-fabsf(v[j])), q = 1.f / (1.f + x);
                s = v[j] >= 0.f ? q : x * q;
            }
            s += b[j];
            if (v[j] == -INFINITY) s = -INFINITY;
            u[j] = a.bias != nullptr ? s : v[j];
            if (groups && i + L * j < E) by[i + L * j] = a.group_best == 2 ? s : u[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            u[j] = v[j];
            if (groups && i + L * j < E) reinterpret_cast<float*>(by_all[slot])[i + L * j] = v[j];
        }
    }
    if (groups) {
        wave_sync();
        bool close;
        mask = groups_that_stay<L>(reinterpret_cast<const float*>(by_all[slot]), a, i, close);
        near = SCORED && close;
        inv = (65535u + (uint32_t)(E / a.n_group)) / (uint32_t)(E / a.n_group);
        wave_sync();
    }
    // the lane's best, in order
    double list[KL];
#pragma unroll
    for (int q = 0; q < KL; ++q) list[q] = kOut;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = i + L * j;
        double x = key_of(u[j], e);
        if (u[j] == -INFINITY || (groups && !stays(mask, e, inv))) x = kOut;
#pragma unroll
        for (int q = 0; q < (j < KL ? j + 1 : KL); ++q) {
            const double hi = fmax(list[q], x);
            x = fmin(list[q], x);
            list[q] = hi;
        }
    }
    double mine = kOut, last = kOut;
    const int rounds = K + (SCORED && a.bias != nullptr ? 1 : 0);  // the first one left out is looked at, too
    for (int r = 0; r < rounds; ++r) {
        const double best = lanes_max<L>(list[0]);
        if (best == list[0]) {
#pragma unroll
            for (int q = 0; q + 1 < KL; ++q) list[q] = list[q + 1];
            list[KL - 1] = kOut;
        }
        if (SCORED && a.bias != nullptr && r > 0 && best > kOut) {
            const float hi = key_value(last), lo = key_value(best);
            near |= hi - lo <= kClose * (1.f + fabsf(hi));
        }
        last = best;
        if (i == r) mine = best;
    }
    int e = mine > kOut ? key_expert(mine) : -1;
    if constexpr (SCORED) {
        if (near) e = choose_exact<L, EPL>(v, a, by_all[slot], i);
    }
    if (bad || i >= K) e = -1;
    // weights: lane j has the j-th expert
    const float l = e >= 0 ? (float)row[e] : -INFINITY;
    float w = 0.f;
    if (a.renorm) {
        // the chosen scores over their sum; sigmoids of very low logits as exp(l), from the largest on
        const float m = fmaxf(lanes_max<L>(l), -3e38f);
        const float s = e < 0 ? 0.f : (softmax || m < -80.f ? expf(l - m) : sigmoid_of(l));
        const float all = lanes_sum<L>(s);
        w = e < 0 ? 0.f : a.scale * (s / all);
    } else if (e >= 0) {
        w = a.scale * (softmax ? expf(l - top) / sum : sigmoid_of(l));
    }
    if (!live) return;
    if (i < K) {
        a.ids[(size_t)t * K + i] = e;
        a.w[(size_t)t * K + i] = w;
    }
    if (bad && i == 0) __hip_atomic_fetch_or(a.err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A token's gradient row is built in LDS: zeros, the choices' terms added one after another (an expert named
// twice gets both, in order), then the softmax's term of every expert.
template <typename S, int L, int EPL>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(const RouteArgs a) {
    constexpr int TB = kRouteThreads / L;
    __shared__ float sums[TB][L * EPL];
    const int i = threadIdx.x % L, slot = threadIdx.x / L;
    const int t = blockIdx.x * TB + slot;
    const bool live = t < a.T;
    const int E = a.n_exp, K = a.top_k;
    const S* row = static_cast<const S*>(a.logits) + (size_t)(live ? t : 0) * E;
    const bool softmax = a.score == GLOWQ_SCORE_SOFTMAX;
    int e = -1;
    float dw = 0.f;
    if (i < K && live) {
        e = a.ids[(size_t)t * K + i];
        dw = a.w[(size_t)t * K + i];
        if (e < -1 || e >= E) {
            __hip_atomic_fetch_or(a.err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            e = -1;
        }
    }
    const float l = e >= 0 ? (float)row[e] : -INFINITY;
    if (l == -INFINITY) e = -1, dw = 0.f;  // an expert that is out has score 0 whatever its logit does
    float* mine = sums[slot];
#pragma unroll
    for (int j = 0; j < EPL; ++j) mine[i + L * j] = 0.f;
    float v[EPL], p[EPL], dot = 0.f, g;
    if (a.renorm) {
        const float m = fmaxf(lanes_max<L>(l), -3e38f);
        const float s = e < 0 ? 0.f : (softmax || m < -80.f ? expf(l - m) : sigmoid_of(l));
        const float all = lanes_sum<L>(s);
        const float share = e < 0 ? 0.f : s / all;
        const float c = lanes_sum<L>(share * dw);
        g = a.scale * share * (dw - c) * (softmax ? 1.f : sigmoid_of(-l));
    } else if (softmax) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            v[j] = i + L * j < E ? (float)row[i + L * j] : -INFINITY;
            top = fmaxf(top, v[j]);
        }
        top = fmaxf(lanes_max<L>(top), -3e38f);
#pragma unroll
        for (int j = 0; j < EPL; ++j) sum += p[j] = __expf(v[j] - top);
        sum = lanes_sum<L>(sum);
        const float rs = sum == 0.f ? 0.f : a.scale / sum;
#pragma unroll
        for (int j = 0; j < EPL; ++j) p[j] *= rs;
        g = dw;
        dot = lanes_sum<L>(e < 0 ? 0.f : dw * expf(l - top)) / (sum == 0.f ? 1.f : sum);
    } else {
        g = a.scale * dw * sigmoid_of(l) * sigmoid_of(-l);
    }
    wave_sync();
    for (int r = 0; r < K; ++r) {
        if (i == r && e >= 0) mine[e] += g;
        wave_sync();
    }
    if (!live) return;
    S* out = static_cast<S*>(a.out) + (size_t)t * E;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int x = i + L * j;
        if (x < E) out[x] = (S)(softmax && !a.renorm ? p[j] * (mine[x] - dot) : mine[x]);
    }
}

template <typename S, int L, int EPL, int KL>
hipError_t launch_route_n(const RouteArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)ceil_div(a.T, kRouteThreads / L)), block(kRouteThreads);
    if (a.bias != nullptr || (a.keep_groups < a.n_group && a.group_best == 2))
        hipLaunchKernelGGL((route_kernel<S, L, EPL, KL, true>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((route_kernel<S, L, EPL, KL, false>), grid, block, 0, stream, a);
    return hipGetLastError();
}

template <typename S, int L, int EPL>
hipError_t launch_route_backward_n(const RouteArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((route_backward_kernel<S, L, EPL>), dim3((unsigned)ceil_div(a.T, kRouteThreads / L)), dim3(kRouteThreads),
                       0, stream, a);
    return hipGetLastError();
}

template <typename S>
hipError_t launch_route_t(const RouteArgs& a, hipStream_t stream) {
    if (a.top_k > 8) return launch_route_n<S, 64, 4, 4>(a, stream);
    if (a.n_exp <= 64) return launch_route_n<S, 16, 4, 4>(a, stream);
    if (a.n_exp <= 128) return a.top_k <= 4 ? launch_route_n<S, 16, 8, 4>(a, stream) : launch_route_n<S, 16, 8, 8>(a, stream);
    return a.top_k <= 4 ? launch_route_n<S, 16, 16, 4>(a, stream) : launch_route_n<S, 16, 16, 8>(a, stream);
}

template <typename S>
hipError_t launch_route_backward_t(const RouteArgs& a, hipStream_t stream) {
    if (a.top_k > 16) return launch_route_backward_n<S, 64, 4>(a, stream);
    if (a.n_exp <= 64) return launch_route_backward_n<S, 16, 4>(a, stream);
    if (a.n_exp <= 128) return launch_route_backward_n<S, 16, 8>(a, stream);
    return launch_route_backward_n<S, 16, 16>(a, stream);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, int32_t dtype, hipStream_t stream) {
    return dtype == GLOWQ_DTYPE_F16 ? launch_route_t<_Float16>(a, stream) : launch_route_t<float>(a, stream);
}

hipError_t launch_moe_route_backward(const RouteArgs& a, int32_t dtype, hipStream_t stream) {
    return dtype == GLOWQ_DTYPE_F16 ? launch_route_backward_t<_Float16>(a, stream) : launch_route_backward_t<float>(a, stream);
}

}  // namespace glowq
