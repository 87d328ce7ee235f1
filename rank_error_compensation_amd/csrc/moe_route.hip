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
// groups by two scores) they are fp32 values a little off the exact ones, in steps of 2^-24:
//   sigmoid  exp is off by 2 |l| + 4 steps of itself (its argument's rounding, its own), which moves s by s (1 - s) of
//            that, 1.5 at most; the quotient and the product add 3, the bias one of the value: 6 + |v|
//   softmax  exp as above, and the sum by one for each of its 20 additions in a row at most, all of s: 32 + |v|
// So two values further apart than 2^-20 (1 + |v|), or 2^-18 (1 + |v|), are in their exact order.  A group's standing by
// two, taken as half their sum (which no two numbers overflow), is off by half of that at 1 + the halves of both magnitudes
// (values of opposite signs cancel, their errors do not), and groups are in their exact order if no one that is out comes within
// its error of one that stays within its own.  A token that is closer at a place that matters is decided again in fp64, by
// the whole wavefront.
// Bound by the keys' arithmetic (64-bit maxima) where scores decide, else by memory and the launch: 32767 x 256 fp32 logits, 8
// choices: from 4 of 8 groups with a bias 32 us (34 MB: 1 TB/s), plain softmax 15.5 us; one token 2.6 us; gradient of
// 16384 x 60, 4 choices 4.4 us (8 MB).  131072 tokens: 60 experts, 4 choices 17 us (plain softmax) to 38 (groups, bias), 256
// experts, 8 choices 52 to 104, 16 choices 146 to 315; gradients of softmax weights 16 (60 experts, 63 MB) and 52 us (256,
// 268 MB: 5.2 TB/s, as a copy), of the others, which only write the row, 13 and 37.  In groups the LDS rows of a wavefront's
// four tokens start at the same bank: conflicts for 0.43 of the access cycles.
#include <algorithm>
#include <cfloat>

#include "glowq.h"
#include "layer.h"

namespace glowq {

namespace {

constexpr int kRouteThreads = 256;
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

// A chosen expert's score next to the others' for logits m at most: softmax over the largest, sigmoid over exp(min(m, 0)), so
// that scores which no number holds keep their ratios.
__device__ __forceinline__ float score_beside(float l, float m, bool softmax) {
    if (softmax) return expf(l - m);
    return expf(fminf(l, 0.f) - fminf(m, 0.f)) * (1.f / (1.f + expf(-fabsf(l))));
}

// How near two values may be before fp64 decides (above), for values v about 1 + |v| large.
__device__ __forceinline__ float close_to(const RouteArgs& a) { return a.score == GLOWQ_SCORE_SIGMOID ? 0x1p-20f : 0x1p-18f; }

// Standings of the groups from the token's values `by` [E] in LDS (-inf: out): bit g of the answer is set where group g
// stays.  `near`: fp32 scores do not tell apart which ones do.
template <int L, typename F>
__device__ __forceinline__ uint32_t groups_that_stay(const F* by, const RouteArgs& a, int i, bool& near) {
    const int n = a.n_exp / a.n_group;
    F b1 = (F)-INFINITY, b2 = (F)-INFINITY;
    if (i < a.n_group) {
        int at = i < n ? i : 0;  // starts spread over the LDS banks
#pragma unroll 4
        for (int q = 0; q < n; ++q) {
            const F v = by[i * n + at];
            at = at + 1 == n ? 0 : at + 1;
            b2 = fmax(b2, fmin(b1, v));
            b1 = fmax(b1, v);
        }
    }
    F stand = b1, size = fabs(b1);
    if (a.group_best == 2) {
        const F half = b2 > (F)-INFINITY ? (F)0.5 * b2 : (F)0;
        stand = (F)0.5 * b1 + half;
        size = (F)0.5 * fabs(b1) + fabs(half);
    }
    int rank = 0;
#pragma unroll 4
    for (int h = 0; h < a.n_group; ++h) {
        const F other = __shfl(stand, h, L);
        rank += other > stand || (other == stand && h < i) ? 1 : 0;
    }
    const bool in = i < a.n_group && rank < a.keep_groups;
    // the lowest that a group which stays may stand, the highest of one that does not; groups without experts are in their place
    const F err = (F)(0.5f * close_to(a)) * ((F)1 + size);
    const bool some = stand > (F)-INFINITY;
    const F low = lanes_max<L>(in && some ? err - stand : (F)-INFINITY);
    const F high = lanes_max<L>(!in && some ? stand + err : (F)-INFINITY);
    near = high >= -low;
    return (uint32_t)lanes_with<L>(in);
}

// Expert e's group stays.  e / n without a division: e < 256, 1 <= n <= 256.
__device__ __forceinline__ bool stays(uint32_t mask, int e, uint32_t inv) { return mask >> ((e * inv) >> 16) & 1u; }

// 1 / v to the last bits of fp64, without a division's special cases (v in 1 .. 2).
__device__ __forceinline__ double inverse(double v) {
    double r = __builtin_amdgcn_rcp(v);
    r = fma(fma(-v, r, 1.0), r, r);
    return fma(fma(-v, r, 1.0), r, r);
}

// The choice of one token in fp64, by the definition.  The whole wavefront calls it, whatever number of lanes share a
// token else: it is rare (under one token in a hundred) but has to be short, since its wavefront ends last.
// row: the token's logits, `by` [E] its LDS.  Lane j < top_k gets the j-th expert.
template <typename S>
__device__ __forceinline__ int choose_exact(const S* row, const RouteArgs& a, double* by) {
    constexpr int M = GLOWQ_MOE_MAX_EXPERTS / 64;
    const int lane = threadIdx.x & 63, E = a.n_exp;
    const bool softmax = a.score == GLOWQ_SCORE_SOFTMAX;
    float v[M], b[M], most = -INFINITY;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        const int e = lane + 64 * j;
        v[j] = e < E ? (float)row[e] : -INFINITY;
        b[j] = a.bias != nullptr && e < E ? a.bias[e] : 0.f;
        most = fmaxf(most, v[j]);
    }
    const double top = lanes_max<64>(most);
    double s[M], u[M], sum = 0.0;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        const double l = (double)v[j], x = exp(softmax ? l - top : -fabs(l));
        s[j] = v[j] == -INFINITY ? 0.0 : (softmax ? x : (v[j] >= 0.f ? inverse(1.0 + x) : x * inverse(1.0 + x)));
        sum += s[j];
    }
    sum = softmax ? lanes_sum<64>(sum) : 1.0;
#pragma unroll
    for (int j = 0; j < M; ++j) {
        if (softmax) s[j] /= sum;
        s[j] = v[j] == -INFINITY ? -INFINITY : s[j] + (double)b[j];
        u[j] = a.bias != nullptr ? s[j] : (double)v[j];
    }
    if (a.keep_groups < a.n_group) {
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (lane + 64 * j < E) by[lane + 64 * j] = a.group_best == 2 ? s[j] : u[j];
        wave_sync();
        bool near;
        const uint32_t mask = groups_that_stay<64>(by, a, lane, near);
        wave_sync();
        const uint32_t inv = (65535u + (uint32_t)(E / a.n_group)) / (uint32_t)(E / a.n_group);
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (lane + 64 * j < E && !stays(mask, lane + 64 * j, inv)) u[j] = -INFINITY;
    }
    int mine = -1;
#pragma unroll 1
    for (int r = 0; r < a.top_k; ++r) {
        double best = u[0];
#pragma unroll
        for (int j = 1; j < M; ++j) best = fmax(best, u[j]);
        best = lanes_max<64>(best);
        if (best == -INFINITY) break;
        int at = 0;  // the lowest expert that has it
#pragma unroll
        for (int j = M - 1; j >= 0; --j) {
            const uint64_t who = __ballot(u[j] == best);
            if (who != 0) at = 64 * j + __ffsll((unsigned long long)who) - 1;
        }
#pragma unroll
        for (int j = 0; j < M; ++j)
            if (lane + 64 * j == at) u[j] = -INFINITY;
        if (lane == r) mine = at;
    }
    return mine;
}

// SCORED: scores decide (a bias, or groups by two scores).
template <typename S, int L, int EPL, int KL, bool SCORED>
__global__ __launch_bounds__(kRouteThreads, 6) void route_kernel(const RouteArgs a) {
    constexpr int TB = kRouteThreads / L;
    // values of each token, and when those are used up, of one token of a wavefront in fp64
    constexpr int W = TB / (kRouteThreads / 64), kEach = SCORED && L * EPL * W < 2 * GLOWQ_MOE_MAX_EXPERTS
                                                             ? 2 * GLOWQ_MOE_MAX_EXPERTS / W : L * EPL;
    __shared__ __attribute__((aligned(16))) float by_all[TB][kEach];
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
        top = fmaxf(lanes_max<L>(top), -FLT_MAX);  // a row without experts: no NaN
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
        float* by = by_all[slot];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            float s;
            if (softmax) {
                s = __expf(v[j] - top) * rs;
            } else {
                const float x = __expf(-fabsf(v[j])), q = __builtin_amdgcn_rcpf(1.f + x);
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
            if (groups && i + L * j < E) by_all[slot][i + L * j] = v[j];
        }
    }
    if (groups) {
        wave_sync();
        bool close;
        mask = groups_that_stay<L>(static_cast<const float*>(by_all[slot]), a, i, close);
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
            near |= hi - lo <= close_to(a) * (1.f + fabsf(hi));
        }
        last = best;
        if (i == r) mine = best;
    }
    int e = mine > kOut ? key_expert(mine) : -1;
    if constexpr (SCORED) {
        // one token after another, all lanes for each
        for (uint64_t todo = __ballot(near && live && i == 0); todo != 0; todo &= todo - 1) {
            const int first = __ffsll((unsigned long long)todo) - 1;  // its first lane
            const int who = ((int)threadIdx.x & ~63) / L + first / L;
            const int got = choose_exact(static_cast<const S*>(a.logits) + (size_t)(blockIdx.x * TB + who) * E, a,
                                         reinterpret_cast<double*>(by_all[((int)threadIdx.x & ~63) / L]));
            const int mine_now = __shfl(got, i, 64);
            if (slot == who) e = mine_now;
        }
    }
    if (bad || i >= K) e = -1;
    // weights: lane j has the j-th expert
    const float l = e >= 0 ? (float)row[e] : -INFINITY;
    float w = 0.f;
    if (a.renorm) {
        // the chosen scores over their sum
        const float m = fmaxf(lanes_max<L>(l), -FLT_MAX);
        const float s = e < 0 ? 0.f : score_beside(l, m, softmax);
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
    const bool there = t < a.T;
    const int E = a.n_exp, K = a.top_k;
    const S* row = static_cast<const S*>(a.logits) + (size_t)(there ? t : 0) * E;
    const bool softmax = a.score == GLOWQ_SCORE_SOFTMAX;
    int e = -1;
    float dw = 0.f;
    if (i < K && there) {
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
    bool live = false;
    if (a.renorm) {
        const float m = fmaxf(lanes_max<L>(l), -FLT_MAX);
        const float s = e < 0 ? 0.f : score_beside(l, m, softmax);
        const float all = lanes_sum<L>(s);
        const float share = e < 0 ? 0.f : s / all;
        const float c = lanes_sum<L>(share * dw);
        g = a.scale * share * (dw - c) * (softmax ? 1.f : sigmoid_of(-l));
    } else if (softmax) {
        live = lanes_with<L>(e >= 0) != 0;  // else the row is zeros: a refused one's logits may hold NaN
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            v[j] = i + L * j < E ? (float)row[i + L * j] : -INFINITY;
            top = fmaxf(top, v[j]);
        }
        top = fmaxf(lanes_max<L>(top), -FLT_MAX);
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
    if (!there) return;
    S* out = static_cast<S*>(a.out) + (size_t)t * E;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int x = i + L * j;
        if (x < E) out[x] = (S)(live ? p[j] * (mine[x] - dot) : mine[x]);
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

// 16 lanes a token and lists no longer than the choices need, more lanes past 8 choices (16384 tokens fp32, softmax / sigmoid
// with a bias, us: 60 experts, 4 choices 4.2 / 7.5, in the next form 5.5 / 9.0, on 64 lanes 9.9 / 15; 128 experts, 4 choices
// 4.9 / 9.1, longer lists 5.7 / 9.3; 256 experts, 4 choices 6.8 / 12, longer lists 8.1 / 12.9, 8 choices 9.5 / 15.4, 64 lanes
// 13.7 / 22.7).
template <typename S>
hipError_t launch_route_t(const RouteArgs& a, hipStream_t stream) {
    if (a.top_k > 8) return launch_route_n<S, 64, 4, 4>(a, stream);
    if (a.n_exp <= 64) return launch_route_n<S, 16, 4, 4>(a, stream);
    if (a.n_exp <= 128) return a.top_k <= 4 ? launch_route_n<S, 16, 8, 5>(a, stream) : launch_route_n<S, 16, 8, 8>(a, stream);
    return a.top_k <= 4 ? launch_route_n<S, 16, 16, 5>(a, stream) : launch_route_n<S, 16, 16, 9>(a, stream);
}

// 16384 tokens, us: 60 experts, 8 choices 4.3, in the last form 5.4, on 64 lanes 7.4; 256 experts, 16 choices 9.4, 64 lanes 11.2.
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
