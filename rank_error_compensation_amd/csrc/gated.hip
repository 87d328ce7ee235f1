// The gated activation between the gate/up and the down projection of an MLP,
//   h = g s(g) u,   s(g) = 1 / (1 + exp(-g)),
// and its gradients  dg = dh u s (1 + g (1 - s)),  du = dh g s,  over n values of any shape.
// With e = exp(-|g|) and q = 1 / (1 + e):  s = q and 1 - s = e q for g >= 0, s = e q and 1 - s = q
// below -- no overflow and no cancellation at either end.  fp32 arithmetic, one rounding.
// Bound by memory: 3 values moved per output value, 5 for the gradients; a thread takes 16 bytes of each.
// Tensors above kStreamBytes go past the caches (the fp32 gradients of 16383 x 1408 values, 461 MB, cold: 75 us,
// 6.1 TB/s; 85 us through them).  A few rows are bound by the launch (4 x 1408 values: 2.2 us).
#include <algorithm>

#include "glowq.h"
#include "layer.h"

namespace glowq {

namespace {

constexpr int kGateThreads = 256;

template <typename S>
struct Gate {
    static constexpr int N = 16 / sizeof(S);
    S v[N];
};

__device__ __forceinline__ void sigmoid_pair(float g, float& s, float& one_minus_s) {
    const float e = expf(-fabsf(g)), q = 1.0f / (1.0f + e), eq = e * q;
    s = g >= 0.f ? q : eq;
    one_minus_s = g >= 0.f ? eq : q;
}

template <typename S, bool NT>
__device__ __forceinline__ Gate<S> load_gate(const S* p, int64_t i, int64_t n) {
    if (i + Gate<S>::N <= n) {
        const u4* q = reinterpret_cast<const u4*>(p + i);
        return __builtin_bit_cast(Gate<S>, NT ? __builtin_nontemporal_load(q) : *q);
    }
    Gate<S> r;
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k) r.v[k] = i + k < n ? p[i + k] : (S)0.f;
    return r;
}

template <typename S, bool NT>
__device__ __forceinline__ void store_gate(S* p, int64_t i, int64_t n, const Gate<S>& r) {
    if (i + Gate<S>::N <= n) {
        u4* q = reinterpret_cast<u4*>(p + i);
        if constexpr (NT) __builtin_nontemporal_store(__builtin_bit_cast(u4, r), q);
        else *q = __builtin_bit_cast(u4, r);
        return;
    }
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k)
        if (i + k < n) p[i + k] = r.v[k];
}

template <typename S, bool NT>
__global__ __launch_bounds__(kGateThreads) void swiglu_kernel(const S* gate, const S* up, int64_t n, S* h) {
    const int64_t i = ((int64_t)blockIdx.x * kGateThreads + threadIdx.x) * Gate<S>::N;
    if (i >= n) return;
    const Gate<S> g = load_gate<S, NT>(gate, i, n), u = load_gate<S, NT>(up, i, n);
    Gate<S> r;
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k) {
        float s, t;
        sigmoid_pair((float)g.v[k], s, t);
        r.v[k] = (S)((float)g.v[k] * s * (float)u.v[k]);
    }
    store_gate<S, NT>(h, i, n, r);
}

template <typename S, bool NT>
__global__ __launch_bounds__(kGateThreads) void swiglu_backward_kernel(const S* dh, const S* gate, const S* up, int64_t n,
                                                                       S* dgate, S* dup) {
    const int64_t i = ((int64_t)blockIdx.x * kGateThreads + threadIdx.x) * Gate<S>::N;
    if (i >= n) return;
    const Gate<S> d = load_gate<S, NT>(dh, i, n), g = load_gate<S, NT>(gate, i, n), u = load_gate<S, NT>(up, i, n);
    Gate<S> rg, ru;
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k) {
        const float gf = (float)g.v[k], df = (float)d.v[k];
        float s, t;
        sigmoid_pair(gf, s, t);
        rg.v[k] = (S)(s * fmaf(gf, t, 1.f) * df * (float)u.v[k]);  // the bounded factors first: no early overflow
        ru.v[k] = (S)(gf * s * df);
    }
    store_gate<S, NT>(dgate, i, n, rg);
    store_gate<S, NT>(dup, i, n, ru);
}

template <typename S>
unsigned gate_grid(int64_t n) {
    return (unsigned)ceil_div(n, (int64_t)kGateThreads * Gate<S>::N);
}

}  // namespace

template <typename S>
static hipError_t launch_swiglu_t(const void* gate, const void* up, int64_t n, void* h, hipStream_t stream) {
    const dim3 grid(gate_grid<S>(n)), block(kGateThreads);
    const S *g = static_cast<const S*>(gate), *u = static_cast<const S*>(up);
    if (n * (int64_t)sizeof(S) > kStreamBytes)
        hipLaunchKernelGGL((swiglu_kernel<S, true>), grid, block, 0, stream, g, u, n, static_cast<S*>(h));
    else
        hipLaunchKernelGGL((swiglu_kernel<S, false>), grid, block, 0, stream, g, u, n, static_cast<S*>(h));
    return hipGetLastError();
}

hipError_t launch_swiglu(const void* gate, const void* up, int64_t n, int32_t dtype, void* h, hipStream_t stream) {
    return dtype == GLOWQ_DTYPE_F16 ? launch_swiglu_t<_Float16>(gate, up, n, h, stream)
                                    : launch_swiglu_t<float>(gate, up, n, h, stream);
}

template <typename S>
static hipError_t launch_swiglu_backward_t(const void* dh, const void* gate, const void* up, int64_t n, void* dgate,
                                           void* dup, hipStream_t stream) {
    const dim3 grid(gate_grid<S>(n)), block(kGateThreads);
    const S *d = static_cast<const S*>(dh), *g = static_cast<const S*>(gate), *u = static_cast<const S*>(up);
    if (n * (int64_t)sizeof(S) > kStreamBytes)
        hipLaunchKernelGGL((swiglu_backward_kernel<S, true>), grid, block, 0, stream, d, g, u, n, static_cast<S*>(dgate),
                           static_cast<S*>(dup));
    else
        hipLaunchKernelGGL((swiglu_backward_kernel<S, false>), grid, block, 0, stream, d, g, u, n, static_cast<S*>(dgate),
                           static_cast<S*>(dup));
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const void* dh, const void* gate, const void* up, int64_t n, int32_t dtype,
                                  void* dgate, void* dup, hipStream_t stream) {
    return dtype == GLOWQ_DTYPE_F16 ? launch_swiglu_backward_t<_Float16>(dh, gate, up, n, dgate, dup, stream)
                                    : launch_swiglu_backward_t<float>(dh, gate, up, n, dgate, dup, stream);
}

}  // namespace glowq
