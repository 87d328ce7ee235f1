// The gated activation between the gate/up and the down projection of an MLP,
//   h = g s(g) u,   s(g) = 1 / (1 + exp(-g)),
// and its gradients  dg = dh u s (1 + g (1 - s)),  du = dh g s,  over n values of any shape.
// With e = exp(-|g|) and q = 1 / (1 + e):  s = q and 1 - s = e q for g >= 0, s = e q and 1 - s = q
// below -- no overflow and no cancellation at either end.  fp32 arithmetic, one rounding.
// Bound by memory: 3 values moved per output value, 5 for the gradients.
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

template <typename S>
__device__ __forceinline__ Gate<S> load_gate(const S* p, int64_t i, int64_t n) {
    if (i + Gate<S>::N <= n) return __builtin_bit_cast(Gate<S>, *reinterpret_cast<const u4*>(p + i));
    Gate<S> r;
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k) r.v[k] = i + k < n ? p[i + k] : (S)0.f;
    return r;
}

template <typename S>
__device__ __forceinline__ void store_gate(S* p, int64_t i, int64_t n, const Gate<S>& r) {
    if (i + Gate<S>::N <= n) {
        *reinterpret_cast<u4*>(p + i) = __builtin_bit_cast(u4, r);
        return;
    }
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k)
        if (i + k < n) p[i + k] = r.v[k];
}

template <typename S>
__global__ __launch_bounds__(kGateThreads) void swiglu_kernel(const S* gate, const S* up, int64_t n, S* h) {
    const int64_t i = ((int64_t)blockIdx.x * kGateThreads + threadIdx.x) * Gate<S>::N;
    if (i >= n) return;
    const Gate<S> g = load_gate(gate, i, n), u = load_gate(up, i, n);
    Gate<S> r;
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k) {
        float s, t;
        sigmoid_pair((float)g.v[k], s, t);
        r.v[k] = (S)((float)g.v[k] * s * (float)u.v[k]);
    }
    store_gate(h, i, n, r);
}

template <typename S>
__global__ __launch_bounds__(kGateThreads) void swiglu_backward_kernel(const S* dh, const S* gate, const S* up, int64_t n,
                                                                       S* dgate, S* dup) {
    const int64_t i = ((int64_t)blockIdx.x * kGateThreads + threadIdx.x) * Gate<S>::N;
    if (i >= n) return;
    const Gate<S> d = load_gate(dh, i, n), g = load_gate(gate, i, n), u = load_gate(up, i, n);
    Gate<S> rg, ru;
#pragma unroll
    for (int k = 0; k < Gate<S>::N; ++k) {
        const float gf = (float)g.v[k], df = (float)d.v[k];
        float s, t;
        sigmoid_pair(gf, s, t);
        rg.v[k] = (S)(df * (float)u.v[k] * s * fmaf(gf, t, 1.f));
        ru.v[k] = (S)(df * gf * s);
    }
    store_gate(dgate, i, n, rg);
    store_gate(dup, i, n, ru);
}

template <typename S>
unsigned gate_grid(int64_t n) {
    return (unsigned)ceil_div(n, (int64_t)kGateThreads * Gate<S>::N);
}

}  // namespace

hipError_t launch_swiglu(const void* gate, const void* up, int64_t n, int32_t dtype, void* h, hipStream_t stream) {
    if (dtype == GLOWQ_DTYPE_F16)
        hipLaunchKernelGGL((swiglu_kernel<_Float16>), dim3(gate_grid<_Float16>(n)), dim3(kGateThreads), 0, stream,
                           static_cast<const _Float16*>(gate), static_cast<const _Float16*>(up), n, static_cast<_Float16*>(h));
    else
        hipLaunchKernelGGL((swiglu_kernel<float>), dim3(gate_grid<float>(n)), dim3(kGateThreads), 0, stream,
                           static_cast<const float*>(gate), static_cast<const float*>(up), n, static_cast<float*>(h));
    return hipGetLastError();
}

hipError_t launch_swiglu_backward(const void* dh, const void* gate, const void* up, int64_t n, int32_t dtype,
                                  void* dgate, void* dup, hipStream_t stream) {
    if (dtype == GLOWQ_DTYPE_F16)
        hipLaunchKernelGGL((swiglu_backward_kernel<_Float16>), dim3(gate_grid<_Float16>(n)), dim3(kGateThreads), 0, stream,
                           static_cast<const _Float16*>(dh), static_cast<const _Float16*>(gate),
                           static_cast<const _Float16*>(up), n, static_cast<_Float16*>(dgate), static_cast<_Float16*>(dup));
    else
        hipLaunchKernelGGL((swiglu_backward_kernel<float>), dim3(gate_grid<float>(n)), dim3(kGateThreads), 0, stream,
                           static_cast<const float*>(dh), static_cast<const float*>(gate), static_cast<const float*>(up), n,
                           static_cast<float*>(dgate), static_cast<float*>(dup));
    return hipGetLastError();
}

}  // namespace glowq
