// Rows of a mixture-of-experts layer: the lists that send tokens to experts, the rows' way into
// expert order and back with the router's weights, and the gradients of both.
//
//   pair p = (t, j) = t top_k + j: token t's j-th choice, an expert id or -1 (no row)
//   sort      pairs with an expert take rows 0, 1, ... by (expert, p); offsets[e] is expert e's
//             first row, row_token[row] = t, pair_row[p] = row (-1 without an expert)
//   dispatch  rows[i] = x[row_token[i]];  its gradient is combine without weights
//   combine   y[t] = add[t] + sum_j w[t, j] rows[pair_row[t, j]]       (fp32, j in order)
//   gradient  d_rows[pair_row[t, j]] = w[t, j] dy[t],  dw[t, j] = sum_c dy[t, c] rows[.][c]
//
// All of it moves memory: every row crosses HBM once (the gradient's rows twice: read for dw,
// written for d_rows) and the token side once, since one workgroup or wavefront holds a token's
// values while it goes over its choices.  No floating atomics: a row belongs to one pair, so
// results do not depend on the order of execution.
#include <algorithm>

#include "glowq.h"
#include "layer.h"

namespace glowq {

namespace {

constexpr int kSortWaves = kSortThreads / 64;
constexpr int kBuckets = kMoeMaxExperts + 1;
constexpr int kHistStride = kBuckets + 3;

__device__ __forceinline__ void raise_routing(int32_t* err) {
    __hip_atomic_fetch_or(err, 2, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ int bucket_of(int id, int n_exp, bool& bad) {
    const bool in = id >= 0 && id < n_exp;
    bad |= !in && id != -1;
    return in ? id : n_exp;
}

// Exclusive prefix over the first kBuckets threads of the workgroup (others pass 0).
__device__ int bucket_scan(int v, int* wsum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int incl = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int n = __shfl_up(incl, off, 64);
        if (lane >= off) incl += n;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int base = 0;
    constexpr int kScanWaves = (kBuckets + 63) / 64;
#pragma unroll
    for (int w = 0; w < kScanWaves; ++w) base += w < wave ? wsum[w] : 0;
    return base + incl - v;
}

// Counts of one chunk per bucket.  Launch-bound: 262144 pairs on 256 workgroups 2.5 us.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const SortArgs a) {
    __shared__ int hist[kBuckets];
    const int nb = a.n_exp + 1;
    for (int b = threadIdx.x; b < nb; b += kSortThreads) hist[b] = 0;
    __syncthreads();
    const int begin = blockIdx.x * a.chunk, end = min(begin + a.chunk, a.n);
    bool bad = false;
    for (int p = begin + threadIdx.x; p < end; p += kSortThreads) atomicAdd(&hist[bucket_of(a.ids[p], a.n_exp, bad)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < nb; b += kSortThreads) a.part[blockIdx.x * nb + b] = hist[b];
}

// Places one chunk.  Every wavefront owns a contiguous piece of the chunk and its own counters, so
// that rows of one expert keep the pairs' order: counters[wave][bucket] first count the piece, then
// hold the next free row (expert start + earlier chunks + earlier wavefronts); 64 pairs at a time
// take theirs, a lane's place among the lanes of its bucket found from ballots of the bucket's bits.
// Bound by latency, not by its 12 bytes a pair: in one workgroup a token's four choices take 2.5 us; 262144
// pairs over 60 experts on 256 workgroups, each of which adds up all workgroups' counts, 6.9 us
// (all of a thread's counts loaded at once: 0.4 us less there, 0.8 more at 16384 pairs).
template <bool ONE>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const SortArgs a) {
    __shared__ int cnt[kSortWaves * kHistStride];
    __shared__ int wsum[kSortWaves];
    __shared__ int red[ONE ? 2 : 2 * kSortThreads];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.n_exp, nb = E + 1;
    for (int i = tid; i < kSortWaves * kHistStride; i += kSortThreads) cnt[i] = 0;
    __syncthreads();
    const int begin = ONE ? 0 : blockIdx.x * a.chunk, end = ONE ? a.n : min(begin + a.chunk, a.n);
    const int piece = ((end - begin + kSortThreads - 1) / kSortThreads) * 64;
    const int p0 = begin + wave * piece, p1 = min(p0 + piece, end);
    int* mine = cnt + wave * kHistStride;
    bool bad = false;
    for (int p = p0 + lane; p < p1; p += 64) atomicAdd(&mine[bucket_of(a.ids[p], E, bad)], 1);
    if (bad) raise_routing(a.err);
    int total = 0, before = 0;
    if constexpr (!ONE) {
        // chunk counts of all workgroups: slices of the list side by side, P buckets each
        int P = 64;
        while (P < nb) P <<= 1;
        const int slices = kSortThreads / P, b = tid & (P - 1), s = tid / P;
        const int per = (a.n_blocks + slices - 1) / slices;
        const int k0 = s * per, k1 = min(k0 + per, a.n_blocks);
        int tot = 0, pre = 0;
        if (b < nb) {
#pragma unroll 4
            for (int k = k0; k < k1; ++k) {
                const int v = a.part[k * nb + b];
                tot += v;
                pre += k < (int)blockIdx.x ? v : 0;
            }
        }
        red[tid] = tot;
        red[kSortThreads + tid] = pre;
        __syncthreads();
        if (tid < nb) {
            for (int i = 0; i < slices; ++i) {
                total += red[i * P + tid];
                before += red[kSortThreads + i * P + tid];
            }
        }
    }
    __syncthreads();
    if constexpr (ONE) {
        if (tid < nb)
            for (int w = 0; w < kSortWaves; ++w) total += cnt[w * kHistStride + tid];
    }
    const int start = bucket_scan(tid < nb ? total : 0, wsum);
    if (tid < nb) {
        if (blockIdx.x == 0) a.offsets[tid] = start;
        int run = start + before;
        for (int w = 0; w < kSortWaves; ++w) {
            const int c = cnt[w * kHistStride + tid];
            cnt[w * kHistStride + tid] = run;
            run += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz((unsigned)E);  // buckets 0 .. E
    const unsigned long long below = (1ull << lane) - 1ull;
    for (int p = p0; p < p1; p += 64) {
        const int q = p + lane;
        const bool act = q < p1;
        const int b = act ? bucket_of(a.ids[q], E, bad) : 0;
        unsigned long long peers = __ballot(act);
        for (int i = 0; i < bits; ++i) {
            const unsigned long long m = __ballot((b >> i) & 1);
            peers &= ((b >> i) & 1) ? m : ~m;
        }
        const int rank = __popcll(peers & below);
        const int row = act ? mine[b] + rank : 0;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (act && rank == 0) mine[b] = row + __popcll(peers);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (act) {
            a.row_token[row] = b < E ? (int)((unsigned)q / (unsigned)a.top_k) : -1;
            a.pair_row[q] = b < E ? row : -1;
        }
    }
}

// --------------------------------------------------------------------- rows
constexpr int kRowsThreads = 256;
constexpr int kDispatchRows = 2;  // rows in flight per thread

// Threads per row: a power of two, the whole workgroup for long rows.
inline int row_threads(int64_t chunks, int most) {
    int t = 1;
    while (t < most && t < chunks) t <<= 1;
    return t;
}

// Bound by memory: 8188 rows of 4 KB out of 2047 take 8.4 us warm (33.5 MB written, 8.4 MB read: 5.0 TB/s).
// Two rows a thread keep enough loads in flight (one or eight: no faster).
// V: the piece of a row that one thread moves at a time (16 bytes where rows are multiples of it).
// NT: rows written past the caches (32764 rows of 4 KB, cold: 38 us, 43 through them; 8188 rows: 10.6, 11.1).
template <typename V, bool NT>
__global__ __launch_bounds__(kRowsThreads) void dispatch_kernel(const RowsArgs a, int chunks, int tpr) {
    const int per = kRowsThreads / tpr, sub = threadIdx.x / tpr, c0 = threadIdx.x & (tpr - 1);
    const int64_t base = (int64_t)blockIdx.x * (per * kDispatchRows) + sub;
    const V* src[kDispatchRows];
    V* dst[kDispatchRows];
#pragma unroll
    for (int i = 0; i < kDispatchRows; ++i) {
        const int64_t row = base + (int64_t)i * per;
        src[i] = nullptr;
        dst[i] = nullptr;
        if (row >= a.n_rows) continue;
        const int t = a.row_token[row];
        if (t >= 0 && t < a.T) src[i] = static_cast<const V*>(a.x) + (size_t)t * chunks;
        else if (t != -1 && c0 == 0) raise_routing(a.err);
        dst[i] = static_cast<V*>(a.out) + (size_t)row * chunks;
    }
    for (int c = c0; c < chunks; c += tpr) {
        V v[kDispatchRows];
#pragma unroll
        for (int i = 0; i < kDispatchRows; ++i) v[i] = src[i] != nullptr ? src[i][c] : V{};
#pragma unroll
        for (int i = 0; i < kDispatchRows; ++i)
            if (dst[i] != nullptr) {
                if constexpr (NT) __builtin_nontemporal_store(v[i], dst[i] + c);
                else dst[i][c] = v[i];
            }
    }
}

// N values of type S as fp32: one 16-byte load (N S's to 16 bytes), or one value (N = 1) where rows are not
// multiples of 16 bytes -- 2 or 4 bytes a lane, far from the memory's rate: combine of 4096 tokens x 4 x 2050
// fp16 79 us, of 2048 columns 22; its gradients 79 and 30; fp32 72 and 37, 78 and 53.  NT: past the caches,
// for 16-byte pieces of rows that outgrow them (kStreamBytes): cold, combine of 65536 x 2048 fp16 rows takes 69 us against
// 77, its gradients for 8191 tokens (rows read so, written as usual) 58 against 71, the fp32 dispatch
// gradient of 16384 rows 30 against 34.
template <typename S, int N>
struct Pack {
    S v[N];
};
template <typename S, int N, bool NT>
__device__ __forceinline__ void load_f32(const S* p, float (&f)[N]) {
    static_assert(N > 1 || !NT, "single values go through the caches");
    if constexpr (N > 1) {
        const u4 raw = NT ? __builtin_nontemporal_load(reinterpret_cast<const u4*>(p)) : *reinterpret_cast<const u4*>(p);
        const Pack<S, N> q = __builtin_bit_cast(Pack<S, N>, raw);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = (float)q.v[i];
    } else {
        f[0] = (float)p[0];
    }
}
template <typename S, int N, bool NT>
__device__ __forceinline__ void store_f32(S* p, const float (&f)[N]) {
    if constexpr (N > 1) {
        Pack<S, N> q;
#pragma unroll
        for (int i = 0; i < N; ++i) q.v[i] = (S)f[i];
        if constexpr (NT) __builtin_nontemporal_store(__builtin_bit_cast(u4, q), reinterpret_cast<u4*>(p));
        else *reinterpret_cast<u4*>(p) = __builtin_bit_cast(u4, q);
    } else {
        p[0] = (S)f[0];
    }
}

constexpr int kChoices = 4;  // choices whose rows are loaded together

// y[t] for kRowsThreads / tpr tokens per workgroup, columns in N-value pieces.  A thread adds up all choices of
// its columns in registers, the rows of kChoices of them in flight: every row is read once and y written once.
// Bound by memory: 16384 tokens x 4 choices x 2048 fp16 (402 MB with the added rows) 68 us, 5.9 TB/s (rows
// partly in the caches of the call before); as the gradient of a dispatch, 4096 tokens x 4 x 2048 fp32, 28 us.
template <typename S, int N, bool NT>
__global__ __launch_bounds__(kRowsThreads) void combine_kernel(const RowsArgs a, int chunks, int tpr) {
    const int per = kRowsThreads / tpr, sub = threadIdx.x / tpr;
    const int64_t t = (int64_t)blockIdx.x * per + sub;
    if (t >= a.T) return;
    const int k = a.top_k;
    const int32_t* pr = a.pair_row + t * k;
    const float* w = a.w != nullptr ? a.w + t * k : nullptr;
    const S* rows = static_cast<const S*>(a.x);
    const int c0 = (threadIdx.x & (tpr - 1)) + blockIdx.y * tpr, step = tpr * gridDim.y;
    for (int c = c0; c < chunks; c += step) {
        const size_t col = (size_t)c * N;
        float acc[N];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = 0.f;
        for (int j0 = 0; j0 < k; j0 += kChoices) {
            float v[kChoices][N], wj[kChoices];
            bool ok[kChoices];
#pragma unroll
            for (int u = 0; u < kChoices; ++u) {
                const int j = min(j0 + u, k - 1);
                const int row = pr[j];
                ok[u] = j0 + u < k && row >= 0 && row < a.n_rows;
                if (j0 + u < k && row != -1 && !ok[u] && c == 0) raise_routing(a.err);
                wj[u] = w != nullptr ? w[j] : 1.f;
                if (ok[u]) load_f32<S, N, NT>(rows + (size_t)row * a.d + col, v[u]);
            }
#pragma unroll
            for (int u = 0; u < kChoices; ++u)
                if (ok[u]) {
#pragma unroll
                    for (int i = 0; i < N; ++i) acc[i] = fmaf(wj[u], v[u][i], acc[i]);
                }
        }
        if (a.add != nullptr) {
            float b[N];
            load_f32<S, N, NT>(static_cast<const S*>(a.add) + (size_t)t * a.d + col, b);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] += b[i];
        }
        store_f32<S, N, NT>(static_cast<S*>(a.out) + (size_t)t * a.d + col, acc);
    }
}

// Rows of token -1 (behind the last expert's) belong to no pair: their gradient is zero.  A token out of
// range is reported here, since no pair need point at its row.  With a.whole the rows that no choice of
// their token takes are zeroed, too -- those that no wavefront of a token writes.  A wavefront clears its rows
// one after another, a value a lane: with one in 16 of 32764 pairs dropped and the lists left at T top_k rows
// of 2048 fp16 values the call takes 100 us, 60 with the lists cut to the rows in use.
template <typename S>
__device__ void zero_free_rows(const RowsArgs& a, int64_t first) {
    const int64_t row = first + threadIdx.x;
    const int t = row < a.n_rows ? a.row_token[row] : 0;
    const bool far = t < 0 || t >= a.T;
    if (row < a.n_rows && far && t != -1) raise_routing(a.err);
    bool unowned = t == -1;
    if (a.whole && row < a.n_rows) {
        unowned = true;
        for (int j = 0; j < a.top_k; ++j) unowned &= far || a.pair_row[(int64_t)t * a.top_k + j] != row;
    }
    unsigned long long free_rows = __ballot(row < a.n_rows && unowned);
    const int lane = threadIdx.x & 63;
    const int64_t row0 = first + (threadIdx.x & ~63);
    while (free_rows != 0) {
        const int i = __builtin_ctzll(free_rows);
        free_rows &= free_rows - 1;
        S* dst = static_cast<S*>(a.out) + (size_t)(row0 + i) * a.d;
        for (int64_t c = lane; c < a.d; c += 64) dst[c] = (S)0.f;
    }
}

// One wavefront per token (and, in the last workgroups, 64 rows per wavefront to look for free
// ones).  Lane j < top_k holds choice j: its row counts when it lies in range,
// row_token names this token and no earlier choice of the token has it -- so that a row is written
// by one wavefront once, whatever the lists hold; anything else but -1 raises the error word.
// NT: 1 for rows that outgrow the caches, 2 where dy is read once too (it is read again for every
// kChoices choices).
// A wavefront holds its token's dy piece while it goes over the choices: dy once, the rows once read and once
// written.  Bound by memory: 8191 tokens x 4 x 2048 fp16 (302 MB) 56 to 58 us, 5.2 TB/s.
template <typename S, int N, int NT>
__global__ __launch_bounds__(kRowsThreads) void combine_backward_kernel(const RowsArgs a, int chunks, int token_blocks) {
    if ((int)blockIdx.x >= token_blocks) {
        zero_free_rows<S>(a, (int64_t)((int)blockIdx.x - token_blocks) * kRowsThreads);
        return;
    }
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * (kRowsThreads / 64) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    if (t >= a.T) return;
    const int k = a.top_k;
    int slot = -1;
    float weight = 0.f;
    if (lane < k) {
        slot = a.pair_row[t * k + lane];
        weight = a.w != nullptr ? a.w[t * k + lane] : 1.f;
    }
    bool bad = slot < -1 || slot >= a.n_rows;
    if (slot >= 0 && !bad) bad = a.row_token[slot] != (int)t;
    for (int j = 0; j + 1 < k; ++j) {
        const int earlier = __builtin_amdgcn_readlane(slot, j);
        bad |= lane > j && slot >= 0 && slot == earlier;
    }
    if (bad) raise_routing(a.err);
    const unsigned long long live = __ballot(slot >= 0 && !bad);
    const S* dy = static_cast<const S*>(a.x) + (size_t)t * a.d;
    float mine = 0.f;  // lane j: dw of choice j
    for (int j0 = 0; j0 < k; j0 += kChoices) {
        const S* src[kChoices];
        S* dst[kChoices];
        float wj[kChoices], dot[kChoices];
        bool ok[kChoices];
#pragma unroll
        for (int u = 0; u < kChoices; ++u) {
            const int j = min(j0 + u, k - 1);
            ok[u] = j0 + u < k && ((live >> j) & 1);
            const int row = ok[u] ? __builtin_amdgcn_readlane(slot, j) : 0;
            wj[u] = __shfl(weight, j, 64);
            src[u] = static_cast<const S*>(a.rows) + (size_t)row * a.d;
            dst[u] = static_cast<S*>(a.out) + (size_t)row * a.d;
            dot[u] = 0.f;
        }
        for (int c = lane; c < chunks; c += 64) {
            const size_t col = (size_t)c * N;
            float g[N], v[kChoices][N];
            load_f32<S, N, NT == 2>(dy + col, g);
#pragma unroll
            for (int u = 0; u < kChoices; ++u)
                if (ok[u]) load_f32<S, N, (NT > 0)>(src[u] + col, v[u]);
#pragma unroll
            for (int u = 0; u < kChoices; ++u)
                if (ok[u]) {
                    float o[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dot[u] = fmaf(g[i], v[u][i], dot[u]);
                        o[i] = wj[u] * g[i];
                    }
                    store_f32<S, N, false>(dst[u] + col, o);
                }
        }
#pragma unroll
        for (int u = 0; u < kChoices; ++u) {
            float s = dot[u];
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) s += __shfl_xor(s, off, 64);
            if (lane == j0 + u) mine = s;
        }
    }
    if (lane < k) a.dw[t * k + lane] = mine;
}

}  // namespace

hipError_t launch_moe_sort(const SortArgs& a, hipStream_t stream) {
    if (a.n_blocks == 1) {
        hipLaunchKernelGGL((sort_place_kernel<true>), dim3(1), dim3(kSortThreads), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(sort_count_kernel, dim3(a.n_blocks), dim3(kSortThreads), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((sort_place_kernel<false>), dim3(a.n_blocks), dim3(kSortThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch(const RowsArgs& a, hipStream_t stream) {
    const int64_t es = a.dtype == GLOWQ_DTYPE_F16 ? 2 : 4, bytes = a.d * es;
    const int64_t unit = bytes % 16 == 0 ? 16 : es, chunks = bytes / unit;
    const int tpr = row_threads(chunks, kRowsThreads);
    const unsigned grid = (unsigned)ceil_div(a.n_rows, (int64_t)(kRowsThreads / tpr) * kDispatchRows);
    const dim3 g(grid), block(kRowsThreads);
    const bool past = ((int64_t)a.n_rows + a.T) * bytes > kStreamBytes;
    if (unit == 16 && past) hipLaunchKernelGGL((dispatch_kernel<u4, true>), g, block, 0, stream, a, (int)chunks, tpr);
    else if (unit == 16) hipLaunchKernelGGL((dispatch_kernel<u4, false>), g, block, 0, stream, a, (int)chunks, tpr);
    else if (unit == 4) hipLaunchKernelGGL((dispatch_kernel<uint32_t, false>), g, block, 0, stream, a, (int)chunks, tpr);
    else hipLaunchKernelGGL((dispatch_kernel<uint16_t, false>), g, block, 0, stream, a, (int)chunks, tpr);
    return hipGetLastError();
}

// Rows that outgrow the eight L2 caches.
template <typename S>
static bool stream_rows(const RowsArgs& a) {
    return (int64_t)a.n_rows * a.d * (int64_t)sizeof(S) > kStreamBytes;
}

template <typename S, int N>
static hipError_t launch_combine_n(const RowsArgs& a, hipStream_t stream) {
    const int64_t chunks = a.d / N;
    const int tpr = row_threads(chunks, kRowsThreads);
    const int64_t blocks = ceil_div(a.T, kRowsThreads / tpr);
    // few tokens: a token's columns over several workgroups
    const int64_t ny = blocks >= 256 ? 1 : std::min<int64_t>(ceil_div(chunks, tpr), 16);
    const dim3 grid((unsigned)blocks, (unsigned)ny);
    if constexpr (N > 1) {
        if (stream_rows<S>(a)) {
            hipLaunchKernelGGL((combine_kernel<S, N, true>), grid, dim3(kRowsThreads), 0, stream, a, (int)chunks, tpr);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((combine_kernel<S, N, false>), grid, dim3(kRowsThreads), 0, stream, a, (int)chunks, tpr);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const RowsArgs& a, hipStream_t stream) {
    if (a.dtype == GLOWQ_DTYPE_F16)
        return a.d % 8 == 0 ? launch_combine_n<_Float16, 8>(a, stream) : launch_combine_n<_Float16, 1>(a, stream);
    return a.d % 4 == 0 ? launch_combine_n<float, 4>(a, stream) : launch_combine_n<float, 1>(a, stream);
}

template <typename S, int N>
static hipError_t launch_combine_backward_n(const RowsArgs& a, hipStream_t stream) {
    const int blocks = (int)ceil_div(a.T, kRowsThreads / 64);
    const unsigned grid = (unsigned)(blocks + ceil_div(a.n_rows, kRowsThreads));
    const dim3 g(grid), block(kRowsThreads);
    const int chunks = (int)(a.d / N);
    if constexpr (N > 1) {
        if (stream_rows<S>(a)) {
            if (a.top_k > kChoices)
                hipLaunchKernelGGL((combine_backward_kernel<S, N, 1>), g, block, 0, stream, a, chunks, blocks);
            else hipLaunchKernelGGL((combine_backward_kernel<S, N, 2>), g, block, 0, stream, a, chunks, blocks);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((combine_backward_kernel<S, N, 0>), g, block, 0, stream, a, chunks, blocks);
    return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const RowsArgs& a, hipStream_t stream) {
    if (a.dtype == GLOWQ_DTYPE_F16)
        return a.d % 8 == 0 ? launch_combine_backward_n<_Float16, 8>(a, stream)
                            : launch_combine_backward_n<_Float16, 1>(a, stream);
    return a.d % 4 == 0 ? launch_combine_backward_n<float, 4>(a, stream) : launch_combine_backward_n<float, 1>(a, stream);
}

}  // namespace glowq
