// Norm of all gradients as one vector, and clipping by it.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  g *= min(1, max_norm / (norm + 1e-6))
//
// Both are bound by HBM: the norm reads every element once, the clipping reads
// and writes every element once.  A list is cut into chunks of a fixed number
// of elements that blocks take in turn; the table of the tensors travels in the
// launch parameters, so a list costs one launch per kMaxTensors.  The clipping
// takes the chunks in descending order: what the norm read last is still in L2.
// A short list is one launch of one cluster that does both.
#include <math.h>

#include "ll_device.cuh"

namespace ll {
namespace {

constexpr int kThreads = 512;
constexpr int kBlocksPerSm = 4;
constexpr int kChunk = 32768;       // elements of a chunk
constexpr int kSmallCtas = 8;       // CTAs of the one-launch path's cluster
constexpr int kSmallChunk = 4096;
constexpr int64_t kSmallBytes = int64_t(4) << 20;  // most bytes of the one-launch path

// The tensors of a launch, up to N of them.
template <int N>
struct GradList {
    const void* data[N];
    int64_t n[N];
    int64_t first[N];  // number of the tensor's first chunk
    int64_t chunks;
    int chunk, count;
    uint8_t dtype[N];
};
constexpr int kFewTensors = 64;  // a launch with a short table costs the host less

// The elements [lo, hi) of one tensor that a chunk covers: the first chunk also
// takes the elements ahead of the first 16-byte boundary, so that every other
// chunk starts on one.
struct Range {
    int tensor;
    int64_t lo, body, hi;  // [lo, body) lie ahead of the boundary
};

template <int N>
__device__ __forceinline__ Range chunk_range(const GradList<N>& L, int64_t chunk) {
    int a = 0, b = L.count;  // last tensor whose first chunk is <= chunk
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (L.first[m] <= chunk)
            a = m;
        else
            b = m;
    }
    Range r;
    r.tensor = a;
    const int es = L.dtype[a] == LL_F32 ? 4 : 2;
    const int64_t n = L.n[a];
    int64_t head = ((16 - (reinterpret_cast<uintptr_t>(L.data[a]) & 15)) & 15) / es;
    if (head > n) head = n;
    const int64_t k = chunk - L.first[a];
    r.body = head + k * L.chunk;
    r.lo = k == 0 ? 0 : r.body;
    r.hi = r.body + L.chunk < n ? r.body + L.chunk : n;
    return r;
}

// A thread's sum of squares: FP32 sums of one chunk's share (at most 72 terms),
// added as a pair while every chunk's largest element lies in [2^-50, 2^55],
// where neither the squares nor their sums leave the FP32 range nor lose what
// matters; other chunks are squared again in 64 bits.
struct Squares {
    Pair sum = {0.f, 0.f};
    double wide = 0;
    bool used_wide = false;
};

template <typename T>
__device__ void add_squares(const T* __restrict__ p, const Range& r, Squares& q) {
    constexpr int E = 16 / sizeof(T);
    const int64_t vecs = (r.hi - r.body) / E;
    float s = 0.f, big = 0.f;
    auto add1 = [&](float x) {
        s = fmaf(x, x, s);
        big = fmaxf(big, fabsf(x));
    };
    if (r.lo + threadIdx.x < r.body) add1(Elem<T>::to_f(p[r.lo + threadIdx.x]));
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vecs; i += kThreads) {
        Pack<T, E> x;
        x.load(p + r.body + i * E);
#pragma unroll
        for (int j = 0; j < E; ++j) add1(Elem<T>::to_f(x.e[j]));
    }
    const int64_t tail = r.body + vecs * E + threadIdx.x;
    if (tail < r.hi) add1(Elem<T>::to_f(p[tail]));
    // a NaN is in s whatever the largest of the others is
    if (big == 0.f || (big >= 0x1p-50f && big <= 0x1p55f)) {
        q.sum = add(q.sum, Pair{s, 0.f});
        return;
    }
    auto add64 = [&](T x) {
        const double f = Elem<T>::to_f(x);
        q.wide += f * f;
    };
    q.used_wide = true;
    if (r.lo + threadIdx.x < r.body) add64(p[r.lo + threadIdx.x]);
    for (int64_t i = threadIdx.x; i < vecs; i += kThreads)
        for (int j = 0; j < E; ++j) add64(p[r.body + i * E + j]);
    if (tail < r.hi) add64(p[tail]);
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The block's sum, in thread 0.  In pairs; in 64 bits where a thread needed them.
__device__ double block_sum(const Squares& q) {
    __shared__ Pair pairs[kThreads / 32];
    __shared__ double wides[kThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool wide = __syncthreads_or(q.used_wide);
    const Pair p = warp_sum(q.sum);
    if (lane == 0) pairs[warp] = p;
    if (wide) {
        const double d = warp_sum(q.wide);
        if (lane == 0) wides[warp] = d;
    }
    __syncthreads();
    double s = 0;
    if (warp == 0) {
        const Pair x = warp_sum(lane < kThreads / 32 ? pairs[lane] : Pair{0.f, 0.f});
        s = static_cast<double>(x.hi) + x.lo;
        if (wide) s += warp_sum(lane < kThreads / 32 ? wides[lane] : 0.0);
    }
    __syncthreads();
    return s;
}

// Squares of the list's chunks `first`, `first + step`, ...
template <int N>
__device__ __forceinline__ void list_squares(const GradList<N>& L, int64_t first, int64_t step,
                                             Squares& q) {
    for (int64_t c = first; c < L.chunks; c += step) {
        const Range r = chunk_range(L, c);
        const void* p = L.data[r.tensor];
        switch (L.dtype[r.tensor]) {
            case LL_F32: add_squares(static_cast<const float*>(p), r, q); break;
            case LL_F16: add_squares(static_cast<const __half*>(p), r, q); break;
            default: add_squares(static_cast<const __nv_bfloat16*>(p), r, q);
        }
    }
}

template <typename T>
__device__ void scale_range(T* __restrict__ p, const Range& r, float coef) {
    constexpr int E = 16 / sizeof(T);
    const int64_t vecs = (r.hi - r.body) / E;
    auto one = [&](T x) { return Elem<T>::from_f(Elem<T>::to_f(x) * coef); };
    if (r.lo + threadIdx.x < r.body) p[r.lo + threadIdx.x] = one(p[r.lo + threadIdx.x]);
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vecs; i += kThreads) {
        Pack<T, E> x;
        x.load(p + r.body + i * E);
#pragma unroll
        for (int j = 0; j < E; ++j) x.e[j] = one(x.e[j]);
        x.store(p + r.body + i * E);
    }
    const int64_t tail = r.body + vecs * E + threadIdx.x;
    if (tail < r.hi) p[tail] = one(p[tail]);
}

// Chunks `last`, `last - step`, ... scaled for the norm.
template <int N>
__device__ __forceinline__ void list_scale(const GradList<N>& L, int64_t last, int64_t step,
                                           float norm, float max_norm) {
    const float c = max_norm / (norm + 1e-6f);
    if (c >= 1.f) return;  // a NaN goes on: it belongs in the gradients too
    for (int64_t i = last; i >= 0; i -= step) {
        const Range r = chunk_range(L, i);
        void* p = const_cast<void*>(L.data[r.tensor]);
        switch (L.dtype[r.tensor]) {
            case LL_F32: scale_range(static_cast<float*>(p), r, c); break;
            case LL_F16: scale_range(static_cast<__half*>(p), r, c); break;
            default: scale_range(static_cast<__nv_bfloat16*>(p), r, c);
        }
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_squares_kernel(
    const __grid_constant__ GradList<N> L, double* __restrict__ part) {
    launch_dependents();
    Squares q;
    list_squares(L, blockIdx.x, gridDim.x, q);
    const double s = block_sum(q);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The root of the sum of the blocks' sums.
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* __restrict__ part,
                                                             int64_t parts,
                                                             float* __restrict__ norm) {
    wait_for_prerequisites();
    launch_dependents();
    Squares q;
    for (int64_t i = threadIdx.x; i < parts; i += kThreads) {
        const double s = part[i];
        if (s == 0.0 || (s >= 0x1p-90 && s <= 0x1p110)) {
            q.sum = add(q.sum, pair_of(s));
        } else {
            q.wide += s;
            q.used_wide = true;
        }
    }
    const double s = block_sum(q);
    if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(s));
}

template <int N>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) grad_clip_kernel(
    const __grid_constant__ GradList<N> L, const float* __restrict__ norm, float max_norm) {
    wait_for_prerequisites();
    list_scale(L, L.chunks - 1 - blockIdx.x, gridDim.x, __ldcg(norm), max_norm);
}

// The norm of a short list, and with max_norm > 0 its clipping, by one cluster.
__global__ void __cluster_dims__(kSmallCtas, 1, 1) __launch_bounds__(kThreads)
    grad_small_kernel(const __grid_constant__ GradList<kFewTensors> L, float max_norm,
                      float* __restrict__ norm) {
    __shared__ double mine;
    __shared__ float total;
    Squares q;
    list_squares(L, blockIdx.x, kSmallCtas, q);
    const double s = block_sum(q);
    if (threadIdx.x == 0) mine = s;
    __syncthreads();
    cluster_barrier();
    if (threadIdx.x == 0) {
        double d[kSmallCtas], sum = 0;
#pragma unroll
        for (int r = 0; r < kSmallCtas; ++r)
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(d[r]) : "r"(cluster_addr(&mine, r)));
#pragma unroll
        for (int r = 0; r < kSmallCtas; ++r) sum += d[r];
        total = static_cast<float>(sqrt(sum));
        if (blockIdx.x == 0) norm[0] = total;
    }
    __syncthreads();
    if (max_norm > 0.f)
        list_scale(L, (L.chunks - 1 - blockIdx.x) / kSmallCtas * kSmallCtas + blockIdx.x, kSmallCtas,
                   total, max_norm);
    cluster_barrier();  // no CTA leaves while another reads its shared memory
}

// Fills L with the tensors of the list from `from` on; returns how many it took.
template <int N>
int64_t fill_list(const ll_tensor* t, int64_t count, int64_t from, int chunk, GradList<N>& L) {
    L.chunk = chunk;
    L.count = 0;
    L.chunks = 0;
    int64_t i = from;
    for (; i < count && L.count < N; ++i) {
        if (t[i].n == 0) continue;
        const int k = L.count++;
        L.data[k] = t[i].data;
        L.n[k] = t[i].n;
        L.dtype[k] = static_cast<uint8_t>(t[i].dtype);
        L.first[k] = L.chunks;
        const int es = t[i].dtype == LL_F32 ? 4 : 2;
        int64_t head = ((16 - (reinterpret_cast<uintptr_t>(t[i].data) & 15)) & 15) / es;
        if (head > t[i].n) head = t[i].n;
        const int64_t c = (t[i].n - head + chunk - 1) / chunk;
        L.chunks += c > 0 ? c : 1;
    }
    return i - from;
}

bool is_small(const ll_tensor* t, int64_t count) {
    if (count > kFewTensors) return false;
    int64_t bytes = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].n > kSmallBytes) return false;
        bytes += t[i].n * (t[i].dtype == LL_F32 ? 4 : 2);
    }
    return bytes <= kSmallBytes;
}

cudaError_t launch_small(const ll_tensor* t, int64_t count, float max_norm, float* norm,
                         cudaStream_t s) {
    GradList<kFewTensors> L;
    fill_list(t, count, 0, kSmallChunk, L);
    note_launches(1);
    grad_small_kernel<<<kSmallCtas, kThreads, 0, s>>>(L, max_norm, norm);
    return cudaGetLastError();
}

template <int N, typename F>
cudaError_t each_list(const ll_tensor* t, int64_t count, int num_sms, const F& launch) {
    GradList<N> L;
    for (int64_t i = 0; i < count;) {
        i += fill_list(t, count, i, kChunk, L);
        if (L.count == 0) break;
        int64_t grid = int64_t(num_sms) * kBlocksPerSm;
        if (grid > kGradMaxBlocks) grid = kGradMaxBlocks;
        if (grid > L.chunks) grid = L.chunks;
        note_launches(1);
        const cudaError_t e = launch(L, static_cast<unsigned>(grid));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int N>
cudaError_t norm_of(const ll_tensor* t, int64_t count, float* norm, double* part, int num_sms,
                    cudaStream_t s) {
    int64_t parts = 0;
    const cudaError_t e = each_list<N>(t, count, num_sms, [&](const GradList<N>& L, unsigned grid) {
        grad_squares_kernel<N><<<grid, kThreads, 0, s>>>(L, part + parts);
        parts += grid;
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    note_launches(1);
    return launch_after(grad_norm_kernel, 1, kThreads, s, static_cast<const double*>(part), parts,
                        norm);
}

template <int N>
cudaError_t clip_by(const ll_tensor* t, int64_t count, float max_norm, const float* norm,
                    int num_sms, cudaStream_t s) {
    return each_list<N>(t, count, num_sms, [&](const GradList<N>& L, unsigned grid) {
        return launch_after(grad_clip_kernel<N>, grid, kThreads, s, L, norm, max_norm);
    });
}

}  // namespace

cudaError_t launch_grad_norm(const ll_tensor* t, int64_t count, float* norm, void* ws,
                             int num_sms, cudaStream_t s) {
    if (is_small(t, count)) return launch_small(t, count, 0.f, norm, s);
    double* part = static_cast<double*>(ws);
    return count <= kFewTensors ? norm_of<kFewTensors>(t, count, norm, part, num_sms, s)
                                : norm_of<kMaxTensors>(t, count, norm, part, num_sms, s);
}

cudaError_t launch_grad_clip(const ll_tensor* t, int64_t count, float max_norm, bool compute,
                             float* norm, void* ws, int num_sms, cudaStream_t s) {
    if (compute && is_small(t, count)) return launch_small(t, count, max_norm, norm, s);
    if (compute) {
        const cudaError_t e = launch_grad_norm(t, count, norm, ws, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    return count <= kFewTensors ? clip_by<kFewTensors>(t, count, max_norm, norm, num_sms, s)
                                : clip_by<kMaxTensors>(t, count, max_norm, norm, num_sms, s);
}

}  // namespace ll
