// Norm of all gradients as one vector, and clipping by it.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  g *= min(1, max_norm / (norm + 1e-6))
//
// Both are bound by HBM: the norm reads every element once, the clipping reads
// and writes every element once.  A list is cut into chunks of a fixed number
// of elements; blocks take chunks in turn and a table of the tensors travels
// in the launch parameters, so a list costs one launch per kMaxTensors.
#include <math.h>

#include "ll_device.cuh"

namespace ll {
namespace {

constexpr int kThreads = 256;

// The elements [lo, hi) of one tensor that chunk `c` of its tensor covers: the
// first chunk also takes the elements ahead of the first 16-byte boundary, so
// that every other chunk starts on one.
struct Range {
    int tensor;
    int64_t lo, body, hi;  // [lo, body) lie ahead of the boundary
};

__device__ __forceinline__ Range chunk_range(const GradList& L, int64_t chunk) {
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

// Sum of squares of one thread's elements of a chunk.  In FP32 while the
// largest element lies in [2^-50, 2^55], where neither the squares nor their
// sum of at most a few hundred leave the FP32 range nor lose what matters;
// else, a second time, in 64 bits.
template <typename T>
__device__ double thread_squares(const T* __restrict__ p, const Range& r) {
    constexpr int E = 16 / sizeof(T);
    const int64_t vecs = (r.hi - r.body) / E;
    float s = 0.f, big = 0.f;
    auto add = [&](float x) {
        s = fmaf(x, x, s);
        big = fmaxf(big, fabsf(x));
    };
    if (r.lo + threadIdx.x < r.body) add(Elem<T>::to_f(p[r.lo + threadIdx.x]));
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vecs; i += kThreads) {
        Pack<T, E> x;
        x.load(p + r.body + i * E);
#pragma unroll
        for (int j = 0; j < E; ++j) add(Elem<T>::to_f(x.e[j]));
    }
    const int64_t tail = r.body + vecs * E + threadIdx.x;
    if (tail < r.hi) add(Elem<T>::to_f(p[tail]));
    if (big == 0.f || (big >= 0x1p-50f && big <= 0x1p55f)) return s;
    double d = 0;
    auto add64 = [&](T x) {
        const double f = Elem<T>::to_f(x);
        d += f * f;
    };
    if (r.lo + threadIdx.x < r.body) add64(p[r.lo + threadIdx.x]);
    for (int64_t i = threadIdx.x; i < vecs; i += kThreads)
        for (int j = 0; j < E; ++j) add64(p[r.body + i * E + j]);
    if (tail < r.hi) add64(p[tail]);
    return d;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Sum over the block of x (every thread gets it).
__device__ double block_sum(double x) {
    __shared__ double part[kThreads / 32];
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0;
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ GradList L,
                                                                double* __restrict__ part) {
    double s = 0;
    for (int64_t c = blockIdx.x; c < L.chunks; c += gridDim.x) {
        const Range r = chunk_range(L, c);
        const void* p = L.data[r.tensor];
        switch (L.dtype[r.tensor]) {
            case LL_F32: s += thread_squares(static_cast<const float*>(p), r); break;
            case LL_F16: s += thread_squares(static_cast<const __half*>(p), r); break;
            default: s += thread_squares(static_cast<const __nv_bfloat16*>(p), r);
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* __restrict__ part,
                                                             int64_t parts,
                                                             float* __restrict__ norm) {
    double s = 0;
    for (int64_t i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    s = block_sum(s);
    if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(s));
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

__global__ void __launch_bounds__(kThreads) grad_clip_kernel(const __grid_constant__ GradList L,
                                                             const float* __restrict__ norm,
                                                             float max_norm) {
    const float c = max_norm / (norm[0] + 1e-6f);
    if (c >= 1.f) return;  // a NaN goes on: it belongs in the gradients too
    for (int64_t i = blockIdx.x; i < L.chunks; i += gridDim.x) {
        const Range r = chunk_range(L, i);
        void* p = const_cast<void*>(L.data[r.tensor]);
        switch (L.dtype[r.tensor]) {
            case LL_F32: scale_range(static_cast<float*>(p), r, c); break;
            case LL_F16: scale_range(static_cast<__half*>(p), r, c); break;
            default: scale_range(static_cast<__nv_bfloat16*>(p), r, c);
        }
    }
}

// Fills L with the tensors [from, ...) of the list and returns how many it took.
int64_t fill_list(const ll_tensor* t, int64_t count, int64_t from, GradList& L) {
    L.chunk = kGradChunk;
    L.count = 0;
    L.chunks = 0;
    int64_t i = from;
    for (; i < count && L.count < kMaxTensors; ++i) {
        if (t[i].n == 0) continue;
        const int k = L.count++;
        L.data[k] = t[i].data;
        L.n[k] = t[i].n;
        L.dtype[k] = static_cast<uint8_t>(t[i].dtype);
        L.first[k] = L.chunks;
        const int es = t[i].dtype == LL_F32 ? 4 : 2;
        int64_t head = ((16 - (reinterpret_cast<uintptr_t>(t[i].data) & 15)) & 15) / es;
        if (head > t[i].n) head = t[i].n;
        const int64_t c = (t[i].n - head + L.chunk - 1) / L.chunk;
        L.chunks += c > 0 ? c : 1;
    }
    return i - from;
}

unsigned list_grid(const GradList& L, int num_sms) {
    int64_t most = int64_t(num_sms) * kGradBlocksPerSm;
    if (most > kGradMaxBlocks) most = kGradMaxBlocks;
    return static_cast<unsigned>(L.chunks < most ? L.chunks : most);
}

}  // namespace

cudaError_t launch_grad_norm(const ll_tensor* t, int64_t count, float* norm, void* ws,
                             int num_sms, cudaStream_t s) {
    double* part = static_cast<double*>(ws);
    int64_t parts = 0;
    GradList L;
    for (int64_t i = 0; i < count;) {
        i += fill_list(t, count, i, L);
        if (L.count == 0) break;
        const unsigned grid = list_grid(L, num_sms);
        note_launches(1);
        grad_squares_kernel<<<grid, kThreads, 0, s>>>(L, part + parts);
        parts += grid;
    }
    note_launches(1);
    grad_norm_kernel<<<1, kThreads, 0, s>>>(part, parts, norm);
    return cudaGetLastError();
}

cudaError_t launch_grad_clip(const ll_tensor* t, int64_t count, float max_norm, const float* norm,
                             int num_sms, cudaStream_t s) {
    GradList L;
    for (int64_t i = 0; i < count;) {
        i += fill_list(t, count, i, L);
        if (L.count == 0) break;
        note_launches(1);
        grad_clip_kernel<<<list_grid(L, num_sms), kThreads, 0, s>>>(L, norm, max_norm);
    }
    return cudaGetLastError();
}

}  // namespace ll
