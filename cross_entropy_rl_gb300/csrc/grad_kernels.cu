// Norm of all gradients as one vector, and clipping by it.
//
//   norm = sqrt(sum_i sum_j g_ij^2),  g *= min(1, max_norm / (norm + 1e-6))
//
// Both are bound by HBM: the norm reads every element once, the clipping reads
// and writes every element once.  The list is laid end to end in chunks, each
// block takes an equal run of them and streams it; the table of the tensors
// travels in the launch parameters, so a list costs one launch per kMaxTensors.
// The clipping goes through each run backwards: what the norm read last is still
// in L2.  A short list is one launch of one cluster that does both.
#include <math.h>

#include "step_device.cuh"

namespace ll {
namespace {

constexpr int kThreads = 512;
// Measured on 1.97 GB (norm) and 0.76 GB (norm + clipping), us: 2 blocks an SM of
// 8 loads 285 / 369, of 4 loads 289 / 370, 3 of 4 loads 351 / 387, 4 of 8 loads
// (spilled) 612 / 548.
constexpr int kBlocksPerSm = 2;
constexpr int kUnroll = 8;          // 16-byte loads of a thread in flight
constexpr int kChunk = 16384;       // bytes of a chunk: what the blocks' shares may differ by
constexpr int kSmallCtas = 8;       // CTAs of the one-launch path's cluster
// Most bytes of the one-launch path: 128 KB in 1 / 40 tensors take 4.2 / 7.0 us in
// one launch and 5.0 / 5.8 in three, 512 KB 4.3 / 8.6 and 6.0 / 6.1, 1 MB 4.8 / 13.3
// and 6.2 / 6.6; the two launches saved are 7 us of the host's time.
constexpr int64_t kSmallBytes = 512 << 10;

// The tensors of a launch, up to N of them.
template <int N>
struct GradList {
    const void* data[N];
    int64_t n[N];
    int64_t first[N];  // number of the tensor's first chunk
    int64_t chunks;
    int count;
    uint8_t dtype[N];
};
constexpr int kFewTensors = 64;  // a launch with a short table costs the host less

// Elements ahead of a tensor's first 16-byte boundary.
__host__ __device__ __forceinline__ int64_t head_of(const void* data, int64_t n, int es) {
    const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(data) & 15)) & 15) / es;
    return h < n ? h : n;
}

// The elements [lo, hi) of a tensor; from `body` on they start on a 16-byte
// boundary.
struct Range {
    int64_t lo, body, hi;
};

// Calls f(tensor, range) for the parts of the list's chunks [c0, c1) that lie in
// one tensor each.  A tensor's first chunk also takes what lies ahead of its
// first 16-byte boundary, so that the others start on one.
template <int N, typename F>
__device__ __forceinline__ void each_part(const GradList<N>& L, int64_t c0, int64_t c1,
                                          bool backwards, const F& f) {
    if (c0 >= c1) return;
    auto tensor_of = [&](int64_t chunk) {  // the last whose first chunk is <= chunk
        int a = 0, b = L.count;
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (L.first[m] <= chunk)
                a = m;
            else
                b = m;
        }
        return a;
    };
    int a = tensor_of(backwards ? c1 - 1 : c0);
    while (c0 < c1) {
        const int64_t t0 = L.first[a], t1 = a + 1 < L.count ? L.first[a + 1] : L.chunks;
        const int64_t p0 = c0 > t0 ? c0 : t0, p1 = c1 < t1 ? c1 : t1;
        const int es = L.dtype[a] == LL_F32 ? 4 : 2;
        const int64_t n = L.n[a], head = head_of(L.data[a], n, es), size = kChunk / es;
        Range r;
        r.body = head + (p0 - t0) * size;
        r.lo = p0 == t0 ? 0 : r.body;
        r.hi = head + (p1 - t0) * size < n ? head + (p1 - t0) * size : n;
        f(a, r);
        if (backwards)
            c1 = p0, --a;
        else
            c0 = p1, ++a;
    }
}

// A thread's sum of squares: FP32 sums of at most 32 elements, added as a pair
// while their largest lies in [2^-50, 2^38], where the squares lose nothing that
// matters and no sum of a block leaves the FP32 range: the 2^57 elements that a
// launch accepts are 2^49 a block, of 2^76 each.  Others are squared in 64 bits.
struct Squares {
    Pair sum = {0.f, 0.f};
    double wide = 0;
    bool used_wide = false;

    template <int K>
    __device__ __forceinline__ void add_all(const float (&x)[K]) {
        float s = 0.f, big = 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            s = fmaf(x[i], x[i], s);
            big = fmaxf(big, fabsf(x[i]));  // a NaN is in s
        }
        if (big == 0.f || (big >= 0x1p-50f && big <= 0x1p38f)) {
            sum = add(sum, Pair{s, 0.f});
        } else {
            used_wide = true;
            for (int i = 0; i < K; ++i) wide += static_cast<double>(x[i]) * x[i];
        }
    }
};

template <typename T>
__device__ __forceinline__ void add_squares(const T* __restrict__ p, const Range& r, Squares& q) {
    constexpr int E = 16 / sizeof(T);
    const T* body = p + r.body;
    const int64_t vecs = (r.hi - r.body) / E;
    int64_t i = threadIdx.x;
    for (; i + (kUnroll - 1) * kThreads < vecs; i += kUnroll * kThreads) {
        Pack<T, E> x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u].load(body + (i + u * kThreads) * E);
#pragma unroll
        for (int u = 0; u < kUnroll; u += 32 / E) {
            float f[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = Elem<T>::to_f(x[u + j / E].e[j % E]);
            q.add_all(f);
        }
    }
    for (; i < vecs; i += kThreads) {
        Pack<T, E> x;
        x.load(body + i * E);
        float f[E];
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = Elem<T>::to_f(x.e[j]);
        q.add_all(f);
    }
    const int64_t head = r.lo + threadIdx.x, tail = r.body + vecs * E + threadIdx.x;
    float f[2] = {0.f, 0.f};
    if (head < r.body) f[0] = Elem<T>::to_f(p[head]);
    if (tail < r.hi) f[1] = Elem<T>::to_f(p[tail]);
    q.add_all(f);
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

// Chunks of block `b` of `blocks`.
template <int N>
__device__ __forceinline__ int64_t share(const GradList<N>& L, int64_t b, int64_t blocks) {
    return L.chunks / blocks * b + (L.chunks % blocks < b ? L.chunks % blocks : b);
}

template <int N>
__device__ __forceinline__ void list_squares(const GradList<N>& L, int64_t b, int64_t blocks,
                                             Squares& q) {
    each_part(L, share(L, b, blocks), share(L, b + 1, blocks), false, [&](int a, const Range& r) {
        const void* p = L.data[a];
        switch (L.dtype[a]) {
            case LL_F32: add_squares(static_cast<const float*>(p), r, q); break;
            case LL_F16: add_squares(static_cast<const __half*>(p), r, q); break;
            default: add_squares(static_cast<const __nv_bfloat16*>(p), r, q);
        }
    });
}

template <typename T>
__device__ __forceinline__ void scale_range(T* __restrict__ p, const Range& r, float coef) {
    constexpr int E = 16 / sizeof(T);
    T* body = p + r.body;
    const int64_t vecs = (r.hi - r.body) / E;
    auto one = [&](T x) { return Elem<T>::from_f(Elem<T>::to_f(x) * coef); };
    const int64_t head = r.lo + threadIdx.x, tail = r.body + vecs * E + threadIdx.x;
    if (tail < r.hi) p[tail] = one(p[tail]);
    // whole rounds from the end of the range back
    constexpr int64_t kRound = kUnroll * kThreads;
    const int64_t rest = vecs % kRound;
    for (int64_t i = vecs - kRound; i >= rest; i -= kRound) {
        Pack<T, E> x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u].load(body + (i + u * kThreads + threadIdx.x) * E);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
#pragma unroll
            for (int j = 0; j < E; ++j) x[u].e[j] = one(x[u].e[j]);
            x[u].store(body + (i + u * kThreads + threadIdx.x) * E);
        }
    }
    for (int64_t i = threadIdx.x; i < rest; i += kThreads) {
        Pack<T, E> x;
        x.load(body + i * E);
#pragma unroll
        for (int j = 0; j < E; ++j) x.e[j] = one(x.e[j]);
        x.store(body + i * E);
    }
    if (head < r.body) p[head] = one(p[head]);
}

// Block b's chunks scaled for the norm, from the last back.
template <int N>
__device__ __forceinline__ void list_scale(const GradList<N>& L, int64_t b, int64_t blocks,
                                           float norm, float max_norm) {
    const float c = max_norm / (norm + 1e-6f);
    if (c >= 1.f) return;  // a NaN goes on: it belongs in the gradients too
    each_part(L, share(L, b, blocks), share(L, b + 1, blocks), true, [&](int a, const Range& r) {
        void* p = const_cast<void*>(L.data[a]);
        switch (L.dtype[a]) {
            case LL_F32: scale_range(static_cast<float*>(p), r, c); break;
            case LL_F16: scale_range(static_cast<__half*>(p), r, c); break;
            default: scale_range(static_cast<__nv_bfloat16*>(p), r, c);
        }
    });
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

// The root of the sum of the blocks' sums: in pairs, as a block's are, while they
// lie in [2^-90, 2^90], of which FP32 holds almost 2^38 (2^28 launches').
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* __restrict__ part,
                                                             int64_t parts,
                                                             float* __restrict__ norm) {
    wait_for_prerequisites();
    launch_dependents();
    Squares q;
    for (int64_t i = threadIdx.x; i < parts; i += kThreads) {
        const double s = part[i];
        if (s == 0.0 || (s >= 0x1p-90 && s <= 0x1p90)) {
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
    list_scale(L, blockIdx.x, gridDim.x, __ldcg(norm), max_norm);
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
        list_scale(L, blockIdx.x, kSmallCtas, total, max_norm);
    __syncthreads();  // the cluster's barrier takes whole warps
    cluster_barrier();  // no CTA leaves while another reads its shared memory
}

// Fills L with the tensors of the list from `from` on; returns how many it took.
template <int N>
int64_t fill_list(const ll_tensor* t, int64_t count, int64_t from, GradList<N>& L) {
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
        const int64_t size = kChunk / es, head = head_of(t[i].data, t[i].n, es);
        const int64_t c = (t[i].n - head + size - 1) / size;
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
    fill_list(t, count, 0, L);
    note_launches(1);
    grad_small_kernel<<<kSmallCtas, kThreads, 0, s>>>(L, max_norm, norm);
    return cudaGetLastError();
}

template <int N, typename F>
cudaError_t each_list(const ll_tensor* t, int64_t count, int num_sms, const F& launch) {
    GradList<N> L;
    for (int64_t i = 0; i < count;) {
        i += fill_list(t, count, i, L);
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
    return launch_after(grad_norm_kernel, 1, kThreads, s, 0, static_cast<const double*>(part), parts,
                        norm);
}

template <int N>
cudaError_t clip_by(const ll_tensor* t, int64_t count, float max_norm, const float* norm,
                    int num_sms, cudaStream_t s) {
    return each_list<N>(t, count, num_sms, [&](const GradList<N>& L, unsigned grid) {
        return launch_after(grad_clip_kernel<N>, grid, kThreads, s, 0, L, norm, max_norm);
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
    const bool clip = max_norm < INFINITY;
    if (compute && clip && is_small(t, count)) return launch_small(t, count, max_norm, norm, s);
    if (compute) {
        const cudaError_t e = launch_grad_norm(t, count, norm, ws, num_sms, s);
        if (e != cudaSuccess) return e;
    }
    if (!clip) return cudaSuccess;
    return count <= kFewTensors ? clip_by<kFewTensors>(t, count, max_norm, norm, num_sms, s)
                                : clip_by<kMaxTensors>(t, count, max_norm, norm, num_sms, s);
}

}  // namespace ll
