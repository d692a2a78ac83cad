// Device helpers of the kernels around the linear log-probability in a training
// step.  They have their own files: the traffic figures that bench.py reports
// hold for the sources that the measured kernels are built from.
#pragma once
#include "ll_device.cuh"
#include "step_internal.h"

namespace ll {

// A sum held as hi + lo, |lo| at most half a step of hi: about 48 bits from
// FP32 additions, whose rounding errors are taken as in Knuth's two-sum.  With FP64
// sums and weights the policy loss of a million tokens kept the FP64 unit 77% busy
// and took 33 us instead of 19 (14 since).  The _rn forms keep the compiler from
// fusing.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ float finite_or_0(float e, float of) {
    return fabsf(of) < INFINITY ? e : 0.f;
}

__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const float s = __fadd_rn(a.hi, b.hi);
    const float t = __fsub_rn(s, a.hi);
    float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    e = finite_or_0(__fadd_rn(e, __fadd_rn(a.lo, b.lo)), s);
    const float hi = __fadd_rn(s, e);
    return {hi, finite_or_0(__fsub_rn(e, __fsub_rn(hi, s)), hi)};
}

__device__ __forceinline__ Pair pair_of(double x) {
    const float hi = static_cast<float>(x);
    return {hi, static_cast<float>(x - hi)};
}

__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = add(x, Pair{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
    return x;
}

// ------------------------------------- overlapped launches on one stream
// In a kernel started by launch_after(): blocks until the kernel ahead of it on
// the stream is done and its writes are visible.
__device__ __forceinline__ void wait_for_prerequisites() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// In the kernel ahead: the next one's blocks may be started.
__device__ __forceinline__ void launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;");
}

// Launches a kernel whose blocks may start before the kernel ahead of it on
// the stream is done (it calls wait_for_prerequisites()).
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads,
                                cudaStream_t s, unsigned smem, const A&... args) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// E consecutive elements of T, moved in vectors of up to 16 bytes when they
// fill them (the pointer is then aligned to 16 bytes, or to the whole pack if
// that is smaller), else one by one.
template <typename T, int E>
struct Pack {
    static constexpr int kBytes = E * int(sizeof(T));
    alignas(kBytes % 16 == 0 ? 16 : kBytes) T e[E];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) e[i] = p[i];
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(e)[i];
        } else if constexpr (kBytes == 8) {
            *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) p[i] = e[i];
        }
    }
};

}  // namespace ll
