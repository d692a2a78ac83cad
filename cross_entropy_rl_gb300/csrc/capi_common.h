// What the entry points of the C ABI share: sizes, the device guard, tracing.
#pragma once
#include "ll_internal.h"

namespace ll {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
inline size_t esize(int dtype) { return dtype == LL_F32 ? 4 : 2; }
inline bool dtype_ok(int dt) { return dt == LL_F32 || dt == LL_F16 || dt == LL_BF16; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Brackets a phase of a call by CUDA events on its stream while tracing is on.
struct Phase {
    const char* label;
    cudaStream_t s;
    cudaEvent_t a = nullptr, b = nullptr;
    Phase(const char* l, cudaStream_t st);
    ~Phase();
};

// Switches to the device owning `ptr` for the lifetime of the guard.
struct DeviceGuard {
    int prev = -1;
    int dev = -1;
    int err = LL_OK;
    explicit DeviceGuard(const void* ptr) {
        cudaPointerAttributes attr;
        if (cudaPointerGetAttributes(&attr, ptr) != cudaSuccess) {
            cudaGetLastError();
            err = LL_ERR_INVALID_ARG;
            return;
        }
        if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) {
            err = LL_ERR_INVALID_ARG;
            return;
        }
        dev = attr.device;
        if (dev < 0 || dev >= 64) {
            err = LL_ERR_INVALID_ARG;
            return;
        }
        if (cudaGetDevice(&prev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) {
            err = LL_ERR_CUDA;
            return;
        }
    }
    ~DeviceGuard() {
        if (prev >= 0 && prev != dev) cudaSetDevice(prev);
    }
};

int device_info(int dev, DevInfo* out);  // LL_OK, or an LL_ERR status
int cuda_status(cudaError_t e);          // LL_OK, or LL_ERR_CUDA with a message
int check_sizes(int64_t N, int64_t D, int64_t V);

}  // namespace ll
