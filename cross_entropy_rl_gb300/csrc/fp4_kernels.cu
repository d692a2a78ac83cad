// Quantisation to microscaled 4-bit floating point, and back.
//
// A lane holds 8 consecutive columns of a row, a warp 256: the largest magnitude of a
// block is a maximum over 4 lanes (LL_FP4_MX, 32 columns) or 2 (LL_FP4_NV, 16), its codes
// are one 32-bit store a lane, and the scales of four blocks one 32-bit store.
//
// 151936 x 4096 BF16 in LL_FP4_NV 559 us (the largest magnitude ahead of it 205 us, 6.1 TB/s), in
// LL_FP4_MX 563, where the bytes would take 235; back 325-331.  The variant of 16 rows a warp, which
// these sizes take, keeps part of its four rows in local memory (208-240 bytes a thread, at 48
// registers for 5 blocks an SM): 40960 x 2048 under a profiler 90 us at 60% of issue slots, 0.73 GB
// of local loads and stores beside 0.25 GB of DRAM's.  The one of 1 row does not (32768 x 2048: 75
// us, 73%).  Back, 48 us for 40960 x 2048 at 65%.  Small ones are a launch (48 x 4096: 2.3 us).
#include "fp4_device.cuh"

namespace ll {
namespace {

constexpr int kWarps = 8;
constexpr int kWarpCols = 256;

// A lane's 8 values of a row as loaded.
template <typename T>
struct Raw8 {
    static constexpr int kWords = 2 * sizeof(T);
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T* p) {  // 16-byte aligned
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    }
    // The largest magnitude as the bits of an FP32 value: NaN above infinity above numbers.
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (sizeof(T) == 4) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
            return m;
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            const uint32_t one = max(m & 0xffffu, m >> 16);
            if constexpr (std::is_same<T, __half>::value)
                return __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(one))));
            else
                return one << 16;
        }
    }
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else if constexpr (std::is_same<T, __half>::value)
            return __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        else
            return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};

// A warp's 256 columns of a row to 8 consecutive ones a lane, through its part of shared
// memory: for rows off the 16-byte boundaries, and their ends.
template <typename T>
__device__ __forceinline__ Raw8<T> load_any(const T* row, int64_t col0, int64_t K, T* stage) {
    const int lane = threadIdx.x & 31;
    T e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t c = col0 + lane + 32 * j;
        e[j] = c < K ? row[c] : Elem<T>::from_f(0.f);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) stage[lane + 32 * j] = e[j];
    __syncwarp();
    Raw8<T> r;
    memcpy(r.w, stage + lane * 8, sizeof(r.w));
    return r;
}

__device__ __forceinline__ float rcp(float x) {  // to 2^-23
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The border between two neighbouring codes, in units of the multiplier: code i to i + 1.
__device__ __forceinline__ double e2m1_border(int i) {
    constexpr double at[7] = {0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0};
    return at[i];
}

// Between two neighbouring codes (of a lane's 8, in `lo` and `hi`) the exact quotient decides:
// border * s has 7 bits, and one fused operation has the sign of |x| - border * s * g.
template <typename T>
__device__ __noinline__ uint32_t settle_codes(const Raw8<T> x, uint32_t lo, uint32_t hi, float s,
                                              float g) {
    uint32_t word = lo;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = (lo >> (4 * j)) & 7u;
        if (c == ((hi >> (4 * j)) & 7u)) continue;
        const float border = c < 4 ? 0.25f + 0.5f * c : c == 4 ? 2.5f : c == 5 ? 3.5f : 5.f;
        const float2 p = x.pair(j / 2);
        const float d = fmaf(-(border * s), g, fabsf(j & 1 ? p.y : p.x));
        if (d > 0.f || (d == 0.f && (c & 1))) word += 1u << (4 * j);  // a tie goes to the even one
    }
    return word;
}
// The same for two neighbouring E4M3 bytes of amax / (6 g).
__device__ __forceinline__ uint32_t settle_scale(float amax, uint32_t two, float g) {
    const uint32_t low = two & 0xffu;
    const float border = 0.5f * (e4m3_value(low) + e4m3_value(two >> 8));  // 5 bits
    const float d = fmaf(-(6.f * border), g, amax);
    return d > 0.f || (d == 0.f && (low & 1)) ? two >> 8 : low;
}

// The code of x for the multiplier s * g far from 1, decided on exact products in FP64.
__device__ __noinline__ uint32_t e2m1_exact(float x, float s, float g) {
    const double m = static_cast<double>(s) * g, a = fabs(static_cast<double>(x));
    uint32_t c = 0;
    for (int i = 0; i < 7; ++i) {
        const double b = e2m1_border(i) * m;
        c += a > b || (a == b && (i & 1));  // a tie goes to the even one of i and i + 1
    }
    return c | (signbit(x) ? 8u : 0u);
}

// E4M3 byte of amax / (6 g), the same way.
__device__ __noinline__ uint32_t e4m3_exact(float amax, float g) {
    const double six_g = 6.0 * g, t = static_cast<double>(amax) / six_g;
    if (!(t < 448.0)) return 0x7eu;
    int e = t > 0.0 ? ilogb(t) : -6;
    if (e < -6) e = -6;
    double n = floor(ldexp(t, 3 - e));
    const double border = ldexp(n + 0.5, e - 3) * six_g;
    const bool odd = fmod(n, 2.0) != 0.0;
    if (amax > border || (amax == border && odd)) n += 1.0;
    return static_cast<uint32_t>((e + 6) * 8) + static_cast<uint32_t>(n);  // n carries into e
}

// The codes of a lane's 8 values and the byte of its block's scale.
template <typename T, int FORMAT>
__device__ __forceinline__ uint32_t quantize8(const Raw8<T>& x, float g, float inv6g, float inv_g,
                                              bool far, uint32_t& byte) {
    constexpr int kLanes = FORMAT == LL_FP4_MX ? 4 : 2;  // of a block
    // factors next to 1 that enclose the rounding errors of the approximate quotients
    // (below 2^-21): where both give one code, so does the exact quotient
    constexpr float kBelow = 1.f - 0x1p-20f, kAbove = 1.f + 0x1p-20f;
    uint32_t top = x.top();
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool bad = top >= 0x7f800000u;
    uint32_t word;
    if (FORMAT == LL_FP4_MX) {
        byte = max(static_cast<int>(top >> 23) - 2, 0);
        const float inv = __uint_as_float((254u - byte) << 23);  // a power of two
        float q[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = x.pair(i);
            q[2 * i] = p.x * inv;
            q[2 * i + 1] = p.y * inv;
        }
        word = e2m1x8(q);
        if (bad) byte = kScaleNanMx;
    } else {
        const float amax = __uint_as_float(top);
        const float t = amax * inv6g;
        const uint32_t two = e4m3x2(t * kBelow, t * kAbove);
        byte = two & 0xffu;
        if (far && !bad)
            byte = e4m3_exact(amax, g);
        else if (byte != two >> 8)
            byte = settle_scale(amax, two, g);
        const float s = e4m3_value(byte);
        const float inv = rcp(s) * inv_g, below = inv * kBelow, above = inv * kAbove;
        float lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = x.pair(i);
            lo[2 * i] = p.x * below;
            lo[2 * i + 1] = p.y * below;
            hi[2 * i] = p.x * above;
            hi[2 * i + 1] = p.y * above;
        }
        word = e2m1x8(lo);
        const uint32_t upper = e2m1x8(hi);
        if (byte == 0) {
            word = 0;
        } else if (far && !bad) {
            word = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 p = x.pair(i);
                word |= e2m1_exact(p.x, s, g) << (8 * i) | e2m1_exact(p.y, s, g) << (8 * i + 4);
            }
        } else if (word != upper) {
            word = settle_codes(x, word, upper, s, g);
        }
        if (bad) byte = kScaleNanNv;
    }
    return bad ? 0u : word;
}

// Rows R, columns K of x to codes and scales.  RPW: rows of a warp, four loads in flight.
template <typename T, int FORMAT, int RPW>
__global__ void __launch_bounds__(kWarps * 32, sizeof(T) == 2 ? 5 : 4)
    quantize_kernel(const T* __restrict__ x, int64_t ldx, int64_t R, int64_t K, int vec,
                    const float* __restrict__ scale, uint8_t* __restrict__ codes,
                    uint8_t* __restrict__ scales, int64_t k_tiles, int64_t col_tiles,
                    int64_t tiles) {
    constexpr int kLanes = FORMAT == LL_FP4_MX ? 4 : 2;  // of a block
    constexpr int kUnroll = RPW < 4 ? RPW : 4;
    __shared__ __align__(16) T stage[kWarps][kWarpCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row_bytes = fp4_row_bytes(K);
    float g = 1.f, inv6g = 0.f, inv_g = 0.f;
    bool far = false;
    if (FORMAT == LL_FP4_NV) {
        g = *scale;
        inv6g = 1.f / (6.f * g);
        inv_g = 1.f / g;
        far = !(g > 0x1p-100f && g < 0x1p100f);  // the approximations may leave FP32's range
    }
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t rt = tile / col_tiles, col0 = (tile - rt * col_tiles) * kWarpCols;
        const int64_t col = col0 + lane * 8, row0 = (rt * kWarps + warp) * RPW;
        const bool whole = vec && col0 + kWarpCols <= K;
        const int64_t b = col / (8 * kLanes);
#pragma unroll 1
        for (int i0 = 0; i0 < RPW; i0 += kUnroll) {
            Raw8<T> raw[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t r = row0 + i0 + i;
                if (r >= R)
                    raw[i].zero();
                else if (whole)
                    raw[i].load(x + r * ldx + col);
                else
                    raw[i] = load_any(x + r * ldx, col0, K, stage[warp]);
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t r = row0 + i0 + i;
                uint32_t byte;
                const uint32_t word = quantize8<T, FORMAT>(raw[i], g, inv6g, inv_g, far, byte);
                if (r < R && col < 2 * row_bytes)
                    *reinterpret_cast<uint32_t*>(codes + r * row_bytes + col / 2) = word;
                // the scales of four blocks to one word
                uint32_t four = byte << (8 * ((lane / kLanes) & 3));
#pragma unroll
                for (int o = kLanes; o < 4 * kLanes; o *= 2)
                    four |= __shfl_xor_sync(0xffffffffu, four, o);
                if (lane % (4 * kLanes) == 0 && b < kFp4TileBlocks * k_tiles &&
                    r < (R + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows)
                    *reinterpret_cast<uint32_t*>(scales + scale_at(r, b, k_tiles)) = four;
            }
        }
    }
}

// Largest finite magnitude of x, as the bits of an FP32 value, into *top (0 before).
template <typename T>
__device__ __forceinline__ uint32_t finite_top(const Raw8<T>& x) {
    uint32_t m = x.top();
    if (m >= 0x7f800000u) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = x.pair(i);
            const uint32_t a = __float_as_uint(p.x) & 0x7fffffffu, b = __float_as_uint(p.y) & 0x7fffffffu;
            m = max(m, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
        }
    }
    return m;
}
__device__ __forceinline__ void block_top(uint32_t m, uint32_t* top) {
    __shared__ uint32_t part[kWarps];
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) m = max(m, part[w]);
        atomicMax(top, m);
    }
}
// ... of n values side by side, from a 16-byte boundary on
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    amax_flat_kernel(const T* __restrict__ x, int64_t n, uint32_t* __restrict__ top) {
    constexpr int kUnroll = 4;
    const int64_t packs = n / 8, step = gridDim.x * (kWarps * 32ll);
    uint32_t m = 0;
    for (int64_t p = blockIdx.x * (kWarps * 32ll) + threadIdx.x; p < packs; p += kUnroll * step) {
        Raw8<T> raw[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            if (p + i * step < packs)
                raw[i].load(x + (p + i * step) * 8);
            else
                raw[i].zero();
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) m = max(m, finite_top(raw[i]));
    }
    if (blockIdx.x == 0)
        for (int64_t i = packs * 8 + threadIdx.x; i < n; i += kWarps * 32) {
            const uint32_t b = __float_as_uint(Elem<T>::to_f(x[i])) & 0x7fffffffu;
            m = max(m, b < 0x7f800000u ? b : 0u);
        }
    block_top(m, top);
}
// ... of rows
template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
    amax_rows_kernel(const T* __restrict__ x, int64_t ldx, int64_t R, int64_t K,
                     uint32_t* __restrict__ top) {
    uint32_t m = 0;
    const int lane = threadIdx.x & 31;
    for (int64_t r = blockIdx.x * int64_t(kWarps) + (threadIdx.x >> 5); r < R; r += gridDim.x * int64_t(kWarps))
#pragma unroll 8
        for (int64_t c = lane; c < K; c += 32) {
            const uint32_t b = __float_as_uint(Elem<T>::to_f(x[r * ldx + c])) & 0x7fffffffu;
            m = max(m, b < 0x7f800000u ? b : 0u);
        }
    block_top(m, top);
}
__global__ void scale_kernel(float* scale) {
    const float top = *scale;
    const float g = static_cast<float>(top / 2688.0);
    *scale = g > 0.f ? g : 1.f;
}

// A launch over tiles of kWarps * RPW rows (of the rows given) x 256 columns.
struct Tiles {
    int64_t cols, all;
    unsigned grid;
};
Tiles tiles_of(int64_t rows, int64_t cols, int rpw, int num_sms) {
    Tiles t;
    t.cols = (cols + kWarpCols - 1) / kWarpCols;
    t.all = t.cols * ((rows + kWarps * rpw - 1) / (kWarps * rpw));
    const int64_t cap = int64_t(num_sms) * 32;
    t.grid = unsigned(t.all < cap ? t.all : cap);
    return t;
}

template <typename T, int FORMAT, int RPW>
cudaError_t run_quantize(const T* x, int64_t ldx, const Fp4Matrix& q, int vec, int num_sms,
                         cudaStream_t s) {
    const int64_t kt = fp4_k_tiles(q.cols, FORMAT);
    const int64_t rows = (q.rows + kFp4TileRows - 1) / kFp4TileRows * kFp4TileRows;
    const Tiles t = tiles_of(rows, kt * kFp4TileBlocks * fp4_block(FORMAT), RPW, num_sms);
    note_launches(1);
    quantize_kernel<T, FORMAT, RPW><<<t.grid, kWarps * 32, 0, s>>>(
        x, ldx, q.rows, q.cols, vec, q.scale, const_cast<uint8_t*>(q.codes),
        const_cast<uint8_t*>(q.scales), kt, t.cols, t.all);
    return cudaGetLastError();
}

// Rows of a warp: 16 where that gives each SM 16 blocks at least, else 1.  LL_FP4_NV and back, us
// with 16 and with 1: 4096 x 4096 22.6 and 20.1, 22.0 and 16.2; 32768 x 2048 72.9 and 74.1, 61.3
// and 59.3; 151936 x 4096 558 and 636, 459 and 506.
bool many_rows(const Fp4Matrix& q, int num_sms) {
    return (q.rows + 127) / 128 * ((q.cols + kWarpCols - 1) / kWarpCols) >= 16 * num_sms;
}

template <typename T>
cudaError_t quantize(const T* x, int64_t ldx, const Fp4Matrix& q, float* scale, bool given,
                     int num_sms, cudaStream_t s) {
    const int vec = (reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ldx * sizeof(T)) % 16 == 0) ? 1 : 0;
    if (q.format == LL_FP4_NV && !given) {
        cudaError_t e = cudaMemsetAsync(scale, 0, sizeof(float), s);
        if (e != cudaSuccess) return e;
        const int64_t n = q.rows * q.cols, want = (n + 8191) / 8192, cap = int64_t(num_sms) * 8;
        const unsigned grid = unsigned(want < cap ? want : cap);
        uint32_t* top = reinterpret_cast<uint32_t*>(scale);
        note_launches(2);
        if ((ldx == q.cols || q.rows == 1) && reinterpret_cast<uintptr_t>(x) % 16 == 0)
            amax_flat_kernel<T><<<grid, kWarps * 32, 0, s>>>(x, n, top);
        else
            amax_rows_kernel<T><<<grid, kWarps * 32, 0, s>>>(x, ldx, q.rows, q.cols, top);
        scale_kernel<<<1, 1, 0, s>>>(scale);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const bool many = many_rows(q, num_sms);
    if (q.format == LL_FP4_MX)
        return many ? run_quantize<T, LL_FP4_MX, 16>(x, ldx, q, vec, num_sms, s)
                    : run_quantize<T, LL_FP4_MX, 1>(x, ldx, q, vec, num_sms, s);
    return many ? run_quantize<T, LL_FP4_NV, 16>(x, ldx, q, vec, num_sms, s)
                : run_quantize<T, LL_FP4_NV, 1>(x, ldx, q, vec, num_sms, s);
}

// The reverse: a lane has 8 columns of a row, a warp 256.
template <typename T, int FORMAT, int RPW>
__global__ void __launch_bounds__(kWarps * 32)
    dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const float* __restrict__ scale, int64_t R, int64_t K, int64_t k_tiles,
                      T* __restrict__ out, int64_t ldo, int vec, int64_t col_tiles, int64_t tiles) {
    constexpr int kUnroll = RPW < 4 ? RPW : 4;
    __shared__ __align__(16) T stage[kWarps][kWarpCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row_bytes = fp4_row_bytes(K);
    const float g = FORMAT == LL_FP4_NV ? *scale : 1.f;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t rt = tile / col_tiles, col0 = (tile - rt * col_tiles) * kWarpCols;
        const int64_t col = col0 + lane * 8, row0 = (rt * kWarps + warp) * RPW;
        const bool whole = vec && col0 + kWarpCols <= K;
        const int64_t b = col / fp4_block(FORMAT);
#pragma unroll 1
        for (int i0 = 0; i0 < RPW; i0 += kUnroll) {
            uint32_t word[kUnroll], byte[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t r = row0 + i0 + i;
                const bool some = r < R && col < K;
                word[i] = some ? __ldg(reinterpret_cast<const uint32_t*>(codes + r * row_bytes + col / 2)) : 0u;
                byte[i] = some ? __ldg(scales + scale_at(r, b, k_tiles)) : 0u;
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int64_t r = row0 + i0 + i;
                if (r >= R) break;
                float v[8];
                e2m1_values(word[i], v);
                if (FORMAT == LL_FP4_MX) {
                    const float s = e8m0_value(byte[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] *= s;
                } else {
                    const float s = e4m3_value(byte[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = (v[j] * s) * g;  // the first product is exact
                }
                if (whole) {
                    store8(out + r * ldo + col, v);
                } else {  // 32 neighbours at once
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) stage[warp][lane * 8 + j] = Elem<T>::from_f(v[j]);
                    __syncwarp();
                    T* o = out + r * ldo + col0;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col0 + lane + 32 * j < K) o[lane + 32 * j] = stage[warp][lane + 32 * j];
                }
            }
        }
    }
}

template <typename T, int FORMAT, int RPW>
cudaError_t run_dequantize(const Fp4Matrix& q, T* out, int64_t ldo, int num_sms, cudaStream_t s) {
    const int vec =
        (reinterpret_cast<uintptr_t>(out) % 16 == 0 && (ldo * sizeof(T)) % 16 == 0) ? 1 : 0;
    const Tiles t = tiles_of(q.rows, q.cols, RPW, num_sms);
    note_launches(1);
    dequantize_kernel<T, FORMAT, RPW><<<t.grid, kWarps * 32, 0, s>>>(
        q.codes, q.scales, q.scale, q.rows, q.cols, fp4_k_tiles(q.cols, FORMAT), out, ldo, vec, t.cols,
        t.all);
    return cudaGetLastError();
}
template <typename T>
cudaError_t dequantize(const Fp4Matrix& q, T* out, int64_t ldo, int num_sms, cudaStream_t s) {
    const bool many = many_rows(q, num_sms);
    if (q.format == LL_FP4_MX)
        return many ? run_dequantize<T, LL_FP4_MX, 16>(q, out, ldo, num_sms, s)
                    : run_dequantize<T, LL_FP4_MX, 1>(q, out, ldo, num_sms, s);
    return many ? run_dequantize<T, LL_FP4_NV, 16>(q, out, ldo, num_sms, s)
                : run_dequantize<T, LL_FP4_NV, 1>(q, out, ldo, num_sms, s);
}

}  // namespace

cudaError_t launch_fp4_quantize(const void* x, int64_t ldx, int dtype, const Fp4Matrix& q,
                                float* scale, bool scale_given, int num_sms, cudaStream_t s) {
    if (dtype == LL_F32)
        return quantize(static_cast<const float*>(x), ldx, q, scale, scale_given, num_sms, s);
    if (dtype == LL_F16)
        return quantize(static_cast<const __half*>(x), ldx, q, scale, scale_given, num_sms, s);
    return quantize(static_cast<const __nv_bfloat16*>(x), ldx, q, scale, scale_given, num_sms, s);
}

cudaError_t launch_fp4_dequantize(const Fp4Matrix& q, void* out, int64_t ldo, int out_dtype,
                                  int num_sms, cudaStream_t s) {
    if (out_dtype == LL_F32) return dequantize(q, static_cast<float*>(out), ldo, num_sms, s);
    if (out_dtype == LL_F16) return dequantize(q, static_cast<__half*>(out), ldo, num_sms, s);
    return dequantize(q, static_cast<__nv_bfloat16*>(out), ldo, num_sms, s);
}

}  // namespace ll
