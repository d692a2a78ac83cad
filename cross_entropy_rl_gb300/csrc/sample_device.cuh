// What the kernels that draw tokens share: keys, weights, a row's settings.
#pragma once
#include "ll_device.cuh"
#include "rollout_internal.h"

namespace ll {

using u64 = unsigned long long;

// x as an integer that ascends with it; 0 for what is never drawn (NaN, -infinity).
__device__ __forceinline__ uint32_t key_of(float x) {
    if (!(x > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

constexpr int kFixBits = 46;

// round(2^S exp((x - m) / T)) for x <= m, with c = log2(e) / T as hi + lo.  The distance
// is taken without error, its product with c to 2^-48, 2^a = 2^n 2^(j / 32) e^y with the
// middle factor from a table and |y| <= ln 2 / 64: about 2^-37 of the weight in all.
struct alignas(16) WeightStep {  // 2^(j / 32) as hi + lo, and times 2^46
    float hi, lo;
    long long fix;
};
namespace {
__device__ const WeightStep kWeightSteps[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f, 70368744177664ll},
    {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f, 71909619029526ll},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f, 73484234647076ll},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f, 75093329856877ll},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f, 76737659663686ll},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f, 78417995604711ll},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f, 80135126111625ll},
    {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f, 81889856880508ll},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f, 83683011249884ll},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f, 85515430587047ll},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f, 87387974682833ll},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f, 89301522155045ll},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f, 91256970860713ll},
    {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f, 93255238317374ll},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f, 95297262133585ll},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f, 97384000448854ll},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f, 99516432383215ll},
    {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f, 101695558496638ll},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f, 103922401258502ll},
    {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f, 106198005527352ll},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f, 108523439041155ll},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f, 110899792918296ll},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f, 113328182169538ll},
    {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f, 115809746221205ll},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f, 118345649449807ll},
    {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f, 120937081728377ll},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f, 123585258984778ll},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f, 126291423772226ll},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f, 129056845852306ll},
    {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f, 131882822790765ll},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f, 134770680566339ll},
    {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f, 137721774192917ll}};
}  // namespace
// The 32 of them to shared memory, by the first 32 threads.
__device__ __forceinline__ void fill_table(WeightStep* tab) { tab[threadIdx.x] = kWeightSteps[threadIdx.x]; }

struct Weights {
    float m, c_hi, c_lo;
    int S;
    uint32_t tab;  // shared-memory address
    // Without branches, and without conversions: an integer is the low bits of x + 1.5 * 2^23.
    __device__ __forceinline__ unsigned long long operator()(float x) const {
        constexpr float kMagic = 12582912.f;
        constexpr int kMagicBits = 0x4b400000;
        const float d = __fsub_rn(x, m), b = __fsub_rn(d, x);
        const float e = __fadd_rn(__fsub_rn(x, __fsub_rn(d, b)), __fsub_rn(-m, b));
        const float a = __fmul_rn(d, c_hi);
        const bool some = a > -static_cast<float>(S + 2);
        const float a_lo = __fmaf_rn(d, c_hi, -a) + __fmaf_rn(d, c_lo, __fmul_rn(e, c_hi));
        const float t32 = __fmaf_rn(a, 32.f, kMagic);
        const float r = __fmaf_rn(__fsub_rn(t32, kMagic), -0.03125f, a);
        const int i = __float_as_int(t32) - kMagicBits, n = i >> 5;
        uint32_t hi_bits, lo_bits, fix_0, fix_1;
        asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
            : "=r"(hi_bits), "=r"(lo_bits), "=r"(fix_0), "=r"(fix_1)
            : "r"(tab + (i & 31) * 16));
        constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.90465421e-9f;
        const float y = __fmul_rn(r, kLn2Hi);
        const float y_lo = __fmaf_rn(r, kLn2Hi, -y) + __fmaf_rn(r, kLn2Lo, __fmul_rn(a_lo, kLn2Hi));
        const float p = __fmaf_rn(y, __fmaf_rn(y, __fmaf_rn(y, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f);
        // e^y - 1 and y_lo e^y: y_lo is not small enough for y_lo alone (2^-20 where |a| is 17)
        const float y2 = __fmul_rn(y, y);
        const float q_lo = __fmaf_rn(y2, p, __fmaf_rn(y_lo, __fmaf_rn(y2, p, y), y_lo));
        const float q = __fadd_rn(y, q_lo), rest_q = __fadd_rn(__fsub_rn(y, q), q_lo);  // e^y - 1
        const float t = __uint_as_float(hi_bits);
        const float u = __fmul_rn(t, q);  // below 0.022
        const float u_lo = __fmaf_rn(t, q, -u) + __fmaf_rn(t, rest_q, __fmul_rn(__uint_as_float(lo_bits), q));
        // times 2^46 in two steps of 32 bits
        const float s27 = __fmaf_rn(u, 0x1p27f, kMagic);
        const float rest = __fmaf_rn(__fsub_rn(s27, kMagic), -0x1p-27f, u) + u_lo;
        const float s46 = __fmaf_rn(rest, 0x1p46f, kMagic);
        const long long w = static_cast<long long>((static_cast<u64>(fix_1) << 32) | fix_0) +
                            (static_cast<long long>(__float_as_int(s27) - kMagicBits) << 19) +
                            (__float_as_int(s46) - kMagicBits);
        const int sh = min(max(kFixBits - S - n, 0), 63);
        const u64 rounded = (static_cast<u64>(w) + ((1ull << sh) >> 1)) >> sh;
        return x == m ? 1ull << S : some ? rounded : 0ull;
    }
};

constexpr double kLog2e64 = 1.4426950408889634074;

// A row's settings.  FP64 is slow here: one thread works them out.
struct Settings {
    double T, p, min_p, u;
    double cd;  // log2(e) / T
    int64_t k;
    float c, c_lo;  // cd as hi + lo
    float off_c;    // |c / cd - 1|
};
__device__ __forceinline__ Settings settings_of(const SampleArgs& a, int64_t n) {
    Settings s;
    s.T = a.temperatures ? a.temperatures[n] : a.temperature;
    s.p = a.top_ps ? a.top_ps[n] : a.top_p;
    s.min_p = a.min_ps ? a.min_ps[n] : a.min_p;
    s.k = a.top_ks ? a.top_ks[n] : a.top_k;
    if (s.k <= 0 || s.k > a.V) s.k = a.V;
    if (!(s.T > 0)) {
        s.T = 1;
        s.k = 1;
    }
    if (!(s.p < 1)) s.p = 1;
    if (!(s.min_p > 0)) s.min_p = 0;
    s.u = a.uniforms[n];
    if (!(s.u > 0)) s.u = 0;
    if (!a.temperatures && s.T == a.temperature) {  // worked out by the host
        s.cd = a.cd;
        s.c = a.c;
        s.c_lo = a.c_lo;
    } else {
        s.cd = s.T == 1 ? kLog2e64 : kLog2e64 / s.T;
        s.c = static_cast<float>(s.cd);
        s.c_lo = static_cast<float>(s.cd - s.c);
    }
    s.off_c = fabsf(s.c_lo / s.c) * 1.0001f;
    return s;
}

// Rows that some(n) holds for, dealt to the clusters in turn, kChunk rows at a time: this
// cluster's among [n0, n0 + kChunk) to d.rows, and how many.  `seen`: those dealt so far.
// some(n) may not change while a cluster still looks.
constexpr int kChunk = 2048;
struct Deal {
    uint32_t per_warp[32];
    uint16_t rows[kChunk];
};
template <int NT, class F>
__device__ __forceinline__ uint32_t deal_rows(F some, int64_t n0, int64_t N, uint32_t clusters,
                                              uint32_t own, uint32_t& seen, Deal& d) {
    constexpr int kEach = kChunk / NT;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t n = n0 + tid * kEach + i;
        bits |= n < N && some(n) ? 1u << i : 0u;
    }
    const uint32_t mine = __popc(bits);
    uint32_t up = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
    }
    __syncthreads();
    if (lane == 31) d.per_warp[warp] = up;
    __syncthreads();
    uint32_t rank = up - mine, total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) rank += d.per_warp[w];
        total += d.per_warp[w];
    }
    // this cluster's are those whose rank, over all chunks, is `own` modulo the clusters
    const uint32_t first = (own + clusters - seen % clusters) % clusters;
    for (int i = 0; i < kEach; ++i)
        if ((bits >> i) & 1u) {
            if (rank >= first && (rank - first) % clusters == 0)
                d.rows[(rank - first) / clusters] = static_cast<uint16_t>(tid * kEach + i);
            ++rank;
        }
    seen = (seen + total) % clusters;
    return total > first ? (total - first + clusters - 1) / clusters : 0;
}

__host__ __device__ inline int weight_bits(int64_t V) {
    int b = 0;
    while ((int64_t(1) << b) < V) ++b;
    return 62 - b < kFixBits ? 62 - b : kFixBits;
}

}  // namespace ll
