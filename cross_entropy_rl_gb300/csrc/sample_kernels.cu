// Drawing a token from each row of logits: one pass over the row in FP32 with a bound of
// its error, then the tokens near the outcome once more.
//
// A row is cut into groups of 256 logits and 64 ranges of groups.  The pass keeps the
// largest logit of each group and, of each range, the sum of 2^(x c - ref), c = log2(e) / T
// (ref an integer, so that ranges and rescaling lose nothing), as a pair of FP32 values.
//  - Nothing cut off: the drawn token's range, group and place follow from the sums; the
//    group sums of one range are formed again.
//  - A small top_k, top_p or min_p: a floor below which no token can be left (for top_k, the
//    k-th largest of the groups' maxima) leaves a few groups to read again.  Their tokens at
//    or above the floor are sorted, and cut and drawn with integer weights.
//  - A top_p that leaves many tokens: a histogram of the mass over x c finds the narrow
//    piece that the border lies in, a second pass sums what is above it and lists the piece;
//    the list is sorted, the border found in it, and the draw made as if nothing were cut.
//    A min_p that leaves many: the same with the piece around its own border.
//  - Where the outcome lies within the bound of the error, one more pass forms every weight as
//    an integer, round(2^S w): its sums, over all tokens and over those above the piece, decide.
//    A cluster does that itself; a row of one block waits for a second launch, in clusters.
//  - Other rows go to the exact kernel (sample_exact.cu): a top_k above 256 or a min_p that
//    leaves many, lists that overflow, u of 1 or more, logits or temperatures out of proportion.
// One block a row, or for few rows a cluster of 8, whose first CTA (the leader) decides; the
// ranges, and so all sums, are the same.
//
// Rows of 151936, us: 1024 uncut (bf16) 160, of which HBM would take 46; 512 with top_p 0.9 311; 512
// with min_p 0.001 198; 48 (FP32) with top_k 50 and top_p 0.95 31.  The launches one by one under a
// profiler, whose caches are cold, us: uncut 95 (14 warp instructions for 32 logits, the schedulers
// issue in 64% of cycles) and then 61 for the 29 rows of 1024 that the FP32 bound leaves to
// clusters, each a whole pass again and a chain of short steps (25%); top_p 230 and 159 for 68 of
// 512 rows; 8 to 9 for an exact kernel that finds no row.
//
// Errors: with weights off by e_w at most (relative) and a target t = u Z, the difference of
// t and a sum P next to it is off by u e_w (Z - P) + (1 - u) e_w P: what P and Z share
// cancels.  A draw is taken where it lies further from both borders of its token.
#include "sample_device.cuh"
#include "step_device.cuh"

namespace ll {
namespace {

constexpr int kRanges = 64;        // two a lane where a warp looks at all
constexpr int kGroup = 256;
constexpr int kList = 1024;       // tokens of a list
constexpr int kShort = 128;       // lists sorted by counting
constexpr int kBins = 1024;       // of the mass histogram
constexpr int kSmallK = 256;      // largest top_k taken from the groups' maxima
constexpr int kMaxGroups = 8192;  // groups of a row
constexpr int kMaxPer = kMaxGroups / kRanges;  // groups of a range
constexpr int kHeadroom = 6;      // weights up to 2^6: rounding of x c - ref is least near 0

// Largest relative error of ex2.approx.ftz over all floats in [-125, 125]: 2^-22.70.
constexpr double kEx2Error = 1.6e-7;

struct alignas(8) RangeInfo {
    float hi, lo;  // sum of 2^(x c - ref)
    float dist;    // sum of 2^(x c - ref) |x c - ref|
    float top;     // largest x
    int ref;
};

enum Mode : int { kDone, kExact, kFew, kWide, kSums };

struct Shared {
    RangeInfo range[kRanges];
    Settings set;
    Deal deal;
    WeightStep tab[32];
    // the leader's
    u64 list[kList];
    u64 sum[kList];
    u64 part[32];
    uint32_t bins[kBins];      // every CTA's
    uint32_t bins_all[kBins];  // the leader's, over the CTAs
    u64 gsum[kMaxPer];
    u64 before[kRanges + 1];  // sums ahead of each range, see to_fix
    u64 range_list[kRanges];
    u64 range_all[kRanges], range_above[kRanges];  // integer weights
    // of the row, worked out by one thread (FP64 is slow here)
    double mass;          // of all tokens, then of those left, units of 2^-ref
    double log_z;         // log of the sum of all weights, the largest being 1
    double e_w, e_a;      // errors of a sum: e_w of it, and e_a
    float dist_upto[32];  // sums of weight times |x c - ref| up to range 2 i + 1
    float e_unit, e_c;    // e_a = e_unit times the whole of these + e_c
    double p_lo, p_hi;    // bounds of top_p of the mass, as integer weights (top_k off)
    double scale;         // of a weight relative to 2^ref to one relative to the largest
    int sure;             // see refine()
    double one;           // 2^S
    double per_one;       // an integer weight of 1 in units of 2^-ref
    u64 least;            // min_p
    u64 target, total, ahead;
    float top, floor_x;
    int ref;
    Mode mode;
    int n_list;
    int count;
    uint32_t kth;
    // the mass histogram
    float bin_a, bin_b;   // bin = x c - ref times a, plus b
    float unit;           // mass of 1
    float x_floor;        // the lowest exponent in it
    int large;            // a weight of more than 2^21 units
    // the piece that the border lies in: exponents in (x_lo, x_hi]; all above x_hi are left
    float x_lo, x_hi;
    int by_min;           // the piece is around min_p's border
    int kept;             // of the list
    // the tokens left: x > last, or x == last and index < last_end
    float last;
    uint32_t last_end;
};

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float pow2i(int k) {  // 2^k for k <= 0, 0 below FP32's range
    return k < -126 ? 0.f : __int_as_float((k + 127) << 23);
}

__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ u64 scan_up64(u64 x) {  // inclusive, over a warp
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const u64 other = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += other;
    }
    return x;
}

// Sums of weights as integers in units of 2^(ref - 34): 8 additions in FP64 take as long here
// as a hundred of these.  A sum is below 2^62; the few hundred roundings to a unit on the way
// to a draw are within 2^-32 of the mass, which is at least 2^6.
constexpr int kFix = 34;
__device__ __forceinline__ u64 to_fix(float x) {  // x >= 0, below 2^28
    const uint32_t bits = __float_as_uint(x), m = (bits & 0x7fffffu) | 0x800000u;
    const int e = static_cast<int>(bits >> 23), s = e - (150 - kFix);
    const u64 big = static_cast<u64>(m) << max(s, 0);
    const uint32_t small = s > -25 ? (m + ((1u << max(-s, 0)) >> 1)) >> max(-s, 0) : 0u;
    return e == 0 ? 0 : s >= 0 ? big : small;
}
__device__ __forceinline__ u64 fix_pair(float hi, float lo) {
    const u64 l = to_fix(fabsf(lo));
    return to_fix(hi) + (lo < 0.f ? ~l + 1 : l);
}
__device__ __forceinline__ double from_fix(u64 x) {
    return static_cast<double>(x) * (1.0 / static_cast<double>(1ull << kFix));
}

// log(x 2^-shift) for a normal x > 0, to 1e-7 (and of the result, where that is small): FP64
// logarithms take microseconds here.
__device__ __forceinline__ double log_of(double x, int shift = 0) {
    const int hi = __double2hiint(x);
    int e = (hi >> 20) - 1023;
    double m = __hiloint2double(hi - (e << 20), __double2loint(x));  // [1, 2)
    if (m > 1.5) {  // nearer to 2: a little below a power of two is a small negative number
        m *= 0.5;
        ++e;
    }
    const float f = static_cast<float>(m);
    const float l = logf(f) + static_cast<float>(m - f) / f;
    return (e - shift) * 0.69314718055994530942 + l;
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ u64 pack2(float lo, float hi) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(u64 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 x, u64 y, u64 z) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ u64 add2(u64 x, u64 y) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

// What weighs nothing beside the row's largest logit is raised to `low`, so that no infinity
// and no NaN enters the sums.  A row whose largest is below `least_top`, or at whose
// temperature the distance between the two weighs anything, goes to the exact kernel.
template <typename T>
struct Bounds {
    static constexpr float low = -0x1p20f, least_top = -0x1p19f;
};
template <>
struct Bounds<__half> {
    static constexpr float low = -65504.f, least_top = -0x1p15f;
};

// A lane's 8 logits of a group, raised to Bounds::low.
template <typename T>
struct Raw {
    static constexpr int kWords = sizeof(T) * 2;
    uint32_t v[kWords];
    static __device__ __forceinline__ uint32_t max_2(uint32_t x, uint32_t y) {  // two 16-bit values
        uint32_t r;
        if constexpr (std::is_same<T, __half>::value)
            asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        else
            asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    }
    static __device__ __forceinline__ float2 get2(uint32_t x) {
        if constexpr (std::is_same<T, __half>::value)
            return __half22float2(*reinterpret_cast<const __half2*>(&x));
        else
            return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    // Bounds::low in every place of a word
    static constexpr uint32_t kLow = sizeof(T) == 4                  ? 0xc9800000u
                                     : std::is_same<T, __half>::value ? 0xfbfffbffu
                                                                      : 0xc980c980u;
    __device__ __forceinline__ void raise() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 2)
                v[i] = max_2(v[i], kLow);
            else
                v[i] = __float_as_uint(fmaxf(__uint_as_float(v[i]), Bounds<T>::low));
        }
    }
    __device__ __forceinline__ void none() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) v[i] = kLow;
    }
    __device__ __forceinline__ void load(const T* p) {  // 16-byte aligned
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(p)[i];
            v[4 * i] = u.x;
            v[4 * i + 1] = u.y;
            v[4 * i + 2] = u.z;
            v[4 * i + 3] = u.w;
        }
        raise();
    }
    // at any alignment and at the row's end (n of them)
    __device__ __forceinline__ void load_edge(const T* p, int64_t n) {
        T e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = j < n ? p[j] : Elem<T>::from_f(-INFINITY);
        memcpy(v, e, sizeof(v));
        raise();
    }
    __device__ __forceinline__ float top() const {
        if constexpr (sizeof(T) == 2) {
            const float2 m = get2(max_2(max_2(v[0], v[1]), max_2(v[2], v[3])));
            return fmaxf(m.x, m.y);
        } else {
            float f[8];
            get(f);
            return max3f(max3f(f[0], f[1], f[2]), max3f(f[3], f[4], f[5]), fmaxf(f[6], f[7]));
        }
    }
    __device__ __forceinline__ float2 pair(int i) const {  // logits 2 i and 2 i + 1
        if constexpr (sizeof(T) == 2)
            return get2(v[i]);
        else
            return make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    }
    __device__ __forceinline__ float2 pair_at(int i) const {  // any i, without local memory
        float2 p = pair(0);
#pragma unroll
        for (int k = 1; k < 4; ++k)
            if (i == k) p = pair(k);
        return p;
    }
    __device__ __forceinline__ void get(float* f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 p = pair(i);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
};

// Exponents x c - ref and weights of 8 logits.
template <typename T>
__device__ __forceinline__ void weights8(const Raw<T>& raw, float c, float ref, float* a, float* w) {
    const u64 c2 = pack2(c, c), r2 = pack2(-ref, -ref);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = raw.pair(i);
        const float2 e = unpack2(fma2(pack2(x.x, x.y), c2, r2));
        a[2 * i] = e.x;
        a[2 * i + 1] = e.y;
        w[2 * i] = ex2(e.x);
        w[2 * i + 1] = ex2(e.y);
    }
}
__device__ __forceinline__ float tree8(const float* w) {
    const u64 s = add2(add2(pack2(w[0], w[1]), pack2(w[2], w[3])),
                       add2(pack2(w[4], w[5]), pack2(w[6], w[7])));
    const float2 p = unpack2(s);
    return p.x + p.y;
}
__device__ __forceinline__ void add_to(Pair& sum, float t) {
    const float s = __fadd_rn(sum.hi, t), b = __fsub_rn(s, sum.hi);
    sum.lo += __fadd_rn(__fsub_rn(sum.hi, __fsub_rn(s, b)), __fsub_rn(t, b));
    sum.hi = s;
}

// The sums of a range in the pass, by one warp.
struct RangeSum {
    float c, ref_f = 0.f, top = -INFINITY, dist = 0.f;
    int ref = 0;
    Pair sum = {0.f, 0.f};
    // two groups, and their maxima
    template <typename T>
    __device__ __forceinline__ float2 groups(const Raw<T>& raw0, const Raw<T>& raw1) {
        const float m0 = warp_max(raw0.top()), m1 = warp_max(raw1.top()), m = fmaxf(m0, m1);
        if (m > top) {
            const int r = static_cast<int>(fminf(fmaxf(ceilf(m * c), -0x1p21f), 0x1p21f)) - kHeadroom;
            if (r > ref || top == -INFINITY) {
                if (top > -INFINITY) {
                    const float k = pow2i(ref - r);
                    sum.hi *= k;
                    sum.lo *= k;
                    dist *= k;
                }
                ref = r;
                ref_f = static_cast<float>(r);
            }
            top = m;
        }
        float a[16], w[16];
        weights8(raw0, c, ref_f, a, w);
        weights8(raw1, c, ref_f, a + 8, w + 8);
        float d[4] = {};
#pragma unroll
        for (int j = 0; j < 16; ++j) d[j % 4] = fmaf(w[j], fabsf(a[j]), d[j % 4]);
        dist += (d[0] + d[1]) + (d[2] + d[3]);
        add_to(sum, tree8(w));
        add_to(sum, tree8(w + 8));
        return make_float2(m0, m1);
    }
    __device__ __forceinline__ RangeInfo finish() {
        const Pair p = warp_sum(sum);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dist += __shfl_xor_sync(0xffffffffu, dist, o);
        return {p.hi, p.lo, dist, top, ref};
    }
};

// `x` of the CTA of this rank.
template <int C, typename V>
__device__ __forceinline__ V at_rank(const V* x, int rank) {
    if constexpr (C == 1) {
        return *x;
    } else {
        const uint32_t p = cluster_addr(x, rank);
        uint32_t w[sizeof(V) / 4];
#pragma unroll
        for (int i = 0; i < int(sizeof(V) / 4); ++i)
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(w[i]) : "r"(p + 4 * i) : "memory");
        V v;
        memcpy(&v, w, sizeof(V));
        return v;
    }
}

// A row as the threads of its CTAs see it.  C CTAs of NT threads.
template <typename T, int C, int NT>
struct Row {
    static constexpr int kMine = kRanges / C;  // ranges of a CTA
    static constexpr int kWarps = NT / 32;
    static constexpr int kOwn = kMine / kWarps;  // ranges of a warp, side by side
    static constexpr int kRing = sizeof(T) == 4 ? 4 : 8;  // groups on their way to a warp: 4 KB
    const SampleArgs& a;
    Shared& sh;
    float* gmax;  // the leader's: of every group
    float* mine;  // of this CTA's groups
    T* ring;
    const T* row;
    int64_t n, V;
    int G, per, rank, tid, warp, lane;
    bool vec, again;

    __device__ __forceinline__ void sync() const {
        __syncthreads();
        if constexpr (C > 1) {
            __syncwarp();  // the cluster's barrier wants whole warps: lanes come from ways of their own
            cluster_barrier();
        }
    }
    __device__ __forceinline__ Raw<T> load(int g) const {
        const int64_t v = int64_t(g) * kGroup + lane * 8;
        Raw<T> raw;
        if (vec && int64_t(g + 1) * kGroup <= V)
            raw.load(row + v);
        else
            raw.load_edge(row + v, V - v);
        return raw;
    }
    // each(g, n, raw, raw of g + 1) for the groups of this warp's ranges in turn, n = 2 at a
    // time (a range's odd one, n = 1, with a second that holds nothing); end(r) after a range.
    // Whole groups at 16-byte addresses come through a ring in shared memory: a lane copies
    // what it will read itself.  The twos are the same at any address, and with them what is
    // rounded.
    template <class F, class E>
    __device__ __forceinline__ void stream(F each, E end) const {
        const int r0 = rank * kMine + warp * kOwn;
        const int g0 = r0 * per, ge = min(G, g0 + kOwn * per);
        const int whole = static_cast<int>(V / kGroup), gv = vec ? min(ge, whole) : g0;
        constexpr uint32_t kStep = kGroup * sizeof(T), kAll = kRing * kStep;
        T* own = ring + (warp * kRing * 32 + lane) * 8;
        const uint32_t to = smem_u32(own);
        const T* from = row + int64_t(g0) * kGroup + lane * 8;
        int next = g0;        // to fetch
        uint32_t next_at = 0;
        auto fetch = [&]() {
            if (next < gv) {
#pragma unroll
                for (int i = 0; i < int(sizeof(T)) / 2; ++i)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + next_at + 16 * i),
                                 "l"(reinterpret_cast<const char*>(from) + 16 * i)
                                 : "memory");
                from += kGroup;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++next;
            next_at = (next_at + kStep) % kAll;
        };
        auto slot = [&](uint32_t at) {
            return reinterpret_cast<const T*>(reinterpret_cast<const char*>(own) + at);
        };
#pragma unroll
        for (int i = 0; i < kRing - 2; ++i) fetch();
        int g = g0;
        uint32_t at = 0;  // of group g's slot
        for (int r = r0; r < r0 + kOwn; ++r) {
            const int g1 = min(ge, (r + 1) * per);
            for (; g + 1 < min(g1, gv); g += 2) {
                fetch();
                fetch();
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
                Raw<T> raw0, raw1;
                raw0.load(slot(at));
                raw1.load(slot((at + kStep) % kAll));
                at = (at + 2 * kStep) % kAll;
                each(g, 2, raw0, raw1);
            }
            for (int n; g < g1; g += n) {
                Raw<T> raw0, raw1;
                raw1.none();
                n = 1;
                if (g < gv) {
                    fetch();
                    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
                    raw0.load(slot(at));
                    at = (at + kStep) % kAll;
                } else {
                    raw0 = load(g);
                    if (g + 1 < min(g1, whole)) {
                        raw1 = load(g + 1);
                        n = 2;
                    }
                }
                each(g, n, raw0, raw1);
            }
            end(r);
        }
    }

    __device__ __forceinline__ void pass() {
        const uint32_t to = C == 1 ? 0 : cluster_addr(gmax, 0);
        const int first = rank * kMine * per;
        RangeSum s;
        s.c = sh.set.c;
        stream(
            [&](int g, int n_here, const Raw<T>& raw0, const Raw<T>& raw1) {
                const float2 m = s.groups(raw0, raw1);
                if (lane < n_here) {
                    const float own = lane ? m.y : m.x;
                    mine[g + lane - first] = own;
                    if constexpr (C > 1)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                                         to + static_cast<uint32_t>(g + lane) * 4),
                                     "f"(own)
                                     : "memory");
                }
            },
            [&](int r) {
                const RangeInfo info = s.finish();
                if (lane == 0) sh.range[r % kMine] = info;
                s = RangeSum{};
                s.c = sh.set.c;
            });
    }

    // ------------------------------------------------------------- the leader
    // Warp 0: sh.before from the sums of ranges 2 lane and 2 lane + 1; the sum up to these.
    __device__ __forceinline__ u64 set_before(u64 x0, u64 x1) {
        const u64 up = scan_up64(x0 + x1);
        if (lane == 0) sh.before[0] = 0;
        sh.before[2 * lane + 1] = up - x1;
        sh.before[2 * lane + 2] = up;
        return up;
    }
    // Warp 0: the row's sums, and what follows from them and the settings.
    __device__ __forceinline__ void combine() {
        RangeInfo r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r[i] = at_rank<C>(&sh.range[(2 * lane + i) % kMine], (2 * lane + i) / kMine);
        const float top = warp_max(fmaxf(r[0].top, r[1].top));
        int ref = -(1 << 28);  // a range may have no group
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (r[i].top > -INFINITY) ref = max(ref, r[i].ref);
        ref = __reduce_max_sync(0xffffffffu, ref);
        u64 own[2];
        float d = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float k = r[i].top > -INFINITY ? pow2i(r[i].ref - ref) : 0.f;
            own[i] = fix_pair(r[i].hi * k, r[i].lo * k);
            d += r[i].dist * k * 1.0001f;
        }
        const u64 up = set_before(own[0], own[1]);
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float other = __shfl_up_sync(0xffffffffu, d, o);
            if (lane >= o) d += other;
        }
        sh.dist_upto[lane] = d;  // lane 31: of all
        if (lane < 31) return;
        const Settings& set = sh.set;
        const double Z = from_fix(up);
        const float Zf = static_cast<float>(Z);
        sh.top = top;
        sh.ref = ref;
        sh.n_list = 0;
        sh.mode = kExact;
        if (!(top >= Bounds<T>::least_top && set.c * (Bounds<T>::least_top - Bounds<T>::low) > 256.f &&
              fabsf(top * set.c) < 0x1p20f && Zf > 0.f && Zf < INFINITY && set.u < 1))
            return;
        // Relative errors of the weights: the exponential and the sum of 8, and per unit of
        // |x c - ref| the rounding of x c - ref and of c; the rest is in pairs or FP64.
        sh.mass = Z;
        sh.e_w = kEx2Error + 3.1 * 0x1p-24;
        sh.e_unit = 0.7f * (0x1p-24f + set.off_c) * 1.01f;
        // c's error also where integer weights, relative to the largest, meet these
        sh.e_c = 0.7f * set.off_c * (kHeadroom + 1) * Zf;
        sh.e_a = sh.e_unit * d + sh.e_c;
        const float E = static_cast<float>(sh.e_w) + static_cast<float>(sh.e_a) / Zf * 1.01f + 1e-12f;
        if (!(E < 1e-3f)) return;
        const bool cut = set.k < V || set.p < 1 || set.min_p > 0;
        if (set.k < V && set.k > kSmallK) return;
        sh.mode = cut ? kFew : kDone;
        // the largest weighs 2^(top c - ref), with the rounded c: 1 / scale
        sh.scale = exp2(sh.ref - static_cast<double>(top) * set.c);
        sh.log_z = log_of(Z * sh.scale);
        sh.one = static_cast<double>(1ull << weight_bits(V));
        // A floor under the tokens left, a little lower than the bounds: these are sums of rounded
        // numbers, and off by a few 2^-24 of each where they cancel (and where a logarithm is near
        // 0, of one unit of it).
        float at = -INFINITY;
        auto lower = [](float x, float y, float unit) {
            const float sum = x + y;
            return sum - 1e-4f * fabsf(sum) - 1e-6f * (fabsf(x) + fabsf(y) + unit);
        };
        if (set.k >= V && set.p < 1) {
            // all that lies below weight w_f weighs less than V w_f = (1 - p) Z
            const double m = set.p * Z;
            const float w_f = static_cast<float>(Z - m) * (1.f - 2.f * E) / static_cast<float>(V);
            if (w_f > 1e-30f) at = lower(log2f(w_f), static_cast<float>(ref), 1.f) / set.c;
            const double scale = sh.scale * sh.one;
            sh.p_lo = m * scale * (1.0 - E) - 2.0 * kList;  // the list's weights are rounded
            sh.p_hi = m * scale * (1.0 + E) + 2.0 * kList;
        }
        sh.least = 0;
        if (set.min_p > 0) {
            const double r_min = fmin(set.min_p, 1.0);
            if (r_min > 1e-30 && !(set.k < V && set.p < 1))  // top_p is of the whole top_k's mass
                at = fmaxf(at, lower(top, logf(static_cast<float>(r_min)) * static_cast<float>(set.T),
                                     static_cast<float>(set.T)));
            sh.least = static_cast<u64>(ceil(r_min * sh.one));
        }
        sh.per_one = 1.0 / (sh.scale * sh.one);
        sh.sure = Zf * static_cast<float>(sh.scale) < 1.9f;
        sh.by_min = 0;
        sh.floor_x = fminf(at, top);
    }
    // Warp 1: a value that at least k of the maxima reach, and so k tokens; a quarter more
    // than k will do.
    __device__ __forceinline__ void kth_max() {
        uint32_t key = 0;
        if (sh.set.k < G && sh.set.k <= kSmallK) {
            constexpr int kHeld = 20;  // maxima of a lane: 163840 logits
            const uint32_t k = static_cast<uint32_t>(sh.set.k);
            uint32_t x[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int g = lane + 32 * i;
                x[i] = g < G ? key_of(gmax[g]) : 0u;
            }
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t probe = key | (1u << bit);
                uint32_t have = 0;
#pragma unroll
                for (int i = 0; i < kHeld; ++i) have += x[i] >= probe;
                for (int g = lane + 32 * kHeld; g < G; g += 32) have += key_of(gmax[g]) >= probe;
                have = __reduce_add_sync(0xffffffffu, have);
                if (have >= k) key = probe;
                // (near G, k + k / 4 would take in groups of any maximum)
                if (have >= k && have <= min(k + k / 4, (k + static_cast<uint32_t>(G)) / 2)) break;
            }
        }
        if (lane == 0) sh.kth = key;
    }

    // The same from the tokens themselves, where fewer than k groups have one that counts.
    __device__ __forceinline__ float kth_token() {
        const int k = static_cast<int>(sh.set.k);
        uint32_t key = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t probe = key | (1u << bit);
            int have = 0;
            for (int g = warp; g < G; g += kWarps) {
                if (gmax[g] <= Bounds<T>::low) continue;
                float f[8];
                load(g).get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j) have += key_of(f[j]) >= probe;
            }
            have = block_sum(have);
            if (have >= k) key = probe;
            if (have >= k && have <= k + k / 4) break;
        }
        return key ? value_of(key) : -INFINITY;
    }

    // Sum over the block of a value a thread.
    __device__ __forceinline__ int block_sum(int x) const {
        x = __reduce_add_sync(0xffffffffu, x);
        __syncthreads();
        if (tid == 0) sh.count = 0;
        __syncthreads();
        if (lane == 0 && x) atomicAdd(&sh.count, x);
        __syncthreads();
        return sh.count;
    }
    // Inclusive prefix sums of sh.sum[0, P), P a multiple of 32: of 32 by a warp, then of those.
    __device__ __forceinline__ void scan_list(int P) const {
        __syncthreads();
        for (int i0 = warp * 32; i0 < P; i0 += NT) {
            const u64 up = scan_up64(sh.sum[i0 + lane]);
            sh.sum[i0 + lane] = up;
            if (lane == 31) sh.part[i0 / 32] = up;
        }
        __syncthreads();
        if (P > 32) {
            if (warp == 0) {
                const u64 own = lane < P / 32 ? sh.part[lane] : 0;
                sh.part[lane] = scan_up64(own) - own;
            }
            __syncthreads();
            for (int i = tid; i < P; i += NT) sh.sum[i] += sh.part[i / 32];
            __syncthreads();
        }
    }
    // sh.list[0, L) in falling order (its values differ).  Uses sh.sum.
    __device__ __forceinline__ void sort_list(int L) const {
        if (L <= kShort) {
            __syncthreads();
            for (int i = tid; i < L; i += NT) {
                const u64 x = sh.list[i];
                int at = 0;
                for (int j = 0; j < L; ++j) at += sh.list[j] > x;
                sh.sum[at] = x;
            }
            __syncthreads();
            for (int i = tid; i < L; i += NT) sh.list[i] = sh.sum[i];
            __syncthreads();
            return;
        }
        int P = 2 * kShort;
        while (P < L) P *= 2;
        for (int i = L + tid; i < P; i += NT) sh.list[i] = 0;
        for (int k = 2; k <= P; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                __syncthreads();
                for (int i = tid; i < P / 2; i += NT) {
                    const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
                    const u64 x = sh.list[lo], y = sh.list[hi];
                    if ((x < y) == ((lo & k) == 0)) {
                        sh.list[lo] = y;
                        sh.list[hi] = x;
                    }
                }
            }
        __syncthreads();
    }
    __device__ __forceinline__ Weights weights() const {
        Weights W;
        W.m = sh.top;
        W.c_hi = sh.set.c;
        W.c_lo = sh.set.c_lo;
        W.S = weight_bits(V);
        W.tab = smem_u32(sh.tab);
        return W;
    }
    // The sorted list's prefix sums of integer weights, P the list's length rounded up; returns
    // how many reach min_p.
    __device__ __forceinline__ int weigh_list(int L, int P) const {
        const Weights W = weights();
        const u64 least = sh.least;
        int n_min = 0;
        for (int i = tid; i < P; i += NT) {
            const u64 w = i < L ? W(value_of(static_cast<uint32_t>(sh.list[i] >> 32))) : 0;
            sh.sum[i] = w;
            n_min += i < L && w >= least;
        }
        n_min = block_sum(n_min);
        scan_list(P);
        return n_min;
    }
    __device__ __forceinline__ void write(int64_t v, float x, double log_left) const {
        const double z = x == sh.top ? 0.0
                                     : (static_cast<double>(x) - sh.top) * sh.set.cd * 0.69314718055994530942;
        a.tokens[n] = v;
        a.logp[n] = static_cast<float>(z - sh.log_z);
        a.logq[n] = static_cast<float>(z - log_left);
    }
    static __device__ __forceinline__ int round_up32(int L) { return (L + 31) / 32 * 32; }

    // draw_few for at most 64 tokens, by warp 0 (in all lanes): two a lane.
    __device__ __forceinline__ bool draw_some(int L) {
        const Settings& set = sh.set;
        const Weights W = weights();
        // by rank to their places in falling order
        u64 x[2];
        int place[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = lane + 32 * i < L ? sh.list[lane + 32 * i] : 0;
        for (int j = 0; j < L; ++j) {
            const u64 y = sh.list[j];
            place[0] += y > x[0];
            place[1] += y > x[1];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 32 * i < L) sh.list[place[i]] = x[i];
        __syncwarp();
        u64 w[2], before[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i] = 2 * lane + i < L ? sh.list[2 * lane + i] : 0;
            w[i] = 2 * lane + i < L ? W(value_of(static_cast<uint32_t>(x[i] >> 32))) : 0;
        }
        before[0] = scan_up64(w[0] + w[1]) - w[0] - w[1];
        before[1] = before[0] + w[0];
        // how many are left: places of the list for which a condition holds are its first ones
        auto count = [&](bool c0, bool c1) {
            return __popc(__ballot_sync(0xffffffffu, c0 && 2 * lane < L)) +
                   __popc(__ballot_sync(0xffffffffu, c1 && 2 * lane + 1 < L));
        };
        int left = set.min_p > 0 ? count(w[0] >= sh.least, w[1] >= sh.least) : L;
        if (set.k < left) left = static_cast<int>(set.k);
        if (set.p < 1) {
            double lo = sh.p_lo, hi = sh.p_hi;
            if (set.k < V) {
                const int last = static_cast<int>(min(int64_t(L), set.k)) - 1;
                const u64 m0 = __shfl_sync(0xffffffffu, before[0] + w[0], last / 2);
                const u64 m1 = __shfl_sync(0xffffffffu, before[1] + w[1], last / 2);
                lo = hi = fmax(ceil(set.p * static_cast<double>(last & 1 ? m1 : m0)), 1.0);
            }
            // integers below 2^62 against numbers: compared as integers
            const u64 need_lo = lo > 0 ? static_cast<u64>(ceil(lo)) : 0;
            const u64 need_hi = hi > 0 ? static_cast<u64>(ceil(hi)) : 0;
            const int n_lo = count(before[0] < need_lo, before[1] < need_lo);
            const int n_hi = count(before[0] < need_hi, before[1] < need_hi);
            if (min(left, n_lo) != min(left, n_hi)) return false;
            left = min(left, n_lo);
        }
        left = max(left, 1);
        const u64 t0 = __shfl_sync(0xffffffffu, before[0] + w[0], (left - 1) / 2);
        const u64 t1 = __shfl_sync(0xffffffffu, before[1] + w[1], (left - 1) / 2);
        const u64 total = (left - 1) & 1 ? t1 : t0;
        const double want = set.u * static_cast<double>(total);
        const u64 target = want < static_cast<double>(total) ? static_cast<u64>(want) : total - 1;
        // the weights ahead of each by index (the list's lower halves fall as the index rises)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < left) sh.sum[2 * lane + i] = w[i];
        __syncwarp();
        u64 ahead[2] = {0, 0};
        for (int j = 0; j < left; ++j) {
            const uint32_t y = static_cast<uint32_t>(sh.list[j]);
            const u64 wy = sh.sum[j];
            ahead[0] += y > static_cast<uint32_t>(x[0]) ? wy : 0;
            ahead[1] += y > static_cast<uint32_t>(x[1]) ? wy : 0;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < left && ahead[i] <= target && target < ahead[i] + w[i])
                write(0xffffffffu - static_cast<uint32_t>(x[i]), value_of(static_cast<uint32_t>(x[i] >> 32)),
                      log_of(static_cast<double>(total), weight_bits(V)));
        return true;
    }
    // The list holds every token that may be left: what lies below the floor is below min_p's
    // border, or beyond the nucleus, or beyond top_k.  Returns false where it cannot decide.
    __device__ __forceinline__ bool draw_few(int L) {
        const Settings& set = sh.set;
        if (L <= 64) {
            __syncthreads();
            if (warp == 0) {
                const bool done = draw_some(L);
                if (lane == 0) sh.count = done;
            }
            __syncthreads();
            return sh.count != 0;
        }
        sort_list(L);
        int P = round_up32(L);
        int left = weigh_list(L, P);
        if (set.k < V) left = static_cast<int>(min(int64_t(left), set.k));
        if (set.p < 1) {
            if (set.k < V) {
                if (tid == 0) {
                    const u64 m = sh.sum[static_cast<int>(min(int64_t(L), set.k)) - 1];
                    sh.p_lo = sh.p_hi = fmax(ceil(set.p * static_cast<double>(m)), 1.0);
                }
                __syncthreads();
            }
            const double lo = sh.p_lo, hi = sh.p_hi;
            int both = 0;
            for (int i = tid; i < L; i += NT) {
                const double before = i > 0 ? static_cast<double>(sh.sum[i - 1]) : 0.0;
                both += (before < lo ? 1 : 0) + (before < hi ? 1 << 16 : 0);
            }
            both = block_sum(both);
            const int n_lo = both & 0xffff, n_hi = both >> 16;
            if (min(left, n_lo) != min(left, n_hi)) return false;
            left = min(left, n_lo);
        }
        left = max(left, 1);
        if (tid == 0) {
            const u64 total = sh.sum[left - 1];
            const double want = set.u * static_cast<double>(total);
            sh.total = total;
            sh.target = want < static_cast<double>(total) ? static_cast<u64>(want) : total - 1;
        }
        __syncthreads();
        // by index
        for (int i = tid; i < left; i += NT) {
            const u64 x = sh.list[i];
            sh.list[i] = (x << 32) | (x >> 32);
        }
        sort_list(left);
        P = round_up32(left);
        const Weights W = weights();
        for (int i = tid; i < P; i += NT)
            sh.sum[i] = i < left ? W(value_of(static_cast<uint32_t>(sh.list[i]))) : 0;
        scan_list(P);
        const u64 target = sh.target;
        for (int i = tid; i < left; i += NT)
            if (sh.sum[i] > target && (i == 0 || sh.sum[i - 1] <= target))
                write(0xffffffffu - static_cast<uint32_t>(sh.list[i] >> 32),
                      value_of(static_cast<uint32_t>(sh.list[i])),
                      log_of(static_cast<double>(sh.total), weight_bits(V)));
        return true;
    }

    // The draw from the sums ahead of each range (sh.before) over the tokens that are left (all,
    // or those of sh.last).  Returns false where it lies too close to a border.
    template <bool CUT>
    __device__ __forceinline__ bool draw_in_ranges() {
        const float c = sh.set.c, ref_f = static_cast<float>(sh.ref), last = sh.last;
        const uint32_t last_end = sh.last_end;
        if (warp == 0) {
            const u64 t = static_cast<u64>(sh.set.u * static_cast<double>(sh.before[kRanges]));
            const uint32_t some = __ballot_sync(0xffffffffu, sh.before[2 * lane + 2] > t);
            if (lane == (some ? __ffs(some) - 1 : 31)) {
                sh.count = 2 * lane + (sh.before[2 * lane + 1] > t ? 0 : 1);
                sh.target = t;
            }
        }
        __syncthreads();
        const int r = sh.count;
        const int g0 = r * per, g1 = min(G, g0 + per);
        auto weigh = [&](int g, const Raw<T>& raw, float (&w)[8]) {
            float x[8];
            weights8(raw, c, ref_f, x, w);
            if (CUT) {
                const uint32_t v = static_cast<uint32_t>(g * kGroup + lane * 8);
                float f[8];
                raw.get(f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!(f[j] > last || (f[j] == last && v + j < last_end))) w[j] = 0.f;
            }
        };
        constexpr int kUnroll = 2;
        for (int g = g0 + warp * kUnroll; g < g1; g += kWarps * kUnroll) {
            Raw<T> raw[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) raw[i] = load(min(g + i, g1 - 1));
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                float w[8];
                weigh(min(g + i, g1 - 1), raw[i], w);
                const u64 sum = warp_sum64(to_fix(tree8(w)));
                if (lane == 0) sh.gsum[min(g + i, g1 - 1) - g0] = sum;
            }
        }
        __syncthreads();
        if (warp == 0) {
            const u64 K = sh.before[kRanges], t = sh.target;
            u64 before = sh.before[r];
            int g = g0;
            bool found = false;
            for (; g < g1; g += 32) {
                const u64 own = g + lane < g1 ? sh.gsum[g + lane - g0] : 0, up = scan_up64(own);
                const uint32_t over = __ballot_sync(0xffffffffu, before + up > t);
                if (over) {
                    const int at = __ffs(over) - 1;
                    before += __shfl_sync(0xffffffffu, up - own, at);
                    g += at;
                    found = true;
                    break;
                }
                before += __shfl_sync(0xffffffffu, up, 31);
            }
            bool here = false;
            if (found) {
                const Raw<T> raw = load(g);
                float f[8], w[8];
                raw.get(f);
                weigh(g, raw, w);
                u64 x_w[8], own = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) own += x_w[j] = to_fix(w[j]);
                u64 at = before + (scan_up64(own) - own), from = 0, wide = 0;
                float x = 0.f;
                int jx = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (at <= t && t < at + x_w[j]) {
                        from = at;
                        x = f[j];
                        wide = x_w[j];
                        jx = j;
                    }
                    at += x_w[j];
                }
                if (wide > 0) {
                    // what lies ahead errs by 1 - u of its share, what follows by u of it
                    const float u = static_cast<float>(sh.set.u), all = sh.dist_upto[31];
                    const float ahead = sh.dist_upto[r / 2], under = r > 1 ? sh.dist_upto[r / 2 - 1] : 0.f;
                    constexpr float kUnit = 1.f / (1ull << kFix);
                    const float upto = static_cast<float>(from + wide) * kUnit;
                    const float after = static_cast<float>(K - from) * kUnit;
                    const float e = (static_cast<float>(sh.e_w) * (upto * (1.f - u) + after * u) +
                                     sh.e_unit * (ahead * (1.f - u) + (all - under) * u) +
                                     (CUT ? sh.e_c : 0.f) + 1e-9f * static_cast<float>(K) * kUnit) * 1.001f;
                    if (static_cast<float>(t - from) * kUnit > e &&
                        static_cast<float>(from + wide - t) * kUnit > e) {
                        write(int64_t(g) * kGroup + lane * 8 + jx, x,
                              CUT ? log_of(from_fix(K) * sh.scale) : sh.log_z);
                        here = true;
                    }
                }
            }
            here = __any_sync(0xffffffffu, here);
            if (lane == 0) sh.count = here;
        }
        __syncthreads();
        return sh.count != 0;
    }

    // --------------------------------------------------------- every CTA's part
    __device__ __forceinline__ void append(int at, float x, int v) const {
        const u64 item = (u64(key_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(v));
        if (at >= kList) return;
        if constexpr (C == 1)
            sh.list[at] = item;
        else
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(&sh.list[at], 0)), "l"(item)
                         : "memory");
    }
    // Places in the leader's list for `count` tokens of each lane: the first of this lane's.
    __device__ __forceinline__ int take(int count) const {
        int up = count;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int other = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += other;
        }
        int at = 0;
        if (lane == 31 && up > 0) {
            if constexpr (C == 1)
                at = atomicAdd(&sh.n_list, up);
            else
                asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;"
                             : "=r"(at)
                             : "r"(cluster_addr(&sh.n_list, 0)), "r"(up)
                             : "memory");
        }
        return __shfl_sync(0xffffffffu, at, 31) + up - count;
    }
    // The tokens at or above the floor into the leader's list.
    __device__ __forceinline__ void gather() {
        const float floor_x = at_rank<C>(&sh.floor_x, 0);
        const int first = rank * kMine * per;
        for (int r = warp * kOwn; r < (warp + 1) * kOwn; ++r) {
            const int g0 = (rank * kMine + r) * per, g1 = min(G, g0 + per);
            for (int gb = g0; gb < g1; gb += 32) {
                uint32_t some = __ballot_sync(
                    0xffffffffu, gb + lane < g1 && mine[gb + lane - first] >= floor_x);
                bool full = false;  // the list: the rest does not matter
                while (some && !full) {
                    const int g = gb + __ffs(some) - 1;
                    some &= some - 1;
                    float f[8];
                    load(g).get(f);
                    uint32_t in = 0;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        in |= f[j] >= floor_x && f[j] > Bounds<T>::low ? 1u << j : 0u;
                    int at = take(__popc(in));
                    // past its end: after exactly kList tokens the next ones still have to show
                    full = __any_sync(0xffffffffu, at > kList);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if ((in >> j) & 1u) append(at++, f[j], g * kGroup + lane * 8 + j);
                }
            }
        }
    }

    // ------------------------------------------------- a top_p that leaves many
    // The leader's parameters of the histogram.
    __device__ __forceinline__ void start_wide() {
        if constexpr (C > 1)
            for (int i = tid; i < kBins; i += NT) sh.bins_all[i] = 0;
        if (tid == 0) {
            const float c = sh.set.c;
            const float hi = fmaf(sh.top, c, -static_cast<float>(sh.ref));
            const float lo = fmaf(sh.floor_x, c, -static_cast<float>(sh.ref));
            const float scale = (kBins - 2) / fmaxf(hi - lo, 1e-3f);
            sh.bin_a = -scale;
            sh.bin_b = hi * scale;
            sh.x_floor = lo;
            // the mass comes to about 2^29
            sh.unit = exp2f(29.f - ceilf(log2f(static_cast<float>(sh.mass))));
            sh.large = exp2f(hi) * sh.unit >= 0x1p21f;
        }
    }
    // The bin of an exponent x c - ref, rising as it falls, as 1.5 * 2^23 + bin: the integer is
    // the low bits (conversions run on the unit that the exponentials need).
    static constexpr float kMagic = 12582912.f;
    static constexpr uint32_t kMagicBits = 0x4b400000u;
    static __device__ __forceinline__ float bin_of(float x, float a, float b) {
        return __fadd_rn(__fmaf_rn(x, a, b), kMagic);
    }
    // The largest exponent whose bin is at least `bin`.
    static __device__ float edge_of(int bin, float a, float b) {
        if (bin <= 0) return INFINITY;
        const float at = kMagic + static_cast<float>(bin);
        float x = (static_cast<float>(bin) - 0.5f - b) / a;
        for (int i = 0; i < 256 && bin_of(x, a, b) >= at; ++i) x = nextafterf(x, INFINITY);
        for (int i = 0; i < 512 && bin_of(x, a, b) < at; ++i) x = nextafterf(x, -INFINITY);
        return x;
    }
    // Histogram of the mass over the bins, each CTA's added to the leader's sh.bins_all.
    __device__ __forceinline__ void histogram() {
        for (int i = tid; i < kBins; i += NT) sh.bins[i] = 0;
        __syncthreads();
        const float c = sh.set.c, ref_f = static_cast<float>(at_rank<C>(&sh.ref, 0));
        const float ba = at_rank<C>(&sh.bin_a, 0), bb = at_rank<C>(&sh.bin_b, 0);
        const float unit = at_rank<C>(&sh.unit, 0), x_floor = at_rank<C>(&sh.x_floor, 0);
        const bool large = at_rank<C>(&sh.large, 0);
        const u64 a2 = pack2(ba, ba), b2 = pack2(bb, bb), m2 = pack2(kMagic, kMagic), u2 = pack2(unit, unit);
        const uint32_t bins = smem_u32(sh.bins) - 4u * kMagicBits;  // modulo 2^32
        stream(
            [&](int, int, const Raw<T>& raw0, const Raw<T>& raw1) {
                float x[16], w[16];
                weights8(raw0, c, ref_f, x, w);
                weights8(raw1, c, ref_f, x + 8, w + 8);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 bin = unpack2(add2(fma2(pack2(x[j], x[j + 1]), a2, b2), m2));
                    float2 mass = unpack2(fma2(pack2(w[j], w[j + 1]), u2, m2));
                    uint32_t m0 = __float_as_uint(mass.x) - kMagicBits, m1 = __float_as_uint(mass.y) - kMagicBits;
                    if (large) {
                        m0 = __float2uint_rn(w[j] * unit);
                        m1 = __float2uint_rn(w[j + 1] * unit);
                    }
                    if (x[j] >= x_floor)
                        asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(bins + 4u * __float_as_uint(bin.x)),
                                     "r"(m0)
                                     : "memory");
                    if (x[j + 1] >= x_floor)
                        asm volatile("red.shared.add.u32 [%0], %1;" ::"r"(bins + 4u * __float_as_uint(bin.y)),
                                     "r"(m1)
                                     : "memory");
                }
            },
            [](int) {});
        if constexpr (C > 1) {
            __syncthreads();
            for (int i = tid; i < kBins; i += NT)
                if (sh.bins[i])
                    asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr(&sh.bins_all[i], 0)),
                                 "r"(sh.bins[i])
                                 : "memory");
        }
    }
    // The leader: the piece of the histogram that the border lies in.
    __device__ __forceinline__ void find_piece() {
        for (int i = tid; i < kBins; i += NT) sh.sum[i] = C == 1 ? sh.bins[i] : sh.bins_all[i];
        scan_list(kBins);
        if (tid == 0) {
            // each weight was rounded to a unit, and V of them may add up
            const double m = sh.set.p * sh.mass * sh.unit;
            const double off = 0.5 * static_cast<double>(V) + 1e-6 * sh.mass * sh.unit + 2.0;
            sh.p_lo = m - off;
            sh.p_hi = m + off;
        }
        __syncthreads();
        int both = 0;
        for (int i = tid; i < kBins; i += NT) {
            const double up = static_cast<double>(sh.sum[i]);
            both += (up < sh.p_lo ? 1 : 0) + (up < sh.p_hi ? 1 << 16 : 0);
        }
        both = block_sum(both);
        if (tid == 0) {
            sh.x_hi = edge_of(both & 0xffff, sh.bin_a, sh.bin_b);
            sh.x_lo = edge_of(min(both >> 16, kBins - 1) + 1, sh.bin_a, sh.bin_b);
            sh.n_list = 0;
        }
    }
    // The sums of what is above the piece, and the list of what is in it.
    __device__ __forceinline__ void split() {
        const float c = sh.set.c, ref_f = static_cast<float>(at_rank<C>(&sh.ref, 0));
        const float lo = at_rank<C>(&sh.x_lo, 0), hi = at_rank<C>(&sh.x_hi, 0);
        Pair sum = {0.f, 0.f};
        stream(
            [&](int g, int, const Raw<T>& raw0, const Raw<T>& raw1) {
                float x[16], w[16];
                weights8(raw0, c, ref_f, x, w);
                weights8(raw1, c, ref_f, x + 8, w + 8);
                uint32_t in = 0;  // of the piece
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    in |= x[j] > lo && x[j] <= hi ? 1u << j : 0u;
                    w[j] = x[j] > hi ? w[j] : 0.f;
                }
                if (__any_sync(0xffffffffu, in)) {
                    int at = take(__popc(in));
                    while (in) {
                        const int j = __ffs(in) - 1;
                        in &= in - 1;
                        const float2 p = (j < 8 ? raw0 : raw1).pair_at(j % 8 / 2);
                        append(at++, j & 1 ? p.y : p.x, (g + j / 8) * kGroup + lane * 8 + j % 8);
                    }
                }
                add_to(sum, tree8(w));
                add_to(sum, tree8(w + 8));
            },
            [&](int r) {
                const Pair p = warp_sum(sum);
                if (lane == 0) {
                    sh.range[r % kMine].hi = p.hi;
                    sh.range[r % kMine].lo = p.lo;
                }
                sum = {0.f, 0.f};
            });
    }
    // How many of the sorted list are left, from its sums and the bounds; 0: undecided.
    __device__ __forceinline__ int border() {
        const int L = sh.n_list;
        int both = 0;
        for (int i = tid; i < L; i += NT) {
            const double before = i > 0 ? static_cast<double>(sh.sum[i - 1]) : 0.0;
            both += (before < sh.p_lo ? 1 : 0) + (before < sh.p_hi ? 1 << 16 : 0);
        }
        both = block_sum(both);
        const int left = both & 0xffff;
        if (left != both >> 16) return 0;
        return left < L || static_cast<double>(sh.sum[L - 1]) >= sh.p_hi ? left : 0;
    }
    // The list's first `left` to the sums of their ranges, and the last of them.
    __device__ __forceinline__ void keep_list(int left) {
        for (int i = tid; i < left; i += NT) {
            const u64 item = sh.list[i];
            const uint32_t v = 0xffffffffu - static_cast<uint32_t>(item);
            const u64 w = sh.sum[i] - (i > 0 ? sh.sum[i - 1] : 0);
            atomicAdd(&sh.range_list[v / (static_cast<uint32_t>(per) * kGroup)], w);
            if (i == left - 1) {
                sh.last = value_of(static_cast<uint32_t>(item >> 32));
                sh.last_end = v + 1;
            }
        }
        __syncthreads();
    }
    // The leader: the border in the list, and the draw.
    // The sums of split() to sh.before, and the list in order with its prefix sums; returns how
    // many of the list reach min_p.
    __device__ __forceinline__ int take_split(int L) {
        if (warp == 0) {
            u64 own[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 x = at_rank<C>(
                    reinterpret_cast<const float2*>(&sh.range[(2 * lane + i) % kMine].hi),
                    (2 * lane + i) / kMine);
                own[i] = fix_pair(x.x, x.y);
                sh.range_list[2 * lane + i] = 0;
            }
            set_before(own[0], own[1]);
        }
        sort_list(L);
        return weigh_list(L, round_up32(L));
    }
    // What is kept of the list to the sums ahead, and the draw.
    __device__ __forceinline__ bool draw_kept() {
        if (warp == 0) {
            const double unit = sh.per_one * static_cast<double>(1ull << kFix);
            const u64 x0 = static_cast<u64>(static_cast<double>(sh.range_list[2 * lane]) * unit);
            const u64 x1 = static_cast<u64>(static_cast<double>(sh.range_list[2 * lane + 1]) * unit);
            const u64 more = scan_up64(x0 + x1);
            sh.before[2 * lane + 1] += more - x1;
            sh.before[2 * lane + 2] += more;
        }
        __syncthreads();
        return draw_in_ranges<true>();
    }
    // The leader's piece around min_p's border.
    __device__ __forceinline__ void start_min() {
        if (tid == 0) {
            constexpr float kHalf = 1e-4f;  // of the piece, in units of x c
            const float c = sh.set.c;
            const float at = fmaf(sh.top, c, -static_cast<float>(sh.ref)) +
                             log2f(fminf(static_cast<float>(sh.set.min_p), 1.f));
            sh.x_lo = at - kHalf;
            sh.x_hi = at + kHalf;
            sh.by_min = 1;
        }
    }
    // The largest logit whose exponent is not above x_hi, so that `x > last` holds for exactly
    // the tokens that split() and exact_sums() take as above the piece.  (x_hi + ref) / c, rounded,
    // is off by more than the piece is wide once |x c| is some thousands.
    __device__ float last_below() const {
        const float c = sh.set.c, ref_f = static_cast<float>(sh.ref), hi = sh.x_hi;
        uint32_t a = key_of(Bounds<T>::low), b = key_of(sh.top);  // the largest is above the piece
        while (b - a > 1) {
            const uint32_t mid = a + (b - a) / 2;
            if (fmaf(value_of(mid), c, -ref_f) > hi)
                b = mid;
            else
                a = mid;
        }
        return value_of(a);
    }
    // After its split, in the leader.
    __device__ __forceinline__ Mode draw_min() {
        const int L = sh.n_list;
        if (L > kList) return kExact;
        const int left = take_split(L);
        if (sh.set.p < 1) {  // does the nucleus end first?
            if (tid == 0) {
                const double mass = from_fix(sh.before[kRanges]) +
                                    (left > 0 ? static_cast<double>(sh.sum[left - 1]) * sh.per_one : 0.0);
                const double need = sh.set.p * sh.mass;
                const double e = sh.e_w * (mass + need) + 2.0 * sh.e_a + 1e-9 * sh.mass + 2.0 * kList * sh.per_one;
                sh.count = mass < need - e ? 0 : mass > need + e ? 1 : 2;
            }
            __syncthreads();
            const int which = sh.count;
            __syncthreads();
            if (which == 1) {
                if (tid == 0) sh.by_min = 0;
                start_wide();
                return kWide;
            }
            if (which == 2) return kExact;
        }
        if (tid == 0) {
            sh.kept = left;
            sh.last_end = 0;
            // none of the list is left: those above its first, or above the piece
            if (left == 0) sh.last = L > 0 ? value_of(static_cast<uint32_t>(sh.list[0] >> 32)) : last_below();
        }
        __syncthreads();
        if (again) return kSums;
        keep_list(left);
        return draw_kept() ? kDone : kSums;
    }
    __device__ __forceinline__ bool draw_wide() {
        const Settings& set = sh.set;
        const int L = sh.n_list;
        take_split(L);
        if (again) return false;  // as before
        const double above = from_fix(sh.before[kRanges]);
        if (tid == 0) {
            // before + above against p Z: as for the draw, p in the place of u
            const double Z = sh.mass, p = set.p;
            const double e = sh.e_w * (above * (1.0 - p) + (Z - above) * p) +
                             sh.e_a * fmax(p, 1.0 - p) + 1e-9 * Z + 2.0 * kList * sh.per_one;
            sh.p_lo = (p * Z - above - e) / sh.per_one;
            sh.p_hi = (p * Z - above + e) / sh.per_one;
        }
        __syncthreads();
        const int left = border();
        if (left < 1) return false;
        keep_list(left);
        return draw_kept();
    }

    // ------------------------------------------------------- sums of integer weights
    __device__ __forceinline__ Weights weights_here() const {  // in any CTA
        Weights W;
        W.m = at_rank<C>(&sh.top, 0);
        W.c_hi = sh.set.c;
        W.c_lo = sh.set.c_lo;
        W.S = weight_bits(V);
        W.tab = smem_u32(sh.tab);
        return W;
    }
    // Of each range, to the leader: over all tokens, and over those above the piece (`cut`).
    __device__ __noinline__ void exact_sums(bool cut) {
        const Weights W = weights_here();
        const float c = sh.set.c, ref_f = static_cast<float>(at_rank<C>(&sh.ref, 0));
        const float hi = at_rank<C>(&sh.x_hi, 0);
        u64 all = 0, above = 0;
        stream(
            [&](int, int, const Raw<T>& raw0, const Raw<T>& raw1) {
                float f[16];
                raw0.get(f);
                raw1.get(f + 8);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const u64 w = f[j] > Bounds<T>::low ? W(f[j]) : 0;
                    all += w;
                    if (cut && fmaf(f[j], c, -ref_f) > hi) above += w;
                }
            },
            [&](int r) {
                all = warp_sum64(all);
                above = warp_sum64(above);
                if (lane == 0) {
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(&sh.range_all[r], 0)),
                                 "l"(all)
                                 : "memory");
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(&sh.range_above[r], 0)),
                                 "l"(above)
                                 : "memory");
                }
                all = above = 0;
            });
    }
    // The draw from the sums of each range over the tokens left, sh.range_list.  Returns false if
    // the tokens do not add up to these.
    template <bool CUT>
    __device__ __noinline__ bool draw_exact() {
        const Weights W = weights();
        const float last = sh.last;
        const uint32_t last_end = sh.last_end;
        if (warp == 0) {
            const u64 first = sh.range_list[2 * lane], own = first + sh.range_list[2 * lane + 1];
            const u64 up = scan_up64(own), total = __shfl_sync(0xffffffffu, up, 31);
            const double want = sh.set.u * static_cast<double>(total);
            const u64 target = want < static_cast<double>(total) ? static_cast<u64>(want) : total - 1;
            const uint32_t over = __ballot_sync(0xffffffffu, up > target);
            if (lane == (over ? __ffs(over) - 1 : 31)) {
                const bool second = up - own + first <= target;
                sh.total = total;
                sh.target = target;
                sh.count = 2 * lane + (second ? 1 : 0);
                sh.ahead = up - own + (second ? first : 0);
            }
        }
        __syncthreads();
        const int r = sh.count;
        const int g0 = r * per, g1 = min(G, g0 + per);
        auto left = [&](float x, int v) {
            return x > Bounds<T>::low &&
                   (!CUT || x > last || (x == last && static_cast<uint32_t>(v) < last_end));
        };
        for (int g = g0 + warp; g < g1; g += kWarps) {
            float f[8];
            load(g).get(f);
            u64 sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += left(f[j], g * kGroup + lane * 8 + j) ? W(f[j]) : 0;
            sum = warp_sum64(sum);
            if (lane == 0) sh.gsum[g - g0] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            u64 before = sh.ahead;
            const u64 target = sh.target;
            bool here = false;
            for (int g = g0; g < g1; g += 32) {
                const u64 own = g + lane < g1 ? sh.gsum[g + lane - g0] : 0, up = scan_up64(own);
                const uint32_t over = __ballot_sync(0xffffffffu, before + up > target);
                if (over == 0) {
                    before += __shfl_sync(0xffffffffu, up, 31);
                    continue;
                }
                const int at = __ffs(over) - 1;
                before += __shfl_sync(0xffffffffu, up - own, at);
                g += at;
                float f[8];
                load(g).get(f);
                u64 w[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    w[j] = left(f[j], g * kGroup + lane * 8 + j) ? W(f[j]) : 0;
                    sum += w[j];
                }
                before += scan_up64(sum) - sum;
#pragma unroll 1
                for (int j = 0; j < 8; ++j) {
                    if (before <= target && before + w[j] > target) {
                        write(int64_t(g) * kGroup + lane * 8 + j, f[j],
                              log_of(static_cast<double>(sh.total), W.S));
                        here = true;
                    }
                    before += w[j];
                }
                break;
            }
            here = __any_sync(0xffffffffu, here);
            if (lane == 0) sh.count = here;
        }
        __syncthreads();
        return sh.count != 0;
    }
    // After exact_sums, in the leader.  WAS: what could not be decided.
    __device__ __forceinline__ bool decide_exact(Mode was) {
        const Settings& set = sh.set;
        if (warp == 0) {
            const u64 every = warp_sum64(sh.range_all[2 * lane] + sh.range_all[2 * lane + 1]);
            const u64 above = warp_sum64(sh.range_above[2 * lane] + sh.range_above[2 * lane + 1]);
#pragma unroll
            for (int r = 2 * lane; r < 2 * lane + 2; ++r)
                sh.range_list[r] = was == kWide ? sh.range_above[r] : sh.range_all[r];
            if (lane == 0) {
                sh.log_z = log_of(static_cast<double>(every), weight_bits(V));
                const double need = fmax(ceil(set.p * static_cast<double>(every)), 1.0);
                sh.p_lo = sh.p_hi = was == kWide ? need - static_cast<double>(above) : need;
            }
        }
        __syncthreads();
        if (was == kFew) return draw_few(sh.n_list);
        if (was == kWide) {
            const int left = sh.by_min ? sh.kept : border();
            if (left < 1 && !sh.by_min) return false;
            keep_list(left);
            return draw_exact<true>();
        }
        return draw_exact<false>();
    }
    __device__ __noinline__ bool run_exact(Mode was) {
        exact_sums(was == kWide);
        sync();
        const bool done = rank == 0 && decide_exact(was);
        sync();
        return done;
    }

    // Where one token holds more than half of the mass, its logp is small beside the error of its
    // exponential and of the 8 it was added with: both are taken out of the sum.
    __device__ __forceinline__ void refine() {
        const float top = sh.top;
        for (int g0 = warp * 32; g0 < G; g0 += NT) {
            const uint32_t at = __ballot_sync(0xffffffffu, g0 + lane < G && gmax[g0 + lane] == top);
            if (!at) continue;
            const Raw<T> raw = load(g0 + __ffs(at) - 1);
            float f[8], x[8], w[8];
            raw.get(f);
            weights8(raw, sh.set.c, static_cast<float>(sh.ref), x, w);
            const float t = tree8(w);  // as the pass added them
            const double exact = sh.per_one * sh.one;
            const float hi = static_cast<float>(exact), lo = static_cast<float>(exact - hi);
            Pair s = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                add_to(s, f[j] == top ? hi : w[j]);
                s.lo += f[j] == top ? lo : 0.f;
            }
            float off = (s.hi - t) + s.lo;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) off += __shfl_xor_sync(0xffffffffu, off, o);
            if (lane == 0) sh.log_z = log_of((sh.mass + off) * sh.scale);
        }
        __syncthreads();
    }
    // What follows the pass, in the leader: sh.mode.
    __device__ __forceinline__ void decide() {
        if (warp == 0) combine();
        if (warp == 1) kth_max();
        __syncthreads();
        Mode next = sh.mode;
        if (next != kExact && sh.sure) refine();
        if (next == kFew) {
            const Settings& set = sh.set;
            if (set.k >= V) {
                // where many groups reach the floor, so do many more tokens
                int some = 0;
                for (int g = tid; g < G; g += NT) some += gmax[g] >= sh.floor_x;
                if (block_sum(some) > kList / 4) {
                    set.min_p > 0 ? start_min() : start_wide();
                    next = kWide;
                }
            }
            float at = sh.kth ? value_of(sh.kth) : -INFINITY;
            if (set.k < V && (set.k >= G || at <= Bounds<T>::low) && V > kShort) at = kth_token();
            if (tid == 0) sh.floor_x = fminf(fmaxf(sh.floor_x, at), sh.top);
        } else if (next == kDone) {
            if (again || !draw_in_ranges<false>()) next = kSums;
        }
        __syncthreads();
        if (tid == 0) sh.mode = next;
        __syncthreads();
    }

    // Returns (in the leader) whether the row is drawn, else which kernel it is left to.
    __device__ __forceinline__ int run() {
        pass();
        sync();
        if (rank == 0) decide();
        sync();
        Mode mode = at_rank<C>(&sh.mode, 0), was = kDone;
        if (mode == kFew) {
            gather();
            sync();
            if (rank == 0) {
                const Settings& set = sh.set;
                const int L = sh.n_list;
                Mode next = kExact;
                if (L <= kList) {
                    next = draw_few(L) ? kDone : kSums;
                } else if (set.k >= V) {
                    set.min_p > 0 ? start_min() : start_wide();
                    next = kWide;
                }
                __syncthreads();
                if (tid == 0) {
                    sh.mode = next;
                    // only here: until the barrier ahead, others may still have to read it for L
                    if (next == kWide) sh.n_list = 0;
                }
            }
            sync();
            mode = at_rank<C>(&sh.mode, 0);
            was = kFew;
        }
        if (mode == kWide && at_rank<C>(&sh.by_min, 0)) {
            split();
            sync();
            if (rank == 0) {
                const Mode next = draw_min();
                __syncthreads();
                if (tid == 0) sh.mode = next;
            }
            sync();
            mode = at_rank<C>(&sh.mode, 0);
            was = kWide;
        }
        if (mode == kWide) {
            histogram();
            sync();
            if (rank == 0) find_piece();
            sync();
            split();
            sync();
            if (rank == 0) {
                const bool fits = sh.n_list <= kList && sh.n_list >= 1;
                const Mode next = !fits ? kExact : draw_wide() ? kDone : kSums;
                __syncthreads();
                if (tid == 0) sh.mode = next;
            }
            sync();
            mode = at_rank<C>(&sh.mode, 0);
            was = kWide;
        }
        if constexpr (C > 1) {
            if (mode == kSums) mode = run_exact(was) ? kDone : kExact;
        }
        return mode == kDone ? kDrawn : mode == kSums ? kAgain : kLeft;
    }
};

template <typename T, int C, int NT>
__global__ void __launch_bounds__(NT, C == 1 ? 2 : 3)
    sample_kernel(const SampleArgs a, uint8_t* __restrict__ left, int64_t per, int again) {
    extern __shared__ __align__(16) uint8_t dynamic[];
    __shared__ Shared sh;
    float* maxima = reinterpret_cast<float*>(dynamic + NT / 32 * Row<T, C, NT>::kRing * kGroup * sizeof(T));
    const int64_t G = (a.V + kGroup - 1) / kGroup;
    launch_dependents();
    if (threadIdx.x < 32) fill_table(sh.tab);
    const uint32_t clusters = gridDim.x / C, own = blockIdx.x / C;
    // No CTA touches the leader's shared memory before the leader has started: where SMs still
    // hold blocks of the kernel ahead, that may be long after its own start.
    if constexpr (C > 1) cluster_barrier();
    if (again) wait_for_prerequisites();
    uint32_t seen = 0;
    for (int64_t n0 = 0; n0 < a.N; n0 += kChunk) {
        uint32_t count = 0;
        if (again) {
            count = deal_rows<NT>([&](int64_t n) { return left[n] == kAgain; }, n0, a.N, clusters, own,
                                  seen, sh.deal);
        } else {
            const int64_t in = a.N - n0 < kChunk ? a.N - n0 : kChunk;
            const uint32_t first = (own + clusters - static_cast<uint32_t>(n0 % clusters)) % clusters;
            count = in > first ? (static_cast<uint32_t>(in) - first + clusters - 1) / clusters : 0;
        }
        for (uint32_t i = 0; i < count; ++i) {
            const uint32_t first = (own + clusters - static_cast<uint32_t>(n0 % clusters)) % clusters;
            __syncthreads();
            const int64_t n = n0 + (again ? sh.deal.rows[i] : first + i * clusters);
            const T* row = static_cast<const T*>(a.logits) + n * a.ld;
            __syncthreads();
            if (threadIdx.x == 0) sh.set = settings_of(a, n);
            __syncthreads();
            Row<T, C, NT> r{a, sh, maxima, C == 1 ? maxima : maxima + G, reinterpret_cast<T*>(dynamic),
                            row, n, a.V, static_cast<int>(G), static_cast<int>(per),
                            C == 1 ? 0 : static_cast<int>(cluster_ctarank()),
                            static_cast<int>(threadIdx.x), static_cast<int>(threadIdx.x >> 5),
                            static_cast<int>(threadIdx.x & 31),
                            reinterpret_cast<uintptr_t>(row) % 16 == 0, again != 0};
            const int state = r.run();
            // the second launch keeps what the first wrote as it is: others still look there
            if (r.rank == 0 && threadIdx.x == 0) {
                if (!again) left[n] = static_cast<uint8_t>(state);
                left[a.N + n] = again && state == kLeft;
            }
        }
    }
    if constexpr (C > 1) {  // the others may still read the leader's shared memory
        __syncthreads();
        cluster_barrier();
    }
}

template <typename T, int C, int NT>
cudaError_t run(const SampleArgs& a, uint8_t* left, bool again, const DevInfo& dev, cudaStream_t s) {
    auto kern = sample_kernel<T, C, NT>;
    const int64_t G = (a.V + kGroup - 1) / kGroup, per = (G + kRanges - 1) / kRanges;
    constexpr int kRingBytes = NT / 32 * Row<T, C, NT>::kRing * kGroup * int(sizeof(T));
    static int configured[64] = {0};
    if (!configured[dev.device]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kRingBytes + 2 * (kMaxGroups + kRanges) * 4);
        if (e != cudaSuccess) return e;
        configured[dev.device] = 1;
    }
    const int64_t cap = int64_t(dev.num_sms) * (C == 1 ? 2 : 3) / C;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.N < cap ? a.N : cap) * C));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = kRingBytes + size_t(G + (C == 1 ? 0 : per * (kRanges / C))) * 4;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = again ? 2 : 1;
    note_launches(1);
    return cudaLaunchKernelEx(&cfg, kern, a, left, per, again ? 1 : 0);
}

template <typename T>
cudaError_t run_t(const SampleArgs& a, uint8_t* left, const DevInfo& dev, cudaStream_t s) {
    // Clusters of 8 while all have a place at once (about 50), us uncut, top_k 50, top_p 0.9: 48
    // rows of 32768 20, 26, 53 and 23, 30, 88 by single blocks; 57 35, 42, 83 and 23, 30, 86 (64).
    if (a.N <= dev.num_sms / 3) return run<T, 8, 256>(a, left, false, dev, s);
    const cudaError_t e = run<T, 1, 512>(a, left, false, dev, s);
    return e != cudaSuccess ? e : run<T, 8, 256>(a, left, true, dev, s);
}

}  // namespace

size_t sample_ws_bytes(int64_t N, int64_t V, int dtype) {
    (void)V, (void)dtype;
    return 2 * size_t(N);
}

cudaError_t launch_sample(const SampleArgs& args, void* workspace, const DevInfo& dev, cudaStream_t s) {
    SampleArgs a = args;
    a.cd = kLog2e64 / a.temperature;
    a.c = static_cast<float>(a.cd);
    a.c_lo = static_cast<float>(a.cd - a.c);
    uint8_t* left = static_cast<uint8_t*>(workspace);
    cudaError_t e;
    if ((a.V + kGroup - 1) / kGroup > kMaxGroups) {  // the groups' maxima do not fit
        e = cudaMemsetAsync(left, kLeft, 2 * size_t(a.N), s);
    } else {
        e = a.dtype == LL_F32   ? run_t<float>(a, left, dev, s)
            : a.dtype == LL_F16 ? run_t<__half>(a, left, dev, s)
                                : run_t<__nv_bfloat16>(a, left, dev, s);
    }
    if (e != cudaSuccess) return e;
    return launch_sample_exact(a, left, dev, s);
}

}  // namespace ll
