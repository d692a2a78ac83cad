// Rows that the fast kernel leaves: every weight as an integer, round(2^S w) with
// V 2^S <= 2^62, so that sums are exact in any order, and prefix sums, totals and borders
// agree with each other.
//
// A cluster of 8 CTAs a row, each warp with one run of its groups of 256 logits.  The last
// token left is found by its key, 11 bits a pass: histograms of the tokens and of their mass
// in shared memory, added up in the leader's.  Bound by instructions: a weight takes about 45, so
// that a pass over a row of 151936 is 27 us of one SM's issue, and 8 share it.  48 rows of 151936 to
// the top 1000 290 us, 512 3040; 48 at u = 1 92.
#include "sample_device.cuh"
#include "step_device.cuh"

namespace ll {
namespace {

constexpr int kC = 8;
constexpr int kThreadsX = 512;
constexpr int kWarpsX = kThreadsX / 32;
constexpr int kRuns = kC * kWarpsX;
constexpr int kDigit = 11;
constexpr int kBinsX = 1 << kDigit;
constexpr int kGroupX = 256;

struct Hist {
    u64 mass[kBinsX];
    uint32_t count[kBinsX];
};
struct SharedX {
    Hist own, all;  // all: the leader's
    Settings set;
    WeightStep tab[32];
    float m;  // the row's largest
    uint32_t floor_key;
    // the leader's
    u64 run_sum[kRuns];
    uint32_t run_ties[kRuns];
    u64 every;
    uint32_t top;
    // of the digits found so far: their value, and what lies above
    uint32_t prefix, above_count, done;
    u64 above_mass;
    // the tokens left: keys above `last`, and the first n_last of key `last`
    uint32_t last, n_last;
    // the draw
    u64 before, target, total;
    uint32_t ties_before;
    int run;
    u64 group_sum[kWarpsX], warp_count[kWarpsX];
    uint32_t group_ties[kWarpsX];
    Deal deal;
};

__device__ __forceinline__ uint32_t ld_leader(const uint32_t* x) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(x, 0)) : "memory");
    return v;
}
__device__ __forceinline__ u64 ld_leader(const u64* x) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr(x, 0)) : "memory");
    return v;
}
__device__ __forceinline__ void add_leader(uint32_t* x, uint32_t v) {
    asm volatile("red.shared::cluster.add.u32 [%0], %1;" ::"r"(cluster_addr(x, 0)), "r"(v) : "memory");
}
__device__ __forceinline__ void add_leader(u64* x, u64 v) {
    asm volatile("red.shared::cluster.add.u64 [%0], %1;" ::"r"(cluster_addr(x, 0)), "l"(v) : "memory");
}
__device__ __forceinline__ void max_leader(uint32_t* x, uint32_t v) {
    asm volatile("red.shared::cluster.max.u32 [%0], %1;" ::"r"(cluster_addr(x, 0)), "r"(v) : "memory");
}
__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <typename T>
struct RowX {
    const SampleArgs& a;
    SharedX& sh;
    const T* row;
    int64_t n, V, G, per;
    int rank, tid, warp, lane;
    bool vec;
    // At temperatures above 2^60 logits are taken as 2^-64 of themselves, and c as 2^64 of itself: the
    // distance of two logits that weighs something may not fit FP32, nor c
    float part;
    Weights W;
    u64 least;
    // u of 1 or more takes the last token left, also where its weight is no whole unit: tokens
    // then count 1 each, min_p leaving those from floor_key on
    bool by_count;
    uint32_t floor_key;

    __device__ __forceinline__ void sync() const {
        __syncthreads();
        __syncwarp();  // the cluster's barrier wants whole warps: lanes come from ways of their own
        cluster_barrier();
    }
    __device__ __forceinline__ void load(int64_t g, float (&f)[8]) const {
        const int64_t v = g * kGroupX + lane * 8;
        if (vec && (g + 1) * kGroupX <= V) {
            load8(row + v, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = v + j < V ? Elem<T>::to_f(row[v + j]) : -INFINITY;
        }
    }
    // each(f) for the groups of this warp's run in turn, four loads in flight
    template <class F>
    __device__ __forceinline__ void stream(F each) const {
        const int64_t g0 = (rank * kWarpsX + warp) * per, g1 = min(G, g0 + per);
        constexpr int kUnroll = sizeof(T) == 2 ? 4 : 2;
        for (int64_t g = g0; g < g1;) {
            if (vec && g + kUnroll <= g1 && (g + kUnroll) * kGroupX <= V) {
                uint4 raw[kUnroll][sizeof(T) / 2];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i)
#pragma unroll
                    for (int k = 0; k < int(sizeof(T)) / 2; ++k)
                        raw[i][k] = reinterpret_cast<const uint4*>(row + (g + i) * kGroupX + lane * 8)[k];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    float f[8];
                    const T* e = reinterpret_cast<const T*>(raw[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = Elem<T>::to_f(e[j]);
                    each(f);
                }
                g += kUnroll;
            } else {
                float f[8];
                load(g, f);
                each(f);
                ++g;
            }
        }
    }

    // The key of the last of the first `need` tokens (BY_MASS: of the first tokens whose mass
    // reaches `need`), with what lies above it: sh.prefix, above_*.  False: there are fewer.
    template <bool BY_MASS>
    __device__ __forceinline__ bool select(u64 need) {
        uint32_t prefix = 0, above_c = 0;
        u64 above_m = 0;
        for (int bits = 32; bits > 0;) {
            const int shift = bits > kDigit ? bits - kDigit : 0;
            for (int i = tid; i < kBinsX; i += kThreadsX) {
                sh.own.mass[i] = sh.all.mass[i] = 0;
                sh.own.count[i] = sh.all.count[i] = 0;
            }
            sync();
            stream([&](const float (&f)[8]) {
#pragma unroll 4
                for (int j = 0; j < 8; ++j) {
                    const uint32_t key = key_of(f[j]);
                    if (key && (bits == 32 || key >> bits == prefix)) {
                        const uint32_t bin = (key >> shift) & ((1u << (bits - shift)) - 1);
                        atomicAdd(&sh.own.count[bin], 1u);
                        atomicAdd(&sh.own.mass[bin], weight(f[j]));
                    }
                }
            });
            __syncthreads();
            for (int i = tid; i < kBinsX; i += kThreadsX)
                if (sh.own.count[i]) {
                    add_leader(&sh.all.count[i], sh.own.count[i]);
                    add_leader(&sh.all.mass[i], sh.own.mass[i]);
                }
            sync();
            if (rank == 0) {
                // the highest bin with which the sum from above reaches the need: a thread has 4
                constexpr int kEach = kBinsX / kThreadsX;
                const int top_bin = kBinsX - 1 - tid * kEach;
                u64 c = 0, m = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    c += sh.all.count[top_bin - i];
                    m += sh.all.mass[top_bin - i];
                }
                u64 cs = c, ms = m;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const u64 x = __shfl_up_sync(0xffffffffu, cs, o);
                    const u64 y = __shfl_up_sync(0xffffffffu, ms, o);
                    if (lane >= o) {
                        cs += x;
                        ms += y;
                    }
                }
                if (tid == 0) sh.done = 1;
                if (lane == 31) {
                    sh.warp_count[warp] = cs;
                    sh.group_sum[warp] = ms;
                }
                __syncthreads();
                cs += above_c - c;  // ahead of this thread
                ms += above_m - m;
                for (int w = 0; w < warp; ++w) {
                    cs += sh.warp_count[w];
                    ms += sh.group_sum[w];
                }
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const u64 ci = sh.all.count[top_bin - i], mi = sh.all.mass[top_bin - i];
                    const u64 have = BY_MASS ? ms : cs, more = BY_MASS ? mi : ci;
                    if (have < need && have + more >= need) {
                        sh.done = 0;
                        sh.prefix = (prefix << (bits - shift)) | static_cast<uint32_t>(top_bin - i);
                        sh.above_count = static_cast<uint32_t>(cs);
                        sh.above_mass = ms;
                    }
                    cs += ci;
                    ms += mi;
                }
            }
            sync();
            if (ld_leader(&sh.done)) return false;
            prefix = ld_leader(&sh.prefix);
            above_c = ld_leader(&sh.above_count);
            above_m = ld_leader(&sh.above_mass);
            bits = shift;
        }
        return true;
    }

    __device__ __forceinline__ u64 weight(float x) const { return W(x * part); }
    // Weight of the token if it is left, equal ones counted apart.
    __device__ __forceinline__ u64 above_last(float x, uint32_t last, uint32_t& ties) const {
        const uint32_t key = key_of(x);
        ties += key == last;
        if (key <= last) return 0;
        if (by_count) return key >= floor_key ? 1 : 0;
        const u64 w = weight(x);
        return w >= least ? w : 0;
    }
    // The key of the lowest logit that min_p leaves: x - max compared in FP64.
    __device__ uint32_t lowest_left(float m) const {
        const Settings& set = sh.set;
        uint32_t b = key_of(m);
        if (!(m < INFINITY)) return b;
        if (!(set.min_p > 0 && set.T < INFINITY)) return 1u;
        const double floor_d = set.T * log(fmin(set.min_p, 1.0));
        for (uint32_t a = 0; b - a > 1;) {
            const uint32_t mid = a + (b - a) / 2;
            if (static_cast<double>(value_of(mid)) - m >= floor_d)
                b = mid;
            else
                a = mid;
        }
        return b;
    }
    // Sums over the tokens left, or how many, a run of groups each, to the leader.
    template <bool COUNT>
    __device__ __forceinline__ void sum_left(uint32_t last, uint32_t to_sum, uint32_t to_ties) const {
        uint32_t ties = 0, some = 0;
        u64 sum = 0;
        const uint32_t lowest = max(last + 1, floor_key);
        stream([&](const float (&f)[8]) {
#pragma unroll 4
            for (int j = 0; j < 8; ++j) {
                if constexpr (COUNT) {
                    const uint32_t key = key_of(f[j]);
                    some += key >= lowest;
                    ties += key == last;
                } else {
                    sum += above_last(f[j], last, ties);
                }
            }
        });
        sum = warp_sum64(COUNT ? some : sum);
        ties = __reduce_add_sync(0xffffffffu, last ? ties : 0u);
        if (lane == 0) {
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to_sum), "l"(sum) : "memory");
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to_ties), "r"(ties) : "memory");
        }
        sync();
    }

    __device__ __forceinline__ void run() {
        const Settings& set = sh.set;
        if (tid == 0) {
            sh.top = 0;
            sh.every = 0;
        }
        sync();
        uint32_t key = 0;
        stream([&](const float (&f)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) key = max(key, key_of(f[j]));
        });
        key = __reduce_max_sync(0xffffffffu, key);
        if (lane == 0) max_leader(&sh.top, key);
        sync();
        const uint32_t top = ld_leader(&sh.top);
        if (top == 0) {
            if (rank == 0 && tid == 0) {
                a.tokens[n] = -1;
                a.logp[n] = a.logq[n] = 0.f;
            }
            return;
        }
        const float m = value_of(top);
        if (tid == 0) sh.m = m;
        W.c_hi = set.c;
        W.c_lo = set.c_lo;
        part = 1.f;
        if (set.cd < 0x1p-60) {
            const double c = set.cd * 0x1p64;
            W.c_hi = static_cast<float>(c);
            W.c_lo = static_cast<float>(c - W.c_hi);
            part = 0x1p-64f;
        }
        W.m = m * part;
        W.S = weight_bits(V);
        W.tab = smem_u32(sh.tab);
        u64 sum = 0;
        stream([&](const float (&f)[8]) {
#pragma unroll 4
            for (int j = 0; j < 8; ++j)
                if (key_of(f[j])) sum += weight(f[j]);
        });
        sum = warp_sum64(sum);
        const int own_run = rank * kWarpsX + warp;
        const uint32_t to_sum = cluster_addr(&sh.run_sum[own_run], 0);
        const uint32_t to_ties = cluster_addr(&sh.run_ties[own_run], 0);
        if (lane == 0) {
            add_leader(&sh.every, sum);
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to_sum), "l"(sum) : "memory");
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to_ties), "r"(0u) : "memory");
        }
        sync();
        const u64 every = ld_leader(&sh.every);
        uint32_t last = 0, n_last = 0;
        u64 mass = every;
        if (set.k < V && select<false>(static_cast<u64>(set.k))) {
            last = ld_leader(&sh.prefix);
            n_last = static_cast<uint32_t>(set.k) - ld_leader(&sh.above_count);
            mass = ld_leader(&sh.above_mass) + weight(value_of(last)) * n_last;
            sync();
        }
        if (set.p < 1) {
            const u64 need = static_cast<u64>(fmax(ceil(set.p * static_cast<double>(mass)), 1.0));
            if (select<true>(need)) {
                const uint32_t at = ld_leader(&sh.prefix);
                const u64 w = weight(value_of(at));
                const uint32_t some =
                    w ? static_cast<uint32_t>((need - ld_leader(&sh.above_mass) + w - 1) / w) : 1u;
                if (at > last || (at == last && some < n_last)) {
                    last = at;
                    n_last = some;
                }
                sync();
            }
        }
        least = 0;
        if (set.min_p > 0)
            least = static_cast<u64>(ceil(fmin(set.min_p, 1.0) * static_cast<double>(1ull << W.S)));
        const u64 w_last = last ? weight(value_of(last)) : 0;
        u64 w_tie = w_last >= least ? w_last : 0;
        if (last || least) sum_left<false>(last, to_sum, to_ties);
        if (set.u >= 1) {
            if (tid == 0) sh.floor_key = lowest_left(sh.m);
            if (rank == 0) find_run(n_last, w_tie);  // their mass
            sync();
            by_count = true;
            floor_key = sh.floor_key;
            w_tie = last && last >= floor_key ? 1 : 0;
            sum_left<true>(last, to_sum, to_ties);
        }
        if (rank == 0) draw(every, last, n_last, w_tie);
        sync();
    }

    // The leader: the run that the target lies in.
    __device__ __forceinline__ void find_run(uint32_t n_last, u64 w_tie) {
        const Settings& set = sh.set;
        if (warp == 0) {  // a lane: 4 runs
            constexpr int kEach = kRuns / 32;
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) t += sh.run_ties[lane * kEach + i];
            uint32_t ts = t;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, ts, o);
                if (lane >= o) ts += x;
            }
            t = ts - t;  // ahead of this lane
            u64 own[kEach];
            uint32_t ahead[kEach];
            u64 sum = 0;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint32_t k = sh.run_ties[lane * kEach + i];
                own[i] = sh.run_sum[lane * kEach + i] + w_tie * min(k, n_last - min(t, n_last));
                ahead[i] = t;
                t += k;
                sum += own[i];
            }
            u64 up = sum;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const u64 x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            const u64 total = __shfl_sync(0xffffffffu, up, 31);
            const double want = set.u * static_cast<double>(total);
            const u64 target = set.u < 1 && want < static_cast<double>(total) ? static_cast<u64>(want)
                                                                              : total - 1;
            u64 at = up - sum;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (at <= target && at + own[i] > target) {
                    sh.run = lane * kEach + i;
                    sh.before = at;
                    sh.ties_before = ahead[i];
                    sh.target = target;
                    if (!by_count) sh.total = total;
                }
                at += own[i];
            }
        }
    }
    // The leader: the run, the group and the token that the target lies in.
    __device__ __forceinline__ void draw(u64 every, uint32_t last, uint32_t n_last, u64 w_tie) {
        const Settings& set = sh.set;
        find_run(n_last, w_tie);
        __syncthreads();
        const u64 target = sh.target;
        u64 before = sh.before;
        uint32_t t0 = sh.ties_before;
        const int64_t g0 = sh.run * per, g1 = min(G, g0 + per);
        for (int64_t gb = g0; gb < g1; gb += kWarpsX) {  // a group a warp
            const int64_t g = gb + warp;
            u64 sum = 0;
            uint32_t ties = 0;
            float f[8];
            if (g < g1) {
                load(g, f);
#pragma unroll 1
                for (int j = 0; j < 8; ++j) sum += above_last(f[j], last, ties);
                if (!last) ties = 0;
            }
            const u64 lane_sum = sum;
            const uint32_t lane_ties = ties;
            sum = warp_sum64(sum);
            ties = __reduce_add_sync(0xffffffffu, ties);
            __syncthreads();
            if (lane == 0) {
                sh.group_sum[warp] = sum;
                sh.group_ties[warp] = ties;
            }
            __syncthreads();
            int w = 0;
            for (; w < kWarpsX; ++w) {
                const uint32_t some = min(sh.group_ties[w], n_last - min(t0, n_last));
                const u64 next = before + sh.group_sum[w] + w_tie * some;
                if (next > target) break;
                before = next;
                t0 += sh.group_ties[w];
            }
            if (w == kWarpsX) continue;
            if (w != warp) return;
            // this warp's group: its lanes in turn, then the lane's logits
            u64 at = before;
            uint32_t t = t0;
            for (int l = 0; l < 32; ++l) {
                const u64 s = __shfl_sync(0xffffffffu, lane_sum, l);
                const uint32_t k = __shfl_sync(0xffffffffu, lane_ties, l);
                const u64 next = at + s + w_tie * min(k, n_last - min(t, n_last));
                if (next > target) {
                    if (lane != l) return;
                    break;
                }
                at = next;
                t += k;
            }
            for (int j = 0; j < 8; ++j) {
                uint32_t tie = 0;
                u64 s = above_last(f[j], last, tie);
                if (tie && last && t < n_last) s = w_tie;
                t += last ? tie : 0;
                at += s;
                if (at > target) {
                    const float x = f[j];
                    const double z = x == sh.m ? 0.0 : (static_cast<double>(x) - sh.m) / set.T;
                    const double one = static_cast<double>(1ull << W.S);
                    a.tokens[n] = g * kGroupX + lane * 8 + j;
                    a.logp[n] = static_cast<float>(z - log(static_cast<double>(every) / one));
                    a.logq[n] = static_cast<float>(z - log(static_cast<double>(sh.total) / one));
                    return;
                }
            }
            return;
        }
    }
};

template <typename T>
__global__ void __cluster_dims__(kC, 1, 1) __launch_bounds__(kThreadsX, 2)
    exact_kernel(const SampleArgs a, const uint8_t* __restrict__ left, int64_t per) {
    extern __shared__ uint8_t raw[];
    SharedX& sh = *reinterpret_cast<SharedX*>(raw);
    const int tid = threadIdx.x;
    if (tid < 32) fill_table(sh.tab);
    const int rank = static_cast<int>(cluster_ctarank());
    wait_for_prerequisites();
    // the rows that are left, dealt to the clusters in turn
    const uint32_t clusters = gridDim.x / kC, own = blockIdx.x / kC;
    uint32_t seen = 0;
    for (int64_t n0 = 0; n0 < a.N; n0 += kChunk) {
        const uint32_t count =
            deal_rows<kThreadsX>([&](int64_t n) { return left[n] == kLeft || left[a.N + n] == kLeft; }, n0,
                                 a.N, clusters, own, seen, sh.deal);
        for (uint32_t i = 0; i < count; ++i) {
            __syncthreads();
            const int64_t n = n0 + sh.deal.rows[i];
            if (tid == 0) sh.set = settings_of(a, n);
            const T* row = static_cast<const T*>(a.logits) + n * a.ld;
            RowX<T> r{a, sh, row, n, a.V, (a.V + kGroupX - 1) / kGroupX, per, rank, tid, tid >> 5, tid & 31,
                      reinterpret_cast<uintptr_t>(row) % 16 == 0, 1.f, {}, 0, false, 0};
            r.run();
        }
    }
    __syncthreads();  // no CTA leaves while another may read its shared memory
    cluster_barrier();
}

template <typename T>
cudaError_t run(const SampleArgs& a, const uint8_t* left, const DevInfo& dev, cudaStream_t s) {
    auto kern = exact_kernel<T>;
    static int configured[64] = {0};
    if (!configured[dev.device]) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   int(sizeof(SharedX)));
        if (e != cudaSuccess) return e;
        configured[dev.device] = 1;
    }
    const int64_t G = (a.V + kGroupX - 1) / kGroupX, per = (G + kRuns - 1) / kRuns;
    const int64_t cap = 2 * dev.num_sms / kC;
    note_launches(1);
    return launch_after(kern, unsigned((a.N < cap ? a.N : cap) * kC), kThreadsX, s,
                        unsigned(sizeof(SharedX)), a, left, per);
}

}  // namespace

cudaError_t launch_sample_exact(const SampleArgs& a, const uint8_t* left, const DevInfo& dev,
                                cudaStream_t s) {
    if (a.dtype == LL_F32) return run<float>(a, left, dev, s);
    if (a.dtype == LL_F16) return run<__half>(a, left, dev, s);
    return run<__nv_bfloat16>(a, left, dev, s);
}

}  // namespace ll
