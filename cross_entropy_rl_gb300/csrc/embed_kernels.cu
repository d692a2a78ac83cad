// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[n, :] = scale * W[y_n - v0, :]  (+0 rows for other tokens)
//   backward  dW[v, :] (+)= scale * sum_{n: y_n - v0 = v} g[n, :]
#include <atomic>
#include <type_traits>

#include "step_device.cuh"

namespace ll {
namespace {

// ------------------------------------------------------------------- lookup
// One multiply per element: bound by HBM (a row read, a row written).  A warp
// takes one row's tile of 32 U chunks of E elements; all its loads are issued
// before the first store.  Rows of the output's type with a scale of 1 are copied
// (COPY).  32768 x 4096 bf16 of 151936 rows: 58 us, 0.94 of the copy bandwidth
// (scaled 60, U = 2 60, U = 8 67 us).  Rows that do not start on 16-byte boundaries
// go element by element, U = 16 of them in flight a lane: 10007 x 1001 FP32 to
// FP16 8.7 us (U = 4: 12.6, 8: 9.3).
constexpr int kLookupWarps = 8;

template <typename TI, typename TO, int E, int U, bool COPY>
__global__ void __launch_bounds__(32 * kLookupWarps) embed_fwd_kernel(
    const TI* __restrict__ W, int64_t ldw, const int64_t* __restrict__ tokens, int64_t N,
    int64_t D, int64_t V, int64_t v0, float scale, TO* __restrict__ out, int64_t ldo) {
    const int lane = threadIdx.x & 31;
    const int64_t n = blockIdx.x * int64_t(kLookupWarps) + (threadIdx.x >> 5);
    if (n >= N) return;
    const int64_t v = tokens[n] - v0;
    const bool in = v >= 0 && v < V;
    const TI* src = W + (in ? v : 0) * ldw;
    TO* dst = out + n * ldo;
    const int64_t chunks = (D + E - 1) / E;
    for (int64_t c0 = int64_t(blockIdx.y) * (32 * U) + lane; c0 < chunks;
         c0 += int64_t(gridDim.y) * (32 * U)) {
        Pack<TI, E> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = (c0 + 32 * u) * E;
            if (in && c + E <= D) x[u].load(src + c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = (c0 + 32 * u) * E;
            if (c + E <= D) {
                Pack<TO, E> y;
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    if constexpr (COPY)
                        y.e[j] = in ? x[u].e[j] : Elem<TO>::from_f(0.f);
                    else
                        y.e[j] = Elem<TO>::from_f(in ? Elem<TI>::to_f(x[u].e[j]) * scale : 0.f);
                }
                y.store(dst + c);
            } else {
                for (int64_t i = c; i < D; ++i)
                    dst[i] = Elem<TO>::from_f(in ? Elem<TI>::to_f(src[i]) * scale : 0.f);
            }
        }
    }
}

template <typename TI, typename TO>
cudaError_t fwd_typed(const EmbedArgs& a, bool vec, cudaStream_t s) {
    constexpr int E = 16 / (sizeof(TI) < sizeof(TO) ? sizeof(TI) : sizeof(TO));
    const int64_t chunks = vec ? (a.D + E - 1) / E : a.D;
    constexpr int U = 4, U1 = 16;
    const int tile = 32 * (vec ? U : U1);
    const int64_t tiles = (chunks + tile - 1) / tile;
    const dim3 grid(static_cast<unsigned>((a.N + kLookupWarps - 1) / kLookupWarps),
                    static_cast<unsigned>(tiles < 65535 ? tiles : 65535));
    const TI* W = static_cast<const TI*>(a.rows);
    TO* out = static_cast<TO*>(a.table);
    auto run = [&](auto* kernel) {
        kernel<<<grid, 32 * kLookupWarps, 0, s>>>(W, a.ld_rows, a.tokens, a.N, a.D, a.V, a.v0,
                                                  a.scale, out, a.ld_table);
        return cudaGetLastError();
    };
    if (!vec) return run(embed_fwd_kernel<TI, TO, 1, U1, false>);
    constexpr bool kSame = std::is_same_v<TI, TO>;
    return kSame && a.scale == 1.f ? run(embed_fwd_kernel<TI, TO, E, U, kSame>)
                                   : run(embed_fwd_kernel<TI, TO, E, U, false>);
}

bool rows16(const void* p, int64_t ld, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && size_t(ld) * es % 16 == 0;
}

// ----------------------------------------------------------------- gradient
// Few tokens are matched in one launch (embed_match_kernel).  Others take three
// launches.  The first sorts the tokens (one cluster), the second adds up
// the rows of grad_out in the sorted order, the third finishes long tokens.
//
// A unit is at most K sorted positions of one token: a token's occurrences are
// cut every K from its first, so the order of its additions is a function of
// its own occurrences (and of K).  The row of a token of one unit is finished
// by the warp that adds it; the pieces of a longer one are written as FP32
// partial sums, which a block then adds in order.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;         // CTAs of the sorting cluster for many tokens
constexpr int kDigitBits = 9;        // most bits of a sorting pass
constexpr int kBins = 1 << kDigitBits;
constexpr int kStaged = 4096;        // keys a CTA holds in shared memory
// Most tokens that one CTA sorts (the sort with nothing to add up: 2048 tokens 12.0
// us, by the cluster 13.5; 4096 tokens 15.8, by the cluster 14.0).
constexpr int64_t kOneCta = 2048;
// Most tokens that are matched in one launch instead of sorted.  BF16 added into FP32,
// matched and sorted: 64 x 4096 3.8 and 10.9 us, 300 x 512 5.6 and 13.2, 1024 x 1024 9.0
// and 15.4, 1024 x 4096 16.7 and 16.6; with 0.7 of them one token 14.3 and 17.9.  Of 2048
// the width decides: 2048 x 256 12.3 and 18.1, but 2048 x 4096 36.8 and 21.4, and with a
// hot token 30.4 and 20.9.
constexpr int kMatch = 1024;
constexpr int kWarpStaged = kStaged / kSortWarps;
constexpr int kRounds = 4;           // rounds of 32 keys of a warp at a time
constexpr int kFillCtas = 256;       // CTAs in all when rows are filled beside the sort
constexpr int kFillBytes = 65536;    // of a block that fills rows beside the sums, about
// vocabulary rows of one bitmap, which takes the place of the counts
constexpr int kFillRows = kSortWarps * kBins * 32;
constexpr int64_t kShort = 8192;     // most tokens of the finer division below
constexpr int kPiece = 16;           // rows of a piece there
constexpr int kFewPieces = 8;        // pieces of a token that one warp adds up
constexpr int kGradWarps = 8;
constexpr int kGradRows = 4;         // rows in flight of a warp of the sums

// Shared memory of the sort: counts, keys, the digits' words (the second buffer
// of the keys, empty as they are counted, where one CTA sorts alone), places of
// the keys among their equals.
constexpr int kSortSmem = kSortWarps * kBins * 8 + kStaged * 8 + kStaged * 2;
static_assert(kStaged * 8 == kSortWarps * kBins * 4, "the words fill a buffer of keys");

// Sorted positions of a warp of the sums, in whole units, and of a piece.  Few
// tokens are bound by the rows that a warp adds one after another, many by the
// work per warp: 4096 x 2048 took 44 us with 8 and 16 and 54 us with 16 and 32,
// 32768 x 4096 152 and 141 us.  Pieces grow so that at most 2048 of their partial
// sums are kept.
__host__ __device__ inline int window_rows(int64_t N) { return N <= kShort ? 8 : 16; }
__host__ __device__ inline int64_t piece_rows(int64_t N) {
    int64_t k = N <= kShort ? kPiece : 32;
    while ((N + k - 1) / k > 2048) k *= 2;
    return k;
}

// An entry of the sorted order: the position in the batch and the table's row.
// The top bits are set in the last entry of a unit: kEnd, and kLong if the
// token has other units.
struct Entry {
    unsigned pos, row;
};
constexpr unsigned kTop = 1u << 31;

// A token of several units: its first sorted position, its occurrences, its row.
struct Long {
    int start, count, row, pad;
};

struct SortHead {
    int valid;         // tokens of the table: entries
    int longs, huges;  // tokens of 2 .. kFewPieces units, of more
};

struct SortPtrs {
    SortHead* head;
    // of more tokens than a cluster sorts
    unsigned long long *buf0, *buf1;  // [N] keys
    int *counts, *totals;             // [kBins, blocks of kStaged], [kBins]
    uint16_t* places;                 // [N]
    Entry* entries;                   // [N]
    int* windows;                     // [ceil(N / window) + 1] start of the unit of each
                                      // window-th entry
    Long* longs;                      // [ceil(N / K)], in any order: the longs from the
                                      // front on, the huges from the back
    unsigned* used;                   // [ceil(V / 32)] rows that are not to be filled any more
    float* part;                      // [2 ceil(N / K), Dp] sums of pieces
    int64_t Dp;
};

struct SortArgs {
    const int64_t* tokens;
    int64_t N, V, v0;
    int bits, passes;  // of a row index; sorting passes
    int K, window, slots;
    SortPtrs p;
    // rows of no token are set to +0 (accumulate = 0), else null
    char* table;
    int64_t row_bytes, pitch;
    float now;  // share of the rows that is filled beside the sort
    bool mark;  // the sort itself marks the rows of tokens as used
};

extern __shared__ __align__(16) unsigned char sort_smem[];

__device__ __forceinline__ int ld_cluster(const int* local, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(local, rank)));
    return v;
}

__device__ __forceinline__ unsigned long long ld_cluster64(const void* local, uint32_t rank) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr(local, rank)));
    return v;
}
__device__ __forceinline__ void st_cluster64(void* local, uint32_t rank, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_addr(local, rank)), "l"(v)
                 : "memory");
}

__device__ __forceinline__ uint32_t cluster_ctas() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

// Exclusive sum over the lanes of a warp.
__device__ __forceinline__ int warp_scan(int x, int lane) {
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    return s - x;
}

typedef unsigned long long Key;  // row << 32 | position
constexpr Key kNone = ~0ull;     // no token of the table

__device__ __forceinline__ Key key_of(const SortArgs& a, int64_t i, int64_t y) {
    const int64_t v = y - a.v0;
    if (y < a.v0 || v >= a.V) return kNone;
    return static_cast<Key>(v) << 32 | static_cast<unsigned>(i);
}

// Digits of a sorting pass: `bins` values from bit `shift` of the row on.
struct Digits {
    int shift, bins;
    __device__ __forceinline__ Digits(const SortArgs& a, int pass) : shift(0) {
        for (int p = 0;; ++p) {
            const int bits = (a.bits - shift + (a.passes - p) - 1) / (a.passes - p);
            bins = 1 << bits;
            if (p == pass) break;
            shift += bits;
        }
    }
    __device__ __forceinline__ int of(Key k) const {
        return k == kNone ? -1 : static_cast<int>(k >> (32 + shift)) & (bins - 1);
    }
};

// Counts a warp's keys by digit.  The lanes of equal digit find each other by
// setting their bits in the digit's word of the warp (a vote for each bit of the
// digit took 4x the time, match.any more), and one of them counts for all.
struct WarpCounts {
    int* count;      // [bins]
    unsigned* word;  // [bins], 0 between the calls
    // A key's place among the warp's keys of its digit so far (d = -1: no key).
    __device__ __forceinline__ int add(int d) {
        const int lane = threadIdx.x & 31;
        const unsigned under = (1u << lane) - 1;
        if (d >= 0) atomicOr(word + d, 1u << lane);
        __syncwarp();
        const unsigned peers = d >= 0 ? word[d] : 0;
        const int had = d >= 0 ? count[d] : 0;
        __syncwarp();
        if (d >= 0 && (peers & under) == 0) {
            count[d] = had + __popc(peers);
            word[d] = 0;
        }
        __syncwarp();
        return had + __popc(peers & under);
    }
};

// counts [kSortWarps][bins]: each warp's become those of the warps below it; the
// sum over the warps of thread tid's digit comes back.
__device__ __forceinline__ int sum_over_warps(int* counts, int bins) {
    int sum = 0;
    if (threadIdx.x >= bins) return 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const int c = counts[w * bins + threadIdx.x];
        counts[w * bins + threadIdx.x] = sum;
        sum += c;
    }
    return sum;
}

// Exclusive sum of x over the block's threads; `all` is the sum of all.
__device__ __forceinline__ int block_scan(int x, int& all) {
    __shared__ int scan[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int low = warp_scan(x, lane);
    __syncthreads();
    if (lane == 31) scan[warp] = low + x;
    __syncthreads();
    int under = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        if (w < warp) under += scan[w];
        all += scan[w];
    }
    return under + low;
}

// The sorted keys [beg, end) of a warp: heads[r] are the lanes that start a token
// in round r of the block at i (the lane's first).  `prev` is the row ahead of the
// block, and then its last row.
__device__ __forceinline__ void heads_of(const Key (&k)[kRounds], int64_t i, int64_t end,
                                         unsigned& prev, unsigned (&heads)[kRounds]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const unsigned row = static_cast<unsigned>(k[r] >> 32);
        const unsigned up = __shfl_up_sync(0xffffffffu, row, 1);
        const bool differs = row != (lane == 0 ? prev : up);
        heads[r] = __ballot_sync(0xffffffffu, i + r * 32 < end && differs);
        prev = __shfl_sync(0xffffffffu, row, 31);
    }
}

// Entries of the sorted keys [beg, end) of a warp, with their units' ends.
// `head` is where the token that the run starts inside started (any value if it
// starts with one), before and after the rows next to the run (~0: none).
// block(i, k) gives kRounds rounds of keys, kNone from `end` on; key_at(i) one.
template <typename B, typename K>
__device__ __forceinline__ void write_entries(const SortArgs& a, int64_t beg, int64_t end, int head,
                                              unsigned before, unsigned after, const B& block,
                                              const K& key_at) {
    const int lane = threadIdx.x & 31;
    const unsigned upto = ~0u >> (31 - lane);  // lanes up to this one
    const int mask = a.K - 1;                  // K is a power of two
#pragma unroll 1
    for (int64_t i0 = beg + lane; i0 - lane < end; i0 += 32 * kRounds) {
        Key k[kRounds];
        unsigned heads[kRounds];
        block(i0, k);
        heads_of(k, i0, end, before, heads);
        const int64_t i1 = i0 - lane + 32 * kRounds;
        unsigned beyond = after;  // the row after the block
        if (i1 < end) beyond = static_cast<unsigned>(key_at(i1) >> 32);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = static_cast<int>(i0) + r * 32, b = i - lane;
            const unsigned row = static_cast<unsigned>(k[r] >> 32);
            const unsigned down = __shfl_down_sync(0xffffffffu, row, 1);
            const unsigned up = static_cast<unsigned>(k[(r + 1) % kRounds] >> 32);
            const unsigned first = r + 1 < kRounds ? __shfl_sync(0xffffffffu, up, 0) : beyond;
            const unsigned seen = heads[r] & upto;
            const int h = seen ? b + 31 - __clz(seen) : head;
            if (i < end) {
                const unsigned next = i + 1 == end ? after : lane == 31 ? first : down;
                const int in = (i - h) & mask;  // place in its unit
                const bool token_ends = row != next;
                const bool unit_ends = token_ends || in == mask;
                const bool more = unit_ends && (i - h >= a.K || !token_ends);
                a.p.entries[i] = Entry{static_cast<unsigned>(k[r]) | (unit_ends ? kTop : 0u),
                                       row | (more ? kTop : 0u)};
                if (i % a.window == 0) a.p.windows[i / a.window] = i - in;
                if (a.mark && token_ends) atomicOr(a.p.used + row / 32, 1u << row % 32);
                if (token_ends && i - h >= a.K) {
                    const bool huge = i - h >= a.K * kFewPieces;
                    const int at = atomicAdd(huge ? &a.p.head->huges : &a.p.head->longs, 1);
                    a.p.longs[huge ? a.slots - 1 - at : at] =
                        Long{h, i + 1 - h, static_cast<int>(row), 0};
                }
            }
            if (heads[r]) head = b + 31 - __clz(heads[r]);
        }
    }
}

__device__ __forceinline__ void write_head(const SortArgs& a, int64_t M) {
    a.p.head->valid = static_cast<int>(M);
    a.p.windows[(M + a.window - 1) / a.window] = static_cast<int>(M);
}

// Least-significant-digit radix sort by one CTA or one cluster, stable, so that
// the positions of a token stay ascending.  Each warp owns a run of the keys; a
// pass counts the run's digits, scans the counts over warps, CTAs and digits,
// and writes each key to its place.  Tokens outside the table drop out in the
// first pass.  The keys stay in shared memory: a CTA's runs lie side by side
// there, and a key goes to its place in the other buffer of the CTA whose run that
// is.  The loops are kept short: the sort is some ten thousand cycles long and its
// instructions are fetched cold (eight rounds unrolled, counting 300 tokens took
// 3.2k cycles instead of 0.9k).  4096 / 32768 tokens: 11 / 20 us.
template <int CTAS>
__device__ void sort_tokens(const SortArgs& a) {
    int* hist = reinterpret_cast<int*>(sort_smem);  // [kSortWarps][bins]
    Key* keys = reinterpret_cast<Key*>(sort_smem + kSortWarps * kBins * 4);
    Key* other = keys + kStaged;  // keys of the next pass
    uint16_t* places = reinterpret_cast<uint16_t*>(keys + kStaged * 2);
    __shared__ int total[kBins], base[kBins];
    __shared__ int last_head[kSortWarps];
    static_assert(kBins == kSortThreads, "a thread per digit");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = CTAS == 1 ? 0 : cluster_ctarank();
    constexpr int kWarps = CTAS * kSortWarps;
    const int me = rank * kSortWarps + warp;
    auto all_ctas = [&]() {
        __syncthreads();
        if (CTAS > 1) cluster_barrier();
    };

    // ahead of barriers of all CTAs
    if (rank == 0 && tid == 0) a.p.head->longs = a.p.head->huges = 0;

    int M = static_cast<int>(a.N), beg, end;
    unsigned run;  // keys of a warp
    auto set_run = [&]() {
        run = ((M + 31) / 32 + kWarps - 1) / kWarps * 32;
        beg = min(me * static_cast<int>(run), M);
        end = min(beg + static_cast<int>(run), M);
    };
    // Keys of kRounds rounds from i on, i the lane's first.
    auto block = [&](int64_t i, Key (&k)[kRounds]) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t at = i + r * 32;
            k[r] = at >= end ? kNone : keys[warp * run + (at - beg)];
        }
    };
    set_run();
    if (beg < end) {
        int64_t y[kWarpStaged / 32];
#pragma unroll
        for (int q = 0; q < kWarpStaged / 32; ++q)
            y[q] = __ldcg(a.tokens + min(beg + q * 32 + lane, end - 1));
#pragma unroll
        for (int q = 0; q < kWarpStaged / 32; ++q) {
            const int i = beg + q * 32 + lane;
            if (i < end) keys[warp * run + q * 32 + lane] = key_of(a, i, y[q]);
        }
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const Digits digits(a, pass);
        const int bins = digits.bins;
        set_run();
        unsigned* words = reinterpret_cast<unsigned*>(other);  // empty as yet
        for (int i = tid; i < kSortWarps * bins; i += kSortThreads) hist[i] = words[i] = 0;
        __syncthreads();
        int* count = hist + warp * bins;
        WarpCounts counts{count, words + warp * bins};
        uint16_t* place = places + warp * run - beg;
#pragma unroll 1
        for (int i = beg + lane; i - lane < end; i += 32 * kRounds) {
            Key k[kRounds];
            block(i, k);
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                const int at = counts.add(digits.of(k[r]));
                if (i + r * 32 < end) place[i + r * 32] = at;
            }
        }
        __syncthreads();
        const int mine = sum_over_warps(hist, bins);
        if (tid < bins) total[tid] = mine;
        all_ctas();
        int before = 0, all = 0;
        if (tid < bins) {
#pragma unroll
            for (uint32_t r = 0; r < CTAS; ++r) {
                const int c = CTAS == 1 ? mine : ld_cluster(total + tid, r);
                if (CTAS > 1 && r < rank) before += c;
                all += c;
            }
        }
        int grand;
        const int low = block_scan(all, grand);
        if (tid < bins) base[tid] = low + before;
        __syncthreads();
        if (pass == 0) M = grand;
        const unsigned share = ((M + 31) / 32 + kWarps - 1) / kWarps * 32 * kSortWarps;  // of a CTA
#pragma unroll 1
        for (int i = beg + lane; i - lane < end; i += 32 * kRounds) {
            Key k[kRounds];
            int at[kRounds];
            block(i, k);
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                const int d = digits.of(k[r]);
                at[r] = d >= 0 ? count[d] + base[d] + place[i + r * 32] : -1;
            }
#pragma unroll
            for (int r = 0; r < kRounds; ++r) {
                if (at[r] < 0) continue;
                if (CTAS == 1) {
                    other[at[r]] = k[r];
                } else {
                    const unsigned to = static_cast<unsigned>(at[r]) / share;
                    st_cluster64(other + (at[r] - to * share), to, k[r]);
                }
            }
        }
        Key* t = keys;
        keys = other;
        other = t;
        all_ctas();  // every key of the pass is in its place
    }

    // All that a warp needs from the runs ahead of its own is where the last token
    // started.
    set_run();
    const unsigned share = run * kSortWarps;
    auto row_at = [&](int i) -> unsigned {
        if (i < 0 || i >= M) return ~0u;
        const unsigned at = CTAS == 1 ? 0 : static_cast<unsigned>(i) / share;
        const Key* k = keys + (i - at * share);
        return static_cast<unsigned>((CTAS == 1 ? *k : ld_cluster64(k, at)) >> 32);
    };
    const unsigned row_before = row_at(beg - 1), row_after = row_at(end);
    int last = -1;
    unsigned prev = row_before;
#pragma unroll 1
    for (int i = beg + lane; i - lane < end; i += 32 * kRounds) {
        Key k[kRounds];
        unsigned heads[kRounds];
        block(i, k);
        heads_of(k, i, end, prev, heads);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (heads[r]) last = i - lane + r * 32 + 31 - __clz(heads[r]);
    }
    if (lane == 0) last_head[warp] = last;
    all_ctas();
    int head = -1;  // of the token that the run may start inside
#pragma unroll
    for (int r = 0; r < (kWarps + 31) / 32; ++r) {
        const int w = r * 32 + lane;
        if (w < me) {
            const int h = CTAS == 1 ? last_head[w % kSortWarps]
                                    : ld_cluster(last_head + w % kSortWarps, w / kSortWarps);
            head = max(head, h);
        }
    }
    head = __reduce_max_sync(0xffffffffu, head);
    write_entries(a, beg, end, head, row_before, row_after, block,
                  [&](int64_t i) { return keys[warp * run + (i - beg)]; });
    if (rank == 0 && tid == 0) write_head(a, M);
    all_ctas();  // no CTA leaves while another reads its shared memory
}

// More tokens than a cluster holds: the same sort over the whole device, three
// launches a pass and one for the entries.  A block owns kStaged keys.
// 131072 / 1000003 tokens: 38 / 58 us; the cluster, its keys in L2, took 87 / 585.
struct BigSort {
    const Key* src;    // nullptr: keys made of the tokens (the first pass)
    Key* dst;
    int* counts;       // [kBins][blocks]: keys of a digit, then of the blocks below
    int* totals;       // [kBins]
    uint16_t* places;  // [N] place among the block's keys of its digit
    int64_t blocks;
    int pass;
};
constexpr uint16_t kNoPlace = 0xffff;
constexpr int kCountSmem = kSortWarps * kBins * 8 + kStaged * 4;

__device__ __forceinline__ Key big_key(const SortArgs& a, const BigSort& s, int64_t i) {
    return s.src ? __ldcg(s.src + i) : key_of(a, i, a.tokens[i]);
}
__device__ __forceinline__ int64_t big_keys(const SortArgs& a, const BigSort& s) {
    return s.pass == 0 ? a.N : a.p.head->valid;
}

__global__ void __launch_bounds__(kSortThreads, 2)
    embed_count_kernel(const __grid_constant__ SortArgs a, const __grid_constant__ BigSort s) {
    int* hist = reinterpret_cast<int*>(sort_smem);
    unsigned* words = reinterpret_cast<unsigned*>(hist + kSortWarps * kBins);
    unsigned* found = words + kSortWarps * kBins;  // [kStaged] place << kDigitBits | digit
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    wait_for_prerequisites();
    launch_dependents();
    const Digits digits(a, s.pass);
    const int bins = digits.bins;
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) hist[i] = words[i] = 0;
    __syncthreads();
    const int64_t M = big_keys(a, s), b0 = int64_t(blockIdx.x) * kStaged;
    WarpCounts counts{hist + warp * bins, words + warp * bins};
#pragma unroll 1
    for (int j = warp * kWarpStaged + lane; j < (warp + 1) * kWarpStaged; j += 32 * kRounds) {
        Key k[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            k[r] = b0 + j + r * 32 < M ? big_key(a, s, b0 + j + r * 32) : kNone;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int d = digits.of(k[r]);
            const int at = counts.add(d);
            found[j + r * 32] = d < 0 ? ~0u : static_cast<unsigned>(at << kDigitBits | d);
        }
    }
    __syncthreads();
    const int sum = sum_over_warps(hist, bins);
    if (tid < bins) s.counts[tid * s.blocks + blockIdx.x] = sum;
    __syncthreads();
    for (int j = warp * kWarpStaged + lane; j < (warp + 1) * kWarpStaged; j += 32) {
        const unsigned f = found[j];
        if (b0 + j < M)
            s.places[b0 + j] = f == ~0u ? kNoPlace
                                        : hist[warp * bins + (f & (kBins - 1))] + (f >> kDigitBits);
    }
}

// A digit's counts become those of the blocks below.
__global__ void __launch_bounds__(kSortThreads)
    embed_scan_kernel(const __grid_constant__ BigSort s) {
    wait_for_prerequisites();
    launch_dependents();
    int* row = s.counts + blockIdx.x * s.blocks;
    int sum = 0;
    for (int64_t b = 0; b < s.blocks; b += kSortThreads) {
        const int c = b + threadIdx.x < s.blocks ? row[b + threadIdx.x] : 0;
        int all;
        const int under = block_scan(c, all);
        if (b + threadIdx.x < s.blocks) row[b + threadIdx.x] = sum + under;
        sum += all;
    }
    if (threadIdx.x == 0) s.totals[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kSortThreads)
    embed_place_kernel(const __grid_constant__ SortArgs a, const __grid_constant__ BigSort s) {
    __shared__ int base[kBins];
    const int tid = threadIdx.x;
    wait_for_prerequisites();
    launch_dependents();
    const Digits digits(a, s.pass);
    int all;
    const int low = block_scan(tid < digits.bins ? s.totals[tid] : 0, all);
    if (tid < digits.bins) base[tid] = low + s.counts[tid * s.blocks + blockIdx.x];
    const int64_t M = big_keys(a, s), b0 = int64_t(blockIdx.x) * kStaged;
    __syncthreads();
#pragma unroll 4
    for (int j = tid; j < kStaged; j += kSortThreads) {
        if (b0 + j >= M) break;
        const int p = s.places[b0 + j];
        if (p == kNoPlace) continue;
        const Key k = big_key(a, s, b0 + j);
        s.dst[base[digits.of(k)] + p] = k;
    }
    if (s.pass == 0 && blockIdx.x == 0 && tid == 0) {
        a.p.head->longs = a.p.head->huges = 0;
        write_head(a, all);
    }
}

__global__ void __launch_bounds__(kSortThreads)
    embed_entries_kernel(const __grid_constant__ SortArgs a, const Key* __restrict__ key) {
    const int lane = threadIdx.x & 31;
    wait_for_prerequisites();
    launch_dependents();
    const int64_t M = a.p.head->valid;
    const int64_t beg = blockIdx.x * int64_t(kStaged) + (threadIdx.x >> 5) * kWarpStaged;
    if (beg >= M) return;
    const int64_t end = beg + kWarpStaged < M ? beg + kWarpStaged : M;
    auto row_at = [&](int64_t i) { return static_cast<unsigned>(key[i] >> 32); };
    const unsigned row = row_at(beg), before = beg > 0 ? row_at(beg - 1) : ~0u;
    int64_t lo = beg;  // where the run's first token started: 32 probes a step
    if (row == before) {
        lo = 0;
        int64_t hi = beg - 1;  // the row at hi is the token's
        while (lo < hi) {
            const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
            const bool less = at < hi && row_at(at) < row;
            const int n = __popc(__ballot_sync(0xffffffffu, less));
            if (n == 0) break;
            const int64_t p = lo + (n - 1) * step;
            lo = p + 1;
            hi = p + step < hi ? p + step : hi;
        }
    }
    auto block = [&](int64_t i, Key (&k)[kRounds]) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) k[r] = i + r * 32 < end ? key[i + r * 32] : kNone;
    };
    write_entries(a, beg, end, static_cast<int>(lo), before, end < M ? row_at(end) : ~0u, block,
                  [&](int64_t i) { return key[i]; });
}

// [p, p + bytes) set to +0 by thread `me` of `threads`, p and bytes even; in 16-byte
// stores wherever p lies (16384 x 1001 bf16 into 150000 FP32 rows 111 us, with 2-byte
// ones for all of an unaligned row 132).
__device__ __forceinline__ void fill_zero(char* p, int64_t bytes, int me, int threads) {
    const int64_t off = -reinterpret_cast<intptr_t>(p) & 15, head = off < bytes ? off : bytes;
    const int64_t vec = (bytes - head) / 16, tail = head + vec * 16;
    if (me * 2 < head) *reinterpret_cast<uint16_t*>(p + me * 2) = 0;
#pragma unroll 4
    for (int64_t i = me; i < vec; i += threads)
        reinterpret_cast<uint4*>(p + head)[i] = make_uint4(0, 0, 0, 0);
    if (me * 2 < bytes - tail) *reinterpret_cast<uint16_t*>(p + tail + me * 2) = 0;
}

// The first `rows` rows at p, but for those of the bits `used`; rows between two of
// those at once where they lie side by side.
__device__ __forceinline__ void fill_rows_of(char* p, int64_t pitch, int64_t row_bytes, int rows,
                                             unsigned used, int me, int threads) {
    unsigned left = rows < 32 ? ~used & ((1u << rows) - 1) : ~used;
    while (left) {
        const int r = __ffs(left) - 1;
        const unsigned rest = ~(left >> r);  // 0: all 32
        const int n = pitch != row_bytes ? 1 : rest ? __ffs(rest) - 1 : 32;
        fill_zero(p + r * pitch, n * row_bytes, me, threads);
        left = r + n < 32 ? left & (~0u << (r + n)) : 0;
    }
}

// Rows that are filled together, of about `bytes`: a power of two up to 32.
__host__ __device__ inline int rows_together(int64_t row_bytes, int64_t bytes) {
    int n = 32;
    while (n > 1 && n * row_bytes > bytes) n /= 2;
    return n;
}

// Rows of no token set to +0, by the clusters that do not sort: each takes a
// range of the vocabulary and marks its tokens in a bitmap (each CTA reads a
// share of the tokens; the CTAs' bitmaps are joined).  It fills the first rows
// of the range, about what HBM takes in while the tokens are sorted; the others
// are filled beside the sums, and the bitmap tells which.
__device__ void fill_rows(const SortArgs& a, int64_t cluster, int64_t clusters) {
    unsigned* marks = reinterpret_cast<unsigned*>(sort_smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = cluster_ctas(), rank = cluster_ctarank();
    int64_t range = (a.V + clusters - 1) / clusters;
    range = range < kFillRows ? (range + 31) / 32 * 32 : kFillRows;
    for (int64_t r0 = cluster * range; r0 < a.V; r0 += clusters * range) {
        const int64_t rows = r0 + range < a.V ? range : a.V - r0;
        const int64_t now = static_cast<int64_t>(ceilf(static_cast<float>(rows) * a.now));
        const int words = static_cast<int>((rows + 31) / 32);
        for (int i = tid; i < words; i += kSortThreads) marks[i] = 0;
        __syncthreads();
        for (int64_t i = int64_t(rank) * kSortThreads + tid; i < a.N; i += ctas * kSortThreads) {
            const int64_t t = a.tokens[i], r = t - a.v0 - r0;
            if (t >= a.v0 && r >= 0 && r < rows) atomicOr(marks + (r >> 5), 1u << (r & 31));
        }
        __syncthreads();
        if (ctas > 1) cluster_barrier();
        auto joined = [&](int64_t w) {
            unsigned m = 0;
            for (uint32_t r = 0; r < ctas; ++r)
                m |= ld_cluster(reinterpret_cast<const int*>(marks) + w, r);
            return m;
        };
        for (int64_t w = int64_t(rank) * kSortThreads + tid; w < words; w += ctas * kSortThreads) {
            const int64_t done = now - w * 32;  // of the word's rows
            a.p.used[r0 / 32 + w] =
                joined(w) | (done >= 32 ? ~0u : done > 0 ? (1u << done) - 1 : 0u);
        }
        const int step = rows_together(a.row_bytes, 8192);  // of a warp
        for (int64_t v = (int64_t(rank) * kSortWarps + warp) * step; v < now;
             v += ctas * kSortWarps * step)
            fill_rows_of(a.table + (r0 + v) * a.pitch, a.pitch, a.row_bytes,
                         static_cast<int>(now - v < step ? now - v : step),
                         joined(v >> 5) >> (v & 31), lane, 32);
        __syncthreads();
        if (ctas > 1) cluster_barrier();  // the bitmaps may be overwritten
    }
}

template <int CTAS>
__global__ void __launch_bounds__(kSortThreads, 2)
    embed_sort_kernel(const __grid_constant__ SortArgs a) {
    launch_dependents();
    if (blockIdx.x < CTAS)
        sort_tokens<CTAS>(a);
    else
        fill_rows(a, blockIdx.x / CTAS - 1, gridDim.x / CTAS - 1);
}

struct GradArgs {
    int64_t ldg, D, ldw;
    float scale;
    int tiles, K, window, slots;
    SortPtrs p;
    // rows that are left to fill with +0 (accumulate = 0); fills = 0: none
    int64_t V, row_bytes;
    int fill_rows;   // of a block
    unsigned fills;  // blocks that fill rows, spread among the others
};

// What is stored for the scaled sum `s` on top of `old`.  + 0: a sum of nothing
// but zeros is +0 whatever the scale's sign.
template <typename TO>
__device__ __forceinline__ TO grad_value(float s, float old) {
    return Elem<TO>::from_f(old + (s + 0.f));
}

// Whether this block is one of `fills` that fill rows, which take turns with the others
// from the front while there are both; `block` becomes its number among its kind.
__device__ __forceinline__ bool fills_rows(unsigned fills, int64_t& block) {
    const int64_t sums = gridDim.x - fills, turns = sums < fills ? sums : fills;
    const bool fill = block < 2 * turns ? block & 1 : sums < fills;
    block = block < 2 * turns ? block >> 1 : block - turns;
    return fill;
}

// A warp takes a window of the sorted order, whole units of `window` entries or
// so, and a tile of columns: C packs of E elements a lane.  Its rows lie side
// by side in the sorted order whatever units they belong to, so R of them, and
// the table's row at each unit's end, are in flight together: one add per
// element read is bound by HBM, and most units are one or two rows.  Measured at
// 32768 tokens x 4096 bf16 added into 151936 FP32 rows, the whole call: 3 blocks
// an SM of 4 rows 141 us, 4 of 4 (spilled) 162, 2 of 8 144 (without the table's
// rows in registers 4 of 4 spill nothing: 4096 x 2048 40 us, 3 of 4 44); a warp
// per unit and tile, its rows waited for unit by unit, 209; adding to the table in L2
// (red.v4.f32) instead of reading it 164.
template <typename TI, typename TO, int E, int C, int R, bool ADD>
__global__ void __launch_bounds__(32 * kGradWarps, ADD ? 3 : 4) embed_grad_kernel(
    const TI* __restrict__ g, TO* __restrict__ dW, const __grid_constant__ GradArgs a) {
    const int lane = threadIdx.x & 31;
    wait_for_prerequisites();
    launch_dependents();
    int64_t block = blockIdx.x;
    if (!ADD && a.fills) {
        if (fills_rows(a.fills, block)) {
            const int64_t v0 = block * a.fill_rows;
            const int rows = static_cast<int>(a.V - v0 < a.fill_rows ? a.V - v0 : a.fill_rows);
            fill_rows_of(reinterpret_cast<char*>(dW + v0 * a.ldw), a.ldw * int64_t(sizeof(TO)),
                         a.row_bytes, rows, a.p.used[v0 / 32] >> (v0 % 32), threadIdx.x, 32 * kGradWarps);
            return;
        }
    }
    const int M = a.p.head->valid;
    const int64_t items = int64_t((M + a.window - 1) / a.window) * a.tiles;
    const int64_t it = block * kGradWarps + (threadIdx.x >> 5);
    if (it < items) {
        const int64_t c0 = (it % a.tiles * C * 32 + lane) * E;
        bool has[C];
#pragma unroll
        for (int k = 0; k < C; ++k) has[k] = c0 + k * 32 * E < a.D;
        const int64_t w = it / a.tiles;
        const int p0 = a.p.windows[w], p1 = a.p.windows[w + 1];
        int start = p0;  // of the unit
        float acc[C][E];
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) acc[k][j] = 0.f;
        for (int b = p0; b < p1; b += 32) {
            const Entry mine = b + lane < p1 ? a.p.entries[b + lane] : Entry{0, 0};
            const int n = p1 - b < 32 ? p1 - b : 32;
#pragma unroll 1
            for (int r = 0; r < n; r += R) {
                Pack<TI, E> x[R][C];
                Pack<TO, E> old[ADD ? R : 1][C];
                auto entry = [&](int q) {
                    return Entry{__shfl_sync(0xffffffffu, mine.pos, (r + q) & 31),
                                 __shfl_sync(0xffffffffu, mine.row, (r + q) & 31)};
                };
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const Entry e = entry(q);
                    if (r + q < n) {
                        const TI* src = g + int64_t(e.pos & ~kTop) * a.ldg + c0;
#pragma unroll
                        for (int k = 0; k < C; ++k)
                            if (has[k]) x[q][k].load(src + k * 32 * E);
                        if (ADD && (e.pos & kTop) && !(e.row & kTop)) {
                            const TO* row = dW + int64_t(e.row) * a.ldw + c0;
#pragma unroll
                            for (int k = 0; k < C; ++k)
                                if (has[k]) old[ADD ? q : 0][k].load(row + k * 32 * E);
                        }
                    }
                }
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    if (r + q >= n) break;
#pragma unroll
                    for (int k = 0; k < C; ++k)
#pragma unroll
                        for (int j = 0; j < E; ++j) acc[k][j] += Elem<TI>::to_f(x[q][k].e[j]);
                    const Entry e = entry(q);
                    if (!(e.pos & kTop)) continue;
                    if (!(e.row & kTop)) {
                        TO* row = dW + int64_t(e.row) * a.ldw + c0;
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            Pack<TO, E> y;
#pragma unroll
                            for (int j = 0; j < E; ++j)
                                y.e[j] = grad_value<TO>(
                                    a.scale * acc[k][j],
                                    ADD ? Elem<TO>::to_f(old[ADD ? q : 0][k].e[j]) : 0.f);
                            if (has[k]) y.store(row + k * 32 * E);
                        }
                    } else {
                        // Full pieces have the even slot of their K positions; beside
                        // it is the odd one, for a short last piece that starts there.
                        const int len = b + r + q + 1 - start;
                        float* dst =
                            a.p.part + (int64_t(start / a.K) * 2 + (len < a.K)) * a.p.Dp + c0;
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            Pack<float, E> y;
#pragma unroll
                            for (int j = 0; j < E; ++j) y.e[j] = acc[k][j];
                            if (has[k]) y.store(dst + k * 32 * E);
                        }
                    }
                    start = b + r + q + 1;
#pragma unroll
                    for (int k = 0; k < C; ++k)
#pragma unroll
                        for (int j = 0; j < E; ++j) acc[k][j] = 0.f;
                }
            }
        }
    }
}

// The scaled sum s of E columns stored to (or on top of) a row.
template <typename TO, int E, bool ADD>
__device__ __forceinline__ void put_row(TO* p, float scale, const float (&s)[E]) {
    Pack<TO, E> y;
    if (ADD) y.load(p);
#pragma unroll
    for (int j = 0; j < E; ++j)
        y.e[j] = grad_value<TO>(scale * s[j], ADD ? Elem<TO>::to_f(y.e[j]) : 0.f);
    y.store(p);
}

// Tokens of several pieces.  Of up to kFewPieces: a warp takes 32 packs of
// columns and adds the pieces in order.  Of more: a block takes kLanes packs;
// its 256 / kLanes groups of lanes each add every so-manieth piece, and the
// groups' sums are added in order.  The order depends on the number of pieces.
template <typename TO, int E, bool ADD>
__global__ void __launch_bounds__(32 * kGradWarps) embed_join_kernel(
    TO* __restrict__ dW, const __grid_constant__ GradArgs a) {
    constexpr int kLanes = 8, kGroups = 32 * kGradWarps / kLanes;
    __shared__ float sums[kGroups][kLanes * E];
    wait_for_prerequisites();
    const int lane = threadIdx.x & 31;
    auto pieces = [&](const Long& l) { return (l.count + a.K - 1) / a.K; };
    // sum of the pieces i, i + step, ... of the columns from c on
    auto add_up = [&](const Long& l, int64_t c, int i, int step, float (&s)[E]) {
        const int n = pieces(l);
        const int odd = l.count % a.K != 0 ? n - 1 : n;  // the short last piece
        const float* src = a.p.part + int64_t(l.start / a.K) * 2 * a.p.Dp + c;
#pragma unroll
        for (int j = 0; j < E; ++j) s[j] = 0.f;
#pragma unroll 8
        for (; i < n; i += step) {
            Pack<float, E> x;
            x.load(src + (i * int64_t(2) + (i == odd)) * a.p.Dp);
#pragma unroll
            for (int j = 0; j < E; ++j) s[j] += x.e[j];
        }
    };
    const SortHead head = *a.p.head;
    const int64_t narrow = (a.D + kLanes * E - 1) / (kLanes * E);
    for (int64_t it = blockIdx.x; it < head.huges * narrow; it += gridDim.x) {
        const Long l = a.p.longs[a.slots - 1 - it / narrow];
        const int group = threadIdx.x / kLanes, at = threadIdx.x % kLanes;
        const int64_t c = (it % narrow * kLanes + at) * E;
        float s[E] = {};
        if (c < a.D) add_up(l, c, group, kGroups, s);
#pragma unroll
        for (int j = 0; j < E; ++j) sums[group][j * kLanes + at] = s[j];
        __syncthreads();
        if (group == 0 && c < a.D) {
            for (int g = 1; g < kGroups; ++g)
#pragma unroll
                for (int j = 0; j < E; ++j) s[j] += sums[g][j * kLanes + at];
            put_row<TO, E, ADD>(dW + int64_t(l.row) * a.ldw + c, a.scale, s);
        }
        __syncthreads();
    }
    const int64_t wide = (a.D + 32 * E - 1) / (32 * E);
    for (int64_t it = blockIdx.x * int64_t(kGradWarps) + (threadIdx.x >> 5); it < head.longs * wide;
         it += int64_t(gridDim.x) * kGradWarps) {
        const Long l = a.p.longs[it / wide];
        const int64_t c = (it % wide * 32 + lane) * E;
        if (c >= a.D) continue;
        float s[E];
        add_up(l, c, 0, 1, s);
        put_row<TO, E, ADD>(dW + int64_t(l.row) * a.ldw + c, a.scale, s);
    }
}

// Few tokens, in one launch and without a sort: a warp takes a position and a tile of
// columns, looks in all tokens (in shared memory) for those of the same row and, if
// none is ahead of its own, adds up their rows in order.  Rows of a token of more than
// kPiece are shared out, in order, over the block's warps once they are done.  Bound
// by latency: tokens, rows and the table's rows are three trips to memory (a launch
// alone 2.2 us).  A warp that looked once for several tiles of columns was faster
// without hot tokens (1024 x 4096 14.4 us) and slower with them (20.3).
struct MatchArgs {
    const int64_t* tokens;
    int N, tiles;
    int64_t V, v0, ldg, D, ldw, row_bytes;
    float scale;
    int fill_rows;   // as in GradArgs, any number
    unsigned fills;
};
constexpr int kMatchThreads = 512;
constexpr int kMatchWarps = kMatchThreads / 32;
constexpr int kMatchInFlight = 4;  // rows of a warp
constexpr int kMatchRows = 4096;  // most rows that a block fills
static_assert(kMatch % 128 == 0 && kMatch / kMatchWarps >= kPiece, "a warp's share of a token");

// The positions of row v among the first `end` of rows, 128 at a time: take(p, k) by
// the lane of the k-th position p; more(n, p) with their number so far and the first
// of them says whether to go on.  Returns their number.
template <typename T, typename M>
__device__ __forceinline__ int match(const int* rows, int end, int v, const T& take, const M& more) {
    const int lane = threadIdx.x & 31;
    const unsigned under = (1u << lane) - 1;
    int n = 0;
#pragma unroll 2
    for (int c = 0; c < end; c += 128) {
        const int4 r = *reinterpret_cast<const int4*>(rows + c + lane * 4);
        const bool is[4] = {r.x == v, r.y == v, r.z == v, r.w == v};
        if (!__any_sync(0xffffffffu, is[0] || is[1] || is[2] || is[3])) continue;
        int k = n, all = 0;
        unsigned any = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const unsigned m = __ballot_sync(0xffffffffu, is[j]);
            k += __popc(m & under);
            all += __popc(m);
            any |= m;
        }
        const int first = is[0] ? 0 : is[1] ? 1 : is[2] ? 2 : 3, low = __ffs(any) - 1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (is[j]) take(c + lane * 4 + j, k++);
        n += all;
        if (!more(n, c + low * 4 + __shfl_sync(0xffffffffu, first, low))) break;
    }
    return n;
}

template <typename TI, typename TO, int E, int C, int R, bool ADD>
__global__ void __launch_bounds__(kMatchThreads, 2) embed_match_kernel(
    const TI* __restrict__ g, TO* __restrict__ dW, const __grid_constant__ MatchArgs a) {
    constexpr int kCols = 32 * C * E;
    __shared__ __align__(16) int rows[kMatch];
    __shared__ int lists[kMatchWarps][kMatch / kMatchWarps];
    __shared__ float sums[kMatchWarps * kCols];
    __shared__ int longs[kMatchWarps];  // the rows of a warp's token, if that has more than kPiece
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t block = blockIdx.x;
    if (!ADD && fills_rows(a.fills, block)) {
        unsigned* marks = reinterpret_cast<unsigned*>(rows);
        static_assert(kMatchRows <= kMatch * 32, "the marks fit");
        const int64_t r0 = block * a.fill_rows;
        const int n = static_cast<int>(a.V - r0 < a.fill_rows ? a.V - r0 : a.fill_rows);
        for (int i = tid; i < (n + 31) / 32; i += kMatchThreads) marks[i] = 0;
        __syncthreads();
        for (int i = tid; i < a.N; i += kMatchThreads) {
            const int64_t t = a.tokens[i], r = t - a.v0 - r0;
            if (t >= a.v0 && r >= 0 && r < n) atomicOr(marks + (r >> 5), 1u << (r & 31));
        }
        __syncthreads();
        const int step = rows_together(a.row_bytes, 8192), pitch = sizeof(TO);
        for (int v = warp * step; v < n; v += kMatchWarps * step)
            fill_rows_of(reinterpret_cast<char*>(dW + (r0 + v) * a.ldw), a.ldw * pitch, a.row_bytes,
                         n - v < step ? n - v : step, marks[v >> 5] >> (v & 31), lane, 32);
        return;
    }
    const int end = (a.N + 127) / 128 * 128;
    for (int i = tid; i < end; i += kMatchThreads) {
        int row = -1;
        if (i < a.N) {
            const int64_t y = a.tokens[i], v = y - a.v0;
            if (y >= a.v0 && v < a.V) row = static_cast<int>(v);
        }
        rows[i] = row;
    }
    __syncthreads();
    // neighbouring blocks take neighbouring tiles, so that a token's are spread
    const int blocks = gridDim.x - (ADD ? 0 : a.fills);
    auto item = [&](int w) { return w * blocks + static_cast<int>(block); };
    auto token_of = [&](int w) { return item(w) / a.tiles; };
    auto column = [&](int w) { return item(w) % a.tiles * int64_t(kCols); };
    float acc[C][E];
    auto clear = [&]() {
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) acc[k][j] = 0.f;
    };
    const int* mine = lists[warp];
    auto load_rows = [&](auto& x, int p, int n, int64_t c0) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (p + q >= n) break;
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (c0 + (k * 32 + lane) * E < a.D)
                    x[q][k].load(g + mine[p + q] * a.ldg + c0 + (k * 32 + lane) * E);
        }
    };
    auto add_rows = [&](const auto& x, int p, int n) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
            if (p + q >= n) break;
#pragma unroll
            for (int k = 0; k < C; ++k)
#pragma unroll
                for (int j = 0; j < E; ++j) acc[k][j] += Elem<TI>::to_f(x[q][k].e[j]);
        }
    };

    const int i = token_of(warp);
    const int v = i < a.N ? rows[i] : -1;
    int n = 0;
    if (v >= 0) {
        bool first = true;
        n = match(
            rows, end, v,
            [&](int p, int k) {
                if (k < kPiece) lists[warp][k] = p;
            },
            [&](int so_far, int p) {
                if (n == 0 && p != i) first = false;
                n = so_far;
                return first;
            });
        if (!first) n = 0;
        __syncwarp();
    }
    if (lane == 0) longs[warp] = n > kPiece ? n : 0;
    if (n > 0 && n <= kPiece) {
        const int64_t c0 = column(warp);
        TO* row = dW + int64_t(v) * a.ldw + c0;
        Pack<TO, E> old[C];
        if (ADD) {
#pragma unroll
            for (int k = 0; k < C; ++k)
                if (c0 + (k * 32 + lane) * E < a.D) old[k].load(row + (k * 32 + lane) * E);
        }
        clear();
        for (int p = 0; p < n; p += R) {
            Pack<TI, E> x[R][C];
            load_rows(x, p, n, c0);
            add_rows(x, p, n);
        }
#pragma unroll
        for (int k = 0; k < C; ++k) {
            Pack<TO, E> y;
#pragma unroll
            for (int j = 0; j < E; ++j)
                y.e[j] = grad_value<TO>(a.scale * acc[k][j], ADD ? Elem<TO>::to_f(old[k].e[j]) : 0.f);
            if (c0 + (k * 32 + lane) * E < a.D) y.store(row + (k * 32 + lane) * E);
        }
    }
    __syncthreads();
    for (int w = 0; w < kMatchWarps; ++w) {
        const int all = longs[w];
        if (all == 0) continue;
        const int row = rows[token_of(w)], per = (all + kMatchWarps - 1) / kMatchWarps;
        const int64_t c0 = column(w);
        const int p0 = warp * per, p1 = min(p0 + per, all);
        match(
            rows, end, row,
            [&](int p, int k) {
                if (k >= p0 && k < p1) lists[warp][k - p0] = p;
            },
            [&](int so_far, int) { return so_far < p1; });
        __syncwarp();
        clear();
        for (int p = 0; p < p1 - p0; p += R) {
            Pack<TI, E> x[R][C];
            load_rows(x, p, p1 - p0, c0);
            add_rows(x, p, p1 - p0);
        }
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) sums[warp * kCols + (k * 32 + lane) * E + j] = acc[k][j];
        __syncthreads();
        if (tid < kCols && c0 + tid < a.D) {
            const int used = (all + per - 1) / per;
            float f = sums[tid];
            for (int u = 1; u < used; ++u) f += sums[u * kCols + tid];
            TO* p = dW + int64_t(row) * a.ldw + c0 + tid;
            *p = grad_value<TO>(a.scale * f, ADD ? Elem<TO>::to_f(*p) : 0.f);
        }
        __syncthreads();
    }
}

// Whole 16-byte packs of rows that start on 16-byte boundaries.
bool grad_vec(const EmbedArgs& a) {
    return a.D % (a.dtype == LL_F32 ? 4 : 8) == 0 &&
           rows16(a.rows, a.ld_rows, a.dtype == LL_F32 ? 4 : 2) &&
           rows16(a.table, a.ld_table, a.table_dtype == LL_F32 ? 4 : 2);
}

template <typename TI, typename TO>
cudaError_t grad_typed(const EmbedArgs& e, bool vec, int accumulate, GradArgs a, int num_sms,
                       cudaStream_t s) {
    constexpr int E = 16 / sizeof(TI), C1 = 4;
    const int64_t cols = vec ? 32 * E : 32 * C1;
    a.tiles = static_cast<int>((a.D + cols - 1) / cols);
    const TI* g = static_cast<const TI*>(e.rows);
    TO* dW = static_cast<TO*>(e.table);
    const int64_t items = (e.N + a.window - 1) / a.window * a.tiles;
    const int64_t sums_blocks = (items + kGradWarps - 1) / kGradWarps;
    a.V = e.V;
    a.row_bytes = e.D * int64_t(sizeof(TO));
    a.fill_rows = rows_together(a.row_bytes, kFillBytes);
    a.fills = accumulate ? 0 : static_cast<unsigned>((e.V + a.fill_rows - 1) / a.fill_rows);
    const int64_t blocks = sums_blocks + a.fills;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const unsigned threads = 32 * kGradWarps;
    const int64_t long_items = e.N / a.K * ((a.D + 127) / 128);
    const int64_t full = int64_t(num_sms) * 8;
    const unsigned join_blocks = static_cast<unsigned>(full < long_items ? full : long_items);
    if (e.N <= kMatch) {
        const int64_t all = (e.N * a.tiles + kMatchWarps - 1) / kMatchWarps;
        MatchArgs m{e.tokens, static_cast<int>(e.N), a.tiles, e.V, e.v0, a.ldg, a.D, a.ldw,
                    a.row_bytes, a.scale, 1, 0};
        while (m.fill_rows * 2 * a.row_bytes <= kFillBytes && m.fill_rows < kMatchRows)
            m.fill_rows *= 2;
        if (!accumulate) m.fills = static_cast<unsigned>((e.V + m.fill_rows - 1) / m.fill_rows);
        if (all * kMatchWarps + m.fills > 0x7fffffff) return cudaErrorInvalidConfiguration;
        auto run = [&](auto* kernel) {
            note_launches(1);
            kernel<<<static_cast<unsigned>(all + m.fills), kMatchThreads, 0, s>>>(g, dW, m);
            return cudaGetLastError();
        };
        constexpr int R = kMatchInFlight;
        if (vec)
            return accumulate ? run(embed_match_kernel<TI, TO, E, 1, R, true>)
                              : run(embed_match_kernel<TI, TO, E, 1, R, false>);
        return accumulate ? run(embed_match_kernel<TI, TO, 1, C1, R, true>)
                          : run(embed_match_kernel<TI, TO, 1, C1, R, false>);
    }
    auto run = [&](auto* sums, auto* join) {
        note_launches(join_blocks ? 2 : 1);
        const cudaError_t err =
            launch_after(sums, static_cast<unsigned>(blocks), threads, s, 0, g, dW, a);
        if (err != cudaSuccess || !join_blocks) return err;
        return launch_after(join, join_blocks, threads, s, 0, dW, a);
    };
    constexpr int R = kGradRows;
    if (vec)
        return accumulate
                   ? run(embed_grad_kernel<TI, TO, E, 1, R, true>, embed_join_kernel<TO, 4, true>)
                   : run(embed_grad_kernel<TI, TO, E, 1, R, false>, embed_join_kernel<TO, 4, false>);
    return accumulate
               ? run(embed_grad_kernel<TI, TO, 1, C1, R, true>, embed_join_kernel<TO, 1, true>)
               : run(embed_grad_kernel<TI, TO, 1, C1, R, false>, embed_join_kernel<TO, 1, false>);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_embed_fwd(const EmbedArgs& a, cudaStream_t s) {
    note_launches(1);
    const bool vec = rows16(a.rows, a.ld_rows, a.dtype == LL_F32 ? 4 : 2) &&
                     rows16(a.table, a.ld_table, a.table_dtype == LL_F32 ? 4 : 2);
    switch (a.dtype * 3 + a.table_dtype) {
        case LL_F32 * 3 + LL_F32: return fwd_typed<float, float>(a, vec, s);
        case LL_F32 * 3 + LL_F16: return fwd_typed<float, __half>(a, vec, s);
        case LL_F32 * 3 + LL_BF16: return fwd_typed<float, __nv_bfloat16>(a, vec, s);
        case LL_F16 * 3 + LL_F16: return fwd_typed<__half, __half>(a, vec, s);
        case LL_F16 * 3 + LL_F32: return fwd_typed<__half, float>(a, vec, s);
        case LL_BF16 * 3 + LL_BF16: return fwd_typed<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
        default: return fwd_typed<__nv_bfloat16, float>(a, vec, s);
    }
}

// Workspace of the gradient.
static SortPtrs grad_layout(int64_t N, int64_t D, int64_t V, void* ws, size_t* bytes) {
    char* p = static_cast<char*>(ws);
    size_t off = 0;
    auto take = [&](size_t n) {
        char* at = p + off;
        off += up256(n);
        return at;
    };
    const int64_t slots = (N + piece_rows(N) - 1) / piece_rows(N);
    SortPtrs q;
    q.Dp = (D + 7) / 8 * 8;
    q.head = reinterpret_cast<SortHead*>(take(sizeof(SortHead)));
    const int64_t big = N > kStaged * kSortCtas ? N : 0;
    q.buf0 = reinterpret_cast<unsigned long long*>(take(size_t(big) * 8));
    q.buf1 = reinterpret_cast<unsigned long long*>(take(size_t(big) * 8));
    q.counts = reinterpret_cast<int*>(take(size_t((big + kStaged - 1) / kStaged) * kBins * 4));
    q.totals = reinterpret_cast<int*>(take(big ? kBins * 4 : 0));
    q.places = reinterpret_cast<uint16_t*>(take(size_t(big) * 2));
    q.entries = reinterpret_cast<Entry*>(take(size_t(N) * sizeof(Entry)));
    const int64_t w = window_rows(N);
    q.windows = reinterpret_cast<int*>(take(size_t((N + w - 1) / w + 1) * 4));
    q.longs = reinterpret_cast<Long*>(take(size_t(slots) * sizeof(Long)));
    q.used = reinterpret_cast<unsigned*>(take(size_t((V + 31) / 32) * 4));
    q.part = reinterpret_cast<float*>(take(size_t(2 * slots) * size_t(q.Dp) * 4));
    *bytes = off;
    return q;
}

size_t embed_bwd_bytes(int64_t N, int64_t D, int64_t V) {
    size_t bytes;
    grad_layout(N, D, V, nullptr, &bytes);
    return bytes;
}

static int bits_of(int64_t V) {
    int b = 1;
    while ((int64_t(1) << b) < V) ++b;
    return b;
}

// Lets a kernel have `bytes` of dynamic shared memory, once on a device.
template <typename F>
static cudaError_t give_smem(F* kernel, int bytes, const DevInfo& dev,
                             std::atomic<uint64_t>& ready) {
    const uint64_t bit = uint64_t(1) << dev.device;
    if (ready.load() & bit) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit);
    return e;
}

static cudaError_t launch_big_sort(const SortArgs& a, const DevInfo& dev, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    cudaError_t e = give_smem(embed_count_kernel, kCountSmem, dev, ready);
    if (e == cudaSuccess && a.table)
        e = cudaMemsetAsync(a.p.used, 0, size_t((a.V + 31) / 32) * 4, s);
    BigSort b{nullptr, a.p.buf0, a.p.counts, a.p.totals, a.p.places,
              (a.N + kStaged - 1) / kStaged, 0};
    const unsigned blocks = static_cast<unsigned>(b.blocks);
    int bits = a.bits;
    for (; e == cudaSuccess && b.pass < a.passes; ++b.pass) {
        const int db = (bits + (a.passes - b.pass) - 1) / (a.passes - b.pass);
        bits -= db;
        note_launches(3);
        if (b.pass == 0) {  // whatever is ahead of it
            embed_count_kernel<<<blocks, kSortThreads, kCountSmem, s>>>(a, b);
            e = cudaGetLastError();
        } else {
            e = launch_after(embed_count_kernel, blocks, kSortThreads, s, kCountSmem, a, b);
        }
        if (e == cudaSuccess) e = launch_after(embed_scan_kernel, 1u << db, kSortThreads, s, 0, b);
        if (e == cudaSuccess)
            e = launch_after(embed_place_kernel, blocks, kSortThreads, s, 0, a, b);
        b.src = b.dst;
        b.dst = b.dst == a.p.buf0 ? a.p.buf1 : a.p.buf0;
    }
    if (e != cudaSuccess) return e;
    note_launches(1);
    return launch_after(embed_entries_kernel, blocks, kSortThreads, s, 0, a, b.src);
}

cudaError_t launch_embed_sort(const EmbedArgs& e, int accumulate, void* ws, const DevInfo& dev,
                              cudaStream_t s) {
    if (e.N <= kMatch) return cudaSuccess;  // not sorted
    size_t bytes;
    SortArgs a;
    a.tokens = e.tokens;
    a.N = e.N;
    a.V = e.V;
    a.v0 = e.v0;
    a.bits = bits_of(e.V);
    a.passes = (a.bits + kDigitBits - 1) / kDigitBits;
    a.K = static_cast<int>(piece_rows(e.N));
    a.window = window_rows(e.N);
    a.slots = static_cast<int>((e.N + a.K - 1) / a.K);
    a.p = grad_layout(e.N, e.D, e.V, ws, &bytes);
    const int64_t es = e.table_dtype == LL_F32 ? 4 : 2;
    a.table = accumulate ? nullptr : static_cast<char*>(e.table);
    a.row_bytes = e.D * es;
    a.pitch = e.ld_table * es;
    a.now = 0.f;
    a.mark = e.N > kStaged * kSortCtas && !accumulate;
    if (e.N > kStaged * kSortCtas) return launch_big_sort(a, dev, s);
    // The sort takes about 10 us and 0.3 us per thousand tokens.
    const double beside = 48e6 + 1600.0 * static_cast<double>(e.N);
    const double total = static_cast<double>(e.V) * static_cast<double>(a.row_bytes);
    a.now = beside < total ? static_cast<float>(beside / total) : 1.f;

    note_launches(1);
    const int ctas = e.N <= kOneCta ? 1 : kSortCtas;
    auto* kernel = ctas == 1 ? embed_sort_kernel<1> : embed_sort_kernel<kSortCtas>;
    static std::atomic<uint64_t> ready[2];
    const cudaError_t err = give_smem(kernel, kSortSmem, dev, ready[ctas == 1]);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(accumulate ? ctas : kFillCtas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_embed_bwd(const EmbedArgs& e, int accumulate, void* ws, const DevInfo& dev,
                             cudaStream_t s) {
    const int num_sms = dev.num_sms;
    size_t bytes;
    const bool vec = grad_vec(e);
    GradArgs a;
    a.ldg = e.ld_rows;
    a.D = e.D;
    a.ldw = e.ld_table;
    a.scale = e.scale;
    a.tiles = 0;
    a.K = static_cast<int>(piece_rows(e.N));
    a.window = window_rows(e.N);
    a.slots = static_cast<int>((e.N + a.K - 1) / a.K);
    a.p = grad_layout(e.N, e.D, e.V, ws, &bytes);
    switch (e.dtype * 3 + e.table_dtype) {
        case LL_F32 * 3 + LL_F32:
            return grad_typed<float, float>(e, vec, accumulate, a, num_sms, s);
        case LL_F16 * 3 + LL_F16:
            return grad_typed<__half, __half>(e, vec, accumulate, a, num_sms, s);
        case LL_F16 * 3 + LL_F32:
            return grad_typed<__half, float>(e, vec, accumulate, a, num_sms, s);
        case LL_BF16 * 3 + LL_BF16:
            return grad_typed<__nv_bfloat16, __nv_bfloat16>(e, vec, accumulate, a, num_sms, s);
        default:
            return grad_typed<__nv_bfloat16, float>(e, vec, accumulate, a, num_sms, s);
    }
}

}  // namespace ll
