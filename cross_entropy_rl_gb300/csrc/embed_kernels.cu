// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[n, :] = scale * W[y_n - v0, :]  (+0 rows for other tokens)
//   backward  dW[v, :] (+)= scale * sum_{n: y_n - v0 = v} g[n, :]
#include "ll_device.cuh"

namespace ll {
namespace {

// ------------------------------------------------------------------- lookup
// One multiply per element: bound by HBM (a row read, a row written).  A warp
// takes one row's tile of kLookupTile chunks of E elements; all its loads are
// issued before the first store.
constexpr int kLookupUnroll = 4;
constexpr int kLookupTile = 32 * kLookupUnroll;
constexpr int kLookupWarps = 8;

template <typename TI, typename TO, int E>
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
    for (int64_t c0 = int64_t(blockIdx.y) * kLookupTile + lane; c0 < chunks;
         c0 += int64_t(gridDim.y) * kLookupTile) {
        Pack<TI, E> x[kLookupUnroll];
#pragma unroll
        for (int u = 0; u < kLookupUnroll; ++u) {
            const int64_t c = (c0 + 32 * u) * E;
            if (in && c + E <= D) x[u].load(src + c);
        }
#pragma unroll
        for (int u = 0; u < kLookupUnroll; ++u) {
            const int64_t c = (c0 + 32 * u) * E;
            if (c + E <= D) {
                Pack<TO, E> y;
#pragma unroll
                for (int j = 0; j < E; ++j)
                    y.e[j] = Elem<TO>::from_f(in ? Elem<TI>::to_f(x[u].e[j]) * scale : 0.f);
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
    const int64_t tiles = (chunks + kLookupTile - 1) / kLookupTile;
    const dim3 grid(static_cast<unsigned>((a.N + kLookupWarps - 1) / kLookupWarps),
                    static_cast<unsigned>(tiles < 65535 ? tiles : 65535));
    const TI* W = static_cast<const TI*>(a.rows);
    TO* out = static_cast<TO*>(a.table);
    if (vec)
        embed_fwd_kernel<TI, TO, E><<<grid, 32 * kLookupWarps, 0, s>>>(
            W, a.ld_rows, a.tokens, a.N, a.D, a.V, a.v0, a.scale, out, a.ld_table);
    else
        embed_fwd_kernel<TI, TO, 1><<<grid, 32 * kLookupWarps, 0, s>>>(
            W, a.ld_rows, a.tokens, a.N, a.D, a.V, a.v0, a.scale, out, a.ld_table);
    return cudaGetLastError();
}

bool rows16(const void* p, int64_t ld, size_t es) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && size_t(ld) * es % 16 == 0;
}

#ifndef LL_GC
#define LL_GC 3
#define LL_GR 4
#endif
// ----------------------------------------------------------------- gradient
// Three launches.  The first sorts the tokens (one cluster), the second adds up
// the rows of grad_out in the sorted order, the third finishes long tokens.
//
// A unit is at most K sorted positions of one token: a token's occurrences are
// cut every K from its first, so the order of its additions is a function of
// its own occurrences (and of K).  The row of a token of one unit is finished
// by the warp that adds it; the pieces of a longer one are written as FP32
// partial sums, which a block then adds in order.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;        // CTAs of the sorting cluster
constexpr int kSortBlock = 8;       // keys a lane loads at a time
constexpr int kDigitBits = 9;       // most bits of a sorting pass
constexpr int kBins = 1 << kDigitBits;
constexpr int kSortSmem = kSortWarps * kBins * 4;
constexpr int kFillClusters = 32;  // clusters in all when rows are filled
constexpr int kFillRows = kSortSmem * 8;  // vocabulary rows of one cluster's bitmap
constexpr int kWindow = 16;         // sorted positions of a warp of the sums

// Positions of a piece: few enough that a token of a third of a large batch is
// spread over the device, and that at most 2048 pieces' partial sums are kept.
__host__ __device__ inline int64_t piece_rows(int64_t N) {
    int64_t k = 32;
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
    int valid;  // tokens of the table: entries
    int longs;
};

struct SortPtrs {
    SortHead* head;
    unsigned long long *buf0, *buf1;  // [N] (row << 32 | position)
    Entry* entries;                   // [N]
    int* windows;                     // [ceil(N / kWindow) + 1] start of the unit of each kWindow-th entry
    Long* longs;                      // [ceil(N / K)], in any order
    float* part;                      // [2 ceil(N / K), Dp] sums of pieces
    int64_t Dp;
};

struct SortArgs {
    const int64_t* tokens;
    int64_t N, V, v0;
    int bits, passes;  // of a row index; sorting passes
    int K;
    SortPtrs p;
    // rows of no token are set to +0 (accumulate = 0), else null
    char* table;
    int64_t row_bytes, pitch;
};

extern __shared__ __align__(16) unsigned char sort_smem[];

__device__ __forceinline__ int ld_cluster(const int* local, uint32_t rank) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(local, rank)));
    return v;
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

// Lanes whose digit (of `bits` bits, below 0: none) is this lane's.  One vote a
// bit: match.any took ~75 cycles of the SM for each warp where most lanes
// differ, and made half of the sort's time.
__device__ __forceinline__ unsigned same_digit(int d, int bits) {
    unsigned m = __ballot_sync(0xffffffffu, d >= 0);
    if (d < 0) m = 0;
    for (int b = 0; b < bits; ++b) {
        const unsigned set = __ballot_sync(0xffffffffu, d >> b & 1);
        m &= d >> b & 1 ? set : ~set;
    }
    return m;
}

// The run of keys [beg, end) of warp `me` of `warps`, of M in all.
struct Run {
    int64_t beg, end;
    bool kept;  // one block of kSortBlock keys a lane: it stays in registers
    __device__ Run(int64_t M, int64_t me, int64_t warps) {
        const int64_t per = ((M + 31) / 32 + warps - 1) / warps * 32;
        beg = me * per < M ? me * per : M;
        end = beg + per < M ? beg + per : M;
        kept = per <= 32 * kSortBlock;
    }
};

// Least-significant-digit radix sort by one cluster, stable, so that the
// positions of a token stay ascending.  Each warp owns a run of the keys; a
// pass counts the run's digits (one lane adds for all of its digit), scans the
// counts over warps, CTAs and digits, and writes each key to its place.  Tokens
// outside the table drop out in the first pass.
__device__ void sort_tokens(const SortArgs& a) {
    int* hist = reinterpret_cast<int*>(sort_smem);  // [kSortWarps][bins]
    __shared__ int total[kBins], base[kBins], scan[kSortWarps], grand;
    static_assert(kBins == kSortThreads, "a thread per digit");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const int64_t warps = kSortCtas * kSortWarps, me = rank * kSortWarps + warp;
    const unsigned lt = (1u << lane) - 1;

    if (rank == 0 && tid == 0) a.p.head->longs = 0;  // ahead of cluster barriers

    int64_t M = a.N;
    int shift = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int db = (a.bits - shift + (a.passes - pass) - 1) / (a.passes - pass);
        const int bins = 1 << db;
        const unsigned long long* src = (pass & 1) ? a.p.buf0 : a.p.buf1;
        unsigned long long* dst = (pass & 1) ? a.p.buf1 : a.p.buf0;
        const Run run(M, me, warps);
        unsigned long long k[kSortBlock];
        int d[kSortBlock];  // digit; of a kept run, with the place among its equals above
        auto fetch = [&](int64_t i0) {
#pragma unroll
            for (int r = 0; r < kSortBlock; ++r) {
                const int64_t i = i0 + r * 32 + lane;
                d[r] = -1;
                if (i >= run.end) continue;
                if (pass > 0) {
                    k[r] = __ldcg(src + i);
                    d[r] = 0;
                } else {
                    const int64_t y = a.tokens[i];
                    const int64_t v = y - a.v0;
                    k[r] = (static_cast<unsigned long long>(v) << 32) | static_cast<unsigned>(i);
                    if (y >= a.v0 && v < a.V) d[r] = 0;
                }
            }
        };
        auto digits = [&]() {
#pragma unroll
            for (int r = 0; r < kSortBlock; ++r)
                if (d[r] == 0) d[r] = static_cast<int>(k[r] >> (32 + shift)) & (bins - 1);
        };
        if (run.kept) fetch(run.beg);  // on its way while the counts are cleared
        for (int i = tid; i < kSortWarps * bins; i += kSortThreads) hist[i] = 0;
        __syncthreads();
        int* mine = hist + warp * bins;
        for (int64_t i0 = run.beg; i0 < run.end; i0 += 32 * kSortBlock) {
            if (!run.kept) fetch(i0);
            digits();
#pragma unroll
            for (int r = 0; r < kSortBlock; ++r) {
                const unsigned peers = same_digit(d[r], db);
                const int had = d[r] >= 0 ? mine[d[r]] : 0;
                __syncwarp();
                if (d[r] >= 0) {
                    if ((peers & lt) == 0) mine[d[r]] = had + __popc(peers);
                    if (run.kept) d[r] |= (had + __popc(peers & lt)) << kDigitBits;
                }
                __syncwarp();
            }
        }
        __syncthreads();
        if (tid < bins) {  // counts of the warps below, and of the CTA
            int c[kSortWarps], sum = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * bins + tid];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                hist[w * bins + tid] = sum;
                sum += c[w];
            }
            total[tid] = sum;
        }
        __syncthreads();
        cluster_barrier();
        int before = 0, all = 0;
        if (tid < bins) {
#pragma unroll
            for (uint32_t r = 0; r < kSortCtas; ++r) {
                const int c = ld_cluster(total + tid, r);
                if (r < rank) before += c;
                all += c;
            }
        }
        const int low = warp_scan(all, lane);  // digits below, within 32
        if (lane == 31) scan[warp] = low + all;
        __syncthreads();
        if (warp == 0) {
            const int c = lane < kSortWarps ? scan[lane] : 0;
            const int s = warp_scan(c, lane);
            if (lane < kSortWarps) scan[lane] = s;
            if (lane == 31) grand = s + c;
        }
        __syncthreads();
        if (tid < bins) base[tid] = scan[warp] + low + before;
        M = pass == 0 ? grand : M;
        __syncthreads();
        for (int64_t i0 = run.beg; i0 < run.end; i0 += 32 * kSortBlock) {
            if (run.kept) {
#pragma unroll
                for (int r = 0; r < kSortBlock; ++r)
                    if (d[r] >= 0) {
                        const int b = d[r] & (kBins - 1);
                        dst[mine[b] + base[b] + (d[r] >> kDigitBits)] = k[r];
                    }
                break;
            }
            fetch(i0);
            digits();
#pragma unroll
            for (int r = 0; r < kSortBlock; ++r) {
                const unsigned peers = same_digit(d[r], db);
                const int had = d[r] >= 0 ? mine[d[r]] : 0;
                __syncwarp();
                if (d[r] >= 0) {
                    if ((peers & lt) == 0) mine[d[r]] = had + __popc(peers);
                    dst[had + base[d[r]] + __popc(peers & lt)] = k[r];
                }
                __syncwarp();
            }
        }
        shift += db;
        __syncthreads();
        cluster_barrier();  // every key of the pass is in its place
    }

    // The entries with their units' ends.  All that a warp needs from the runs
    // ahead of its own is where the last token started.
    __shared__ int last_head[kSortWarps];
    const unsigned long long* key = (a.passes & 1) ? a.p.buf0 : a.p.buf1;
    const Run run(M, me, warps);
    unsigned long long k[kSortBlock];
    unsigned heads[kSortBlock];  // lanes whose key starts a token
    unsigned after;              // row of the key after the block
    auto fetch = [&](int64_t i0) {
        unsigned before = ~0u;  // row of the key ahead of the block
        after = ~0u;
#pragma unroll
        for (int r = 0; r < kSortBlock; ++r) {
            const int64_t i = i0 + r * 32 + lane;
            k[r] = i < M ? __ldcg(key + i) : ~0ull;
        }
        if (i0 > 0) before = static_cast<unsigned>(__ldcg(key + i0 - 1) >> 32);
        if (i0 + 32 * kSortBlock < M)
            after = static_cast<unsigned>(__ldcg(key + i0 + 32 * kSortBlock) >> 32);
#pragma unroll
        for (int r = 0; r < kSortBlock; ++r) {
            const unsigned row = static_cast<unsigned>(k[r] >> 32);
            const unsigned up = __shfl_up_sync(0xffffffffu, row, 1);
            const unsigned prev = lane == 0 ? before : up;
            heads[r] = __ballot_sync(0xffffffffu, i0 + r * 32 + lane < run.end && row != prev);
            before = __shfl_sync(0xffffffffu, row, 31);
        }
    };
    int last = -1;
    for (int64_t i0 = run.beg; i0 < run.end; i0 += 32 * kSortBlock) {
        fetch(i0);
#pragma unroll
        for (int r = 0; r < kSortBlock; ++r)
            if (heads[r]) last = static_cast<int>(i0) + r * 32 + 31 - __clz(heads[r]);
    }
    if (lane == 0) last_head[warp] = last;
    __syncthreads();
    cluster_barrier();
    int head = -1;  // of the token that the run may start inside
    static_assert(kSortCtas * kSortWarps % 32 == 0, "whole warps");
#pragma unroll
    for (int r = 0; r < kSortCtas * kSortWarps / 32; ++r) {
        const int w = r * 32 + lane;
        const int h = ld_cluster(last_head + w % kSortWarps, w / kSortWarps);
        if (w < me) head = max(head, h);
    }
    head = __reduce_max_sync(0xffffffffu, head);
    for (int64_t i0 = run.beg; i0 < run.end; i0 += 32 * kSortBlock) {
        if (!run.kept) fetch(i0);
#pragma unroll
        for (int r = 0; r < kSortBlock; ++r) {
            const int b = static_cast<int>(i0) + r * 32, i = b + lane;
            const unsigned row = static_cast<unsigned>(k[r] >> 32);
            const unsigned down = __shfl_down_sync(0xffffffffu, row, 1);
            const unsigned first = r + 1 < kSortBlock
                                       ? __shfl_sync(0xffffffffu, static_cast<unsigned>(k[r + 1 < kSortBlock ? r + 1 : r] >> 32), 0)
                                       : after;
            const unsigned behind = lane == 31 ? first : down;  // ~0 past the last key
            const unsigned upto = heads[r] & (lt | (1u << lane));
            const int h = upto ? b + 31 - __clz(upto) : head;
            if (i < run.end) {
                const int in = (i - h) % a.K;  // place in its unit
                const bool token_ends = row != behind;
                const bool end = token_ends || in == a.K - 1;
                const bool more = end && (i - h >= a.K || !token_ends);
                a.p.entries[i] = Entry{static_cast<unsigned>(k[r]) | (end ? kTop : 0u),
                                       row | (more ? kTop : 0u)};
                if (i % kWindow == 0) a.p.windows[i / kWindow] = i - in;
                if (token_ends && i - h >= a.K)
                    a.p.longs[atomicAdd(&a.p.head->longs, 1)] =
                        Long{h, i + 1 - h, static_cast<int>(row), 0};
            }
            if (heads[r]) head = b + 31 - __clz(heads[r]);
        }
    }
    if (rank == 0 && tid == 0) {
        a.p.head->valid = static_cast<int>(M);
        a.p.windows[(M + kWindow - 1) / kWindow] = static_cast<int>(M);
    }
    __syncthreads();
    cluster_barrier();  // no CTA leaves while another reads its shared memory
}

// Rows of no token set to +0, by the clusters that do not sort: each takes a
// range of the vocabulary and marks its tokens in a bitmap (each CTA reads a
// share of the tokens; the CTAs' bitmaps are joined as the rows are filled).
__device__ void fill_rows(const SortArgs& a, int64_t cluster, int64_t clusters) {
    unsigned* marks = reinterpret_cast<unsigned*>(sort_smem);
    const int tid = threadIdx.x;
    const uint32_t ctas = cluster_ctas(), rank = cluster_ctarank();
    int64_t range = (a.V + clusters - 1) / clusters;
    range = range < kFillRows ? (range + 31) / 32 * 32 : kFillRows;
    for (int64_t r0 = cluster * range; r0 < a.V; r0 += clusters * range) {
        const int64_t rows = r0 + range < a.V ? range : a.V - r0;
        const int words = static_cast<int>((rows + 31) / 32);
        for (int i = tid; i < words; i += kSortThreads) marks[i] = 0;
        __syncthreads();
        for (int64_t i = int64_t(rank) * kSortThreads + tid; i < a.N; i += ctas * kSortThreads) {
            const int64_t t = a.tokens[i], r = t - a.v0 - r0;
            if (t >= a.v0 && r >= 0 && r < rows) atomicOr(marks + (r >> 5), 1u << (r & 31));
        }
        __syncthreads();
        cluster_barrier();
        // a warp takes a row at a time
        for (int64_t v = int64_t(rank) * kSortWarps + (tid >> 5); v < rows; v += ctas * kSortWarps) {
            int used = 0;
            if ((tid & 31) < ctas)
                used = ld_cluster(reinterpret_cast<const int*>(marks) + (v >> 5), tid & 31);
            if (__ballot_sync(0xffffffffu, used >> (v & 31) & 1)) continue;
            char* p = a.table + (r0 + v) * a.pitch;
            const int64_t vec = reinterpret_cast<uintptr_t>(p) % 16 == 0 ? a.row_bytes / 16 : 0;
#pragma unroll 4
            for (int64_t i = tid & 31; i < vec; i += 32)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
            for (int64_t i = vec * 16 + (tid & 31) * 2; i < a.row_bytes; i += 64)
                *reinterpret_cast<uint16_t*>(p + i) = 0;
        }
        __syncthreads();
        cluster_barrier();  // the bitmaps may be overwritten
    }
}

__global__ void __launch_bounds__(kSortThreads, 2) embed_sort_kernel(const __grid_constant__ SortArgs a) {
    const int64_t cluster = blockIdx.x / cluster_ctas(), clusters = gridDim.x / cluster_ctas();
    if (cluster == 0)
        sort_tokens(a);
    else
        fill_rows(a, cluster - 1, clusters - 1);
}

struct GradArgs {
    int64_t ldg, D, ldw;
    float scale;
    int tiles, K;
    SortPtrs p;
};

constexpr int kGradWarps = 8;

// What is stored for the scaled sum `s` on top of `old`.  + 0: a sum of nothing
// but zeros is +0 whatever the scale's sign.
template <typename TO>
__device__ __forceinline__ TO grad_value(float s, float old) {
    return Elem<TO>::from_f(old + (s + 0.f));
}

// A warp takes a window of the sorted order, whole units of kWindow entries or
// so, and a tile of columns: C packs of E elements a lane.  Its rows lie side
// by side in the sorted order whatever units they belong to, so R of them, and
// the table's row at each unit's end, are in flight together: one add per
// element read is bound by HBM, and most units are one or two rows.
template <typename TI, typename TO, int E, int C, int R, bool ADD>
__global__ void __launch_bounds__(32 * kGradWarps, LL_GC) embed_grad_kernel(
    const TI* __restrict__ g, TO* __restrict__ dW, const __grid_constant__ GradArgs a) {
    const int lane = threadIdx.x & 31;
    const int M = a.p.head->valid;
    const int64_t items = int64_t((M + kWindow - 1) / kWindow) * a.tiles;
    for (int64_t it = blockIdx.x * int64_t(kGradWarps) + (threadIdx.x >> 5); it < items;
         it += int64_t(gridDim.x) * kGradWarps) {
        const int64_t w = it / a.tiles;
        const int64_t c0 = ((it - w * a.tiles) * C * 32 + lane) * E;
        bool has[C];
#pragma unroll
        for (int k = 0; k < C; ++k) has[k] = c0 + k * 32 * E < a.D;
        const int p0 = a.p.windows[w], p1 = a.p.windows[w + 1];
        int start = p0;  // of the unit
        float acc[C][E];
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) acc[k][j] = 0.f;
        for (int b = p0; b < p1; b += 32) {
            Entry mine{0, 0};
            if (b + lane < p1) mine = a.p.entries[b + lane];
            const int n = p1 - b < 32 ? p1 - b : 32;
#pragma unroll 1
            for (int r = 0; r < n; r += R) {
                Pack<TI, E> x[R][C];
                Pack<TO, E> old[R][C];
                const TI* src[R];
                Entry e[R];
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    e[q].pos = __shfl_sync(0xffffffffu, mine.pos, (r + q) & 31);
                    e[q].row = __shfl_sync(0xffffffffu, mine.row, (r + q) & 31);
                    if (r + q < n) {
                        src[q] = g + int64_t(e[q].pos & ~kTop) * a.ldg + c0;
#pragma unroll
                        for (int k = 0; k < C; ++k)
                            if (has[k]) x[q][k].load(src[q] + k * 32 * E);
                        if (ADD && (e[q].pos & kTop) && !(e[q].row & kTop)) {
                            const TO* row = dW + int64_t(e[q].row) * a.ldw + c0;
#pragma unroll
                            for (int k = 0; k < C; ++k)
                                if (has[k]) old[q][k].load(row + k * 32 * E);
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
                    if (!(e[q].pos & kTop)) continue;
                    if (!(e[q].row & kTop)) {
                        TO* row = dW + int64_t(e[q].row) * a.ldw + c0;
#pragma unroll
                        for (int k = 0; k < C; ++k) {
                            Pack<TO, E> y;
#pragma unroll
                            for (int j = 0; j < E; ++j)
                                y.e[j] = grad_value<TO>(a.scale * acc[k][j],
                                                        ADD ? Elem<TO>::to_f(old[q][k].e[j]) : 0.f);
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

// Tokens of several pieces: a block takes 32 packs of columns of one, each warp
// an equal run of its pieces, and the warps' sums are added in order.
template <typename TO, int E, bool ADD>
__global__ void __launch_bounds__(32 * kGradWarps) embed_join_kernel(
    TO* __restrict__ dW, const __grid_constant__ GradArgs a) {
    __shared__ float sums[kGradWarps][32 * E];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tiles = (a.D + 32 * E - 1) / (32 * E);
    const int64_t items = a.p.head->longs * tiles;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const Long l = a.p.longs[it / tiles];
        const int64_t c = (it % tiles * 32 + lane) * E;
        const int n = (l.count + a.K - 1) / a.K;
        const int per = (n + kGradWarps - 1) / kGradWarps;
        const int p0 = warp * per, p1 = p0 + per < n ? p0 + per : n;
        const bool odd = l.count % a.K != 0;
        float s[E];
#pragma unroll
        for (int j = 0; j < E; ++j) s[j] = 0.f;
        if (c < a.D) {
            const float* src = a.p.part + int64_t(l.start / a.K) * 2 * a.p.Dp + c;
#pragma unroll 8
            for (int i = p0; i < p1; ++i) {
                Pack<float, E> x;
                x.load(src + (i * int64_t(2) + (odd && i == n - 1)) * a.p.Dp);
#pragma unroll
                for (int j = 0; j < E; ++j) s[j] += x.e[j];
            }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) sums[warp][j * 32 + lane] = s[j];
        __syncthreads();
        if (warp == 0 && c < a.D) {
            const int used = (n + per - 1) / per;
            TO* row = dW + int64_t(l.row) * a.ldw + c;
            Pack<TO, E> y;
            if (ADD) y.load(row);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                float f = s[j];
                for (int w = 1; w < used; ++w) f += sums[w][j * 32 + lane];
                y.e[j] = grad_value<TO>(a.scale * f, ADD ? Elem<TO>::to_f(y.e[j]) : 0.f);
            }
            y.store(row);
        }
        __syncthreads();
    }
}

// Whole 16-byte packs of rows that start on 16-byte boundaries.
bool grad_vec(const EmbedArgs& a) {
    return a.D % (a.dtype == LL_F32 ? 4 : 8) == 0 && rows16(a.rows, a.ld_rows, a.dtype == LL_F32 ? 4 : 2) &&
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
    const int64_t items = (e.N + kWindow - 1) / kWindow * a.tiles;
    const int64_t most = (items + kGradWarps - 1) / kGradWarps;
    const int64_t full = int64_t(num_sms) * 8;
    const unsigned grid = static_cast<unsigned>(full < most ? full : most);
    const unsigned threads = 32 * kGradWarps;
    const int64_t long_items = e.N / a.K * ((a.D + 127) / 128);
    const unsigned jgrid = static_cast<unsigned>(full < long_items ? full : long_items);
    auto run = [&](auto* sums, auto* join) {
        note_launches(jgrid ? 2 : 1);
        sums<<<grid, threads, 0, s>>>(g, dW, a);
        if (jgrid) join<<<jgrid, threads, 0, s>>>(dW, a);
        return cudaGetLastError();
    };
    if (vec)
        return accumulate
                   ? run(embed_grad_kernel<TI, TO, E, 1, LL_GR, true>, embed_join_kernel<TO, 4, true>)
                   : run(embed_grad_kernel<TI, TO, E, 1, LL_GR, false>, embed_join_kernel<TO, 4, false>);
    return accumulate
               ? run(embed_grad_kernel<TI, TO, 1, C1, LL_GR, true>, embed_join_kernel<TO, 1, true>)
               : run(embed_grad_kernel<TI, TO, 1, C1, LL_GR, false>, embed_join_kernel<TO, 1, false>);
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
static SortPtrs grad_layout(int64_t N, int64_t D, void* ws, size_t* bytes) {
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
    q.buf0 = reinterpret_cast<unsigned long long*>(take(size_t(N) * 8));
    q.buf1 = reinterpret_cast<unsigned long long*>(take(size_t(N) * 8));
    q.entries = reinterpret_cast<Entry*>(take(size_t(N) * sizeof(Entry)));
    q.windows = reinterpret_cast<int*>(take(size_t((N + kWindow - 1) / kWindow + 1) * 4));
    q.longs = reinterpret_cast<Long*>(take(size_t(slots) * sizeof(Long)));
    q.part = reinterpret_cast<float*>(take(size_t(2 * slots) * size_t(q.Dp) * 4));
    *bytes = off;
    return q;
}

size_t embed_bwd_bytes(int64_t N, int64_t D, int64_t V) {
    (void)V;
    size_t bytes;
    grad_layout(N, D, nullptr, &bytes);
    return bytes;
}

static int bits_of(int64_t V) {
    int b = 1;
    while ((int64_t(1) << b) < V) ++b;
    return b;
}

cudaError_t launch_embed_sort(const EmbedArgs& e, int accumulate, void* ws, int num_sms,
                              cudaStream_t s) {
    size_t bytes;
    SortArgs a;
    a.tokens = e.tokens;
    a.N = e.N;
    a.V = e.V;
    a.v0 = e.v0;
    a.bits = bits_of(e.V);
    a.passes = (a.bits + kDigitBits - 1) / kDigitBits;
    a.K = static_cast<int>(piece_rows(e.N));
    a.p = grad_layout(e.N, e.D, ws, &bytes);
    const int64_t es = e.table_dtype == LL_F32 ? 4 : 2;
    a.table = accumulate ? nullptr : static_cast<char*>(e.table);
    a.row_bytes = e.D * es;
    a.pitch = e.ld_table * es;

    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kSortCtas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(accumulate ? kSortCtas : kSortCtas * kFillClusters);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    note_launches(1);
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, a);
}

cudaError_t launch_embed_bwd(const EmbedArgs& e, int accumulate, void* ws, int num_sms,
                             cudaStream_t s) {
    size_t bytes;
    const bool vec = grad_vec(e);
    GradArgs a;
    a.ldg = e.ld_rows;
    a.D = e.D;
    a.ldw = e.ld_table;
    a.scale = e.scale;
    a.tiles = 0;
    a.K = static_cast<int>(piece_rows(e.N));
    a.p = grad_layout(e.N, e.D, ws, &bytes);
    switch (e.dtype * 3 + e.table_dtype) {
        case LL_F32 * 3 + LL_F32: return grad_typed<float, float>(e, vec, accumulate, a, num_sms, s);
        case LL_F16 * 3 + LL_F16: return grad_typed<__half, __half>(e, vec, accumulate, a, num_sms, s);
        case LL_F16 * 3 + LL_F32: return grad_typed<__half, float>(e, vec, accumulate, a, num_sms, s);
        case LL_BF16 * 3 + LL_BF16:
            return grad_typed<__nv_bfloat16, __nv_bfloat16>(e, vec, accumulate, a, num_sms, s);
        default: return grad_typed<__nv_bfloat16, float>(e, vec, accumulate, a, num_sms, s);
    }
}

}  // namespace ll
