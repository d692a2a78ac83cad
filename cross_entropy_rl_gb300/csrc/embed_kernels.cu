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

// ----------------------------------------------------------------- gradient
// Two launches.  The first sorts the tokens (one cluster) and cuts the sorted
// order into units; the second adds up each unit's rows of grad_out.
//
// A unit is at most K sorted positions of one token: a token's occurrences are
// cut every K from its first, so the order of its additions is a function of
// its own occurrences (and of K).  A token of one unit is finished by the warp
// that adds it; the pieces of a longer one are written as FP32 partial sums and
// added, in order, by the warp that finishes last.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;        // CTAs of the sorting cluster
constexpr int kDigitBits = 9;       // most bits of a sorting pass
constexpr int kBins = 1 << kDigitBits;
constexpr int kFillRows = 1 << 19;  // vocabulary rows of one cluster's bitmap

// Positions of a piece: short enough that a token of a third of a large batch
// is spread over the device, and at most 2048 pieces' partial sums are kept.
__host__ __device__ inline int64_t piece_rows(int64_t N) {
    int64_t k = 64;
    while ((N + k - 1) / k > 2048) k *= 2;
    return k;
}

struct SortHead {
    int units;  // units cut from the sorted order
    int valid;  // tokens of the table
};

struct SortPtrs {
    SortHead* head;
    unsigned long long *buf0, *buf1;  // [N] (row << 32 | position)
    int2* units;                      // [N + 1] (first sorted position, piece of its token)
    int* pieces;                      // [ceil(N / K)] pieces of the token that starts there
    int* arrived;                     // [ceil(N / K), tiles]
    float* part;                      // [2 ceil(N / K), Dp] sums of pieces
    int64_t Dp;
};

struct SortArgs {
    const int64_t* tokens;
    int64_t N, V, v0;
    int bits, passes;  // of a row index; sorting passes
    int K;
    int64_t counters;  // entries of `arrived`
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

// Least-significant-digit radix sort by one cluster, stable, so that the
// positions of a token stay ascending.  Each warp owns a run of the keys; a
// pass counts the run's digits (lanes of equal digit found by match, one of
// them adds), scans the counts over warps, CTAs and digits, and writes each
// key to its place.  Tokens outside the table drop out in the first pass.
__device__ void sort_tokens(const SortArgs& a) {
    int* hist = reinterpret_cast<int*>(sort_smem);  // [kSortWarps][bins]
    __shared__ int total[kBins], base[kBins], scan[kSortWarps], grand;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = cluster_ctas(), rank = cluster_ctarank();
    const int64_t warps = int64_t(ctas) * kSortWarps, me = int64_t(rank) * kSortWarps + warp;
    const unsigned lt = (1u << lane) - 1;

    for (int64_t i = int64_t(rank) * kSortThreads + tid; i < a.counters; i += ctas * kSortThreads)
        a.p.arrived[i] = 0;

    int64_t M = a.N;
    int shift = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int db = (a.bits - shift + (a.passes - pass) - 1) / (a.passes - pass);
        const int bins = 1 << db;
        const unsigned long long* src = (pass & 1) ? a.p.buf0 : a.p.buf1;
        unsigned long long* dst = (pass & 1) ? a.p.buf1 : a.p.buf0;
        for (int i = tid; i < kSortWarps * bins; i += kSortThreads) hist[i] = 0;
        __syncthreads();
        const int64_t per = ((M + 31) / 32 + warps - 1) / warps * 32;
        const int64_t beg = me * per < M ? me * per : M;
        const int64_t end = beg + per < M ? beg + per : M;
        int* mine = hist + warp * bins;

        auto key_at = [&](int64_t i, bool& in) -> unsigned long long {
            in = i < end;
            if (!in) return 0;
            if (pass > 0) return __ldcg(src + i);
            const int64_t r = a.tokens[i] - a.v0;
            in = a.tokens[i] >= a.v0 && r < a.V;
            return (static_cast<unsigned long long>(r) << 32) | static_cast<unsigned>(i);
        };
        for (int64_t i0 = beg; i0 < end; i0 += 32) {
            bool in;
            const unsigned long long k = key_at(i0 + lane, in);
            const int d = in ? static_cast<int>(k >> (32 + shift)) & (bins - 1) : -1;
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            if (in && (peers & lt) == 0) mine[d] += __popc(peers);
            __syncwarp();
        }
        __syncthreads();
        if (tid < bins) {  // counts of the warps below, and of the CTA
            int run = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const int c = hist[w * bins + tid];
                hist[w * bins + tid] = run;
                run += c;
            }
            total[tid] = run;
        }
        __syncthreads();
        cluster_barrier();
        int before = 0, all = 0;
        if (tid < bins) {
            for (uint32_t r = 0; r < ctas; ++r) {
                const int c = ld_cluster(total + tid, r);
                if (r < rank) before += c;
                all += c;
            }
        }
        const int low = warp_scan(all, lane);  // digits below, within 32
        if (lane == 31) scan[warp] = low + all;
        __syncthreads();
        if (warp == 0) {
            const int c = scan[lane];
            const int s = warp_scan(c, lane);
            scan[lane] = s;
            if (lane == 31) grand = s + c;
        }
        __syncthreads();
        if (tid < bins) base[tid] = scan[warp] + low + before;
        M = pass == 0 ? grand : M;
        __syncthreads();
        for (int64_t i0 = beg; i0 < end; i0 += 32) {
            bool in;
            const unsigned long long k = key_at(i0 + lane, in);
            const int d = in ? static_cast<int>(k >> (32 + shift)) & (bins - 1) : -1;
            const unsigned peers = __match_any_sync(0xffffffffu, d);
            int at = 0;
            if (in) at = mine[d] + base[d] + __popc(peers & lt);
            __syncwarp();
            if (in) {
                if ((peers & lt) == 0) mine[d] += __popc(peers);
                dst[at] = k;
            }
            __syncwarp();
        }
        shift += db;
        __syncthreads();
        cluster_barrier();  // every key of the pass is in its place
    }

    // Units.  A warp needs, of the runs ahead of it, where the last token
    // started (a run may start inside it) and how many units they hold.
    __shared__ int first_head[kSortWarps], last_head[kSortWarps], count[kSortWarps];
    __shared__ int carry[kSortWarps], offset[kSortWarps];
    const unsigned long long* key = (a.passes & 1) ? a.p.buf0 : a.p.buf1;
    const int64_t per = ((M + 31) / 32 + warps - 1) / warps * 32;
    const int64_t beg = me * per < M ? me * per : M;
    const int64_t end = beg + per < M ? beg + per : M;
    auto is_head = [&](int64_t i) {
        return i < end && (i == 0 || (__ldcg(key + i) >> 32) != (__ldcg(key + i - 1) >> 32));
    };
    int first = -1, last = -1, units = 0;
    for (int64_t i0 = beg; i0 < end; i0 += 32) {
        const int i = static_cast<int>(i0) + lane;
        const unsigned heads = __ballot_sync(0xffffffffu, is_head(i));
        if (first < 0 && heads) first = static_cast<int>(i0) + __ffs(heads) - 1;
        const unsigned upto = heads & (lt | (1u << lane));
        const int h = upto ? static_cast<int>(i0) + 31 - __clz(upto) : last;
        const bool u = i < end && h >= 0 && (i - h) % a.K == 0;
        units += __popc(__ballot_sync(0xffffffffu, u));
        if (heads) last = static_cast<int>(i0) + 31 - __clz(heads);
    }
    if (lane == 0) {
        first_head[warp] = first;
        last_head[warp] = last;
        count[warp] = units;
    }
    __syncthreads();
    cluster_barrier();
    if (warp == 0) {
        // runs in order, one CTA's 32 at a time
        int head = -1, sum = 0;
        for (uint32_t r = 0; r <= rank; ++r) {
            const int f = ld_cluster(first_head + lane, r), l = ld_cluster(last_head + lane, r);
            int c = ld_cluster(count + lane, r);
            int h = l;  // last head at or before this run's end
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, h, o);
                if (lane >= o) h = max(h, y);
            }
            h = max(h, head);
            int in = __shfl_up_sync(0xffffffffu, h, 1);  // the head this run starts inside
            if (lane == 0) in = head;
            const int64_t b = (int64_t(r) * kSortWarps + lane) * per;
            if (b < M && in >= 0) {  // its pieces that start ahead of the run's first head
                const int64_t e0 = b + per < M ? b + per : M;
                const int64_t e = f >= 0 ? f : e0;
                c += static_cast<int>((e - in + a.K - 1) / a.K - (b - in + a.K - 1) / a.K);
            }
            const int s = warp_scan(c, lane);
            if (r == rank) {
                carry[lane] = in;
                offset[lane] = sum + s;
            }
            sum += __shfl_sync(0xffffffffu, s + c, 31);
            head = __shfl_sync(0xffffffffu, h, 31);
        }
        if (rank == ctas - 1 && lane == 0) {
            *a.p.head = SortHead{sum, static_cast<int>(M)};
            a.p.units[sum] = make_int2(static_cast<int>(M), 0);
        }
    }
    __syncthreads();
    int h0 = carry[warp], at = offset[warp];
    for (int64_t i0 = beg; i0 < end; i0 += 32) {
        const int i = static_cast<int>(i0) + lane;
        const unsigned heads = __ballot_sync(0xffffffffu, is_head(i));
        const unsigned upto = heads & (lt | (1u << lane));
        const int h = upto ? static_cast<int>(i0) + 31 - __clz(upto) : h0;
        const bool u = i < end && (i - h) % a.K == 0;
        const unsigned us = __ballot_sync(0xffffffffu, u);
        if (u) a.p.units[at + __popc(us & lt)] = make_int2(i, (i - h) / a.K);
        at += __popc(us);
        if (heads) h0 = static_cast<int>(i0) + 31 - __clz(heads);
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
        // a warp takes 32 rows at a time
        for (int64_t w = int64_t(rank) * kSortWarps + (tid >> 5); w < words; w += ctas * kSortWarps) {
            unsigned used = 0;
            for (uint32_t r = 0; r < ctas; ++r)
                used |= ld_cluster(reinterpret_cast<const int*>(marks) + w, r);
            const int64_t left = rows - w * 32;
            for (int b = 0; b < 32 && b < left; ++b) {
                if (used >> b & 1) continue;
                char* p = a.table + (r0 + w * 32 + b) * a.pitch;
                const int64_t vec = reinterpret_cast<uintptr_t>(p) % 16 == 0 ? a.row_bytes / 16 : 0;
                for (int64_t i = tid & 31; i < vec; i += 32)
                    reinterpret_cast<uint4*>(p)[i] = make_uint4(0, 0, 0, 0);
                for (int64_t i = vec * 16 + (tid & 31) * 2; i < a.row_bytes; i += 64)
                    *reinterpret_cast<uint16_t*>(p + i) = 0;
            }
        }
        __syncthreads();
        cluster_barrier();  // the bitmaps may be overwritten
    }
}

__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ SortArgs a) {
    const int64_t cluster = blockIdx.x / cluster_ctas(), clusters = gridDim.x / cluster_ctas();
    if (cluster == 0)
        sort_tokens(a);
    else
        fill_rows(a, cluster - 1, clusters - 1);
}

// Elements a lane holds of a row: C packs of E, packs of neighbouring lanes
// side by side.
template <typename T, int E>
__device__ __forceinline__ void load_pack(const T* p, int64_t c, int64_t D, float (&f)[E]) {
    if (c + E <= D) {
        Pack<T, E> x;
        x.load(p + c);
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = Elem<T>::to_f(x.e[j]);
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] = c + j < D ? Elem<T>::to_f(p[c + j]) : 0.f;
    }
}

struct GradArgs {
    int64_t ldg, D, ldw;
    float scale;
    int tiles, K;
    const unsigned long long* key;
    SortPtrs p;
};

constexpr int kGradWarps = 8;

template <typename TI, typename TO, int E, int C, bool ADD>
__global__ void __launch_bounds__(32 * kGradWarps) embed_grad_kernel(
    const TI* __restrict__ g, TO* __restrict__ dW, const __grid_constant__ GradArgs a) {
    constexpr int R = 4;  // rows in flight
    const int lane = threadIdx.x & 31;
    const int64_t items = int64_t(a.p.head->units) * a.tiles;
    for (int64_t it = blockIdx.x * int64_t(kGradWarps) + (threadIdx.x >> 5); it < items;
         it += int64_t(gridDim.x) * kGradWarps) {
        const int64_t u = it / a.tiles;
        const int tile = static_cast<int>(it - u * a.tiles);
        const int2 now = a.p.units[u], next = a.p.units[u + 1];
        const int len = next.x - now.x;
        const bool whole = now.y == 0 && next.y == 0;
        const int64_t c0 = (int64_t(tile) * C * 32 + lane) * E;
        TO* row = dW + static_cast<int64_t>(a.key[now.x] >> 32) * a.ldw;

        float old[C][E];
        if (ADD && whole) {
#pragma unroll
            for (int k = 0; k < C; ++k) load_pack<TO, E>(row, c0 + k * 32 * E, a.D, old[k]);
        }
        float acc[C][E];
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int j = 0; j < E; ++j) acc[k][j] = 0.f;
        for (int b = 0; b < len; b += 32) {
            const int n = len - b < 32 ? len - b : 32;
            const unsigned pos = lane < n ? static_cast<unsigned>(a.key[now.x + b + lane]) : 0;
            for (int r = 0; r < n; r += R) {
                float f[R][C][E];
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const unsigned at = __shfl_sync(0xffffffffu, pos, r + q < n ? r + q : r);
                    if (r + q < n) {
#pragma unroll
                        for (int k = 0; k < C; ++k)
                            load_pack<TI, E>(g + at * a.ldg, c0 + k * 32 * E, a.D, f[q][k]);
                    }
                }
#pragma unroll
                for (int q = 0; q < R; ++q)
                    if (r + q < n) {
#pragma unroll
                        for (int k = 0; k < C; ++k)
#pragma unroll
                            for (int j = 0; j < E; ++j) acc[k][j] += f[q][k][j];
                    }
            }
        }
        if (!whole) {
            // The piece's sum goes to its slot: full pieces by K positions, and
            // beside each the short last piece that may start in the same K.
            const int64_t slot = now.x / a.K * int64_t(2) + (len < a.K);
            float* dst = a.p.part + slot * a.p.Dp;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const int64_t c = c0 + k * 32 * E;
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (c + j < a.D) dst[c + j] = acc[k][j];
            }
            // The counter of the token's tile returns to zero with its last
            // piece: the last piece in order takes away what the others add.
            const int h = (now.x - now.y * a.K) / a.K;
            const bool final_piece = next.y == 0;
            __threadfence();
            __syncwarp();
            int left = 0;
            if (lane == 0) {
                if (final_piece) {
                    a.p.pieces[h] = now.y + 1;
                    __threadfence();
                }
                const int d = final_piece ? -now.y : 1;
                left = atomicAdd(a.p.arrived + int64_t(h) * a.tiles + tile, d) + d;
            }
            left = __shfl_sync(0xffffffffu, left, 0);
            if (left != 0) continue;
            __threadfence();
            const int n = __ldcg(a.p.pieces + h);
            const int64_t start = now.x - int64_t(now.y) * a.K;
            // only the last piece can be short; its unit is n - 1 - now.y after this one
            const int2 lp = a.p.units[u + (n - 1 - now.y)], ln = a.p.units[u + (n - now.y)];
            const int short_last = ln.x - lp.x < a.K;
#pragma unroll
            for (int k = 0; k < C; ++k) {
                const int64_t c = c0 + k * 32 * E;
                float s[E];
#pragma unroll
                for (int j = 0; j < E; ++j) s[j] = 0.f;
#pragma unroll 8
                for (int i = 0; i < n; ++i) {
                    const float* src =
                        a.p.part + ((start / a.K + i) * 2 + (i == n - 1 ? short_last : 0)) * a.p.Dp;
#pragma unroll
                    for (int j = 0; j < E; ++j)
                        if (c + j < a.D) s[j] += __ldcg(src + c + j);
                }
#pragma unroll
                for (int j = 0; j < E; ++j) acc[k][j] = s[j];
            }
            if (ADD) {
#pragma unroll
                for (int k = 0; k < C; ++k) load_pack<TO, E>(row, c0 + k * 32 * E, a.D, old[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int64_t c = c0 + k * 32 * E;
            Pack<TO, E> y;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                // + 0: a sum of nothing but zeros is +0 whatever the scale's sign
                const float s = a.scale * acc[k][j] + 0.f;
                y.e[j] = Elem<TO>::from_f(ADD ? old[k][j] + s : s);
            }
            if (c + E <= a.D) {
                y.store(row + c);
            } else {
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (c + j < a.D) row[c + j] = y.e[j];
            }
        }
    }
}

constexpr int kGradPacks = 2;  // packs of a lane (C), 16-byte rows
constexpr int kGradCols = 8;   // columns of a lane otherwise

bool grad_vec(const EmbedArgs& a) {
    return rows16(a.rows, a.ld_rows, a.dtype == LL_F32 ? 4 : 2) &&
           rows16(a.table, a.ld_table, a.table_dtype == LL_F32 ? 4 : 2);
}

int64_t grad_tiles(int64_t D, bool vec, int dtype) {
    const int64_t cols = vec ? 32 * kGradPacks * (dtype == LL_F32 ? 4 : 8) : 32 * kGradCols;
    return (D + cols - 1) / cols;
}

template <typename TI, typename TO>
cudaError_t grad_typed(const EmbedArgs& e, bool vec, int accumulate, const GradArgs& a,
                       int num_sms, cudaStream_t s) {
    constexpr int E = 16 / sizeof(TI);
    const TI* g = static_cast<const TI*>(e.rows);
    TO* dW = static_cast<TO*>(e.table);
    auto run = [&](auto* kernel) {
        int per_sm = 0;
        const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &per_sm, kernel, 32 * kGradWarps, 0);
        if (err != cudaSuccess) return err;
        const int64_t most = (e.N * a.tiles + kGradWarps - 1) / kGradWarps;
        const int64_t grid = int64_t(num_sms) * (per_sm > 0 ? per_sm : 1);
        kernel<<<static_cast<unsigned>(grid < most ? grid : most), 32 * kGradWarps, 0, s>>>(g, dW, a);
        return cudaGetLastError();
    };
    if (vec)
        return accumulate ? run(embed_grad_kernel<TI, TO, E, kGradPacks, true>)
                          : run(embed_grad_kernel<TI, TO, E, kGradPacks, false>);
    return accumulate ? run(embed_grad_kernel<TI, TO, 1, kGradCols, true>)
                      : run(embed_grad_kernel<TI, TO, 1, kGradCols, false>);
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

// Workspace of the gradient.  The counters are sized for the narrower tiles.
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
    q.units = reinterpret_cast<int2*>(take(size_t(N + 1) * 8));
    q.pieces = reinterpret_cast<int*>(take(size_t(slots) * 4));
    q.arrived = reinterpret_cast<int*>(take(size_t(slots) * size_t((D + 255) / 256) * 4));
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
    a.counters = (e.N + a.K - 1) / a.K * grad_tiles(e.D, grad_vec(e), e.dtype);
    const int64_t es = e.table_dtype == LL_F32 ? 4 : 2;
    a.table = accumulate ? nullptr : static_cast<char*>(e.table);
    a.row_bytes = e.D * es;
    a.pitch = e.ld_table * es;

    const int smem = kSortWarps * kBins * 4;
    cudaError_t err = cudaFuncSetAttribute(embed_sort_kernel,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = kSortCtas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(accumulate ? kSortCtas : num_sms / kSortCtas * kSortCtas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    note_launches(1);
    return cudaLaunchKernelEx(&cfg, embed_sort_kernel, a);
}

cudaError_t launch_embed_bwd(const EmbedArgs& e, int accumulate, void* ws, int num_sms,
                             cudaStream_t s) {
    note_launches(1);
    size_t bytes;
    const bool vec = grad_vec(e);
    GradArgs a;
    a.ldg = e.ld_rows;
    a.D = e.D;
    a.ldw = e.ld_table;
    a.scale = e.scale;
    a.tiles = static_cast<int>(grad_tiles(e.D, vec, e.dtype));
    a.K = static_cast<int>(piece_rows(e.N));
    a.p = grad_layout(e.N, e.D, ws, &bytes);
    const int passes = (bits_of(e.V) + kDigitBits - 1) / kDigitBits;
    a.key = (passes & 1) ? a.p.buf0 : a.p.buf1;
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
