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
// A block per vocabulary row: the row's occurrences (ascending position, from
// the sorted tokens) added by each thread for its columns.
template <typename TI, typename TO>
__global__ void __launch_bounds__(256) embed_bwd_kernel(
    const TI* __restrict__ g, int64_t ldg, const int64_t* __restrict__ keys,
    const int* __restrict__ offs, int64_t D, int64_t V, float scale, int accumulate,
    TO* __restrict__ dW, int64_t ldw) {
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
        const int beg = offs[v], end = offs[v + 1];
        if (accumulate && beg == end) continue;
        for (int64_t c = threadIdx.x; c < D; c += blockDim.x) {
            float acc = 0.f;
            for (int i = beg; i < end; ++i)
                acc += Elem<TI>::to_f(g[(keys[i] & 0xffffffffll) * ldg + c]);
            acc = scale * acc + 0.f;
            if (accumulate) acc += Elem<TO>::to_f(dW[v * ldw + c]);
            dW[v * ldw + c] = Elem<TO>::from_f(acc);
        }
    }
}

template <typename TI, typename TO>
cudaError_t bwd_typed(const EmbedArgs& a, const int64_t* keys, const int* offs, int accumulate,
                      cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(a.V < 65536 ? a.V : 65536);
    embed_bwd_kernel<TI, TO><<<grid, 256, 0, s>>>(
        static_cast<const TI*>(a.rows), a.ld_rows, keys, offs, a.D, a.V, a.scale, accumulate,
        static_cast<TO*>(a.table), a.ld_table);
    return cudaGetLastError();
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

size_t embed_bwd_bytes(int64_t N, int64_t D, int64_t V) {
    (void)D;
    return up256(size_t(N) * 8) + up256(token_sort_bytes(N)) + up256(size_t(V + 1) * 4);
}

cudaError_t launch_embed_sort(const EmbedArgs& a, void* ws, cudaStream_t s) {
    char* p = static_cast<char*>(ws);
    int64_t* local = reinterpret_cast<int64_t*>(p);
    int64_t* keys = reinterpret_cast<int64_t*>(p + up256(size_t(a.N) * 8));
    int* offs = reinterpret_cast<int*>(p + up256(size_t(a.N) * 8) + up256(token_sort_bytes(a.N)));
    cudaError_t e = launch_localize_targets(a.tokens, a.N, a.v0, a.V, a.v0 + a.V, local, nullptr, s);
    if (e != cudaSuccess) return e;
    return launch_token_sort(local, a.N, a.V, keys, offs, s);
}

cudaError_t launch_embed_bwd(const EmbedArgs& a, int accumulate, void* ws, cudaStream_t s) {
    note_launches(1);
    char* p = static_cast<char*>(ws);
    const int64_t* keys = reinterpret_cast<const int64_t*>(p + up256(size_t(a.N) * 8));
    const int* offs =
        reinterpret_cast<const int*>(p + up256(size_t(a.N) * 8) + up256(token_sort_bytes(a.N)));
    switch (a.dtype * 3 + a.table_dtype) {
        case LL_F32 * 3 + LL_F32: return bwd_typed<float, float>(a, keys, offs, accumulate, s);
        case LL_F16 * 3 + LL_F16: return bwd_typed<__half, __half>(a, keys, offs, accumulate, s);
        case LL_F16 * 3 + LL_F32: return bwd_typed<__half, float>(a, keys, offs, accumulate, s);
        case LL_BF16 * 3 + LL_BF16:
            return bwd_typed<__nv_bfloat16, __nv_bfloat16>(a, keys, offs, accumulate, s);
        default: return bwd_typed<__nv_bfloat16, float>(a, keys, offs, accumulate, s);
    }
}

}  // namespace ll
