// Clipped policy loss over sampled tokens, with its gradient.
//
// Per token (unmasked, advantage A, upstream of nothing: this is the loss):
//   delta = logp - old, r = exp(delta), d = ref - logp
//   p = -min(r A, clamp(r, 1 - lo, 1 + hi) A),  k = exp(d) - d - 1
//   loss = sum w (p + beta k),  grad = w ((clipped ? 0 : -A r) - beta (exp(d) - 1))
// with w = 1 / denominator, or 1 / (tokens of the sequence * denominator).
//
// ~20 FP32 operations and at most 21 bytes per token: a batch of a million
// tokens is 21 MB, so the launches and the two dependent passes (the weights
// need the counts) are what costs.
#include <math.h>

#include "ll_device.cuh"

namespace ll {
namespace {

constexpr int kThreads = 256;

// Sequence of token t: the last b with offs[b] <= t, -1 if t lies in none.
// Whatever the offsets hold, the result is in [-1, n_seqs).
__device__ __forceinline__ int64_t seq_of(const int64_t* __restrict__ offs, int64_t n_seqs,
                                          int64_t t) {
    int64_t lo = 0, hi = n_seqs + 1;  // first index with offs > t
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (offs[mid] <= t)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo - 1 < n_seqs ? lo - 1 : -1;
}

// exp(d) - d - 1.  For small |d| the exponential's rounding alone (6e-8) would
// be more than the result (d^2 / 2), so there it is d^2 times the Taylor
// polynomial of (e^d - 1 - d) / d^2 up to d^9 (below 2^-34 of it left out).
__device__ __forceinline__ float exp_rest2(float d) {
    if (fabsf(d) >= 0.5f) return expf(d) - d - 1.f;
    float q = 1.f / 39916800.f;
    q = fmaf(q, d, 1.f / 3628800.f);
    q = fmaf(q, d, 1.f / 362880.f);
    q = fmaf(q, d, 1.f / 40320.f);
    q = fmaf(q, d, 1.f / 5040.f);
    q = fmaf(q, d, 1.f / 720.f);
    q = fmaf(q, d, 1.f / 120.f);
    q = fmaf(q, d, 1.f / 24.f);
    q = fmaf(q, d, 1.f / 6.f);
    q = fmaf(q, d, 0.5f);
    return d * d * q;
}

// delta against a border held in 64 bits.  The FP32 difference is within 2^-24
// of its magnitude of the exact one, so only a delta next to the border needs
// the 64-bit difference.
__device__ __forceinline__ bool above(float delta, float a, float b, double border) {
    const float f = static_cast<float>(border);
    if (fabsf(delta - f) > 1e-6f * (1.f + fabsf(f))) return delta > f;
    return static_cast<double>(a) - static_cast<double>(b) > border;
}
__device__ __forceinline__ bool below(float delta, float a, float b, double border) {
    const float f = static_cast<float>(border);
    if (fabsf(delta - f) > 1e-6f * (1.f + fabsf(f))) return delta < f;
    return static_cast<double>(a) - static_cast<double>(b) < border;
}

struct Token {
    float p, k, grad;  // policy part, divergence, unweighted gradient
    bool clipped;
};

__device__ __forceinline__ Token token_loss(const PolicyArgs& a, float logp, float old, float ref,
                                            float A) {
    Token t;
    const float delta = logp - old;
    t.clipped = A > 0.f ? above(delta, logp, old, a.log_hi)
                        : (A < 0.f && below(delta, logp, old, a.log_lo));
    const float r = expf(delta);
    const float pg = A == 0.f ? 0.f : -A * r;
    t.p = t.clipped ? -A * (A > 0.f ? a.bound_hi : a.bound_lo) : pg;
    t.grad = t.clipped ? 0.f : pg;
    t.k = 0.f;
    if (a.ref) {
        const float d = ref - logp;
        t.k = exp_rest2(d);
        if (a.beta != 0.f) t.grad -= a.beta * expm1f(d);
    }
    return t;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Counts: unmasked tokens (in a sequence), per sequence, and sequences that
// have one.  Integer atomics: the same counts in any order.
__global__ void __launch_bounds__(kThreads) policy_count_kernel(const __grid_constant__ PolicyArgs a,
                                                                PolicyWs* __restrict__ ws,
                                                                int* __restrict__ seq_count) {
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    unsigned long long mine = 0;
    for (int64_t t = blockIdx.x * int64_t(kThreads) + threadIdx.x; t < a.N; t += stride) {
        if (a.mask && !a.mask[t]) continue;
        if (a.offs) {
            const int64_t b = seq_of(a.offs, a.n_seqs, t);
            if (b < 0) continue;
            if (atomicAdd(seq_count + b, 1) == 0) atomicAdd(&ws->full, 1ull);
        }
        ++mine;
    }
    if (mine) atomicAdd(&ws->tokens, mine);
}

__global__ void __launch_bounds__(kThreads) policy_loss_kernel(const __grid_constant__ PolicyArgs a,
                                                               PolicyWs* __restrict__ ws,
                                                               const int* __restrict__ seq_count) {
    __shared__ double part[3][kThreads / 32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const double n = a.denominator > 0 ? a.denominator
                                       : static_cast<double>(a.offs ? ws->full : ws->tokens);
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    double sp = 0, sk = 0, sc = 0;
    for (int64_t t = blockIdx.x * int64_t(kThreads) + threadIdx.x; t < a.N; t += stride) {
        int64_t b = 0;
        bool in = !a.mask || a.mask[t];
        if (in && a.offs) {
            b = seq_of(a.offs, a.n_seqs, t);
            in = b >= 0;
        }
        if (!in) {
            a.grad[t] = 0.f;
            continue;
        }
        const double dw = 1.0 / (a.offs ? n * seq_count[b] : n);
        const float w = static_cast<float>(dw);
        const Token k = token_loss(a, a.logp[t], a.old[t], a.ref ? a.ref[t] : 0.f, a.adv[t]);
        a.grad[t] = w * k.grad + 0.f;
        sp += dw * k.p;
        sk += dw * k.k;
        sc += k.clipped ? dw : 0.0;
    }
    sp = warp_sum(sp);
    sk = warp_sum(sk);
    sc = warp_sum(sc);
    if (lane == 0) {
        part[0][warp] = sp;
        part[1][warp] = sk;
        part[2][warp] = sc;
    }
    __syncthreads();
    if (threadIdx.x < 3) {
        double s = 0;
        for (int i = 0; i < kThreads / 32; ++i) s += part[threadIdx.x][i];
        ws->part[3 * blockIdx.x + threadIdx.x] = s;
        __threadfence();
    }
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&ws->done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last || threadIdx.x >= 32) return;
    __threadfence();
    double s[3] = {0, 0, 0};
    for (unsigned i = lane; i < gridDim.x; i += 32)
#pragma unroll
        for (int j = 0; j < 3; ++j) s[j] += __ldcg(&ws->part[3 * i + j]);
#pragma unroll
    for (int j = 0; j < 3; ++j) s[j] = warp_sum(s[j]);
    if (lane == 0) {
        a.stats[0] = static_cast<float>(s[0] + a.beta_d * s[1]);
        a.stats[1] = static_cast<float>(s[0]);
        a.stats[2] = static_cast<float>(s[1]);
        a.stats[3] = static_cast<float>(s[2]);
    }
}

}  // namespace

size_t policy_ws_bytes(int64_t n_seqs) { return sizeof(PolicyWs) + size_t(n_seqs) * 4; }

cudaError_t launch_policy_loss(const PolicyArgs& a, void* workspace, cudaStream_t s) {
    PolicyWs* ws = static_cast<PolicyWs*>(workspace);
    int* seq_count = reinterpret_cast<int*>(ws + 1);
    note_launches(2);
    cudaError_t e = cudaMemsetAsync(ws, 0, policy_ws_bytes(a.n_seqs), s);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (a.N + kThreads - 1) / kThreads;
    const unsigned grid = static_cast<unsigned>(blocks < kPolicyBlocks ? blocks : kPolicyBlocks);
    policy_count_kernel<<<grid, kThreads, 0, s>>>(a, ws, seq_count);
    policy_loss_kernel<<<grid, kThreads, 0, s>>>(a, ws, seq_count);
    return cudaGetLastError();
}

}  // namespace ll
