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
// need the counts) are what costs, and instructions: 250 per 32 tokens of the
// second pass, whose issue slots are 56% used.  4096 / a million tokens 5.6 / 14.0 us,
// a million in 700 sequences 21.5.
#include <math.h>

#include "step_device.cuh"

namespace ll {
namespace {

constexpr int kThreads = 512;
constexpr int kSlots = 8;                 // tokens of a lane of one plain FP32 sum
constexpr int kSmallCtas = 8;             // CTAs of the one-launch path's cluster
constexpr int kSmallThreads = 512;
constexpr int64_t kSmallTokens = 4096;    // most tokens (and sequences) of the one-launch path

// Sequences of 32 tokens at a time, for a warp that walks along the tokens.
// Its lanes hold the ends of the next 32 sequences; where they are not known
// (the start, or all of them past) the warp searches, 32 probes a step.  The sequence
// of token t is the last b with offs[b] <= t, or -1 if t lies in none; whatever
// the offsets hold, it is in [-1, n_seqs).
struct SeqWalk {
    int base = -2;         // lane l holds the end of sequence base + l; -2: nothing
    int ends = 0;
    bool uniform = false;  // the 32 tokens lie in one sequence
    int b = -1, until = 0;  // that, and its end (0: more than one)

    __device__ __forceinline__ static int offset(const PolicyArgs& a, int64_t i) {
        const int64_t o = a.offs[i];
        return o < 0 ? 0 : o > 0x7fffffff ? 0x7fffffff : static_cast<int>(o);
    }
    __device__ __forceinline__ void load(const PolicyArgs& a, int64_t from, int lane) {
        const int64_t i = from + 1 + lane;
        base = static_cast<int>(from);
        ends = i <= a.n_seqs ? offset(a, i) : 0x7fffffff;
    }
    // How many of the n_seqs + 1 offsets are <= t.
    __device__ static int64_t search(const PolicyArgs& a, int t, int lane) {
        int64_t lo = 0, hi = a.n_seqs + 1;
        while (lo < hi) {
            const int64_t step = (hi - lo + 31) / 32, p = lo + lane * step;
            const int c = __popc(__ballot_sync(0xffffffffu, p < hi && offset(a, p) <= t));
            if (c == 0) break;
            const int64_t at = lo + (c - 1) * step;
            lo = at + 1;
            hi = at + step < hi ? at + step : hi;
        }
        return lo;
    }
    __device__ __forceinline__ int at(const PolicyArgs& a, int t0, int lane) {
        const int t1 = t0 + 31, t = t0 + lane;
        if (t1 < until) return b;  // still inside
        unsigned past = ~0u;  // the start: search
        if (base != -2) past = __ballot_sync(0xffffffffu, ends <= t0);
        if (base == -2 || __shfl_sync(0xffffffffu, ends, 31) <= t1)
            load(a, past == ~0u ? search(a, t0, lane) - 1 : int64_t(base) + __popc(past), lane);
        const unsigned m0 = __ballot_sync(0xffffffffu, ends <= t0);
        const unsigned m1 = __ballot_sync(0xffffffffu, ends <= t1);
        uniform = m0 == m1;
        until = 0;
        int64_t b;
        if (uniform) {
            b = int64_t(base) + __popc(m0);
            until = __shfl_sync(0xffffffffu, ends, __popc(m0) & 31);  // of them all: <= t0
        } else if (m1 != ~0u) {
            int n = 0;  // ends <= t
#pragma unroll
            for (int s = 16; s > 0; s >>= 1)
                if (__shfl_sync(0xffffffffu, ends, n + s - 1) <= t) n += s;
            b = int64_t(base) + n;
        } else {  // 32 ends or more among 32 tokens
            int64_t lo = 0, hi = a.n_seqs + 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi) >> 1;
                if (offset(a, mid) <= t)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            b = lo - 1;
        }
        this->b = b < a.n_seqs ? static_cast<int>(b) : -1;
        return this->b;
    }
};

// exp(d) - d - 1 and exp(d) - 1.  For small |d| the exponential's rounding alone
// (6e-8) would be more than the first (d^2 / 2), so there it is d^2 times the
// Taylor polynomial of (e^d - 1 - d) / d^2 up to d^9 (below 2^-27 of it left out),
// and the second is that and d.
struct Exp {
    float rest2, rest1;
};
__device__ __forceinline__ Exp exp_rests(float d) {
    if (fabsf(d) >= 1.f) {
        const float e = expf(d);
        return {e - d - 1.f, e - 1.f};
    }
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
    q = d * d * q;
    return {q, d + q};
}

// Whether x - y lies above a border given to about 48 bits: s, the rounded
// difference, and what its rounding left (Knuth's two-sum), against the border's
// two parts.  (In
// FP64 next to the border only, the compiler still ran the conversions for every
// token: that unit was 61% busy.)
__device__ __forceinline__ bool above(float s, float x, float y, Pair border) {
    const float t = __fsub_rn(s, x);
    const float e = __fsub_rn(__fsub_rn(x, __fsub_rn(s, t)), __fadd_rn(y, t));
    const float rest = finite_or_0(__fsub_rn(e, border.lo), s);
    return __fadd_rn(__fsub_rn(s, border.hi), rest) > 0.f;
}

struct Token {
    float p, k, grad;  // policy part, divergence, unweighted gradient
    bool clipped;
};

__device__ __forceinline__ Token token_loss(const PolicyArgs& a, float logp, float old, float ref,
                                            float A) {
    Token t;
    // below the lower border: above it with the signs turned
    const bool up = A > 0.f;
    const float x = up ? logp : old, y = up ? old : logp, s = x - y;
    t.clipped = above(s, x, y, {up ? a.log_hi[0] : -a.log_lo[0], up ? a.log_hi[1] : -a.log_lo[1]}) &&
                (up || A < 0.f);
    const float r = expf(up ? s : -s);
    const float pg = A == 0.f ? 0.f : -A * r;
    t.p = t.clipped ? -A * (up ? a.bound_hi : a.bound_lo) : pg;
    t.grad = t.clipped ? 0.f : pg;
    t.k = 0.f;
    if (a.ref) {
        const Exp e = exp_rests(ref - logp);
        t.k = e.rest2;
        if (a.beta != 0.f) t.grad -= a.beta * e.rest1;
    }
    return t;
}

// Groups of 32 tokens of warp `me` of `warps`: a run, so that a warp walks
// along the sequences.
struct Groups {
    int beg, end;
    __device__ Groups(int64_t N, int me, int warps) {
        const int all = static_cast<int>((N + 31) / 32), per = (all + warps - 1) / warps;
        beg = static_cast<int>(min(int64_t(me) * per, int64_t(all)));
        end = min(beg + per, all);
    }
};

__device__ __forceinline__ bool unmasked(const PolicyArgs& a, int t) {
    return t < a.N && (!a.mask || a.mask[t]);
}

// Unmasked tokens of a warp's groups (no sequences).
__device__ __forceinline__ int count_tokens(const PolicyArgs& a, const Groups& g) {
    int n = 0;
#pragma unroll 4
    for (int i = g.beg; i < g.end; ++i) n += unmasked(a, i * 32 + (threadIdx.x & 31));
    return __reduce_add_sync(0xffffffffu, n);
}

// Unmasked tokens per sequence, and sequences that have one.  Integer atomics:
// the same counts in any order.  cleared() is called ahead of every one of them.
template <typename F>
__device__ __forceinline__ void count_sequences(const PolicyArgs& a, const Groups& g, const F& cleared,
                                                PolicyWs* __restrict__ ws,
                                                int* __restrict__ seq_count) {
    const int lane = threadIdx.x & 31;
    SeqWalk walk;
    int held = -1, count = 0;  // not yet added
    auto flush = [&]() {
        cleared();
        if (count && lane == 0 && atomicAdd(seq_count + held, count) == 0)
            atomicAdd(&ws->full, 1ull);
        count = 0;
    };
    bool ahead = unmasked(a, g.beg * 32 + lane), ahead2 = unmasked(a, g.beg * 32 + 32 + lane);
#pragma unroll 1
    for (int i = g.beg; i < g.end; ++i) {
        const bool in = ahead;  // the masks of two groups are on their way
        ahead = ahead2;
        ahead2 = unmasked(a, i * 32 + 64 + lane);
        const int b = walk.at(a, i * 32, lane);
        if (walk.uniform) {
            const unsigned m = __ballot_sync(0xffffffffu, in && b >= 0);
            if (b != held && count) flush();
            held = b;
            count += __popc(m);
        } else {
            // one lane adds for all of its sequence
            const int s = in ? b : -1;
            const unsigned peers = __match_any_sync(0xffffffffu, s);
            cleared();
            if (s >= 0 && lane == __ffs(peers) - 1 && atomicAdd(seq_count + s, __popc(peers)) == 0)
                atomicAdd(&ws->full, 1ull);
        }
    }
    flush();
}

// x times the weight w.
__device__ __forceinline__ Pair times(float x, Pair w) {
    const float p = __fmul_rn(x, w.hi);
    return {p, finite_or_0(fmaf(x, w.lo, fmaf(x, w.hi, -p)), p)};
}

// one / c: an FP32 quotient and its remainder's.
__device__ __forceinline__ Pair per_token(Pair one, int c) {
    const float n = static_cast<float>(c), rest = static_cast<float>(c - static_cast<int>(n));
    const float q = __fdiv_rn(one.hi, n);
    return {q, __fdiv_rn(fmaf(-q, n, one.hi) + one.lo - q * rest, n)};
}

// Gradients of a warp's groups; adds to s[0..2] the lane's share of the sums.
// FP32 sums, unweighted, are over kSlots tokens of one sequence at most.  The
// next group's tokens and its sequence's count are loaded ahead, the first's ahead
// of `counted`, which gives 1 / denominator, and of `ready`, which waits for the
// counts; the loop is kept small, since in a short call its instructions are
// fetched cold.
template <typename R, typename F>
__device__ __forceinline__ void loss_tokens(const PolicyArgs& a, const R& ready, const F& counted,
                                            const int* __restrict__ seq_count, const Groups& g,
                                            Pair (&s)[3]) {
    const int lane = threadIdx.x & 31;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    bool in = false;
    auto fetch = [&](int i) {
        const int t = i * 32 + lane;
        in = i < g.end && unmasked(a, t);
        if (!in) return;
        x[0] = a.logp[t];
        x[1] = a.old[t];
        if (a.ref) x[2] = a.ref[t];
        x[3] = a.adv[t];
    };
    fetch(g.beg);
    SeqWalk walk;
    int b = -1, c = 0;  // sequence and its tokens
    auto follow = [&](int i) {
        if (a.offs && i < g.end) b = walk.at(a, i * 32, lane);
    };
    auto tokens_of = [&]() { c = b >= 0 ? __ldcg(seq_count + b) : 0; };
    follow(g.beg);
    ready();
    tokens_of();
    const Pair one = counted();
    int held = -1, slots = 0;
    Pair w = a.offs ? Pair{0.f, 0.f} : one;
    float f[3] = {0.f, 0.f, 0.f};
    auto flush = [&]() {
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            s[j] = add(s[j], times(f[j], w));
            f[j] = 0.f;
        }
        slots = 0;
    };
#pragma unroll 1
    for (int i = g.beg; i < g.end; ++i) {
        const float logp = x[0], old = x[1], ref = x[2], adv = x[3];
        bool use = in;
        fetch(i + 1);
        const int t = i * 32 + lane;
        if (a.offs) {
            if (b != held) {
                if (held >= 0) flush();
                held = b;
                w = c > 0 ? per_token(one, c) : Pair{0.f, 0.f};
            }
            if (b < 0) use = false;
            follow(i + 1);
            if (b != held) tokens_of();
        }
        float grad = 0.f;
        if (use) {
            const Token k = token_loss(a, logp, old, ref, adv);
            grad = w.hi * k.grad + 0.f;
            f[0] += k.p;
            f[1] += k.k;
            f[2] += k.clipped ? 1.f : 0.f;
        }
        if (t < a.N) a.grad[t] = grad;
        if (++slots == kSlots) flush();
    }
    flush();
}

// Sums of a warp's s[0..2]: lane 0 gets the first, 16 the second, 8 the third.  The
// lanes share out the values as they go: 6 additions instead of 15.
__device__ __forceinline__ Pair warp_sums(const Pair (&s)[3]) {
    auto other = [](Pair x, int o) {
        return Pair{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
    };
    const bool b16 = threadIdx.x & 16, b8 = threadIdx.x & 8;
    Pair x = add(b16 ? s[1] : s[0], other(b16 ? s[0] : s[1], 16));
    const Pair third = add(s[2], other(s[2], 16));
    x = add(b8 ? third : x, other(b8 ? x : third, 8));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) x = add(x, other(x, o));
    return x;
}

// Sums of the block's s[0..2] in out[0..2], by a fixed tree.
template <int kBlock>
__device__ void block_sums(Pair (&s)[3], Pair* out) {
    __shared__ Pair all[3][kBlock / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    const Pair mine = warp_sums(s);
    if (lane == 0 || lane == 8 || lane == 16) all[lane == 0 ? 0 : lane == 16 ? 1 : 2][warp] = mine;
    __syncthreads();
    if (warp < 3) {
        const Pair x = warp_sum(lane < kBlock / 32 ? all[warp][lane] : Pair{0.f, 0.f});
        if (lane == 0) out[warp] = x;
    }
}

// 1 / denominator, of `counted` tokens or sequences where it is not given.
__device__ __forceinline__ Pair weight(const PolicyArgs& a, unsigned long long counted) {
    const double n = a.denominator > 0 ? a.denominator : static_cast<double>(counted);
    return n > 0 ? pair_of(1.0 / n) : Pair{0.f, 0.f};
}

__device__ __forceinline__ Pair load_pair(const PolicyWs* ws, int i) {
    const float2 x = __ldcg(&ws->part[i]);
    return {x.x, x.y};
}

__device__ __forceinline__ void write_stats(const PolicyArgs& a, const Pair* s) {
    const double p = double(s[0].hi) + s[0].lo, k = double(s[1].hi) + s[1].lo;
    // without a weight the divergence is watched only: 0 times an infinite one is NaN
    a.stats[0] = static_cast<float>(a.beta != 0.f ? p + a.beta_d * k : p);
    a.stats[1] = s[0].hi;
    a.stats[2] = s[1].hi;
    a.stats[3] = s[2].hi;
}

__device__ __forceinline__ Groups grid_groups(const PolicyArgs& a) {
    return Groups(a.N, blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32));
}

__global__ void __launch_bounds__(kThreads) policy_clear_kernel(PolicyWs* __restrict__ ws,
                                                                int* __restrict__ seq_count,
                                                                int64_t n_seqs) {
    launch_dependents();
    const int64_t i = blockIdx.x * int64_t(kThreads) + threadIdx.x;
    if (i == 0) ws->full = 0;
    if (i < n_seqs) seq_count[i] = 0;
}

__global__ void __launch_bounds__(kThreads) policy_count_kernel(const __grid_constant__ PolicyArgs a,
                                                                PolicyWs* __restrict__ ws,
                                                                int* __restrict__ seq_count) {
    const Groups g = grid_groups(a);
    launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) ws->done = 0;
    if (a.offs) {
        count_sequences(a, g, [] { wait_for_prerequisites(); }, ws, seq_count);
        wait_for_prerequisites();  // of every block, so that the next kernel's wait is for both
    } else {
        __shared__ int all;
        if (threadIdx.x == 0) all = 0;
        __syncthreads();
        const int n = count_tokens(a, g);
        if (n && (threadIdx.x & 31) == 0) atomicAdd(&all, n);
        __syncthreads();
        if (threadIdx.x == 0) ws->tokens[blockIdx.x] = all;
    }
}

__global__ void __launch_bounds__(kThreads, 2) policy_loss_kernel(const __grid_constant__ PolicyArgs a,
                                                                  PolicyWs* __restrict__ ws,
                                                                  const int* __restrict__ seq_count) {
    __shared__ bool last;
    __shared__ Pair one;
    Pair s[3] = {};
    loss_tokens(
        a, [] { wait_for_prerequisites(); },
        [&]() {
            if (threadIdx.x < 32) {
                unsigned long long n = 0;
                if (a.offs) {
                    n = ws->full;
                } else {
                    int c = 0;  // of up to ten blocks, each of fewer than 2^31 / gridDim.x tokens
                    for (unsigned i = threadIdx.x; i < gridDim.x; i += 32) c += ws->tokens[i];
                    n = __reduce_add_sync(0xffffffffu, c);
                }
                if (threadIdx.x == 0) one = weight(a, n);
            }
            __syncthreads();
            return one;
        },
        seq_count, grid_groups(a), s);
    block_sums<kThreads>(s, reinterpret_cast<Pair*>(ws->part) + 3 * blockIdx.x);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&ws->done, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
#pragma unroll
    for (int j = 0; j < 3; ++j)
        s[j] = threadIdx.x < gridDim.x ? load_pair(ws, 3 * threadIdx.x + j) : Pair{0.f, 0.f};
    static_assert(kPolicyBlocks <= kThreads, "a thread per partial sum");
    __shared__ Pair sums[3];
    block_sums<kThreads>(s, sums);
    __syncthreads();
    if (threadIdx.x == 0) write_stats(a, sums);
}

// Both passes, and the clearing of the counts, in one cluster: few tokens are
// bound by the launches, not by what eight SMs can do.
__global__ void __cluster_dims__(kSmallCtas, 1, 1) __launch_bounds__(kSmallThreads)
    policy_small_kernel(const __grid_constant__ PolicyArgs a, PolicyWs* __restrict__ ws,
                        int* __restrict__ seq_count) {
    __shared__ Pair one;
    __shared__ int warp_tokens[kSmallThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Groups g(a.N, blockIdx.x * (kSmallThreads / 32) + warp, kSmallCtas * (kSmallThreads / 32));
    if (a.offs) {
        for (int64_t i = blockIdx.x * kSmallThreads + threadIdx.x; i < a.n_seqs;
             i += kSmallCtas * kSmallThreads)
            seq_count[i] = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) ws->full = 0;
        __syncthreads();
        cluster_barrier();
        count_sequences(a, g, [] {}, ws, seq_count);
        __syncthreads();
        cluster_barrier();
        if (threadIdx.x == 0) one = weight(a, __ldcg(&ws->full));
    } else {
        const int n = count_tokens(a, g);
        if (lane == 0) warp_tokens[warp] = n;
        __syncthreads();
        cluster_barrier();
        if (warp == 0) {
            int all = 0;
#pragma unroll
            for (int i = 0; i < kSmallCtas * (kSmallThreads / 32) / 32; ++i) {
                const int w = i * 32 + lane;
                int c;
                asm volatile("ld.shared::cluster.s32 %0, [%1];"
                             : "=r"(c)
                             : "r"(cluster_addr(warp_tokens + w % (kSmallThreads / 32),
                                                w / (kSmallThreads / 32))));
                all += c;
            }
            all = __reduce_add_sync(0xffffffffu, all);
            if (lane == 0) one = weight(a, all);
        }
    }
    __syncthreads();
    Pair s[3] = {};
    loss_tokens(a, [] {}, [&]() { return one; }, seq_count, g, s);
    block_sums<kSmallThreads>(s, reinterpret_cast<Pair*>(ws->part) + 3 * blockIdx.x);
    __syncthreads();
    cluster_barrier();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        for (int j = 0; j < 3; ++j) {
            s[j] = load_pair(ws, j);
            for (int i = 1; i < kSmallCtas; ++i) s[j] = add(s[j], load_pair(ws, 3 * i + j));
        }
        write_stats(a, s);
    }
}

}  // namespace

size_t policy_ws_bytes(int64_t n_seqs) { return sizeof(PolicyWs) + size_t(n_seqs) * 4; }

cudaError_t launch_policy_loss(const PolicyArgs& a, void* workspace, cudaStream_t s) {
    PolicyWs* ws = static_cast<PolicyWs*>(workspace);
    int* seq_count = reinterpret_cast<int*>(ws + 1);
    if (a.N <= kSmallTokens && a.n_seqs <= kSmallTokens) {
        note_launches(1);
        policy_small_kernel<<<kSmallCtas, kSmallThreads, 0, s>>>(a, ws, seq_count);
        return cudaGetLastError();
    }
    const int64_t blocks = (a.N + kThreads - 1) / kThreads;
    const unsigned grid = static_cast<unsigned>(blocks < kPolicyBlocks ? blocks : kPolicyBlocks);
    note_launches(a.offs ? 3 : 2);
    if (a.offs) {
        const int64_t clear = (a.n_seqs + kThreads - 1) / kThreads;
        policy_clear_kernel<<<static_cast<unsigned>(clear), kThreads, 0, s>>>(ws, seq_count, a.n_seqs);
        const cudaError_t e = launch_after(policy_count_kernel, grid, kThreads, s, 0, a, ws, seq_count);
        if (e != cudaSuccess) return e;
    } else {
        policy_count_kernel<<<grid, kThreads, 0, s>>>(a, ws, seq_count);
    }
    return launch_after(policy_loss_kernel, grid, kThreads, s, 0, a, ws,
                        static_cast<const int*>(seq_count));
}

}  // namespace ll
