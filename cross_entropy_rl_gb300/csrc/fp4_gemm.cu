// Logits from 4-bit operands on the block-scaled tensor cores (tcgen05.mma with E2M1
// operands, FP32 accumulators in TMEM).
//
// A stage holds 256 columns of K: 128 bytes of codes a row, 128-byte swizzled by TMA, and
// the scales of those columns as they lie in memory, tiles of 512 bytes: row r's 16 bytes are
// 4 TMEM columns of lane r, the order in which the MMA reads them.  Four warps bring them
// there, each the same to its own 32 lanes: a tcgen05.cp of 512 bytes keeps the tensor pipe
// as long as an MMA does, and 12 go with 4 MMAs of a pair (2048 x 4096 x 151936: 914 us
// with copies; the product of 48 tokens 90).  The scales of a stage have TMEM columns of their own: they are
// written again only when the stage is, after the MMAs that read them.
//
// Many tokens (pair_kernel): 256 tokens x 256 vocabulary entries by a pair of CTAs
// (cta_group::2): each holds 128 rows of either operand, and the accumulator's rows of its
// own tokens, as rows of the output.  With the scales there is room for one accumulator
// in TMEM: eight warps empty it into registers before the next tile's MMAs begin.
// 4096 x 2048 x 32768 (mx) 124 us, 2048 x 4096 x 151936 (nv) 532: 4.4 and 4.8 PFLOP/s.  Of the
// first's time the tensor pipe is active 45%; L2 moves 1.42 GB (11 TB/s), 0.27 of them the output, and
// no MMA runs while the accumulator is emptied.
// Few tokens (few_kernel): the 128 rows of a tile are vocabulary entries, the columns
// tokens, so that no tensor work is spent on padding tokens and a warp's store of one
// column is 32 neighbouring logits of a token.  The weights are read once: bound by memory
// (48 x 4096 x 151936: 71 us, 4.9 TB/s).
#include <string.h>

#include <mutex>

#include "fp4_device.cuh"
#include "loads_device.cuh"

namespace ll {
namespace {

constexpr int kBKb = 128;                  // bytes of codes of a row in a stage: 256 columns
constexpr int kTileBytes = 128 * kBKb;     // codes of 128 rows
constexpr int kThreadsG = 320;  // producer, MMA issuer, 4 epilogue warps, 4 for the scales
constexpr int kTmem = 512;
constexpr int kMaxStages = 8;
constexpr int kSmemMax = 227 * 1024;

template <int FORMAT>
struct Fmt {
    static constexpr int kTilesPerStage = FORMAT == LL_FP4_MX ? 2 : 4;  // tiles of scales
    static constexpr int kScaleBytes = kTilesPerStage * kFp4TileBytes;  // of 128 rows
    static constexpr int kMmasPerTile = FORMAT == LL_FP4_MX ? 2 : 1;
    static constexpr uint32_t idesc(int M, int N) {
        return (1u << 7) | (1u << 10)                          // A, B: E2M1
               | (static_cast<uint32_t>(N >> 3) << 17)         //
               | ((FORMAT == LL_FP4_MX ? 1u : 0u) << 23)       // scales: E8M0 or E4M3
               | (static_cast<uint32_t>(M >> 4) << 24);
    }
};

// D (+)= A B^T over 64 columns, A and B scaled by the block scales in TMEM.  id: the byte of
// the scales' 32-bit cells that the first block's is in (two blocks of 32 an MMA, or four
// of 16).
template <int FORMAT>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                        uint32_t sfa, uint32_t sfb, uint32_t id,
                                        uint32_t accumulate) {
    const uint32_t di = idesc | (id << 4) | (id << 29);
    if constexpr (FORMAT == LL_FP4_MX) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(di), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%4], [%5], p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(di), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    }
}

// 16 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint4 (&v)[4]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
        "r"(v[1].w), "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y),
        "r"(v[3].z), "r"(v[3].w)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ float load_bias(const void* b, int dtype, int64_t v) {
    if (dtype == LL_F32) return static_cast<const float*>(b)[v];
    if (dtype == LL_F16) return __half2float(static_cast<const __half*>(b)[v]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(b)[v]);
}

struct GemmArgs {
    const uint8_t *h_scales, *w_scales;
    const float *h_scale, *w_scale;
    const void* bias;
    int bias_dtype;
    int64_t N, K, V;
    int64_t k_tiles;  // tiles of scales along K
    void* out;
    int64_t ldo;
    int stages, nt;  // few_kernel: columns of the MMA (tokens, rounded up to 16)
    int wide_out;    // pair_kernel: the output's rows start on 16-byte boundaries
    int* status;
    uint64_t wait_ns;
};

struct BarsFew {
    uint64_t full[kMaxStages], empty[kMaxStages], scaled[kMaxStages];
    uint64_t tfull[2], tempty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

// Tiles of 128 vocabulary entries x all tokens (at most 96), dealt to the CTAs in turn.
template <int FORMAT, typename T>
__global__ void __launch_bounds__(kThreadsG, 1)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH,
               const GemmArgs P) {
    using F = Fmt<FORMAT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ BarsFew bars;
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = P.stages;
    const uint32_t h_bytes = P.nt * kBKb;
    const uint32_t stage_bytes = kTileBytes + h_bytes + 2 * F::kScaleBytes;
    const int64_t k_stages = (P.K + 255) / 256;
    const int64_t tiles = (P.V + 127) / 128;
    volatile int* abort = &bars.abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
            mbar_init(&bars.scaled[s], 4);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars.tfull[b], 1);
            mbar_init(&bars.tempty[b], 4);
        }
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmH);
    }
    if (warp == 1) {
        tmem_alloc(&bars.tmem_base, kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    // TMEM columns: two accumulators of up to 128, then 32 a stage: scales of W, of h
    const uint32_t tscales = tmem + 256;

    if (warp == 0) {
        // ------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0;
        Issued issued;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            for (int64_t kb = 0; kb < k_stages; ++kb) {
                if (!__all_sync(0xffffffffu,
                                mbar_wait(&bars.empty[stage], phase ^ 1, P.wait_ns, abort))) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t* sw = smem + stage * stage_bytes;
                    uint8_t* sh = sw + kTileBytes;
                    uint8_t* ss = sh + h_bytes;
                    uint64_t* bar = &bars.full[stage];
                    const int64_t st0 = kb * F::kTilesPerStage;
                    const uint32_t sb = static_cast<uint32_t>(
                        min(int64_t(F::kTilesPerStage), P.k_tiles - st0) * kFp4TileBytes);
                    mbar_arrive_expect_tx(bar, kTileBytes + h_bytes + 2 * sb);
                    tma_load_2d(sw, &tmW, bar, static_cast<int32_t>(kb * kBKb),
                                static_cast<int32_t>(t * 128));
                    tma_load_2d(sh, &tmH, bar, static_cast<int32_t>(kb * kBKb), 0);
                    bulk_load(ss, P.w_scales + (t * P.k_tiles + st0) * kFp4TileBytes, sb, bar);
                    bulk_load(ss + F::kScaleBytes, P.h_scales + st0 * kFp4TileBytes, sb, bar);
                }
                __syncwarp();
                issued.add(stage, phase);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
        // no load is in flight when the CTA ends, whichever warp gave up
        wait_for_loads(bars.full, issued, P.wait_ns);
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        int stage = 0, buf = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        const uint32_t sbase = smem_u32(smem);
        const uint32_t idesc = F::idesc(128, 0) | (static_cast<uint32_t>(P.nt >> 3) << 17);
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            if (!__all_sync(0xffffffffu,
                            mbar_wait(&bars.tempty[buf], bphase ^ 1, P.wait_ns, abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + buf * 128;
            for (int64_t kb = 0; kb < k_stages; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[stage], phase, P.wait_ns, abort) &&
                                                 mbar_wait(&bars.scaled[stage], phase, P.wait_ns, abort))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) {
                    const uint32_t sw = sbase + stage * stage_bytes, sh = sw + kTileBytes;
                    const uint32_t ts = tscales + stage * 32;
                    const int mmas = static_cast<int>(min(int64_t(4), (P.K - kb * 256 + 63) / 64));
                    for (int i = 0; i < mmas; ++i) {
                        const uint32_t col = 4 * (i / F::kMmasPerTile);
                        const uint32_t id = FORMAT == LL_FP4_MX ? 2 * (i & 1) : 0;
                        mma_fp4<FORMAT>(d, smem_desc_sw128(sw + i * 32, 16, 1024),
                                        smem_desc_sw128(sh + i * 32, 16, 1024), idesc, ts + col,
                                        ts + 16 + col, id, (kb > 0 || i > 0) ? 1u : 0u);
                    }
                    tc_commit(&bars.empty[stage]);
                }
                __syncwarp();
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            if (lane == 0) tc_commit(&bars.tfull[buf]);
            __syncwarp();
            if (++buf == 2) {
                buf = 0;
                bphase ^= 1;
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
        if (lane == 0) tc_commit(&bars.drain);
        __syncwarp();
        mbar_wait(&bars.drain, 0, P.wait_ns, nullptr);
    } else if (warp >= 6) {
        // ------------------------------------------------------- scales to TMEM
        const int q = warp & 3;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            for (int64_t kb = 0; kb < k_stages; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[stage], phase, P.wait_ns, abort))) {
                    ok = false;
                    break;
                }
                const uint8_t* ss = smem + stage * stage_bytes + kTileBytes + h_bytes + lane * 16;
                const uint32_t ts = tscales + stage * 32 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
                for (int m = 0; m < 2; ++m) {  // of W, of h
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = i < F::kTilesPerStage
                                   ? *reinterpret_cast<const uint4*>(ss + m * F::kScaleBytes +
                                                                     i * kFp4TileBytes)
                                   : make_uint4(0, 0, 0, 0);
                    __syncwarp();
                    tmem_st16(ts + 16 * m, v);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.scaled[stage]);
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
    } else {
        // ------------------------------------------------------- epilogue
        const int q = warp & 3;  // TMEM lanes [32 q, 32 q + 32)
        int buf = 0;
        uint32_t bphase = 0;
        bool ok = true;
        ScaleProduct scale = {1.f, 1.f};
        if (FORMAT == LL_FP4_NV) scale = scale_product(*P.h_scale, *P.w_scale);
        const float g = scale.g;
        T* out = static_cast<T*>(P.out);
        for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
            const int64_t v = t * 128 + q * 32 + lane;
            const float b = P.bias && v < P.V ? load_bias(P.bias, P.bias_dtype, v) : 0.f;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars.tfull[buf], bphase, P.wait_ns, abort))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem + buf * 128 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < P.nt; c += 32) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(taddr + c, r);
                tmem_ld_wait(r);
                if (FORMAT == LL_FP4_NV && scale.two != 1.f) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale.two);
                }
                if (v < P.V) {
                    T* o = out + int64_t(c) * P.ldo + v;
                    const int left = static_cast<int>(min(int64_t(32), P.N - c));
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < left)
                            o[int64_t(j) * P.ldo] = Elem<T>::from_f(__uint_as_float(r[j]) * g + b);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.tempty[buf]);
            if (++buf == 2) {
                buf = 0;
                bphase ^= 1;
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmem);
}

// ------------------------------------------------------------- many tokens
constexpr int kPairStages = 5;
constexpr int kPairThreads = 448;  // producer, MMA issuer, 8 epilogue warps, 4 for the scales
constexpr int kOutBuf = 32 * 128;  // a warp's 32 rows of 128 bytes

struct BarsPair {
    uint64_t full[kPairStages];   // leader: both CTAs' tiles landed
    uint64_t empty[kPairStages];  // both: the MMAs are done with the stage
    uint64_t landed[kPairStages];  // each: its scales landed
    uint64_t scaled[kPairStages];  // leader: both CTAs' scales are in TMEM
    uint64_t tfull;               // both: the accumulator is ready
    uint64_t tempty;              // leader: both CTAs' warps have emptied it
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

template <int FORMAT>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t id,
                                             uint32_t accumulate) {
    const uint32_t di = idesc | (id << 4) | (id << 29);
    if constexpr (FORMAT == LL_FP4_MX) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
            "[%5], p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(di), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
            "[%4], [%5], p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(di), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    }
}
// 32 values as T, in words.
template <typename T>
__device__ __forceinline__ void pack32(const float (&v)[32], uint32_t* w) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 p = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
                memcpy(&w[j], &p, 4);
            } else {
                const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                memcpy(&w[j], &p, 4);
            }
        }
    }
}
// Arrival that orders no memory: what it announces is in TMEM, complete by a tcgen05 wait.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar_cl) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cl)
                 : "memory");
}
template <int FORMAT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmW,
                const GemmArgs P) {
    using F = Fmt<FORMAT>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ BarsPair bars;
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    // operand tiles first (1024-byte aligned), then the scales, then the output
    uint8_t* scales = smem + kPairStages * 2 * kTileBytes;
    uint8_t* outbuf = scales + kPairStages * 3 * F::kScaleBytes;
    outbuf = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(outbuf) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int64_t k_stages = (P.K + 255) / 256;
    const int64_t m_tiles = (P.N + 255) / 256, tiles = m_tiles * ((P.V + 255) / 256);
    volatile int* abort = &bars.abort;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 1);
            mbar_init(&bars.landed[s], 1);
            mbar_init(&bars.scaled[s], 8);  // 4 warps in each CTA
        }
        mbar_init(&bars.tfull, 1);
        mbar_init(&bars.tempty, 16);  // 8 warps in each CTA
        mbar_init(&bars.drain, 1);
        bars.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmH);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc_pair(&bars.tmem_base, kTmem);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;
    // TMEM columns: the accumulator's 256, then 48 a stage: scales of h (16), of W (32)
    const uint32_t tscales = tmem + 256;

    if (warp == 0) {
        // ------------------------------------------------------- producer
        int stage = 0;
        uint32_t phase = 0;
        Issued issued;
        bool ok = true;
        const uint32_t full0 = cluster_addr(&bars.full[0], 0);
        for (int64_t t = pair; t < tiles && ok; t += pairs) {
            const int64_t mt = (t % m_tiles) * 2 + rank, vt = (t / m_tiles) * 2;  // tiles of 128 rows
            for (int64_t kb = 0; kb < k_stages; ++kb) {
                if (!__all_sync(0xffffffffu,
                                mbar_wait_cl(&bars.empty[stage], phase ^ 1, P.wait_ns, abort))) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t* sa = smem + stage * 2 * kTileBytes;
                    uint8_t* ss = scales + stage * 3 * F::kScaleBytes;
                    const uint32_t bar = full0 + stage * 8u;
                    if (leader) mbar_arrive_expect_tx(&bars.full[stage], 4 * kTileBytes);
                    const int32_t x = static_cast<int32_t>(kb * kBKb);
                    tma_load_2d_pair(sa, &tmH, bar, x, static_cast<int32_t>(mt * 128));
                    tma_load_2d_pair(sa + kTileBytes, &tmW, bar, x, static_cast<int32_t>((vt + rank) * 128));
                    // scales of rows past the matrix are not used: what lies there stays
                    const int64_t st = kb * F::kTilesPerStage;
                    const uint32_t sb = static_cast<uint32_t>(
                        min(int64_t(F::kTilesPerStage), P.k_tiles - st) * kFp4TileBytes);
                    const int some_h = mt * 128 < P.N, some_w = (vt + 1) * 128 < P.V;
                    mbar_arrive_expect_tx(&bars.landed[stage], (1 + some_h + some_w) * sb);
                    if (some_h)
                        bulk_load(ss, P.h_scales + (mt * P.k_tiles + st) * kFp4TileBytes, sb,
                                  &bars.landed[stage]);
                    const uint8_t* ws = P.w_scales + (vt * P.k_tiles + st) * kFp4TileBytes;
                    bulk_load(ss + F::kScaleBytes, ws, sb, &bars.landed[stage]);
                    if (some_w)
                        bulk_load(ss + 2 * F::kScaleBytes, ws + P.k_tiles * kFp4TileBytes, sb,
                                  &bars.landed[stage]);
                }
                __syncwarp();
                issued.add(stage, phase);
                if (++stage == kPairStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
        // No load is in flight when the CTAs end, whichever warp gave up: each waits for its scales,
        // the leader for both CTAs' tiles, which are counted there, and for the next ones of the
        // other, which may have loaded on where this one stopped.  (Both end together, below.)
        wait_for_loads(bars.landed, issued, P.wait_ns);
        if (leader) wait_for_pair_loads(bars.full, issued, kPairStages, 2 * kTileBytes, !ok, P.wait_ns);
    } else if (warp == 1) {
        // ------------------------------------------- MMA issuer (leader only)
        if (leader) {
            int stage = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            const uint32_t sbase = smem_u32(smem);
            constexpr uint32_t kIdesc = F::idesc(256, 256);
            for (int64_t t = pair; t < tiles && ok; t += pairs) {
                if (!__all_sync(0xffffffffu, mbar_wait_cl(&bars.tempty, tphase ^ 1, P.wait_ns, abort))) {
                    ok = false;
                    break;
                }
                tphase ^= 1;
                tc_fence_after();
                for (int64_t kb = 0; kb < k_stages; ++kb) {
                    if (!__all_sync(0xffffffffu,
                                    mbar_wait_cl(&bars.full[stage], phase, P.wait_ns, abort) &&
                                        mbar_wait_cl(&bars.scaled[stage], phase, P.wait_ns, abort))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t sa = sbase + stage * 2 * kTileBytes, sb = sa + kTileBytes;
                        const uint32_t ts = tscales + stage * 48;
                        const int mmas = static_cast<int>(min(int64_t(4), (P.K - kb * 256 + 63) / 64));
                        for (int i = 0; i < mmas; ++i) {
                            const uint32_t c = i / F::kMmasPerTile;
                            const uint32_t id = FORMAT == LL_FP4_MX ? 2 * (i & 1) : 0;
                            mma_fp4_pair<FORMAT>(tmem, smem_desc_sw128(sa + i * 32, 16, 1024),
                                                 smem_desc_sw128(sb + i * 32, 16, 1024), kIdesc,
                                                 ts + 4 * c, ts + 16 + 8 * c, id,
                                                 (kb > 0 || i > 0) ? 1u : 0u);
                        }
                        tc_commit_pair_both(&bars.empty[stage]);
                    }
                    __syncwarp();
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (lane == 0) tc_commit_pair_both(&bars.tfull);
                __syncwarp();
            }
            if (!ok) {
                if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
                bars.abort = 1;
            }
            if (lane == 0) tc_commit_pair_local(&bars.drain);
            __syncwarp();
            mbar_wait(&bars.drain, 0, P.wait_ns, nullptr);
        }
    } else if (warp >= 10) {
        // ----------------------------------------------- scales to TMEM (both CTAs)
        const int q = warp & 3;  // the same scales to the lanes of every warp
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        const uint32_t scaled0 = cluster_addr(&bars.scaled[0], 0);
        for (int64_t t = pair; t < tiles && ok; t += pairs) {
            for (int64_t kb = 0; kb < k_stages; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&bars.landed[stage], phase, P.wait_ns, abort))) {
                    ok = false;
                    break;
                }
                // a lane: the 16 bytes of its row of each tile, 4 columns
                const uint8_t* ss = scales + stage * 3 * F::kScaleBytes + lane * 16;
                const uint32_t ts = tscales + stage * 48 + (static_cast<uint32_t>(q * 32) << 16);
                uint4 v[3][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < F::kTilesPerStage) {
                        v[0][i] = *reinterpret_cast<const uint4*>(ss + i * kFp4TileBytes);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v[1 + (2 * i + h) / 4][(2 * i + h) % 4] = *reinterpret_cast<const uint4*>(
                                ss + (1 + h) * F::kScaleBytes + i * kFp4TileBytes);
                    } else {
                        v[0][i] = make_uint4(0, 0, 0, 0);
                    }
                }
                __syncwarp();
                tmem_st16(ts, v[0]);
                tmem_st16(ts + 16, v[1]);
                if (F::kTilesPerStage == 4) tmem_st16(ts + 32, v[2]);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(scaled0 + stage * 8u);
                if (++stage == kPairStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
    } else {
        // ------------------------------------------------- epilogue (both CTAs)
        const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lanes [32 q, + 32), 128 columns
        uint8_t* buf = outbuf + (warp - 2) * kOutBuf;
        uint8_t* rowp = buf + lane * 128;
        const int sw = lane & 7;
        uint32_t tphase = 0;
        bool ok = true;
        ScaleProduct scale = {1.f, 1.f};
        if (FORMAT == LL_FP4_NV) scale = scale_product(*P.h_scale, *P.w_scale);
        const float g = scale.g;
        constexpr int kCols = 128 / int(sizeof(T));  // of a box
        const bool wide = P.wide_out != 0;
        T* out = static_cast<T*>(P.out);
        for (int64_t t = pair; t < tiles; t += pairs) {
            const int64_t row0 = (t % m_tiles) * 256 + rank * 128 + q * 32;
            const int64_t col0 = (t / m_tiles) * 256 + half * 128;
            if (!__all_sync(0xffffffffu, mbar_wait_cl(&bars.tfull, tphase, P.wait_ns, abort))) {
                ok = false;
                break;
            }
            tphase ^= 1;
            tc_fence_after();
            const uint32_t taddr = tmem + half * 128 + (static_cast<uint32_t>(q * 32) << 16);
            // 32 columns of this lane's row, as they go out: 16-bit outputs are packed, so
            // that all 128 fit in registers
            constexpr int kPacked = 32 * int(sizeof(T)) / 16;
            auto take = [&](int c, uint4 (&u)[kPacked]) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld32(taddr + c * 32, r);
                tmem_ld_wait(r);
                if (FORMAT == LL_FP4_NV && scale.two != 1.f) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale.two);
                }
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = FORMAT == LL_FP4_NV ? __uint_as_float(r[j]) * g : __uint_as_float(r[j]);
                if (P.bias) {
                    const int64_t col = col0 + c * 32 + lane;
                    const float b = col < P.V ? load_bias(P.bias, P.bias_dtype, col) : 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, b, j);
                }
                uint32_t w[8 * int(sizeof(T))];
                pack32<T>(v, w);
                memcpy(u, w, sizeof(w));
            };
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(cluster_addr(&bars.tempty, 0));
            };
            constexpr int kHeld = sizeof(T) == 2 ? 4 : 1;  // FP32 goes out 32 columns at a time
            uint4 u[kHeld][kPacked];
            if constexpr (kHeld == 4) {
#pragma unroll
                for (int c = 0; c < 4; ++c) take(c, u[c]);
                release();
            }
            constexpr int kBoxes = 128 / kCols;
#pragma unroll
            for (int b = 0; b < kBoxes; ++b) {
                const int64_t x0 = col0 + b * kCols;
                if constexpr (kHeld == 1) {
                    take(b, u[0]);
                    if (b == kBoxes - 1) release();
                }
                if (row0 >= P.N || x0 >= P.V) continue;
                __syncwarp();  // the buffer's last reads are done
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(rowp + ((k ^ sw) << 4)) =
                        kHeld == 4 ? u[(2 * b + k / 4) % kHeld][k % 4] : u[0][k % kPacked];
                __syncwarp();
                constexpr int kE = 16 / int(sizeof(T));
                const int64_t x = x0 + (lane & 7) * kE;
                T* o = out + (row0 + (lane >> 3)) * P.ldo + x;
                const uint8_t* from = buf + (lane >> 3) * 128;
                if (wide && row0 + 32 <= P.N && x0 + kCols <= P.V) {  // 4 rows of 128 bytes at once
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int swz = ((lane & 7) ^ ((4 * i + (lane >> 3)) & 7)) << 4;
                        *reinterpret_cast<uint4*>(o) =
                            *reinterpret_cast<const uint4*>(from + i * 512 + swz);
                        o += 4 * P.ldo;
                    }
                } else if (wide) {
                    for (int i = 0; i < 8; ++i, o += 4 * P.ldo) {
                        if (row0 + 4 * i + (lane >> 3) >= P.N) break;
                        const int swz = ((lane & 7) ^ ((4 * i + (lane >> 3)) & 7)) << 4;
                        const uint4 w = *reinterpret_cast<const uint4*>(from + i * 512 + swz);
                        if (x + kE <= P.V) {
                            *reinterpret_cast<uint4*>(o) = w;
                        } else {
                            T e[kE];
                            memcpy(e, &w, 16);
#pragma unroll
                            for (int j = 0; j < kE; ++j)
                                if (x + j < P.V) o[j] = e[j];
                        }
                    }
                } else {
                    const int rows = static_cast<int>(min(int64_t(32), P.N - row0));
                    for (int i = 0; i < rows; ++i)
#pragma unroll
                        for (int c = lane; c < kCols; c += 32)
                            if (x0 + c < P.V) {
                                const int chunk = c * int(sizeof(T)) / 16;
                                out[(row0 + i) * P.ldo + x0 + c] = *reinterpret_cast<const T*>(
                                    buf + i * 128 + ((chunk ^ (i & 7)) << 4) + c * sizeof(T) % 16);
                            }
                }
            }
        }
        if (!ok) {
            if (lane == 0) set_status(P.status, LL_ERR_DEVICE_TIMEOUT);
            bars.abort = 1;
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_barrier();  // the leader's MMAs are done with both CTAs' memory
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, kTmem);
}

// ---------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Codes [rows, row_bytes]: boxes of 128 bytes x box_rows, 128-byte swizzle, zero fill.
bool codes_map(CUtensorMap* map, const Fp4Matrix& m, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t bytes = fp4_row_bytes(m.cols);
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(bytes), static_cast<cuuint64_t>(m.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(bytes)};
    const cuuint32_t box[2] = {kBKb, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(m.codes), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FORMAT, typename T>
cudaError_t run_few(const Fp4Matrix& h, const Fp4Matrix& w, GemmArgs P, const DevInfo& dev,
                    cudaStream_t s) {
    auto kern = few_kernel<FORMAT, T>;
    static int configured[64] = {0};
    if (!configured[dev.device]) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax - 1024);
        if (e != cudaSuccess) return e;
        configured[dev.device] = 1;
    }
    CUtensorMap mw, mh;
    P.nt = static_cast<int>((h.rows + 15) / 16 * 16);
    if (!codes_map(&mw, w, 128) || !codes_map(&mh, h, P.nt)) return cudaErrorInvalidValue;
    const int stage = kTileBytes + P.nt * kBKb + 2 * Fmt<FORMAT>::kScaleBytes;
    P.stages = (kSmemMax - 1024 - 1024) / stage;
    if (P.stages > kMaxStages) P.stages = kMaxStages;
    const int64_t tiles = (w.rows + 127) / 128;
    const unsigned grid = unsigned(tiles < dev.num_sms ? tiles : dev.num_sms);
    note_launches(1);
    kern<<<grid, kThreadsG, P.stages * stage + 1024, s>>>(mw, mh, P);
    return cudaGetLastError();
}

template <int FORMAT, typename T>
cudaError_t run_pair(const Fp4Matrix& h, const Fp4Matrix& w, GemmArgs P, const DevInfo& dev,
                     cudaStream_t s) {
    using F = Fmt<FORMAT>;
    auto kern = pair_kernel<FORMAT, T>;
    constexpr int kBytes = kPairStages * (2 * kTileBytes + 3 * F::kScaleBytes) + 8 * kOutBuf + 2048;
    static_assert(kBytes + int(sizeof(BarsPair)) <= kSmemMax, "shared memory");
    static int configured[64] = {0};
    if (!configured[dev.device]) {
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
        configured[dev.device] = 1;
    }
    CUtensorMap mh, mw;
    if (!codes_map(&mh, h, 128) || !codes_map(&mw, w, 128)) return cudaErrorInvalidValue;
    P.wide_out = reinterpret_cast<uintptr_t>(P.out) % 16 == 0 && P.ldo * sizeof(T) % 16 == 0;
    const int64_t tiles = (P.N + 255) / 256 * ((P.V + 255) / 256);
    const int64_t pairs = tiles < dev.num_sms / 2 ? tiles : dev.num_sms / 2;
    note_launches(1);
    kern<<<unsigned(2 * pairs), kPairThreads, kBytes, s>>>(mh, mw, P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_linear(const Fp4Matrix& h, const Fp4Matrix& w, const void* bias,
                              int bias_dtype, void* out, int64_t ldo, int out_dtype,
                              const DevInfo& dev, cudaStream_t s) {
    GemmArgs P;
    memset(&P, 0, sizeof(P));
    P.h_scales = h.scales;
    P.w_scales = w.scales;
    P.h_scale = h.scale;
    P.w_scale = w.scale;
    P.bias = bias;
    P.bias_dtype = bias_dtype;
    P.N = h.rows;
    P.K = h.cols;
    P.V = w.rows;
    P.k_tiles = fp4_k_tiles(h.cols, h.format);
    P.out = out;
    P.ldo = ldo;
    P.status = dev.status;
    P.wait_ns = wait_limit_ns();
    // us by few_kernel and pair_kernel, 32768 x 2048 and 151936 x 4096 weights: 16 tokens 12.0 and
    // 14.7, 68.5 and 74.0; 64 13.8 and 14.7, 71.8 and 75.5; 128 17.5 and 14.7, 76.7 and 74.1
    const bool few = h.rows <= 96;
#define LL_RUN(F, T) (few ? run_few<F, T>(h, w, P, dev, s) : run_pair<F, T>(h, w, P, dev, s))
#define LL_RUN_T(T) (h.format == LL_FP4_MX ? LL_RUN(LL_FP4_MX, T) : LL_RUN(LL_FP4_NV, T))
    if (out_dtype == LL_F32) return LL_RUN_T(float);
    if (out_dtype == LL_F16) return LL_RUN_T(__half);
    return LL_RUN_T(__nv_bfloat16);
#undef LL_RUN_T
#undef LL_RUN
}

}  // namespace ll
