// FP8 GEMM with block scales:
//     y[m, n] = sum_B as[m, B] bs[n / 128, B] sum_{k in block B} E4M3(a[m, k]) E4M3(b[n, k]),
// blocks of 128 values along K. The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, products
// of E4M3 values exact, fp32 accumulation) into tensor memory, one K block per accumulator; the outer
// sum, scaled, is kept in fp32 registers: per K block the accumulator is read back and added with its
// factor while the next block's MMAs run into a second accumulator.
//
// fp8_gemm_narrow_kernel: the weight takes the MMA's M side (a tile of 128 rows of b on the 128 tensor-memory
// lanes), MT activation rows (16, 32, 64 or 128) the N side, so that few tokens cost no more MMA or
// tensor-memory work than they need. K is split over a cluster of CTAs along grid z where the tiles
// alone would leave SMs idle; the partial sums meet in shared memory, summed in rank order.
//   warp 0     TMA producer: weight tile (128 rows x 128 B) and activation tile (MT x 128 B) per K block;
//   warp 1     tensor memory and the MMA issue (one thread);
//   warps 2-3  the factors as[m, B] bs[n0 / 128, B] of the tile's MT rows, sixteen K blocks at a time;
//   warps 4-   one weight row per thread (two threads for MT = 128, half the columns each): accumulator
//              -> registers, one FMA per value, and at the end the tile through shared memory to y.
//
// fp8_gemm_wide_kernel, for many tokens: SM pairs (tcgen05.mma.cta_group::2) on 256 x 256 tiles, tokens on the M
// side, CTA r of a pair holding 128 token rows and half of the 256 weight rows, so that a K block costs each SM
// 32 KB of loads for 512 cycles of MMA (a 128 x 128 tile on one SM: 32 KB for 256, and loads are what
// bounds it). Persistent; the two accumulators take all of tensor memory, so that the MMAs of one K block
// run while the block before is scaled and added by the eight promotion warps, 128 fp32 sums a thread
// (register split by setmaxnreg: 128 x 72 + 256 x 216 = 384 x 168, the launch's own total).
//   warp 0     TMA producer of this CTA's operands;   warp 1     (leader) MMA issue;
//   warp 2     (peer) tells the leader that a stage's operands have landed here;
//   warp 3     the factors as[m, B] bs[n / 128, B] of this CTA's rows, through shared memory;
//   warps 4-11 one token row and half of the 256 columns per thread.
//
// Every barrier wait is bounded (gdn_debug_set_wait); an expired one records GDN_ERR_TIMEOUT, issued copies
// and MMAs are waited for (bounded), tensor memory is freed and the CTA ends.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kChunk = 16;                 // K blocks per set of staged factors

template <int MT>
struct NarrowCfg {
    static constexpr int STAGES = MT == 16 ? 6 : MT == 32 ? 5 : MT == 64 ? 4 : 6;
    static constexpr int CTAS = MT == 128 ? 1 : 2;             // per SM
    static constexpr int W_BYTES = 128 * 128, X_BYTES = MT * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int EPI_WARPS = MT == 128 ? 8 : 4;
    static constexpr int COLS = MT == 128 ? 64 : MT;           // accumulator columns per thread
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int PITCH = 132;                          // fp32 pitch of a column of the partial tile
    static constexpr int OFF_SCL = STAGES * STAGE_BYTES;
    static constexpr int OFF_BAR = OFF_SCL + 2 * kChunk * MT * 4;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;
    static constexpr int TMEM_COLS = 2 * MT;
    static_assert(MT * PITCH * 4 <= STAGES * STAGE_BYTES, "the partial tile fits over the stage ring");
    static_assert(STAGE_BYTES % 1024 == 0, "stage bases stay 1024-byte aligned");
    static_assert(CTAS * (SMEM + 1024) <= 233472, "CTAs per SM");
};

__device__ __forceinline__ uint32_t f8_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void f8_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 16 bytes at this CTA's shared address `p` as seen in CTA `rank` of the cluster.
__device__ __forceinline__ float4 f8_ld_cluster(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ void f8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// Instruction descriptor: fp32 accumulation, E4M3 A and B (format 0), both K-major.
__host__ __device__ constexpr uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Wait for tensor-memory loads, tied to the registers of the last one so that no use of them moves above it.
template <int N>
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 16)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                          "+r"(r[i + 6]), "+r"(r[i + 7]), "+r"(r[i + 8]), "+r"(r[i + 9]), "+r"(r[i + 10]), "+r"(r[i + 11]),
                          "+r"(r[i + 12]), "+r"(r[i + 13]), "+r"(r[i + 14]), "+r"(r[i + 15]));
}

// One lane of a whole warp. The warps that issue copies and MMAs run their loops with all lanes, the wait
// included, and elect a lane around the instructions alone: the operands of those instructions are warp-uniform
// registers, and from inside a one-lane branch each MMA took about 90 cycles to issue, more than it ran.
__device__ __forceinline__ bool f8_elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
// Whether the phase with the given parity has completed, without waiting.
__device__ __forceinline__ bool f8_done(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// The whole warp waits (bounded); false in every lane if any lane's wait ran out.
__device__ __forceinline__ bool f8_warp_wait(uint64_t *bar, uint32_t parity, int *status) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

// Four consecutive values of a row of y.
template <bool OUT_BF16>
__device__ __forceinline__ void store_y4(void *y, int64_t idx, float4 v) {
    if constexpr (OUT_BF16) {
        const __nv_bfloat162 p0 = __floats2bfloat162_rn(v.x, v.y), p1 = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(y) + idx) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&p0), *reinterpret_cast<const uint32_t *>(&p1));
    } else {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(y) + idx) = v;
    }
}

template <int MT, bool OUT_BF16>
__global__ void __launch_bounds__(NarrowCfg<MT>::THREADS, NarrowCfg<MT>::CTAS)
fp8_gemm_narrow_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                       const float *__restrict__ as, const float *__restrict__ bs, int M, int N, int kb_all,
                       void *__restrict__ y, int split, int *status) {
    using Cfg = NarrowCfg<MT>;
    constexpr int STAGES = Cfg::STAGES, COLS = Cfg::COLS;
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *scl = reinterpret_cast<float *>(sm + Cfg::OFF_SCL);            // [2][kChunk][MT]
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Cfg::OFF_BAR);
    uint64_t *full = bars, *empty = bars + STAGES, *acc_full = bars + 2 * STAGES, *acc_empty = acc_full + 2;
    uint64_t *scl_full = acc_full + 4, *scl_empty = acc_full + 6, *drain = acc_full + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 9);
    auto tile_w = [&](int s) { return sm + s * Cfg::STAGE_BYTES; };
    auto tile_x = [&](int s) { return sm + s * Cfg::STAGE_BYTES + Cfg::W_BYTES; };

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n0 = blockIdx.x * 128, m0 = blockIdx.y * MT;
    // this CTA's K blocks: [kb0, kb0 + nkb), at least one (split <= kb_all)
    const int crank = split > 1 ? (int)f8_cluster_rank() : 0;
    const int kb0 = (int)((int64_t)crank * kb_all / split);
    const int nkb = (int)((int64_t)(crank + 1) * kb_all / split) - kb0;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], Cfg::EPI_WARPS);
            mbar_init(&scl_full[b], 2);
            mbar_init(&scl_empty[b], Cfg::EPI_WARPS);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    if (warp == 0) {
        int i = 0;
        for (int s = 0, ph = 1; i < nkb; ++i) {
            if (!f8_warp_wait(&empty[s], (uint32_t)ph, status)) break;
            if (f8_elect()) {
                mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
                tma_load_2d(tile_w(s), &map_w, &full[s], (kb0 + i) * 128, n0);
                tma_load_2d(tile_x(s), &map_x, &full[s], (kb0 + i) * 128, m0);
            }
            if (++s == STAGES) {
                s = 0;
                ph ^= 1;
            }
        }
        // before the CTA may exit: the last load armed on each stage has landed
        for (int s = 0; s < STAGES && s < i; ++s) {
            const int last = i - 1 - ((i - 1 - s) % STAGES);
            mbar_wait(&full[s], (uint32_t)((last / STAGES) & 1), status);
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = f8_idesc(128, MT);
        const uint64_t w_desc = smem_desc(smem_u32(tile_w(0)), 16, 1024, 2), x_desc = smem_desc(smem_u32(tile_x(0)), 16, 1024, 2);
        int i = 0;
        for (int s = 0, ph = 0; i < nkb; ++i) {
            const int b = i & 1;
            // the first use of each accumulator waits for nothing (the phase before the first)
            if (!f8_warp_wait(&acc_empty[b], (uint32_t)(((i >> 1) & 1) ^ 1), status)) break;
            if (!f8_warp_wait(&full[s], (uint32_t)ph, status)) break;
            tc_fence_after();
            const uint64_t off = (uint64_t)(s * (Cfg::STAGE_BYTES >> 4));
            if (f8_elect()) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    f8_mma(tmem + b * MT, w_desc + off + 2 * kk, x_desc + off + 2 * kk, idesc, kk ? 1u : 0u);
                tc_commit(&empty[s]);
                tc_commit(&acc_full[b]);
            }
            __syncwarp();
            if (++s == STAGES) {
                s = 0;
                ph ^= 1;
            }
        }
        // before tensor memory is freed: every MMA issued has completed (bounded)
        if (i) {
            if (f8_elect()) tc_commit(drain);
            __syncwarp();
            mbar_wait(drain, 0, status);
        }
    } else if (warp < 4) {
        // factors of chunk c (K blocks kChunk c ..) for the tile's rows, rows past M zero
        bool ok = true;
        const float *bs_row = bs + (int64_t)blockIdx.x * kb_all + kb0;
        for (int c = 0; c * kChunk < nkb; ++c) {
            const int b = c & 1, cnt = min(kChunk, nkb - c * kChunk);
            if (lane == 0) ok = mbar_wait(&scl_empty[b], (uint32_t)(((c >> 1) & 1) ^ 1), status);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            for (int r = (warp - 2) * 32 + lane; r < MT; r += 64) {
                const bool live = m0 + r < M;
                const float *as_row = as + (int64_t)(live ? m0 + r : 0) * kb_all + kb0;
                float f[kChunk];
#pragma unroll
                for (int j = 0; j < kChunk; ++j)
                    f[j] = live && j < cnt ? as_row[c * kChunk + j] * bs_row[c * kChunk + j] : 0.0f;
#pragma unroll
                for (int j = 0; j < kChunk; ++j) scl[(b * kChunk + j) * MT + r] = f[j];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&scl_full[b]);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + half * COLS;
        float acc[COLS];
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[c] = 0.0f;
        bool ok = true;
        for (int i = 0; i < nkb; ++i) {
            const int b = i & 1, ch = i / kChunk;
            if (lane == 0) {
                ok = i % kChunk || mbar_wait(&scl_full[ch & 1], (uint32_t)((ch >> 1) & 1), status);
                ok = ok && mbar_wait(&acc_full[b], (uint32_t)((i >> 1) & 1), status);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const float *f = scl + ((ch & 1) * kChunk + i % kChunk) * MT + half * COLS;
#pragma unroll
            for (int c0 = 0; c0 < COLS; c0 += 16) {
                uint32_t d[16];
                tmem_ld16(tm + b * MT + c0, d);
                tmem_ld_wait_for(d);
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float4 s4 = *reinterpret_cast<const float4 *>(f + c0 + c);
                    acc[c0 + c] = fmaf(__uint_as_float(d[c]), s4.x, acc[c0 + c]);
                    acc[c0 + c + 1] = fmaf(__uint_as_float(d[c + 1]), s4.y, acc[c0 + c + 1]);
                    acc[c0 + c + 2] = fmaf(__uint_as_float(d[c + 2]), s4.z, acc[c0 + c + 2]);
                    acc[c0 + c + 3] = fmaf(__uint_as_float(d[c + 3]), s4.w, acc[c0 + c + 3]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&acc_empty[b]);
                if (i % kChunk == kChunk - 1) mbar_arrive(&scl_empty[ch & 1]);
            }
        }
        // the tile into shared memory over the idle stage ring (every load was read by an MMA that has
        // completed): column c (an activation row) at c * PITCH, weight rows consecutive
        if (ok) {
            float *part = reinterpret_cast<float *>(sm) + quarter * 32 + lane;
#pragma unroll
            for (int c = 0; c < COLS; ++c) part[(half * COLS + c) * Cfg::PITCH] = acc[c];
        }
    }
    // All threads reach the barriers, on the failure path too (the partial tile is then stale and the
    // status word already says so). CTA r of a cluster stores the r-th share of the activation rows.
    if (split > 1) f8_cluster_sync();
    else __syncthreads();
    const int c_lo = crank * MT / split, c_hi = (crank + 1) * MT / split;
    for (int u = tid; u < (c_hi - c_lo) * 32; u += Cfg::THREADS) {
        const int c = c_lo + u / 32, j = 4 * (u % 32);
        const float *src = reinterpret_cast<const float *>(sm) + c * Cfg::PITCH + j;
        if (m0 + c >= M || n0 + j >= N) continue;
        float4 v;
        if (split == 1) {
            v = *reinterpret_cast<const float4 *>(src);
        } else {
            v = f8_ld_cluster(src, 0);
            for (int z = 1; z < split; ++z) {
                const float4 t = f8_ld_cluster(src, (uint32_t)z);
                v.x += t.x;
                v.y += t.y;
                v.z += t.z;
                v.w += t.w;
            }
        }
        store_y4<OUT_BF16>(y, (int64_t)(m0 + c) * N + n0 + j, v);
    }
    if (split > 1) f8_cluster_sync();   // no CTA leaves before its partial tile has been read
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

// ------------------------------------------------------------------- wide ----

constexpr int kWStages = 6;
constexpr int kWStageBytes = 2 * 128 * 128;                   // this CTA's 128 token rows and 128 weight rows
constexpr int kWEpiWarps = 8;
constexpr int kWPieceBytes = 32 * 64;                         // a promotion warp's 32 rows x 64 bytes of y
constexpr int kWOutOff = kWStages * kWStageBytes;
constexpr int kWFacOff = kWOutOff + kWEpiWarps * kWPieceBytes;
constexpr int kWFacAhead = 3;                                 // K blocks whose factors are on their way
constexpr int kWFacSlots = kWFacAhead + 4;
constexpr int kWFacPitch = 132;                               // 128 token rows, the two weight blocks
constexpr int kWBarOff = kWFacOff + kWFacSlots * kWFacPitch * 4;
constexpr int kWSmem = kWBarOff + 256 + 1024;
constexpr int kWThreads = 384;
static_assert(kWSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ uint32_t f8_mapa(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// Arrival on a barrier of a CTA of the pair (no generic-memory data goes with it).
__device__ __forceinline__ void f8_arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// The MMAs issued so far complete -> one arrival on `bar` in both CTAs of the pair.
__device__ __forceinline__ void f8_commit_pair(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3)
                 : "memory");
}
__device__ __forceinline__ void f8_mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// acc += f * d on 32 accumulator columns. (Scalar FMAs: as packed f32x2 ones they need the loaded columns in
// aligned register pairs, and the moves and spills cost a fifth of the kernel's time.)
__device__ __forceinline__ void f8_promote(float (&acc)[32], const uint32_t (&d)[32], float f) {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(d[j]), f, acc[j]);
}

template <bool OUT_BF16>
__global__ void __launch_bounds__(kWThreads, 1)
fp8_gemm_wide_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const float *__restrict__ as, const float *__restrict__ bs, int M, int N, int num_k,
                     void *__restrict__ y, int *status) {
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + kWBarOff);
    uint64_t *full = bars, *empty = bars + kWStages;
    uint64_t *acc_full = bars + 2 * kWStages, *acc_empty = acc_full + 2, *drain = acc_full + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 5);
    auto tile_a = [&](int s) { return sm + s * kWStageBytes; };
    auto tile_b = [&](int s) { return sm + s * kWStageBytes + 128 * 128; };

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)f8_cluster_rank();
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int tiles_n = (N + 255) / 256;
    const int num_tiles = tiles_n * ((M + 255) / 256);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kWStages; ++s) {
            mbar_init(&full[s], rank == 0 ? 2 : 1);   // this CTA's TMA; in the leader also the peer's word that its own landed
            mbar_init(&empty[s], 1);                  // the leader's commit
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 2);                 // the leader's commit, and warp 3: the K block's factors
            mbar_init(&acc_empty[b], 2 * kWEpiWarps);   // leader only: every promotion warp of the pair
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    f8_cluster_sync();   // both CTAs' barriers are initialised and tensor memory is allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0) {
            int it = 0, s = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int t = pair; t < num_tiles && ok; t += npairs) {
                const int m0 = t / tiles_n * 256 + rank * 128, n0 = t % tiles_n * 256 + rank * 128;
                for (int k = 0; k < num_k; ++k, ++it) {
                    if (!(ok = f8_warp_wait(&empty[s], ph, status))) break;
                    if (f8_elect()) {
                        mbar_arrive_expect_tx(&full[s], kWStageBytes);
                        tma_load_2d(tile_a(s), &map_a, &full[s], k * 128, m0);
                        tma_load_2d(tile_b(s), &map_b, &full[s], k * 128, n0);
                    }
                    if (++s == kWStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // before the CTA may exit: the latest load armed on each stage has landed
            for (int s = 0; s < kWStages && s < it; ++s) {
                const int last = it - 1 - ((it - 1 - s) % kWStages);
                mbar_wait(&full[s], (uint32_t)((last / kWStages) & 1), status);
            }
        } else if (warp == 1 && rank == 0) {
            constexpr uint32_t idesc = f8_idesc(256, 256);
            const uint64_t a_desc = smem_desc(smem_u32(tile_a(0)), 16, 1024, 2), b_desc = smem_desc(smem_u32(tile_b(0)), 16, 1024, 2);
            const int total = (num_tiles - pair + npairs - 1) / npairs * num_k;   // K blocks of this pair's tiles
            int it = 0, s = 0;
            uint32_t ph = 0;
            for (; it < total; ++it) {
                const int b = it & 1;
                if (!f8_warp_wait(&full[s], ph, status)) break;
                if (!f8_warp_wait(&acc_empty[b], (uint32_t)(((it >> 1) & 1) ^ 1), status)) break;
                tc_fence_after();
                if (f8_elect()) {
                    const uint64_t off = (uint64_t)(s * (kWStageBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        f8_mma_pair(tmem + b * 256, a_desc + off + 2 * kk, b_desc + off + 2 * kk, idesc, kk ? 1u : 0u);
                    f8_commit_pair(&acc_full[b]);
                    f8_commit_pair(&empty[s]);
                }
                __syncwarp();
                if (++s == kWStages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // before the pair may free tensor memory: every MMA issued has completed (bounded)
            if (f8_elect()) f8_commit_pair(drain);
            __syncwarp();
            mbar_wait(drain, 0, status);
        } else if (warp == 2 && lane == 0 && rank == 1) {
            const uint32_t at = f8_mapa(full, 0);
            int it = 0;
            bool ok = true;
            for (int t = pair; t < num_tiles && ok; t += npairs)
                for (int k = 0; k < num_k && ok; ++k, ++it) {
                    const int s = it % kWStages;
                    ok = mbar_wait(&full[s], (uint32_t)((it / kWStages) & 1), status);
                    if (ok) f8_arrive_at(at + (uint32_t)(s * 8));
                }
        } else if (warp == 3) {
            // as[m, B] of the tile's rows and bs[n / 128, B] of its two weight blocks, three K blocks ahead by
            // asynchronous copies (a load that was waited for one block later took longer than the MMAs).
            // K block `it` is handed over once the block two before it is in its accumulator: the MMAs of
            // that one waited for the promotion of the one four before `it`, whose slot can be written again.
            float *fac = reinterpret_cast<float *>(sm + kWFacOff);
            const int rows_n = (N + 127) / 128;
            const int total = (num_tiles - pair + npairs - 1) / npairs * num_k;
            int pt = pair, pk = 0, pslot = 0;
            const float *pa[4], *pb;
            auto aim = [&] {   // at the rows of tile pt
                const int tm = pt / tiles_n, m0 = tm * 256 + rank * 128 + lane, nb = (pt - tm * tiles_n) * 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) pa[j] = as + (int64_t)min(m0 + 32 * j, M - 1) * num_k;
                pb = bs + (int64_t)min(nb + (lane & 1), rows_n - 1) * num_k;
            };
            aim();
            auto fetch = [&](int i) {
                if (i < total) {
                    float *to = fac + pslot * kWFacPitch;
#pragma unroll
                    for (int j = 0; j < 4; ++j) cp_async4(to + 32 * j + lane, pa[j] + pk);
                    if (lane < 2) cp_async4(to + 128 + lane, pb + pk);
                    if (++pk == num_k && i + 1 < total) {
                        pk = 0;
                        pt += npairs;
                        aim();
                    }
                    if (++pslot == kWFacSlots) pslot = 0;
                }
                cp_async_commit();
            };
            for (int i = 0; i < kWFacAhead; ++i) fetch(i);
            for (int it = 0; it < total; ++it) {
                const int b = it & 1;
                if (it >= 2 && !f8_warp_wait(&acc_full[b], (uint32_t)(((it >> 1) & 1) ^ 1), status)) break;
                fetch(it + kWFacAhead);
                cp_async_wait<kWFacAhead>();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_full[b]);
            }
            cp_async_wait<0>();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
        const uint32_t leader_empty = f8_mapa(acc_empty, 0);
        const int r0 = rank * 128 + quarter * 32;
        uint8_t *piece = sm + kWOutOff + (warp - 4) * kWPieceBytes;
        const float *fac = reinterpret_cast<const float *>(sm + kWFacOff);
        int fslot = 0;
        auto factor = [&] {   // of this thread's row and half, the next K block's
            const float f = fac[fslot * kWFacPitch + quarter * 32 + lane] * fac[fslot * kWFacPitch + 128 + half];
            if (++fslot == kWFacSlots) fslot = 0;
            return f;
        };
        int it = 0;
        bool ok = true;
        for (int t = pair; t < num_tiles && ok; t += npairs) {
            float acc[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[c][j] = 0.0f;
            uint32_t d[2][32];   // 32 columns are loaded while the 32 before are added, also from one K block to the next
            ok = f8_warp_wait(&acc_full[it & 1], (uint32_t)((it >> 1) & 1), status);
            if (!ok) break;
            tc_fence_after();
            tmem_ld32(tm + (it & 1) * 256, d[0]);
            float f = factor();
            for (int k = 0; k < num_k; ++k, ++it) {
                const int b = it & 1;
                const uint32_t next_ph = (uint32_t)(((it + 1) >> 1) & 1);
                bool next = false;   // whether the next K block's accumulator is there, looked at early
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    tmem_ld_wait_for(d[c & 1]);
                    tmem_ld32(tm + b * 256 + 32 * (c + 1), d[(c + 1) & 1]);
                    if (c == 1) next = f8_done(&acc_full[b ^ 1], next_ph);
                    f8_promote(acc[c], d[c & 1], f);
                }
                tmem_ld_wait_for(d[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) f8_arrive_at(leader_empty + (uint32_t)(b * 8));
                const float f3 = f;
                if (k + 1 < num_k) {
                    if (!__all_sync(0xffffffffu, next) && !(ok = f8_warp_wait(&acc_full[b ^ 1], next_ph, status))) break;
                    tc_fence_after();
                    tmem_ld32(tm + (b ^ 1) * 256, d[0]);
                    f = factor();
                }
                f8_promote(acc[3], d[1], f3);
            }
            if (!ok) break;
            // a row of y lies in one thread: pieces of 32 rows x 64 bytes turn in the warp's shared memory
            // (16-byte chunk c of row r at chunk c ^ (r / 2 % 4): no bank conflicts either way) so that a store
            // covers eight runs of 64 bytes instead of 32 of 16
            constexpr int CPP = OUT_BF16 ? 32 : 16;      // columns per piece
            const int m_base = t / tiles_n * 256 + r0, n_base = t % tiles_n * 256 + half * 128;
#pragma unroll
            for (int pc = 0; pc < 128 / CPP; ++pc) {
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float *v = OUT_BF16 ? &acc[pc][8 * c] : &acc[pc / 2][16 * (pc % 2) + 4 * c];
                    uint4 u;
                    if constexpr (OUT_BF16) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 p2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                            w[j] = *reinterpret_cast<const uint32_t *>(&p2);
                        }
                        u = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
                    }
                    *reinterpret_cast<uint4 *>(piece + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = u;
                }
                __syncwarp();
                const int c = lane & 3, n = n_base + pc * CPP + c * (CPP / 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * i + lane / 4;
                    const uint4 u = *reinterpret_cast<const uint4 *>(piece + r * 64 + ((c ^ (r >> 1 & 3)) << 4));
                    if (m_base + r < M && n < N)
                        *reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(y) + ((int64_t)(m_base + r) * N + n) * (OUT_BF16 ? 2 : 4)) = u;
                }
            }
        }
    }

    // neither CTA frees tensor memory or exits while the pair's MMAs, reads or arrivals may touch it
    tc_fence_before();
    f8_cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------- host side ----

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn f8_encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// Codes [rows, K] as a byte matrix, boxes of box_rows x 128 bytes (one K block), 128-byte swizzle;
// what lies past the last row or column reads as zero.
bool f8_map(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t K, uint32_t box_rows) {
    EncodeTiledFn fn = f8_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {K, rows};
    cuuint64_t strides[1] = {K};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t elem[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MT, bool OUT_BF16>
cudaError_t launch_narrow_t(const Fp8GemmArgs &g, cudaStream_t st) {
    using Cfg = NarrowCfg<MT>;
    static PerDevice<int> sm_count;   // the shared-memory attribute is set per device alongside
    int sms = 0;
    const cudaError_t e = sm_count.get(
        [](int dev, int &r) {
            cudaError_t x = cudaFuncSetAttribute(fp8_gemm_narrow_kernel<MT, OUT_BF16>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM);
            if (x == cudaSuccess) x = cudaDeviceGetAttribute(&r, cudaDevAttrMultiProcessorCount, dev);
            return x;
        },
        &sms);
    if (e != cudaSuccess) return e;
    CUtensorMap mw, mx;
    if (!f8_map(&mw, g.bq, (uint64_t)g.N, (uint64_t)g.K, 128) || !f8_map(&mx, g.aq, (uint64_t)g.M, (uint64_t)g.K, MT))
        return cudaErrorInvalidValue;
    const int nt = (g.N + 127) / 128, mt = (g.M + MT - 1) / MT, kb = (g.K + 127) / 128;
    int split = 1;   // doubled while the CTAs fit at once and every range keeps two K blocks
    while (split < 8 && (int64_t)nt * mt * split * 2 <= (int64_t)Cfg::CTAS * sms && kb >= 4 * split) split *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nt, (unsigned)mt, (unsigned)split);
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 1;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = (unsigned)split;
    cfg.attrs = attrs;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_narrow_kernel<MT, OUT_BF16>, mw, mx, g.as, g.bs, g.M, g.N, kb, g.y, split,
                              g.status);
}

template <int MT>
cudaError_t launch_narrow(const Fp8GemmArgs &g, cudaStream_t st) {
    return g.out_bf16 ? launch_narrow_t<MT, true>(g, st) : launch_narrow_t<MT, false>(g, st);
}

template <bool OUT_BF16>
cudaError_t launch_wide(const Fp8GemmArgs &g, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = 2;
    attrs[0].val.clusterDim.y = 1;
    attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = kWSmem;
    cfg.stream = st;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    static PerDevice<int> max_pairs;   // as many pairs as run at once
    int pairs = 0;
    const cudaError_t e = max_pairs.get(
        [&cfg](int, int &r) {
            cudaError_t x = cudaFuncSetAttribute(fp8_gemm_wide_kernel<OUT_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWSmem);
            if (x != cudaSuccess) return x;
            cudaLaunchConfig_t q = cfg;
            q.gridDim = dim3(2);
            int clusters = 0;
            if ((x = cudaOccupancyMaxActiveClusters(&clusters, fp8_gemm_wide_kernel<OUT_BF16>, &q)) != cudaSuccess) return x;
            r = clusters > 0 ? clusters : 1;
            return cudaSuccess;
        },
        &pairs);
    if (e != cudaSuccess) return e;
    CUtensorMap ma, mb;
    if (!f8_map(&ma, g.aq, (uint64_t)g.M, (uint64_t)g.K, 128) || !f8_map(&mb, g.bq, (uint64_t)g.N, (uint64_t)g.K, 128))
        return cudaErrorInvalidValue;
    const int64_t tiles = (int64_t)((g.N + 255) / 256) * ((g.M + 255) / 256);
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    return cudaLaunchKernelEx(&cfg, fp8_gemm_wide_kernel<OUT_BF16>, ma, mb, g.as, g.bs, g.M, g.N, (g.K + 127) / 128, g.y, g.status);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmArgs &g, cudaStream_t st) {
    if (g.M > 128) return g.out_bf16 ? launch_wide<true>(g, st) : launch_wide<false>(g, st);
    if (g.M <= 16) return launch_narrow<16>(g, st);
    if (g.M <= 32) return launch_narrow<32>(g, st);
    if (g.M <= 64) return launch_narrow<64>(g, st);
    return launch_narrow<128>(g, st);
}

}  // namespace gdn
