// FP8 GEMM with block scales:
//     y[m, n] = sum_B as[m, B] bs[n / 128, B] sum_{k in block B} E4M3(a[m, k]) E4M3(b[n, k]),
// blocks of 128 values along K. The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, products
// of E4M3 values exact, fp32 accumulation) into tensor memory, one K block per accumulator; the outer
// sum, scaled, is kept in fp32 registers: per K block the accumulator is read back and added with its
// factor while the next block's MMAs run into a second accumulator.
//
// fp8_gemm_narrow_kernel: the weight takes the MMA's M side (a tile of 128 rows of b on the 128 tensor-memory
// lanes), MT activation rows (16, 32, 64 or 128) the N side, so that few tokens cost no more MMA or
// tensor-memory work than they need. K is split over a cluster of CTAs along grid z where the tiles alone would
// leave SMs idle; the partial sums are written into the shared memory of the CTA that stores them, which adds them in
// rank order, so results do not depend on scheduling. They have a place of their own there, so that nothing waits for
// another CTA's loads and MMAs (over the idle stage ring, behind a cluster barrier, the exchange took half of the 5.0 us
// of 1 x 2048 x 4096, which now takes 4.1 to 4.4). One K block takes an SM 450 cycles at MT = 16 (waits, four MMAs and
// their commits one after another in one warp) to 870 at MT = 128.
//   warp 0     TMA producer: weight tile (128 rows x 128 B) and activation tile (MT x 128 B) per K block;
//   warp 1     tensor memory and the MMA issue;
//   warps 2-3  the factors as[m, B] bs[n0 / 128, B] of the tile's MT rows, eight K blocks at a time;
//   warps 4-   one weight row and 32 of the MT columns per thread (16 for MT = 16): accumulator -> registers, one
//              FMA per value, and at the end the tile through shared memory to y.
//
// fp8_gemm_wide_kernel, for many tokens: SM pairs (tcgen05.mma.cta_group::2) on tiles of 256 tokens x BN columns (128,
// 192 or 256), tokens on the M side, CTA r of a pair holding 128 token rows and half of the BN weight rows, so that a K
// block of a 256-wide tile costs each SM 32 KB of loads for 512 cycles of MMA. Persistent, the pairs walking the tiles
// along N first; the accumulators (two, or four of 128 columns) fill tensor memory, so that the MMAs of one K block run
// while the one before is scaled and added.
//   warp 0     TMA producer of this CTA's operands;
//   warp 1     (leader) MMA issue;
//   warp 2     (peer) tells the leader that a stage's operands have landed here;
//   warp 3     the factors as[m, B] bs[n / 128, B], through shared memory;
//   warps 4-   (BN / 16 promotion warps) one token row and 64 columns per thread, in fp32 registers (at BN = 256 the
//              register split by setmaxnreg is 128 x 64 + 512 x 104 = 640 x 96, the launch's own total).
// A K block of a 256-wide tile takes 815 cycles: the MMAs alone 512, with their signals and loads 620, and the read-back,
// which shares tensor memory with them, the rest (reading 128 x 256 sums flat out slows a group of MMAs by 28 %). From a
// tile's last K block to the next tile's first it is 3,260 cycles, 2,220 of them the way of the sums to y.
// One of a 128-wide tile takes 535, the MMAs alone 256: its 24 KB of loads, at 46 bytes a cycle (a TMA load path
// measured at about 50), are 520 of them; the signals between the warps alone take 350. A 192-wide tile's 28 KB are 610
// of 700. So below 256 columns it is the loads that set the pace.
// With the accumulators neither read back nor added a call of 8192 x 2048 x 4096 takes 58 us instead of 70, without its
// MMAs 60, with a third of its loads 68: at 256 columns it is the way from an accumulator's MMAs through its promotion to
// the next ones, with two accumulators in turn, that sets the pace.
// 32768 x 2048 x 4096 takes 400,000 cycles: 244 us for a call after idle (2.25 PFLOP/s; the SMs at 1.64 GHz already), 268 to
// 284 us back to back, where the 1 kW limit holds them at 1.4 to 1.5 GHz.
//
// Every barrier wait is bounded (gdn_debug_set_wait); an expired one records GDN_ERR_TIMEOUT, issued copies
// and MMAs are waited for (bounded), tensor memory is freed and the CTA ends.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kChunk = 8;                  // K blocks per set of staged factors
constexpr int kMaxSplit = 8;
// Stages loaded before the CTAs of a pair meet: from the producer's loop the first load left 1,600 cycles later (256 x
// 12352 x 2048 11.4 us against 11.0); but a stage takes 200 to 300 cycles to issue, and with all of them first the rest
// of the pair waited for that.
constexpr int kEarly = 2;

template <int MT>
struct NarrowCfg {
    // Two CTAs an SM for the narrow tiles, so that as many clusters of eight run at once as their K splits need: 16 x
    // 2048 x 4096 takes 4.5 us in eight ranges, 5.2 in four.
    static constexpr int CTAS = MT <= 32 ? 2 : 1;
    static constexpr int STAGES = MT == 16 ? 5 : MT == 32 ? 4 : MT == 64 ? 7 : 4;
    static constexpr int W_BYTES = 128 * 128, X_BYTES = MT * 128;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    static constexpr int COLS = MT == 16 ? 16 : 32;            // accumulator columns per thread, one tensor-memory load
    static constexpr int EPI_WARPS = 4 * MT / COLS;
    static constexpr int THREADS = 128 + 32 * EPI_WARPS;
    static constexpr int PITCH = 132;                          // unsplit: fp32 pitch of a column of the tile, over the stage ring
    static constexpr int OFF_PART = STAGES * STAGE_BYTES;      // split: the partial sums of this CTA's columns
    // fp32 pitch of a weight row in a CTA's share of c columns (padded off the bank stride), and all shares' size
    static constexpr int part_pitch(int c) { return c <= 4 ? c : c + 4; }
    static constexpr int part_bytes(int split) { return split * 128 * part_pitch(MT / split) * 4; }
    // Narrow tiles send with st.async and wait for the bytes (1 x 2048 x 4096 in 4.1 us, 4.3 with plain stores and a second
    // cluster barrier); the wider tiles' many sums go faster as plain stores (128 x 2048 x 4096 in 7.9 us, 8.5 by st.async).
    static constexpr bool ASYNC = MT <= 32;
    static constexpr int larger(int a, int b) { return a > b ? a : b; }
    static constexpr int PART_BYTES = larger(part_bytes(2), larger(part_bytes(4), part_bytes(8)));
    static constexpr int OFF_SCL = OFF_PART + PART_BYTES;
    static constexpr int OFF_BAR = OFF_SCL + 2 * kChunk * MT * 4;
    static constexpr int SMEM = OFF_BAR + 512 + 1024;
    static constexpr int TMEM_COLS = 2 * MT;
    static_assert(MT * PITCH * 4 <= STAGES * STAGE_BYTES, "the tile fits over the stage ring");
    static_assert(PART_BYTES >= part_bytes(2) && PART_BYTES >= part_bytes(4) && PART_BYTES >= part_bytes(8), "every split's shares fit");
    static_assert(STAGE_BYTES % 1024 == 0, "stage bases stay 1024-byte aligned");
    static_assert(2 * STAGES + 10 <= 32, "a lane a barrier");
    static_assert(MT % kMaxSplit == 0, "whole columns for every CTA of a cluster");
    static_assert(SMEM <= 232448 && CTAS * (SMEM + 1024) <= 233472 && 8 * (2 * STAGES + 10) + 4 <= 512, "layout");
};

__device__ __forceinline__ uint32_t f8_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void f8_cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// ... with nothing to release: an arrival that releases holds its warp up for about 1,000 cycles.
__device__ __forceinline__ void f8_cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void f8_cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The shared::cluster address of this CTA's object `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t f8_mapa(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// V values into another CTA's shared memory; with ASYNC their bytes complete on a barrier there.
template <int V, bool ASYNC>
__device__ __forceinline__ void f8_st_cluster(uint32_t at, const float *v, uint32_t bar) {
    if constexpr (ASYNC && V == 4)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at), "f"(v[0]),
                     "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(bar)
                     : "memory");
    else if constexpr (ASYNC)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at), "f"(v[0]), "f"(v[1]),
                     "r"(bar)
                     : "memory");
    else if constexpr (V == 4)
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
    else
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v[0]), "f"(v[1]) : "memory");
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

__device__ __forceinline__ void f8_tmem_ld(uint32_t at, uint32_t (&d)[16]) { tmem_ld16(at, d); }
__device__ __forceinline__ void f8_tmem_ld(uint32_t at, uint32_t (&d)[32]) { tmem_ld32(at, d); }

// mbar_wait_warp on two barriers, the first look at both in one instruction (even lanes at one, odd lanes at the other;
// __syncwarp makes what each half has seen complete so for the other, which the vote does not).
__device__ __forceinline__ bool f8_warp_wait2(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1, int *status) {
    const bool odd = threadIdx.x & 1;
    if (__all_sync(0xffffffffu, mbar_try_wait(odd ? b1 : b0, odd ? p1 : p0))) {
        __syncwarp();
        return true;
    }
    return mbar_wait_warp(b0, p0, status) && mbar_wait_warp(b1, p1, status);
}
// A look at two barriers, which the warp has to agree on (and to __syncwarp after).
__device__ __forceinline__ bool f8_look2(uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1) {
    const bool odd = threadIdx.x & 1;
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(odd ? b1 : b0)), "r"(odd ? p1 : p0)
        : "memory");
    return ok;
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

// This thread's sums (one weight row, COLS columns from its group's first) to the CTAs that store them: columns
// [r cpr, (r + 1) cpr) of the tile to CTA r, into the share of this CTA there, [weight row][column].
template <int MT, int V>
__device__ __forceinline__ void f8_send_parts(uint8_t *sm, uint64_t *parts, const float (&acc)[NarrowCfg<MT>::COLS], int warp, int lane,
                                              int crank, int cpr) {
    using Cfg = NarrowCfg<MT>;
    const int c0 = ((warp - 4) >> 2) * Cfg::COLS, row = (warp & 3) * 32 + lane, pitch = Cfg::part_pitch(cpr), sh = __ffs(cpr) - 1;
    const float *share = reinterpret_cast<const float *>(sm + Cfg::OFF_PART) + (crank * 128 + row) * pitch;
#pragma unroll
    for (int c = 0; c < Cfg::COLS; c += V) {
        const uint32_t to = (uint32_t)((c0 + c) >> sh);   // cpr is a power of two
        f8_st_cluster<V, Cfg::ASYNC>(f8_mapa(share + ((c0 + c) & (cpr - 1)), to), acc + c, f8_mapa(parts, to));
    }
}

// The shares of this CTA's cpr columns (activation rows m_first ..), added in rank order and stored.
template <int MT, int V, bool OUT_BF16>
__device__ __forceinline__ void f8_sum_parts(const uint8_t *sm, void *y, int tid, int m_first, int n0, int M, int N, int split, int cpr) {
    using Cfg = NarrowCfg<MT>;
    const int pitch = Cfg::part_pitch(cpr);
    for (int u = tid; u < 128 * (cpr / V); u += Cfg::THREADS) {
        const int row = u % 128, c = u / 128 * V;
        const float *src = reinterpret_cast<const float *>(sm + Cfg::OFF_PART) + row * pitch + c;
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.0f;
#pragma unroll 8
        for (int z = 0; z < split; ++z) {   // in rank order
            const float *t = src + z * 128 * pitch;
            if constexpr (V == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(t);
                v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(t);
                v[0] += x.x; v[1] += x.y;
            }
        }
        if (n0 + row >= N) continue;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (m_first + c + i < M) store1<OUT_BF16>(y, (size_t)(m_first + c + i) * N + n0 + row, v[i]);
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
    uint64_t *scl_full = acc_full + 4, *scl_empty = acc_full + 6, *drain = acc_full + 8, *parts = acc_full + 9;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 10);
    auto tile_w = [&](int s) { return sm + s * Cfg::STAGE_BYTES; };
    auto tile_x = [&](int s) { return sm + s * Cfg::STAGE_BYTES + Cfg::W_BYTES; };

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int n0 = blockIdx.x * 128, m0 = blockIdx.y * MT;
    // this CTA's K blocks: [kb0, kb0 + nkb), at least one (split <= kb_all)
    const int crank = split > 1 ? (int)f8_cluster_rank() : 0;
    const int split_log = __ffs(split) - 1;   // (a power of two)
    const int kb0 = (int)((int64_t)crank * kb_all >> split_log);
    const int nkb = (int)((int64_t)(crank + 1) * kb_all >> split_log) - kb0;

    if (warp == 0) {
        // a lane a barrier; arrivals: the promotion warps at acc_empty and scl_empty, two factor warps at scl_full, else one
        const int b = lane - 2 * STAGES;
        if (b < 10) mbar_init(&bars[lane], b == 2 || b == 3 || b == 6 || b == 7 ? Cfg::EPI_WARPS : b == 4 || b == 5 ? 2 : 1);
        fence_barrier_init();
        // the sums of this CTA's MT / split columns from every CTA of the cluster
        if (Cfg::ASYNC && split > 1 && b == 9) mbar_arrive_expect_tx(parts, MT * 128 * 4);
    }
    __syncwarp();
    // (below: nothing is sent to a CTA before it has come this far; the fence above releases its barriers)
    if (split > 1) f8_cluster_arrive_relaxed();
    if (warp == 1) {
        tmem_alloc(tmem_slot, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    float acc[COLS];          // warps 4-: the scaled sums of this thread's weight row
    bool acc_ok = false;

    if (warp == 0) {
        int i = 0;
        for (int s = 0, ph = 1; i < nkb; ++i) {
            if (!mbar_wait_warp(&empty[s], (uint32_t)ph, status)) break;
            if (elect_one()) {
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
            if (!f8_warp_wait2(&acc_empty[b], (uint32_t)(((i >> 1) & 1) ^ 1), &full[s], (uint32_t)ph, status)) break;
            tc_fence_after();
            const uint64_t off = (uint64_t)(s * (Cfg::STAGE_BYTES >> 4));
            if (elect_one()) {
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
            if (elect_one()) tc_commit(drain);
            __syncwarp();
            mbar_wait(drain, 0, status);
        }
    } else if (warp < 4) {
        // factors of chunk c (K blocks kChunk c ..) for the tile's rows, rows past M zero
        const float *bs_row = bs + (int64_t)blockIdx.x * kb_all + kb0;
        for (int c = 0; c * kChunk < nkb; ++c) {
            const int b = c & 1, cnt = min(kChunk, nkb - c * kChunk);
            if (!mbar_wait_warp(&scl_empty[b], (uint32_t)(((c >> 1) & 1) ^ 1), status)) break;
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
        const int quarter = warp & 3, group = (warp - 4) >> 2;
        const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + group * COLS;
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[c] = 0.0f;
        bool ok = true;
        for (int i = 0; i < nkb; ++i) {
            const int b = i & 1, ch = i / kChunk;
            ok = i % kChunk || mbar_wait_warp(&scl_full[ch & 1], (uint32_t)((ch >> 1) & 1), status);
            if (!ok || !(ok = mbar_wait_warp(&acc_full[b], (uint32_t)((i >> 1) & 1), status))) break;
            tc_fence_after();
            uint32_t d[COLS];
            f8_tmem_ld(tm + b * MT, d);
            const float4 *f4 = reinterpret_cast<const float4 *>(scl + ((ch & 1) * kChunk + i % kChunk) * MT + group * COLS);
            tmem_ld_wait_for(d);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
            for (int c = 0; c < COLS / 4; ++c) {
                const float4 f = f4[c];
                acc[4 * c] = fmaf(__uint_as_float(d[4 * c]), f.x, acc[4 * c]);
                acc[4 * c + 1] = fmaf(__uint_as_float(d[4 * c + 1]), f.y, acc[4 * c + 1]);
                acc[4 * c + 2] = fmaf(__uint_as_float(d[4 * c + 2]), f.z, acc[4 * c + 2]);
                acc[4 * c + 3] = fmaf(__uint_as_float(d[4 * c + 3]), f.w, acc[4 * c + 3]);
            }
            __syncwarp();
            if (i % kChunk == kChunk - 1 && lane == 0) mbar_arrive(&scl_empty[ch & 1]);
        }
        acc_ok = ok;
    }
    __syncwarp();
    if (split == 1) {
        // the tile over the idle stage ring (its loads have landed and been read by MMAs that have completed): column c
        // (an activation row) at c * PITCH, weight rows consecutive
        __syncthreads();
        if (acc_ok) {
            float *part = reinterpret_cast<float *>(sm) + (warp & 3) * 32 + lane;
#pragma unroll
            for (int c = 0; c < COLS; ++c) part[(((warp - 4) >> 2) * COLS + c) * Cfg::PITCH] = acc[c];
        }
        __syncthreads();
        for (int u = tid; u < MT * 32; u += Cfg::THREADS) {
            const int c = u / 32, j = 4 * (u % 32);
            if (m0 + c < M && n0 + j < N)
                store_y4<OUT_BF16>(y, (int64_t)(m0 + c) * N + n0 + j,
                                   *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sm) + c * Cfg::PITCH + j));
        }
    } else {
        const int cpr = MT >> split_log;
        f8_cluster_wait();
        if (acc_ok) {
            if (cpr >= 4) f8_send_parts<MT, 4>(sm, parts, acc, warp, lane, crank, cpr);
            else f8_send_parts<MT, 2>(sm, parts, acc, warp, lane, crank, cpr);
        }
        __syncwarp();
        if constexpr (Cfg::ASYNC) f8_cluster_arrive_relaxed();   // (the sums signal for themselves)
        else f8_cluster_arrive();
        bool here = true;   // the sums of every CTA of the cluster have arrived in this one
        if constexpr (Cfg::ASYNC) here = mbar_wait_warp(parts, 0, status);
        else f8_cluster_wait();
        if (here && cpr >= 4) f8_sum_parts<MT, 4, OUT_BF16>(sm, y, tid, m0 + crank * cpr, n0, M, N, split, cpr);
        else if (here) f8_sum_parts<MT, 2, OUT_BF16>(sm, y, tid, m0 + crank * cpr, n0, M, N, split, cpr);
        if constexpr (Cfg::ASYNC) f8_cluster_wait();   // no CTA ends while another may still send to it
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, Cfg::TMEM_COLS);
    }
}

// ------------------------------------------------------------------- wide ----

constexpr int kWFacAhead = 3;                 // K blocks whose factors are on their way
constexpr int kWFacPitch = 132;               // 128 token rows, the four 64-column groups
constexpr int kWPieceBytes = 32 * 64;         // a promotion warp's 32 rows x 64 bytes of y

template <int BN>
struct WideCfg {
    static constexpr int GROUPS = BN / 64;                        // column groups, a warpgroup of promotion warps each
    static constexpr int WARPS = 4 * GROUPS;
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr int BUFS = BN == 128 ? 4 : 2;                // accumulators in tensor memory
    static constexpr int A_BYTES = 128 * 128, B_BYTES = BN / 2 * 128;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 4 : BN == 192 ? 6 : 7;
    static constexpr int FAC_SLOTS = kWFacAhead + 2 * BUFS;
    static constexpr int OFF_OUT = STAGES * STAGE_BYTES;
    static constexpr int OFF_FAC = OFF_OUT + WARPS * 2 * kWPieceBytes;
    static constexpr int OFF_BAR = OFF_FAC + FAC_SLOTS * kWFacPitch * 4;
    static constexpr int SMEM = OFF_BAR + 256 + 1024;
    static constexpr bool SPLIT_REGS = BN == 256;
    static constexpr int CH = 32;                // columns of a tensor-memory load
    static_assert(2 * STAGES + 2 * BUFS + 1 <= 32, "a lane a barrier");
    static_assert(STAGE_BYTES % 1024 == 0 && kWPieceBytes % 512 == 0 && SMEM <= 232448 && BUFS * BN <= 512 && OFF_FAC % 16 == 0, "layout");
};

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
// A tile of 64-byte rows from shared memory to the matrix of `map`.
__device__ __forceinline__ void f8_store_2d(const CUtensorMap *map, const void *smem, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(smem_u32(smem)), "r"(x), "r"(y)
        : "memory");
}
// acc += f * d on CH accumulator columns, two at a time. (The sums are kept as pairs everywhere: packed and unpacked here
// they cost a fifth of the kernel's time in moves and spills.)
template <int CH>
__device__ __forceinline__ void f8_promote(f2_t *acc, const uint32_t (&d)[CH], f2_t f) {
#pragma unroll
    for (int j = 0; j < CH; j += 2) acc[j / 2] = fma2(f2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])), f, acc[j / 2]);
}

template <int BN, bool OUT_BF16>
__global__ void __launch_bounds__(WideCfg<BN>::THREADS, 1)
fp8_gemm_wide_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap map_y,
                     const float *__restrict__ as, const float *__restrict__ bs, int M, int N, int num_k,
                     int *status) {
    using Cfg = WideCfg<BN>;
    constexpr int STAGES = Cfg::STAGES, BUFS = Cfg::BUFS;
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Cfg::OFF_BAR);
    uint64_t *full = bars, *empty = bars + STAGES;
    uint64_t *acc_full = bars + 2 * STAGES, *acc_empty = acc_full + BUFS, *drain = acc_empty + BUFS;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    auto tile_a = [&](int s) { return sm + s * Cfg::STAGE_BYTES; };
    auto tile_b = [&](int s) { return sm + s * Cfg::STAGE_BYTES + Cfg::A_BYTES; };

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)f8_cluster_rank();
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int tiles_n = (N + BN - 1) / BN;
    const int num_tiles = tiles_n * ((M + 255) / 256);
    const int total = (num_tiles - pair + npairs - 1) / npairs * num_k;   // K blocks of this pair's tiles

    if (warp == 0) {
        // A lane a barrier. Arrivals: at full[] this CTA's TMA, in the leader also the peer's word that its own landed; at
        // empty[] and drain the leader's commit; at acc_full[] that and warp 3 (the K block's factors); at acc_empty[]
        // (leader only) every promotion warp of the pair.
        const int b = lane - 2 * STAGES;
        if (b <= 2 * BUFS)
            mbar_init(&bars[lane], lane < STAGES ? (rank == 0 ? 2 : 1) : b < 0 || b == 2 * BUFS ? 1 : b < BUFS ? 2 : 2 * Cfg::WARPS);
        fence_barrier_init();
        if (lane == 0) {
            tma_prefetch_desc(&map_a);
            tma_prefetch_desc(&map_b);
            tma_prefetch_desc(&map_y);
        }
        __syncwarp();
    }
    // The producer's place: tile pt, K block pk of it, stage ps. Its first loads go out before the CTAs of the pair meet
    // (they touch this CTA's barriers alone).
    int pt = pair, pk = 0, pit = 0, ps = 0, pm = pair / tiles_n * 256 + rank * 128, pn = pair % tiles_n * BN + rank * (BN / 2);
    auto load_stage = [&] {
        if (elect_one()) {
            mbar_arrive_expect_tx(&full[ps], Cfg::STAGE_BYTES);
            tma_load_2d(tile_a(ps), &map_a, &full[ps], pk * 128, pm);
            tma_load_2d(tile_b(ps), &map_b, &full[ps], pk * 128, pn);
        }
        ++pit;
        if (++pk == num_k) {
            pk = 0;
            pt += npairs;
            pm = pt / tiles_n * 256 + rank * 128;
            pn = pt % tiles_n * BN + rank * (BN / 2);
        }
        if (++ps == STAGES) ps = 0;
    };
    if (warp == 0) {
        __syncwarp();
        pdl_wait();
        while (pit < kEarly && pit < total) load_stage();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    // Both CTAs' barriers are initialised (the fence above releases them to the cluster) and tensor memory is allocated.
    f8_cluster_arrive_relaxed();
    f8_cluster_wait();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();

    if (warp < 4) {
        if constexpr (Cfg::SPLIT_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 0) {
            for (; pit < total;) {
                if (!mbar_wait_warp(&empty[ps], (uint32_t)(((pit / STAGES) & 1) ^ 1), status)) break;
                load_stage();
            }
            // before the CTA may exit: the latest load armed on each stage has landed ..
            for (int s = 0; s < STAGES && s < pit; ++s) {
                const int last = pit - 1 - ((pit - 1 - s) % STAGES);
                mbar_wait(&full[s], (uint32_t)((last / STAGES) & 1), status);
            }
            // .. and the leader's commit of the MMAs that read it has arrived here: the loop's waits, STAGES blocks on
            for (int i = pit; pit == total && i < total + STAGES; ++i) {
                if (!mbar_wait_warp(&empty[ps], (uint32_t)(((i / STAGES) & 1) ^ 1), status)) break;
                if (++ps == STAGES) ps = 0;
            }
            if (rank == 1) mbar_wait(drain, 0, status);   // (the leader's last commit arrives in both CTAs)
        } else if (warp == 1 && rank == 0) {
            constexpr uint32_t idesc = f8_idesc(256, BN);
            const uint64_t a_desc = smem_desc(smem_u32(tile_a(0)), 16, 1024, 2), b_desc = smem_desc(smem_u32(tile_b(0)), 16, 1024, 2);
            int s = 0, b = 0, it = 0;
            uint32_t ph = 0, bph = 1;   // the first use of each accumulator waits for nothing
            bool ready = false;
            for (; it < total; ++it) {
                if ((BUFS != 4 || !__all_sync(0xffffffffu, ready)) &&
                    (!mbar_wait_warp(&full[s], ph, status) || !mbar_wait_warp(&acc_empty[b], bph, status)))
                    break;
                if constexpr (BUFS == 4) __syncwarp();
                tc_fence_after();
                const int s_now = s, b_now = b;
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
                if (++b == BUFS) {
                    b = 0;
                    bph ^= 1;
                }
                // With four accumulators the next block's barriers have most often completed: they are looked at while
                // this block's MMAs are issued (512 x 4096 x 4096 14.4 -> 13.5 us; with two accumulators 3 to 5 % slower).
                if constexpr (BUFS == 4) ready = f8_look2(&full[s], ph, &acc_empty[b], bph);
                if (elect_one()) {
                    const uint64_t off = (uint64_t)(s_now * (Cfg::STAGE_BYTES >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        f8_mma_pair(tmem + b_now * BN, a_desc + off + 2 * kk, b_desc + off + 2 * kk, idesc, kk ? 1u : 0u);
                    f8_commit_pair(&acc_full[b_now]);
                    f8_commit_pair(&empty[s_now]);
                }
                __syncwarp();
            }
            // before the pair may free tensor memory: every MMA issued has completed (bounded)
            if (elect_one()) f8_commit_pair(drain);
            __syncwarp();
            mbar_wait(drain, 0, status);
            // before this CTA may exit: the promotion warps of both CTAs have given back each accumulator's last sums (the
            // loop's waits, BUFS blocks on)
            for (int i = 0; it == total && i < BUFS; ++i) {
                if (!mbar_wait_warp(&acc_empty[b], bph, status)) break;
                if (++b == BUFS) {
                    b = 0;
                    bph ^= 1;
                }
            }
        } else if (warp == 2 && lane == 0 && rank == 1) {
            const uint32_t at = f8_mapa(full, 0);
            int s = 0;
            uint32_t ph = 0;
            for (int it = 0; it < total; ++it) {
                if (!mbar_wait(&full[s], ph, status)) break;
                f8_arrive_at(at + (uint32_t)(s * 8));
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
        } else if (warp == 3) {
            // as[m, B] of the tile's rows and bs[n / 128, B] of its 64-column groups, some K blocks ahead by
            // asynchronous copies (a load that was waited for one block later took longer than the MMAs).
            // K block `it` is handed over once the one BUFS before it is in its accumulator: that one's MMAs
            // waited for the promotion of the one 2 BUFS before `it`, whose slot can be written again.
            float *fac = reinterpret_cast<float *>(sm + Cfg::OFF_FAC);
            const int rows_n = (N + 127) / 128;
            int pt = pair, pk = 0, pslot = 0;
            const float *pa[4], *pb;
            auto aim = [&] {   // at the rows of tile pt
                const int tm = pt / tiles_n, m0 = tm * 256 + rank * 128 + lane, ng = (pt - tm * tiles_n) * Cfg::GROUPS;
#pragma unroll
                for (int j = 0; j < 4; ++j) pa[j] = as + (int64_t)min(m0 + 32 * j, M - 1) * num_k;
                pb = bs + (int64_t)min((ng + (lane & 3)) / 2, rows_n - 1) * num_k;
            };
            aim();
            auto fetch = [&](int i) {
                if (i < total) {
                    float *to = fac + pslot * kWFacPitch;
#pragma unroll
                    for (int j = 0; j < 4; ++j) cp_async4(to + 32 * j + lane, pa[j] + pk);
                    if (lane < Cfg::GROUPS) cp_async4(to + 128 + lane, pb + pk);
                    if (++pk == num_k && i + 1 < total) {
                        pk = 0;
                        pt += npairs;
                        aim();
                    }
                    if (++pslot == Cfg::FAC_SLOTS) pslot = 0;
                }
                cp_async_commit();
            };
            for (int i = 0; i < kWFacAhead; ++i) fetch(i);
            int b = 0;
            uint32_t ph = 1;
            for (int it = 0; it < total; ++it) {
                if (it >= BUFS && !mbar_wait_warp(&acc_full[b], ph, status)) break;
                fetch(it + kWFacAhead);
                cp_async_wait<kWFacAhead>();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_full[b]);
                if (++b == BUFS) {
                    b = 0;
                    ph ^= 1;
                }
            }
            cp_async_wait<0>();
        }
    } else {
        if constexpr (Cfg::SPLIT_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        constexpr int CH = Cfg::CH, NCH = 64 / CH;
        const int quarter = warp & 3, group = (warp - 4) >> 2;
        const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16) + group * 64;
        const uint32_t leader_empty = f8_mapa(acc_empty, 0);
        const int r0 = rank * 128 + quarter * 32;
        uint8_t *pieces = sm + Cfg::OFF_OUT + (warp - 4) * 2 * kWPieceBytes;
        const float *fac = reinterpret_cast<const float *>(sm + Cfg::OFF_FAC);
        int fslot = 0, b = 0;
        uint32_t bph = 0;
        bool ok = true;
        for (int t = pair; t < num_tiles && ok; t += npairs) {
            f2_t acc[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) acc[j] = 0ull;
            for (int k = 0; k < num_k; ++k) {
                if (!(ok = mbar_wait_warp(&acc_full[b], bph, status))) break;
                tc_fence_after();
                // two loads of 32 columns in one set of registers (four of 16 in two sets, each under way while the one
                // before was added, with scalar sums: 32768 x 2048 x 4096 282 us back to back, so 267)
                uint32_t d[CH];
                f8_tmem_ld(tm + b * BN, d);
                const float f1 = fac[fslot * kWFacPitch + quarter * 32 + lane] * fac[fslot * kWFacPitch + 128 + group];
                const f2_t f = f2(f1, f1);
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    tmem_ld_wait_for(d);
                    if (c == NCH - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) f8_arrive_at(leader_empty + (uint32_t)(b * 8));
                    }
                    f8_promote(acc + CH / 2 * c, d, f);
                    if (c + 1 < NCH) f8_tmem_ld(tm + b * BN + CH * (c + 1), d);
                }
                if (++fslot == Cfg::FAC_SLOTS) fslot = 0;
                if (++b == BUFS) {
                    b = 0;
                    bph ^= 1;
                }
            }
            if (!ok) break;
            // A row of y lies in one thread: pieces of 32 rows x 64 bytes go through the warp's shared memory (16-byte chunk
            // c of row r at chunk c ^ (r / 2 % 4), the 64-byte swizzle) and out by TMA, which leaves off what lies past
            // the last row or column. Read back and stored by the warps, eight rows a store, they kept the SM's store
            // path busy for 1,600 to 2,600 cycles a tile.
            constexpr int CPP = OUT_BF16 ? 32 : 16;      // columns per piece
            const int m_base = t / tiles_n * 256 + r0, n_base = t % tiles_n * BN + group * 64;
#pragma unroll
            for (int pc = 0; pc < 64 / CPP; ++pc) {
                uint8_t *piece = pieces + pc % 2 * kWPieceBytes;
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");   // the one before last is out
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const f2_t *v = acc + (CPP * pc + CPP / 4 * c) / 2;
                    uint4 u;
                    if constexpr (OUT_BF16) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __nv_bfloat162 p2 = __floats2bfloat162_rn(f2lo(v[j]), f2hi(v[j]));
                            w[j] = *reinterpret_cast<const uint32_t *>(&p2);
                        }
                        u = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        u = make_uint4(__float_as_uint(f2lo(v[0])), __float_as_uint(f2hi(v[0])), __float_as_uint(f2lo(v[1])), __float_as_uint(f2hi(v[1])));
                    }
                    *reinterpret_cast<uint4 *>(piece + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)) = u;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (m_base < M && n_base + pc * CPP < N) f8_store_2d(&map_y, piece, n_base + pc * CPP, m_base);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");   // (one a piece: the waits count them)
                }
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    // Neither CTA frees tensor memory or exits while the pair's MMAs or reads may touch it. Every arrival from the other CTA
    // has been waited for above in the one it goes to: at full[] and acc_empty[] by the issuing warp, at empty[] by the
    // producers, at drain by the issuing warp and the peer's producer, at acc_full[] by the promotion warps. So this barrier
    // orders no memory and is relaxed (a release would wait for the stores of y to be performed).
    tc_fence_before();
    f8_cluster_arrive_relaxed();
    f8_cluster_wait();
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

// y [M, N], boxes of 32 rows x 64 bytes, 64-byte swizzle.
bool f8_map_out(CUtensorMap *m, void *ptr, uint64_t M, uint64_t N, bool bf16) {
    EncodeTiledFn fn = f8_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {N, M};
    cuuint64_t strides[1] = {N * (bf16 ? 2 : 4)};
    cuuint32_t box[2] = {bf16 ? 32u : 16u, 32};
    cuuint32_t elem[2] = {1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, ptr, dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t f8_count_clusters(K kernel, int threads, int smem, dim3 cluster, int *count) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster.x;
    attr.val.clusterDim.y = cluster.y;
    attr.val.clusterDim.z = cluster.z;
    cfg.gridDim = cluster;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(count, kernel, &cfg);
}
template <int MT>
cudaError_t f8_set_narrow() {
    const cudaError_t e = cudaFuncSetAttribute(fp8_gemm_narrow_kernel<MT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowCfg<MT>::SMEM);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fp8_gemm_narrow_kernel<MT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, NarrowCfg<MT>::SMEM);
}
template <int BN>
cudaError_t f8_set_wide() {
    const cudaError_t e = cudaFuncSetAttribute(fp8_gemm_wide_kernel<BN, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, WideCfg<BN>::SMEM);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(fp8_gemm_wide_kernel<BN, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, WideCfg<BN>::SMEM);
}
template <int MT>
cudaError_t launch_narrow(const Fp8GemmArgs &g, int split, cudaStream_t st) {
    using Cfg = NarrowCfg<MT>;
    CUtensorMap mw, mx;
    if (!f8_map(&mw, g.bq, (uint64_t)g.N, (uint64_t)g.K, 128) || !f8_map(&mx, g.aq, (uint64_t)g.M, (uint64_t)g.K, MT))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((g.N + 127) / 128), (unsigned)((g.M + MT - 1) / MT), (unsigned)split);
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
    const int kb = (g.K + 127) / 128;
    if (g.out_bf16)
        return cudaLaunchKernelEx(&cfg, fp8_gemm_narrow_kernel<MT, true>, mw, mx, g.as, g.bs, g.M, g.N, kb, g.y, split, g.status);
    return cudaLaunchKernelEx(&cfg, fp8_gemm_narrow_kernel<MT, false>, mw, mx, g.as, g.bs, g.M, g.N, kb, g.y, split, g.status);
}

template <int BN>
cudaError_t launch_wide(const Fp8GemmArgs &g, int pairs, cudaStream_t st) {
    using Cfg = WideCfg<BN>;
    CUtensorMap ma, mb, my;
    if (!f8_map(&ma, g.aq, (uint64_t)g.M, (uint64_t)g.K, 128) || !f8_map(&mb, g.bq, (uint64_t)g.N, (uint64_t)g.K, BN / 2) ||
        !f8_map_out(&my, g.y, (uint64_t)g.M, (uint64_t)g.N, g.out_bf16))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    const int64_t tiles = (int64_t)((g.N + BN - 1) / BN) * ((g.M + 255) / 256);
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(Cfg::THREADS);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = 2;
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    const int kb = (g.K + 127) / 128;
    if (g.out_bf16) return cudaLaunchKernelEx(&cfg, fp8_gemm_wide_kernel<BN, true>, ma, mb, my, g.as, g.bs, g.M, g.N, kb, g.status);
    return cudaLaunchKernelEx(&cfg, fp8_gemm_wide_kernel<BN, false>, ma, mb, my, g.as, g.bs, g.M, g.N, kb, g.status);
}

struct Cost {
    int tile;
    float start, end, block, push;   // push: what a split's exchange of partial sums adds
};
constexpr Cost kCost[kFp8Forms] = {{16, 2.1f, 1.0f, 0.26f, 0.4f},   {32, 2.2f, 1.0f, 0.285f, 0.9f},  {64, 2.7f, 1.0f, 0.31f, 1.1f},
                                   {128, 3.6f, 1.0f, 0.42f, 2.3f},  {128, 3.1f, 0.8f, 0.285f, 0.0f}, {192, 3.7f, 1.0f, 0.36f, 0.0f},
                                   {256, 4.0f, 1.2f, 0.415f, 0.0f}};

}  // namespace

cudaError_t fp8_device(Fp8Device *out) {
    static PerDevice<Fp8Device> rec;
    return rec.get(
        [](int dev, Fp8Device &r) {
            cudaError_t e = cudaDeviceGetAttribute(&r.sms, cudaDevAttrMultiProcessorCount, dev);
            if (e == cudaSuccess) e = f8_set_narrow<16>();
            if (e == cudaSuccess) e = f8_set_narrow<32>();
            if (e == cudaSuccess) e = f8_set_narrow<64>();
            if (e == cudaSuccess) e = f8_set_narrow<128>();
            if (e == cudaSuccess) e = f8_set_wide<128>();
            if (e == cudaSuccess) e = f8_set_wide<192>();
            if (e == cudaSuccess) e = f8_set_wide<256>();
            for (int i = 1; i < 4 && e == cudaSuccess; ++i)
                e = f8_count_clusters(fp8_gemm_narrow_kernel<128, true>, NarrowCfg<128>::THREADS, NarrowCfg<128>::SMEM,
                                      dim3(1, 1, 1u << i), &r.clusters[i]);
            if (e == cudaSuccess)
                e = f8_count_clusters(fp8_gemm_wide_kernel<256, true>, WideCfg<256>::THREADS, WideCfg<256>::SMEM, dim3(2), &r.pairs);
            if (e == cudaSuccess && r.pairs < 1) e = cudaErrorInvalidConfiguration;
            return e;
        },
        out);
}

bool fp8_form_ok(int64_t M, int64_t N, int64_t K, Fp8Form f, const Fp8Device &dev) {
    if (f.form < 0 || f.form >= kFp8Forms) return false;
    if (f.form >= kFp8Narrow) return f.split == 1;
    if ((M + kCost[f.form].tile - 1) / kCost[f.form].tile > 65535) return false;   // grid y
    if (f.split == 1) return true;
    // a cluster of that size runs, and every CTA has a K block
    const int lg = f.split == 2 ? 1 : f.split == 4 ? 2 : f.split == 8 ? 3 : 0;
    return lg && dev.clusters[lg] > 0 && (K + 127) / 128 >= f.split;
}

// The kernel and tile with the least estimated time: a start, and per wave of CTAs (or pairs) an end and a cost for
// each K block, in us at 1965 MHz. Fitted to timings of each form at 1 to 64 K blocks (bf16 output, CUDA-graph
// replay). Over 58 shapes of 1 to 26020 rows the pick was 1 to 2 % behind the fastest form on average, 6 % at most.
// Tiles of 16 and 32 split even where two CTAs then share an SM, if the shares are long: 8 x 10240 x 5120 takes
// 12.3 us in 160 CTAs of 20 K blocks, 15.6 in 80 of 40; 16 x 12352 x 2048 7.4 us in 194 of 8, 7.2 in 97 of 16.
// For example (us: narrow 64, narrow 128, wide 128, wide 192, wide 256)
//     256 x 2048 x 4096   10.2, 13.2, 12.4, 15.7, 17.7      1024 x 2048 x 4096   26.0, 18.6, 13.5, 16.6, 18.8
//     128 x 2048 x 4096    8.1, 10.7, 12.3, 15.4, 17.6      256 x 12352 x 2048   24.3, 21.2, 13.8, 10.9, 12.5
Fp8Form fp8_gemm_form(int64_t M, int64_t N, int64_t K, const Fp8Device &dev) {
    const int64_t kb = (K + 127) / 128, nt = (N + 127) / 128;
    float best = 3.0e38f;
    Fp8Form pick{kFp8Forms - 1, 1};
    for (int i = 0; i < kFp8Narrow; ++i) {
        const Cost &c = kCost[i];
        const int64_t ctas = nt * ((M + c.tile - 1) / c.tile);
        // K split while all clusters run at once and every CTA keeps two K blocks
        const int per_sm = c.tile <= 32 ? 2 : 1;
        for (int lg = 0; lg < 4; ++lg) {
            if (lg && (ctas << lg > (int64_t)per_sm * dev.sms || ctas > (int64_t)per_sm * dev.clusters[lg] || kb < 2 << lg)) break;
            if (!fp8_form_ok(M, N, K, {i, 1 << lg}, dev)) break;
            // of two CTAs on one SM a K block each takes 1.6 times as long as one alone, and they start later
            const bool two = per_sm == 2 && ctas << lg > dev.sms;
            const int64_t at_once = two ? 2 * dev.sms : dev.sms, waves = ((ctas << lg) + at_once - 1) / at_once;
            const float block = two ? 1.6f * c.block : c.block;
            const float t = c.start + (float)waves * (c.end + (float)((kb + (1 << lg) - 1) >> lg) * block) + (lg ? c.push : 0.0f) +
                            (two ? 1.0f : 0.0f);
            if (t < best) {
                best = t;
                pick = {i, 1 << lg};
            }
        }
        if (c.tile >= M) break;   // wider tiles hold nothing more
    }
    for (int i = kFp8Narrow; i < kFp8Forms && M > 64; ++i) {
        const Cost &c = kCost[i];
        const int64_t tiles = (N + c.tile - 1) / c.tile * ((M + 255) / 256);
        const int64_t waves = (tiles + dev.pairs - 1) / dev.pairs;
        const float t = c.start + (float)waves * (c.end + (float)kb * c.block);
        if (t < best) {
            best = t;
            pick = {i, 1};
        }
    }
    return pick;
}

cudaError_t launch_fp8_gemm_form(const Fp8GemmArgs &g, Fp8Form f, const Fp8Device &dev, cudaStream_t st) {
    switch (f.form) {
        case 0: return launch_narrow<16>(g, f.split, st);
        case 1: return launch_narrow<32>(g, f.split, st);
        case 2: return launch_narrow<64>(g, f.split, st);
        case 3: return launch_narrow<128>(g, f.split, st);
        case 4: return launch_wide<128>(g, dev.pairs, st);
        case 5: return launch_wide<192>(g, dev.pairs, st);
        default: return launch_wide<256>(g, dev.pairs, st);
    }
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs &g, cudaStream_t st) {
    Fp8Device dev;
    const cudaError_t e = fp8_device(&dev);
    return e != cudaSuccess ? e : launch_fp8_gemm_form(g, fp8_gemm_form(g.M, g.N, g.K, dev), dev, st);
}

}  // namespace gdn
