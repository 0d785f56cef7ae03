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
        if (lane == 0) {
            int i = 0;
            for (; i < nkb; ++i) {
                const int s = i % STAGES;
                if (!mbar_wait(&empty[s], (uint32_t)(((i / STAGES) & 1) ^ 1), status)) break;
                mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
                tma_load_2d(tile_w(s), &map_w, &full[s], (kb0 + i) * 128, n0);
                tma_load_2d(tile_x(s), &map_x, &full[s], (kb0 + i) * 128, m0);
            }
            // before the CTA may exit: the last load armed on each stage has landed
            for (int s = 0; s < STAGES && s < i; ++s) {
                const int last = i - 1 - ((i - 1 - s) % STAGES);
                mbar_wait(&full[s], (uint32_t)((last / STAGES) & 1), status);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = f8_idesc(128, MT);
            int i = 0;
            for (; i < nkb; ++i) {
                const int s = i % STAGES, b = i & 1;
                // the first use of each accumulator waits for nothing (the phase before the first)
                if (!mbar_wait(&acc_empty[b], (uint32_t)(((i >> 1) & 1) ^ 1), status)) break;
                if (!mbar_wait(&full[s], (uint32_t)((i / STAGES) & 1), status)) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    f8_mma(tmem + b * MT, smem_desc(smem_u32(tile_w(s)) + kk * 32, 16, 1024, 2),
                           smem_desc(smem_u32(tile_x(s)) + kk * 32, 16, 1024, 2), idesc, kk ? 1u : 0u);
                tc_commit(&empty[s]);
                tc_commit(&acc_full[b]);
            }
            // before tensor memory is freed: every MMA issued has completed (bounded)
            if (i) {
                tc_commit(drain);
                mbar_wait(drain, 0, status);
            }
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
                tmem_ld_wait();
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

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmArgs &g, cudaStream_t st) {
    if (g.M <= 16) return launch_narrow<16>(g, st);
    if (g.M <= 32) return launch_narrow<32>(g, st);
    if (g.M <= 64) return launch_narrow<64>(g, st);
    return launch_narrow<128>(g, st);
}

}  // namespace gdn
