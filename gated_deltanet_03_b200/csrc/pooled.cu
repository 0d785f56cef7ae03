// The single-token gated delta rule on states that lie in a pool of slots (one slot per live request, batch
// rows naming theirs), plain or with the gated tail and its FP8 encoding in the same kernel:
//     S = alpha S + beta (v - alpha S k^) k^^T,  o = S q^,  S = pool[slots[row], head]  (128 x 128 fp32, in place),
// "Why Gated DeltaNet Survives 4-Bit Quantization" (abstract, mechanisms ii-iii); tail: "Red Lite dev15d -
// DeltaNet gated tail", Pinned graph semantics, steps 1-5.
//
// HBM-bound: 128 KB of state traffic and about 8 operations a state value per (row, head) item. The grid has one
// CTA per unit of one or more heads of a row; those that run take over the units of CTAs that have not been
// launched yet (cluster launch control), so each SM does as many as its share of the memory rate allows (equal
// shares left the fastest SMs idle for a fifth of the time: 183 us against 166 for 250 live rows x 32 heads). A
// producer warp brings each item's 64 KB state and its q, k, v, z rows into a ring by bulk copies, so loads
// stay in flight while items are computed, written back and encoded:
//   warps 0-15   the state from the stage into registers (8 lanes a row, 2 rows a thread, in the arithmetic of
//                gdn_recurrent128_kernel, so o and S equal gdn_decode_step's bit for bit), the stage released
//                at once, the update, o to shared memory, S stored straight to the pool;
//   warp 16      slots, bulk copies, gates;
//   warps 17-18  item i's o row on warp 17 + i % 2 (tail and encode, or the plain store). Its chain of
//                reductions and divisions takes longer than the update; done in turn by the update's own warps
//                it held up every item's last row (6.5 us an item against 3 us of HBM time).
// Both kinds of item warps go through their loop once before their first item, on whatever shared memory holds and
// without a wait or a store: it brings the loop's code into the SM's instruction cache while the first state is on
// its way. Without it a CTA's first item took 12,700 cycles from its state's arrival to its codes, later ones a
// third of that, which is most of a small batch's time.
// 250 live rows x 32 heads take 161.3 us plain and 161.8 with the tail (the bytes at the measured copy rate: 161), 3 live
// rows x 16 heads 4.3 and 4.6.
// A row with a negative slot is passed over (its outputs stay as they are); so is a row whose slot is not
// below num_slots or is named by an earlier row, and the status word then reads GDN_ERR_INVALID_ARG.
// Every wait is bounded; an expired one records GDN_ERR_TIMEOUT and the warp ends.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kD = 128;
constexpr int kPoolStages = 3;
constexpr int kPoolWarps = 16;
constexpr int kPoolFinishers = 2;
constexpr int kPoolRows = 4;               // o rows between the update and the finishers
constexpr int kPoolThreads = 32 * (kPoolWarps + 1 + kPoolFinishers);
constexpr uint32_t kStateBytes = kD * kD * 4;
constexpr uint32_t kRowBytes = kD * 2;
constexpr unsigned kAll = 0xffffffffu;

struct PoolMeta {
    int32_t row, head, slot;   // row < 0: no more items
    float alpha, beta;
};
struct PoolSmem {
    float state[kPoolStages][kD * kD];
    __nv_bfloat16 q[kPoolStages][kD], k[kPoolStages][kD], v[kPoolStages][kD], z[kPoolStages][kD];
    float o[kPoolRows][kD];
    PoolMeta meta[kPoolStages];
    uint4 claim;               // answer of the launch control
    uint64_t full[kPoolStages], empty[kPoolStages], o_full[kPoolRows], o_empty[kPoolRows], claimed;
};
constexpr int kPoolSmem = (int)sizeof(PoolSmem) + 128;

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// Asks for the unit of a CTA that has not been launched: the answer (16 bytes) completes on `bar`.
__device__ __forceinline__ void claim_unit(uint4 *answer, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The claimed unit (grid y and x of that CTA: row and place in it), or row -1 if none was left.
__device__ __forceinline__ int2 claimed_unit(const uint4 *answer) {
    uint32_t ok, x, y;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%3];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "mov.u32 %2, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::y.b32.b128 %2, r;\n\t}"
        : "=r"(ok), "=r"(x), "=r"(y)
        : "r"(smem_u32(answer))
        : "memory");
    fence_proxy_async_smem();   // read before the next answer is written
    return make_int2(ok ? (int)y : -1, (int)x);
}

__device__ __forceinline__ float pool_dot16(const f2_t (&a)[8], const f2_t (&b)[8]) {
    f2_t acc = mul2(a[0], b[0]);
#pragma unroll
    for (int c = 1; c < 8; ++c) acc = fma2(a[c], b[c], acc);
    return f2lo(acc) + f2hi(acc);
}
// The sums over a row group of 8 lanes of two values: lanes whose bit 2 is p get value p. (In the order of additions of
// the four-row form of gdn_recurrent128_kernel.)
__device__ __forceinline__ float pool_sum2(const float (&x)[2], int l8) {
    const bool b2 = (l8 & 4) != 0;
    float v = (b2 ? x[1] : x[0]) + __shfl_xor_sync(kAll, b2 ? x[0] : x[1], 4);
    v += __shfl_xor_sync(kAll, v, 2);
    v += __shfl_xor_sync(kAll, v, 1);
    return v;
}
// Columns 32 j + 4 l8 + e of a staged bf16 row as 8 pairs.
__device__ __forceinline__ void pool_cols16(const __nv_bfloat16 *row, int l8, f2_t (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint2 u = *reinterpret_cast<const uint2 *>(row + 32 * j + 4 * l8);
        x[2 * j] = bf16x2_to_f2(u.x);
        x[2 * j + 1] = bf16x2_to_f2(u.y);
    }
}

__device__ __forceinline__ float gate_at(const void *p, bool bf16, int64_t idx) {
    return bf16 ? load1<true>(p, idx) : load1<false>(p, idx);
}

template <bool TAIL>
__global__ void __launch_bounds__(kPoolThreads, 1)
gdn_decode128_pooled_kernel(const __grid_constant__ PooledDecodeArgs d) {
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    PoolSmem &sm = *reinterpret_cast<PoolSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (warp == 0) {
        // a lane a barrier; full: the copies, and the item's meta data
        constexpr int F = kPoolStages, E = 2 * F, O = E + kPoolRows, C = O + kPoolRows;
        if (lane <= C)
            mbar_init(&sm.full[0] + lane, lane < F ? 2 : lane < E ? kPoolWarps + 1 : lane < O ? kPoolWarps : 1);
        fence_barrier_init();
    }
    __syncthreads();
    const int Hv = d.Hv;
    int first = -1;                    // the pass before the first item
    asm volatile("" : "+r"(first));    // (not known to the compiler, which would give that pass code of its own)

    if (warp == kPoolWarps) {
        const int group = Hv / d.Hk;
        pdl_wait();
        int it = 0, claims = 0;
        bool ok = true;
        // A unit is a row (grid y) and unit_heads heads of it (grid x: heads of a row, which lie side by side in the pool, go
        // to CTAs that run together; the rows in front took 167 us for 256 x 32 heads, 165.7 so). From a CTA's start to its
        // first load is time that a small batch pays in full, so the loads of the slots go out first, and the claim, the
        // head's place and the barriers of an empty ring hold up nothing (48 items 5.6 -> 5.2 us, with the outputs in front
        // of the stores).
        for (int2 unit = make_int2(blockIdx.y, blockIdx.x); unit.x >= 0 && ok;) {
            const int row = unit.x, h0 = unit.y * d.unit_heads, h1 = min(h0 + d.unit_heads, Hv);
            const int slot = d.slots[row];
            const int other = lane < row ? d.slots[lane] : -1;
            if (elect_one()) claim_unit(&sm.claim, &sm.claimed);   // the next one
            ++claims;
            int kh = h0 / group, kr = h0 - kh * group;             // key head, and heads of it passed
            bool again = lane < row && other == slot;              // an earlier row's slot
            for (int i = lane + 32; i < row; i += 32) again |= d.slots[i] == slot;
            again = __any_sync(kAll, again);
            const bool live = slot >= 0 && slot < d.num_slots && !again;
            if (slot >= 0 && !live && lane == 0) report_status(d.status, GDN_ERR_INVALID_ARG);
            for (int h = h0; live && h < h1; ++h, ++it) {
                const int s = it % kPoolStages;
                const float ga = gate_at(d.a, d.gate_bf16, row * d.ldg + h), gb = gate_at(d.b, d.gate_bf16, row * d.ldg + h);
                const float ge = d.A_log[h], gt = d.dt_bias[h];
                if (it >= kPoolStages) ok = mbar_wait_warp(&sm.empty[s], (uint32_t)(((it / kPoolStages) & 1) ^ 1), d.status);
                if (!ok) break;
                const int64_t vrow = ((int64_t)row * Hv + h) * kD, krow = ((int64_t)row * d.Hk + kh) * kD;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sm.full[s], kStateBytes + (TAIL ? 4 : 3) * kRowBytes);
                    bulk_load(sm.state[s], d.pool + ((int64_t)slot * Hv + h) * kD * kD, kStateBytes, &sm.full[s]);
                    bulk_load(sm.k[s], reinterpret_cast<const __nv_bfloat16 *>(d.k) + krow, kRowBytes, &sm.full[s]);
                    bulk_load(sm.q[s], reinterpret_cast<const __nv_bfloat16 *>(d.q) + krow, kRowBytes, &sm.full[s]);
                    bulk_load(sm.v[s], reinterpret_cast<const __nv_bfloat16 *>(d.v) + vrow, kRowBytes, &sm.full[s]);
                    if constexpr (TAIL)
                        bulk_load(sm.z[s], reinterpret_cast<const __nv_bfloat16 *>(d.z) + row * d.ldz + h * kD, kRowBytes, &sm.full[s]);
                }
                __syncwarp();
                if (++kr == group) {
                    kr = 0;
                    ++kh;
                }
                float g, beta;   // while the state is on its way
                gdn_gates(ga, gb, ge, gt, g, beta);
                if (lane == 0) {
                    sm.meta[s] = {row, h, slot, expf(g), beta};
                    mbar_arrive(&sm.full[s]);
                }
                __syncwarp();
            }
            if (!mbar_wait_warp(&sm.claimed, (uint32_t)((claims - 1) & 1), d.status)) break;
            unit = claimed_unit(&sm.claim);
            __syncwarp();
        }
        // before the warp ends every copy it armed has landed; then one end mark for each finisher
        if (lane == 0) {
            for (int s = 0; s < kPoolStages && s < it; ++s) {
                const int at = it - 1 - ((it - 1 - s) % kPoolStages);
                mbar_wait(&sm.full[s], (uint32_t)((at / kPoolStages) & 1), d.status);
            }
            for (int e = it; e < it + kPoolFinishers && ok; ++e) {
                const int s = e % kPoolStages;
                ok = mbar_wait(&sm.empty[s], (uint32_t)(((e / kPoolStages) & 1) ^ 1), d.status);
                if (!ok) break;
                sm.meta[s].row = -1;
                mbar_arrive(&sm.full[s]);
                mbar_arrive(&sm.full[s]);
            }
        }
        return;
    }

    if (warp > kPoolWarps) {
        const int col = (lane & 15) * 8;   // lanes 16-31 repeat the row, their results unused
        f2_t w2[4] = {0ull, 0ull, 0ull, 0ull};
        for (int it = first, step = warp - kPoolWarps;; it += step, step = kPoolFinishers) {
            const bool run = it >= 0;
            const int s = run ? it % kPoolStages : 0, ob = run ? it % kPoolRows : 0;
            if (run && !mbar_wait_warp(&sm.full[s], (uint32_t)((it / kPoolStages) & 1), d.status)) break;
            const int row = sm.meta[s].row, head = sm.meta[s].head;
            if (run && row < 0) break;
            uint4 zu = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (TAIL) zu = *reinterpret_cast<const uint4 *>(&sm.z[s][col]);
            __syncwarp();
            if (run && lane == 0) mbar_arrive(&sm.empty[s]);
            if (run && !mbar_wait_warp(&sm.o_full[ob], (uint32_t)((it / kPoolRows) & 1), d.status)) break;
            const float4 oa = *reinterpret_cast<const float4 *>(&sm.o[ob][col]);
            const float4 oc = *reinterpret_cast<const float4 *>(&sm.o[ob][col + 4]);
            __syncwarp();
            if (run && lane == 0) mbar_arrive(&sm.o_empty[ob]);
            const int64_t at = ((int64_t)row * Hv + head) * kD;
            const bool store = run && lane < 16;
            if (d.o && store) {
                const float x[8] = {oa.x, oa.y, oa.z, oa.w, oc.x, oc.y, oc.z, oc.w};
                if (d.out_bf16) store8<true>(d.o, at + col, x);
                else store8<false>(d.o, at + col, x);
            }
            if constexpr (TAIL) {
                const f2_t o2[4] = {f2(oa.x, oa.y), f2(oa.z, oa.w), f2(oc.x, oc.y), f2(oc.z, oc.w)};
                const f2_t z2[4] = {bf16x2_to_f2(zu.x), bf16x2_to_f2(zu.y), bf16x2_to_f2(zu.z), bf16x2_to_f2(zu.w)};
                f2_t y2[4];
                gated_row8<16>(o2, z2, w2, 1.0f / (float)kD, d.eps, y2);
                float amax = 0.0f, r;
#pragma unroll
                for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(f2lo(y2[j])), fabsf(f2hi(y2[j]))));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, off));
                const float sc = fp8_block_scale(amax, r);
                const uint2 codes = make_uint2(fp8_pack4(f2lo(y2[0]), f2hi(y2[0]), f2lo(y2[1]), f2hi(y2[1]), r),
                                               fp8_pack4(f2lo(y2[2]), f2hi(y2[2]), f2lo(y2[3]), f2hi(y2[3]), r));
                if (store) *reinterpret_cast<uint2 *>(d.xq + at + col) = codes;
                if (run && lane == 0) d.xs[at / kD] = sc;
                if (!run) {
                    pdl_wait();
#pragma unroll
                    for (int j = 0; j < 4; ++j) w2[j] = f2(d.norm_w[col + 2 * j], d.norm_w[col + 2 * j + 1]);
                }
            } else if (!run) {
                pdl_wait();
            }
        }
        return;
    }

    const int l8 = tid & 7, rbase = tid >> 3, gbase = lane & ~7;   // rows rbase and rbase + 64
    for (int it = first;; ++it) {
        const bool run = it >= 0;
        const int s = run ? it % kPoolStages : 0, ob = run ? it % kPoolRows : 0;
        if (run && !mbar_wait_warp(&sm.full[s], (uint32_t)((it / kPoolStages) & 1), d.status)) break;
        const PoolMeta m = sm.meta[s];
        if (run && m.row < 0) break;

        f2_t st[2][8], k2[8], q2[8];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = *reinterpret_cast<const float4 *>(&sm.state[s][(rbase + 64 * p) * kD + 32 * j + 4 * l8]);
                st[p][2 * j] = f2(x.x, x.y);
                st[p][2 * j + 1] = f2(x.z, x.w);
            }
        pool_cols16(sm.k[s], l8, k2);
        pool_cols16(sm.q[s], l8, q2);
        float vv[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) vv[p] = __bfloat162float(sm.v[s][rbase + 64 * p]);
        __syncwarp();
        if (run && lane == 0) mbar_arrive(&sm.empty[s]);

        float kn = 1.0f, qn = d.scale;
        if (d.l2norm) {
            const float ks = group_sum<8>(pool_dot16(k2, k2)), qs = group_sum<8>(pool_dot16(q2, q2));
            kn = rsqrtf(ks + 1e-6f);
            qn = rsqrtf(qs + 1e-6f) * d.scale;
        }
        float part[2], sk[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) part[p] = pool_dot16(st[p], k2);
        const float skt = pool_sum2(part, l8);
#pragma unroll
        for (int p = 0; p < 2; ++p) sk[p] = __shfl_sync(kAll, skt, gbase + 4 * p);
        const f2_t a2 = f2(m.alpha, m.alpha);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float u = m.beta * (vv[p] - m.alpha * kn * sk[p]) * kn;
            const f2_t u2 = f2(u, u);
#pragma unroll
            for (int c = 0; c < 8; ++c) st[p][c] = fma2(a2, st[p][c], mul2(u2, k2[c]));
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) part[p] = pool_dot16(st[p], q2);
        const float ot = pool_sum2(part, l8) * qn;
        // the row that this buffer held has been finished
        if (run && !mbar_wait_warp(&sm.o_empty[ob], (uint32_t)(((it / kPoolRows) & 1) ^ 1), d.status)) break;
        if (run && (l8 & 3) == 0) sm.o[ob][rbase + 64 * (l8 >> 2)] = ot;
        __syncwarp();
        if (run && lane == 0) mbar_arrive(&sm.o_full[ob]);
        if (run) {
            float *out = d.pool + ((int64_t)m.slot * Hv + m.head) * kD * kD + rbase * kD + 4 * l8;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    __stcs(reinterpret_cast<float4 *>(out + 64 * p * kD + 32 * j),
                           make_float4(f2lo(st[p][2 * j]), f2hi(st[p][2 * j]), f2lo(st[p][2 * j + 1]), f2hi(st[p][2 * j + 1])));
        }
        if (!run) pdl_wait();
    }
}

template <bool TAIL>
cudaError_t launch_pooled_t(PooledDecodeArgs d, cudaStream_t st) {
    static PerDevice<int> sm_count;   // the shared-memory attribute is set per device alongside
    int sms = 0;
    const cudaError_t e = sm_count.get(
        [](int dev, int &r) {
            cudaError_t x = cudaFuncSetAttribute(gdn_decode128_pooled_kernel<TAIL>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kPoolSmem);
            if (x == cudaSuccess) x = cudaDeviceGetAttribute(&r, cudaDevAttrMultiProcessorCount, dev);
            return x;
        },
        &sms);
    if (e != cudaSuccess) return e;
    // heads per unit: doubled while every SM keeps sixteen units or more (each looks through the batch's slots once)
    d.unit_heads = 1;
    while (d.unit_heads < d.Hv && (int64_t)d.B * ((d.Hv + 2 * d.unit_heads - 1) / (2 * d.unit_heads)) >= 16 * (int64_t)sms)
        d.unit_heads *= 2;
    const int units_row = (d.Hv + d.unit_heads - 1) / d.unit_heads;
    return launch_pdl(gdn_decode128_pooled_kernel<TAIL>, dim3((unsigned)units_row, (unsigned)d.B), dim3(kPoolThreads), kPoolSmem, st, d);
}

}  // namespace

cudaError_t launch_decode_pooled(const PooledDecodeArgs &d, cudaStream_t st) {
    return d.xq ? launch_pooled_t<true>(d, st) : launch_pooled_t<false>(d, st);
}

}  // namespace gdn
