// FP8 (E4M3) with one fp32 scale per block of 128 values along K: the encoders of activations
// (1 x 128 blocks) and weights (128 x 128 blocks), and the gated tail that writes its output in this
// form. For a block with largest magnitude amax (a NaN is passed over),
//     s = max(amax / 448, 2^-126),   code_j = E4M3(x_j / s)   (as x_j * (1 / s), saturating),
// so E4M3(code_j) * s stands for x_j. All of it in fp32.
//
// All three are HBM-bound streams (about 3 to 12 operations a value): a block of 128 values of a row is
// 16 lanes of 8 values, so its maximum is four shuffles, a warp's loads are 512 or 1024 consecutive
// bytes, and every thread issues the loads of several blocks before it uses any.
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kFp8Threads = 256;
constexpr int kFp8Lanes = 16;                            // lanes per block of 128 values
constexpr int kFp8Blocks = kFp8Threads / kFp8Lanes;      // blocks per CTA pass
constexpr int kFp8Unroll = 4;

// Eight consecutive values as loaded, or zeros.
template <bool BF16>
struct Fp8In {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *base, int64_t idx, bool live) {
        a = b = make_uint4(0u, 0u, 0u, 0u);
        if (!live) return;
        if constexpr (BF16) {
            a = *reinterpret_cast<const uint4 *>(reinterpret_cast<const __nv_bfloat16 *>(base) + idx);
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(base) + idx);
            a = p[0];
            b = p[1];
        }
    }
    __device__ __forceinline__ void get(f2_t (&v)[4]) const {
        if constexpr (BF16) {
            v[0] = bf16x2_to_f2(a.x); v[1] = bf16x2_to_f2(a.y); v[2] = bf16x2_to_f2(a.z); v[3] = bf16x2_to_f2(a.w);
        } else {
            v[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y)); v[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
            v[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y)); v[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
        }
    }
};

__device__ __forceinline__ float amax_f2(const f2_t (&v)[4]) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(f2lo(v[k])), fabsf(f2hi(v[k]))));
    return m;
}
__device__ __forceinline__ uint2 pack8_f2(const f2_t (&v)[4], float r) {
    return make_uint2(fp8_pack4(f2lo(v[0]), f2hi(v[0]), f2lo(v[1]), f2hi(v[1]), r),
                      fp8_pack4(f2lo(v[2]), f2hi(v[2]), f2lo(v[3]), f2hi(v[3]), r));
}

// Maximum over the 16 lanes of a block (all lanes of the warp take part).
__device__ __forceinline__ float group16_max(float m) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

// Block i of x is row i / kb, values 128 (i % kb) ..; the last block of a row may be short (K % 16 == 0,
// so a lane's eight values are all inside or all outside).
template <bool BF16>
__global__ void __launch_bounds__(kFp8Threads)
fp8_quantize_act_kernel(const void *__restrict__ x, int64_t ldx, int32_t nblocks, int32_t kb, int32_t K,
                        uint8_t *__restrict__ xq, float *__restrict__ xs) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int U = kFp8Unroll;
    const int l = threadIdx.x % kFp8Lanes;
    const int64_t stride = (int64_t)gridDim.x * kFp8Blocks;
    const int64_t first = (int64_t)blockIdx.x * kFp8Blocks;
    // the loop condition is uniform over the CTA (the shuffles need whole warps)
    for (int64_t i0 = first; i0 < nblocks; i0 += U * stride) {
        Fp8In<BF16> in[U];
        int32_t row[U], col[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * stride + threadIdx.x / kFp8Lanes;
            row[u] = (int32_t)min(i, (int64_t)nblocks - 1) / kb;
            col[u] = ((int32_t)min(i, (int64_t)nblocks - 1) - row[u] * kb) * 128 + 8 * l;
            live[u] = i < nblocks && col[u] < K;
            in[u].load(x, row[u] * ldx + col[u], live[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2_t v[4];
            in[u].get(v);
            float r;
            const float s = fp8_block_scale(group16_max(amax_f2(v)), r);
            if (!live[u]) continue;
            *reinterpret_cast<uint2 *>(xq + (int64_t)row[u] * K + col[u]) = pack8_f2(v, r);
            if (l == 0) xs[(int64_t)row[u] * kb + col[u] / 128] = s;
        }
    }
}

// One CTA per 128 x 128 block of w [N, K]: 16 lanes a row, 16 rows a pass, eight passes held in
// registers between the maximum and the encoding, so w is read once.
template <bool BF16>
__global__ void __launch_bounds__(kFp8Threads)
fp8_quantize_weight_kernel(const void *__restrict__ w, int64_t ldw, int32_t N, int32_t K, int32_t kb,
                           uint8_t *__restrict__ wq, float *__restrict__ ws) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[kFp8Threads / 32];
    const int tid = threadIdx.x;
    const int32_t kblk = blockIdx.x % kb, nblk = blockIdx.x / kb;
    const int32_t col = kblk * 128 + 8 * (tid % kFp8Lanes), row0 = nblk * 128 + tid / kFp8Lanes;
    Fp8In<BF16> in[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) in[p].load(w, (row0 + 16 * p) * ldw + col, row0 + 16 * p < N && col < K);
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        f2_t v[4];
        in[p].get(v);
        m = fmaxf(m, amax_f2(v));
    }
    m = group16_max(m);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
    if (tid % 32 == 0) part[tid / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFp8Threads / 32; ++i) m = fmaxf(m, part[i]);
    float r;
    const float s = fp8_block_scale(m, r);
    if (tid == 0) ws[blockIdx.x] = s;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        if (row0 + 16 * p >= N || col >= K) continue;
        f2_t v[4];
        in[p].get(v);
        *reinterpret_cast<uint2 *>(wq + (int64_t)(row0 + 16 * p) * K + col) = pack8_f2(v, r);
    }
}

// The gated tail ("Red Lite dev15d - DeltaNet gated tail", Pinned graph semantics, steps 1-5) into FP8:
// a block of 128 columns is 128 / D heads, each normalised over its own D / 8 lanes (gated_row8, the
// plain tail's arithmetic), then one maximum and one scale over the 16 lanes. The codes come from the
// fp32 values, with no rounding to bf16 between: the same bytes as the plain tail with an fp32 output
// followed by fp8_quantize_act.
template <int D, bool BF16>
__global__ void __launch_bounds__(kFp8Threads)
gated_rmsnorm_fp8_kernel(const void *__restrict__ o, const void *__restrict__ z, const float *__restrict__ w,
                         float eps, int32_t nblocks, int32_t kb, int32_t K, uint8_t *__restrict__ xq,
                         float *__restrict__ xs) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int U = kFp8Unroll;
    const int l = threadIdx.x % kFp8Lanes, wcol = 8 * l % D;
    f2_t w2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w2[k] = f2(w[wcol + 2 * k], w[wcol + 2 * k + 1]);
    const int64_t stride = (int64_t)gridDim.x * kFp8Blocks;
    const int64_t first = (int64_t)blockIdx.x * kFp8Blocks;
    for (int64_t i0 = first; i0 < nblocks; i0 += U * stride) {   // uniform over the CTA
        Fp8In<BF16> ro[U], rz[U];
        int32_t blk[U];
        int64_t off[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * stride + threadIdx.x / kFp8Lanes;
            blk[u] = (int32_t)min(i, (int64_t)nblocks - 1);
            const int32_t row = blk[u] / kb, col = (blk[u] - row * kb) * 128 + 8 * l;
            off[u] = (int64_t)row * K + col;
            live[u] = i < nblocks && col < K;
            ro[u].load(o, off[u], live[u]);
            rz[u].load(z, off[u], live[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2_t o2[4], z2[4], y2[4];
            ro[u].get(o2);
            rz[u].get(z2);
            gated_row8<D / 8>(o2, z2, w2, 1.0f / (float)D, eps, y2);
            float r;
            const float s = fp8_block_scale(group16_max(live[u] ? amax_f2(y2) : 0.0f), r);
            if (!live[u]) continue;
            *reinterpret_cast<uint2 *>(xq + off[u]) = pack8_f2(y2, r);
            if (l == 0) xs[blk[u]] = s;
        }
    }
}

unsigned fp8_grid(int64_t nblocks) {
    const int64_t per = (int64_t)kFp8Blocks * kFp8Unroll;
    const int64_t want = (nblocks + per - 1) / per, cap = 148 * 8;
    return (unsigned)(want < cap ? want : cap);
}

template <int D>
cudaError_t launch_tail_fp8_d(const Fp8TailArgs &t, int32_t kb, cudaStream_t st) {
    const int32_t nblocks = t.M * kb, K = t.Hv * t.D;
    if (t.in_bf16)
        return launch_pdl(gated_rmsnorm_fp8_kernel<D, true>, dim3(fp8_grid(nblocks)), dim3(kFp8Threads), 0, st, t.o, t.z,
                          t.w, t.eps, nblocks, kb, K, t.xq, t.xs);
    return launch_pdl(gated_rmsnorm_fp8_kernel<D, false>, dim3(fp8_grid(nblocks)), dim3(kFp8Threads), 0, st, t.o, t.z,
                      t.w, t.eps, nblocks, kb, K, t.xq, t.xs);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs &a, cudaStream_t st) {
    const int32_t kb = (a.K + 127) / 128;
    if (a.weight) {
        const dim3 grid((unsigned)(kb * ((a.rows + 127) / 128)));
        if (a.in_bf16)
            return launch_pdl(fp8_quantize_weight_kernel<true>, grid, dim3(kFp8Threads), 0, st, a.x, a.ldx, a.rows, a.K, kb,
                              a.xq, a.xs);
        return launch_pdl(fp8_quantize_weight_kernel<false>, grid, dim3(kFp8Threads), 0, st, a.x, a.ldx, a.rows, a.K, kb,
                          a.xq, a.xs);
    }
    const int32_t nblocks = a.rows * kb;
    if (a.in_bf16)
        return launch_pdl(fp8_quantize_act_kernel<true>, dim3(fp8_grid(nblocks)), dim3(kFp8Threads), 0, st, a.x, a.ldx,
                          nblocks, kb, a.K, a.xq, a.xs);
    return launch_pdl(fp8_quantize_act_kernel<false>, dim3(fp8_grid(nblocks)), dim3(kFp8Threads), 0, st, a.x, a.ldx,
                      nblocks, kb, a.K, a.xq, a.xs);
}

cudaError_t launch_gated_rmsnorm_fp8(const Fp8TailArgs &t, cudaStream_t st) {
    const int32_t kb = (t.Hv * t.D + 127) / 128;
    switch (t.D) {
        case 16: return launch_tail_fp8_d<16>(t, kb, st);
        case 32: return launch_tail_fp8_d<32>(t, kb, st);
        case 64: return launch_tail_fp8_d<64>(t, kb, st);
        case 128: return launch_tail_fp8_d<128>(t, kb, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gdn
