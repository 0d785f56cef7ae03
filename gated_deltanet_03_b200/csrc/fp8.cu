// FP8 (E4M3) with one fp32 scale per block of 128 values along K: the encoders of activations
// (1 x 128 blocks) and weights (128 x 128 blocks), and the gated tail that writes its output in this
// form. For a block with largest magnitude amax (a NaN is passed over),
//     s = max(amax / 448, 2^-126),   code_j = E4M3(x_j / s)   (as x_j * (1 / s), saturating),
// so E4M3(code_j) * s stands for x_j. All of it in fp32.
//
// All three are HBM-bound streams, with arithmetic close behind: with 8 bf16 values a thread the scale, the index and
// the reductions were most of 11 instructions a value (tail of 32768 x 32 heads 131 us). So a lane takes 32 bytes of a
// block, one wide load: 16 bf16 values (8 lanes a block: 116 us, 89 % of the measured copy rate; encoder 96 %) or 8
// fp32 ones (16 lanes; 16 values a lane there took 124 us against 96 at 16384 rows). Long inputs go four blocks a
// thread, all loads before any use; short ones one block a thread (256 x 2048: 1.7 us against 2.8).
#include "common.cuh"
#include "kernels.h"

namespace gdn {
namespace {

constexpr int kFp8Threads = 256;
constexpr int kFp8Long = 4;                              // blocks per thread and turn for long inputs

// Layout of a block of 128 values by input type: NC chunks of 8 values (32 bytes) a lane.
template <bool BF16>
struct Fp8Lay {
    static constexpr int NC = BF16 ? 2 : 1;
    static constexpr int LANES = 16 / NC;
    static constexpr int BLOCKS = kFp8Threads / LANES;   // blocks per CTA pass
};

__device__ __forceinline__ void ld_global_32b(const void *p, uint32_t (&r)[8]) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
}

// A lane's 32 bytes as loaded (WIDE: they are 32-byte aligned), or zeros.
template <bool BF16>
struct Fp8In {
    uint32_t w[8];
    template <bool WIDE>
    __device__ __forceinline__ void load(const void *base, int64_t idx, bool live) {
        const uint8_t *p = reinterpret_cast<const uint8_t *>(base) + idx * (BF16 ? 2 : 4);
        if (!live) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0u;
        } else if constexpr (WIDE) {
            ld_global_32b(p, w);
        } else {
            const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
    }
    // chunk c: eight values
    __device__ __forceinline__ void get(int c, f2_t (&v)[4]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (BF16) v[k] = bf16x2_to_f2(w[4 * c + k]);
            else v[k] = f2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
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
template <int NC>
__device__ __forceinline__ void store_codes(uint8_t *p, const f2_t (&v)[NC][4], float r) {
    const uint2 x = pack8_f2(v[0], r);
    if constexpr (NC == 2) {
        const uint2 y = pack8_f2(v[1], r);
        *reinterpret_cast<uint4 *>(p) = make_uint4(x.x, x.y, y.x, y.y);
    } else {
        *reinterpret_cast<uint2 *>(p) = x;
    }
}

// Maximum over the lanes of a block (all lanes of the warp take part).
template <int LANES>
__device__ __forceinline__ float block_max(float m) {
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    return m;
}

// Block i of x is row i / kb, values 128 (i % kb) ..; the last block of a row may be short (K % 16 == 0,
// so a lane's values are all inside or all outside).
template <bool BF16, bool WIDE, int U>
__global__ void __launch_bounds__(kFp8Threads, BF16 ? 3 : 4)
fp8_quantize_act_kernel(const void *__restrict__ x, int64_t ldx, int32_t nblocks, int32_t kb, int32_t K,
                        uint8_t *__restrict__ xq, float *__restrict__ xs) {
    using L = Fp8Lay<BF16>;
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x % L::LANES;
    const int64_t stride = (int64_t)gridDim.x * L::BLOCKS;
    const int64_t first = (int64_t)blockIdx.x * L::BLOCKS;
    // the loop condition is uniform over the CTA (the shuffles need whole warps)
    for (int64_t i0 = first; i0 < nblocks; i0 += U * stride) {
        Fp8In<BF16> in[U];
        int32_t row[U], col[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * stride + threadIdx.x / L::LANES;
            row[u] = (int32_t)min(i, (int64_t)nblocks - 1) / kb;
            col[u] = ((int32_t)min(i, (int64_t)nblocks - 1) - row[u] * kb) * 128 + 8 * L::NC * l;
            live[u] = i < nblocks && col[u] < K;
            in[u].template load<WIDE>(x, row[u] * ldx + col[u], live[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2_t v[L::NC][4];
            float m = 0.0f, r;
#pragma unroll
            for (int c = 0; c < L::NC; ++c) {
                in[u].get(c, v[c]);
                m = fmaxf(m, amax_f2(v[c]));
            }
            const float s = fp8_block_scale(block_max<L::LANES>(m), r);
            if (!live[u]) continue;
            store_codes<L::NC>(xq + (int64_t)row[u] * K + col[u], v, r);
            if (l == 0) xs[(int64_t)row[u] * kb + col[u] / 128] = s;
        }
    }
}

// One CTA per 128 x 128 block of w [N, K], held in registers between the maximum and the encoding, so w is
// read once.
template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(kFp8Threads, BF16 ? 3 : 2)
fp8_quantize_weight_kernel(const void *__restrict__ w, int64_t ldw, int32_t N, int32_t K, int32_t kb,
                           uint8_t *__restrict__ wq, float *__restrict__ ws) {
    using L = Fp8Lay<BF16>;
    constexpr int P = 128 / L::BLOCKS;   // passes of BLOCKS rows
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float part[kFp8Threads / 32];
    const int tid = threadIdx.x;
    const int32_t nblk = blockIdx.x / kb, kblk = blockIdx.x - nblk * kb;
    const int32_t col = kblk * 128 + 8 * L::NC * (tid % L::LANES);
    const int64_t row0 = (int64_t)nblk * 128 + tid / L::LANES;
    Fp8In<BF16> in[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
        in[p].template load<WIDE>(w, (row0 + L::BLOCKS * p) * ldw + col, row0 + L::BLOCKS * p < N && col < K);
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int c = 0; c < L::NC; ++c) {
            f2_t v[4];
            in[p].get(c, v);
            m = fmaxf(m, amax_f2(v));
        }
    m = block_max<32>(m);
    if (tid % 32 == 0) part[tid / 32] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFp8Threads / 32; ++i) m = fmaxf(m, part[i]);
    float r;
    const float s = fp8_block_scale(m, r);
    if (tid == 0) ws[blockIdx.x] = s;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (row0 + L::BLOCKS * p >= N || col >= K) continue;
        f2_t v[L::NC][4];
#pragma unroll
        for (int c = 0; c < L::NC; ++c) in[p].get(c, v[c]);
        store_codes<L::NC>(wq + (row0 + L::BLOCKS * p) * K + col, v, r);
    }
}

// The gated tail ("Red Lite dev15d - DeltaNet gated tail", Pinned graph semantics, steps 1-5) into FP8:
// a block of 128 columns is 128 / D heads, each normalised over its own lanes, then one maximum and one scale
// over the block's. The codes come from the fp32 values, with no rounding to bf16 between: the same bytes as the
// plain tail with an fp32 output followed by fp8_quantize_act. (The plain tail has 8 values a lane and adds its
// lanes' squares from the farthest to the nearest; where a lane has two chunks here, they are the nearest.)
template <int D, bool BF16, bool WIDE, int U>
__global__ void __launch_bounds__(kFp8Threads, U == 1 ? 4 : BF16 ? 2 : 4)
gated_rmsnorm_fp8_kernel(const void *__restrict__ o, const void *__restrict__ z, const float *__restrict__ w,
                         float eps, int32_t nblocks, int32_t kb, int32_t K, uint8_t *__restrict__ xq,
                         float *__restrict__ xs) {
    using L = Fp8Lay<BF16>;
    constexpr int NC = L::NC;
    pdl_launch_dependents();
    pdl_wait();
    const int l = threadIdx.x % L::LANES, wcol = 8 * NC * l % D;
    f2_t w2[NC][4];
#pragma unroll
    for (int k = 0; k < 4 * NC; ++k) w2[k / 4][k % 4] = f2(w[wcol + 2 * k], w[wcol + 2 * k + 1]);
    const int64_t stride = (int64_t)gridDim.x * L::BLOCKS;
    const int64_t first = (int64_t)blockIdx.x * L::BLOCKS;
    for (int64_t i0 = first; i0 < nblocks; i0 += U * stride) {   // uniform over the CTA
        Fp8In<BF16> ro[U], rz[U];
        int32_t blk[U];
        int64_t off[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * stride + threadIdx.x / L::LANES;
            blk[u] = (int32_t)min(i, (int64_t)nblocks - 1);
            const int32_t row = blk[u] / kb, col = (blk[u] - row * kb) * 128 + 8 * NC * l;
            off[u] = (int64_t)row * K + col;
            live[u] = i < nblocks && col < K;
            ro[u].template load<WIDE>(o, off[u], live[u]);
            rz[u].template load<WIDE>(z, off[u], live[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            f2_t o2[NC][4], z2[4], y2[NC][4];
            float sq[NC], m = 0.0f, r;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                ro[u].get(c, o2[c]);
                sq[c] = row_sumsq8(o2[c]);
            }
#pragma unroll
            for (int n = D / 16 / NC; n > 0; n >>= 1)
#pragma unroll
                for (int c = 0; c < NC; ++c) sq[c] += __shfl_xor_sync(0xffffffffu, sq[c], n);
            const float inv_rms = rsqrtf(__fmaf_rn(NC == 2 ? sq[0] + sq[NC - 1] : sq[0], 1.0f / (float)D, eps));
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                rz[u].get(c, z2);
                gated_apply8(o2[c], z2, w2[c], inv_rms, y2[c]);
            }
            const float s = fp8_block_scale(block_max<L::LANES>(live[u] ? (NC == 2 ? fmaxf(amax_f2(y2[0]), amax_f2(y2[NC - 1])) : amax_f2(y2[0])) : 0.0f), r);
            if (!live[u]) continue;
            store_codes<NC>(xq + off[u], y2, r);
            if (l == 0) xs[blk[u]] = s;
        }
    }
}

// As many CTAs as there are passes, up to eight an SM.
template <bool BF16>
unsigned fp8_grid(int64_t nblocks) {
    const int64_t want = (nblocks + Fp8Lay<BF16>::BLOCKS - 1) / Fp8Lay<BF16>::BLOCKS, cap = 148 * 8;
    return (unsigned)(want < cap ? want : cap);
}
// Long: more than one turn of one block a thread on the largest grid.
template <bool BF16>
bool fp8_long(int64_t nblocks) {
    return nblocks > 148 * 8 * Fp8Lay<BF16>::BLOCKS;
}

bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <int D, bool BF16, bool WIDE>
cudaError_t launch_tail_t(const Fp8TailArgs &t, cudaStream_t st) {
    const int32_t K = t.Hv * t.D, kb = (K + 127) / 128, nblocks = t.M * kb;
    // (fp32: two blocks a thread hold as many bytes, and four spill)
    if (fp8_long<BF16>(nblocks))
        return launch_pdl(gated_rmsnorm_fp8_kernel<D, BF16, WIDE, BF16 ? kFp8Long : 2>, dim3(fp8_grid<BF16>(nblocks)), dim3(kFp8Threads),
                          0, st, t.o, t.z, t.w, t.eps, nblocks, kb, K, t.xq, t.xs);
    return launch_pdl(gated_rmsnorm_fp8_kernel<D, BF16, WIDE, 1>, dim3(fp8_grid<BF16>(nblocks)), dim3(kFp8Threads), 0, st, t.o, t.z,
                      t.w, t.eps, nblocks, kb, K, t.xq, t.xs);
}

template <int D>
cudaError_t launch_tail_d(const Fp8TailArgs &t, cudaStream_t st) {
    const bool wide = aligned32(t.o) && aligned32(t.z);   // rows are multiples of 16 values
    if (t.in_bf16) return wide ? launch_tail_t<D, true, true>(t, st) : launch_tail_t<D, true, false>(t, st);
    return wide ? launch_tail_t<D, false, true>(t, st) : launch_tail_t<D, false, false>(t, st);
}

template <bool BF16, bool WIDE>
cudaError_t launch_quantize_t(const Fp8QuantArgs &a, cudaStream_t st) {
    const int32_t kb = (a.K + 127) / 128;
    if (a.weight)
        return launch_pdl(fp8_quantize_weight_kernel<BF16, WIDE>, dim3((unsigned)(kb * ((a.rows + 127) / 128))), dim3(kFp8Threads), 0,
                          st, a.x, a.ldx, a.rows, a.K, kb, a.xq, a.xs);
    const int32_t nblocks = a.rows * kb;
    if (fp8_long<BF16>(nblocks))
        return launch_pdl(fp8_quantize_act_kernel<BF16, WIDE, kFp8Long>, dim3(fp8_grid<BF16>(nblocks)), dim3(kFp8Threads), 0, st, a.x,
                          a.ldx, nblocks, kb, a.K, a.xq, a.xs);
    return launch_pdl(fp8_quantize_act_kernel<BF16, WIDE, 1>, dim3(fp8_grid<BF16>(nblocks)), dim3(kFp8Threads), 0, st, a.x, a.ldx,
                      nblocks, kb, a.K, a.xq, a.xs);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs &a, cudaStream_t st) {
    const bool wide = aligned32(a.x) && a.ldx % (a.in_bf16 ? 16 : 8) == 0;   // every row starts on 32 bytes
    if (a.in_bf16) return wide ? launch_quantize_t<true, true>(a, st) : launch_quantize_t<true, false>(a, st);
    return wide ? launch_quantize_t<false, true>(a, st) : launch_quantize_t<false, false>(a, st);
}

cudaError_t launch_gated_rmsnorm_fp8(const Fp8TailArgs &t, cudaStream_t st) {
    switch (t.D) {
        case 16: return launch_tail_d<16>(t, st);
        case 32: return launch_tail_d<32>(t, st);
        case 64: return launch_tail_d<64>(t, st);
        case 128: return launch_tail_d<128>(t, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace gdn
