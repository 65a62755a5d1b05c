// The products of a few rows (decode: up to 16) by E4M3 weights with fp32 block scales.
//
// Here the weights are the larger operand by far: N K bytes against M K, each used 2 M times, so
// the time is their way from memory (and, for one token, mostly the launch).  The tensor-memory kernel
// spends some 300 cycles per 128-K block on its hand-overs (copy, MMA, scaled sums); a chain of 23
// blocks then takes longer than the weights' copy.  So here every warp is on its own: it loads its
// weights from global memory straight into the operands of mma.sync m16n8k16 (weights the 16 rows,
// tokens the 8 columns; E4M3 to f16 is exact, and two conversions and an f16 product took less than the E4M3
// form of mma.sync), scales each K block's sums in registers, and the CTA's eight warps, which split
// K, add up at the end in a fixed order.
//
// One token, in a run of calls on weights that L2 holds in part: 5120 x 2880 in 4.6 us (10.2 in the other kernel),
// gated 2 x 2880 x 2880 in 6.3 us (11.8); all weights from memory: 5.7 us (14.8 MB, 2.6 TB/s) and 7.5 us (16.6 MB,
// 2.2 TB/s).  Latency: of the launch, behind which the loads start, of one round of loads (eight of ten samples of a
// warp wait for memory) and of the join, and for the gated form of the cluster's exchange.
//
// Operands without shuffles: the K order within a product is free as long as both sides use the
// same.  Lane (g, t) takes the 16 bytes t of a 64-byte K segment of rows g and g + 8 (of token g); each of their
// words, as two f16 pairs, is one MMA's a0, a2 (a1, a3; b0, b1).  So every load is 16 bytes wide and four lanes
// take 64 contiguous bytes.
//
// Gated: a CTA takes 16 gate rows and their 16 linear rows; a row's 128-column block of h lies in a
// cluster of eight CTAs, which exchange its maximum through distributed shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_kernels.cuh"
#include "fp8_ptx.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr int FEW_WARPS = 8;            // warps of a CTA: parts of K
constexpr int FEW_ROWS = 16;            // weight rows of a CTA (gated: of each half)

// D += A B for f16 operands (products of E4M3 numbers are exact), fp32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sixteen E4M3 bytes to eight f16 pairs, exactly.
__device__ __forceinline__ void to_f16(const uint4 &v, uint32_t (&h)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
            : "r"(w[i]));
}

// Sixteen bytes, or zeros.  Volatile, so that a round's loads are all issued before its products: left to
// the compiler, they move down to their uses and a warp waits for memory several times a round.
__device__ __forceinline__ uint4 load16(const uint8_t *p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
        "mov.b32 %3, 0;\n\t@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p), "r"((int)in));
    return v;
}

template <typename T>
__device__ __forceinline__ void store_as(void *c, long long at, float v) { static_cast<T *>(c)[at] = static_cast<T>(v); }

constexpr int few_ahead(int nt, bool gated) { return nt > 1 ? 1 : gated ? 2 : 3; }
// ... and CTAs to an SM: every CTA of a grid of FP8_FEW_CTAS to an SM is there at once
constexpr int few_ctas(bool gated) { return gated ? 2 : FP8_FEW_CTAS; }

}  // namespace

// NT: tokens / 8, rounded up.
template <int NT, bool GATED>
__global__ void __launch_bounds__(FEW_WARPS * 32, few_ctas(GATED)) fp8_few_kernel(const Fp8FewParams p) {
    constexpr int H = GATED ? 2 : 1;                // row groups: the gate's and the linear part's
    constexpr int TOK = NT * 8;
    __shared__ float part[FEW_WARPS][H * FEW_ROWS][TOK + 1];
    __shared__ float row_max[8][TOK];               // gated: the cluster's CTAs' maxima
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * FEW_ROWS;
    if constexpr (GATED) cluster_arrive();          // (waited for before the first access to a peer)
    pdl_wait();
    pdl_trigger();

    // this warp's K blocks
    const int kb0 = (int)((long long)p.KB * warp / FEW_WARPS), kb1 = (int)((long long)p.KB * (warp + 1) / FEW_WARPS);
    const uint8_t *w[H][2];                         // rows g and g + 8 of each group
    bool in_n[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int n = n0 + g + 8 * r;
        in_n[r] = n < p.N;
#pragma unroll
        for (int h = 0; h < H; ++h) w[h][r] = p.b + ((long long)h * p.N + min(n, p.N - 1)) * p.K + 16 * t;
    }
    float sum[H][NT][4];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[h][n][i] = 0.0f;

    constexpr int AHEAD = few_ahead(NT, GATED);     // K blocks whose loads are in flight together
    for (int kb = kb0; kb < kb1; kb += AHEAD) {
        uint4 wv[AHEAD][H][2][2], av[AHEAD][NT][2];
        float sa[AHEAD][NT][2], sb[AHEAD][H];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int k0 = (kb + u) * FP8_KS;
            const bool in_u = kb + u < kb1;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool in_k = in_u && k0 + 64 * s + 16 * t < p.K;       // K is a multiple of 16
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int r = 0; r < 2; ++r) wv[u][h][r][s] = load16(w[h][r] + k0 + 64 * s, in_k && in_n[r]);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const bool in_k = in_u && k0 + 64 * s + 16 * t < p.K;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int m = 8 * n + g;
                    av[u][n][s] = load16(p.a + (long long)m * p.lda + k0 + 64 * s + 16 * t, in_k && m < p.M);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int m = 8 * n + 2 * t + j;
                    sa[u][n][j] = in_u && m < p.M ? p.a_scale[(long long)m * p.KB + kb + u] : 0.0f;
                }
#pragma unroll
            for (int h = 0; h < H; ++h)
                sb[u][h] = in_u ? p.b_scale[((long long)h * p.NB + n0 / FP8_BLOCK) * p.KB + kb + u] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            float d[H][NT][4];
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[h][n][i] = 0.0f;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                uint32_t x[H][8], y[H][8];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    to_f16(wv[u][h][0][s], x[h]);
                    to_f16(wv[u][h][1][s], y[h]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t v[8];
                    to_f16(av[u][n][s], v);
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            mma_f16(d[h][n], x[h][j], y[h][j], x[h][j + 1], y[h][j + 1], v[j], v[j + 1]);
                }
            }
            // (a block past the warp's last one adds nothing, whatever the scales are)
            if (kb + u < kb1) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int h = 0; h < H; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sum[h][n][i] = fmaf(d[h][n][i], sa[u][n][i & 1] * sb[u][h], sum[h][n][i]);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[warp][h * FEW_ROWS + g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = sum[h][n][i];
    __syncthreads();

    // the warps' parts, in order; a thread takes one column of c (or h) of one token
    auto total = [&](int row, int m) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < FEW_WARPS; ++i) v += part[i][row][m];
        return v;
    };
    const int col = threadIdx.x % FEW_ROWS, n = n0 + col;
    if constexpr (!GATED) {
        if (n < p.N)
            for (int m = threadIdx.x / FEW_ROWS; m < p.M; m += FEW_WARPS * 32 / FEW_ROWS) {
                float v = total(col, m);
                if (p.bias) v += __uint_as_float((uint32_t)p.bias[n] << 16);
                const long long at = (long long)m * p.ldc + n;
                if (p.residual) {
                    const long long ar = (long long)m * p.ldr + n;
                    v += p.type == FP8_BF16   ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.residual)[ar])
                         : p.type == FP8_FP16 ? __half2float(static_cast<const __half *>(p.residual)[ar])
                                              : static_cast<const float *>(p.residual)[ar];
                }
                if (p.type == FP8_BF16) store_as<__nv_bfloat16>(p.c, at, v);
                else if (p.type == FP8_FP16) store_as<__half>(p.c, at, v);
                else store_as<float>(p.c, at, v);
            }
    } else {
        constexpr int PASSES = (TOK * FEW_ROWS + FEW_WARPS * 32 - 1) / (FEW_WARPS * 32);
        const uint32_t rank = cluster_ctarank();
        float hv[PASSES];
        cluster_wait();                             // every CTA of the cluster runs
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int m = threadIdx.x / FEW_ROWS + i * (FEW_WARPS * 32 / FEW_ROWS);
            float amax = 0.0f;
            if (m < TOK && n < p.N) {
                float gt = total(col, m), u = total(FEW_ROWS + col, m);
                if (p.bias) {
                    gt += __uint_as_float((uint32_t)p.bias[n] << 16);
                    u += __uint_as_float((uint32_t)p.bias[p.N + n] << 16);
                }
                gt = fmin_nan(gt, p.limit);
                u = fmax_nan(fmin_nan(u, p.limit), -p.limit);
                hv[i] = gt * rcp_approx(1.0f + exp2_approx(p.minus_alpha_log2e * gt)) * (u + p.shift);
                amax = fabsf(hv[i]);
            }
            // over the 16 columns (neighbouring lanes), then to every CTA of the cluster
#pragma unroll
            for (int o = 8; o; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (col < 8 && m < TOK) st_cluster_f32(map_to_rank(smem_addr(&row_max[rank][m]), (uint32_t)col), amax);
        }
        cluster_sync();
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
            const int m = threadIdx.x / FEW_ROWS + i * (FEW_WARPS * 32 / FEW_ROWS);
            if (m < p.M && n < p.N) {
                float amax = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) amax = fmax_nan(amax, row_max[c][m]);
                const float s = fmax_nan(amax / FP8_MAX, FP8_SCALE_MIN);
                p.h[(long long)m * p.N + n] = (uint8_t)f32x2_to_e4m3x2(hv[i] * (1.0f / s), 0.0f);
                if (n % FP8_BLOCK == 0) p.h_scale[(long long)m * p.NB + n / FP8_BLOCK] = s;
            }
        }
    }
}

template <int NT, bool GATED>
static cudaError_t launch_few_t(const Fp8FewParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    // gated: whole clusters, one for each 128-column block
    cfg.gridDim = dim3(GATED ? p.NB * 8 : (p.N + FEW_ROWS - 1) / FEW_ROWS);
    cfg.blockDim = dim3(FEW_WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 8;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = GATED ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fp8_few_kernel<NT, GATED>, p);
}

// Loads the kernels (once per device, before the first launch, which may be captured).
cudaError_t fp8_few_setup() {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, fp8_few_kernel<1, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, fp8_few_kernel<2, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, fp8_few_kernel<1, true>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, fp8_few_kernel<2, true>);
    return e;
}

cudaError_t launch_fp8_few(const Fp8FewParams &p, int gated, cudaStream_t s) {
    if (gated) return p.M <= 8 ? launch_few_t<1, true>(p, s) : launch_few_t<2, true>(p, s);
    return p.M <= 8 ? launch_few_t<1, false>(p, s) : launch_few_t<2, false>(p, s);
}

}  // namespace moe
