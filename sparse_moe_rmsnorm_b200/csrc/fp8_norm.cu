// RMS norm with the residual's addition, the normalised rows in E4M3 with a scale per 128 elements.
//
//   n = x + r,  y = n / sqrt(mean(n^2) + eps) * w          (fp32 throughout)
//   s_b = max(max_{i in b} |y_i| / 448, 2^-126),  q = e4m3(y (1 / s_b))
//
// The norm is the routed block's (no bias, no mean subtraction: pnsm.cn overview, section 2.3;
// "gpt-oss-20B" hub page, section 3.2) and stands beside it: here the rows leave in the form the
// dense 8-bit products read.  Bound by HBM: x, r, the sum and q move once (8192 rows of 2880, bf16:
// 166 MB in 30.2 us in a run of calls, 27.3 from a graph whose calls write the same results, 0.84 and 0.92 of the
// measured copy rate), and next by instruction issue (75% of the slots): the arithmetic is on pairs (f32x2), which
// took it from 39 us.  One row: 1.5 us from a graph, a launch; in a run of calls the host's 5.  One CTA holds a row in
// registers, 8 or 16 elements per thread, so the row is read once and the second pass (the scaling) needs no memory; a block's 128
// elements sit in 16 neighbouring lanes, so its maximum is four shuffles.  A row's sum adds the
// elements of a thread in two halves, then a tree over lanes and warps.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8_kernels.cuh"
#include "fp8_ptx.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

// Two fp32 numbers side by side: one instruction for both.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ F2 bf16_pair(uint32_t u) { return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u)); }

// Eight elements: as they lie in memory (two uint4 for fp32), as four pairs, and back.
template <typename T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void unpack(F2 (&f)[4]) const {
        if constexpr (sizeof(T) == 4) {
            f[0] = pair(__uint_as_float(u[0].x), __uint_as_float(u[0].y));
            f[1] = pair(__uint_as_float(u[0].z), __uint_as_float(u[0].w));
            f[2] = pair(__uint_as_float(u[1].x), __uint_as_float(u[1].y));
            f[3] = pair(__uint_as_float(u[1].z), __uint_as_float(u[1].w));
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (std::is_same<T, __half>::value) {
                    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                    f[i] = pair(v.x, v.y);
                } else {
                    f[i] = bf16_pair(w[i]);
                }
            }
        }
    }
    static __device__ __forceinline__ void store(T *p, const F2 (&f)[4]) {
        if constexpr (sizeof(T) == 4) {
            const float2 a = both(f[0]), b = both(f[1]), c = both(f[2]), d = both(f[3]);
            reinterpret_cast<float4 *>(p)[0] = make_float4(a.x, a.y, b.x, b.y);
            reinterpret_cast<float4 *>(p)[1] = make_float4(c.x, c.y, d.x, d.y);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = both(f[i]);
                if constexpr (std::is_same<T, __half>::value) {
                    const __half2 h = __floats2half2_rn(v.x, v.y);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
                    w[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

}  // namespace

// CH: 8-element pieces per thread (1 or 2).  RES: with a residual.
template <typename T, int CH, bool RES>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(const Fp8NormParams p) {
    __shared__ float part[32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, step = blockDim.x;
    const long long row = blockIdx.x;
    const int pieces = p.d / 8;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx + 8 * tid;
    const T *r = RES ? static_cast<const T *>(p.residual) + row * p.ldr + 8 * tid : nullptr;
    Raw8<T> rx[CH], rr[RES ? CH : 1];
    uint4 w[CH];                    // the norm's weights, on their way while the row is summed
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (c * step + tid < pieces) {
            rx[c].load(x + 8 * c * step);
            if constexpr (RES) rr[c].load(r + 8 * c * step);
        }
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (c * step + tid < pieces) w[c] = *reinterpret_cast<const uint4 *>(p.norm_scale + 8 * (c * step + tid));
    F2 n[CH][4];
    F2 s2 = pair(0.0f, 0.0f);
#pragma unroll
    for (int c = 0; c < CH; ++c)
        if (c * step + tid < pieces) {
            rx[c].unpack(n[c]);
            if constexpr (RES) {
                F2 v[4];
                rr[c].unpack(v);
#pragma unroll
                for (int j = 0; j < 4; ++j) n[c][j] = add2(n[c][j], v[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s2 = fma2(n[c][j], n[c][j], s2);
            if constexpr (RES) {
                if (p.sum_out) Raw8<T>::store(static_cast<T *>(p.sum_out) + row * p.lds + 8 * (c * step + tid), n[c]);
            }
        }
    float ss = both(s2).x + both(s2).y;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    float tot = lane < (step >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const float rms = 1.0f / sqrtf(tot / (float)p.d + p.eps);
    const int blocks = fp8_blocks(p.d);
    const F2 rms2 = pair(rms, rms);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * step + tid;
        const bool in = i < pieces;
        float amax = 0.0f;
        if (in) {
            const uint32_t u[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                n[c][j] = mul2(mul2(n[c][j], rms2), bf16_pair(u[j]));
                const float2 v = both(n[c][j]);
                amax = fmax_nan(amax, fmax_nan(fabsf(v.x), fabsf(v.y)));
            }
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (in) {
            const float s = fmax_nan(amax / FP8_MAX, FP8_SCALE_MIN), inv = 1.0f / s;
            const F2 f = pair(inv, inv);
            float2 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = both(mul2(n[c][j], f));
            *reinterpret_cast<uint2 *>(p.q + row * p.d + 8 * i) =
                make_uint2(f32x4_to_e4m3x4(v[0].x, v[0].y, v[1].x, v[1].y), f32x4_to_e4m3x4(v[2].x, v[2].y, v[3].x, v[3].y));
            if ((lane & 15) == 0) p.q_scale[row * blocks + i / 16] = s;
        }
    }
}

template <typename T, int CH>
static cudaError_t launch_norm_ch(const Fp8NormParams &p, cudaStream_t s) {
    const int pieces = p.d / 8, threads = ((pieces + CH - 1) / CH + 31) / 32 * 32;
    return p.residual ? launch_pdl(add_rmsnorm_fp8_kernel<T, CH, true>, dim3(p.T), dim3(threads), 0, s, p)
                      : launch_pdl(add_rmsnorm_fp8_kernel<T, CH, false>, dim3(p.T), dim3(threads), 0, s, p);
}

template <typename T>
static cudaError_t launch_norm_t(const Fp8NormParams &p, int num_sms, cudaStream_t s) {
    const int pieces = p.d / 8;
    // Few rows: a piece per thread, the shortest way through a row.  Many: two, so that more rows are in flight on
    // an SM.  Measured (bf16, d = 2880, residual; one, two, three pieces): T = 600 4.6, 5.4, 5.4 us; T = 1024 6.3
    // all three; T = 8192 31.1, 28.0, 27.7 us; T = 2048, d = 6144 20.4, 16.4, 16.7 us.
    return pieces > 1024 || p.T >= 8 * num_sms ? launch_norm_ch<T, 2>(p, s) : launch_norm_ch<T, 1>(p, s);
}

template <typename T>
static cudaError_t load_t() {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, add_rmsnorm_fp8_kernel<T, 1, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, add_rmsnorm_fp8_kernel<T, 1, true>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, add_rmsnorm_fp8_kernel<T, 2, false>);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, add_rmsnorm_fp8_kernel<T, 2, true>);
    return e;
}

// Loads the kernels (once per device, before the first launch, which may be captured).
cudaError_t fp8_norm_setup() {
    cudaError_t e = load_t<__nv_bfloat16>();
    if (e == cudaSuccess) e = load_t<__half>();
    if (e == cudaSuccess) e = load_t<float>();
    return e;
}

cudaError_t launch_add_rmsnorm_fp8(const Fp8NormParams &p, int type, int num_sms, cudaStream_t s) {
    if (type == FP8_BF16) return launch_norm_t<__nv_bfloat16>(p, num_sms, s);
    if (type == FP8_FP16) return launch_norm_t<__half>(p, num_sms, s);
    return launch_norm_t<float>(p, num_sms, s);
}

}  // namespace moe
