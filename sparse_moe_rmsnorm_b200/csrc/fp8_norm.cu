// RMS norm with the residual's addition, the normalised rows in E4M3 with a scale per 128 elements.
//
//   n = x + r,  y = n / sqrt(mean(n^2) + eps) * w          (fp32 throughout)
//   s_b = max(max_{i in b} |y_i| / 448, 2^-126),  q = e4m3(y / s_b)
//
// The norm is the routed block's (no bias, no mean subtraction: pnsm.cn overview, section 2.3;
// "gpt-oss-20B" hub page, section 3.2) and stands beside it: here the rows leave in the form the
// dense 8-bit products read.  Bound by HBM: x, r, the sum and q move once, about 6 operations
// per element.  One CTA holds a row in registers, 8 elements per thread, so the row is read once
// and the second pass (the scaling) needs no memory; a block's 128 elements sit in 16 neighbouring
// lanes, so its maximum is four shuffles.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_kernels.cuh"
#include "fp8_ptx.cuh"
#include "kernels.cuh"

namespace moe {

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(e[i]);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = static_cast<T>(v[i]);
        *reinterpret_cast<uint4 *>(p) = u;
    }
}

// CH: 8-element pieces per thread.
template <typename T, int CH>
__global__ void __launch_bounds__(1024) add_rmsnorm_fp8_kernel(const Fp8NormParams p) {
    __shared__ float part[32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long row = blockIdx.x;
    const int pieces = p.d / 8;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *r = static_cast<const T *>(p.residual) + (p.residual ? row * p.ldr : 0);
    float n[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * blockDim.x + tid;
        if (i < pieces) {
            load8(x + 8 * i, n[c]);
            if (p.residual) {
                float v[8];
                load8(r + 8 * i, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) n[c][j] += v[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) ss += n[c][j] * n[c][j];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) part[warp] = ss;
    __syncthreads();
    float tot = lane < (blockDim.x >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const float rms = 1.0f / sqrtf(tot / (float)p.d + p.eps);
    const int blocks = fp8_blocks(p.d);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int i = c * blockDim.x + tid;
        const bool in = i < pieces;
        float y[8], amax = 0.0f;
        if (in) {
            if (p.sum_out) store8(static_cast<T *>(p.sum_out) + row * p.lds + 8 * i, n[c]);
            float w[8];
            load8(reinterpret_cast<const __nv_bfloat16 *>(p.norm_scale) + 8 * i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                y[j] = n[c][j] * rms * w[j];
                amax = fmax_nan(amax, fabsf(y[j]));
            }
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (in) {
            const float s = fmax_nan(amax / FP8_MAX, FP8_SCALE_MIN);
            const float inv = 1.0f / s;
            uint2 q;
            q.x = f32x4_to_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            q.y = f32x4_to_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
            *reinterpret_cast<uint2 *>(p.q + row * p.d + 8 * i) = q;
            if ((lane & 15) == 0) p.q_scale[row * blocks + i / 16] = s;
        }
    }
}

template <typename T>
static cudaError_t launch_norm_t(const Fp8NormParams &p, cudaStream_t s) {
    const int pieces = p.d / 8;
    const int ch = (pieces + 1023) / 1024;
    const int threads = ((pieces + ch - 1) / ch + 31) / 32 * 32;
    return ch == 1 ? launch_pdl(add_rmsnorm_fp8_kernel<T, 1>, dim3(p.T), dim3(threads), 0, s, p)
                   : launch_pdl(add_rmsnorm_fp8_kernel<T, 2>, dim3(p.T), dim3(threads), 0, s, p);
}

cudaError_t launch_add_rmsnorm_fp8(const Fp8NormParams &p, int type, cudaStream_t s) {
    if (type == FP8_BF16) return launch_norm_t<__nv_bfloat16>(p, s);
    if (type == FP8_FP16) return launch_norm_t<__half>(p, s);
    return launch_norm_t<float>(p, s);
}

}  // namespace moe
