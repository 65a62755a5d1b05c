// C ABI of the dense 8-bit operators: context, argument validation, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <new>

#include "moe_b200.h"
#include "fp8_kernels.cuh"
#include "host_plan.cuh"

namespace moe {
cudaError_t launch_add_rmsnorm_fp8(const Fp8NormParams &p, int type, int num_sms, cudaStream_t s);
cudaError_t fp8_gemm_setup(int *clusters);
cudaError_t fp8_few_setup();
cudaError_t fp8_norm_setup();
cudaError_t launch_fp8_selftest_wait(unsigned int *err, unsigned long long limit_ns, cudaStream_t s);
cudaError_t launch_fp8_few(const Fp8FewParams &p, int gated, cudaStream_t s);
cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const Fp8Plan &pl, int gated, cudaStream_t s);
}  // namespace moe

using namespace moe;

// Nothing but the count of waits that ran out lives on the device, so calls on one context from several
// streams, host threads or captured graphs share no workspace.  The count only grows: a stream that asks for the
// status hears whether it grew since that stream asked last, and takes nothing from another's answer.
struct moe_fp8_ctx {
    int device;
    int num_sms;
    unsigned int *err;
    unsigned long long wait_limit_ns;
    int clusters[FP8_SPLIT_MAX + 1];    // clusters of n CTAs that the device holds at once
    std::mutex lock;
    std::map<unsigned long long, unsigned int> heard;       // the count at each stream's (by its id) last answer
};

namespace {

static_assert((int)MOE_BF16 == (int)FP8_BF16 && (int)MOE_FP16 == (int)FP8_FP16 && (int)MOE_FP32 == (int)FP8_FP32,
              "types of the C ABI");

// The context's device is current while a call runs, whichever the caller had.
struct DeviceGuard {
    int old = -1;
    bool ok;
    explicit DeviceGuard(int device) {
        ok = cudaGetDevice(&old) == cudaSuccess && (old == device || cudaSetDevice(device) == cudaSuccess);
        if (old == device) old = -1;
    }
    ~DeviceGuard() {
        if (old >= 0) cudaSetDevice(old);
    }
};

bool aligned(const void *p, uintptr_t to) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool aligned_or_null(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
int type_bytes(int type) { return type == MOE_FP32 ? 4 : type == MOE_BF16 || type == MOE_FP16 ? 2 : 0; }
int status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// u8 {K, rows, planes}, rows ld bytes apart, planes rows * ld bytes apart: a box of 128 bytes x
// box_rows, 128-byte swizzle, zeros outside.
bool encode_u8(CUtensorMap *m, const void *base, int K, long long rows, long long ld, int planes, int box_rows) {
    EncodeTiledFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)rows, (cuuint64_t)planes};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)(planes > 1 ? rows * ld : ld)};
    const cuuint32_t box[3] = {FP8_KS, (cuuint32_t)box_rows, 1};
    const cuuint32_t es[3] = {1, 1, 1};
    return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_product(moe_fp8_ctx *c, int M, int N, int K, const uint8_t *a, long long lda, const float *a_scale,
                  const uint8_t *b, const float *b_scale, const uint16_t *bias) {
    if (!c || M < 0 || N < 1 || K < 16 || K % 16 || M > FP8_SIZE_MAX || N > FP8_SIZE_MAX || K > FP8_SIZE_MAX)
        return MOE_ERR_ARG;
    if (M == 0) return MOE_OK;
    if (!aligned(a, 16) || !aligned(a_scale, 4) || !aligned(b, 16) || !aligned(b_scale, 4) || !aligned_or_null(bias, 2))
        return MOE_ERR_ARG;
    if (lda < K || lda % 16 || lda >= (1LL << 40)) return MOE_ERR_ARG;
    return MOE_OK;
}

// The sizes, operands and tensor maps that both products share.
int product_params(moe_fp8_ctx *c, Fp8GemmParams &p, Fp8Plan &pl, int gated, int M, int N, int K, const uint8_t *a,
                   long long lda, const float *a_scale, const uint8_t *b, const float *b_scale, const uint16_t *bias) {
    memset(&p, 0, sizeof p);
    if (!fp8_plan(M, N, K, gated, c->num_sms, c->clusters, &pl)) return MOE_ERR_ARG;
    const int b_rows = gated ? pl.bn / 4 : pl.bn / pl.ctas / fp8_split(pl.bn);
    if (!encode_u8(&p.map_a, a, K, M, lda, 1, pl.a_rows)) return MOE_ERR_ARG;
    if (!encode_u8(&p.map_b, b, K, N, K, gated ? 2 : 1, b_rows)) return MOE_ERR_ARG;
    p.a_scale = a_scale;
    p.b_scale = b_scale;
    p.M = M;
    p.N = N;
    p.K = K;
    p.KB = fp8_blocks(K);
    p.NB = fp8_blocks(N);
    p.m_tiles = pl.m_tiles;
    p.tiles = pl.tiles;
    p.a_rows = pl.a_rows;
    p.n_stages = pl.n_stages;
    p.split = pl.split;
    p.bias = bias;
    p.err = c->err;
    p.wait_limit_ns = c->wait_limit_ns;
    return MOE_OK;
}

Fp8FewParams few_params(int M, int N, int K, const uint8_t *a, long long lda, const float *a_scale, const uint8_t *b,
                        const float *b_scale, const uint16_t *bias) {
    Fp8FewParams p;
    memset(&p, 0, sizeof p);
    p.a = a;
    p.b = b;
    p.a_scale = a_scale;
    p.b_scale = b_scale;
    p.bias = bias;
    p.lda = lda;
    p.M = M;
    p.N = N;
    p.K = K;
    p.KB = fp8_blocks(K);
    p.NB = fp8_blocks(N);
    return p;
}

}  // namespace

extern "C" {

int moe_fp8_init(moe_fp8_ctx_t **out) {
    if (!out) return MOE_ERR_ARG;
    *out = nullptr;
    int dev = 0, major = 0, minor = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (major != 10 || minor != 0) return MOE_ERR_UNSUPPORTED;
    if (!encode_fn()) return MOE_ERR_CUDA;
    moe_fp8_ctx *c = new (std::nothrow) moe_fp8_ctx;
    if (!c) return MOE_ERR_NOMEM;
    c->device = dev;
    c->num_sms = sms;
    c->wait_limit_ns = 2000000000ull;
    memset(c->clusters, 0, sizeof c->clusters);
    // (every kernel is loaded here, so that a first call may be captured)
    cudaError_t e = fp8_gemm_setup(c->clusters);
    if (e == cudaSuccess) e = fp8_few_setup();
    if (e == cudaSuccess) e = fp8_norm_setup();
    if (e != cudaSuccess) {
        delete c;
        return e == cudaErrorNotSupported ? MOE_ERR_UNSUPPORTED : MOE_ERR_CUDA;
    }
    if (cudaMalloc(&c->err, 64) != cudaSuccess) {
        cudaGetLastError();
        delete c;
        return MOE_ERR_NOMEM;
    }
    // (waited for: streams that do not block on the default one are not behind it)
    if (cudaMemset(c->err, 0, 64) != cudaSuccess || cudaStreamSynchronize(0) != cudaSuccess) {
        cudaFree(c->err);
        delete c;
        return MOE_ERR_CUDA;
    }
    *out = c;
    return MOE_OK;
}

int moe_fp8_destroy(moe_fp8_ctx_t *c) {
    if (!c) return MOE_OK;
    {
        DeviceGuard g(c->device);
        cudaDeviceSynchronize();
        cudaFree(c->err);
    }
    delete c;
    return MOE_OK;
}

int moe_fp8_sync_status(moe_fp8_ctx_t *c, void *stream) {
    if (!c) return MOE_ERR_ARG;
    DeviceGuard g(c->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int count = 0;
    unsigned long long id = 0;                  // (never used again, as a handle may be)
    if (!g.ok || cudaStreamGetId(s, &id) != cudaSuccess ||
        cudaMemcpyAsync(&count, c->err, sizeof count, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (!count) return MOE_OK;
    try {
        const std::lock_guard<std::mutex> hold(c->lock);
        unsigned int &heard = c->heard[id];
        if ((int)(count - heard) <= 0) return MOE_OK;
        heard = count;
    } catch (...) {
        return MOE_ERR_NOMEM;
    }
    return MOE_ERR_TIMEOUT;
}

int moe_fp8_set_wait_limit_ns(moe_fp8_ctx_t *c, unsigned long long ns) {
    if (!c || ns < FP8_WAIT_LIMIT_MIN_NS) return MOE_ERR_ARG;
    c->wait_limit_ns = ns;
    return MOE_OK;
}

int moe_fp8_selftest_wait_timeout(moe_fp8_ctx_t *c, void *stream) {
    if (!c) return MOE_ERR_ARG;
    DeviceGuard g(c->device);
    if (!g.ok) return MOE_ERR_CUDA;
    return status(launch_fp8_selftest_wait(c->err, c->wait_limit_ns, static_cast<cudaStream_t>(stream)));
}

int moe_add_rmsnorm_fp8(moe_fp8_ctx_t *c, int T, int d, int type, const void *x, int64_t ldx, const void *residual,
                        int64_t ldr, const uint16_t *norm_scale, float eps, void *sum_out, int64_t lds, uint8_t *q,
                        float *q_scale, void *stream) {
    const int eb = type_bytes(type);
    if (!c || T < 0 || d < 16 || d > 16384 || d % 16 || !eb || !(eps >= 0.0f)) return MOE_ERR_ARG;
    if (T == 0) return MOE_OK;
    if (!aligned(x, 16) || !aligned_or_null(residual, 16) || !aligned(norm_scale, 16) || !aligned_or_null(sum_out, 16) ||
        !aligned(q, 16) || !aligned(q_scale, 4))
        return MOE_ERR_ARG;
    const int row = 16 / eb;
    if (sum_out && !residual) return MOE_ERR_ARG;      // the sum is x
    if (ldx < d || ldx % row || (residual && (ldr < d || ldr % row)) || (sum_out && (lds < d || lds % row)))
        return MOE_ERR_ARG;
    // a row's sum replaces x or the residual in place, or lies elsewhere
    if (sum_out && ((sum_out == x && lds != ldx) || (sum_out == residual && lds != ldr))) return MOE_ERR_ARG;
    DeviceGuard g(c->device);
    if (!g.ok) return MOE_ERR_CUDA;
    Fp8NormParams p;
    p.x = x;
    p.residual = residual;
    p.norm_scale = norm_scale;
    p.sum_out = sum_out;
    p.q = q;
    p.q_scale = q_scale;
    p.ldx = ldx;
    p.ldr = ldr;
    p.lds = lds;
    p.T = T;
    p.d = d;
    p.eps = eps;
    return status(launch_add_rmsnorm_fp8(p, type, c->num_sms, static_cast<cudaStream_t>(stream)));
}

int moe_fp8_matmul(moe_fp8_ctx_t *c, int M, int N, int K, const uint8_t *a, int64_t lda, const float *a_scale,
                   const uint8_t *b, const float *b_scale, const uint16_t *bias, const void *residual, int64_t ldr,
                   void *out, int64_t ldc, int type, void *stream) {
    const int eb = type_bytes(type);
    int rc = check_product(c, M, N, K, a, lda, a_scale, b, b_scale, bias);
    if (rc || !eb) return MOE_ERR_ARG;
    if (M == 0) return MOE_OK;
    if (!aligned(out, eb) || !aligned_or_null(residual, eb) || ldc < N || (residual && ldr < N)) return MOE_ERR_ARG;
    if (residual == out && ldr != ldc) return MOE_ERR_ARG;
    DeviceGuard g(c->device);
    if (!g.ok) return MOE_ERR_CUDA;
    if (fp8_few(M, N, 0, c->num_sms)) {
        Fp8FewParams p = few_params(M, N, K, a, lda, a_scale, b, b_scale, bias);
        p.residual = residual;
        p.ldr = ldr;
        p.c = out;
        p.ldc = ldc;
        p.type = type;
        return status(launch_fp8_few(p, 0, static_cast<cudaStream_t>(stream)));
    }
    Fp8GemmParams p;
    Fp8Plan pl;
    if ((rc = product_params(c, p, pl, 0, M, N, K, a, lda, a_scale, b, b_scale, bias))) return rc;
    p.residual = residual;
    p.ldr = ldr;
    p.c = out;
    p.ldc = ldc;
    p.type = type;
    p.vec = aligned(out, 4 * eb) && ldc % 4 == 0 && (!residual || (aligned(residual, 4 * eb) && ldr % 4 == 0));
    return status(launch_fp8_gemm(p, pl, 0, static_cast<cudaStream_t>(stream)));
}

int moe_fp8_gated_matmul(moe_fp8_ctx_t *c, int M, int F, int K, const uint8_t *a, int64_t lda, const float *a_scale,
                         const uint8_t *w13, const float *w13_scale, const uint16_t *b13, float alpha, float limit,
                         float shift, uint8_t *h, float *h_scale, void *stream) {
    int rc = check_product(c, M, F, K, a, lda, a_scale, w13, w13_scale, b13);
    const float minus_alpha_log2e = -1.44269504f * alpha;
    if (rc || F % 16 || !(limit > 0.0f) || !std::isfinite(minus_alpha_log2e) || !std::isfinite(shift)) return MOE_ERR_ARG;
    if (M == 0) return MOE_OK;
    if (!aligned(h, 16) || !aligned(h_scale, 4)) return MOE_ERR_ARG;
    DeviceGuard g(c->device);
    if (!g.ok) return MOE_ERR_CUDA;
    if (fp8_few(M, F, 1, c->num_sms)) {
        Fp8FewParams p = few_params(M, F, K, a, lda, a_scale, w13, w13_scale, b13);
        p.minus_alpha_log2e = minus_alpha_log2e;
        p.limit = limit;
        p.shift = shift;
        p.h = h;
        p.h_scale = h_scale;
        return status(launch_fp8_few(p, 1, static_cast<cudaStream_t>(stream)));
    }
    Fp8GemmParams p;
    Fp8Plan pl;
    if ((rc = product_params(c, p, pl, 1, M, F, K, a, lda, a_scale, w13, w13_scale, b13))) return rc;
    p.minus_alpha_log2e = minus_alpha_log2e;
    p.limit = limit;
    p.shift = shift;
    p.h = h;
    p.h_scale = h_scale;
    return status(launch_fp8_gemm(p, pl, 1, static_cast<cudaStream_t>(stream)));
}

int moe_fp8_debug_plan(int gated, int M, int N, int K, int num_sms, int *out) {
    if (!out || M < 1 || N < 1 || K < 16 || K % 16 || num_sms < 1 || (gated && N % 16) || N > FP8_SIZE_MAX)
        return MOE_ERR_ARG;
    Fp8Plan pl;
    int clusters[FP8_SPLIT_MAX + 1];
    for (int n = 1; n <= FP8_SPLIT_MAX; ++n) clusters[n] = num_sms / n;
    const int few = fp8_few(M, N, gated ? 1 : 0, num_sms) ? 1 : 0;
    if (!fp8_plan(M, N, K, gated ? 1 : 0, num_sms, clusters, &pl)) return MOE_ERR_ARG;
    const int v[] = {few, pl.bn, pl.ctas, pl.split, pl.a_rows, pl.n_stages, pl.m_tiles, pl.tiles, pl.grid,
                     fp8_smem(pl.bn, pl.ctas, gated ? 1 : 0, pl.split > 1 || (gated && pl.ctas == 1), pl.a_rows, pl.n_stages).total};
    memcpy(out, v, sizeof v);
    return MOE_OK;
}

}  // extern "C"
