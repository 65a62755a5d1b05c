// Products of E4M3 matrices with fp32 block scales, on tcgen05 (kind::f8f6f4).
//
//   D_kb[m, n] = sum_{k in block kb} a[m, k] b[n, k]
//   c[m, n]    = sum_kb sa[m, kb] sb[n / 128, kb] D_kb[m, n]  (+ bias[n]) (+ residual[m, n])
//
// One 128-K block is one shared-memory stage and four MMAs (K = 32) into an accumulator of its
// own in TMEM.  The scales are any fp32 numbers, so the tensor core cannot apply them: the
// epilogue warps read each block's accumulator, multiply by sa * sb (one number per thread and
// 64 or 128 columns: a thread holds one row) and add it to fp32 sums in registers, while the
// MMAs fill the next accumulator.  That is one FMA per 128 products; 256 threads take about
// half the time that the MMAs of a 128 x 256 tile do.
//
// Gated (both projections of a gated feed-forward block): a CTA's accumulator columns are half
// gate rows and half linear rows of W13, so a thread holds a row's gate and linear value of the
// same columns, computes h = min(g, L) sigmoid(alpha min(g, L)) (clamp(u, -L, L) + shift), and
// writes h in E4M3 with the scale of its 128-column block; only the block's maximum crosses
// warps (or, for narrow tiles, the CTAs of a cluster, through distributed shared memory).
//
// Warp roles: 4 or 8 epilogue warps (warp w reads TMEM lane quarter w % 4), then the TMA
// producer, then the MMA warp, both running as whole warps with an elected lane issuing.
// Persistent: CTAs (clusters) walk the output tiles, rows fastest, so the B tile of neighbouring
// CTAs is the same and A stays in L2.
//
// Every wait is bounded (WaitCtl); when one runs out the CTA stops issuing, waits (bounded) for
// what it has in flight, frees TMEM and returns with the error latched.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8_kernels.cuh"
#include "fp8_ptx.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr unsigned int FP8_ERR_WAIT = 1u;

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

template <typename T>
__device__ __forceinline__ float to_f32(T v) { return static_cast<float>(v); }

// Rows of 16-byte pieces between global memory and a warp's staging tile (32 rows of 128 bytes,
// piece p of row r at slot p ^ (r & 7)): PCS lanes per row, so a row's bytes move together.
template <typename T, int PCS, bool STORE>
__device__ __forceinline__ void move_tile(uint8_t *stage, T *g, long long ld, int rows, int cols, bool vec, int lane) {
    constexpr int VEC = 16 / sizeof(T);
    const int pc = lane % PCS;
#pragma unroll
    for (int it = 0; it < PCS; ++it) {
        const int r = it * (32 / PCS) + lane / PCS;
        uint4 *slot = reinterpret_cast<uint4 *>(stage + r * 128 + ((pc ^ (r & 7)) << 4));
        if (r >= rows || pc * VEC >= cols) continue;
        T *src = g + (long long)r * ld + pc * VEC;
        if (vec && (pc + 1) * VEC <= cols) {
            if constexpr (STORE) *reinterpret_cast<uint4 *>(src) = *slot;
            else *slot = *reinterpret_cast<const uint4 *>(src);
        } else {
            uint4 u = make_uint4(0, 0, 0, 0);
            T *e = reinterpret_cast<T *>(&u);
            if constexpr (STORE) u = *slot;
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (pc * VEC + j < cols) {
                    if constexpr (STORE) src[j] = e[j];
                    else e[j] = src[j];
                }
            if constexpr (!STORE) *slot = u;
        }
    }
}

// c = sums (+ bias) (+ residual), rounded once: CW columns of 32 rows, a thread's row to the
// staging tile in 16-byte pieces, then out of it row by row.
template <typename T, int CW>
__device__ __forceinline__ void store_columns(const Fp8GemmParams &p, const float (&acc)[CW], uint8_t *stage, int m0,
                                              int n0, int lane) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int PCS = CW / VEC < 8 ? CW / VEC : 8;
    const int rows = min(32, p.M - m0);
#pragma unroll
    for (int ch = 0; ch < CW / (PCS * VEC); ++ch) {
        const int c0 = n0 + ch * PCS * VEC;
        const int cols = min(PCS * VEC, p.N - c0);
        if (cols <= 0) break;
        if (p.residual) {
            move_tile<T, PCS, false>(stage, const_cast<T *>(static_cast<const T *>(p.residual)) + (long long)m0 * p.ldr + c0,
                                     p.ldr, rows, cols, p.vec_r, lane);
            __syncwarp();
        }
#pragma unroll
        for (int pc = 0; pc < PCS; ++pc) {
            uint4 *slot = reinterpret_cast<uint4 *>(stage + lane * 128 + ((pc ^ (lane & 7)) << 4));
            float b[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int n = pc * VEC + j;
                b[j] = p.bias && n < cols ? bf16_bits_to_f32(p.bias[c0 + n]) : 0.0f;
            }
            uint4 u = *slot;
            T *e = reinterpret_cast<T *>(&u);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float v = acc[ch * PCS * VEC + pc * VEC + j];
                if (p.bias) v += b[j];
                if (p.residual) v += to_f32(e[j]);
                e[j] = static_cast<T>(v);
            }
            *slot = u;
        }
        __syncwarp();
        move_tile<T, PCS, true>(stage, static_cast<T *>(p.c) + (long long)m0 * p.ldc + c0, p.ldc, rows, cols, p.vec_c, lane);
        __syncwarp();
    }
}

// Wait (bounded, without the abort flag) for a phase: for copies and MMAs in flight after an abort.
__device__ __forceinline__ void wait_drain(uint64_t *bar, uint32_t parity, unsigned long long limit_ns) {
    const uint64_t start = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - start > limit_ns) return;
    }
}

}  // namespace

template <int BN, int CTAS, bool GATED, int CL>
__global__ void __launch_bounds__(fp8_threads(BN), fp8_ctas_per_sm(BN)) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
    constexpr int WGS = fp8_wgs(BN);            // epilogue warpgroups
    constexpr int CW = BN / WGS;                // accumulator columns per epilogue thread
    constexpr int HW = CW / 2;                  // gated: h columns per thread
    constexpr int BUFS = fp8_bufs(BN);
    constexpr int CSIZE = CTAS == 2 ? 2 : CL;   // CTAs per cluster
    constexpr int EX = WGS > CL ? WGS : CL;     // gated: warps or CTAs that share a row's block
    static_assert(!GATED || HW * EX == FP8_BLOCK, "a gated row's block is shared by EX threads");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int NS = p.n_stages;
    const Fp8Smem plan = fp8_smem(BN, CTAS, CL, GATED, p.a_rows, NS);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + plan.bar_off);
    uint64_t *empty = full + NS;
    uint64_t *d_full = empty + NS;              // a K block's accumulator is complete
    uint64_t *d_empty = d_full + BUFS;          // ... and has been read
    uint64_t *drain_bar = d_empty + BUFS;
    uint64_t *ex_bar = drain_bar + 1;           // [4 quarters][2 parities]
    float *ex = reinterpret_cast<float *>(smem + plan.ex_off);       // [2 parities][EX][128 rows]
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + plan.misc_off);
    volatile int *abort_s = reinterpret_cast<volatile int *>(smem + plan.misc_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CSIZE > 1 ? cluster_ctarank() : 0;
    constexpr int TMA_WARP = WGS * 4, MMA_WARP = TMA_WARP + 1;
    constexpr uint32_t COLS = BUFS * BN;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);             // the (even CTA's) producer
            mbar_init(&empty[i], 1);            // MMA commit
        }
        for (int i = 0; i < BUFS; ++i) {
            mbar_init(&d_full[i], 1);           // MMA commit
            mbar_init(&d_empty[i], WGS * 4 * CTAS);   // every epilogue warp (of both CTAs)
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < 8; ++i) mbar_init(&ex_bar[i], EX);
        *abort_s = 0;
        fence_barrier_init();
    }
    if (warp == MMA_WARP) tmem_alloc_g<CTAS>(tmem_base_s, COLS);
    tc_fence_before();
    __syncthreads();
    if constexpr (CSIZE > 1) cluster_sync();    // the peers' barriers are initialised
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_base_s;
    const WaitCtl wc{abort_s, p.err, FP8_ERR_WAIT, p.wait_limit_ns};
    const int first = blockIdx.x / CSIZE, step = gridDim.x / CSIZE;

    if (warp == TMA_WARP) {
        if (lane == 0) {
            tma_prefetch_desc(&p.map_a);
            tma_prefetch_desc(&p.map_b);
        }
        int slot = 0;
        uint32_t ph = 0;
        long long issued = 0;
        bool ok = true;
        const uint32_t bytes = (uint32_t)(CTAS * (plan.a_stage + plan.b_stage));
        for (int t = first; t < p.tiles && ok; t += step) {
            const int m0 = (t % p.m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0);
            const int nt = t / p.m_tiles;
            const int nb = GATED ? nt * FP8_BLOCK + (int)rank * HW : nt * BN + (CTAS == 2 ? (int)rank * (BN / 2) : 0);
            for (int kb = 0; kb < p.KB; ++kb) {
                if (!__all_sync(0xffffffffu, mbar_wait(&empty[slot], ph ^ 1, wc))) { ok = false; break; }
                if (CTAS == 1 || rank == 0) mbar_arrive_expect_tx_w(&full[slot], bytes);
                uint8_t *as = smem + slot * plan.a_stage, *bs = smem + plan.b_off + slot * plan.b_stage;
                const int k0 = kb * FP8_KS;
                if constexpr (CTAS == 2) {
                    tma_load_3d_pair_w(as, &p.map_a, &full[slot], k0, m0, 0);
                    tma_load_3d_pair_w(bs, &p.map_b, &full[slot], k0, nb, 0);
                    if constexpr (GATED) tma_load_3d_pair_w(bs + HW * FP8_KS, &p.map_b, &full[slot], k0, nb, 1);
                } else {
                    tma_load_3d_w(as, &p.map_a, &full[slot], k0, m0, 0);
                    tma_load_3d_w(bs, &p.map_b, &full[slot], k0, nb, 0);
                    if constexpr (GATED) tma_load_3d_w(bs + HW * FP8_KS, &p.map_b, &full[slot], k0, nb, 1);
                }
                ++issued;
                if (++slot == NS) { slot = 0; ph ^= 1; }
            }
        }
        if (!ok && rank == 0) {
            // fill i went to slot i % NS with phase parity (i / NS) & 1
            for (long long i = issued - 1; i >= 0 && i >= issued - NS; --i)
                wait_drain(&full[i % NS], (uint32_t)((i / NS) & 1), p.wait_limit_ns);
        }
    } else if (warp == MMA_WARP) {
        if (CTAS == 1 || rank == 0) {
            // kind::f8f6f4 descriptor: fp32 accumulators (1 << 4), E4M3 x E4M3 (0), both K-major, N >> 3, M >> 4
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(FP8_BM * CTAS >> 4) << 24);
            int slot = 0, buf = 0;
            uint32_t ph = 0, dph = 0;
            bool ok = true, any = false;
            for (int t = first; t < p.tiles && ok; t += step) {
                for (int kb = 0; kb < p.KB; ++kb) {
                    const bool free_d = CTAS == 2 ? mbar_wait_cluster(&d_empty[buf], dph ^ 1, wc)
                                                  : mbar_wait(&d_empty[buf], dph ^ 1, wc);
                    if (!__all_sync(0xffffffffu, free_d)) { ok = false; break; }
                    if (!__all_sync(0xffffffffu, mbar_wait(&full[slot], ph, wc))) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_sw128(smem_addr(smem + slot * plan.a_stage));
                    const uint64_t bd = smem_desc_sw128(smem_addr(smem + plan.b_off + slot * plan.b_stage));
#pragma unroll
                    for (int k = 0; k < 4; ++k)      // past K the operands are zeros
                        mma_f8_w<CTAS>(tmem + (uint32_t)(buf * BN), ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                    any = true;
                    mma_commit_g<CTAS>(&empty[slot]);
                    mma_commit_g<CTAS>(&d_full[buf]);
                    if (++slot == NS) { slot = 0; ph ^= 1; }
                    if (++buf == BUFS) { buf = 0; dph ^= 1; }
                }
            }
            if (!ok && any) {
                mma_commit_g<CTAS>(drain_bar);
                wait_drain(drain_bar, 0, p.wait_limit_ns);
            }
        }
    } else {
        const int wg = warp >> 2, q = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(wg * CW);
        const uint32_t d_empty0 = CTAS == 2 ? map_to_rank(smem_addr(d_empty), 0) : 0;
        int buf = 0, par = 0;
        uint32_t dph = 0, exph = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += step) {
            const int nt = t / p.m_tiles;
            const int m0 = (t % p.m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0) + 32 * q;
            const int n0 = GATED ? nt * FP8_BLOCK + (WGS > 1 ? wg : (int)rank) * HW : nt * BN + wg * CW;
            const bool active = m0 < p.M && n0 < p.N;      // the warp has something to write
            const float *sa = p.a_scale + (long long)min(m0 + lane, p.M - 1) * p.KB;
            const float *sb0 = p.b_scale + (long long)min(n0 / FP8_BLOCK, p.NB - 1) * p.KB;
            const float *sb1 = GATED ? sb0 + (long long)p.NB * p.KB : sb0;
            float acc[CW];
#pragma unroll
            for (int i = 0; i < CW; ++i) acc[i] = 0.0f;
            float a_next = sa[0], b0_next = sb0[0], b1_next = sb1[0];
            for (int kb = 0; kb < p.KB; ++kb) {
                const float s0 = a_next * b0_next, s1 = a_next * b1_next;
                if (kb + 1 < p.KB) { a_next = sa[kb + 1]; b0_next = sb0[kb + 1]; b1_next = sb1[kb + 1]; }
                if (!__all_sync(0xffffffffu, mbar_wait(&d_full[buf], dph, wc))) { ok = false; break; }
                tc_fence_after();
                if (active) {
#pragma unroll
                    for (int c = 0; c < CW; c += 32) {
                        uint32_t r[32];
                        tmem_ld32(lane_base + (uint32_t)(buf * BN + c), r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            acc[c + i] = fmaf(__uint_as_float(r[i]), GATED && c + i >= HW ? s1 : s0, acc[c + i]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CTAS == 2) mbar_arrive_cluster(d_empty0 + 8u * (uint32_t)buf);
                    else mbar_arrive(&d_empty[buf]);
                }
                if (++buf == BUFS) { buf = 0; dph ^= 1; }
            }
            if (!ok) break;
            if constexpr (GATED) {
                const int row = 32 * q + lane;
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < HW; ++i) {
                    float g = acc[i], u = acc[HW + i];
                    const bool in = n0 + i < p.N;
                    if (p.bias && in) {
                        g += bf16_bits_to_f32(p.bias[n0 + i]);
                        u += bf16_bits_to_f32(p.bias[p.N + n0 + i]);
                    }
                    // comparisons that keep a NaN
                    g = g > p.limit ? p.limit : g;
                    u = u > p.limit ? p.limit : u < -p.limit ? -p.limit : u;
                    const float h = in ? __fdividef(g, 1.0f + __expf(-p.alpha * g)) * (u + p.shift) : 0.0f;
                    acc[i] = h;
                    amax = fmax_nan(amax, fabsf(h));
                }
                // the row's maximum over its 128-column block
                float *slot = ex + (par * EX) * FP8_BM + row;
                uint64_t *bar = &ex_bar[2 * q + par];
                if constexpr (CL > 1) {
#pragma unroll
                    for (int c = 0; c < CL; ++c)
                        st_cluster_f32(map_to_rank(smem_addr(slot + rank * FP8_BM), (uint32_t)c), amax);
                    __syncwarp();
                    if (lane < CL) mbar_arrive_cluster(map_to_rank(smem_addr(bar), (uint32_t)lane));
                    if (!__all_sync(0xffffffffu, mbar_wait_cluster(bar, exph, wc))) { ok = false; break; }
                } else {
                    slot[wg * FP8_BM] = amax;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                    if (!__all_sync(0xffffffffu, mbar_wait(bar, exph, wc))) { ok = false; break; }
                }
#pragma unroll
                for (int e = 0; e < EX; ++e) amax = fmax_nan(amax, slot[e * FP8_BM]);
                par ^= 1;
                if (par == 0) exph ^= 1;
                if (active && m0 + lane < p.M) {
                    const float s = fmax_nan(amax / FP8_MAX, FP8_SCALE_MIN);
                    const float inv = 1.0f / s;
                    uint8_t *h = p.h + (long long)(m0 + lane) * p.N + n0;
#pragma unroll
                    for (int i = 0; i < HW; i += 16)
                        if (n0 + i < p.N) {
                            uint4 u;
                            u.x = f32x4_to_e4m3x4(acc[i] * inv, acc[i + 1] * inv, acc[i + 2] * inv, acc[i + 3] * inv);
                            u.y = f32x4_to_e4m3x4(acc[i + 4] * inv, acc[i + 5] * inv, acc[i + 6] * inv, acc[i + 7] * inv);
                            u.z = f32x4_to_e4m3x4(acc[i + 8] * inv, acc[i + 9] * inv, acc[i + 10] * inv, acc[i + 11] * inv);
                            u.w = f32x4_to_e4m3x4(acc[i + 12] * inv, acc[i + 13] * inv, acc[i + 14] * inv, acc[i + 15] * inv);
                            *reinterpret_cast<uint4 *>(h + i) = u;
                        }
                    if (n0 % FP8_BLOCK == 0) p.h_scale[(long long)(m0 + lane) * p.NB + n0 / FP8_BLOCK] = s;
                }
            } else if (active) {
                uint8_t *stage = smem + plan.stage_off + warp * 4096;
                if (p.type == FP8_BF16) store_columns<__nv_bfloat16, CW>(p, acc, stage, m0, n0, lane);
                else if (p.type == FP8_FP16) store_columns<__half, CW>(p, acc, stage, m0, n0, lane);
                else store_columns<float, CW>(p, acc, stage, m0, n0, lane);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if constexpr (CSIZE > 1) cluster_sync();    // no CTA leaves while a peer may still reach its shared memory
    tc_fence_after();
    if (warp == MMA_WARP) tmem_dealloc_g<CTAS>(tmem, COLS);
}

template <int BN, int CTAS, bool GATED, int CL>
static cudaError_t launch_t(const Fp8GemmParams &p, const Fp8Plan &pl, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(fp8_threads(BN));
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS == 2 ? 2 : CL;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CTAS == 2 || CL > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<BN, CTAS, GATED, CL>, p);
}

template <int BN, int CTAS, bool GATED, int CL>
static cudaError_t setup_t() {
    return cudaFuncSetAttribute(fp8_gemm_kernel<BN, CTAS, GATED, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                fp8_smem_bytes(BN));
}

// Once per device, before the first launch.
cudaError_t fp8_gemm_setup() {
    cudaError_t e = setup_t<32, 1, false, 1>();
    if (e == cudaSuccess) e = setup_t<64, 1, false, 1>();
    if (e == cudaSuccess) e = setup_t<128, 1, false, 1>();
    if (e == cudaSuccess) e = setup_t<32, 1, true, 8>();
    if (e == cudaSuccess) e = setup_t<64, 1, true, 4>();
    return e;
}

cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const Fp8Plan &pl, int gated, cudaStream_t s) {
    if (gated) {
        if (pl.bn == 32) return launch_t<32, 1, true, 8>(p, pl, s);
        return launch_t<64, 1, true, 4>(p, pl, s);
    }
    if (pl.bn == 32) return launch_t<32, 1, false, 1>(p, pl, s);
    if (pl.bn == 64) return launch_t<64, 1, false, 1>(p, pl, s);
    return launch_t<128, 1, false, 1>(p, pl, s);
}

}  // namespace moe
