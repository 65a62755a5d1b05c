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
// producer, then two MMA warps, one elected lane of each running its loop.
// Persistent: CTAs (clusters) walk the output tiles, rows fastest, so the B tile of neighbouring
// CTAs is the same and A stays in L2.
//
// Every wait is bounded (WaitCtl); when one runs out the CTA stops issuing, waits (bounded) for
// what it has in flight, frees TMEM and returns with the error latched.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8_kernels.cuh"
#include "fp8_ptx.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr unsigned int FP8_ERR_WAIT = 1u;

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

// A warp's staging tile: 32 rows of 64 bytes, 16-byte piece p of row r at slot p ^ (r / 2 & 3), so that
// the eight lanes of a 128-byte access meet in no bank, whether they hold one piece of eight rows or
// two rows' pieces.
__device__ __forceinline__ uint4 *piece(uint8_t *stage, int r, int p) {
    return reinterpret_cast<uint4 *>(stage + r * 64 + ((p ^ (r >> 1 & 3)) << 4));
}

// Between the staging tile and rows of global memory, PCS pieces to a row: PCS neighbouring lanes take
// a row, so its bytes move together.  At the edges, and where rows do not start on 16 bytes, element
// by element.
template <typename T, int PCS, bool STORE>
__device__ __forceinline__ void move_tile(uint8_t *stage, T *g, long long ld, int rows, int cols, bool vec, int lane) {
    constexpr int VEC = 16 / sizeof(T);
    const int pc = lane % PCS, r0 = lane / PCS;
    T *at = g + r0 * ld + pc * VEC;
    if (vec && rows == 32 && cols == PCS * VEC) {
#pragma unroll
        for (int it = 0; it < PCS; ++it) {
            uint4 *slot = piece(stage, it * (32 / PCS) + r0, pc);
            if constexpr (STORE) *reinterpret_cast<uint4 *>(at) = *slot;
            else *slot = *reinterpret_cast<const uint4 *>(at);
            at += (32 / PCS) * ld;
        }
        return;
    }
#pragma unroll 1
    for (int r = r0; r < rows; r += 32 / PCS, at += (32 / PCS) * ld) {
        uint4 *slot = piece(stage, r, pc);
        if (vec && (pc + 1) * VEC <= cols) {
            if constexpr (STORE) *reinterpret_cast<uint4 *>(at) = *slot;
            else *slot = *reinterpret_cast<const uint4 *>(at);
        } else {
            T *e = reinterpret_cast<T *>(slot);
#pragma unroll 1
            for (int j = 0; j < VEC && pc * VEC + j < cols; ++j) {
                if constexpr (STORE) at[j] = e[j];
                else e[j] = at[j];
            }
        }
    }
}

// The eight or four elements of a piece, rounded (with RES: added to what the piece holds).
template <typename T, bool RES>
__device__ __forceinline__ uint4 pack_piece(const float *v, const uint4 &old) {
    uint4 u;
    if constexpr (sizeof(T) == 4) {
        float4 f = make_float4(v[0], v[1], v[2], v[3]);
        if constexpr (RES) {
            f.x += __uint_as_float(old.x), f.y += __uint_as_float(old.y);
            f.z += __uint_as_float(old.z), f.w += __uint_as_float(old.w);
        }
        u = make_uint4(__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z), __float_as_uint(f.w));
    } else {
        const uint32_t o[4] = {old.x, old.y, old.z, old.w};
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a = v[2 * i], b = v[2 * i + 1];
            if constexpr (RES) {
                const T *e = reinterpret_cast<const T *>(&o[i]);
                a += static_cast<float>(e[0]), b += static_cast<float>(e[1]);
            }
            if constexpr (std::is_same<T, __half>::value) {
                const __half2 h = __floats2half2_rn(a, b);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return u;
}

// c = sums (+ residual), rounded once: CW columns of 32 rows, each thread's row to the staging tile in
// 16-byte pieces, then out of it row by row.
template <typename T, int CW, bool RES>
__device__ __forceinline__ void store_columns(const Fp8GemmParams &p, const float (&acc)[CW], uint8_t *stage, int m0,
                                              int n0, int lane) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int PCS = CW / VEC < 4 ? CW / VEC : 4;
    const int rows = min(32, p.M - m0);
    T *c = static_cast<T *>(p.c) + (long long)m0 * p.ldc + n0;
    T *res = const_cast<T *>(static_cast<const T *>(p.residual)) + (RES ? (long long)m0 * p.ldr + n0 : 0);
#pragma unroll
    for (int c0 = 0; c0 < CW; c0 += PCS * VEC) {
        const int cols = min(PCS * VEC, p.N - n0 - c0);
        if (cols > 0) {
            if constexpr (RES) {
                move_tile<T, PCS, false>(stage, res + c0, p.ldr, rows, cols, p.vec_r, lane);
                __syncwarp();
            }
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) {
                uint4 *slot = piece(stage, lane, pc);
                uint4 old = make_uint4(0, 0, 0, 0);
                if constexpr (RES) old = *slot;
                *slot = pack_piece<T, RES>(acc + c0 + pc * VEC, old);
            }
            __syncwarp();
            move_tile<T, PCS, true>(stage, c + c0, p.ldc, rows, cols, p.vec_c, lane);
            __syncwarp();
        }
    }
}

template <typename T, int CW>
__device__ __forceinline__ void store_columns(const Fp8GemmParams &p, const float (&acc)[CW], uint8_t *stage, int m0,
                                              int n0, int lane) {
    if (p.residual) store_columns<T, CW, true>(p, acc, stage, m0, n0, lane);
    else store_columns<T, CW, false>(p, acc, stage, m0, n0, lane);
}

// v[0 .. n) = bias[0 .. n) (zeros past `valid`, and without a bias).
template <int N>
__device__ __forceinline__ void load_bias(float *v, const uint16_t *bias, int valid) {
    if (bias && valid >= N && (reinterpret_cast<uintptr_t>(bias) & 15) == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(bias + i);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i + 2 * j] = __uint_as_float(w[j] << 16);
                v[i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = bias && i < valid ? bf16_bits_to_f32(bias[i]) : 0.0f;
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
    constexpr int LD = CW > 64 ? 32 : 16;       // columns of a TMEM load (registers: 2 LD beside the CW sums)
    constexpr int HW = CW / 2;                  // gated: h columns per thread
    constexpr int BUFS = fp8_bufs(BN);
    constexpr int SPLIT = fp8_split(BN);        // parts of an accumulator: one per warpgroup, or the whole
    constexpr int PN = BN / SPLIT;              // columns of an MMA
    constexpr int CSIZE = CTAS == 2 ? 2 : CL;   // CTAs per cluster
    constexpr int EX = WGS > CL ? WGS : CL;     // gated: warps or CTAs that share a row's block
    static_assert(BUFS % 2 == 0, "with an accumulator's uses, too, one MMA warp's");
    static_assert(!GATED || HW * EX == FP8_BLOCK, "a gated row's block is shared by EX threads");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int NS = p.n_stages;
    const Fp8Smem plan = fp8_smem(BN, CTAS, CL, GATED, p.a_rows, NS);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + plan.bar_off);
    uint64_t *empty = full + NS;
    uint64_t *d_full = empty + NS;              // [SPLIT][BUFS] a K block's accumulator (part) is complete
    uint64_t *d_empty = d_full + SPLIT * BUFS;  // ... and has been read
    uint64_t *drain_bar = d_empty + SPLIT * BUFS;   // [2 MMA warps]
    uint64_t *ex_bar = drain_bar + 2;           // [4 quarters][2 parities]
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
            mbar_init(&empty[i], SPLIT);        // MMA commits
        }
        for (int i = 0; i < SPLIT * BUFS; ++i) {
            mbar_init(&d_full[i], 1);           // MMA commit
            mbar_init(&d_empty[i], WGS / SPLIT * 4 * CTAS);   // every epilogue warp that reads it (of both CTAs)
        }
        mbar_init(&drain_bar[0], 1);
        mbar_init(&drain_bar[1], 1);
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

    // Register shares of the wide variants (3 warpgroups of 168 at launch): 224 for the two that hold
    // the sums, 56 for the producers', 2 x 224 + 56 = 3 x 168.
    if (warp >= WGS * 4) {
        if constexpr (WGS > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == TMA_WARP && elect_one()) {
            tma_prefetch_desc(&p.map_a);
            tma_prefetch_desc(&p.map_b);
            const uint32_t a0 = smem_addr(smem), b0 = smem_addr(smem + plan.b_off), full0 = smem_addr(full), empty0 = smem_addr(empty);
            const uint32_t a_stage = plan.a_stage, b_stage = plan.b_stage;
            const uint32_t bytes = CTAS * (a_stage + b_stage);
            const int KB = p.KB, tiles = p.tiles, m_tiles = p.m_tiles;
            int slot = 0;
            uint32_t ph = 0, fills = 0;                 // fills: at most NS are of interest
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                const int nt = t / m_tiles;
                const int m0 = (t - nt * m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0);
                // B rows: of a pair, each CTA brings half of each part's columns (gated: the gate rows or the linear ones)
                const int nb = GATED ? nt * FP8_BLOCK + (CTAS == 2 ? 0 : (int)rank * HW) : nt * BN + (CTAS == 2 ? (int)rank * (PN / 2) : 0);
                for (int kb = 0, k0 = 0; kb < KB; ++kb, k0 += FP8_KS) {
                    const uint32_t bar = full0 + 8u * slot;
                    if (!wait_phase<false>(empty0 + 8u * slot, ph ^ 1, wc)) { ok = false; break; }
                    if (CTAS == 1 || rank == 0) mbar_arrive_expect_tx(bar, bytes);
                    const uint32_t as = a0 + slot * a_stage, bs = b0 + slot * b_stage;
                    tma_load_3d<CTAS>(as, &p.map_a, bar, k0, m0, 0);
                    if constexpr (CTAS == 2) {
#pragma unroll
                        for (int h = 0; h < SPLIT; ++h)
                            tma_load_3d<2>(bs + h * (PN / 2) * FP8_KS, &p.map_b, bar, k0, nb + h * (GATED ? HW : PN), GATED ? (int)rank : 0);
                    } else {
                        tma_load_3d<1>(bs, &p.map_b, bar, k0, nb, 0);
                        if constexpr (GATED) tma_load_3d<1>(bs + HW * FP8_KS, &p.map_b, bar, k0, nb, 1);
                    }
                    fills = min(fills + 1, (uint32_t)NS);
                    if (++slot == NS) { slot = 0; ph ^= 1; }
                }
            }
            // Back over the last fills: until the MMAs have freed every slot, so that no arrival is still on
            // its way to this CTA's barriers when it ends; after an abort, until the copies have landed.
            for (uint32_t i = 0; i < fills; ++i) {
                if (--slot < 0) { slot = NS - 1; ph ^= 1; }
                if (ok) wait_drain(&empty[slot], ph, p.wait_limit_ns);
                else if (rank == 0 || CTAS == 1) wait_drain(&full[slot], ph, p.wait_limit_ns);
            }
        } else if ((warp == MMA_WARP || warp == MMA_WARP + 1) && (CTAS == 1 || rank == 0) && elect_one()) {
            // Two MMA warps: one alone takes longer to issue a block's MMAs and commits than the tensor core
            // to run them.  They take the two parts of every block's accumulator, or every other block.
            // kind::f8f6f4 descriptor: fp32 accumulators (1 << 4), E4M3 x E4M3 (0), both K-major, N >> 3, M >> 4
            constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(PN >> 3) << 17) | ((uint32_t)(FP8_BM * CTAS >> 4) << 24);
            constexpr int BY = SPLIT == 2 ? 1 : 2;              // blocks between two of this warp's
            const int m = warp - MMA_WARP, part = SPLIT == 2 ? m : 0;
            const int skip = SPLIT == 2 ? 0 : m;
            const long long blocks = (long long)((p.tiles - first + step - 1) / step) * p.KB;
            const uint32_t full0 = smem_addr(full), empty0 = smem_addr(empty);
            const uint32_t d_full0 = smem_addr(d_full + part * BUFS), d_empty0 = smem_addr(d_empty + part * BUFS);
            const uint64_t ad0 = smem_desc_sw128(smem_addr(smem));
            const uint64_t bd0 = smem_desc_sw128(smem_addr(smem + plan.b_off + part * (PN / CTAS) * FP8_KS));
            const uint32_t a_step = plan.a_stage >> 4, b_step = plan.b_stage >> 4;     // in the descriptors' address units
            const uint32_t d0 = tmem + (uint32_t)(part * BUFS * PN);
            int slot = skip % NS, buf = skip % BUFS;
            uint32_t ph = 0, dph = 0;
            bool ok = true, any = false;
            for (long long g = skip; g < blocks; g += BY) {
                if (!wait_phase<CTAS == 2>(d_empty0 + 8u * buf, dph ^ 1, wc) || !wait_phase<false>(full0 + 8u * slot, ph, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = ad0 + slot * a_step, bd = bd0 + slot * b_step;
#pragma unroll
                for (int k = 0; k < 4; ++k)      // past K the operands are zeros
                    mma_f8<CTAS>(d0 + (uint32_t)(buf * PN), ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                any = true;
                mma_commit_g<CTAS>(d_full0 + 8u * buf);
                mma_commit_g<CTAS>(empty0 + 8u * slot);
                if ((slot += BY) >= NS) { slot -= NS; ph ^= 1; }
                if ((buf += BY) >= BUFS) { buf -= BUFS; dph ^= 1; }
            }
            if (!ok && any) {
                mma_commit_g<CTAS>(smem_addr(&drain_bar[m]));
                wait_drain(&drain_bar[m], 0, p.wait_limit_ns);
            }
        }
    } else {
        if constexpr (WGS > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int wg = warp >> 2, q = warp & 3;
        const int part = SPLIT == 2 ? wg : 0;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(SPLIT == 2 ? wg * BUFS * PN : wg * CW);
        const uint32_t d_full0 = smem_addr(d_full + part * BUFS);
        const uint32_t d_empty0 = CTAS == 2 ? map_to_rank(smem_addr(d_empty + part * BUFS), 0) : smem_addr(d_empty);
        int buf = 0, par = 0, cb = 0;
        uint32_t dph = 0, exph = 0;
        bool ok = true;
        // first row and column of the warp's part of tile t
        auto place = [&](int t, int &m0, int &n0) {
            const int nt = t / p.m_tiles;
            m0 = (t % p.m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0) + 32 * q;
            n0 = GATED ? nt * FP8_BLOCK + (WGS > 1 ? wg : (int)rank) * HW : nt * BN + wg * CW;
        };
        // The scales come a chunk of K blocks ahead (the next tile's first chunk during this one's
        // last), asynchronously: a load per block and row in the loop below put an L2 round trip on
        // every block.  Neighbouring lanes take a row's blocks of the chunk.
        float *scales = reinterpret_cast<float *>(smem + plan.scale_off + warp * FP8_CHUNK_BYTES);
        auto fetch = [&](int t, int kb0, int into) {
            if (t < p.tiles) {
                int m0, n0;
                place(t, m0, n0);
                const uint32_t dst = smem_addr(scales + into * FP8_CHUNK * FP8_CHUNK_ROW);
                const int k = lane % FP8_CHUNK, kb = kb0 + k;
                if (kb < p.KB) {
#pragma unroll
                    for (int i = 0; i < FP8_CHUNK; ++i) {
                        const int r = i * (32 / FP8_CHUNK) + lane / FP8_CHUNK;
                        if (m0 + r < p.M)
                            cp_async4(dst + (uint32_t)(k * FP8_CHUNK_ROW + r) * 4, p.a_scale + (long long)(m0 + r) * p.KB + kb);
                    }
                    const int half = lane / FP8_CHUNK;
                    if (half < (GATED ? 2 : 1) && n0 < p.N)
                        cp_async4(dst + (uint32_t)(k * FP8_CHUNK_ROW + 32 + half) * 4,
                                  p.b_scale + ((long long)half * p.NB + n0 / FP8_BLOCK) * p.KB + kb);
                }
            }
            cp_async_commit();
        };
        fetch(first, 0, 0);
        for (int t = first; t < p.tiles && ok; t += step) {
            int m0, n0;
            place(t, m0, n0);
            const bool active = m0 < p.M && n0 < p.N;      // the warp has something to write
            float acc[CW];
            if constexpr (GATED) {
                load_bias<HW>(acc, p.bias ? p.bias + n0 : nullptr, p.N - n0);
                load_bias<HW>(acc + HW, p.bias ? p.bias + p.N + n0 : nullptr, p.N - n0);
            } else {
                load_bias<CW>(acc, p.bias ? p.bias + n0 : nullptr, p.N - n0);
            }
            for (int kb = 0; kb < p.KB; ++kb) {
                const int k = kb % FP8_CHUNK;
                if (k == 0) {
                    __syncwarp();               // the buffer's last readers are done
                    fetch(kb + FP8_CHUNK < p.KB ? t : t + step, kb + FP8_CHUNK < p.KB ? kb + FP8_CHUNK : 0, cb ^ 1);
                    cp_async_wait<1>();
                    __syncwarp();
                    cb ^= 1;
                }
                const float *sc = scales + ((cb ^ 1) * FP8_CHUNK + k) * FP8_CHUNK_ROW;
                const float sa = sc[lane], s0 = sa * sc[32], s1 = GATED ? sa * sc[33] : s0;
                if (!__all_sync(0xffffffffu, wait_phase<false>(d_full0 + 8u * buf, dph, wc))) { ok = false; break; }
                tc_fence_after();
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CTAS == 2) mbar_arrive_remote(d_empty0 + 8u * (uint32_t)buf);
                        else mbar_arrive(&d_empty[buf]);
                    }
                };
                if (active) {
                    // the next LD columns are on their way while these are added
                    const uint32_t from = lane_base + (uint32_t)(buf * PN);
                    uint32_t r[2][LD];
                    tmem_ld<LD>(from, r[0]);
#pragma unroll
                    for (int c = 0; c < CW; c += LD) {
                        tmem_wait_ld();
                        if (c + LD < CW) tmem_ld<LD>(from + (uint32_t)(c + LD), r[(c / LD + 1) & 1]);
                        else release();
#pragma unroll
                        for (int i = 0; i < LD; ++i)
                            acc[c + i] = fmaf(__uint_as_float(r[(c / LD) & 1][i]), GATED && c + i >= HW ? s1 : s0, acc[c + i]);
                    }
                } else {
                    release();
                }
                if (++buf == BUFS) { buf = 0; dph ^= 1; }
            }
            if (!ok) break;
            if constexpr (GATED) {
                const int row = 32 * q + lane;
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < HW; ++i) {
                    const float g = fmin_nan(acc[i], p.limit);
                    const float u = fmax_nan(fmin_nan(acc[HW + i], p.limit), -p.limit);
                    acc[i] = __fdividef(g, 1.0f + __expf(-p.alpha * g)) * (u + p.shift);
                    if (n0 + i < p.N) amax = fmax_nan(amax, fabsf(acc[i]));
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
                    if (!__all_sync(0xffffffffu, wait_phase<true>(smem_addr(bar), exph, wc))) { ok = false; break; }
                } else {
                    slot[wg * FP8_BM] = amax;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                    if (!__all_sync(0xffffffffu, wait_phase<false>(smem_addr(bar), exph, wc))) { ok = false; break; }
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
                uint8_t *stage = smem + plan.stage_off + warp * FP8_TILE_BYTES;
                if (p.type == FP8_BF16) store_columns<__nv_bfloat16, CW>(p, acc, stage, m0, n0, lane);
                else if (p.type == FP8_FP16) store_columns<__half, CW>(p, acc, stage, m0, n0, lane);
                else store_columns<float, CW>(p, acc, stage, m0, n0, lane);
            }
        }
    }

    cp_async_wait<0>();
    __syncwarp();
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
    if (e == cudaSuccess) e = setup_t<256, 2, false, 1>();
    if (e == cudaSuccess) e = setup_t<256, 2, true, 1>();
    return e;
}

cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const Fp8Plan &pl, int gated, cudaStream_t s) {
    if (gated) {
        if (pl.bn == 256) return launch_t<256, 2, true, 1>(p, pl, s);
        if (pl.bn == 32) return launch_t<32, 1, true, 8>(p, pl, s);
        return launch_t<64, 1, true, 4>(p, pl, s);
    }
    if (pl.bn == 256) return launch_t<256, 2, false, 1>(p, pl, s);
    if (pl.bn == 32) return launch_t<32, 1, false, 1>(p, pl, s);
    if (pl.bn == 64) return launch_t<64, 1, false, 1>(p, pl, s);
    return launch_t<128, 1, false, 1>(p, pl, s);
}

}  // namespace moe
