// Products of E4M3 matrices with fp32 block scales, on tcgen05 (kind::f8f6f4).
//
//   D_kb[m, n] = sum_{k in block kb} a[m, k] b[n, k]
//   c[m, n]    = sum_kb sa[m, kb] sb[n / 128, kb] D_kb[m, n]  (+ bias[n]) (+ residual[m, n])
//
// One 128-K block is one shared-memory stage and four MMAs (K = 32) into an accumulator of its
// own in TMEM.  The scales are any fp32 numbers, so the tensor core cannot apply them: the
// epilogue warps read each block's accumulator, multiply by sa * sb (one number per thread and
// 64 or 128 columns: a thread holds one row) and add it to fp32 sums in registers, while the
// MMAs fill the next accumulator.  That is one FMA and one word of TMEM per 128 products.  Large products: 8192 x
// 5120 x 2880 takes 143 to 157 us, 1.5 to 1.7 PFLOP/s, the MMAs and copies alone 88 (at the power limit's clock).  A
// 256-column K block takes 0.6 us, some 960 clocks, where the MMAs need 512 at their nominal rate and the sums 579
// in isolation; the tensor pipe is 45% and the issue slots 51% busy, so neither is the bound by itself (whether they
// contend for TMEM or the hand-overs show has not been told apart).  A tile's start and end, which no MMA covers, are
// another 3 us, nine times here.
//
// Gated (both projections of a gated feed-forward block): a CTA's accumulator columns are half
// gate rows and half linear rows of W13, so a thread holds a row's gate and linear value of the
// same columns, computes h = min(g, L) sigmoid(alpha min(g, L)) (clamp(u, -L, L) + shift), and
// writes h in E4M3 with the scale of its 128-column block; only the block's maximum crosses
// warps.
//
// Three forms (fp8_plan chooses):
//   pairs   many tiles: two CTAs of a cluster share MMAs of 256 rows x 256 columns (cta_group::2), each
//           holding its 128 rows' sums and half of B.  Persistent; a K block's accumulator is two
//           parts of 128 columns, one per epilogue warpgroup, each filled and freed by itself.  (Gated,
//           8192 x 2 x 2880 x 2880: 163 to 171 us, 1.6 to 1.7 PFLOP/s.)
//   single  128 x 128 tiles, one CTA each, persistent: few rows by many columns, or too few tiles for pairs.
//           64 rows by 201088 columns (fp32 out), K = 2880: 132 us at 1965 MHz in a run of calls with a new result
//           each (631 MB at 4.8 TB/s), 124 into the same two results; a tile's 23 K blocks at 0.34 us of hand-overs
//           are what it waits for.  1024 x 5120 x 2880: 28 us.
//   split   few tiles: the CTAs of a cluster split K (a block costs a CTA some 0.2 us of hand-overs whatever
//           its size, so the chain of blocks is what takes the time), then join their sums through
//           distributed shared memory, in a fixed order, each finishing some of the rows.  32 x 5120 x 2880:
//           7.3 us in a run of calls (10.5 with K whole) and 8.9 with all weights from memory, 15 MB that HBM could
//           bring in 2.3: 8 blocks' hand-overs, the join and the launch.
//
// Warp roles: 8 epilogue warps (warp w reads TMEM lane quarter w % 4), the TMA producer, two MMA
// warps, one elected lane of each running its loop, then the warp that fetches the scales (16 K
// blocks ahead: loads of them in the epilogue's loop put a round trip to L2 on every block).
// Tiles are walked rows fastest, so the B tile of neighbouring CTAs is the same and A stays in L2.
//
// Every wait is bounded (WaitCtl); when one runs out the CTA stops issuing, waits (bounded) for
// what it has in flight, frees TMEM and returns with the timeout counted.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8_kernels.cuh"
#include "fp8_ptx.cuh"
#include "kernels.cuh"

namespace moe {

namespace {

constexpr unsigned int FP8_ERR_WAIT = 1u;      // what a wait that runs out adds to the context's count

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }

// h of a gate and a linear value: min(g, L) sigmoid(alpha min(g, L)) (clamp(u, -L, L) + shift).
__device__ __forceinline__ float gated_value(const Fp8GemmParams &p, float g, float u) {
    g = fmin_nan(g, p.limit);
    u = fmax_nan(fmin_nan(u, p.limit), -p.limit);
    return g * rcp_approx(1.0f + exp2_approx(p.minus_alpha_log2e * g)) * (u + p.shift);
}

// V elements (1, 2 or 4) of type T.
template <typename T, int V>
struct Pack {
    typename std::conditional<V * sizeof(T) == 16, uint4, typename std::conditional<V * sizeof(T) == 8, uint2,
        typename std::conditional<V == 2, uint32_t, T>::type>::type>::type raw;
    __device__ __forceinline__ float get(int j) const { return static_cast<float>(reinterpret_cast<const T *>(&raw)[j]); }
    __device__ __forceinline__ void set(const float (&v)[V]) {
        if constexpr (V > 1 && std::is_same<T, __half>::value) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) reinterpret_cast<__half2 *>(&raw)[j] = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        } else if constexpr (V > 1 && std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) reinterpret_cast<__nv_bfloat162 *>(&raw)[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) reinterpret_cast<T *>(&raw)[j] = static_cast<T>(v[j]);
        }
    }
};

// The staged sums (+ bias) (+ residual), rounded once, to rows m0.. and columns n0.. of c; lane i brings the
// bias of column n0 + i.  V == 4: 32 whole rows, four elements per lane; V == 1: what there is, a column per
// lane.  Several steps at a time, their residuals first; every element of the residual is read by the thread that
// writes c's, so the two may be the same.
template <typename T, int CC, int V, bool RES>
__device__ __forceinline__ void put_tile(const Fp8GemmParams &p, const float *tile, float bias, int m0, int n0, int lane) {
    constexpr int LPR = CC / V, RPI = 32 / LPR, B = V == 1 && RES ? 8 : 4;     // lanes per row, rows per step, steps at a time
    typedef decltype(Pack<T, V>::raw) Raw;
    const int pc = lane % LPR, r0 = lane / LPR, col = n0 + V * pc;
    float b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = __shfl_sync(0xffffffffu, bias, V * pc + j);
    const int rows = V == 4 ? 32 : col < p.N ? min(32, p.M - m0) : 0;
    T *c = static_cast<T *>(p.c) + (long long)(m0 + r0) * p.ldc + col;
    const T *res = RES ? static_cast<const T *>(p.residual) + (long long)(m0 + r0) * p.ldr + col : nullptr;
    const long long cs = RPI * p.ldc, rs = RPI * p.ldr;
    const float *f = tile + r0 * (CC + 4) + V * pc;
#pragma unroll 1
    for (int r = r0; r < rows; r += B * RPI, f += B * RPI * (CC + 4)) {
        Pack<T, V> old[B];
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < B; ++i, res += rs)
                if (V == 4 || r + i * RPI < rows) old[i].raw = *reinterpret_cast<const Raw *>(res);
        }
#pragma unroll
        for (int i = 0; i < B; ++i, c += cs) {
            if (V == 4 || r + i * RPI < rows) {
                float o[V];
                if constexpr (V == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(f + i * RPI * (CC + 4));
                    o[0] = v.x, o[1] = v.y, o[2] = v.z, o[3] = v.w;
                } else {
                    o[0] = f[i * RPI * (CC + 4)];
                }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    o[j] += b[j];
                    if constexpr (RES) o[j] += old[i].get(j);
                }
                Pack<T, V> out;
                out.set(o);
                *reinterpret_cast<Raw *>(c) = out.raw;
            }
        }
    }
}

// The same for 16-bit types where rows start anywhere or end inside the tile.  16 lanes take a row, each two
// neighbours that share a word of c: columns 2 i and 2 i + 1, or, where the row starts inside a word, 1 + 2 i and
// 2 + 2 i (a lane's rows are two apart, so they start alike).  What is left at a row's ends, one column each, is
// written a lane a row.  (An element a lane: twice the loads and stores.  The residual's are asm so that they stay
// in one stream: as branches, each waited for its own.)
template <typename T, int CC, bool RES>
__device__ __forceinline__ void put_pairs(const Fp8GemmParams &p, const float *tile, float bias, int m0, int n0, int lane) {
    static_assert(CC == 32 && sizeof(T) == 2, "a row is 16 lanes' words");
    constexpr int B = RES ? 8 : 4;              // steps at a time
    const int rows = min(32, p.M - m0), cols = min(CC, p.N - n0);
    const auto half = [](const T *at) { return (int)(reinterpret_cast<uintptr_t>(at) >> 1 & 1); };
    T *c = static_cast<T *>(p.c) + (long long)m0 * p.ldc + n0;
    const T *res = RES ? static_cast<const T *>(p.residual) + (long long)m0 * p.ldr + n0 : nullptr;

    T *end_c = c + lane * p.ldc;
    const T *end_res = RES ? res + lane * p.ldr : nullptr;
    const int lead = half(end_c);
    const bool end0 = lane < rows && lead, end1 = lane < rows && ((cols - lead) & 1);
    uint32_t old0 = 0, old1 = 0;
    if constexpr (RES) {
        ld_u16_if(old0, end_res, end0);
        ld_u16_if(old1, end_res + (cols - 1), end1);
    }

    const int r0 = lane >> 4;
    c += r0 * p.ldc;
    const int k = 2 * (lane & 15) + half(c);
    const float b0 = __shfl_sync(0xffffffffu, bias, k), b1 = __shfl_sync(0xffffffffu, bias, (k + 1) & 31);
    const bool in = k + 1 < cols;
    c += k;
    if (RES) res += r0 * p.ldr + k;
    const bool apart = RES && half(res);        // the residual's rows start otherwise than c's
    const float *f = tile + r0 * (CC + 4) + k;
#pragma unroll 1
    for (int r = r0; r < rows; r += 2 * B) {
        uint32_t lo[B], hi[B];
        if constexpr (RES) {
#pragma unroll
            for (int i = 0; i < B; ++i, res += 2 * p.ldr) {
                const bool on = in && r + 2 * i < rows;
                hi[i] = 0;
                ld_u32_if(lo[i], res, on && !apart);
                ld_u16_if(lo[i], res, on && apart);
                ld_u16_if(hi[i], res + 1, on && apart);
            }
        }
#pragma unroll
        for (int i = 0; i < B; ++i, c += 2 * p.ldc, f += 2 * (CC + 4)) {
            if (in && r + 2 * i < rows) {
                float o[2] = {f[0] + b0, f[1] + b1};
                if constexpr (RES) {
                    Pack<T, 2> old;
                    old.raw = lo[i] | hi[i] << 16;
                    o[0] += old.get(0), o[1] += old.get(1);
                }
                Pack<T, 2> out;
                out.set(o);
                *reinterpret_cast<uint32_t *>(c) = out.raw;
            }
        }
    }

    const float be = __shfl_sync(0xffffffffu, bias, cols - 1), bl = __shfl_sync(0xffffffffu, bias, 0);
    f = tile + lane * (CC + 4);
    Pack<T, 2> old;
    old.raw = old0 | old1 << 16;
    if (end0) *end_c = static_cast<T>(f[0] + bl + (RES ? old.get(0) : 0.0f));
    if (end1) end_c[cols - 1] = static_cast<T>(f[cols - 1] + be + (RES ? old.get(1) : 0.0f));
}

template <typename T, int CC, bool RES>
__device__ __forceinline__ void put_tile(const Fp8GemmParams &p, const float *tile, float bias, int m0, int n0, int lane) {
    if (p.vec && m0 + 32 <= p.M && n0 + CC <= p.N) put_tile<T, CC, 4, RES>(p, tile, bias, m0, n0, lane);
    else if constexpr (sizeof(T) == 2) put_pairs<T, CC, RES>(p, tile, bias, m0, n0, lane);
    else put_tile<T, CC, 1, RES>(p, tile, bias, m0, n0, lane);
}

// A warp's sums, CC columns at a time: each thread's row into the staging tile, rows out of it.  The loop over
// the parts stays a loop (its body is every part's), and the residual has kernels of its own: code that runs once
// a tile does not stay in the instruction caches, and the largest products lost 4% to a second copy of put_tile.
// (Measured against this staging: 128 bytes of a row at a time in c's type, unrolled, 6% longer on narrow tiles;
// 16-byte pieces of 32 rows straight from the registers 30% longer.)
template <int CW, int CC, bool RES>
__device__ __forceinline__ void store_columns(const Fp8GemmParams &p, const float (&acc)[CW], const float (&bias)[(CW + 31) / 32],
                                              float *tile, int m0, int n0, int lane) {
#pragma unroll 1
    for (int part = 0; part < CW / CC; ++part) {
        if (n0 + part * CC >= p.N) break;
        float b = 0.0f;
#pragma unroll
        for (int s = 0; s < CW / CC; ++s)
            if (s == part) {
#pragma unroll
                for (int i = 0; i < CC; i += 4)
                    *reinterpret_cast<float4 *>(tile + lane * (CC + 4) + i) =
                        make_float4(acc[s * CC + i], acc[s * CC + i + 1], acc[s * CC + i + 2], acc[s * CC + i + 3]);
                b = bias[s * CC / 32];
            }
        __syncwarp();
        if (p.type == FP8_BF16) put_tile<__nv_bfloat16, CC, RES>(p, tile, b, m0, n0 + part * CC, lane);
        else if (p.type == FP8_FP16) put_tile<__half, CC, RES>(p, tile, b, m0, n0 + part * CC, lane);
        else put_tile<float, CC, RES>(p, tile, b, m0, n0 + part * CC, lane);
        __syncwarp();
    }
}

// (Volatile keeps it behind the cluster barrier; no memory clobber, so that a round's loads stay together.)
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// Four neighbouring sums at byte `at` of every CTA's tile, and their sum in the CTAs' order.
struct Parts {
    float4 v[FP8_SPLIT_MAX];
    __device__ __forceinline__ void load(uint32_t tile, uint32_t at, int split) {
#pragma unroll
        for (int c = 0; c < FP8_SPLIT_MAX; ++c)
            if (c < split) v[c] = ld_cluster_f32x4(map_to_rank(tile + at, (uint32_t)c));
    }
    __device__ __forceinline__ float4 sum(int split) const {
        float4 t = v[0];
#pragma unroll
        for (int c = 1; c < FP8_SPLIT_MAX; ++c)
            if (c < split) t.x += v[c].x, t.y += v[c].y, t.z += v[c].z, t.w += v[c].w;
        return t;
    }
};

template <typename T>
__device__ __forceinline__ void put_four(const Fp8GemmParams &p, long long row, int n, float (&o)[4]) {
    T *c = static_cast<T *>(p.c) + row * p.ldc + n;
    const T *res = static_cast<const T *>(p.residual);
    if (res) res += row * p.ldr + n;
    if (p.vec && n + 4 <= p.N) {
        Pack<T, 4> v;
        if (res) {
            v.raw = *reinterpret_cast<const decltype(v.raw) *>(res);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] += v.get(j);
        }
        v.set(o);
        *reinterpret_cast<decltype(v.raw) *>(c) = v.raw;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < p.N) c[j] = static_cast<T>(res ? o[j] + static_cast<float>(res[j]) : o[j]);
    }
}

// A tile whose K the cluster's CTAs have split: every CTA finishes some of the rows, a warp a row, a lane four
// columns (gated: four columns of h), reading all CTAs' sums through distributed shared memory.
template <int BN, bool GATED>
__device__ __forceinline__ void join_parts(const Fp8GemmParams &p, uint32_t tile, int rank, int t, int warp, int lane) {
    const int nt = t / p.m_tiles, m0 = (t - nt * p.m_tiles) * FP8_BM;
    const int rows = min(FP8_BM, p.M - m0), each = (rows + p.split - 1) / p.split;
    const int n = nt * 128 + 4 * lane;          // BN columns of c, or BN / 2 of h: 128
    float b[2][4];
#pragma unroll
    for (int h = 0; h < (GATED ? 2 : 1); ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) b[h][j] = p.bias && n + j < p.N ? bf16_bits_to_f32(p.bias[h * p.N + n + j]) : 0.0f;
    const int end = min(rows, (rank + 1) * each);
    // plain: two rows at a time, gated: a row's gate and linear sums, so that 16 remote loads are in flight
    constexpr int STEP = FP8_WGS * 4;
#pragma unroll 1
    for (int r = rank * each + warp; r < end; r += GATED ? STEP : 2 * STEP) {
        Parts x, y;
        if constexpr (!GATED) {
            const uint32_t at = (uint32_t)(r * (BN + 4) + 4 * lane) * 4;
            x.load(tile, at, p.split);
            if (r + STEP < end) y.load(tile, at + STEP * (BN + 4) * 4, p.split);
            if (n >= p.N) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (r + i * STEP >= end) break;
                const long long m = m0 + r + i * STEP;
                const float4 v = i ? y.sum(p.split) : x.sum(p.split);
                float o[4] = {v.x + b[0][0], v.y + b[0][1], v.z + b[0][2], v.w + b[0][3]};
                if (p.type == FP8_BF16) put_four<__nv_bfloat16>(p, m, n, o);
                else if (p.type == FP8_FP16) put_four<__half>(p, m, n, o);
                else put_four<float>(p, m, n, o);
            }
        } else {
            // a warpgroup's columns are 64 gate and 64 linear ones
            const uint32_t at = (uint32_t)(r * (BN + 4) + lane / 16 * 128 + lane % 16 * 4) * 4;
            x.load(tile, at, p.split);
            y.load(tile, at + 256, p.split);
            const float4 gv = x.sum(p.split), uv = y.sum(p.split);
            const float gs[4] = {gv.x, gv.y, gv.z, gv.w}, us[4] = {uv.x, uv.y, uv.z, uv.w};
            const long long m = m0 + r;
            float h[4], amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = gated_value(p, gs[j] + b[0][j], us[j] + b[1][j]);
                if (n + j < p.N) amax = fmax_nan(amax, fabsf(h[j]));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) amax = fmax_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const float s = fmax_nan(amax / FP8_MAX, FP8_SCALE_MIN), inv = 1.0f / s;
            if (n < p.N)                        // F is a multiple of 16
                *reinterpret_cast<uint32_t *>(p.h + m * p.N + n) = f32x4_to_e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
            if (lane == 0) p.h_scale[m * p.NB + nt] = s;
        }
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

// RES: with a residual (a kernel of its own, as its code made the others' slower: see store_columns).  2048 x 5120 x
// 2880 bf16: 57 us with one, 47 without: the reads of it are eight rounds of loads a tile (fewer, of 32 steps, spill).
template <int BN, int CTAS, bool GATED, bool SK, bool RES>
__global__ void __launch_bounds__(FP8_THREADS, 1) fp8_gemm_kernel(const __grid_constant__ Fp8GemmParams p) {
    constexpr int WGS = FP8_WGS;                // epilogue warpgroups
    constexpr int CW = BN / WGS;                // accumulator columns per epilogue thread
    constexpr int LD = CW > 64 && !GATED && !RES ? 32 : 16;     // columns of a TMEM load (registers: 2 LD beside the CW sums)
    constexpr int CC = FP8_TILE_COLS;           // columns of a staging tile
    constexpr int HW = CW / 2;                  // gated: h columns per thread
    constexpr int BUFS = fp8_bufs(BN);
    constexpr int SPLIT = fp8_split(BN);        // parts of an accumulator: one per warpgroup, or the whole
    constexpr int PN = BN / SPLIT;              // columns of an MMA
    static_assert(BUFS % 2 == 0, "an accumulator's uses are one MMA warp's, too");
    static_assert(!GATED || HW * WGS == FP8_BLOCK, "the warpgroups share a gated row's block");
    static_assert(!SK || CTAS == 1, "CTAs of a cluster split K, or are a pair");
    extern __shared__ uint8_t smem_raw[];
    // 1024-aligned, as an offset from the array: a pointer rounded as a number is no longer known to be shared
    // memory, and its loads and stores become generic ones
    uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
    const int NS = p.n_stages;
    const Fp8Smem plan = fp8_smem(BN, CTAS, GATED, SK, p.a_rows, NS);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + plan.bar_off);
    uint64_t *empty = full + NS;
    uint64_t *d_full = empty + NS;              // [SPLIT][BUFS] a K block's accumulator (part) is complete
    uint64_t *d_empty = d_full + SPLIT * BUFS;  // ... and has been read
    uint64_t *drain_bar = d_empty + SPLIT * BUFS;   // [2 MMA warps]
    uint64_t *ex_bar = drain_bar + 2;           // [4 quarters][2 parities]
    uint64_t *sc_full = ex_bar + 8;             // [FP8_CHUNKS] a chunk of scales is there
    uint64_t *sc_empty = sc_full + FP8_CHUNKS;  // ... and has been read
    const uint32_t scales0 = smem_addr(smem + plan.scale_off);
    float *ex = reinterpret_cast<float *>(smem + plan.ex_off);       // [2 parities][2 warpgroups][128 rows]
    uint32_t *tmem_base_s = reinterpret_cast<uint32_t *>(smem + plan.misc_off);
    volatile int *abort_s = reinterpret_cast<volatile int *>(smem + plan.misc_off + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS > 1 || SK ? cluster_ctarank() : 0;
    constexpr int TMA_WARP = WGS * 4, MMA_WARP = TMA_WARP + 1, SCALE_WARP = TMA_WARP + 3;
    constexpr uint32_t COLS = BUFS * BN;

    if (warp == TMA_WARP) {                     // (a lane a barrier: one thread after another took 0.2 us)
        if (lane < NS) {
            mbar_init(&full[lane], 1);          // the (even CTA's) producer
            mbar_init(&empty[lane], SPLIT);     // MMA commits
        }
        if (lane < SPLIT * BUFS) {
            mbar_init(&d_full[lane], 1);        // MMA commit
            mbar_init(&d_empty[lane], WGS / SPLIT * 4 * CTAS);    // every epilogue warp that reads it (of both CTAs)
        }
        if (lane < 2) mbar_init(&drain_bar[lane], 1);
        if (lane < 8) mbar_init(&ex_bar[lane], WGS);
        if (lane < FP8_CHUNKS) {
            mbar_init(&sc_full[lane], 32);      // every lane of the scale warp
            mbar_init(&sc_empty[lane], WGS * 4);    // every epilogue warp
        }
        if (lane == 0) *abort_s = 0;
        fence_barrier_init();
    }
    if (warp == MMA_WARP) tmem_alloc_g<CTAS>(tmem_base_s, COLS);
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS > 1) cluster_sync();     // the peer's barriers are initialised
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = *tmem_base_s;
    const WaitCtl wc{abort_s, p.err, FP8_ERR_WAIT, p.wait_limit_ns};
    // SK: a cluster takes one tile, each of its CTAs a part of K
    const int group = SK ? p.split : CTAS;
    const int first = blockIdx.x / group, step = gridDim.x / group;
    const int kb0 = SK ? p.KB * (int)rank / p.split : 0, kb1 = SK ? p.KB * ((int)rank + 1) / p.split : p.KB;

    // Register shares (3 warpgroups of 168 at launch): 224 for the two that hold
    // the sums, 56 for the producers', 2 x 224 + 56 = 3 x 168.
    if (warp >= WGS * 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == TMA_WARP && elect_one()) {
            tma_prefetch_desc(&p.map_a);
            tma_prefetch_desc(&p.map_b);
            const uint32_t a0 = smem_addr(smem), b0 = smem_addr(smem + plan.b_off), full0 = smem_addr(full), empty0 = smem_addr(empty);
            const uint32_t a_stage = plan.a_stage, b_stage = plan.b_stage;
            const uint32_t bytes = CTAS * (a_stage + b_stage);
            const int tiles = p.tiles, m_tiles = p.m_tiles;
            pdl_wait();                                 // (each role where it first touches a predecessor's memory)
            int slot = 0;
            uint32_t ph = 0, fills = 0;                 // fills: at most NS are of interest
            bool ok = true;
            for (int t = first; t < tiles && ok; t += step) {
                const int nt = t / m_tiles;
                const int m0 = (t - nt * m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0);
                // B rows: of a pair, each CTA brings half of each part's columns (gated: the gate rows or the linear ones)
                const int nb = GATED ? nt * FP8_BLOCK : nt * BN + (CTAS == 2 ? (int)rank * (PN / 2) : 0);
                for (int kb = kb0, k0 = kb0 * FP8_KS; kb < kb1; ++kb, k0 += FP8_KS) {
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
#pragma unroll
                        for (int h = 0; h < SPLIT; ++h) {
                            tma_load_3d<1>(bs + h * PN * FP8_KS, &p.map_b, bar, k0, nb + h * (GATED ? HW : PN), 0);
                            if constexpr (GATED) tma_load_3d<1>(bs + (h * PN + HW) * FP8_KS, &p.map_b, bar, k0, nb + h * HW, 1);
                        }
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
            const long long blocks = (long long)((p.tiles - first + step - 1) / step) * (kb1 - kb0);
            const uint32_t full0 = smem_addr(full), empty0 = smem_addr(empty);
            const uint32_t d_full0 = smem_addr(d_full + part * BUFS), d_empty0 = smem_addr(d_empty + part * BUFS);
            const uint64_t ad0 = smem_desc_sw128(smem_addr(smem));
            const uint64_t bd0 = smem_desc_sw128(smem_addr(smem + plan.b_off + part * (PN / CTAS) * FP8_KS));
            const uint32_t a_step = plan.a_stage >> 4, b_step = plan.b_stage >> 4;     // in the descriptors' address units
            const uint32_t d0 = tmem + (uint32_t)(part * BUFS * PN);
            int slot = skip % NS, buf = skip % BUFS;
            uint32_t ph = 0, dph = 0;
            bool ok = true, any = false;
            pdl_wait();                                 // (it reads no such memory, but its waits' time starts here)
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
        } else if (warp == SCALE_WARP) {
            // The scales, a chunk of K blocks at a time: four neighbouring lanes take a row's four blocks.
            const int k = lane % FP8_CHUNK, r0 = lane / FP8_CHUNK;
            constexpr int RPI = 32 / FP8_CHUNK;                 // rows per instruction
            const uint32_t full0 = smem_addr(sc_full), empty0 = smem_addr(sc_empty);
            const uint32_t dst0 = scales0 + (uint32_t)lane * 4;
            pdl_wait();
            int cb = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = first; t < p.tiles && ok; t += step) {
                const int nt = t / p.m_tiles;
                const int m0 = (t - nt * p.m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0);
                const int rows = p.M - m0 - r0;                 // this lane's first row is there if > 0
                const float *sa = p.a_scale + (long long)(m0 + r0) * p.KB + k;
                const long long next = (long long)RPI * p.KB;
                // the weight's scales: gated, the gate's and the linear part's; else each warpgroup's block
                const int blk = (GATED ? nt * FP8_BLOCK : nt * BN + r0 * CW) / FP8_BLOCK;
                const bool has_b = r0 < (GATED ? 2 : WGS) && blk < p.NB;
                const float *sb = p.b_scale + ((long long)(GATED ? r0 * p.NB : 0) + blk) * p.KB + k;
                for (int kb = kb0; kb < kb1; kb += FP8_CHUNK) {
                    if (!__all_sync(0xffffffffu, wait_phase<false>(empty0 + 8u * cb, ph ^ 1, wc))) { ok = false; break; }
                    const uint32_t dst = dst0 + (uint32_t)(cb * FP8_CHUNK_BYTES);
                    if (kb + k < kb1) {
                        const float *src = sa + kb;
#pragma unroll
                        for (int i = 0; i < FP8_BM / RPI; ++i, src += next)
                            if (i * RPI < rows) cp_async4(dst + i * 128, src);
                        if (has_b) cp_async4(dst + FP8_BM * FP8_CHUNK * 4, sb + kb);      // behind the rows
                    }
                    cp_async_arrive(full0 + 8u * cb);
                    if (++cb == FP8_CHUNKS) { cb = 0; ph ^= 1; }
                }
            }
            cp_async_wait_all();
        }
        __syncwarp();
        if constexpr (SK) cluster_sync();       // (with the epilogue warps' below)
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int wg = warp >> 2, q = warp & 3;
        const int part = SPLIT == 2 ? wg : 0;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(SPLIT == 2 ? wg * BUFS * PN : wg * CW);
        const uint32_t d_full0 = smem_addr(d_full + part * BUFS);
        const uint32_t d_empty_here = smem_addr(d_empty + part * BUFS);
        const uint32_t d_empty0 = CTAS == 2 ? map_to_rank(d_empty_here, 0) : d_empty_here;
        const uint32_t sc_full0 = smem_addr(sc_full), sc_empty0 = smem_addr(sc_empty);
        int buf = 0, par = 0, cb = 0;
        uint32_t dph = 0, exph = 0, cph = 0;
        bool ok = true;
        auto release = [&](uint32_t bar) {          // the warp has read its columns of an accumulator
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CTAS == 2) mbar_arrive_remote(bar);
                else mbar_arrive_at(bar);
            }
        };
        pdl_wait();
        for (int t = first; t < p.tiles && ok; t += step) {
            // first row and column of the warp's part of the tile
            const int nt = t / p.m_tiles;
            const int m0 = (t - nt * p.m_tiles) * (FP8_BM * CTAS) + (CTAS == 2 ? (int)rank * FP8_BM : 0) + 32 * q;
            const int n0 = GATED ? nt * FP8_BLOCK + wg * HW : nt * BN + wg * CW;
            const bool active = m0 < p.M && n0 < p.N;      // the warp has something to write
            // lane i: the biases of the columns 32 j + i (gated: of the gate, then of the linear part), read
            // here so that they have arrived when the sums are complete
            float bias[(CW + 31) / 32];
#pragma unroll
            for (int j = 0; j < (CW + 31) / 32; ++j) {
                const int i = 32 * j + lane, col = n0 + (GATED ? i % HW : i);
                bias[j] = !SK && p.bias && col < p.N ? bf16_bits_to_f32(p.bias[(GATED && i >= HW ? p.N : 0) + col]) : 0.0f;
            }
            if constexpr (RES) {
                // the residual's part of this lane's row starts on its way to L2: read after the sums, from memory, it
                // took 6 us a tile
                if (active && m0 + lane < p.M) {
                    const int eb = p.type == FP8_FP32 ? 4 : 2, bytes = min(CW, p.N - n0) * eb;
                    const char *row = static_cast<const char *>(p.residual) + ((m0 + lane) * p.ldr + n0) * eb;
                    for (int i = 0; i < bytes; i += 128) prefetch_l2(row + i);
                }
            }
            float acc[CW];
#pragma unroll
            for (int i = 0; i < CW; ++i) acc[i] = 0.0f;
            for (int kb = kb0; kb < kb1; kb += FP8_CHUNK) {
                wait_phase_through(sc_full0 + 8u * cb, cph, wc);
                const float *sc = reinterpret_cast<const float *>(smem + plan.scale_off + cb * FP8_CHUNK_BYTES);
                const float *sa = sc + (32 * q + lane) * FP8_CHUNK, *sb = sc + (FP8_BM + (GATED ? 0 : wg)) * FP8_CHUNK;
                const int blocks = min(FP8_CHUNK, kb1 - kb);
#pragma unroll 1
                for (int k = 0; k < blocks; ++k) {
                    const float s0 = sa[k] * sb[k], s1 = GATED ? sa[k] * sb[FP8_CHUNK + k] : 0.0f;
                    const uint32_t freed = d_empty0 + 8u * buf;
                    wait_phase_through(d_full0 + 8u * buf, dph, wc);
                    tc_fence_after();
                    if (active) {
                        // the next LD columns are on their way while these are added
                        const uint32_t from = lane_base + (uint32_t)(buf * PN);
                        uint32_t r[2][LD];
                        tmem_ld<LD>(from, r[0]);
#pragma unroll
                        for (int c = 0; c < CW; c += LD) {
                            tmem_wait_ld();
                            if (c + LD < CW) tmem_ld<LD>(from + (uint32_t)(c + LD), r[(c / LD + 1) & 1]);
                            else release(freed);
#pragma unroll
                            for (int i = 0; i < LD; ++i)
                                acc[c + i] = fmaf(__uint_as_float(r[(c / LD) & 1][i]), GATED && c + i >= HW ? s1 : s0, acc[c + i]);
                        }
                    } else {
                        release(freed);
                    }
                    if (++buf == BUFS) { buf = 0; dph ^= 1; }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive_at(sc_empty0 + 8u * cb);
                if (++cb == FP8_CHUNKS) { cb = 0; cph ^= 1; }
                if (__any_sync(0xffffffffu, *abort_s)) { ok = false; break; }
            }
            if constexpr (SK) {
                // every warpgroup's last block is complete, so no copy or MMA uses the rings: the sums go there
                asm volatile("bar.sync 1, %0;" ::"n"(WGS * 128) : "memory");
                const int row = 32 * q + lane;
                if (row < p.a_rows) {
                    float *to = reinterpret_cast<float *>(smem) + row * (BN + 4) + wg * CW;
#pragma unroll
                    for (int i = 0; i < CW; i += 4)
                        *reinterpret_cast<float4 *>(to + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
                }
                break;
            }
            if (!ok) break;
            if constexpr (GATED && !SK) {
                const int row = 32 * q + lane;
                float amax = 0.0f, h[HW];
                float *bs = reinterpret_cast<float *>(smem + plan.stage_off + warp * fp8_tile_bytes(1));
#pragma unroll
                for (int j = 0; j < (CW + 31) / 32; ++j) bs[32 * j + lane] = bias[j];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < HW; ++i) {
                    h[i] = gated_value(p, acc[i] + bs[i], acc[HW + i] + bs[HW + i]);
                    if (n0 + i < p.N) amax = fmax_nan(amax, fabsf(h[i]));
                }
                __syncwarp();
                // the row's maximum over its 128-column block
                float *slot = ex + par * WGS * FP8_BM + row;
                uint64_t *bar = &ex_bar[2 * q + par];
                slot[wg * FP8_BM] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
                if (!__all_sync(0xffffffffu, wait_phase<false>(smem_addr(bar), exph, wc))) { ok = false; break; }
#pragma unroll
                for (int e = 0; e < WGS; ++e) amax = fmax_nan(amax, slot[e * FP8_BM]);
                par ^= 1;
                if (par == 0) exph ^= 1;
                if (active && m0 + lane < p.M) {
                    const float s = fmax_nan(amax / FP8_MAX, FP8_SCALE_MIN);
                    const float inv = 1.0f / s;
                    uint8_t *to = p.h + (long long)(m0 + lane) * p.N + n0;
#pragma unroll
                    for (int i = 0; i < HW; i += 16)
                        if (n0 + i < p.N) {
                            uint32_t u[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                u[j] = f32x4_to_e4m3x4(h[i + 4 * j] * inv, h[i + 4 * j + 1] * inv, h[i + 4 * j + 2] * inv,
                                                       h[i + 4 * j + 3] * inv);
                            *reinterpret_cast<uint4 *>(to + i) = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                    if (n0 % FP8_BLOCK == 0) p.h_scale[(long long)(m0 + lane) * p.NB + n0 / FP8_BLOCK] = s;
                }
            } else if (!SK && active) {
                store_columns<CW, CC, RES>(p, acc, bias, reinterpret_cast<float *>(smem + plan.stage_off + warp * fp8_tile_bytes(0)), m0, n0, lane);
            }
        }
        if constexpr (SK) {
            cluster_sync();                     // every CTA's sums are in its shared memory
            join_parts<BN, GATED>(p, smem_addr(smem), (int)rank, first, warp, lane);
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS > 1 || SK) cluster_sync();   // no CTA leaves while a peer may still reach its shared memory
    tc_fence_after();
    if (warp == MMA_WARP) tmem_dealloc_g<CTAS>(tmem, COLS);
}

// A wait on a barrier that nothing arrives at: it runs out, is counted, and the kernel ends.
__global__ void fp8_selftest_wait_kernel(unsigned int *err, unsigned long long limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    const WaitCtl wc{&abort_flag, err, FP8_ERR_WAIT, limit_ns};
    wait_phase_through(smem_addr(&bar), 0, wc);
}

cudaError_t launch_fp8_selftest_wait(unsigned int *err, unsigned long long limit_ns, cudaStream_t s) {
    fp8_selftest_wait_kernel<<<1, 32, 0, s>>>(err, limit_ns);
    return cudaGetLastError();
}

template <int BN, int CTAS, bool GATED, bool SK, bool RES>
static cudaError_t launch_t(const Fp8GemmParams &p, const Fp8Plan &pl, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.grid);
    cfg.blockDim = dim3(FP8_THREADS);
    cfg.dynamicSmemBytes = FP8_SMEM_SM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = SK ? pl.split : CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = attr[1].val.clusterDim.x > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fp8_gemm_kernel<BN, CTAS, GATED, SK, RES>, p);
}

template <int BN, int CTAS, bool GATED, bool SK, bool RES>
static cudaError_t setup_t() {
    // the registers that the kernel's warpgroups share out have to be there at launch (setmaxnreg waits for them), and
    // another compiler may give the kernel fewer
    cudaFuncAttributes attr;
    cudaError_t e = cudaFuncGetAttributes(&attr, fp8_gemm_kernel<BN, CTAS, GATED, SK, RES>);
    if (e == cudaSuccess && attr.numRegs != 168) e = cudaErrorNotSupported;
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(fp8_gemm_kernel<BN, CTAS, GATED, SK, RES>, cudaFuncAttributeMaxDynamicSharedMemorySize, FP8_SMEM_SM);
}

// Once per device, before the first launch: the kernels' shared memory, and how many clusters of 1 to
// FP8_SPLIT_MAX CTAs the device holds at once (an SM to a CTA; a cluster lies in one GPC).
cudaError_t fp8_gemm_setup(int *clusters) {
    cudaError_t e = setup_t<128, 1, false, false, false>();
    if (e == cudaSuccess) e = setup_t<128, 1, false, false, true>();
    if (e == cudaSuccess) e = setup_t<128, 1, false, true, false>();
    if (e == cudaSuccess) e = setup_t<256, 1, true, true, false>();
    if (e == cudaSuccess) e = setup_t<256, 2, false, false, false>();
    if (e == cudaSuccess) e = setup_t<256, 2, false, false, true>();
    if (e == cudaSuccess) e = setup_t<256, 2, true, false, false>();
    cudaFuncAttributes selftest;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&selftest, fp8_selftest_wait_kernel);
    for (int n = 1; n <= FP8_SPLIT_MAX && e == cudaSuccess; ++n) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n);
        cfg.blockDim = dim3(FP8_THREADS);
        cfg.dynamicSmemBytes = FP8_SMEM_SM;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = n;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&clusters[n], fp8_gemm_kernel<128, 1, false, true, false>, &cfg);
    }
    return e;
}

cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const Fp8Plan &pl, int gated, cudaStream_t s) {
    if (gated) return pl.ctas == 2 ? launch_t<256, 2, true, false, false>(p, pl, s) : launch_t<256, 1, true, true, false>(p, pl, s);
    if (pl.split > 1) return launch_t<128, 1, false, true, false>(p, pl, s);       // (the residual is join_parts')
    if (pl.ctas == 2) return p.residual ? launch_t<256, 2, false, false, true>(p, pl, s) : launch_t<256, 2, false, false, false>(p, pl, s);
    return p.residual ? launch_t<128, 1, false, false, true>(p, pl, s) : launch_t<128, 1, false, false, false>(p, pl, s);
}

}  // namespace moe
