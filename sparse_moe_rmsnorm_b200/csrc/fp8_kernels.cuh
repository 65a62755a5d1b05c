// Parameter blocks and host-side launch plan of the dense 8-bit operators.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace moe {

constexpr int FP8_BLOCK = 128;                 // elements (of a row, or rows and columns of a weight) per scale
constexpr float FP8_MAX = 448.0f;              // largest E4M3 value
constexpr float FP8_SCALE_MIN = 1.17549435e-38f;   // 2^-126: the scale of a block of zeros

enum { FP8_BF16 = 0, FP8_FP16 = 1, FP8_FP32 = 2 };   // MOE_BF16, MOE_FP16, MOE_FP32 of the C ABI

__host__ __device__ inline int fp8_blocks(int n) { return (n + FP8_BLOCK - 1) / FP8_BLOCK; }

struct Fp8NormParams {
    const void *x, *residual;       // [T, d], rows ldx / ldr elements apart; residual may be NULL
    const uint16_t *norm_scale;     // bf16 [d]
    void *sum_out;                  // [T, d], rows lds elements apart, or NULL
    uint8_t *q;                     // E4M3 [T, d]
    float *q_scale;                 // [T, ceil(d / 128)]
    long long ldx, ldr, lds;
    int T, d;
    float eps;
};

struct Fp8GemmParams {
    CUtensorMap map_a;              // u8 {K, M, 1}, box {128, a_rows, 1}
    CUtensorMap map_b;              // u8 {K, N, 1}, box {128, BN / CTAS / split, 1}; gated {K, F, 2}, box {128, h columns of a part, 1}
    const float *a_scale;           // [M, KB]
    const float *b_scale;           // [NB, KB]; gated [2, NB, KB]
    int M, N, K, KB, NB;            // N: output columns (gated: F)
    int m_tiles, tiles;
    int a_rows, n_stages;           // rows of an A stage (128, or M rounded up to 8 below that)
    int split;                      // CTAs of a cluster that share a tile's K
    const uint16_t *bias;           // bf16 [N] (gated [2 F]) or NULL
    const void *residual;           // type [M, N], rows ldr elements apart, or NULL
    void *c;                        // type [M, N], rows ldc elements apart
    long long ldr, ldc;
    int type;                       // FP8_BF16, FP8_FP16 or FP8_FP32
    int vec;                        // rows of c (and of the residual) start on four elements
    float minus_alpha_log2e, limit, shift;      // gated activation
    uint8_t *h;                     // gated: E4M3 [M, F]
    float *h_scale;                 // gated: [M, NB]
    unsigned int *err;
    unsigned long long wait_limit_ns;
};

// The same products for up to FP8_FEW rows (fp8_few.cu), as long as its CTAs are all there at once; beyond that the
// persistent kernel is as good or better, but for one to four rows and a long K, where it is up to a sixth behind.  Here |
// there, us: 1 x 5120 x 2880 4.6 | 11, 16 x 5120 x 2880 8.9 | 9.2, 16 x 40000 x 2880 31.0 | 29.7, 8 x 40000 x 528 13.8 |
// 10.6, 1 x 40000 x 528 13.2 | 10.3, 8 x 201088 x 2880 127 | 122, but 1 x 40000 x 2880 25.2 | 29.5, 4 x 100000 x 2880
// 60.9 | 65.6; gated 16 x 2880 x 2880 9.0 | 9.5, 16 x 11520 x 2880 24.6 | 21.4, but 1 x 20000 x 2880 36.3 | 39.2.
constexpr int FP8_FEW = 16;
constexpr int FP8_FEW_CTAS = 3;         // CTAs (16 columns each) to an SM, at most
inline bool fp8_few(int M, int N, int gated, int num_sms) {
    const long long ctas = gated ? fp8_blocks(N) * 8LL : (N + 15LL) / 16;
    return M <= FP8_FEW && ctas <= (long long)(gated ? 2 : FP8_FEW_CTAS) * num_sms;
}
struct Fp8FewParams {
    const uint8_t *a, *b;           // E4M3 [M, K] (rows lda bytes apart), [N, K] (gated [2, F, K])
    const float *a_scale, *b_scale;
    const uint16_t *bias;
    const void *residual;
    void *c;
    uint8_t *h;
    float *h_scale;
    long long lda, ldr, ldc;
    int M, N, K, KB, NB, type;
    float minus_alpha_log2e, limit, shift;
};

// One launch: BN columns of accumulators per CTA (gated: BN / 2 gate and BN / 2 linear columns), CTAS CTAs
// per MMA, K split over `split` CTAs of a cluster.
struct Fp8Plan {
    int bn, ctas, split;
    int a_rows, n_stages;
    int m_tiles, tiles, grid;
};

// The shortest limit of a wait.  A CTA that gives up waits as long again for its copies and MMAs in flight before it
// frees TMEM and leaves; they take microseconds, so from here on they have landed by then, its pair's too.
constexpr unsigned long long FP8_WAIT_LIMIT_MIN_NS = 1000000;

constexpr int FP8_SIZE_MAX = 1 << 30;   // rows, columns and K, at most
constexpr int FP8_BM = 128;             // rows of A per CTA (TMEM lanes)
constexpr int FP8_KS = 128;             // K elements per stage: one scale block
constexpr int FP8_STAGES_MAX = 16;
constexpr int FP8_SPLIT_MAX = 8;        // CTAs of a cluster
constexpr int FP8_WGS = 2;              // epilogue warpgroups
constexpr int FP8_THREADS = FP8_WGS * 128 + 128;
// A CTA has its SM alone, with all of its tensor memory: whatever its rings need, it takes all of the shared
// memory, so no other of these CTAs (nor the expert GEMM's) can lie beside it and wait for TMEM columns
// while a peer in its cluster waits for it.
constexpr int FP8_SMEM_SM = 227 * 1024;
constexpr int FP8_TMEM_COLS = 512;

__host__ __device__ constexpr int fp8_bufs(int bn) { return FP8_TMEM_COLS / bn; }       // accumulators of BN columns
__host__ __device__ constexpr int fp8_split(int bn) { return bn == 256 ? 2 : 1; }       // parts that one fills and frees in
// The scales on their way to the epilogue: a ring of chunks of four K blocks, in a chunk a row's four
// scales side by side, for the CTA's 128 rows and two of the weight's blocks (each warpgroup's, or the
// gate's and the linear part's).
constexpr int FP8_CHUNK = 4, FP8_CHUNKS = 4;
constexpr int FP8_CHUNK_BYTES = (FP8_BM + 2) * FP8_CHUNK * 4;
constexpr int FP8_SCALE_BYTES = FP8_CHUNKS * FP8_CHUNK_BYTES;
// An epilogue warp's staging tile: 32 rows of 32 sums, rows 16 bytes further apart than they are long
// (gated: the biases of its 128 columns; a split tile: none).
constexpr int FP8_TILE_COLS = 32;
__host__ __device__ constexpr int fp8_tile_bytes(int gated) { return gated ? 128 * 4 : 32 * (FP8_TILE_COLS + 4) * 4; }

// Offsets from a 1024-aligned base: the A ring, the B ring, each epilogue warp's staging tile, the
// scales, the barriers, the row maxima that warps exchange, the TMEM base and abort flag.
struct Fp8Smem {
    int a_stage, b_stage, b_off, stage_off, scale_off, bar_off, ex_off, misc_off, total;
};

__host__ __device__ inline Fp8Smem fp8_smem(int bn, int ctas, int gated, int split, int a_rows, int n_stages) {
    Fp8Smem s;
    s.a_stage = a_rows * FP8_KS;
    s.b_stage = bn / ctas * FP8_KS;
    s.b_off = n_stages * s.a_stage;
    s.stage_off = s.b_off + n_stages * s.b_stage;
    s.scale_off = s.stage_off + (split ? 0 : FP8_WGS * 4 * fp8_tile_bytes(gated));
    s.bar_off = s.scale_off + FP8_SCALE_BYTES;
    // full and empty per stage, full and empty per accumulator (part), drain [2 MMA warps], exchange
    // [4 quarters][2 parities], full and empty per chunk of scales
    s.ex_off = s.bar_off + (2 * n_stages + 2 * fp8_split(bn) * fp8_bufs(bn) + 2 + 8 + 2 * FP8_CHUNKS) * 8;
    s.ex_off = (s.ex_off + 15) / 16 * 16;
    s.misc_off = s.ex_off + (gated ? 2 * FP8_WGS * FP8_BM * 4 : 0);
    s.total = s.misc_off + 16;
    // the MMA reads 128 rows of A from a stage's start, also where a stage holds fewer; a CTA that shares
    // its tile's K puts its sums over the rings
    const int a_end = (n_stages - 1) * s.a_stage + FP8_BM * FP8_KS, sums = split ? a_rows * (bn + 4) * 4 : 0;
    if (s.total < a_end) s.total = a_end;
    if (s.total < sums) s.total = sums;
    s.total += 1024;
    return s;
}

// The form, ring depth and grid of one product; clusters[n]: how many clusters of n CTAs the device holds at
// once.  Returns false when the sizes are out of range.
inline bool fp8_plan(int M, int N, int K, int gated, int num_sms, const int *clusters, Fp8Plan *pl) {
    if (M > FP8_SIZE_MAX || N > FP8_SIZE_MAX || K > FP8_SIZE_MAX) return false;
    long long rows = (M + FP8_BM - 1) / FP8_BM;
    const long long cols = fp8_blocks(N), wide = gated ? cols : (N + 255) / 256;     // columns in 128s, in pairs' tiles
    // The form that should take least: us per K block (of hand-overs, mostly) and per tile, as fitted to measured times
    // (the gated forms' within a seventh).  Either side of its choices, us: 1024 x 5120 x 2880 single 27.3, pairs
    // 30.4; 1500 x 5120 x 2880 37.1, 32.8; 8192 x 5120 x 2880 180, 155; 256 x 2880 x 6144 split 13.6, pairs 27.2;
    // 24 x 5120 x 11520 split 16.3, single 29.3.  Gated, split | pairs (weights from memory): 256 x 2880 x 512 10.7 |
    // 6.8, 333 x 1360 x 1552 12.3 | 11.2, 256 x 2880 x 2880 17.8 | 16.4, 512 x 2880 x 2880 26.7 | 17.4, 260 x 1360 x
    // 2880 14.0 | 15.9, 256 x 2880 x 6144 25.8 | 28.0; 64 x 2880 x 2880 split 10.4, not split 20.9.
    const int kb = fp8_blocks(K);
    auto waves = [](long long tiles, int at_once) { return at_once > 0 ? (double)((tiles + at_once - 1) / at_once) : 1e30; };
    const long long pair_tiles = (rows + 1) / 2 * wide, one_tiles = rows * cols;
    int n = 1;                                  // CTAs to split K over
    while (n < FP8_SPLIT_MAX && n < kb && one_tiles <= clusters[n + 1]) ++n;
    const double pair = waves(pair_tiles, num_sms / 2) * (gated ? 0.48 * kb + 4.7 : 0.55 * kb + 3.0);
    const double one = gated   ? waves(one_tiles, clusters[n]) * (0.7 * ((kb + n - 1) / n) + 9.5)
                       : n > 1 ? waves(one_tiles, clusters[n]) * (0.34 * ((kb + n - 1) / n) + 4.0)
                               : waves(one_tiles, num_sms) * (0.34 * kb + 2.0);
    pl->bn = gated ? 256 : 128;
    pl->ctas = 1;
    pl->split = n;
    if (M > FP8_BM && pair < one) {
        pl->bn = 256;
        pl->ctas = 2;
        pl->split = 1;
        rows = (rows + 1) / 2;
    }
    const long long tiles = pl->ctas == 2 ? pair_tiles : one_tiles;
    if (tiles > (1 << 27)) return false;
    const int split = pl->split > 1 || (gated && pl->ctas == 1);      // the split form (also with one CTA)
    pl->m_tiles = (int)rows;
    pl->tiles = (int)tiles;
    pl->a_rows = M < FP8_BM ? (M + 7) / 8 * 8 : FP8_BM;
    // Where the two MMA warps take every other K block, an even number of stages keeps a stage with one
    // of them: a warp that met only every other use of a barrier could take a phase for the one before
    // or after it (a wait tells them apart by parity alone).
    const int by = fp8_split(pl->bn) == 2 ? 1 : 2;
    int ns = FP8_STAGES_MAX;
    while (ns > 2 && fp8_smem(pl->bn, pl->ctas, gated, split, pl->a_rows, ns).total > FP8_SMEM_SM) ns -= by;
    if (fp8_smem(pl->bn, pl->ctas, gated, split, pl->a_rows, ns).total > FP8_SMEM_SM) return false;
    pl->n_stages = ns;
    if (split) {
        pl->grid = (int)tiles * pl->split;      // a cluster per tile
    } else {
        const long long most = num_sms / pl->ctas;
        pl->grid = (int)(tiles < most ? tiles : most) * pl->ctas;
    }
    return true;
}

}  // namespace moe
