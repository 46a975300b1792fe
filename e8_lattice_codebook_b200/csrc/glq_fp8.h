// glq_fp8.h -- parameters and launchers of the 8-bit float operators: the
// activation quantiser, the linear layer with e4m3 weights and one fp32
// scale per 128 x 128 block, and the mixture-of-experts layer built on them.
//
// Device layout of a weight matrix [rows][cols] (rows on the MMA's M side):
// tiles of 128 rows x 128 columns, 16 KB each and contiguous, tile (rt, kb)
// at ((rt * KB) + kb) * 16 KB with KB = ceil(cols / 128).  Inside a tile a
// row is 128 bytes and its eight 16-byte chunks are stored at chunk ^ (row &
// 7): the 128-byte swizzle of the tensor core's K-major operand.  One bulk
// copy of 16 KB therefore brings a ready operand tile, without a tensor map,
// from one contiguous DRAM range.  Rows and columns past the matrix hold 0.
// The scales are [ceil(rows / 128)][KB] fp32.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#define GLQ_FP8_BLOCK 128
#define GLQ_FP8_TILE_BYTES 16384
#define GLQ_FP8_MAX_DIM (1 << 20)

namespace glq {

// x [B][n] (dtype 0 f16, 1 bf16, 2 f32) -> q [B][KB * 128] e4m3, s [KB][B]
struct Fp8QuantParams {
    const void *x;
    uint8_t *q;
    float *s;
    int64_t B;
    int n, KB;
};
cudaError_t launch_fp8_quantize(const Fp8QuantParams &p, int dtype, cudaStream_t s, bool pdl);

// rows x cols e4m3 at row distance ld (bytes, multiple of 8, src 8-byte
// aligned) into tiles; tile row r goes to dst tile row r * rt_step + rt_off,
// its scales likewise
struct Fp8PackParams {
    const uint8_t *src;
    const float *src_scale;  // [ceil(rows/128)][KB]
    uint8_t *dst;
    float *dst_scale;
    int64_t ld;
    int rows, cols, KB;
    int rt_step, rt_off;
    // batch of matrices (experts): distances between two of them
    int count;
    int64_t src_stride, src_scale_stride, dst_tiles;
};
cudaError_t launch_fp8_pack(const Fp8PackParams &p, cudaStream_t s);

// w [m][n] fp32 = the values the tiles and scales stand for
cudaError_t launch_fp8_dequant(const uint8_t *tiles, const float *scale, float *w, int m, int n, int KB,
                               cudaStream_t s);

// y [B][m] = x W^T for B <= NT tokens, tiles of 128 rows, clusters of C CTAs
// splitting K
struct Fp8SkinnyParams {
    const uint8_t *w;
    const float *ws;
    const void *x;      // source 0 / 1: f16 / bf16 [B][n], rounded on the way
    const float *s;     // source 2: scales [KB][s_ld] of the rows in qmap
    int64_t s_ld;
    void *y;
    int y_dtype;
    int m, n, B, RT, KB;
    int C;              // CTAs per cluster, 1..8, at most KB
    unsigned *err;
};
constexpr int FP8_ROUND_FEW = 4, FP8_ROUND_MAX = 8;  // most tokens of sources 0 and 1: always, in small layers
// whether the few-token kernel rounds f16 / bf16 activations itself (sources 0
// and 1); else the quantiser runs first
bool fp8_rounds_inside(int64_t B, int64_t tiles, int KB, int num_sms);
// Most tokens of the few-token kernel.  4096x14336 takes 19.5 us at 64 tokens
// (few) and 27.1 at 65 (many), the quantiser included; as two few-token calls of
// 64 and 1, 65 would take 32.
constexpr int FP8_FEW = 64;
int fp8_skinny_tile(int64_t B);  // NT: tokens per tile for a batch of B <= FP8_FEW
// clusters of c = 1..8 CTAs (one per SM) the current device holds at once
cudaError_t fp8_skinny_clusters(int num_sms, int count[9]);
struct Fp8SkinnyPlan {
    int C, clusters;
};
Fp8SkinnyPlan plan_fp8_skinny(int64_t tiles, int KB, int nt, const int clusters[9]);
// qmap: source 2 only, boxes of 128 columns x nt tokens of q, 128-byte swizzle
cudaError_t launch_fp8_skinny(const Fp8SkinnyParams &p, const CUtensorMap &qmap, int source, int nt, int clusters,
                              cudaStream_t s, bool pdl);

// y [B][m] = x W^T for many tokens, tiles of FP8_GEMM_TOK tokens x 256 rows
constexpr int FP8_GEMM_TOK = 256;
struct Fp8GemmParams {
    const float *ws;
    const float *s;     // [KB][s_ld]
    int64_t s_ld;
    int y_dtype;        // of ymap
    int m, B, RT, KB;
    int TT, tiles;      // token tiles; all tiles, token tiles within a column of them
    int ksplit;         // parts of K; with more than one, ymap is the fp32 parts,
    int part_rows;      // this many rows apart
    unsigned *err;
};
// the parts of K for a layer and batch (host only)
int plan_fp8_gemm(int64_t tiles, int KB, int64_t B, int64_t m, int num_sms);
// y (count values, a multiple of 4) = the sum of `parts` arrays part_stride
// floats apart
cudaError_t launch_fp8_sum_parts(const float *part, int64_t part_stride, int parts, void *y, int y_dtype, int64_t count,
                                 cudaStream_t s, bool pdl);
// qmap: boxes of 128 columns x 128 tokens of q, 128-byte swizzle; wmap: the
// laid-out weights as rows of 128 bytes, boxes of 64 rows, no swizzle; ymap:
// boxes of 128 bytes x 32 tokens of y, 128-byte swizzle
cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const CUtensorMap &qmap, const CUtensorMap &wmap,
                            const CUtensorMap &ymap, int num_sms, cudaStream_t s, bool pdl);

// the kernels' bounded wait on a barrier `arrivals` of its two arrivals reach
cudaError_t launch_fp8_wait_selftest(unsigned *err, int arrivals, unsigned long long limit, cudaStream_t s);

// A mixture-of-experts layer (glq_moe.cu) for T <= MOE_MAX_T tokens.  d: width
// of x and y, inter: of an expert; KB1 = ceil(d/128) = DB, IB = ceil(inter/128).
constexpr int MOE_MAX_T = 64, MOE_MAX_E = 512, MOE_MAX_K = 16;
constexpr int MOE_SMEM_LIMIT = 224 * 1024;  // 227 KB less the static arrays
struct MoeParams {
    const void *x;       // [T][d] f16 (x_dtype 0) or bf16 (1)
    const void *logits;  // [T][E], dtype 0 f16, 1 bf16, 2 f32
    void *y;             // [T][d]
    int x_dtype, logits_dtype, y_dtype;
    int T, E, k, d;
    int KB1, IB, DB;
    int scoring, renormalize;  // 0 softmax, 1 sigmoid
    float routed_scale;
    const uint8_t *w13;  // tiles [E][2 IB][KB1]: gate and up row tiles in turn
    const float *s13;    // [E][2 IB][KB1]
    const uint8_t *w2;   // tiles [E][DB][IB]
    const float *s2;     // [E][DB][IB]
    // workspace (nt: moe_tile(T), the most a token tile may hold; rows: the tokens of each expert in use,
    // rounded up to 8, one expert after the other)
    uint8_t *xq;         // [expert in use][KB1][its rows][128]: x^ as operand tiles
    float *xs;           // [KB1][T]
    float *main1;        // [T k][2 IB][128]
    float *spill1;       // [grid][nt][128]
    uint8_t *hq;         // [expert in use][IB][its rows][128]: h^ as operand tiles
    float *hs;           // [expert in use][IB][its rows]
    float *main2;        // [T k][DB][128]
    float *spill2;       // [grid][nt][128]
    uint64_t *bar;       // grid barrier: arrivals so far, a multiple of grid between calls
    unsigned *err;
};
int moe_tile(int T);
// the kernel's grid barrier, all its CTAs arriving or all but one
cudaError_t launch_moe_wait_selftest(uint64_t *bar, unsigned *err, int grid, bool all, unsigned long long limit,
                                     cudaStream_t s);
// cooperative: `grid` CTAs, one per SM
cudaError_t launch_moe(const MoeParams &p, int grid, cudaStream_t s);

}  // namespace glq
