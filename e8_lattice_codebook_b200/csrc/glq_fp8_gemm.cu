// glq_fp8_gemm.cu -- the 8-bit float linear layer for many tokens on the 5th
// generation tensor cores:
//     y[b][r] = sum_kb (s[kb][b] ws[r/128][kb]) sum_{k in kb} q[b][k] w[r][k].
//
// The scales change every 128 columns, so the tensor core can only add up one
// K block at a time; its result is scaled and added in registers.  What bounds
// the kernel is the MMA, if that second sum keeps up:
//   * tiles of 256 tokens x 256 weight rows per cluster of two CTAs
//     (cta_group::2, M = 256: 128 tokens per CTA, each CTA holding
//     half of the weight rows' operand), so that a CTA copies 32 KB for the
//     512 cycles of a K block's MMAs;
//   * tokens are the M side: a thread of the drain owns one token and 128
//     columns of one 128-row weight block, so that a K block has one scale per
//     thread, and the sums stay in its registers (128 of them) until the tile
//     ends: 128 fused multiply-adds per thread and K block;
//   * the two 128-row blocks of a tile are MMAs of their own (N = 128), each
//     with two accumulators of 128 TMEM columns and its own four drain warps:
//     from an accumulator's MMAs to its reuse pass the MMA's latency, the read
//     and an arrival from the other CTA, and the more pieces wait for that
//     apart, the more of them the MMAs cover.
// Warps: 0 copies (TMA of the e4m3 rows and of the laid-out weight tiles, both
// completing on the first CTA's barrier), 1 MMA (first CTA) and TMEM, 4-11
// drain.  Every wait is bounded; a timeout sets the layer's error word.
// Measured: 4096x14336, 2048 rounded tokens 138 to 141 us = 1.71 to 1.74
// PFLOP/s; a K block takes about 1190 cycles, and the tensor pipe is busy 45 %
// of them.  Cycle stamps (in a build in which the stamps themselves bring it to
// 1020): per K block the MMA thread waits 360 cycles for accumulators and 160 for
// copies, a drain warp 330 for its accumulator; its two reads take 180 and 110,
// products, scales and arrival the other 390.  So neither side is busy all the
// time: an accumulator goes round MMA, commit, reads, products of the first
// half and the arrival in the first CTA, in two K blocks' time, there being two.
#include "glq_fp8.cuh"
#include "glq_kernels.cuh"

namespace glq {

namespace {

using namespace fp8;

constexpr int TOK = 128;                  // tokens per CTA
constexpr int COLS = 128;                 // weight rows of one of a tile's two MMAs
constexpr int A_BYTES = TOK * 128, B_BYTES = GLQ_FP8_TILE_BYTES / 2;  // half of each block's rows per CTA
constexpr int STAGE = A_BYTES + 2 * B_BYTES;  // 32 KB
constexpr int STAGES = 5;
constexpr int DRAIN_WARPS = 8;
// warps 0-3: copies, MMA, two idle; 4-11: drain.  Registers move between the
// warpgroups: 384 threads start with 168 each; the first warpgroup keeps 56,
// the two that drain hold 224 (128 x 56 + 256 x 224 = 384 x 168).
constexpr int DRAIN_WARP0 = 4;
constexpr int THREADS = (DRAIN_WARP0 + DRAIN_WARPS) * 32;
// y leaves by TMA from shared memory, a drain warp's 32 tokens in chunks of 128
// bytes of columns, two at a time (stores from the threads, which own a token
// each, would touch 32 rows per instruction: a quarter of the kernel's time at
// 32 K blocks).
constexpr int CHUNK = 32 * 128;
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE + (size_t)DRAIN_WARPS * 2 * CHUNK;

// Chunk (c0, c1) of y from shared memory; rows and columns past y are left out.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(smem_addr(src)), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
    if (dtype == 1) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ void mma2_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// arrive on the barrier at the same place in the pair's first CTA
__device__ __forceinline__ void arrive_first(uint64_t *bar) {
    asm volatile(
        "{\n .reg .b32 ra;\n mapa.shared::cluster.u32 ra, %0, 0;\n"
        " mbarrier.arrive.shared::cluster.b64 _, [ra];\n}\n" ::"r"(smem_addr(bar))
        : "memory");
}
__global__ void __launch_bounds__(THREADS, 1) fp8_gemm_kernel(const __grid_constant__ CUtensorMap qmap,
                                                              const __grid_constant__ CUtensorMap wmap,
                                                              const __grid_constant__ CUtensorMap ymap,
                                                              Fp8GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    // (first CTA) full: both CTAs' copies have landed; acc_empty: both CTAs have
    // drained the accumulator.  (both) empty: the MMAs of the stage have
    // finished; acc_full: the accumulator holds a K block.
    __shared__ __align__(8) uint64_t full[STAGES], empty[STAGES], acc_full[4], acc_empty[4], mma_done;  // accumulator 2 half + turn
    __shared__ uint32_t tmem_holder;
    __shared__ volatile int abort_flag;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = sm100::cluster_ctarank();
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 4; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], DRAIN_WARPS);  // four of each CTA
        }
        mbar_init(&mma_done, 1);
        abort_flag = 0;
        sm100::prefetch_tensormap(&qmap);
        sm100::prefetch_tensormap(&wmap);
        sm100::prefetch_tensormap(&ymap);
    }
    if (warp == 1) {
        sm100::tmem_alloc2(&tmem_holder, 512);
        sm100::tmem_relinquish2();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::cluster_sync_all();  // barriers of both CTAs are set up
    sm100::tc_fence_after();
    const uint32_t tmem = tmem_holder;
    pdl_launch_dependents();

    // CTA scope: what the barriers order is copies, MMAs and TMEM loads (the
    // tcgen05 fences), no stores of another CTA.  Cluster-scope acquires, one
    // per drain warp and K block, cost more than the K block's MMAs; on the MMA
    // thread's waits for accumulators alone 4096x14336 with 2048 tokens took 257
    // us instead of 140.
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_bounded(bar, parity, &abort_flag, p.err); };
    const int KB = p.KB, items = p.tiles * p.ksplit;
    // an item: a tile's token and weight-row place and its share of the K blocks
    struct Item {
        int ct, tt, ks, kb0, kb1;
    };
    auto item = [&](int i) {
        Item w;
        const int tile = i / p.ksplit;
        w.ks = i - tile * p.ksplit;
        w.ct = tile / p.TT;
        w.tt = tile - w.ct * p.TT;
        w.kb0 = w.ks * KB / p.ksplit;
        w.kb1 = (w.ks + 1) * KB / p.ksplit;
        return w;
    };

    if (warp < DRAIN_WARP0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
        if (elect_one()) {
            pdl_wait();  // the rounded tokens come from the kernel before
            uint32_t s = 0, par = 1, loaded = 0;
            bool ok = true;
            for (int it = cid; it < items && ok; it += ncl) {
                const Item w = item(it);
                const int ct = w.ct, tok0 = w.tt * (2 * TOK) + (int)rank * TOK;
                const bool both = 2 * ct + 1 < p.RT;             // the second block of weight rows exists
                const uint32_t bytes = 2 * (A_BYTES + (both ? 2 : 1) * B_BYTES);
                int wrow = (2 * ct * KB + w.kb0) * 128 + (int)rank * 64;  // this CTA's 64 rows of a block
                for (int kb = w.kb0; kb < w.kb1; ++kb, wrow += 128) {
                    if (!(ok = wait(&empty[s], par))) break;
                    uint8_t *st = smem + s * STAGE;
                    if (rank == 0) mbar_expect_tx(&full[s], bytes);
                    sm100::tma_load_2d_pair(st, &qmap, &full[s], kb * GLQ_FP8_BLOCK, tok0);
                    sm100::tma_load_2d_pair(st + A_BYTES, &wmap, &full[s], 0, wrow);
                    if (both) sm100::tma_load_2d_pair(st + A_BYTES + B_BYTES, &wmap, &full[s], 0, wrow + KB * 128);
                    ++loaded;
                    if (++s == STAGES) s = 0, par ^= 1;
                }
            }
            if (abort_flag && rank == 0)  // let the copies in flight land before the CTA exits
                for (uint32_t i = loaded > (uint32_t)STAGES ? loaded - STAGES : 0; i < loaded; ++i)
                    sm100::mbar_wait(&full[i % STAGES], (i / STAGES) & 1, WAIT_CYCLES / 64);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            pdl_wait();  // a bounded wait must not count the time of the kernel before
            if (rank == 0) {
                const uint32_t idesc = idesc_e4m3_f32(2 * TOK, COLS);
                uint32_t s = 0, par = 0, a = 0, apar = 1;
                bool ok = true;
                for (int it = cid; it < items && ok; it += ncl) {
                    const Item w = item(it);
                    for (int kb = w.kb0; kb < w.kb1; ++kb) {
                        if (!(ok = wait(&full[s], par))) break;
                        uint8_t *st = smem + s * STAGE;
                        const uint64_t ad = sm100::smem_desc_sw128(st);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!(ok = wait(&acc_empty[2 * h + a], apar))) break;
                            sm100::tc_fence_after();
                            const uint64_t bd = sm100::smem_desc_sw128(st + A_BYTES + h * B_BYTES);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma2_f8_ss(tmem + (2 * h + a) * COLS, ad + 2 * kk, bd + 2 * kk, idesc, kk);
                            sm100::mma2_commit_both(&acc_full[2 * h + a]);
                        }
                        if (!ok) break;
                        sm100::mma2_commit_both(&empty[s]);
                        if (++s == STAGES) s = 0, par ^= 1;
                        a ^= 1;
                        if (a == 0) apar ^= 1;
                    }
                }
                sm100::mma2_commit_both(&mma_done);  // every MMA of the pair has completed
            }
            sm100::mbar_wait(&mma_done, 0, WAIT_CYCLES);
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ---------------- drain ----------------
        pdl_wait();  // scales of the tokens; y may still be in use by the kernel before
        const int quadrant = warp & 3, half = (warp - DRAIN_WARP0) >> 2;
        const uint32_t t0 = tmem + ((uint32_t)(32 * quadrant) << 16) + half * 2 * COLS;
        uint32_t a = 0, apar = 0;
        bool ok = true;
        for (int it = cid; it < items && ok; it += ncl) {
            const Item w = item(it);
            const int token = w.tt * (2 * TOK) + (int)rank * TOK + 32 * quadrant + lane;
            const int rt = 2 * w.ct + half;
            const float *s = p.s + min(token, p.B - 1);
            const float *ws = p.ws + (int64_t)min(rt, p.RT - 1) * KB;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            // Four blocks' scales are loaded while the four before them are used,
            // and multiplied after: a product of values still on their way would
            // stop the warp.
            float f[4], rs[4], rw[4];
            auto fetch = [&](int kb0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int kb = min(kb0 + i, w.kb1 - 1);
                    rs[i] = __ldcg(s + (int64_t)kb * p.s_ld);
                    rw[i] = __ldg(ws + kb);
                }
            };
            fetch(w.kb0);
            for (int kb0 = w.kb0; kb0 < w.kb1 && ok; kb0 += 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = rs[i] * rw[i];
                fetch(kb0 + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kb0 + i >= w.kb1) break;
                    if (lane == 0) ok = wait(&acc_full[2 * half + a], apar);
                    __syncwarp();
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    sm100::tc_fence_after();
                    // a read takes about 190 cycles beside the MMAs, whatever its
                    // size: 64 columns at a time
#pragma unroll
                    for (int c = 0; c < 128; c += 64) {
                        uint32_t d[2][32];
                        sm100::tmem_ld32(t0 + a * COLS + c, d[0]);
                        sm100::tmem_ld32(t0 + a * COLS + c + 32, d[1]);
                        sm100::tmem_wait_ld();
                        if (c == 64) {  // all read: the MMAs of the block after next may start
                            sm100::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_first(&acc_empty[2 * half + a]);
                        }
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            acc[c + j] = fmaf(__uint_as_float(d[j >> 5][j & 31]), f[i], acc[c + j]);
                    }
                    a ^= 1;
                    if (a == 0) apar ^= 1;
                }
            }
            if (!ok) break;
            const int row0 = rt * 128, tok0 = token - lane;
            uint8_t *out = smem + STAGES * STAGE + (warp - DRAIN_WARP0) * 2 * CHUNK + lane * 128;
            // 64 columns of a 16-bit y, or 32 of fp32, to a chunk
            auto put = [&](auto chunk_words, int c, int slot) {
                uint8_t *row = out + slot * CHUNK;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(row + ((j ^ (lane & 7)) << 4)) = chunk_words(c, j);
            };
            auto send = [&](int col, int slot) {
                if (col < p.m && tok0 < p.B)
                    sm100::fence_proxy_async_smem(), __syncwarp();
                if (lane == 0 && col < p.m && tok0 < p.B) {
                    tma_store_2d(&ymap, out - lane * 128 + slot * CHUNK, col, w.ks * p.part_rows + tok0);
                    bulk_commit();
                }
            };
            if (lane == 0) bulk_wait_read();  // the last tile's chunks have been read
            __syncwarp();
            if (p.y_dtype == 2) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c == 2) {
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                    }
                    put([&](int k, int j) {
                        const float *v = acc + k * 32 + j * 4;
                        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                          __float_as_uint(v[3]));
                    }, c, c & 1);
                    send(row0 + c * 32, c & 1);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    put([&](int k, int j) {
                        const float *v = acc + k * 64 + j * 8;
                        return make_uint4(pack2(v[0], v[1], p.y_dtype), pack2(v[2], v[3], p.y_dtype),
                                          pack2(v[4], v[5], p.y_dtype), pack2(v[6], v[7], p.y_dtype));
                    }, c, c);
                    send(row0 + c * 64, c);
                }
            }
        }
        if (lane == 0) bulk_wait_all();  // before the CTA's shared memory is given back
    }
    __syncwarp();
    sm100::tc_fence_before();
    __syncthreads();
    sm100::cluster_sync_all();  // no CTA leaves while its pair may still touch its memory
    if (warp == 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc2(tmem, 512);
    }
}

// y = the parts of a split K, added in order; four columns a thread
__global__ void __launch_bounds__(256) fp8_sum_parts_kernel(const float *part, int64_t part_stride, int parts, void *y,
                                                            int y_dtype, int64_t quads) {
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
        float4 sum = __ldcg(reinterpret_cast<const float4 *>(part) + i);
#pragma unroll 4
        for (int k = 1; k < parts; ++k) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + k * part_stride) + i);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        store_y4(y, y_dtype, i * 4, sum);
    }
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const CUtensorMap &qmap, const CUtensorMap &wmap,
                            const CUtensorMap &ymap, int num_sms, cudaStream_t s, bool pdl) {
    const void *fn = (const void *)fp8_gemm_kernel;
    static std::atomic<uint64_t> configured;
    const cudaError_t e = once_per_device(configured, [fn] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    });
    if (e != cudaSuccess) return e;
    Fp8GemmParams q = p;
    CUtensorMap a = qmap, b = wmap, c = ymap;
    void *args[] = {&a, &b, &c, &q};
    const int items = p.tiles * p.ksplit, clusters = items < num_sms / 2 ? items : num_sms / 2;
    return launch_ex(fn, dim3(2 * clusters), dim3(THREADS), SMEM, s, pdl, args, 2);
}

int plan_fp8_gemm(int64_t tiles, int KB, int64_t B, int64_t m, int num_sms) {
    // A pair of CTAs takes a K block in 0.62 us; an item's start and end cost
    // about 2 us.  Splitting K over more pairs costs the parts' trip through L2
    // (8 bytes each at 5 TB/s) and a launch.  (4096 x 14336, 128 tokens: 16
    // tiles of 112 blocks take 71 us on 16 of 74 pairs, 25 us split in four.)
    const int pairs = num_sms / 2;
    int best = 1;
    double best_t = 1e30;
    for (int s = 1; s <= 8 && s * 4 <= KB + 3; ++s) {
        const double waves = (double)((tiles * s + pairs - 1) / pairs);
        const double t = waves * ((KB + s - 1) / s * 0.62 + 2.0) + (s > 1 ? 3.0 + (double)s * B * m * 8 / 5e6 : 0.0);
        if (t < best_t * 0.95) {
            best_t = t;
            best = s;
        }
    }
    return best;
}

cudaError_t launch_fp8_sum_parts(const float *part, int64_t part_stride, int parts, void *y, int y_dtype, int64_t count,
                                 cudaStream_t s, bool pdl) {
    int64_t quads = count / 4;
    void *args[] = {&part, &part_stride, &parts, &y, &y_dtype, &quads};
    const int64_t blocks = (quads + 255) / 256;
    return launch_ex((const void *)fp8_sum_parts_kernel, dim3((unsigned)(blocks < 148 * 8 ? blocks : 148 * 8)), dim3(256), 0,
                     s, pdl, args);
}

}  // namespace glq
