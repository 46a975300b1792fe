// glq_fp8_gemm.cu -- the 8-bit float linear layer for many tokens on the 5th
// generation tensor cores:
//     y[b][r] = sum_kb (s[kb][b] ws[r/128][kb]) sum_{k in kb} q[b][k] w[r][k].
//
// The scales change every 128 columns, so the tensor core can only add up one
// K block at a time; its result is scaled and added in registers.  What bounds
// the kernel is the MMA, if that second sum keeps up:
//   * tiles of 256 tokens x 256 weight rows per cluster of two CTAs
//     (cta_group::2, M = 256, N = 256: 128 tokens per CTA, each CTA holding
//     half of the weight rows' operand), so that a CTA copies 32 KB for the
//     512 cycles of a K block's MMAs;
//   * tokens are the M side: a thread of the drain owns one token and 128
//     columns of one 128-row weight block, so that a K block has one scale per
//     thread, and the sums stay in its registers (128 of them) until the tile
//     ends: 128 fused multiply-adds per thread and K block;
//   * two accumulators of 256 TMEM columns: the MMAs of one K block run while
//     the other one is drained.
// Warps: 0 copies (TMA of the e4m3 rows and of the laid-out weight tiles, both
// completing on the first CTA's barrier), 1 MMA (first CTA) and TMEM, 4-11
// drain.  Every wait is bounded; a timeout sets the layer's error word.
#include "glq_fp8.cuh"
#include "glq_kernels.cuh"

namespace glq {

namespace {

using namespace fp8;

constexpr int TOK = 128;                  // tokens per CTA
constexpr int COLS = 256;                 // weight rows of a tile
constexpr int A_BYTES = TOK * 128, B_BYTES = GLQ_FP8_TILE_BYTES;
constexpr int STAGE = A_BYTES + B_BYTES;  // 32 KB
constexpr int STAGES = 6;
constexpr int DRAIN_WARPS = 8;
// warps 0-3: copies, MMA, two idle; 4-11: drain.  Registers move between the
// warpgroups: 384 threads start with 168 each; the first warpgroup keeps 56,
// the two that drain hold 224 (128 x 56 + 256 x 224 = 384 x 168).
constexpr int DRAIN_WARP0 = 4;
constexpr int THREADS = (DRAIN_WARP0 + DRAIN_WARPS) * 32;
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE;

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
                                                              Fp8GemmParams p) {
    extern __shared__ uint8_t smem_raw[];
    // (first CTA) full: both CTAs' copies have landed; acc_empty: both CTAs have
    // drained the accumulator.  (both) empty: the MMAs of the stage have
    // finished; acc_full: the accumulator holds a K block.
    __shared__ __align__(8) uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], mma_done;
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
        for (int a = 0; a < 2; ++a) {
            mbar_init(&acc_full[a], 1);
            mbar_init(&acc_empty[a], 2 * DRAIN_WARPS);
        }
        mbar_init(&mma_done, 1);
        abort_flag = 0;
        sm100::prefetch_tensormap(&qmap);
        sm100::prefetch_tensormap(&wmap);
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

    auto fail = [&]() {
        atomicOr(p.err, GLQ_DEVERR_TIMEOUT);
        abort_flag = 1;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        // CTA scope: what the barriers order is copies, MMAs and TMEM loads (the
        // tcgen05 fences), no stores of another CTA.  Cluster-scope acquires, one
        // per drain warp and K block, cost more than the K block's MMAs.
        if (sm100::mbar_try(bar, parity)) return true;
        if (abort_flag) return false;
        if (sm100::mbar_wait(bar, parity, WAIT_CYCLES)) return true;
        fail();
        return false;
    };
    const int KB = p.KB;

    if (warp < DRAIN_WARP0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
        if (elect_one()) {
            pdl_wait();  // the rounded tokens come from the kernel before
            uint32_t s = 0, par = 1, loaded = 0;
            bool ok = true;
            for (int tile = cid; tile < p.tiles && ok; tile += ncl) {
                const int ct = tile / p.TT, tt = tile - ct * p.TT;
                const int tok0 = tt * (2 * TOK) + (int)rank * TOK, rt = 2 * ct + (int)rank;
                const bool mine = rt < p.RT;                     // this CTA's weight rows exist
                const uint32_t bytes = 2 * A_BYTES + (2 * ct + 1 < p.RT ? 2 : 1) * B_BYTES;
                int wrow = rt * KB * 128;
                for (int kb = 0; kb < KB; ++kb, wrow += 128) {
                    if (!(ok = wait(&empty[s], par))) break;
                    uint8_t *st = smem + s * STAGE;
                    if (rank == 0) mbar_expect_tx(&full[s], bytes);
                    sm100::tma_load_2d_pair(st, &qmap, &full[s], kb * GLQ_FP8_BLOCK, tok0);
                    if (mine) sm100::tma_load_2d_pair(st + A_BYTES, &wmap, &full[s], 0, wrow);
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
            if (rank == 0) {
                const uint32_t idesc = idesc_e4m3_f32(2 * TOK, COLS);
                uint32_t s = 0, par = 0, a = 0, apar = 1;
                bool ok = true;
                for (int tile = cid; tile < p.tiles && ok; tile += ncl) {
                    for (int kb = 0; kb < KB; ++kb) {
                        if (!(ok = wait(&acc_empty[a], apar) && wait(&full[s], par))) break;
                        sm100::tc_fence_after();
                        uint8_t *st = smem + s * STAGE;
                        const uint64_t ad = sm100::smem_desc_sw128(st), bd = sm100::smem_desc_sw128(st + A_BYTES);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) mma2_f8_ss(tmem + a * COLS, ad + 2 * kk, bd + 2 * kk, idesc, kk);
                        sm100::mma2_commit_both(&acc_full[a]);
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
        const uint32_t t0 = tmem + ((uint32_t)(32 * quadrant) << 16) + half * 128;
        uint32_t a = 0, apar = 0;
        bool ok = true;
        for (int tile = cid; tile < p.tiles && ok; tile += ncl) {
            const int ct = tile / p.TT, tt = tile - ct * p.TT;
            const int token = tt * (2 * TOK) + (int)rank * TOK + 32 * quadrant + lane;
            const int rt = 2 * ct + half;
            const float *s = p.s + min(token, p.B - 1);
            const float *ws = p.ws + (int64_t)min(rt, p.RT - 1) * KB;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            // scales four blocks ahead: a load takes longer than a block's MMAs
            float next[4], now[4];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    next[i] = kb + i < KB ? __ldg(s + (int64_t)(kb + i) * p.s_ld) * __ldg(ws + kb + i) : 0.f;
            };
            fetch(0);
            for (int kb0 = 0; kb0 < KB && ok; kb0 += 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = next[i];
                fetch(kb0 + 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (kb0 + i >= KB) break;
                    if (lane == 0) ok = wait(&acc_full[a], apar);
                    __syncwarp();
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    sm100::tc_fence_after();
                    const float f = now[i];
                    uint32_t d[2][32];
                    sm100::tmem_ld32(t0 + a * COLS, d[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        sm100::tmem_wait_ld();
                        if (c < 3) {
                            sm100::tmem_ld32(t0 + a * COLS + (c + 1) * 32, d[(c + 1) & 1]);
                        } else {  // all read: the MMAs of the block after next may start
                            sm100::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive_first(&acc_empty[a]);
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            acc[c * 32 + j] = fmaf(__uint_as_float(d[c & 1][j]), f, acc[c * 32 + j]);
                    }
                    a ^= 1;
                    if (a == 0) apar ^= 1;
                }
            }
            if (!ok) break;
            if (token < p.B && rt < p.RT) {
                const int row0 = rt * 128;
#pragma unroll
                for (int j = 0; j < 128; j += 4)
                    if (row0 + j < p.m)  // m is a multiple of 8: four columns are in or out together
                        store_y4(p.y, p.y_dtype, (int64_t)token * p.m + row0 + j,
                                 make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]));
            }
        }
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

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8GemmParams &p, const CUtensorMap &qmap, const CUtensorMap &wmap, int num_sms,
                            cudaStream_t s, bool pdl) {
    const void *fn = (const void *)fp8_gemm_kernel;
    static std::atomic<uint64_t> configured;
    const cudaError_t e = once_per_device(configured, [fn] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    });
    if (e != cudaSuccess) return e;
    Fp8GemmParams q = p;
    CUtensorMap a = qmap, b = wmap;
    void *args[] = {&a, &b, &q};
    const int clusters = p.tiles < num_sms / 2 ? p.tiles : num_sms / 2;
    return launch_ex(fn, dim3(2 * clusters), dim3(THREADS), SMEM, s, pdl, args, 2);
}

}  // namespace glq
