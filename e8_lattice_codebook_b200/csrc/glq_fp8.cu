// glq_fp8.cu -- the activation quantiser, the weight layout and the few-token
// product of the 8-bit float linear layer
//     y[b][r] = sum_kb s[kb][b] ws[r/128][kb] sum_{k in kb} q[b][k] w[r][k]
// (q, w e4m3; s the token's scale of 128-column block kb, ws the weight
// block's).
#include <cmath>
#include <type_traits>

#include "glq_fp8.cuh"
#include "glq_kernels.cuh"

namespace glq {

namespace {

using namespace fp8;

// ---------------------------------------------------------------------------
// Quantiser: reads x once, writes q and s once; bound by HBM, so instructions
// are kept few.  A CTA takes 32 tokens x 2 groups: half a warp per group (8
// values a lane, one or two 16-byte loads), all of a warp's four tokens loaded
// before the first is used.  16-bit magnitudes are compared as they are, two
// tokens to a register; the divisions are made once per token and group, by
// the lane whose turn the token is.  The scales of 32 tokens leave as one
// 128-byte line of the [group][token] array.  2048 x 11008 bf16: 10.8 us =
// 6.3 TB/s; one row of 5120: 1.6 us.
// ---------------------------------------------------------------------------

constexpr int QT = 32, QG = 2, QTHREADS = 256;
constexpr int QPER = QT / (QTHREADS / 32);  // tokens per warp
static_assert(QPER == 4, "a pair of tokens in each of two registers");

// Through L2: the kernel before may still be writing x when this one starts.
// (Volatile, so that a warp's loads stay together in front of the first use:
// left to the compiler a call over 2048 x 11008 took 12.3 us instead of 11.5.)
__device__ __forceinline__ uint4 ld_l2_v4(const void *p) {
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight values of a lane, as loaded.
template <typename T>
struct Eight {
    uint4 w;
    __device__ __forceinline__ void load(const T *p) { w = ld_l2_v4(p); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    // the largest magnitude in each half, as 16-bit patterns
    __device__ __forceinline__ uint32_t top() const {
        constexpr uint32_t M = 0x7FFF7FFFu;
        return __vmaxu2(__vmaxu2(w.x & M, w.y & M), __vmaxu2(w.z & M, w.w & M));
    }
    __device__ __forceinline__ uint2 round(float inv) const {
        const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y), c = unpack2<T>(w.z), d = unpack2<T>(w.w);
        const float v[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
        return make_uint2(e4m3x4(v, inv), e4m3x4(v + 4, inv));
    }
};
template <>
struct Eight<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p) {
        const uint4 a = ld_l2_v4(p), b = ld_l2_v4(p + 4);
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    __device__ __forceinline__ uint2 round(float inv) const { return make_uint2(e4m3x4(v, inv), e4m3x4(v + 4, inv)); }
};

// The bits of the group's largest magnitude (fp32) of token l16 & 3, over the
// 16 lanes of half a warp.
template <typename T>
__device__ __forceinline__ uint32_t half_warp_top(const Eight<T> (&e)[QPER], int l16) {
    uint32_t m[2];  // tokens 0 and 1, 2 and 3
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = e[2 * i].top(), b = e[2 * i + 1].top();
        m[i] = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[i] = __vmaxu2(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
    }
    const uint32_t p = (l16 & 2) ? m[1] : m[0], bits = (l16 & 1) ? p >> 16 : p & 0xFFFFu;
    if constexpr (std::is_same<T, __half>::value) return __float_as_uint(__half2float(__ushort_as_half((unsigned short)bits)));
    else return bits << 16;
}
template <>
__device__ __forceinline__ uint32_t half_warp_top<float>(const Eight<float> (&e)[QPER], int l16) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < QPER; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, mag_bits(e[i].v[j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if ((l16 & 3) == i) mine = m;
    }
    return mine;
}

template <typename T>
__global__ void __launch_bounds__(QTHREADS) fp8_quantize_kernel(Fp8QuantParams p) {
    __shared__ float s_s[QG][QT];
    pdl_launch_dependents();
    pdl_wait();  // x may come from the kernel before
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = lane >> 4, l16 = lane & 15;
    const int64_t t0 = (int64_t)blockIdx.y * QT;
    const int g = blockIdx.x * QG + half;
    const int col = g * GLQ_FP8_BLOCK + l16 * 8;
    Eight<T> e[QPER];
#pragma unroll
    for (int i = 0; i < QPER; ++i) {
        const int64_t t = t0 + warp * QPER + i;
        if (t < p.B && col < p.n) e[i].load(static_cast<const T *>(p.x) + t * p.n + col);
        else e[i].zero();
    }
    const uint32_t top = max(half_warp_top<T>(e, l16), FLOOR_BITS);
    const float inv = group_inv(top);
    if (l16 < QPER) s_s[half][warp * QPER + l16] = group_scale(top);
#pragma unroll
    for (int i = 0; i < QPER; ++i) {
        const int64_t t = t0 + warp * QPER + i;
        const uint2 q = e[i].round(__shfl_sync(0xffffffffu, inv, (lane & 16) + i));
        if (t < p.B && g < p.KB) *reinterpret_cast<uint2 *>(p.q + t * ((int64_t)p.KB * GLQ_FP8_BLOCK) + col) = q;
    }
    __syncthreads();
    if (threadIdx.x < QG * QT) {
        const int gl = threadIdx.x / QT, tl = threadIdx.x % QT;
        const int gg = blockIdx.x * QG + gl;
        if (gg < p.KB && t0 + tl < p.B) p.s[(int64_t)gg * p.B + t0 + tl] = s_s[gl][tl];
    }
}

// ---------------------------------------------------------------------------
// Weight layout (once per layer) and its inverse
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(256) fp8_pack_kernel(Fp8PackParams p) {
    const int rt = blockIdx.y, kb = blockIdx.x;
    for (int mat = blockIdx.z; mat < p.count; mat += gridDim.z) {
        const uint8_t *src = p.src + mat * p.src_stride;
        const int64_t tile = mat * p.dst_tiles + (int64_t)(rt * p.rt_step + p.rt_off) * p.KB + kb;
        uint8_t *dst = p.dst + tile * GLQ_FP8_TILE_BYTES;
        for (int i = threadIdx.x; i < 128 * 16; i += 256) {
            const int r = i >> 4, c8 = i & 15;
            const int row = rt * 128 + r, col = kb * 128 + c8 * 8;
            uint2 v = make_uint2(0, 0);
            if (row < p.rows && col < p.cols) v = *reinterpret_cast<const uint2 *>(src + row * p.ld + col);
            *reinterpret_cast<uint2 *>(dst + sw128(r, c8 >> 1) + (c8 & 1) * 8) = v;
        }
        if (threadIdx.x == 0)
            p.dst_scale[tile] = p.src_scale[mat * p.src_scale_stride + (int64_t)rt * p.KB + kb];
    }
}

__global__ void __launch_bounds__(256) fp8_dequant_kernel(const uint8_t *tiles, const float *scale, float *w, int m,
                                                          int n, int KB) {
    const int rt = blockIdx.y, kb = blockIdx.x;
    const int64_t tile = (int64_t)rt * KB + kb;
    const float sc = scale[tile];
    for (int i = threadIdx.x; i < 128 * 128; i += 256) {
        const int r = i >> 7, c = i & 127;
        const int row = rt * 128 + r, col = kb * 128 + c;
        if (row >= m || col >= n) continue;
        __nv_fp8_e4m3 v;
        v.__x = tiles[tile * GLQ_FP8_TILE_BYTES + sw128(r, c >> 4) + (c & 15)];
        w[(int64_t)row * n + col] = (float)v * sc;
    }
}

// ---------------------------------------------------------------------------
// Few tokens.  Reads every weight once: bound by HBM for small batches
// (32768x5120, 1 token: 26.6 us = 6.3 TB/s).  An
// output tile is 128 weight rows x all tokens; a cluster of C CTAs (one per SM)
// takes tile after tile, each CTA 1 / C of its K blocks, so that few tiles
// still keep most SMs loading.  The parts meet in distributed shared memory:
// group j of four tokens is summed by CTA j mod C of the cluster, in the order
// of the CTAs.
// (Parts through global memory, summed by the CTA that arrives last, cost 3.5
// to 5 us at the end of every call: store, atomic and load each make the trip
// to L2.)
// SOURCE 0 / 1: f16 / bf16 activations of up to ROWS tokens rounded on the way;
// 2: e4m3 rows (by
// TMA: 128 columns x NT tokens, 128-byte swizzle) and their scales.
// ---------------------------------------------------------------------------

template <int NT, int SOURCE, int ROWS = 1>
__global__ void __launch_bounds__(PIPE_THREADS, 1) fp8_skinny_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                     Fp8SkinnyParams p) {
    constexpr bool ROUND = SOURCE != 2;
    constexpr int HALF = NT / 2, STAGES = Pipe<NT>::STAGES, DRAIN = Pipe<NT>::DRAIN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) Pipe<NT> pipe;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t C = p.C, rank = C > 1 ? sm100::cluster_ctarank() : 0;
    const uint32_t NC = gridDim.x / C, tiles = p.RT;
    // this CTA's K blocks of every tile
    const uint32_t k0 = rank * p.KB / C, nk = (rank + 1) * p.KB / C - k0;
    const uint32_t first = blockIdx.x / C;
    const uint32_t nblk = first < tiles ? ((tiles - first - 1) / NC + 1) * nk : 0;

    if (warp == 0) pipe.init(lane, C);
    if (warp == 1) {
        sm100::tmem_alloc(&pipe.tmem, Pipe<NT>::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    if (C > 1) cluster_arrive();  // the wait for the others' barriers is the drain's
    sm100::tc_fence_after();
    pdl_launch_dependents();

    uint32_t it = 0;  // the copy thread: blocks whose copies have been started
    bool copier = false, met = false;  // met: has waited for the cluster's barriers to be set up
    if (warp == 0) {
        if (elect_one()) {
            copier = true;
            Loader<NT> ld(smem);
            uint32_t ahead = 0;
            if constexpr (!ROUND) {
                // weights are constant: the first copies do not wait for the
                // kernel before, which the rounded tokens come from
                ahead = min(nblk, (uint32_t)STAGES);
                for (uint32_t t = first; t < tiles && it < ahead; t += NC) {
                    const uint8_t *w = p.w + ((int64_t)t * p.KB + k0) * GLQ_FP8_TILE_BYTES;
                    for (uint32_t k = 0; k < nk && it < ahead; ++k, ++it, w += GLQ_FP8_TILE_BYTES, ld.next())
                        pipe_load<NT, ROUND>(pipe, ld, w, NT * 128, p.err);
                }
                sm100::prefetch_tensormap(&qmap);
                pdl_wait();
                ld = Loader<NT>(smem);
            }
            uint32_t i = 0;
            bool ok = true;
            for (uint32_t t = first; t < tiles && ok; t += NC) {
                const uint8_t *w = p.w + ((int64_t)t * p.KB + k0) * GLQ_FP8_TILE_BYTES;
                int col = (int)k0 * GLQ_FP8_BLOCK;
                for (uint32_t k = 0; k < nk; ++k, ++i, w += GLQ_FP8_TILE_BYTES, col += GLQ_FP8_BLOCK, ld.next()) {
                    // a stage's second use waits for the tokens of its first, and
                    // a wait must not count the time of the kernel before
                    if (ROUND && i == (uint32_t)STAGES) pdl_wait();
                    if (ROUND || i >= ahead) {
                        ok = pipe_load<NT, ROUND>(pipe, ld, w, ROUND ? 0 : NT * 128, p.err);
                        if (!ok) break;
                        ++it;
                    }
                    if (!ROUND) sm100::tma_load_2d(ld.dst + GLQ_FP8_TILE_BYTES, &qmap, &pipe.full[ld.stage], col, 0);
                }
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            pdl_wait();  // (as above)
            pipe_mma<NT>(pipe, smem, 0, nblk, p.err);
            sm100::mma_commit(&pipe.mma_done);  // every MMA issued has completed
            sm100::mbar_wait(&pipe.mma_done, 0, WAIT_CYCLES);
        }
    } else if (warp < D_WARP0) {
        // the block scales of this CTA come from DRAM, behind the weights in
        // flight: into L2 before those are too many
        for (uint32_t t = first + (warp - X_WARP0) * NC; t < tiles; t += X_WARPS * NC)
            for (uint32_t k = lane * 32; k < nk; k += 32 * 32) prefetch_l2(p.ws + (int64_t)t * p.KB + k0 + k);
        pdl_wait();
        // Everything a block needs from memory is loaded one turn ahead (the
        // block scales come from DRAM, behind the weights in flight) and
        // rounded before its stage is waited for: a load after the wait would
        // add its trip to the time a stage takes to come round (0.37 us a
        // block for 11 stages, whatever the number of SMs).
        using T = typename std::conditional<SOURCE == 0, __half, __nv_bfloat16>::type;
        constexpr int SC = (NT + 31) / 32;
        struct Ahead {
            uint2 x[ROWS];
            float s[SC], ws;
        } a;
        const uint32_t turn = Pipe<NT>::X_TURN;
        auto fetch = [&](uint32_t i, Ahead &f) {
            if (i >= nblk) return;
            const uint32_t q = i / nk, k = k0 + (i - q * nk);
            f.ws = __ldg(p.ws + (int64_t)(first + q * NC) * p.KB + k);
            if constexpr (ROUND) {
                const int col = k * GLQ_FP8_BLOCK + lane * 4;
                const T *src = static_cast<const T *>(p.x) + col;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    f.x[r] = make_uint2(0, 0);
                    // n is a multiple of 8: a lane's four columns are in or out together
                    if (r < p.B && col < p.n) f.x[r] = __ldcg(reinterpret_cast<const uint2 *>(src + (int64_t)r * p.n));
                }
            } else {
#pragma unroll
                for (int j = 0; j < SC; ++j) {
                    const int tok = j * 32 + lane;
                    f.s[j] = tok < p.B ? __ldcg(p.s + (int64_t)k * p.s_ld + tok) : 0.f;
                }
            }
        };
        const uint32_t w0 = warp - X_WARP0;
        if (w0 < turn) fetch(w0, a);
        for (uint32_t i = w0; i < nblk && w0 < turn; i += turn) {
            float *sc = pipe.sc[i % STAGES];
            const Ahead f = a;
            if constexpr (!ROUND) fetch(i + turn, a);
            if constexpr (ROUND) {
                float inv;
                const float s = warp_group_scales<T, ROWS>(f.x, p.B, lane, inv);
                if (!pipe_x_begin(pipe, i, p.err)) break;
                uint8_t *xt = pipe_x_tile<NT>(smem, i);
                if (lane < p.B) sc[lane] = s * f.ws;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    if (r >= p.B) break;
                    *reinterpret_cast<uint32_t *>(xt + sw128(r, lane >> 2) + (lane & 3) * 4) =
                        round4<T>(f.x[r], __shfl_sync(0xffffffffu, inv, r));
                }
            } else {
                if (!pipe_x_begin(pipe, i, p.err)) break;
#pragma unroll
                for (int j = 0; j < SC; ++j)
                    if (j * 32 + lane < NT) sc[j * 32 + lane] = f.s[j] * f.ws;
            }
            pipe_x_done<NT, ROUND>(pipe, i, lane);
            // not before: the proxy fence in pipe_x_done waits for loads in flight
            if constexpr (ROUND) fetch(i + turn, a);
        }
    } else {
        pdl_wait();  // y may still be in use by the kernel before
        const int quadrant = warp & 3, set = (warp - D_WARP0) >> 2;
        const int row_l = 32 * quadrant + lane, dtid = tid - D_WARP0 * 32;
        float *red = reinterpret_cast<float *>(smem + STAGES * Pipe<NT>::STAGE_BYTES);
        const int per = (NT / 4 + C - 1) / C;  // most groups of four tokens one CTA sums
        float acc[HALF];
        uint32_t i = 0, round = 0;
        for (uint32_t t = first; t < tiles; t += NC, ++round) {
            const int live = p.B;
#pragma unroll
            for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
            bool ok = true;
            for (uint32_t k = 0; k < nk && ok;) {
                const int n = min((int)(nk - k), DRAIN);
                if (n == DRAIN) ok = pipe_drain<NT, DRAIN>(pipe, i, quadrant, set, acc, p.err);
                else ok = pipe_drain<NT, 1>(pipe, i, quadrant, set, acc, p.err);
                k += n == DRAIN ? DRAIN : 1;
                i += n == DRAIN ? DRAIN : 1;
            }
            if (!ok) break;
            if (C == 1) {
                const int row = t * 128 + row_l;
                if (row < p.m) {
#pragma unroll
                    for (int j = 0; j < HALF; ++j)
                        if (set * HALF + j < live)
                            store_y(p.y, p.y_dtype, (int64_t)(set * HALF + j) * p.m + row, acc[j]);
                }
                continue;
            }
            // Parts to the CTAs that sum them, four tokens a store (stores of one
            // token each cost 2.5 us more at 64 tokens), but a single token by
            // itself (0.1 to 0.5 us less than with three that are not there).
            const int width = live == 1 ? 1 : 4;
            const int groups = (live + 3) >> 2;
            const int mine = groups > (int)rank ? (groups - (int)rank - 1) / (int)C + 1 : 0;  // this CTA sums
            if (!met) cluster_wait(), met = true;
            if (!pipe.template wait_warp<true>(&pipe.red_empty, (round & 1) ^ 1, p.err)) break;
            if (dtid == 0) mbar_expect_tx(&pipe.red_full, (uint32_t)(mine * (int)C * width) * (128 * 4));
            if (width == 1) {
                if (set == 0)
                    st_async(remote_smem(red + (int)rank * 128 + row_l, 0), acc[0], remote_smem(&pipe.red_full, 0));
            } else {
#pragma unroll
                for (int j = 0; j < HALF; j += 4) {
                    const int g = (set * HALF + j) >> 2, own = g / (int)C, to = g - own * (int)C;
                    if (g < groups)
                        st_async4(remote_smem(red + (((int)rank * per + own) * 128 + row_l) * 4, to), acc + j,
                                  remote_smem(&pipe.red_full, to));
                }
            }
            if (!pipe.template wait_warp<true>(&pipe.red_full, round & 1, p.err)) break;
            // a warp sums 32 rows of a group
            for (int u = dtid >> 5; u < mine * 4; u += D_WARPS) {
                const int own = u >> 2, r = (u & 3) * 32 + lane, row = t * 128 + r;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                if (width == 1) {
                    for (uint32_t c = 0; c < C; ++c) sum[0] += red[c * 128 + r];
                } else {
                    for (uint32_t c = 0; c < C; ++c) {
                        const float4 v = *reinterpret_cast<const float4 *>(red + (((int)c * per + own) * 128 + r) * 4);
                        sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
                    }
                }
                const int tok = (own * (int)C + (int)rank) * 4;
                if (row < p.m) {
#pragma unroll
                    for (int l = 0; l < 4; ++l)
                        if (tok + l < live) store_y(p.y, p.y_dtype, (int64_t)(tok + l) * p.m + row, sum[l]);
                }
            }
            __syncwarp();
            // in the last round nobody waits for it, and a CTA may leave as soon
            // as its own parts are here
            if (t + NC < tiles && lane < C) sm100::mbar_arrive_remote(&pipe.red_empty, lane);
        }
    }
    __syncwarp();
    if (C > 1 && !met) cluster_wait();
    sm100::tc_fence_before();
    __syncthreads();
    if (copier && pipe.abort) pipe_load_drain(pipe, it);
    __syncwarp();
    if (warp == 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(pipe.tmem, Pipe<NT>::TMEM_COLS);
    }
    // A CTA that has its parts is written to no more; one that gave up before
    // waits for the others to finish or leave.
    if (C > 1 && pipe.abort) sm100::cluster_sync_all();
}


}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantParams &p, int dtype, cudaStream_t s, bool pdl) {
    const void *fn = dtype == 0   ? (const void *)fp8_quantize_kernel<__half>
                     : dtype == 1 ? (const void *)fp8_quantize_kernel<__nv_bfloat16>
                                  : (const void *)fp8_quantize_kernel<float>;
    Fp8QuantParams q = p;
    void *args[] = {&q};
    const dim3 grid((unsigned)((p.KB + QG - 1) / QG), (unsigned)((p.B + QT - 1) / QT));
    return launch_ex(fn, grid, dim3(QTHREADS), 0, s, pdl, args);
}

cudaError_t launch_fp8_pack(const Fp8PackParams &p, cudaStream_t s) {
    const dim3 grid(p.KB, (p.rows + 127) / 128, p.count < 1024 ? p.count : 1024);
    fp8_pack_kernel<<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_fp8_dequant(const uint8_t *tiles, const float *scale, float *w, int m, int n, int KB,
                               cudaStream_t s) {
    fp8_dequant_kernel<<<dim3(KB, (m + 127) / 128), 256, 0, s>>>(tiles, scale, w, m, n, KB);
    return cudaGetLastError();
}

int fp8_skinny_tile(int64_t B) { return B <= 16 ? 16 : B <= 32 ? 32 : 64; }

namespace {

struct SkinnyKernel {
    const void *fn;
    size_t smem;
    int key;
};

SkinnyKernel skinny_kernel(int source, int nt, int B) {
    if (source < 2 && B <= FP8_ROUND_FEW)
        return {source ? (const void *)fp8_skinny_kernel<16, 1, FP8_ROUND_FEW>
                       : (const void *)fp8_skinny_kernel<16, 0, FP8_ROUND_FEW>, Pipe<16>::SMEM_BYTES, source};
    if (source < 2)
        return {source ? (const void *)fp8_skinny_kernel<16, 1, FP8_ROUND_MAX>
                       : (const void *)fp8_skinny_kernel<16, 0, FP8_ROUND_MAX>, Pipe<16>::SMEM_BYTES, 5 + source};
    switch (nt) {
        case 16: return {(const void *)fp8_skinny_kernel<16, 2>, Pipe<16>::SMEM_BYTES, 2};
        case 32: return {(const void *)fp8_skinny_kernel<32, 2>, Pipe<32>::SMEM_BYTES, 3};
        default: return {(const void *)fp8_skinny_kernel<64, 2>, Pipe<64>::SMEM_BYTES, 4};
    }
}

// Sets the kernel's shared memory limit once per device.
cudaError_t prepare(const SkinnyKernel &k) {
    static std::atomic<uint64_t> configured[7];
    return once_per_device(configured[k.key], [&k] {
        return cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
    });
}

}  // namespace

cudaError_t fp8_skinny_clusters(int num_sms, int count[9]) {
    // the clusters that fit depend on the device's layout of SMs and on one
    // CTA per SM, not on which variant runs
    static int known[128][9];  // per device, once asked
    static std::atomic<bool> asked[128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 128 && asked[dev].load(std::memory_order_acquire)) {
        for (int c = 0; c <= 8; ++c) count[c] = known[dev][c];
        return cudaSuccess;
    }
    const SkinnyKernel k = skinny_kernel(2, 16, 16);
    e = prepare(k);
    count[0] = 0;
    count[1] = num_sms;
    for (int c = 2; c <= 8 && e == cudaSuccess; ++c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(c);
        cfg.blockDim = dim3(PIPE_THREADS);
        cfg.dynamicSmemBytes = k.smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = c;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&count[c], k.fn, &cfg);
    }
    if (e == cudaSuccess && dev < 128) {  // two callers would write the same values
        for (int c = 0; c <= 8; ++c) known[dev][c] = count[c];
        asked[dev].store(true, std::memory_order_release);
    }
    return e;
}

bool fp8_rounds_inside(int64_t B, int64_t tiles, int KB, int num_sms) {
    // A launch of the quantiser in front costs about 1.1 us; a block's rounding
    // inside the kernel comes once per row tile, and from 5 tokens on is slower
    // than its weights.  Measured, inside against in front: 960x960 at 5 / 8
    // tokens 4.7 / 4.9 against 5.6 / 5.5 us; 4096x14336 (24 blocks per SM) 14.6 /
    // 14.9 against 15.5 / 15.4; 32768x5120 (69) 31.9 / 32.8 against 30.6 / 30.5,
    // but at 4 tokens 29.4 against 30.6; 4096x14336 at 16 tokens 24.4 against 16.
    return B <= FP8_ROUND_FEW || (B <= FP8_ROUND_MAX && tiles * KB <= (int64_t)32 * num_sms);
}

Fp8SkinnyPlan plan_fp8_skinny(int64_t tiles, int KB, int nt, const int clusters[9]) {
    // A call takes about 2.4 us beside its blocks.  One CTA takes a block in
    // 0.22 us (16 tokens) to 0.31 us (64) by itself, all together at the HBM's
    // rate (16 KB at 5.9 TB/s: 0.0028 us), and near both bounds the two add up
    // like a norm.  Summing the parts of a split tile costs 1 us at 16 tokens,
    // 2.5 us at 64, and more the larger the cluster.  Measured with C = 1, 2,
    // 3, 4, 6, 8 at one token: 4096x14336 28.8, 17.0, 13.9, 12.6, 15.2, 17.2 us
    // (plan 4); 5120x32768 61, 35, 27.7, 38, 30, 33 us (plan 3); 11008x2048 7.0,
    // 8.3, 10.5, 9.6, 13.1, 16.0 us (plan 1); 1024x8192 17.3, 11.2, 8.8, 7.3, 6.2,
    // 5.4 us (plan 8).  At 64 tokens: 2560x960 5.8, 7.2, 7.7, 6.9, 7.7, 11.4 us
    // (plan 1); 4096x4096 14.0, 12.3, 11.3, 10.2, 13.5, 17.0 us (plan 4).
    Fp8SkinnyPlan best{1, (int)(tiles < clusters[1] ? tiles : clusters[1])};
    double best_t = 1e30;
    for (int c = 1; c <= 8 && c <= KB; ++c) {
        if (clusters[c] < 1) continue;
        const int64_t nc = tiles < clusters[c] ? tiles : clusters[c];
        const int64_t rounds = (tiles + nc - 1) / nc;
        const double alone = (double)(rounds * ((KB + c - 1) / c)) * (0.19 + 0.0019 * nt);
        const double hbm = (double)tiles * KB * 0.0028;
        const double t = 2.4 + std::cbrt(alone * alone * alone + hbm * hbm * hbm) +
                         (c > 1 ? 0.4 + nt / 32.0 + 0.1 * c : 0.0);
        if (t < best_t * 0.98) {
            best_t = t;
            best = {c, (int)nc};
        }
    }
    return best;
}

cudaError_t launch_fp8_skinny(const Fp8SkinnyParams &p, const CUtensorMap &qmap, int source, int nt, int clusters,
                              cudaStream_t s, bool pdl) {
    const SkinnyKernel k = skinny_kernel(source, nt, p.B);
    const cudaError_t e = prepare(k);
    if (e != cudaSuccess) return e;
    Fp8SkinnyParams q = p;
    CUtensorMap map = qmap;
    void *args[] = {&map, &q};
    return launch_ex(k.fn, dim3(clusters * p.C), dim3(PIPE_THREADS), k.smem, s, pdl, args, p.C);
}

}  // namespace glq
