// glq_fp8.cu -- the activation quantiser, the weight layout and the few-token
// product of the 8-bit float linear layer
//     y[b][r] = sum_kb s[kb][b] ws[r/128][kb] sum_{k in kb} q[b][k] w[r][k]
// (q, w e4m3; s the token's scale of 128-column block kb, ws the weight
// block's).
#include "glq_fp8.cuh"
#include "glq_kernels.cuh"

namespace glq {

namespace {

using namespace fp8;

// ---------------------------------------------------------------------------
// Quantiser: reads x once, writes q and s once; bound by HBM.  A CTA takes 32
// tokens x 2 groups: half a warp per group (8 values a lane, one or two
// 16-byte loads), all of a warp's four tokens loaded before the first is
// used, and the scales of a group of 32 tokens leave as one 128-byte line of
// the [group][token] array.
// ---------------------------------------------------------------------------

constexpr int QT = 32, QG = 2, QTHREADS = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *p, float v[8]) {
    const uint4 w = ldg_nc_v4(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<T>(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float v[8]) {
    const uint4 a = ldg_nc_v4(p), b = ldg_nc_v4(p + 4);
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
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
    constexpr int PER = QT / (QTHREADS / 32);  // tokens per warp
    float v[PER][8];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t t = t0 + warp + i * (QTHREADS / 32);
        if (t < p.B && col < p.n) load8(static_cast<const T *>(p.x) + t * p.n + col, v[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int tl = warp + i * (QTHREADS / 32);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, mag_bits(v[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = max(m, FLOOR_BITS);
        const float inv = group_inv(m);
        if (t0 + tl < p.B && g < p.KB) {
            const uint2 q = make_uint2(e4m3x4(v[i], inv), e4m3x4(v[i] + 4, inv));
            *reinterpret_cast<uint2 *>(p.q + (t0 + tl) * ((int64_t)p.KB * GLQ_FP8_BLOCK) + col) = q;
        }
        if (l16 == 0) s_s[half][tl] = group_scale(m);
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
// Few tokens.  Reads every weight once: bound by HBM for small batches.  The
// 128 x 128 blocks of all output tiles form one sequence, dealt out evenly
// over the CTAs (one per SM), so that every SM streams the same number of
// bytes whatever m and n are; a tile whose blocks fall to several CTAs is
// summed from their parts, in the order of the CTAs, by the CTA that arrives
// last.
// SOURCE 0 / 1: f16 / bf16 activations rounded on the way; 2: e4m3 rows (by
// TMA: 128 columns x NT tokens, 128-byte swizzle) and their scales.
// ---------------------------------------------------------------------------

// y[tok0 .. tok0 + live)[row0 .. row0 + 128) = the sum of a tile's parts, by
// the 256 drain threads: a thread has 4 rows of one token in eight, and the
// loads of four such tokens in flight.
__device__ __forceinline__ void sum_parts(const Fp8SkinnyParams &p, int nt, int c0, int c1, int tok0, int live, int row0,
                                          int dtid) {
    const int r4 = (dtid & 31) * 4, jt = dtid >> 5;
    const int64_t cstep = (int64_t)2 * nt * 128;
    // the first part is its CTA's last tile (slot 1), the others their CTAs' first (slot 0)
    const float *first = p.part + c0 * cstep + (int64_t)nt * 128 + r4, *rest = p.part + (c0 + 1) * cstep + r4;
    for (int j0 = jt; j0 < live; j0 += 32) {
        float4 sum[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j0 + 8 * i < live) sum[i] = __ldcg(reinterpret_cast<const float4 *>(first + (j0 + 8 * i) * 128));
#pragma unroll 4
        for (int c = c0 + 1; c <= c1; ++c) {
            const float *src = rest + (c - c0 - 1) * cstep;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (j0 + 8 * i >= live) continue;
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(src + (j0 + 8 * i) * 128));
                sum[i].x += v.x;
                sum[i].y += v.y;
                sum[i].z += v.z;
                sum[i].w += v.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + r4;  // m is a multiple of 8: four rows are in or out together
            if (j0 + 8 * i < live && row < p.m) store_y4(p.y, p.y_dtype, (int64_t)(tok0 + j0 + 8 * i) * p.m + row, sum[i]);
        }
    }
}

template <int NT, int SOURCE>
__global__ void __launch_bounds__(PIPE_THREADS, 1) fp8_skinny_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                     Fp8SkinnyParams p) {
    constexpr bool ROUND = SOURCE != 2;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) Pipe<NT> pipe;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t KB = p.KB, TT = p.TT, total = p.RT * TT * KB, G = gridDim.x, cta = blockIdx.x;
    const uint32_t b0 = range_begin(cta, total, G), nblk = range_begin(cta + 1, total, G) - b0;

    uint32_t it = 0;  // warp 0: blocks whose copies have been started
    uint32_t tile = b0 / KB, kb = b0 - tile * KB, rt = tile / TT, tt = tile - rt * TT;
    auto next_block = [&]() {
        if (++kb == KB) {
            kb = 0;
            if (++tt == TT) tt = 0, ++rt;
        }
    };
    auto w_tile = [&]() { return p.w + ((int64_t)rt * KB + kb) * GLQ_FP8_TILE_BYTES; };
    if (warp == 0) {
        pipe.init(lane);
        __syncwarp();
        if (lane == 0) {  // weights are constant: the first copies start at once
            const uint32_t n = min(nblk, (uint32_t)Pipe<NT>::STAGES);
            const uint32_t rt0 = rt, tt0 = tt, kb0 = kb;
            for (; it < n; ++it, next_block()) pipe_load<NT, ROUND>(pipe, smem, it, w_tile(), ROUND ? 0 : NT * 128, p.err);
            if (!ROUND) {
                sm100::prefetch_tensormap(&qmap);
                pdl_wait();  // the rounded tokens come from the kernel before
                rt = rt0, tt = tt0, kb = kb0;
                for (uint32_t i = 0; i < n; ++i, next_block())
                    sm100::tma_load_2d(pipe_x_tile<NT>(smem, i), &qmap, &pipe.w_full[i], kb * GLQ_FP8_BLOCK, tt * NT);
            }
        }
    }
    if (warp == 1) {
        sm100::tmem_alloc(&pipe.tmem, Pipe<NT>::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            for (; it < nblk; ++it, next_block()) {
                if (!pipe_load<NT, ROUND>(pipe, smem, it, w_tile(), ROUND ? 0 : NT * 128, p.err)) break;
                if (!ROUND)
                    sm100::tma_load_2d(pipe_x_tile<NT>(smem, it), &qmap, &pipe.w_full[it % Pipe<NT>::STAGES],
                                       kb * GLQ_FP8_BLOCK, tt * NT);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            pipe_mma<NT, ROUND>(pipe, smem, 0, nblk, p.err);
            sm100::mma_commit(&pipe.mma_done);  // every MMA issued has completed
            sm100::mbar_wait(&pipe.mma_done, 0, WAIT_CYCLES);
        }
    } else if (warp < D_WARP0) {
        pdl_wait();
        for (uint32_t i = warp - X_WARP0; i < nblk && warp < X_WARP0 + Pipe<NT>::X_TURN; i += Pipe<NT>::X_TURN) {
            const uint32_t b = b0 + i, t = b / KB, k = b - t * KB, r = t / TT;
            const int tok0 = (int)(t - r * TT) * NT, live = min(NT, p.B - tok0);
            const float ws = __ldg(p.ws + (int64_t)r * KB + k);
            float *sc = pipe.sc[i % Pipe<NT>::STAGES];
            if constexpr (ROUND) {
                using T = typename std::conditional<SOURCE == 0, __half, __nv_bfloat16>::type;
                const int col = k * GLQ_FP8_BLOCK + lane * 4;
                if (!pipe_x_begin(pipe, i, p.err)) break;
                // n is a multiple of 8: a lane's four columns are in or out together
                warp_quantize_rows(static_cast<const T *>(p.x) + (int64_t)tok0 * p.n + col, (int64_t)p.n, col < p.n, live,
                                   pipe_x_tile<NT>(smem, i), sc, ws, lane);
            } else {
                float s[(NT + 31) / 32];
#pragma unroll
                for (int j = 0; j < (NT + 31) / 32; ++j) {
                    const int tok = j * 32 + lane;
                    s[j] = tok < live ? p.s[(int64_t)k * p.s_ld + tok0 + tok] * ws : 0.f;
                }
                if (!pipe_x_begin(pipe, i, p.err)) break;
#pragma unroll
                for (int j = 0; j < (NT + 31) / 32; ++j)
                    if (j * 32 + lane < NT) sc[j * 32 + lane] = s[j];
            }
            pipe_x_done<NT, ROUND>(pipe, i, lane);
        }
    } else {
        pdl_wait();  // y and the workspace may still be in use by the kernel before
        constexpr int HALF = NT / 2;
        const int quadrant = warp & 3, set = (warp - D_WARP0) >> 2;
        const int row_l = 32 * quadrant + lane, dtid = tid - D_WARP0 * 32;
        uint32_t dphase = 0;
        float acc[HALF];
#pragma unroll
        for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
        for (uint32_t i = 0; i < nblk; ++i) {
            if (!pipe_drain<NT, false>(pipe, i, quadrant, set, acc, p.err)) break;
            const bool tile_end = ++kb == KB;
            if (!tile_end && i + 1 < nblk) continue;
            // the end of this CTA's part of the tile
            const int tok0 = tt * NT, live = min(NT, p.B - tok0);
            const uint32_t tb = tile * KB;   // the tile's first block
            const bool head = b0 > tb;       // an earlier CTA has its beginning
            if (!head && tile_end) {
                const int row = rt * 128 + row_l;
                if (row < p.m) {
#pragma unroll
                    for (int j = 0; j < HALF; ++j)
                        if (set * HALF + j < live)
                            store_y(p.y, p.y_dtype, (int64_t)(tok0 + set * HALF + j) * p.m + row, acc[j]);
                }
            } else {
                float *part = p.part + ((int64_t)cta * 2 + (head ? 0 : 1)) * NT * 128;
#pragma unroll
                for (int j = 0; j < HALF; ++j)
                    if (set * HALF + j < live) __stcg(part + (set * HALF + j) * 128 + row_l, acc[j]);
                if (!pipe.drain_sync(dphase, p.err)) break;
                const int c0 = range_owner(tb, total, G), c1 = range_owner(tb + KB - 1, total, G);
                if (dtid == 0) {
                    __threadfence();  // the parts of all drain threads, ordered here by the barrier
                    const bool last = atom_add_acq_rel_gpu(p.cnt + tile, 1u) == (unsigned)(c1 - c0);
                    if (last) p.cnt[tile] = 0;  // as the next call expects it
                    __threadfence();
                    pipe.last = last;
                }
                if (!pipe.drain_sync(dphase, p.err)) break;
                if (pipe.last) sum_parts(p, NT, c0, c1, tok0, live, rt * 128, dtid);
            }
#pragma unroll
            for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
            ++tile;
            kb = 0;
            if (++tt == TT) tt = 0, ++rt;
        }
    }
    sm100::tc_fence_before();
    __syncthreads();
    if (tid == 0 && pipe.abort) pipe_load_drain(pipe, it);
    if (warp == 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(pipe.tmem, Pipe<NT>::TMEM_COLS);
    }
}

template <int NT>
const void *skinny_fn(int source) {
    return source == 0   ? (const void *)fp8_skinny_kernel<NT, 0>
           : source == 1 ? (const void *)fp8_skinny_kernel<NT, 1>
                         : (const void *)fp8_skinny_kernel<NT, 2>;
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

int fp8_skinny_tile(int64_t B) { return B <= 16 ? 16 : B <= 32 ? 32 : B <= 64 ? 64 : 128; }

size_t fp8_skinny_part_bytes(int nt, int grid) { return (size_t)grid * 2 * nt * 128 * sizeof(float); }

cudaError_t launch_fp8_skinny(const Fp8SkinnyParams &p, const CUtensorMap &qmap, int source, int nt, int grid,
                              cudaStream_t s, bool pdl) {
    const void *fn;
    size_t smem;
    int key;
    switch (nt) {
        case 16: fn = skinny_fn<16>(source), smem = Pipe<16>::SMEM_BYTES, key = 0; break;
        case 32: fn = skinny_fn<32>(source), smem = Pipe<32>::SMEM_BYTES, key = 1; break;
        case 64: fn = skinny_fn<64>(source), smem = Pipe<64>::SMEM_BYTES, key = 2; break;
        case 128: fn = skinny_fn<128>(source), smem = Pipe<128>::SMEM_BYTES, key = 3; break;
        default: return cudaErrorInvalidValue;
    }
    static std::atomic<uint64_t> configured[12];
    const cudaError_t e = once_per_device(configured[key * 3 + source], [fn, smem] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    Fp8SkinnyParams q = p;
    CUtensorMap map = qmap;
    void *args[] = {&map, &q};
    return launch_ex(fn, dim3(grid), dim3(PIPE_THREADS), smem, s, pdl, args);
}

}  // namespace glq
