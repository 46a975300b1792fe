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
// SOURCE 0 / 1: f16 / bf16 activations rounded on the way; 2: e4m3 and scales.
// ---------------------------------------------------------------------------

template <int NT, int SOURCE>
__global__ void __launch_bounds__(PIPE_THREADS, 1) fp8_skinny_kernel(Fp8SkinnyParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) Pipe<NT> pipe;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t total = (int64_t)p.RT * p.TT * p.KB;
    const int G = gridDim.x, cta = blockIdx.x;
    const int64_t b0 = range_begin(cta, total, G), b1 = range_begin(cta + 1, total, G);
    const uint32_t nblk = (uint32_t)(b1 - b0);

    if (tid == 0) pipe.init();
    if (warp == 1) {
        sm100::tmem_alloc(&pipe.tmem, 512);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {  // weights are constant: no wait for the kernel before
            uint32_t it = 0;
            for (; it < nblk; ++it) {
                const int64_t b = b0 + it, tile = b / p.KB;
                const int64_t rt = tile / p.TT;
                if (!pipe_load(pipe, smem, it, p.w + (rt * p.KB + (b - tile * p.KB)) * GLQ_FP8_TILE_BYTES, p.err))
                    break;
            }
            if (pipe.abort) pipe_load_drain(pipe, it);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            pipe_mma(pipe, smem, 0, nblk, p.err);
            sm100::mma_commit(&pipe.mma_done);  // every MMA issued has completed
            sm100::mbar_wait(&pipe.mma_done, 0, WAIT_CYCLES);
        }
    } else if (warp < D_WARP0) {
        pdl_wait();
        for (uint32_t it = warp - X_WARP0; it < nblk; it += X_WARPS) {
            const int64_t b = b0 + it, tile = b / p.KB;
            const int kb = (int)(b - tile * p.KB), rt = (int)(tile / p.TT), tok0 = (int)(tile - (int64_t)rt * p.TT) * NT;
            const int live = min(NT, p.B - tok0);
            if (!pipe_x_begin(pipe, it, p.err)) break;
            uint8_t *xt = smem + (it % Pipe<NT>::STAGES) * Pipe<NT>::STAGE_BYTES + GLQ_FP8_TILE_BYTES;
            float *sc = pipe.sc[it % Pipe<NT>::SLOTS];
            const float ws = __ldg(p.ws + (int64_t)rt * p.KB + kb);
            if constexpr (SOURCE == 2) {
                const int64_t ld = (int64_t)p.KB * GLQ_FP8_BLOCK;
                const int chunk = lane & 7;
                const uint8_t *src = p.q + (int64_t)tok0 * ld + kb * GLQ_FP8_BLOCK + chunk * 16;
#pragma unroll 8
                for (int r = lane >> 3; r < live; r += 4) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + r * ld);
                    *reinterpret_cast<uint4 *>(xt + sw128(r, chunk)) = v;
                }
                for (int r = lane; r < live; r += 32) sc[r] = p.s[(int64_t)kb * p.s_ld + tok0 + r] * ws;
            } else {
                using T = typename std::conditional<SOURCE == 0, __half, __nv_bfloat16>::type;
                const int col = kb * GLQ_FP8_BLOCK + lane * 4;
                const bool in = col < p.n;  // n is a multiple of 8
                const T *src = static_cast<const T *>(p.x) + (int64_t)tok0 * p.n + col;
#pragma unroll 4
                for (int r = 0; r < live; ++r) {
                    uint2 w = make_uint2(0, 0);
                    if (in) w = *reinterpret_cast<const uint2 *>(src + (int64_t)r * p.n);
                    const float2 a = unpack2<T>(w.x), c = unpack2<T>(w.y);
                    const float v[4] = {a.x, a.y, c.x, c.y};
                    float s;
                    const uint32_t q = warp_quantize(v, s);
                    *reinterpret_cast<uint32_t *>(xt + sw128(r, lane >> 2) + (lane & 3) * 4) = q;
                    if (lane == 0) sc[r] = s * ws;
                }
            }
            pipe_x_done(pipe, it, lane);
        }
    } else {
        pdl_wait();  // y and the workspace may still be in use by the kernel before
        constexpr int HALF = NT / 2;
        const int dw = warp - D_WARP0, quadrant = warp & 3, set = dw >> 2;
        const int row_l = 32 * quadrant + lane, dtid = tid - D_WARP0 * 32;
        int64_t tile = nblk ? b0 / p.KB : 0;
        int kb = (int)(b0 - tile * p.KB);
        uint32_t dphase = 0;
        float acc[HALF];
#pragma unroll
        for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
        for (uint32_t it = 0; it < nblk; ++it) {
            if (!pipe_drain<NT, false>(pipe, it, quadrant, set, acc, p.err)) break;
            const bool tile_end = ++kb == p.KB;
            if (!tile_end && it + 1 < nblk) continue;
            // the end of this CTA's part of the tile
            const int rt = (int)(tile / p.TT), tok0 = (int)(tile - (int64_t)rt * p.TT) * NT;
            const int live = min(NT, p.B - tok0);
            const int64_t tb = tile * p.KB;  // the tile's first block
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
                __threadfence();
                if (!pipe.drain_sync(dphase, p.err)) break;
                const int c0 = range_owner(tb, total, G), c1 = range_owner(tb + p.KB - 1, total, G);
                if (dtid == 0) {
                    const bool last = atom_add_acq_rel_gpu(p.cnt + tile, 1u) == (unsigned)(c1 - c0);
                    if (last) p.cnt[tile] = 0;  // as the next call expects it
                    pipe.last = last;
                }
                if (!pipe.drain_sync(dphase, p.err)) break;
                if (pipe.last) {
                    __threadfence();
                    const int r = dtid & 127, row = rt * 128 + r;
                    for (int j = dtid >> 7; j < live; j += 2) {
                        float sum = 0.f;
                        for (int c = c0; c <= c1; ++c)
                            sum += __ldcg(p.part + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * NT * 128 + j * 128 + r);
                        if (row < p.m) store_y(p.y, p.y_dtype, (int64_t)(tok0 + j) * p.m + row, sum);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
            ++tile;
            kb = 0;
        }
    }
    sm100::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(pipe.tmem, 512);
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

cudaError_t launch_fp8_skinny(const Fp8SkinnyParams &p, int source, int nt, int grid, cudaStream_t s, bool pdl) {
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
    void *args[] = {&q};
    return launch_ex(fn, dim3(grid), dim3(PIPE_THREADS), smem, s, pdl, args);
}

}  // namespace glq
