// glq_fp8.cuh -- device side shared by the 8-bit float kernels: the
// activation rounding, the fp8 tensor-core instruction, and the pipeline of
// the few-token kernels (weights by bulk copies, tokens as the MMA's N side).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "glq_device.cuh"
#include "glq_fp8.h"
#include "glq_sm100.cuh"

namespace glq {
namespace fp8 {

constexpr float TOP = 448.f;               // largest e4m3 value
constexpr uint32_t FLOOR_BITS = 0x08800000u;  // 2^-110: the smallest group maximum a scale is made from
constexpr uint64_t WAIT_CYCLES = 4000000000ull;  // wait limit: 4e9 SM cycles (about 2 s)

// ---------------------------------------------------------------------------
// Activation rounding.  A group of 128 values of one token shares the scale
// s = a / 448, a its largest magnitude (at least 2^-110, so that 448 / a and
// a / 448 stay normal); each value becomes e4m3(v * (448 / a)), both products
// and quotients fp32, round to nearest even.  The magnitudes are compared as
// bit patterns, so a NaN (larger than every number as bits) makes the whole
// group NaN, and an infinity gives s = inf with itself as NaN.
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ float group_inv(uint32_t top_bits) { return __fdiv_rn(TOP, __uint_as_float(top_bits)); }
__device__ __forceinline__ float group_scale(uint32_t top_bits) { return __fdiv_rn(__uint_as_float(top_bits), TOP); }

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x4(const float v[4], float inv) {
    return e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2 *>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// One warp, one token, one group of 128: lane holds values 4 lane .. 4 lane
// + 3.  Returns the packed e4m3 values and the scale.
__device__ __forceinline__ uint32_t warp_quantize(const float v[4], float &scale) {
    uint32_t m = max(max(mag_bits(v[0]), mag_bits(v[1])), max(mag_bits(v[2]), mag_bits(v[3])));
    m = max(__reduce_max_sync(0xffffffffu, m), FLOOR_BITS);
    scale = group_scale(m);
    return e4m3x4(v, group_inv(m));
}

// Byte offset of (row, 16-byte chunk) in a K-major tile of 128-byte rows
// with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

// ---------------------------------------------------------------------------
// tcgen05.mma kind::f8f6f4, e4m3 x e4m3 -> fp32, K = 32 per instruction
// ---------------------------------------------------------------------------

// D format f32; format code 0 of A and B is e4m3; both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 8 consecutive 32-bit columns
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t r[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// ---------------------------------------------------------------------------
// The few-token pipeline.  The weights are the MMA's M side (128 rows), up to
// NT tokens its N side, one MMA group per 128-column block (K = 128: four
// instructions) into its own TMEM slot of NT columns, so that the MMA never
// waits for the sum over blocks, which the drain warps hold in registers:
// acc[token] += d * (token scale * block scale).  Roles:
//   warp 0       bulk copies of the 16 KB weight tiles, STAGES deep
//   warp 1       MMA issue and TMEM allocation
//   warps 2-9    token operand: one block per warp in turn, rounded or copied
//                into the swizzled tile, with the block's NT scales
//   warps 10-17  drain: warp & 3 is its TMEM lane quadrant (rows), the two
//                sets of four take half of the tokens each
// ---------------------------------------------------------------------------

constexpr int X_WARP0 = 2, X_WARPS = 8;
constexpr int D_WARP0 = 10, D_WARPS = 8;
constexpr int PIPE_THREADS = (D_WARP0 + D_WARPS) * 32;  // 576
constexpr int D_THREADS = D_WARPS * 32;

template <int NT>
struct Pipe {
    static constexpr int STAGE_BYTES = GLQ_FP8_TILE_BYTES + NT * 128;
    // as many stages as fit beside the static arrays: 198 KB at 16 tokens, 192 KB at 128
    static constexpr int STAGES = NT == 16 ? 11 : NT == 32 ? 10 : NT == 64 ? 8 : 6;
    static constexpr int SLOTS = 512 / NT;  // TMEM slots
    static constexpr int HALF = NT / 2;     // tokens of one drain set
    static constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * STAGE_BYTES;

    uint64_t w_full[STAGES], x_full[STAGES], empty[STAGES];
    uint64_t acc_full[SLOTS], acc_empty[SLOTS], sc_full[SLOTS], mma_done;
    uint64_t drain_bar;   // the drain warps among themselves: a wait that can give up
    alignas(16) float sc[SLOTS][NT];  // (read as float4) token scale * block scale of each slot
    uint32_t tmem;
    volatile int abort;
    unsigned last;  // broadcast among the drain warps

    __device__ __forceinline__ void init() {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&w_full[s], 1);
            mbar_init(&x_full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], D_WARPS);
            mbar_init(&sc_full[s], 1);
        }
        mbar_init(&mma_done, 1);
        mbar_init(&drain_bar, D_WARPS);
        abort = 0;
    }
    __device__ __forceinline__ void fail(unsigned *err) {
        atomicOr(err, GLQ_DEVERR_TIMEOUT);
        abort = 1;
    }
    // false once the wait has run out here or elsewhere in the CTA
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, unsigned *err) {
        if (abort) return false;
        if (sm100::mbar_wait(bar, parity, WAIT_CYCLES)) return true;
        fail(err);
        return false;
    }
    // the same for a whole warp: one answer, whatever each lane saw
    __device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, unsigned *err) {
        return __all_sync(0xffffffffu, wait(bar, parity, err));
    }
    // Barrier of the drain warps; phase counts the ones passed.  Not bar.sync:
    // a drain warp that gave up elsewhere would leave the others waiting.
    __device__ __forceinline__ bool drain_sync(uint32_t &phase, unsigned *err) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(&drain_bar);
        return wait_warp(&drain_bar, phase++ & 1, err);
    }
};

// Block `it` of this CTA's sequence: wait for its stage and load its tile.
template <int NT>
__device__ __forceinline__ bool pipe_load(Pipe<NT> &p, uint8_t *smem, uint32_t it, const uint8_t *tile, unsigned *err) {
    const uint32_t s = it % Pipe<NT>::STAGES, use = it / Pipe<NT>::STAGES;
    if (!p.wait(&p.empty[s], (use & 1) ^ 1, err)) return false;
    mbar_expect_tx(&p.w_full[s], GLQ_FP8_TILE_BYTES);
    bulk_g2s(smem + s * Pipe<NT>::STAGE_BYTES, tile, GLQ_FP8_TILE_BYTES, &p.w_full[s]);
    return true;
}

// After an abort: let the copies of blocks [.., loaded) land before the CTA exits.
template <int NT>
__device__ __forceinline__ void pipe_load_drain(Pipe<NT> &p, uint32_t loaded) {
    const uint32_t first = loaded > (uint32_t)Pipe<NT>::STAGES ? loaded - Pipe<NT>::STAGES : 0;
    for (uint32_t i = first; i < loaded; ++i)
        sm100::mbar_wait(&p.w_full[i % Pipe<NT>::STAGES], (i / Pipe<NT>::STAGES) & 1, WAIT_CYCLES);
}

// The MMA warp's one thread: blocks [it, it + count).
template <int NT>
__device__ __forceinline__ bool pipe_mma(Pipe<NT> &p, uint8_t *smem, uint32_t it, uint32_t count, unsigned *err) {
    const uint32_t idesc = idesc_e4m3_f32(128, NT);
    for (const uint32_t end = it + count; it != end; ++it) {
        const uint32_t s = it % Pipe<NT>::STAGES, use = it / Pipe<NT>::STAGES;
        const uint32_t slot = it % Pipe<NT>::SLOTS, suse = it / Pipe<NT>::SLOTS;
        if (!p.wait(&p.acc_empty[slot], (suse & 1) ^ 1, err) || !p.wait(&p.x_full[s], use & 1, err) ||
            !p.wait(&p.w_full[s], use & 1, err))
            return false;
        sm100::tc_fence_after();
        uint8_t *st = smem + s * Pipe<NT>::STAGE_BYTES;
        const uint64_t a = sm100::smem_desc_sw128(st), b = sm100::smem_desc_sw128(st + GLQ_FP8_TILE_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_f8_ss(p.tmem + slot * NT, a + 2 * kk, b + 2 * kk, idesc, kk);
        sm100::mma_commit(&p.acc_full[slot]);
        sm100::mma_commit(&p.empty[s]);
    }
    return true;
}

// A token-operand warp before it writes block `it`: its stage and scale slot
// are free.  After the writes: pipe_x_done.
template <int NT>
__device__ __forceinline__ bool pipe_x_begin(Pipe<NT> &p, uint32_t it, unsigned *err) {
    const uint32_t s = it % Pipe<NT>::STAGES, slot = it % Pipe<NT>::SLOTS;
    return p.wait_warp(&p.empty[s], ((it / Pipe<NT>::STAGES) & 1) ^ 1, err) &&
           p.wait_warp(&p.acc_empty[slot], ((it / Pipe<NT>::SLOTS) & 1) ^ 1, err);
}
template <int NT>
__device__ __forceinline__ void pipe_x_done(Pipe<NT> &p, uint32_t it, int lane) {
    sm100::fence_proxy_async_smem();  // the MMA reads the tile through the async proxy
    __syncwarp();
    if (lane == 0) {
        sm100::mbar_arrive(&p.sc_full[it % Pipe<NT>::SLOTS]);
        sm100::mbar_arrive(&p.x_full[it % Pipe<NT>::STAGES]);
    }
}

// A drain warp: adds block `it` to acc (its half of the tokens).  skip_zero:
// tokens whose scale is 0 take no part (their operand rows are not written).
template <int NT, bool SKIP_ZERO>
__device__ __forceinline__ bool pipe_drain(Pipe<NT> &p, uint32_t it, int quadrant, int set, float (&acc)[NT / 2],
                                           unsigned *err) {
    constexpr int HALF = NT / 2;
    constexpr int STEP = HALF < 16 ? 8 : 16;
    const uint32_t slot = it % Pipe<NT>::SLOTS, par = (it / Pipe<NT>::SLOTS) & 1;
    if (!p.wait_warp(&p.sc_full[slot], par, err) || !p.wait_warp(&p.acc_full[slot], par, err)) return false;
    sm100::tc_fence_after();
    const uint32_t t0 = p.tmem + ((uint32_t)(32 * quadrant) << 16) + slot * NT + set * HALF;
    const float4 *sc = reinterpret_cast<const float4 *>(&p.sc[slot][set * HALF]);
#pragma unroll
    for (int c = 0; c < HALF; c += STEP) {
        uint32_t d[STEP];
        if constexpr (STEP == 8) tmem_ld8(t0 + c, d);
        else sm100::tmem_ld16(t0 + c, d);
        sm100::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < STEP; j += 4) {
            const float4 f = sc[(c + j) >> 2];
            const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int l = 0; l < 4; ++l)
                if (!SKIP_ZERO || fs[l] != 0.f)
                    acc[c + j + l] = fmaf(__uint_as_float(d[j + l]), fs[l], acc[c + j + l]);
        }
    }
    sm100::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) sm100::mbar_arrive(&p.acc_empty[slot]);
    return true;
}

// Blocks dealt out evenly: CTA c of G owns [c total / G, (c + 1) total / G).
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t total, int64_t G) { return c * total / G; }
// the CTA that owns block b
__device__ __forceinline__ int range_owner(int64_t b, int64_t total, int64_t G) {
    return (int)(((b + 1) * G - 1) / total);
}

__device__ __forceinline__ void store_y(void *y, int dtype, int64_t i, float v) {
    if (dtype == 1) static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
    else if (dtype == 0) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<float *>(y)[i] = v;
}

}  // namespace fp8
}  // namespace glq
