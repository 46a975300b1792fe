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

// Byte offset of (row, 16-byte chunk) in a K-major tile of 128-byte rows
// with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

// One warp, a group of 128 columns of up to ROWS <= 32 tokens, whose lane l
// holds columns 4 l .. 4 l + 3 of each (w[r], two 16-bit pairs).  The two
// divisions are made once for all tokens, lane r having token r's: returns
// lane r's scale, and its inverse in inv.
template <typename T, int ROWS>
__device__ __forceinline__ float warp_group_scales(const uint2 (&w)[ROWS], int live, int lane, float &inv) {
    uint32_t mine = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (r >= live) break;
        const float2 a = unpack2<T>(w[r].x), c = unpack2<T>(w[r].y);
        const uint32_t m = __reduce_max_sync(0xffffffffu, max(max(mag_bits(a.x), mag_bits(a.y)),
                                                              max(mag_bits(c.x), mag_bits(c.y))));
        if (lane == r) mine = m;
    }
    mine = max(mine, FLOOR_BITS);
    inv = group_inv(mine);
    return group_scale(mine);
}

// One warp, a group of one token in fp32: lane l holds values 4 l .. 4 l + 3;
// returns them rounded.
__device__ __forceinline__ uint32_t warp_quantize(const float v[4], float &scale) {
    uint32_t m = max(max(mag_bits(v[0]), mag_bits(v[1])), max(mag_bits(v[2]), mag_bits(v[3])));
    m = max(__reduce_max_sync(0xffffffffu, m), FLOOR_BITS);
    scale = group_scale(m);
    return e4m3x4(v, group_inv(m));
}

// The rounded values of one token of warp_group_scales.
template <typename T>
__device__ __forceinline__ uint32_t round4(uint2 w, float inv) {
    const float2 a = unpack2<T>(w.x), c = unpack2<T>(w.y);
    const float v[4] = {a.x, a.y, c.x, c.y};
    return e4m3x4(v, inv);
}

// ---------------------------------------------------------------------------
// Waits, bounded.  CTA scope, or (CLUSTER) cluster scope: for barriers behind
// which values lie that another CTA of the cluster stored here, or that say
// that another CTA has read what it was sent; two per tile, not one per block.
// (try_wait, with and without a suspend hint, took the same time within 5 %,
// now more, now less.)
// ---------------------------------------------------------------------------

template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
    return done != 0;
}

// false once `limit` cycles have passed, here (then *abort is set and the
// error word says so) or elsewhere in the CTA
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned *err,
                                             uint64_t limit = WAIT_CYCLES) {
    if (mbar_test<CLUSTER>(bar, parity)) return true;
    const uint64_t t0 = sm100::clock_cycles();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_test<CLUSTER>(bar, parity)) return true;
        if (*abort) return false;
        if (sm100::clock_cycles() - t0 > limit) {
            atomicOr(err, GLQ_DEVERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ uint64_t atom_add_u64(uint64_t *p, uint64_t v) {
    uint64_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
    return old;
}
__device__ __forceinline__ uint64_t ld_acquire_u64(const uint64_t *p) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
// One thread of each of the G CTAs of a cooperative launch: the grid's barrier.
// `bar` counts arrivals over all calls, each of which adds a multiple of G.
// The same bound and outcome as wait_bounded; after a wait that ran out the
// counter is no multiple of G until it is cleared.
__device__ __forceinline__ bool grid_barrier(uint64_t *bar, uint32_t G, volatile int *abort, unsigned *err,
                                             uint64_t limit = WAIT_CYCLES) {
    // release: what this CTA's warps wrote before they arrived at this thread
    const uint64_t old = atom_add_u64(bar, 1);
    const uint64_t target = (old / G + 1) * G;
    const uint64_t t0 = sm100::clock_cycles();
    while (ld_acquire_u64(bar) < target) {
        if (*abort) return false;
        if (sm100::clock_cycles() - t0 > limit) {
            atomicOr(err, GLQ_DEVERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
    return true;
}

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

// True in one lane of a converged warp.  Copies, MMAs and commits take uniform
// operands: behind elect.sync the compiler knows that one lane is left, behind
// a test of the lane number it does not, and a wait + copy or MMA iteration
// takes twice as long (500 against 250 cycles).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// 1-D bulk copy of weights, which pass through L2 once: first to be evicted
// (measured: 6.2 against 5.8 TB/s over 600 MB).
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t r;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(r));
    return r;
}
__device__ __forceinline__ void bulk_g2s_once(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                              uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// ---------------------------------------------------------------------------
// The few-token pipeline.  The weights are the MMA's M side (128 rows), up to
// NT tokens its N side, one MMA group per 128-column block (K = 128: four
// instructions) into its own TMEM slot of NT columns, so that the MMA never
// waits for the sum over blocks, which the drain warps hold in registers:
// acc[token] += d * (token scale * block scale).  Roles:
//   warp 0       copies: the 16 KB weight tiles and, when the tokens were
//                rounded beforehand, their NT x 128 byte tiles
//   warp 1       MMA issue and TMEM allocation
//   warps 2-9    one block per warp in turn: the block's NT scales, and the
//                token tile itself when it is rounded on the way
//   warps 10-17  drain: warp & 3 is its TMEM lane quadrant (rows), the two
//                sets of four take half of the tokens each
// A stage is one weight tile, its token tile, its scales and its TMEM slot;
// three barriers carry it round:
//   full   the copies have landed and the scale warp has written -> MMA
//   done   the MMA has finished -> drain (weight copy of the next use)
//   empty  the drain has read it -> everything of the next use
// One commit per block and one polling lane per warp: with stages and slots
// apart and every lane polling, the MMA thread alone took 1150 cycles a block,
// against 700 for its share of the HBM rate.
// ---------------------------------------------------------------------------

constexpr int X_WARP0 = 2, X_WARPS = 8;
constexpr int D_WARP0 = 10, D_WARPS = 8;
constexpr int PIPE_THREADS = (D_WARP0 + D_WARPS) * 32;  // 576
constexpr int D_THREADS = D_WARPS * 32;

template <int NT>
struct Pipe {
    static constexpr int STAGE_BYTES = GLQ_FP8_TILE_BYTES + NT * 128;
    // as many as shared memory holds beside the parts buffer
    static constexpr int STAGES = NT == 16 ? 11 : NT == 32 ? 9 : 7;
    static constexpr int TMEM_COLS = NT == 16 ? 256 : 512;
    static_assert(STAGES * NT <= TMEM_COLS, "a slot per stage");
    static constexpr int HALF = NT / 2;     // tokens of one drain set
    static constexpr int DRAIN = 2;         // blocks a drain warp takes at once
    // Token-operand warps in turn.  A warp's next block is X_TURN after its
    // last, whose begin showed block (last - STAGES) drained; the parity of a
    // barrier tells phases apart only one back, so X_TURN may not exceed the
    // stages.
    static constexpr int X_TURN = STAGES < X_WARPS ? STAGES : X_WARPS;
    // parts of the tokens a CTA sums, in groups of four tokens (2 KB): from each
    // of C <= 8 CTAs ceil(NT / 4 / C) groups, all of them fewer than NT / 4 + C
    static constexpr int RED_BYTES = (NT / 4 + 7) * 128 * 16;
    static constexpr size_t SMEM_BYTES = 1024 + (size_t)STAGES * STAGE_BYTES + RED_BYTES;
    static_assert(SMEM_BYTES + 4096 <= 227 * 1024, "shared memory");

    uint64_t full[STAGES], done[STAGES], empty[STAGES], mma_done;
    // parts of a split tile, between the CTAs of a cluster: red_full the bytes
    // of the tokens this CTA sums have arrived, red_empty every CTA has summed
    // its tokens (the buffers may be written again)
    uint64_t red_full, red_empty;
    alignas(16) float sc[STAGES][NT];  // (read as float4) token scale * block scale
    uint32_t tmem;
    volatile int abort;

    // one warp; ctas: CTAs that share a tile
    __device__ __forceinline__ void init(int lane, int ctas) {
        if (lane < STAGES) {
            mbar_init(&full[lane], 2);
            mbar_init(&done[lane], 1);
            mbar_init(&empty[lane], D_WARPS);
        }
        if (lane == 0) {
            mbar_init(&mma_done, 1);
            mbar_init(&red_full, 1);
            mbar_init(&red_empty, ctas * D_WARPS);
            abort = 0;
        }
    }
    template <bool CLUSTER = false>
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, unsigned *err) {
        return wait_bounded<CLUSTER>(bar, parity, &abort, err);
    }
    // The same for a whole warp: one lane waits and __syncwarp orders the
    // others after it.  A poll by all 32 lanes takes the mbarrier unit 32
    // turns: every wait of the CTA then takes hundreds of cycles.
    template <bool CLUSTER = false>
    __device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, unsigned *err) {
        bool ok = true;
        if ((threadIdx.x & 31) == 0) ok = wait<CLUSTER>(bar, parity, err);
        __syncwarp();
        return __shfl_sync(0xffffffffu, ok, 0);
    }
};

// The copy thread's place in the ring; it keeps running indices and pointers:
// with a division or a remainder in its loop a copy took 570 cycles instead of
// 300, and the copies in flight never covered the memory's latency.
template <int NT>
struct Loader {
    uint32_t stage = 0, parity = 1;  // of the wait for the stage's last use
    uint8_t *dst;                    // the stage's weight tile
    uint8_t *smem;
    uint64_t policy;
    __device__ __forceinline__ explicit Loader(uint8_t *s) : dst(s), smem(s), policy(evict_first_policy()) {}
    __device__ __forceinline__ void next() {
        dst += Pipe<NT>::STAGE_BYTES;
        if (++stage == Pipe<NT>::STAGES) stage = 0, parity ^= 1, dst = smem;
    }
};

// The copy thread: waits for its stage and starts its weight tile; extra:
// bytes that other copies will bring for the block.  Where the token tile is
// written by a warp, that warp has waited for the drain and the copy may start
// when the MMA has finished with the tile; else the drain of the TMEM slot is
// waited for here.
template <int NT, bool X_WRITTEN>
__device__ __forceinline__ bool pipe_load(Pipe<NT> &p, const Loader<NT> &l, const uint8_t *tile, uint32_t extra,
                                          unsigned *err) {
    if (!p.wait(X_WRITTEN ? &p.done[l.stage] : &p.empty[l.stage], l.parity, err)) return false;
    mbar_expect_tx(&p.full[l.stage], GLQ_FP8_TILE_BYTES + extra);
    bulk_g2s_once(l.dst, tile, GLQ_FP8_TILE_BYTES, &p.full[l.stage], l.policy);
    return true;
}
template <int NT>
__device__ __forceinline__ uint8_t *pipe_x_tile(uint8_t *smem, uint32_t it) {
    return smem + (it % Pipe<NT>::STAGES) * Pipe<NT>::STAGE_BYTES + GLQ_FP8_TILE_BYTES;
}

// Before the CTA exits, if it gave up: let the copies of the last blocks land
// (`loaded` blocks were started; an earlier use of a stage has landed, or it
// would not have been loaded again).  A block whose scale warp stopped never
// completes: its wait runs out, long after any copy has landed.
template <int NT>
__device__ __forceinline__ void pipe_load_drain(Pipe<NT> &p, uint32_t loaded) {
    for (uint32_t i = loaded > (uint32_t)Pipe<NT>::STAGES ? loaded - Pipe<NT>::STAGES : 0; i < loaded; ++i)
        sm100::mbar_wait(&p.full[i % Pipe<NT>::STAGES], (i / Pipe<NT>::STAGES) & 1, WAIT_CYCLES / 64);
}

// The MMA warp's one thread: blocks [it, it + count).
template <int NT>
__device__ __forceinline__ bool pipe_mma(Pipe<NT> &p, uint8_t *smem, uint32_t it, uint32_t count, unsigned *err) {
    const uint32_t idesc = idesc_e4m3_f32(128, NT);
    const uint32_t tmem = p.tmem;
    uint32_t s = it % Pipe<NT>::STAGES, par = (it / Pipe<NT>::STAGES) & 1;
    for (uint32_t i = 0; i < count; ++i) {
        if (!p.wait(&p.full[s], par, err)) return false;
        sm100::tc_fence_after();
        uint8_t *st = smem + s * Pipe<NT>::STAGE_BYTES;
        const uint64_t a = sm100::smem_desc_sw128(st), b = sm100::smem_desc_sw128(st + GLQ_FP8_TILE_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_f8_ss(tmem + s * NT, a + 2 * kk, b + 2 * kk, idesc, kk);
        sm100::mma_commit(&p.done[s]);
        if (++s == Pipe<NT>::STAGES) s = 0, par ^= 1;
    }
    return true;
}

// A scale / token warp before it writes block `it`: its stage has been
// drained.  After the writes: pipe_x_done.
template <int NT>
__device__ __forceinline__ bool pipe_x_begin(Pipe<NT> &p, uint32_t it, unsigned *err) {
    return p.wait_warp(&p.empty[it % Pipe<NT>::STAGES], ((it / Pipe<NT>::STAGES) & 1) ^ 1, err);
}
template <int NT, bool X_WRITTEN>
__device__ __forceinline__ void pipe_x_done(Pipe<NT> &p, uint32_t it, int lane) {
    if (X_WRITTEN) sm100::fence_proxy_async_smem();  // the MMA reads the tile through the async proxy
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&p.full[it % Pipe<NT>::STAGES]);
}

// A drain warp: adds blocks it .. it + N - 1 to acc (its half of the tokens).
// The last block's wait covers the others (MMAs complete in order); several
// blocks share its cost, about 300 cycles for wait, TMEM load and arrive (one
// block at a time, 64 tokens of 32768x5120 took 37.6 us instead of 34.8; three
// or four keep too many stages waiting: 40.0).
template <int NT, int N>
__device__ __forceinline__ bool pipe_drain(Pipe<NT> &p, uint32_t it, int quadrant, int set, float (&acc)[NT / 2],
                                           unsigned *err) {
    constexpr int HALF = NT / 2, STAGES = Pipe<NT>::STAGES;
    constexpr int STEP = HALF < 16 ? HALF : 16;
    const uint32_t last = it + N - 1;
    if (!p.wait_warp(&p.done[last % STAGES], (last / STAGES) & 1, err)) return false;
    sm100::tc_fence_after();
    const uint32_t t0 = p.tmem + ((uint32_t)(32 * quadrant) << 16) + set * HALF;
    uint32_t s[N];
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] = (it + n) % STAGES;
#pragma unroll
    for (int c = 0; c < HALF; c += STEP) {
        uint32_t d[N][STEP];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (STEP == 8) tmem_ld8(t0 + s[n] * NT + c, d[n]);
            else if constexpr (STEP == 16) sm100::tmem_ld16(t0 + s[n] * NT + c, d[n]);
            else sm100::tmem_ld32(t0 + s[n] * NT + c, d[n]);
        }
        sm100::tmem_wait_ld();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float4 *sc = reinterpret_cast<const float4 *>(&p.sc[s[n]][set * HALF + c]);
#pragma unroll
            for (int j = 0; j < STEP; j += 4) {
                const float4 f = sc[j >> 2];
                const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int l = 0; l < 4; ++l) acc[c + j + l] = fmaf(__uint_as_float(d[n][j + l]), fs[l], acc[c + j + l]);
            }
        }
    }
    sm100::tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int n = 0; n < N; ++n) sm100::mbar_arrive(&p.empty[s[n]]);
    }
    return true;
}

// Address of this CTA's shared memory location `local` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_smem(const void *local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(local)), "r"(rank));
    return r;
}
// Stores into another CTA's shared memory that count their bytes on a barrier
// there: the reader waits for the data itself, no store has to be
// acknowledged before an arrival may follow it.
__device__ __forceinline__ void st_async(uint32_t addr, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_async4(uint32_t addr, const float *v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(
                     addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Blocks dealt out evenly: CTA c of G owns [c total / G, (c + 1) total / G).
// (total < 2^31: the blocks of 2^31 would fill more than the device's memory)
__device__ __forceinline__ uint32_t range_begin(uint32_t c, uint32_t total, uint32_t G) {
    return (uint32_t)((uint64_t)c * total / G);
}
// the CTA that owns block b
__device__ __forceinline__ int range_owner(uint32_t b, uint32_t total, uint32_t G) {
    if (total <= 0xFFFFFFFFu / G) return (int)(((b + 1) * G - 1) / total);  // a 64-bit division takes four times as long
    return (int)((((uint64_t)b + 1) * G - 1) / total);
}

__device__ __forceinline__ void store_y(void *y, int dtype, int64_t i, float v) {
    if (dtype == 1) static_cast<__nv_bfloat16 *>(y)[i] = __float2bfloat16_rn(v);
    else if (dtype == 0) static_cast<__half *>(y)[i] = __float2half_rn(v);
    else static_cast<float *>(y)[i] = v;
}

// four consecutive outputs, i a multiple of 4
__device__ __forceinline__ void store_y4(void *y, int dtype, int64_t i, float4 v) {
    if (dtype == 2) {
        *reinterpret_cast<float4 *>(static_cast<float *>(y) + i) = v;
        return;
    }
    uint2 w;
    if (dtype == 1) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
        w = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(y) + i) = w;
}

}  // namespace fp8
}  // namespace glq
