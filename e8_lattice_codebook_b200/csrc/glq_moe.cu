// glq_moe.cu -- a mixture-of-experts layer for a few tokens in one kernel.
//
//     y[t] = sum over t's experts e of  p[t][e] down_e h^_e(t),
//     h_e(t) = silu(gate_e x^(t)) * (up_e x^(t)),
//
// x^ and h^ the e4m3 roundings of x and h (a scale per token and 128 columns),
// the matrices e4m3 with a scale per 128 x 128 block, p the softmax (or
// sigmoid) of the token's chosen router logits.
//
// Bound by HBM: the weights of every chosen expert are read once, 16 KB tile
// by tile (glq_fp8.h), by the few-token pipeline of glq_fp8.cuh, whose MMA
// takes all tokens as its N side whichever expert the tile belongs to (the
// tensor cores have time to spare; a token that did not choose the expert is
// dropped when the result is read).  The tiles of a phase form one sequence,
// dealt out evenly over the CTAs, one per SM, so that an odd number of experts
// or rows leaves no SM idle; a tile that falls to two or more CTAs is summed
// by whoever reads it, in the order of the CTAs.  Phases, with a barrier over
// the grid (a cooperative launch) after each:
//   0  every CTA: the routing of all tokens, for itself; a share of x^
//   1  gate and up tiles -> fp32 sums per (token, expert)
//   h  silu, product, rounding -> h^ as operand tiles
//   2  down tiles -> sums per token over experts; whole tiles go to y
//   y  the tiles of y that were split
// The copy warp runs ahead across the barriers: while a CTA waits, its first
// stages of the next phase's weights (up to 11 x 16 KB) are on their way.
#include "glq_fp8.cuh"
#include "glq_kernels.cuh"

namespace glq {

namespace {

using namespace fp8;

constexpr int WARPS = D_WARP0 + D_WARPS + 1;  // the pipeline's and one that keeps the grid's barriers
constexpr int THREADS = WARPS * 32;           // 608
constexpr int GRID_WARP = WARPS - 1;
constexpr int H_WARPS = X_WARPS + D_WARPS;    // warps that form h^
constexpr uint8_t NONE = 0xFF;
constexpr int LOCAL_T = 4;

// Shared memory behind the stages.
struct Layout {
    uint32_t mask, wts, rank, list, ids, slot, end;
};
__host__ __device__ inline Layout layout_of(uint32_t base, int nt, int T, int E, int k) {
    const int most = E < T * k ? E : T * k;  // experts in use, at most
    Layout l;
    l.mask = base;                                  // [E] 64-bit: tokens that chose the expert
    l.wts = l.mask + (uint32_t)E * 8;               // [T][k] fp32: p
    l.rank = l.wts + (uint32_t)(T * k) * 4;         // [E] 16-bit: place among the experts in use
    l.list = l.rank + (uint32_t)E * 2;              // [most] 16-bit: experts in use
    l.ids = l.list + (uint32_t)most * 2;            // [T][k] 16-bit: chosen experts, -1 none
    l.slot = (l.ids + (uint32_t)(T * k) * 2 + 15) & ~15u;  // [most][nt]: which of t's choices, or NONE
    l.end = l.slot + (uint32_t)most * nt;
    return l;
}

// Monotonic key of a logit: larger for larger values, 0 for those never chosen
// (NaN, -inf); -0 counts as 0.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (!(v > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float load_logit(const MoeParams &p, int64_t i) {
    if (p.logits_dtype == 2) return __ldg(static_cast<const float *>(p.logits) + i);
    if (p.logits_dtype == 1) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p.logits)[i]);
    return __half2float(static_cast<const __half *>(p.logits)[i]);
}

// One warp: the k largest logits of token t, ties to the lowest index, and
// their weights.  Lane l has experts l, l + 32, ... (NV of them).
template <int NV>
__device__ __forceinline__ void route(const MoeParams &p, int t, int lane, int16_t *ids, float *wts,
                                      unsigned long long *mask) {
    uint32_t key[NV];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = i * 32 + lane;
        key[i] = e < p.E ? logit_key(load_logit(p, (int64_t)t * p.E + e)) : 0;
    }
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) best = max(best, key[i]);
    const float top = key_logit(__reduce_max_sync(0xffffffffu, best));
    if (!p.renormalize && p.scoring == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (key[i]) sum += expf(key_logit(key[i]) - top);
        sum = warp_sum(sum);
    }
    uint32_t mine = 0, expert = 0;  // lane j: choice j's key and index
    for (int j = 0; j < p.k; ++j) {
        best = 0;
        uint32_t at = 0;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)  // downwards: the lowest index of equals stays
            if (key[i] >= best) best = key[i], at = i * 32 + lane;
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m == 0) break;  // nothing left to choose
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == m ? at : 0xFFFFFFFFu);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((uint32_t)(i * 32 + lane) == e) key[i] = 0;
        if (lane == j) mine = m, expert = e;
    }
    const float l = key_logit(mine);
    float w = 0.f;
    if (mine) w = p.scoring == 0 ? expf(l - top) : 1.f / (1.f + expf(-l));
    if (p.renormalize) sum = warp_sum(w);
    if (p.renormalize || p.scoring == 0) w = w / sum;
    if (lane < p.k) {
        ids[lane] = mine ? (int16_t)expert : (int16_t)-1;
        wts[lane] = w * p.routed_scale;
        if (mine) atomicOr(mask + expert, 1ull << t);
    }
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

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

__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

// A scale warp, block i: the group w of T tokens rounded into the operand tile.
template <int NT, typename T16>
__device__ __forceinline__ bool put_rounded(Pipe<NT> &pipe, uint8_t *smem, uint32_t i, const uint2 (&w)[LOCAL_T], int T,
                                            float ws, int lane, unsigned *err) {
    float inv;
    const float s = warp_group_scales<T16, LOCAL_T>(w, T, lane, inv);
    if (!pipe_x_begin(pipe, i, err)) return false;
    uint8_t *xt = pipe_x_tile<NT>(smem, i);
    if (lane < NT) pipe.sc[i % Pipe<NT>::STAGES][lane] = lane < T ? s * ws : 0.f;
#pragma unroll
    for (int t = 0; t < LOCAL_T; ++t) {
        if (t >= T) break;
        *reinterpret_cast<uint32_t *>(xt + sw128(t, lane >> 2) + (lane & 3) * 4) =
            round4<T16>(w[t], __shfl_sync(0xffffffffu, inv, t));
    }
    pipe_x_done<NT, true>(pipe, i, lane);
    return true;
}

// LOCAL (at most LOCAL_T tokens): x^ and h^ are not shared through memory;
// every CTA rounds the tokens' columns that its own blocks need into its
// operand tiles.  The work is done several times over, but two of the four
// barriers, 2 to 4 us each while the weights saturate the memory, and h's trip
// through memory go.
template <int NT, bool LOCAL>
__global__ void __launch_bounds__(THREADS, 1) moe_kernel(MoeParams p) {
    using P = Pipe<NT>;
    constexpr int HALF = NT / 2, STAGES = P::STAGES, DRAIN = P::DRAIN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) P pipe;
    // grid[n]: the grid's barrier n has been passed.  part1, formed, part2:
    // this CTA's warps have written their share of the phase.
    __shared__ uint64_t grid_bar[4], part1, formed, part2;
    __shared__ int s_count;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, G = gridDim.x;
    const int T = p.T, E = p.E, K = p.k;
    const Layout at = layout_of(STAGES * P::STAGE_BYTES, NT, T, E, K);
    unsigned long long *mask = reinterpret_cast<unsigned long long *>(smem + at.mask);
    float *wts = reinterpret_cast<float *>(smem + at.wts);
    int16_t *rank = reinterpret_cast<int16_t *>(smem + at.rank), *list = reinterpret_cast<int16_t *>(smem + at.list);
    int16_t *ids = reinterpret_cast<int16_t *>(smem + at.ids);
    uint8_t *slot = smem + at.slot;

    // ---------------- phase 0: setup, x^, routing ----------------
    if (warp == 0) {
        pipe.init(lane, 1);
        if (lane == 0) {
            for (int i = 0; i < 4; ++i) mbar_init(&grid_bar[i], 1);
            mbar_init(&part1, D_WARPS);
            mbar_init(&formed, H_WARPS);
            mbar_init(&part2, D_WARPS);
        }
    }
    if (warp == 1) {
        sm100::tmem_alloc(&pipe.tmem, P::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    for (int e = tid; e < E; e += THREADS) mask[e] = 0;
    for (int i = tid; i < (int)(at.end - at.slot) / 4; i += THREADS) reinterpret_cast<uint32_t *>(slot)[i] = 0xFFFFFFFFu;
    if (tid == 0) prefetch_l2(p.bar);  // before the weights are in flight
    // this CTA's share of x^: a warp per token and group
    if constexpr (!LOCAL)
    for (int i = warp * G + cta; i < T * p.KB1; i += WARPS * G) {
        const int t = i / p.KB1, kb = i - t * p.KB1, col = kb * GLQ_FP8_BLOCK + lane * 4;
        uint2 w = make_uint2(0, 0);  // d is a multiple of 8: a lane's four columns are in or out together
        if (col < p.d) w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.x) + (int64_t)t * p.d + col));
        const float2 a = p.x_dtype ? unpack2<__nv_bfloat16>(w.x) : unpack2<__half>(w.x);
        const float2 b = p.x_dtype ? unpack2<__nv_bfloat16>(w.y) : unpack2<__half>(w.y);
        const float v[4] = {a.x, a.y, b.x, b.y};
        float s;
        const uint32_t q = warp_quantize(v, s);
        __stcg(reinterpret_cast<uint32_t *>(p.xq + (int64_t)kb * (NT * 128) + sw128(t, lane >> 2)) + (lane & 3), q);
        if (lane == 0) __stcg(p.xs + kb * NT + t, s);
    }
    if (!LOCAL) fence_proxy_async();  // x^ is read by bulk copies
    __syncthreads();
    for (int t = warp; t < T; t += WARPS) {
        if (E <= 128) route<4>(p, t, lane, ids + t * K, wts + t * K, mask);
        else route<16>(p, t, lane, ids + t * K, wts + t * K, mask);
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    if (warp == 0) {  // experts in use, in order
        int n = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const bool used = e0 + lane < E && mask[e0 + lane] != 0;
            const unsigned b = __ballot_sync(0xffffffffu, used);
            if (used) {
                const int r = n + __popc(b & ((1u << lane) - 1));
                rank[e0 + lane] = (int16_t)r;
                list[r] = (int16_t)(e0 + lane);
            }
            n += __popc(b);
        }
        if (lane == 0) s_count = n;
    }
    __syncthreads();
    for (int i = tid; i < T * K; i += THREADS)
        if (ids[i] >= 0) slot[rank[ids[i]] * NT + i / K] = (uint8_t)(i % K);
    __syncthreads();

    const uint32_t A = s_count, R1 = 2 * p.IB, KB1 = p.KB1, IB = p.IB, DB = p.DB, K2 = A * IB;
    const uint32_t total1 = A * R1 * KB1, total2 = DB * K2;
    // CTAs that take part in each phase: as many as there are blocks, so that
    // none between the first and the last of a tile is without one
    const uint32_t G1 = min((uint32_t)G, total1), G2 = min((uint32_t)G, total2);
    const uint32_t b1 = cta < (int)G1 ? range_begin(cta, total1, G1) : 0;
    const uint32_t n1 = cta < (int)G1 ? range_begin(cta + 1, total1, G1) - b1 : 0;
    const uint32_t b2 = cta < (int)G2 ? range_begin(cta, total2, G2) : 0;
    const uint32_t n2 = cta < (int)G2 ? range_begin(cta + 1, total2, G2) - b2 : 0;
    uint32_t it = 0;  // the copy thread: blocks whose copies have been started
    bool copier = false;

    if (A == 0) {  // no token has an expert (the same in every CTA)
        for (int64_t i = (int64_t)cta * THREADS + tid; i < (int64_t)T * p.d; i += (int64_t)G * THREADS)
            store_y(p.y, p.y_dtype, i, 0.f);
    } else if (warp == 0) {
        if (elect_one()) {
            copier = true;
            Loader<NT> ld(smem);
            // A phase's blocks in order: weight tiles from w, in runs of `run`
            // blocks that follow one another; seek(b) finds block b's tile and
            // what is left of its run.  The token tiles, `xs_` of them in turn
            // from `x`, exist once `bar` completes.
            auto phase = [&](uint32_t b, uint32_t n, uint64_t *bar, auto seek, const uint8_t *x, uint32_t xs_) {
                const uint32_t ahead = LOCAL ? n : min(n, (uint32_t)STAGES);
                Loader<NT> lx = ld;
                const uint8_t *w = nullptr;
                uint32_t left = 0;
                auto load = [&](uint32_t i) {
                    if (left == 0) seek(b + i, w, left);
                    if (!pipe_load<NT, LOCAL>(pipe, ld, w, LOCAL ? 0 : NT * 128, p.err)) return false;
                    w += GLQ_FP8_TILE_BYTES;
                    --left;
                    ++it;
                    ld.next();
                    return true;
                };
                for (uint32_t i = 0; i < ahead; ++i)
                    if (!load(i)) return false;
                if (LOCAL) return true;
                if (!pipe.wait(bar, 0, p.err)) return false;
                fence_proxy_async();
                uint32_t xi = b % xs_;
                for (uint32_t i = 0; i < n; ++i) {
                    if (i >= ahead && !load(i)) return false;
                    bulk_g2s(lx.dst + GLQ_FP8_TILE_BYTES, x + (int64_t)xi * (NT * 128), NT * 128, &pipe.full[lx.stage]);
                    if (++xi == xs_) xi = 0;
                    lx.next();
                }
                return true;
            };
            // (an expert's gate and up tiles, and a row block of its down tiles,
            // lie in the order of the blocks)
            const bool ok = phase(
                b1, n1, &grid_bar[0],
                [&](uint32_t b, const uint8_t *&w, uint32_t &left) {
                    const uint32_t per = R1 * KB1, a = b / per, k = b - a * per;
                    w = p.w13 + ((int64_t)list[a] * per + k) * GLQ_FP8_TILE_BYTES;
                    left = per - k;
                },
                p.xq, KB1);
            if (ok)
                phase(
                    b2, n2, &grid_bar[2],
                    [&](uint32_t b, const uint8_t *&w, uint32_t &left) {
                        const uint32_t rt = b / K2, k = b - rt * K2, a = k / IB, ib = k - a * IB;
                        w = p.w2 + (((int64_t)list[a] * DB + rt) * IB + ib) * GLQ_FP8_TILE_BYTES;
                        left = IB - ib;
                    },
                    p.hq, K2);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            pipe_mma<NT>(pipe, smem, 0, n1 + n2, p.err);
            sm100::mma_commit(&pipe.mma_done);  // every MMA issued has completed
            sm100::mbar_wait(&pipe.mma_done, 0, WAIT_CYCLES);
        }
    } else if (warp == GRID_WARP) {
        if (lane == 0) {
            uint64_t *const mine[4] = {nullptr, &part1, &formed, &part2};
            for (int n = LOCAL ? 1 : 0; n < 4; n += LOCAL ? 2 : 1) {
                if (mine[n] && !pipe.wait(mine[n], 0, p.err)) break;
                // release: what this CTA's warps wrote before they arrived
                const uint64_t old = atom_add_u64(p.bar, 1);
                const uint64_t target = (old / G + 1) * G;  // every call adds a multiple of G
                const uint64_t t0 = sm100::clock_cycles();
                bool ok = true;
                while (ok && ld_acquire_u64(p.bar) < target) {
                    if (pipe.abort) ok = false;
                    else if (sm100::clock_cycles() - t0 > WAIT_CYCLES) pipe.fail(p.err), ok = false;
                }
                if (!ok) break;
                sm100::mbar_arrive(&grid_bar[n]);
            }
        }
    } else {
        // One warp: four columns per lane of h of token t for expert a (its place
        // among those in use; s = t K + which of t's choices), group ib.
        auto expert_h = [&](uint32_t a, int s, int t, int ib, float (&h)[4]) {
            float4 v[2], more[2];
            int c0[2], c1[2];
            const float *spill = p.spill + (int64_t)t * 128 + lane * 4;
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // gate, up: every load before the first sum
                const uint32_t r = 2 * ib + g, first = (a * R1 + r) * KB1;
                c0[g] = range_owner(first, total1, G1), c1[g] = range_owner(first + KB1 - 1, total1, G1);
                v[g] = __ldcg(reinterpret_cast<const float4 *>(p.main + ((int64_t)s * R1 + r) * 128 + lane * 4));
                more[g] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c1[g] > c0[g]) more[g] = __ldcg(reinterpret_cast<const float4 *>(spill + (int64_t)(c0[g] + 1) * NT * 128));
            }
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                v[g] = add4(v[g], more[g]);
#pragma unroll 4
                for (int c = c0[g] + 2; c <= c1[g]; ++c)
                    v[g] = add4(v[g], __ldcg(reinterpret_cast<const float4 *>(spill + (int64_t)c * NT * 128)));
            }
            h[0] = silu(v[0].x) * v[1].x;
            h[1] = silu(v[0].y) * v[1].y;
            h[2] = silu(v[0].z) * v[1].z;
            h[3] = silu(v[0].w) * v[1].w;
        };
        // h^: a warp per (token, choice) and group of the expert's width
        auto form = [&]() {
            if (!pipe.wait_warp(&grid_bar[1], 0, p.err)) return false;
            for (int i = (warp - X_WARP0) * G + cta; i < T * K * (int)IB; i += H_WARPS * G) {
                const int s = i / (int)IB, ib = i - s * (int)IB, e = ids[s], t = s / K;
                if (e < 0) continue;
                const uint32_t a = rank[e];
                float h[4], sc;
                expert_h(a, s, t, ib, h);
                const uint32_t q = warp_quantize(h, sc);
                const int64_t tile = (int64_t)a * IB + ib;
                __stcg(reinterpret_cast<uint32_t *>(p.hq + tile * (NT * 128) + sw128(t, lane >> 2)) + (lane & 3), q);
                if (lane == 0) __stcg(p.hs + tile * NT + t, sc * wts[s]);
            }
            fence_proxy_async();  // h^ is read by bulk copies
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&formed);
            return true;
        };
        if (warp < D_WARP0) {
            // ---------------- scales ----------------
            constexpr int SC = (NT + 31) / 32;
            const uint32_t turn = P::X_TURN, w0 = warp - X_WARP0;
            auto put = [&](uint32_t i, const float (&s)[SC]) {
                if (!pipe_x_begin(pipe, i, p.err)) return false;
#pragma unroll
                for (int j = 0; j < SC; ++j)
                    if (j * 32 + lane < NT) pipe.sc[i % STAGES][j * 32 + lane] = s[j];
                pipe_x_done<NT, false>(pipe, i, lane);
                return true;
            };
            // the block scales come from DRAM, behind the weights in flight: into L2
            // before those are too many
            for (uint32_t j = (w0 * 32 + lane) * 32; j < n1; j += X_WARPS * 32 * 32) {
                const uint32_t b = b1 + j, a = b / (R1 * KB1);
                prefetch_l2(p.s13 + (int64_t)list[a] * (R1 * KB1) + (b - a * (R1 * KB1)));
            }
            for (uint32_t j = w0 * 32 + lane; j < n2; j += X_WARPS * 32) {
                const uint32_t b = b2 + j, rt = b / K2, k = b - rt * K2, a = k / IB;
                prefetch_l2(p.s2 + ((int64_t)list[a] * DB + rt) * IB + (k - a * IB));
            }
            bool ok = LOCAL || pipe.wait_warp(&grid_bar[0], 0, p.err);
            uint32_t i = w0;
            if (w0 >= turn) i = n1 + n2;
            for (; ok && i < n1; i += turn) {
                const uint32_t b = b1 + i, a = b / (R1 * KB1), kb = b % KB1;
                const float ws = __ldg(p.s13 + (int64_t)list[a] * (R1 * KB1) + (b - a * (R1 * KB1)));
                if constexpr (LOCAL) {
                    const int col = kb * GLQ_FP8_BLOCK + lane * 4;
                    uint2 w[LOCAL_T];
#pragma unroll
                    for (int t = 0; t < LOCAL_T; ++t) {
                        w[t] = make_uint2(0, 0);
                        if (t < T && col < p.d)
                            w[t] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.x) + (int64_t)t * p.d + col));
                    }
                    ok = p.x_dtype ? put_rounded<NT, __nv_bfloat16>(pipe, smem, i, w, T, ws, lane, p.err)
                                   : put_rounded<NT, __half>(pipe, smem, i, w, T, ws, lane, p.err);
                } else {
                    float s[SC];
#pragma unroll
                    for (int j = 0; j < SC; ++j)
                        s[j] = j * 32 + lane < T ? __ldcg(p.xs + kb * NT + j * 32 + lane) * ws : 0.f;
                    ok = put(i, s);
                }
            }
            if constexpr (LOCAL) ok = ok && pipe.wait_warp(&grid_bar[1], 0, p.err);
            else ok = ok && form() && pipe.wait_warp(&grid_bar[2], 0, p.err);
            for (; ok && i < n1 + n2; i += turn) {
                const uint32_t b = b2 + (i - n1), rt = b / K2, k = b - rt * K2, a = k / IB, ib = k - a * IB;
                const float ws = __ldg(p.s2 + ((int64_t)list[a] * DB + rt) * IB + ib);
                float s[SC];
                if constexpr (LOCAL) {
                    if (!(ok = pipe_x_begin(pipe, i, p.err))) break;
                    uint8_t *xt = pipe_x_tile<NT>(smem, i);
                    s[0] = 0.f;
#pragma unroll 1
                    for (int t = 0; t < T; ++t) {  // rolled: it runs a few times a call, from a cold instruction cache
                        const uint8_t c = slot[a * NT + t];
                        if (c == NONE) continue;
                        float h[4], sc;
                        expert_h(a, t * K + c, t, ib, h);
                        *reinterpret_cast<uint32_t *>(xt + sw128(t, lane >> 2) + (lane & 3) * 4) = warp_quantize(h, sc);
                        if (lane == t) s[0] = sc * wts[t * K + c] * ws;
                    }
                    if (lane < NT) pipe.sc[i % STAGES][lane] = s[0];
                    pipe_x_done<NT, true>(pipe, i, lane);
                } else {
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        const int t = j * 32 + lane;
                        s[j] = t < T && slot[a * NT + t] != NONE ? __ldcg(p.hs + (int64_t)k * NT + t) * ws : 0.f;
                    }
                    ok = put(i, s);
                }
            }
        } else {
            // ---------------- drain ----------------
            const int quadrant = warp & 3, set = (warp - D_WARP0) >> 2;
            const int row = 32 * quadrant + lane, dtid = tid - D_WARP0 * 32;
            float acc[HALF];
            uint32_t i = 0;
            bool ok = true;
            // Phase 0: sums per (token, expert); the piece with a tile's first block
            // in `main`, a CTA's piece of an earlier CTA's tile in `spill`.  Phase
            // 1: sums per token; a CTA's piece of a split tile in `part`.
            auto phase = [&](auto skip, int ph) {
                constexpr bool SKIP = decltype(skip)::value;
                const uint32_t end = ph ? n1 + n2 : n1, KT = ph ? K2 : KB1, b = ph ? b2 : b1;
                uint32_t tile = b / KT, k = b - tile * KT;
                while (ok && i < end) {
                    const uint32_t len = min(KT - k, end - i);
#pragma unroll
                    for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
                    for (uint32_t n = 0; ok && n < len;) {
                        const bool two = DRAIN == 2 && n + 2 <= len;
                        ok = two ? pipe_drain<NT, DRAIN, SKIP>(pipe, i, quadrant, set, acc, p.err)
                                 : pipe_drain<NT, 1, SKIP>(pipe, i, quadrant, set, acc, p.err);
                        n += two ? 2 : 1;
                        i += two ? 2 : 1;
                    }
                    if (!ok) break;
                    const uint32_t a = tile / R1, r = tile - a * R1;   // phase 0
                    const bool whole = k == 0 && len == KT;            // phase 1
                    const int64_t col = (int64_t)tile * 128 + row;
                    float *part = p.part + ((int64_t)cta * 2 + (k == 0 ? 1 : 0)) * NT * 128 + row;
#pragma unroll
                    for (int j = 0; j < HALF; ++j) {
                        const int t = set * HALF + j;
                        if (t >= T) continue;
                        if (ph == 0) {
                            const uint8_t c = slot[a * NT + t];
                            if (c != NONE)
                                __stcg(k == 0 ? p.main + (((int64_t)t * K + c) * R1 + r) * 128 + row
                                              : p.spill + ((int64_t)cta * NT + t) * 128 + row, acc[j]);
                        } else if (!whole) {
                            __stcg(part + t * 128, acc[j]);
                        } else if (col < p.d) {
                            store_y(p.y, p.y_dtype, (int64_t)t * p.d + col, acc[j]);
                        }
                    }
                    ++tile;
                    k = 0;
                }
            };
            phase(std::false_type{}, 0);
            __syncwarp();
            if (ok && lane == 0) sm100::mbar_arrive(&part1);
            if (!LOCAL) ok = ok && form();
            phase(std::true_type{}, 1);
            __syncwarp();
            if (ok && lane == 0) sm100::mbar_arrive(&part2);
            ok = ok && pipe.wait_warp(&grid_bar[3], 0, p.err);
            // the tiles that were split: four columns of one token per thread
            for (int j = cta * (D_WARPS * 32) + dtid; ok && j < T * (int)DB * 32; j += G * D_WARPS * 32) {
                const int t = j / ((int)DB * 32), c4 = j - t * ((int)DB * 32), rt = c4 >> 5, col = c4 * 4;
                const uint32_t first = rt * K2;
                const int c0 = range_owner(first, total2, G2), c1 = range_owner(first + K2 - 1, total2, G2);
                if (c0 == c1 || col >= p.d) continue;
                const int64_t off = (int64_t)t * 128 + (c4 & 31) * 4;
                float4 sum = __ldcg(reinterpret_cast<const float4 *>(p.part + ((int64_t)c0 * 2 + 1) * NT * 128 + off));
#pragma unroll 4
                for (int c = c0 + 1; c <= c1; ++c)
                    sum = add4(sum, __ldcg(reinterpret_cast<const float4 *>(p.part + (int64_t)c * 2 * NT * 128 + off)));
                store_y4(p.y, p.y_dtype, (int64_t)t * p.d + col, sum);
            }
        }
    }
    // converged, or a warp whose one thread is still at work counts twice
    __syncwarp();
    sm100::tc_fence_before();
    __syncthreads();
    if (copier && pipe.abort) pipe_load_drain(pipe, it);
    __syncwarp();
    if (warp == 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(pipe.tmem, P::TMEM_COLS);
    }
}

struct MoeKernel {
    const void *fn;
    size_t smem;
    int key;
};

template <int NT, bool LOCAL>
MoeKernel moe_kernel_of(const MoeParams &p, int key) {
    return {(const void *)moe_kernel<NT, LOCAL>,
            1024 + layout_of(Pipe<NT>::STAGES * Pipe<NT>::STAGE_BYTES, NT, p.T, p.E, p.k).end, key};
}

}  // namespace

int moe_tile(int T) { return T <= 16 ? 16 : T <= 32 ? 32 : 64; }

cudaError_t launch_moe(const MoeParams &p, int grid, cudaStream_t s) {
    const int nt = moe_tile(p.T);
    const MoeKernel k = p.T <= LOCAL_T ? moe_kernel_of<16, true>(p, 0)
                        : nt == 16     ? moe_kernel_of<16, false>(p, 1)
                        : nt == 32     ? moe_kernel_of<32, false>(p, 2)
                                       : moe_kernel_of<64, false>(p, 3);
    static std::atomic<uint64_t> configured[4];
    const cudaError_t e = once_per_device(configured[k.key], [&k] {
        return cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, MOE_SMEM_LIMIT);
    });
    if (e != cudaSuccess) return e;
    if (k.smem > MOE_SMEM_LIMIT) return cudaErrorInvalidValue;
    MoeParams q = p;
    void *args[] = {&q};
    return cudaLaunchCooperativeKernel(k.fn, dim3(grid), dim3(THREADS), args, k.smem, s);
}

}  // namespace glq
