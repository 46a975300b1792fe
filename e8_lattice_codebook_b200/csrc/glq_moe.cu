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
// takes the expert's own tokens as its N side, one behind the other: with all
// tokens there the drain of a block took as long as an SM's share of the HBM
// (64 tokens of 32 experts of 4096 x 2048: 177 us instead of 148).  The tiles
// of a phase form one sequence, expert by expert, dealt out evenly over the
// CTAs, one per SM, so that an odd number of experts or rows leaves no SM idle;
// a tile that falls to two or more CTAs is summed by whoever reads it, in the
// order of the CTAs.  One token of 8 of 128 experts of 2048 x 768 takes 23.6 us,
// of which the weights need 5.8; 16 tokens, 28 experts of 4096 x 2048, 124 us =
// 5.7 TB/s.
// Phases, with a barrier over the grid (a cooperative launch) after each:
//   0  every CTA: the routing of all tokens, for itself; a share of x^
//   1  gate and up tiles -> fp32 sums per (token, expert)
//   h  silu, product, rounding -> h^ as operand tiles
//   2  down tiles -> fp32 sums per (token, expert)
//   y  their sum over the token's experts, in the order of its choices
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
constexpr int LOCAL_T = 4;

// Shared memory behind the stages.
struct Layout {
    uint32_t mask, wts, rank, ids, list, off, roff, pairs, end;
};
__host__ __device__ inline Layout layout_of(uint32_t base, int T, int E, int k) {
    const int most = E < T * k ? E : T * k;  // experts in use, at most
    Layout l;
    l.mask = base;                                  // [E] 64-bit: tokens that chose the expert
    l.wts = l.mask + (uint32_t)E * 8;               // [T][k] fp32: p
    l.rank = l.wts + (uint32_t)(T * k) * 4;         // [E] 16-bit: place among the experts in use
    l.ids = l.rank + (uint32_t)E * 2;               // [T][k] 16-bit: chosen experts, -1 none
    l.list = l.ids + (uint32_t)(T * k) * 2;         // [most] 16-bit: experts in use
    l.off = l.list + (uint32_t)most * 2;            // [most + 1] 16-bit: their tokens' first place in pairs
    l.roff = l.off + (uint32_t)(most + 1) * 2;      // [most + 1] 16-bit: the same with each rounded up to 8
    l.pairs = l.roff + (uint32_t)(most + 1) * 2;    // [T k] 16-bit: 16 t + which of t's choices, by expert
    l.end = l.pairs + (uint32_t)(T * k) * 2;
    return l;
}
static_assert(MOE_MAX_K <= 16 && MOE_MAX_T <= 64 && 8 * MOE_MAX_T * MOE_MAX_K < 65536, "16-bit tables");

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
    if (mine) {
        if (p.scoring == 0) w = expf(l - top);
        // The quotient of two scores is a number where the scores vanish in fp32
        // (logits below -87): relative to the largest, exp(l) = exp(top) exp(l -
        // top) having its factor in all of them.
        else if (p.renormalize) w = expf(fminf(l, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(l)));
        else w = 1.f / (1.f + expf(-l));
    }
    if (p.renormalize) sum = warp_sum(w);
    if (p.renormalize || p.scoring == 0) w = w / sum;
    if (lane < p.k) {
        ids[lane] = mine ? (int16_t)expert : (int16_t)-1;
        wts[lane] = w * p.routed_scale;
        if (mine) atomicOr(mask + expert, 1ull << t);
    }
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ float4 add4(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

// A scale warp, block i: the group w of `live` tokens rounded into the operand tile.
template <int NT, typename T16>
__device__ __forceinline__ bool put_rounded(Pipe<NT> &pipe, uint8_t *smem, uint32_t i, const uint2 (&w)[LOCAL_T],
                                            int live, float ws, int lane, unsigned *err) {
    float inv;
    const float s = warp_group_scales<T16, LOCAL_T>(w, live, lane, inv);
    if (!pipe_x_begin(pipe, i, err)) return false;
    uint8_t *xt = pipe_x_tile<NT>(smem, i);
    if (lane < NT) pipe.sc[i % Pipe<NT>::STAGES][lane] = lane < live ? s * ws : 0.f;
#pragma unroll
    for (int j = 0; j < LOCAL_T; ++j) {
        if (j >= live) break;
        *reinterpret_cast<uint32_t *>(xt + sw128(j, lane >> 2) + (lane & 3) * 4) =
            round4<T16>(w[j], __shfl_sync(0xffffffffu, inv, j));
    }
    pipe_x_done<NT, true>(pipe, i, lane);
    return true;
}

// What every CTA keeps for itself about the routing, and the barriers that do
// not depend on NT.
struct Routing {
    unsigned long long *mask;
    float *wts;
    int16_t *rank, *list, *ids;
    uint16_t *off, *roff, *pairs;
    uint32_t A;  // experts in use
    // token t's place among the tokens of expert e
    __device__ __forceinline__ int place(int e, int t) const { return __popcll(mask[e] & ((1ull << t) - 1)); }
};
struct Barriers {
    // grid[n]: the grid's barrier n has been passed.  part0, part1, formed,
    // part2: this CTA's warps have written their share of the phase.
    uint64_t grid[4], part0, part1, formed, part2;
};

// Everything behind the routing.
template <int NT, int MAX_NT, bool LOCAL>
__device__ __forceinline__ void moe_body(const MoeParams &p, const Routing &z, Barriers &bars, Pipe<NT> &pipe,
                                         uint8_t *smem, uint32_t tmem) {
    using P = Pipe<NT>;
    constexpr int HALF = NT / 2, STAGES = P::STAGES, DRAIN = P::DRAIN;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, G = gridDim.x;
    const int T = p.T, K = p.k;
    if constexpr (MAX_NT > 16) {  // (else it has been done)
        if (warp == 0) pipe.init(lane, 1);
        if (tid == 0) pipe.tmem = tmem;
        __syncthreads();
    }

    const uint32_t A = z.A, R1 = 2 * p.IB, KB1 = p.KB1, IB = p.IB, DB = p.DB;
    const uint32_t total1 = A * R1 * KB1, total2 = A * DB * IB;
    // CTAs that take part in each phase: as many as there are blocks, so that
    // none between the first and the last of a tile is without one
    const uint32_t G1 = min((uint32_t)G, total1), G2 = min((uint32_t)G, total2);
    const uint32_t b1 = cta < (int)G1 ? range_begin(cta, total1, G1) : 0;
    const uint32_t n1 = cta < (int)G1 ? range_begin(cta + 1, total1, G1) - b1 : 0;
    const uint32_t b2 = cta < (int)G2 ? range_begin(cta, total2, G2) : 0;
    const uint32_t n2 = cta < (int)G2 ? range_begin(cta + 1, total2, G2) - b2 : 0;
    uint32_t it = 0;  // the copy thread: blocks whose copies have been started
    bool copier = false;

    if (warp == 0) {
        if (elect_one()) {
            copier = true;
            Loader<NT> ld(smem);
            // A phase's blocks in order, R rows of KT blocks for each expert: the
            // weight tiles from w; the token tiles from x (each expert's KT of them
            // for every row) exist once `bar` completes.
            auto phase = [&](uint32_t b, uint32_t n, uint64_t *bar, const uint8_t *weights, const uint8_t *x, uint32_t R,
                             uint32_t KT) {
                const uint32_t ahead = LOCAL ? n : min(n, (uint32_t)STAGES), per = R * KT;
                Loader<NT> lx = ld;
                const uint8_t *w = nullptr;
                uint32_t a = b / per, left = 0, bytes = 0;
                auto load = [&](uint32_t i) {
                    if (left == 0) {
                        const uint32_t k = i == 0 ? b - a * per : 0;
                        if (i) ++a;
                        w = weights + ((int64_t)z.list[a] * per + k) * GLQ_FP8_TILE_BYTES;
                        left = per - k;
                        if (!LOCAL) bytes = (uint32_t)(z.roff[a + 1] - z.roff[a]) * 128;
                    }
                    if (!pipe_load<NT, LOCAL>(pipe, ld, w, bytes, p.err)) return false;
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
                uint32_t xa = b / per, xk = (b - xa * per) % KT, xleft = per - (b - xa * per);
                uint32_t xbytes = (uint32_t)(z.roff[xa + 1] - z.roff[xa]) * 128;
                const uint8_t *xe = x + (int64_t)z.roff[xa] * KT * 128, *xp = xe + xk * xbytes;
                for (uint32_t i = 0; i < n; ++i) {
                    if (i >= ahead && !load(i)) return false;
                    bulk_g2s(lx.dst + GLQ_FP8_TILE_BYTES, xp, xbytes, &pipe.full[lx.stage]);
                    lx.next();
                    xp += xbytes;
                    if (++xk == KT) xk = 0, xp = xe;
                    if (--xleft == 0 && i + 1 < n) {
                        ++xa;
                        xleft = per;
                        xbytes = (uint32_t)(z.roff[xa + 1] - z.roff[xa]) * 128;
                        xe = xp = x + (int64_t)z.roff[xa] * KT * 128;
                    }
                }
                return true;
            };
            if (n1 == 0 || phase(b1, n1, &bars.grid[0], p.w13, p.xq, R1, KB1))
                if (n2) phase(b2, n2, &bars.grid[2], p.w2, p.hq, DB, IB);
        }
    } else if (warp == 1) {
        if (elect_one()) {
            pipe_mma<NT>(pipe, smem, 0, n1 + n2, p.err);
            sm100::mma_commit(&pipe.mma_done);  // every MMA issued has completed
            sm100::mbar_wait(&pipe.mma_done, 0, WAIT_CYCLES);
        }
    } else if (warp == GRID_WARP) {
        if (lane == 0) {
            uint64_t *const mine[4] = {&bars.part0, &bars.part1, &bars.formed, &bars.part2};
            for (int n = LOCAL ? 1 : 0; n < 4; n += LOCAL ? 2 : 1) {
                if (!pipe.wait(mine[n], 0, p.err)) break;
                if (!grid_barrier(p.bar, G, &pipe.abort, p.err)) break;
                sm100::mbar_arrive(&bars.grid[n]);
            }
        }
    } else {
        // x^: a warp per token and group, into the tiles of the token's experts
        auto form_x = [&]() {
            for (int i = (warp - X_WARP0) * G + cta; i < T * (int)KB1; i += H_WARPS * G) {
                const int t = i / (int)KB1, kb = i - t * (int)KB1, col = kb * GLQ_FP8_BLOCK + lane * 4;
                uint2 w = make_uint2(0, 0);  // d is a multiple of 8: a lane's four columns are in or out together
                if (col < p.d)
                    w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.x) + (int64_t)t * p.d + col));
                const float2 a = p.x_dtype ? unpack2<__nv_bfloat16>(w.x) : unpack2<__half>(w.x);
                const float2 b = p.x_dtype ? unpack2<__nv_bfloat16>(w.y) : unpack2<__half>(w.y);
                const float v[4] = {a.x, a.y, b.x, b.y};
                float s;
                const uint32_t q = warp_quantize(v, s);
                for (int c = 0; c < K; ++c) {
                    const int e = z.ids[t * K + c];
                    if (e < 0) continue;
                    const uint32_t r = z.rank[e], ro = z.roff[r], rows = z.roff[r + 1] - ro;
                    uint8_t *tile = p.xq + ((int64_t)ro * KB1 + kb * rows) * 128;
                    __stcg(reinterpret_cast<uint32_t *>(tile + sw128(z.place(e, t), lane >> 2)) + (lane & 3), q);
                }
                if (lane == 0) __stcg(p.xs + kb * T + t, s);
            }
            fence_proxy_async();  // x^ is read by bulk copies
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&bars.part0);
        };
        // One warp: four columns per lane of h, group ib of the expert with place a,
        // for the token with place j among its own (s = t K + which of t's
        // choices).  The loads, and their sum:
        struct Sums {
            float4 v[2], more[2];  // gate, up
        };
        auto owners = [&](uint32_t a, int ib) {  // lanes 0 to 3: the CTAs with the first and last blocks of both tiles
            return range_owner((a * R1 + 2 * ib + ((lane >> 1) & 1)) * KB1 + (lane & 1 ? KB1 - 1 : 0), total1, G1);
        };
        auto load_h = [&](int owner, int s, int j, int ib) {
            Sums m;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int c0 = __shfl_sync(0xffffffffu, owner, 2 * g), c1 = __shfl_sync(0xffffffffu, owner, 2 * g + 1);
                m.v[g] = __ldcg(reinterpret_cast<const float4 *>(p.main1 + ((int64_t)s * R1 + 2 * ib + g) * 128 + lane * 4));
                m.more[g] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c1 > c0)
                    m.more[g] = __ldcg(reinterpret_cast<const float4 *>(p.spill1 + ((int64_t)(c0 + 1) * NT + j) * 128 + lane * 4));
            }
            return m;
        };
        auto finish_h = [&](Sums &m, int owner, int j, float (&h)[4]) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int c0 = __shfl_sync(0xffffffffu, owner, 2 * g), c1 = __shfl_sync(0xffffffffu, owner, 2 * g + 1);
                m.v[g] = add4(m.v[g], m.more[g]);
#pragma unroll 4
                for (int c = c0 + 2; c <= c1; ++c)
                    m.v[g] = add4(m.v[g], __ldcg(reinterpret_cast<const float4 *>(p.spill1 + ((int64_t)c * NT + j) * 128 + lane * 4)));
            }
            h[0] = silu(m.v[0].x) * m.v[1].x;
            h[1] = silu(m.v[0].y) * m.v[1].y;
            h[2] = silu(m.v[0].z) * m.v[1].z;
            h[3] = silu(m.v[0].w) * m.v[1].w;
        };
        // h^: a warp per (token, choice) and group of the expert's width
        auto form = [&]() {
            if (!pipe.wait_warp(&bars.grid[1], 0, p.err)) return false;
            for (int i = (warp - X_WARP0) * G + cta; i < T * K * (int)IB; i += H_WARPS * G) {
                const int s = i / (int)IB, ib = i - s * (int)IB, e = z.ids[s];
                if (e < 0) continue;
                const uint32_t a = z.rank[e], ro = z.roff[a], rows = z.roff[a + 1] - ro;
                const int j = z.place(e, s / K);
                float h[4], sc;
                const int owner = owners(a, ib);
                Sums m = load_h(owner, s, j, ib);
                finish_h(m, owner, j, h);
                const uint32_t q = warp_quantize(h, sc);
                const int64_t row0 = (int64_t)ro * IB + ib * rows;
                __stcg(reinterpret_cast<uint32_t *>(p.hq + row0 * 128 + sw128(j, lane >> 2)) + (lane & 3), q);
                if (lane == 0) __stcg(p.hs + row0 + j, sc * z.wts[s]);
            }
            fence_proxy_async();  // h^ is read by bulk copies
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&bars.formed);
            return true;
        };
        if constexpr (!LOCAL) form_x();
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
            auto prefetch = [&](const float *scales, uint32_t b, uint32_t n, uint32_t per) {
                for (uint32_t j = (w0 * 32 + lane) * 32; j < n; j += X_WARPS * 32 * 32) {
                    const uint32_t a = (b + j) / per;
                    prefetch_l2(scales + (int64_t)z.list[a] * per + (b + j - a * per));
                }
            };
            const uint32_t per1 = R1 * KB1, per2 = DB * IB;
            prefetch(p.s13, b1, n1, per1);
            prefetch(p.s2, b2, n2, per2);
            bool ok = LOCAL || pipe.wait_warp(&bars.grid[0], 0, p.err);
            uint32_t i = w0;
            if (w0 >= turn) i = n1 + n2;
            for (; ok && i < n1; i += turn) {
                const uint32_t b = b1 + i, a = b / per1, kb = b % KB1;
                const float ws = __ldg(p.s13 + (int64_t)z.list[a] * per1 + (b - a * per1));
                const int o = z.off[a], live = z.off[a + 1] - o;
                if constexpr (LOCAL) {
                    const int col = kb * GLQ_FP8_BLOCK + lane * 4;
                    uint2 w[LOCAL_T];
#pragma unroll
                    for (int j = 0; j < LOCAL_T; ++j) {
                        w[j] = make_uint2(0, 0);
                        if (j < live && col < p.d)
                            w[j] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.x) +
                                                                         (int64_t)(z.pairs[o + j] >> 4) * p.d + col));
                    }
                    ok = p.x_dtype ? put_rounded<NT, __nv_bfloat16>(pipe, smem, i, w, live, ws, lane, p.err)
                                   : put_rounded<NT, __half>(pipe, smem, i, w, live, ws, lane, p.err);
                } else {
                    float s[SC];
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        const int at_j = j * 32 + lane;
                        s[j] = at_j < live ? __ldcg(p.xs + kb * T + (z.pairs[o + at_j] >> 4)) * ws : 0.f;
                    }
                    ok = put(i, s);
                }
            }
            if constexpr (LOCAL) ok = ok && pipe.wait_warp(&bars.grid[1], 0, p.err);
            else ok = ok && form() && pipe.wait_warp(&bars.grid[2], 0, p.err);
            for (; ok && i < n1 + n2; i += turn) {
                const uint32_t b = b2 + (i - n1), a = b / per2, ib = b % IB;
                const float ws = __ldg(p.s2 + (int64_t)z.list[a] * per2 + (b - a * per2));
                const int o = z.off[a], live = z.off[a + 1] - o;
                float s[SC];
                if constexpr (LOCAL) {
                    const int owner = owners(a, ib);
                    auto choice = [&](int j) {
                        const int pair = z.pairs[o + j];
                        return (pair >> 4) * K + (pair & 15);
                    };
                    int c = choice(0);
                    Sums m = load_h(owner, c, 0, ib);
                    if (!(ok = pipe_x_begin(pipe, i, p.err))) break;
                    uint8_t *xt = pipe_x_tile<NT>(smem, i);
                    s[0] = 0.f;
#pragma unroll 1
                    for (int j = 0; j < live; ++j) {  // rolled: it runs a few times a call, from a cold instruction cache
                        const int next = choice(min(j + 1, live - 1));
                        Sums ahead = m;
                        if (j + 1 < live) ahead = load_h(owner, next, j + 1, ib);
                        float h[4], sc;
                        finish_h(m, owner, j, h);
                        *reinterpret_cast<uint32_t *>(xt + sw128(j, lane >> 2) + (lane & 3) * 4) = warp_quantize(h, sc);
                        if (lane == j) s[0] = sc * z.wts[c] * ws;
                        m = ahead, c = next;
                    }
                    if (lane < NT) pipe.sc[i % STAGES][lane] = s[0];
                    pipe_x_done<NT, true>(pipe, i, lane);
                } else {
                    const uint32_t ro = z.roff[a], rows = z.roff[a + 1] - ro;
                    const float *hs = p.hs + (int64_t)ro * IB + ib * rows;
#pragma unroll
                    for (int j = 0; j < SC; ++j) {
                        const int at_j = j * 32 + lane;
                        s[j] = at_j < live ? __ldcg(hs + at_j) * ws : 0.f;
                    }
                    ok = put(i, s);
                }
            }
        } else {
            // ---------------- drain ----------------
            const int quadrant = warp & 3, set = (warp - D_WARP0) >> 2;
            const int row = 32 * quadrant + lane;
            float acc[HALF];
            uint32_t i = 0;
            bool ok = true;
            // Sums per (token, expert) and row tile; the piece with a tile's first
            // block in `main`, a CTA's piece of an earlier CTA's tile in `spill`.
            auto phase = [&](uint32_t b, uint32_t end, uint32_t R, uint32_t KT, float *main, float *spill) {
                uint32_t tile = b / KT, k = b - tile * KT;
                while (ok && i < end) {
                    const uint32_t len = min(KT - k, end - i), a = tile / R, r = tile - a * R;
                    const int o = z.off[a], live = z.off[a + 1] - o;
#pragma unroll
                    for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
                    for (uint32_t n = 0; ok && n < len;) {
                        const bool two = n + DRAIN <= len;
                        ok = two ? pipe_drain<NT, DRAIN>(pipe, i, quadrant, set, acc, p.err)
                                 : pipe_drain<NT, 1>(pipe, i, quadrant, set, acc, p.err);
                        n += two ? DRAIN : 1;
                        i += two ? DRAIN : 1;
                    }
                    if (!ok) break;
#pragma unroll
                    for (int j = 0; j < HALF; ++j) {
                        const int at_j = set * HALF + j;
                        if (at_j >= live) break;
                        const int at_p = z.pairs[o + at_j];
                        __stcg(k == 0 ? main + ((int64_t)((at_p >> 4) * K + (at_p & 15)) * R + r) * 128 + row
                                      : spill + ((int64_t)cta * NT + at_j) * 128 + row, acc[j]);
                    }
                    ++tile;
                    k = 0;
                }
            };
            phase(b1, n1, R1, KB1, p.main1, p.spill1);
            __syncwarp();
            if (ok && lane == 0) sm100::mbar_arrive(&bars.part1);
            if (!LOCAL) ok = ok && form();
            phase(b2, n1 + n2, DB, IB, p.main2, p.spill2);
            __syncwarp();
            if (ok && lane == 0) sm100::mbar_arrive(&bars.part2);
            // y: a warp per token and 128 columns
            const int u0 = (warp - D_WARP0) * G + cta;
            for (int u = u0; ok && u < T * (int)DB; u += D_WARPS * G) {
                const int t = u / (int)DB, rt = u - t * (int)DB, col = rt * 128 + lane * 4;
                // lane c: choice c's pieces, and how many there are before them
                const int e = lane < K ? z.ids[t * K + lane] : -1;
                int c0 = 0, n = 0, at_j = 0;
                if (e >= 0) {
                    const uint32_t first = ((uint32_t)z.rank[e] * DB + rt) * IB;
                    c0 = range_owner(first, total2, G2), n = range_owner(first + IB - 1, total2, G2) - c0 + 1;
                    at_j = z.place(e, t);
                }
                int end = n;
#pragma unroll
                for (int d = 1; d < MOE_MAX_K; d <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, end, d);
                    if (lane >= d) end += v;
                }
                const int pieces = __shfl_sync(0xffffffffu, end, MOE_MAX_K - 1);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int base = 0; base < pieces || (base == 0 && u == u0); base += 32) {
                    // lane l: where piece base + l is, beside its columns
                    const float *from = p.main2;
                    for (int c = 0; c < K; ++c) {
                        const int ce = __shfl_sync(0xffffffffu, end, c), cn = __shfl_sync(0xffffffffu, n, c);
                        const int cc = __shfl_sync(0xffffffffu, c0, c), cj = __shfl_sync(0xffffffffu, at_j, c);
                        const int o = base + lane - (ce - cn);  // which of choice c's pieces
                        if (o == 0 && cn) from = p.main2 + ((int64_t)(t * K + c) * DB + rt) * 128;
                        if (o > 0 && o < cn) from = p.spill2 + ((int64_t)(cc + o) * NT + cj) * 128;
                    }
                    if (base == 0 && u == u0 && !(ok = pipe.wait_warp(&bars.grid[3], 0, p.err))) break;
                    const int here = min(32, pieces - base);
                    constexpr int Q = 8;  // loads in flight
                    for (int l = 0; l < here; l += Q) {
                        float4 v[Q];
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            const float *at_l = reinterpret_cast<const float *>(
                                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), (l + q) & 31));
                            v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (l + q < here) v[q] = __ldcg(reinterpret_cast<const float4 *>(at_l + lane * 4));
                        }
#pragma unroll
                        for (int q = 0; q < Q; ++q) sum = add4(sum, v[q]);
                    }
                }
                if (!ok) break;
                if (col < p.d) store_y4(p.y, p.y_dtype, (int64_t)t * p.d + col, sum);
            }
        }
    }
    // converged, or a warp whose one thread is still at work counts twice
    __syncwarp();
    __syncthreads();
    if (copier && pipe.abort) pipe_load_drain(pipe, it);
    __syncwarp();
}

union PipeSpace {  // one of them is used
    Pipe<16> few;
    Pipe<32> some;
    Pipe<64> many;
    __device__ PipeSpace() {}
};
constexpr size_t ring_bytes(int max_nt) {
    const size_t few = (size_t)Pipe<16>::STAGES * Pipe<16>::STAGE_BYTES, some = (size_t)Pipe<32>::STAGES * Pipe<32>::STAGE_BYTES,
                 many = (size_t)Pipe<64>::STAGES * Pipe<64>::STAGE_BYTES;
    return max_nt == 16 ? few : few > some ? (few > many ? few : many) : some > many ? some : many;
}

// LOCAL (at most LOCAL_T tokens): x^ and h^ are not shared through memory;
// every CTA rounds the tokens' columns that its own blocks need into its
// operand tiles.  The work is done several times over, but two of the four
// barriers, 2 to 4 us each while the weights saturate the memory, and h's trip
// through memory go.
//
// The body's NT is the smallest that holds the tokens of every expert; 64
// tokens rarely bring one expert more than 16.  A block of 16 tokens is drained
// in half the time of one of 64, two at a time (179 -> 148 us, as above; the
// number of stages, 8 to 11, makes no difference).
// LOCAL_T: 4 tokens of 128 experts of 2048 x 768 took 38 us (LOCAL) and 42 us,
// 8 tokens of 32 experts of 4096 x 2048 111 us and 101 us.
template <int MAX_NT, bool LOCAL>
__global__ void __launch_bounds__(THREADS, 1) moe_kernel(MoeParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(16) PipeSpace pipe_space;
    __shared__ uint32_t tmem;
    __shared__ Barriers bars;
    __shared__ int s_count, s_most;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, G = gridDim.x;
    const int T = p.T, E = p.E, K = p.k;
    const Layout at = layout_of((uint32_t)ring_bytes(MAX_NT), T, E, K);
    Routing z;
    z.mask = reinterpret_cast<unsigned long long *>(smem + at.mask);
    z.wts = reinterpret_cast<float *>(smem + at.wts);
    z.rank = reinterpret_cast<int16_t *>(smem + at.rank), z.list = reinterpret_cast<int16_t *>(smem + at.list);
    z.ids = reinterpret_cast<int16_t *>(smem + at.ids);
    z.off = reinterpret_cast<uint16_t *>(smem + at.off), z.roff = reinterpret_cast<uint16_t *>(smem + at.roff);
    z.pairs = reinterpret_cast<uint16_t *>(smem + at.pairs);

    // ---------------- setup, routing ----------------
    if (MAX_NT == 16 && warp == 2) pipe_space.few.init(lane, 1);
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(&bars.grid[i], 1);
        mbar_init(&bars.part0, H_WARPS);
        mbar_init(&bars.part1, D_WARPS);
        mbar_init(&bars.formed, H_WARPS);
        mbar_init(&bars.part2, D_WARPS);
    }
    if (warp == 1) {
        sm100::tmem_alloc(MAX_NT == 16 ? &pipe_space.few.tmem : &tmem, MAX_NT == 16 ? 256 : 512);
        sm100::tmem_relinquish();
    }
    for (int e = tid; e < E; e += THREADS) z.mask[e] = 0;
    if (tid == 0) prefetch_l2(p.bar);  // before the weights are in flight
    __syncthreads();
    for (int t = warp; t < T; t += WARPS) {
        if (E <= 128) route<4>(p, t, lane, z.ids + t * K, z.wts + t * K, z.mask);
        else route<16>(p, t, lane, z.ids + t * K, z.wts + t * K, z.mask);
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    if (warp == 0) {  // experts in use, in order, and where their tokens begin
        const int per = (E + 31) / 32, e0 = lane * per, e1 = min(E, e0 + per);  // a lane's experts
        int used = 0, sum = 0, most = 0;  // sum: tokens, and tokens rounded up to 8 in the upper half
        for (int e = e0; e < e1; ++e) {
            const int c = __popcll(z.mask[e]);
            used += c != 0, sum += c | ((c + 7) & ~7) << 16;
            if (MAX_NT > 16) most = max(most, c);
        }
        int n = used, o = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int a = __shfl_up_sync(0xffffffffu, n, d), b = __shfl_up_sync(0xffffffffu, o, d);
            if (lane >= d) n += a, o += b;
        }
        if (MAX_NT > 16) most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 31) s_count = n, s_most = most, z.off[n] = (uint16_t)(o & 0xFFFF), z.roff[n] = (uint16_t)(o >> 16);
        n -= used, o -= sum;  // of the lanes before
        for (int e = e0; used && e < e1; ++e) {
            const int c = __popcll(z.mask[e]);
            if (c == 0) continue;
            z.rank[e] = (int16_t)n;
            z.list[n] = (int16_t)e;
            z.off[n] = (uint16_t)(o & 0xFFFF), z.roff[n] = (uint16_t)(o >> 16);
            ++n, o += c | ((c + 7) & ~7) << 16;
        }
    }
    __syncthreads();
    for (int i = tid; i < T * K; i += THREADS) {
        const int e = z.ids[i], t = i / K;
        if (e >= 0) z.pairs[z.off[z.rank[e]] + z.place(e, t)] = (uint16_t)(t * 16 + (i - t * K));
    }
    __syncthreads();

    z.A = s_count;
    if (z.A == 0) {  // no token has an expert (the same in every CTA)
        for (int64_t i = (int64_t)cta * THREADS + tid; i < (int64_t)T * p.d; i += (int64_t)G * THREADS)
            store_y(p.y, p.y_dtype, i, 0.f);
    } else if constexpr (MAX_NT == 16) {
        moe_body<16, MAX_NT, LOCAL>(p, z, bars, pipe_space.few, smem, tmem);
    } else if (s_most <= 16) {
        moe_body<16, MAX_NT, LOCAL>(p, z, bars, pipe_space.few, smem, tmem);
    } else if (s_most <= 32) {
        moe_body<32, MAX_NT, LOCAL>(p, z, bars, pipe_space.some, smem, tmem);
    } else {
        moe_body<64, MAX_NT, LOCAL>(p, z, bars, pipe_space.many, smem, tmem);
    }
    sm100::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        sm100::tc_fence_after();
        sm100::tmem_dealloc(MAX_NT == 16 ? pipe_space.few.tmem : tmem, MAX_NT == 16 ? 256 : 512);
    }
}

struct MoeKernel {
    const void *fn;
    size_t smem;
    int key;
};

template <int MAX_NT, bool LOCAL>
MoeKernel moe_kernel_of(const MoeParams &p, int key) {
    return {(const void *)moe_kernel<MAX_NT, LOCAL>, 1024 + layout_of((uint32_t)ring_bytes(MAX_NT), p.T, p.E, p.k).end, key};
}

}  // namespace

int moe_tile(int T) { return T <= 16 ? 16 : 64; }

cudaError_t launch_moe(const MoeParams &p, int grid, cudaStream_t s) {
    const MoeKernel k = p.T <= LOCAL_T          ? moe_kernel_of<16, true>(p, 0)
                        : moe_tile(p.T) == 16 ? moe_kernel_of<16, false>(p, 1)
                                              : moe_kernel_of<64, false>(p, 2);
    static std::atomic<uint64_t> configured[3];
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
