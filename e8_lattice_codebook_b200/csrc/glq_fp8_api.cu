// glq_fp8_api.cu -- the C ABI of the 8-bit float operators (include/glq.h):
// argument checks, ownership of the laid-out weights, kernel choice.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <utility>

#include "../../include/glq.h"
#include "glq_fp8.h"
#include "glq_handles.h"

using glq::DeviceGuard;

namespace {

// most tokens of one launch; a call with more runs in slices of this many
constexpr int64_t MAX_SLICE = 8192;

int64_t blocks_of(int64_t v) { return (v + GLQ_FP8_BLOCK - 1) / GLQ_FP8_BLOCK; }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// One allocation for several arrays: sizes[i] bytes at *out[i], 256-byte
// aligned.  *out[0] is what cudaFree takes.
glq_status dev_alloc(std::initializer_list<std::pair<void **, size_t>> arrays, size_t *total) {
    size_t bytes = 0;
    for (const auto &a : arrays) bytes += (a.second + 255) & ~(size_t)255;
    char *p = nullptr;
    if (cudaMalloc((void **)&p, bytes) != cudaSuccess) {
        cudaGetLastError();
        return GLQ_ERR_OOM;
    }
    *total = bytes;
    for (const auto &a : arrays) {
        *a.first = p;
        p += (a.second + 255) & ~(size_t)255;
    }
    return GLQ_OK;
}

glq_status launched(cudaError_t e) {
    if (e == cudaSuccess) return GLQ_OK;
    cudaGetLastError();
    return GLQ_ERR_CUDA;
}

// TMA descriptor of rows [rows][cols] of `type` (`size` bytes each): boxes of
// 128 bytes x box_rows, zero fill past the last row; 128-byte swizzle, or none
// for weights that are laid out swizzled.
bool encode_rows(CUtensorMap *map, CUtensorMapDataType type, int size, const void *base, int64_t cols, int64_t rows,
                 int box_rows, bool swizzle = true) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        cudaDriverEntryPointQueryResult r;
        void *fn = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            fn = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(cols * size)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows};
    const cuuint32_t step[2] = {1, 1};
    return encode(map, type, 2, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_e4m3(CUtensorMap *map, const uint8_t *q, int64_t cols, int64_t rows, int box_rows, bool swizzle = true) {
    return encode_rows(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q, cols, rows, box_rows, swizzle);
}

void free_fp8(glq_fp8 L) {
    cudaFree(L->d_w);  // and what was allocated with it
    delete L;
}

bool rounds_inside(glq_fp8 L, int64_t B) { return glq::fp8_rounds_inside(B, L->RT, L->KB, L->num_sms); }

// The many-token kernel's tiles and parts of K.
glq::Fp8GemmParams gemm_params(glq_fp8 L, int64_t B) {
    glq::Fp8GemmParams p{};
    p.ws = L->d_ws;
    p.m = (int)L->m;
    p.B = (int)B;
    p.RT = L->RT;
    p.KB = L->KB;
    p.TT = (int)((B + glq::FP8_GEMM_TOK - 1) / glq::FP8_GEMM_TOK);
    p.tiles = (L->RT + 1) / 2 * p.TT;
    p.ksplit = glq::plan_fp8_gemm(p.tiles, p.KB, B, L->m, L->num_sms);
    p.part_rows = (int)((B + 31) / 32 * 32);  // stores come in boxes of 32 rows
    p.err = L->d_err;
    return p;
}

// What a call of B tokens needs of the shared workspace.
void fp8_need(glq_fp8 L, int64_t B, bool quantized, size_t need[glq::FP8_WS_COUNT]) {
    B = std::min(B, MAX_SLICE);
    if (B > glq::FP8_FEW) {
        const glq::Fp8GemmParams p = gemm_params(L, B);
        if (p.ksplit > 1)
            need[glq::FP8_WS_Z] =
                std::max(need[glq::FP8_WS_Z], (size_t)p.ksplit * p.part_rows * (size_t)L->m * sizeof(float));
    }
    if (B <= 0 || quantized || rounds_inside(L, B)) return;
    need[glq::FP8_WS_Q] = std::max(need[glq::FP8_WS_Q], (size_t)B * L->KB * GLQ_FP8_BLOCK);
    need[glq::FP8_WS_S] = std::max(need[glq::FP8_WS_S], (size_t)B * L->KB * sizeof(float));
}

// One slice of at most MAX_SLICE tokens: x (f16 / bf16), or q and s.
glq_status run_fp8(glq_fp8 L, const void *x, int x_dtype, const uint8_t *q, const float *s, int64_t s_ld, void *y,
                   int y_dtype, int64_t B, cudaStream_t st) {
    size_t need[glq::FP8_WS_COUNT] = {};
    fp8_need(L, B, q != nullptr, need);
    void *buf[glq::FP8_WS_COUNT];
    const glq_status ok = glq::fp8_workspace(L->device, need, st, buf);
    if (ok != GLQ_OK) return ok;
    int source = 2;
    if (!q && rounds_inside(L, B)) source = x_dtype;
    if (!q && source == 2) {
        glq::Fp8QuantParams p{};
        p.x = x;
        p.q = static_cast<uint8_t *>(buf[glq::FP8_WS_Q]);
        p.s = static_cast<float *>(buf[glq::FP8_WS_S]);
        p.B = B;
        p.n = (int)L->n;
        p.KB = L->KB;
        const glq_status e = launched(glq::launch_fp8_quantize(p, x_dtype, st, true));
        if (e != GLQ_OK) return e;
        q = p.q;
        s = p.s;
        s_ld = B;
    }
    if (B > glq::FP8_FEW) {
        glq::Fp8GemmParams p = gemm_params(L, B);
        const bool split = p.ksplit > 1;
        void *z = split ? buf[glq::FP8_WS_Z] : y;
        p.s = s;
        p.s_ld = s_ld;
        p.y_dtype = split ? GLQ_F32 : y_dtype;
        CUtensorMap qmap, wmap, ymap;
        if (!encode_e4m3(&qmap, q, (int64_t)L->KB * GLQ_FP8_BLOCK, B, 128) ||
            !encode_e4m3(&wmap, L->d_w, GLQ_FP8_BLOCK, (int64_t)L->RT * L->KB * 128, 64, false) ||
            !encode_rows(&ymap, p.y_dtype == 2 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                         p.y_dtype == 2 ? 4 : 2, z, L->m, split ? (int64_t)p.ksplit * p.part_rows : B, 32))
            return GLQ_ERR_CUDA;
        const glq_status e = launched(glq::launch_fp8_gemm(p, qmap, wmap, ymap, L->num_sms, st, true));
        if (e != GLQ_OK || !split) return e;
        return launched(glq::launch_fp8_sum_parts(static_cast<float *>(z), (int64_t)p.part_rows * L->m, p.ksplit, y,
                                                  y_dtype, B * L->m, st, true));
    }
    const int nt = glq::fp8_skinny_tile(B);
    glq::Fp8SkinnyParams p{};
    p.w = L->d_w;
    p.ws = L->d_ws;
    p.x = x;
    p.s = s;
    p.s_ld = s_ld;
    p.y = y;
    p.y_dtype = y_dtype;
    p.m = (int)L->m;
    p.n = (int)L->n;
    p.B = (int)B;
    p.RT = L->RT;
    p.KB = L->KB;
    p.err = L->d_err;
    const glq::Fp8SkinnyPlan plan = glq::plan_fp8_skinny(p.RT, p.KB, nt, L->clusters);
    p.C = plan.C;
    CUtensorMap qmap{};
    if (source == 2 && !encode_e4m3(&qmap, q, (int64_t)L->KB * GLQ_FP8_BLOCK, B, nt)) return GLQ_ERR_CUDA;
    return launched(glq::launch_fp8_skinny(p, qmap, source, nt, plan.clusters, st, true));
}

// ---------------------------------------------------------------------------
// Mixture of experts
// ---------------------------------------------------------------------------

void free_moe(glq_moe L) {
    cudaFree(L->d_w13);  // and what was allocated with it
    delete L;
}

// Sets p's workspace pointers from `base` (may be null) for p.T tokens;
// returns the bytes they span.
size_t moe_workspace(glq_moe L, glq::MoeParams &p, uint8_t *base) {
    const size_t nt = glq::moe_tile(p.T), slots = (size_t)p.T * p.k;
    const size_t A = std::min<size_t>((size_t)L->experts, slots);
    const size_t rows = slots + 7 * A;  // every expert's tokens rounded up to 8, at most
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t *r = base ? base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return r;
    };
    p.xq = take(rows * p.KB1 * 128);
    p.xs = reinterpret_cast<float *>(take((size_t)p.KB1 * p.T * 4));
    p.main1 = reinterpret_cast<float *>(take(slots * 2 * p.IB * 512));
    p.spill1 = reinterpret_cast<float *>(take((size_t)L->num_sms * nt * 512));
    p.hq = take(rows * p.IB * 128);
    p.hs = reinterpret_cast<float *>(take(rows * p.IB * 4));
    p.main2 = reinterpret_cast<float *>(take(slots * p.DB * 512));
    p.spill2 = reinterpret_cast<float *>(take((size_t)L->num_sms * nt * 512));
    return off;
}

glq::MoeParams moe_params(glq_moe L, int T) {
    glq::MoeParams p{};
    p.T = T;
    p.E = (int)L->experts;
    p.k = L->topk;
    p.d = (int)L->d;
    p.KB1 = p.DB = L->DB;
    p.IB = L->IB;
    p.scoring = L->scoring;
    p.renormalize = L->renormalize;
    p.routed_scale = L->routed_scale;
    p.w13 = L->d_w13;
    p.s13 = L->d_s13;
    p.w2 = L->d_w2;
    p.s2 = L->d_s2;
    p.bar = L->d_bar;
    p.err = L->d_err;
    return p;
}

void moe_need(glq_moe L, int64_t T, size_t need[glq::FP8_WS_COUNT]) {
    for (int t : {16, 32, glq::MOE_MAX_T}) {
        glq::MoeParams p = moe_params(L, (int)std::min<int64_t>(T, t));
        need[glq::FP8_WS_MOE] = std::max(need[glq::FP8_WS_MOE], moe_workspace(L, p, nullptr));
    }
}

// Layers are not made while their stream is captured: the allocation would end the capture.
bool capturing(void *stream) {
    cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &c) != cudaSuccess) cudaGetLastError();
    return c != cudaStreamCaptureStatusNone;
}

bool good_dims(int64_t m, int64_t n) {
    return m > 0 && n > 0 && !(m & 7) && !(n & 7) && m <= GLQ_FP8_MAX_DIM && n <= GLQ_FP8_MAX_DIM;
}

}  // namespace

extern "C" {

glq_status glq_fp8_quantize(const void *x_dev, glq_dtype x_dtype, int64_t B, int64_t n, void *q_dev, float *s_dev,
                            void *stream) {
    if (B < 0 || n <= 0 || (n & 7) || n > GLQ_FP8_MAX_DIM || B > 65535 * 32) return GLQ_ERR_SHAPE;
    if (x_dtype != GLQ_F16 && x_dtype != GLQ_BF16 && x_dtype != GLQ_F32) return GLQ_ERR_DTYPE;
    if (B == 0) return GLQ_OK;
    if (!x_dev || !q_dev || !s_dev) return GLQ_ERR_INVALID_ARG;
    if (!aligned(x_dev, 16) || !aligned(q_dev, 16) || !aligned(s_dev, 4)) return GLQ_ERR_INVALID_ARG;
    glq::Fp8QuantParams p{};
    p.x = x_dev;
    p.q = static_cast<uint8_t *>(q_dev);
    p.s = s_dev;
    p.B = B;
    p.n = (int)n;
    p.KB = (int)blocks_of(n);
    return launched(glq::launch_fp8_quantize(p, (int)x_dtype, static_cast<cudaStream_t>(stream), true));
}

glq_status glq_fp8_create(int64_t m, int64_t n, const void *w_dev, int64_t ldw, const float *scales_dev, void *stream,
                          glq_fp8 *out) {
    if (!out) return GLQ_ERR_INVALID_ARG;
    *out = nullptr;
    if (!good_dims(m, n) || ldw < n || (ldw & 7)) return GLQ_ERR_SHAPE;
    if (!w_dev || !scales_dev || !aligned(w_dev, 8) || !aligned(scales_dev, 4)) return GLQ_ERR_INVALID_ARG;
    if (capturing(stream)) return GLQ_ERR_CAPTURE;
    glq_fp8 L = new (std::nothrow) glq_fp8_s;
    if (!L) return GLQ_ERR_OOM;
    L->m = m;
    L->n = n;
    L->RT = (int)blocks_of(m);
    L->KB = (int)blocks_of(n);
    const int64_t tiles = (int64_t)L->RT * L->KB;
    glq_status st = GLQ_OK;
    if (cudaGetDevice(&L->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&L->num_sms, cudaDevAttrMultiProcessorCount, L->device) != cudaSuccess ||
        glq::fp8_skinny_clusters(L->num_sms, L->clusters) != cudaSuccess) {
        cudaGetLastError();
        st = GLQ_ERR_CUDA;
    }
    if (st == GLQ_OK)
        st = dev_alloc({{(void **)&L->d_w, (size_t)tiles * GLQ_FP8_TILE_BYTES},
                        {(void **)&L->d_ws, (size_t)tiles * sizeof(float)},
                        {(void **)&L->d_err, sizeof(unsigned)}},
                       &L->device_bytes);
    if (st == GLQ_OK) {
        glq::Fp8PackParams p{};
        p.src = static_cast<const uint8_t *>(w_dev);
        p.src_scale = scales_dev;
        p.dst = L->d_w;
        p.dst_scale = L->d_ws;
        p.ld = ldw;
        p.rows = (int)m;
        p.cols = (int)n;
        p.KB = L->KB;
        p.rt_step = 1;
        p.count = 1;
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        if (cudaMemsetAsync(L->d_err, 0, sizeof(unsigned), s) != cudaSuccess ||
            glq::launch_fp8_pack(p, s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess) {
            cudaGetLastError();
            st = GLQ_ERR_CUDA;
        }
    }
    if (st != GLQ_OK) {
        free_fp8(L);
        return st;
    }
    *out = L;
    return GLQ_OK;
}

glq_status glq_fp8_destroy(glq_fp8 layer) {
    if (!layer) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(layer->device);
    free_fp8(layer);
    return GLQ_OK;
}

glq_status glq_fp8_reserve(glq_fp8 layer, int64_t max_B) {
    if (!layer) return GLQ_ERR_INVALID_ARG;
    if (max_B < 0) return GLQ_ERR_SHAPE;
    DeviceGuard guard(layer->device);
    size_t need[glq::FP8_WS_COUNT] = {};
    // every batch up to max_B: the parts of K depend on it
    for (int64_t B = 1; B <= std::min(max_B, MAX_SLICE); ++B) fp8_need(layer, B, false, need);
    void *buf[glq::FP8_WS_COUNT];
    return glq::fp8_workspace(layer->device, need, 0, buf);
}

glq_status glq_fp8_linear(glq_fp8 L, const void *x_dev, glq_dtype x_dtype, void *y_dev, glq_dtype y_dtype, int64_t B,
                          void *stream) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    if (B < 0) return GLQ_ERR_SHAPE;
    if (x_dtype != GLQ_F16 && x_dtype != GLQ_BF16) return GLQ_ERR_DTYPE;
    if (y_dtype != x_dtype && y_dtype != GLQ_F32) return GLQ_ERR_DTYPE;
    if (B == 0) return GLQ_OK;
    if (!x_dev || !y_dev || !aligned(x_dev, 16) || !aligned(y_dev, 16)) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    const size_t ye = y_dtype == GLQ_F32 ? 4 : 2;
    for (int64_t b = 0; b < B; b += MAX_SLICE) {
        const glq_status st = run_fp8(L, static_cast<const char *>(x_dev) + (size_t)b * L->n * 2, (int)x_dtype, nullptr,
                                      nullptr, 0, static_cast<char *>(y_dev) + (size_t)b * L->m * ye, (int)y_dtype,
                                      std::min(MAX_SLICE, B - b), static_cast<cudaStream_t>(stream));
        if (st != GLQ_OK) return st;
    }
    return GLQ_OK;
}

glq_status glq_fp8_linear_quantized(glq_fp8 L, const void *q_dev, const float *s_dev, void *y_dev, glq_dtype y_dtype,
                                    int64_t B, void *stream) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    if (B < 0) return GLQ_ERR_SHAPE;
    if (y_dtype != GLQ_F16 && y_dtype != GLQ_BF16 && y_dtype != GLQ_F32) return GLQ_ERR_DTYPE;
    if (B == 0) return GLQ_OK;
    if (!q_dev || !s_dev || !y_dev || !aligned(q_dev, 16) || !aligned(s_dev, 4) || !aligned(y_dev, 16))
        return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    const size_t ye = y_dtype == GLQ_F32 ? 4 : 2;
    for (int64_t b = 0; b < B; b += MAX_SLICE) {
        const glq_status st =
            run_fp8(L, nullptr, 0, static_cast<const uint8_t *>(q_dev) + (size_t)b * L->KB * GLQ_FP8_BLOCK, s_dev + b, B,
                    static_cast<char *>(y_dev) + (size_t)b * L->m * ye, (int)y_dtype, std::min(MAX_SLICE, B - b),
                    static_cast<cudaStream_t>(stream));
        if (st != GLQ_OK) return st;
    }
    return GLQ_OK;
}

glq_status glq_fp8_dequant(glq_fp8 L, float *w_dev, void *stream) {
    if (!L || !w_dev || !aligned(w_dev, 4)) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    return launched(glq::launch_fp8_dequant(L->d_w, L->d_ws, w_dev, (int)L->m, (int)L->n, L->KB,
                                            static_cast<cudaStream_t>(stream)));
}

glq_status glq_fp8_check(glq_fp8 L, void *stream) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    return glq::take_error(L->d_err, static_cast<cudaStream_t>(stream));
}

glq_status glq_fp8_selftest_wait(glq_fp8 L, int arrivals, int64_t limit, void *stream) {
    if (!L || arrivals < 1 || arrivals > 2 || limit <= 0) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    return launched(glq::launch_fp8_wait_selftest(L->d_err, arrivals, (unsigned long long)limit,
                                                  static_cast<cudaStream_t>(stream)));
}

glq_status glq_fp8_plan(glq_fp8 L, int64_t B, int32_t *kernel, int32_t *cluster, int32_t *clusters, int32_t *ksplit,
                        int64_t *items) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    if (B < 1 || B > MAX_SLICE) return GLQ_ERR_SHAPE;
    const bool many = B > glq::FP8_FEW;
    int c = 2, n = 0, ks = 1;
    int64_t all = L->RT;
    if (many) {
        const glq::Fp8GemmParams p = gemm_params(L, B);
        ks = p.ksplit;
        all = (int64_t)p.tiles * ks;
        n = (int)std::min<int64_t>(all, L->num_sms / 2);
    } else {
        const glq::Fp8SkinnyPlan plan = glq::plan_fp8_skinny(L->RT, L->KB, glq::fp8_skinny_tile(B), L->clusters);
        c = plan.C;
        n = plan.clusters;
    }
    if (kernel) *kernel = many ? 1 : 0;
    if (cluster) *cluster = c;
    if (clusters) *clusters = n;
    if (ksplit) *ksplit = ks;
    if (items) *items = all;
    return GLQ_OK;
}

glq_status glq_fp8_info(glq_fp8 L, int64_t *m, int64_t *n, size_t *device_bytes) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    if (m) *m = L->m;
    if (n) *n = L->n;
    if (device_bytes) *device_bytes = L->device_bytes;
    return GLQ_OK;
}

glq_status glq_moe_create(const glq_moe_config *c, const void *gate_dev, const float *gate_scales_dev,
                          const void *up_dev, const float *up_scales_dev, const void *down_dev,
                          const float *down_scales_dev, void *stream, glq_moe *out) {
    if (!out) return GLQ_ERR_INVALID_ARG;
    *out = nullptr;
    if (!c) return GLQ_ERR_INVALID_ARG;
    if (!good_dims(c->d, c->inter) || c->experts < 1 || c->experts > glq::MOE_MAX_E || c->topk < 1 ||
        c->topk > glq::MOE_MAX_K || c->topk > c->experts)
        return GLQ_ERR_SHAPE;
    // the kernel counts blocks and places in 31 bits
    const int64_t DB = blocks_of(c->d), IB = blocks_of(c->inter);
    if (c->experts * 2 * IB * DB > (int64_t)1 << 30) return GLQ_ERR_SHAPE;
    if (c->scoring != GLQ_MOE_SOFTMAX && c->scoring != GLQ_MOE_SIGMOID) return GLQ_ERR_INVALID_ARG;
    if (!(c->routed_scale - c->routed_scale == 0.f)) return GLQ_ERR_INVALID_ARG;  // not finite
    for (const void *w : {gate_dev, up_dev, down_dev})
        if (!w || !aligned(w, 8)) return GLQ_ERR_INVALID_ARG;
    for (const float *s : {gate_scales_dev, up_scales_dev, down_scales_dev})
        if (!s || !aligned(s, 4)) return GLQ_ERR_INVALID_ARG;
    if (capturing(stream)) return GLQ_ERR_CAPTURE;
    glq_moe L = new (std::nothrow) glq_moe_s;
    if (!L) return GLQ_ERR_OOM;
    L->experts = c->experts;
    L->d = c->d;
    L->inter = c->inter;
    L->topk = c->topk;
    L->scoring = c->scoring;
    L->renormalize = c->renormalize ? 1 : 0;
    L->routed_scale = c->routed_scale;
    L->DB = (int)DB;
    L->IB = (int)IB;
    const int64_t tiles2 = L->experts * DB * IB, tiles13 = 2 * tiles2;
    glq_status st = GLQ_OK;
    if (cudaGetDevice(&L->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&L->num_sms, cudaDevAttrMultiProcessorCount, L->device) != cudaSuccess) {
        cudaGetLastError();
        st = GLQ_ERR_CUDA;
    }
    if (st == GLQ_OK)
        st = dev_alloc({{(void **)&L->d_w13, (size_t)tiles13 * GLQ_FP8_TILE_BYTES},
                        {(void **)&L->d_w2, (size_t)tiles2 * GLQ_FP8_TILE_BYTES},
                        {(void **)&L->d_s13, (size_t)tiles13 * sizeof(float)},
                        {(void **)&L->d_s2, (size_t)tiles2 * sizeof(float)},
                        {(void **)&L->d_err, sizeof(unsigned)},
                        {(void **)&L->d_bar, sizeof(uint64_t)}},
                       &L->device_bytes);
    if (st == GLQ_OK) {
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        bool ok = cudaMemsetAsync(L->d_err, 0, sizeof(unsigned), s) == cudaSuccess &&
                  cudaMemsetAsync(L->d_bar, 0, sizeof(uint64_t), s) == cudaSuccess;
        auto pack = [&](const void *w, const float *sc, int64_t rows, int64_t cols, uint8_t *dst, float *dst_scale,
                        int step, int off) {
            glq::Fp8PackParams p{};
            p.src = static_cast<const uint8_t *>(w);
            p.src_scale = sc;
            p.dst = dst;
            p.dst_scale = dst_scale;
            p.ld = cols;
            p.rows = (int)rows;
            p.cols = (int)cols;
            p.KB = (int)blocks_of(cols);
            p.rt_step = step;
            p.rt_off = off;
            p.count = (int)L->experts;
            p.src_stride = rows * cols;
            p.src_scale_stride = blocks_of(rows) * p.KB;
            p.dst_tiles = step * blocks_of(rows) * p.KB;
            ok = ok && glq::launch_fp8_pack(p, s) == cudaSuccess;
        };
        pack(gate_dev, gate_scales_dev, L->inter, L->d, L->d_w13, L->d_s13, 2, 0);
        pack(up_dev, up_scales_dev, L->inter, L->d, L->d_w13, L->d_s13, 2, 1);
        pack(down_dev, down_scales_dev, L->d, L->inter, L->d_w2, L->d_s2, 1, 0);
        if (!ok || cudaStreamSynchronize(s) != cudaSuccess) {
            cudaGetLastError();
            st = GLQ_ERR_CUDA;
        }
    }
    if (st != GLQ_OK) {
        free_moe(L);
        return st;
    }
    *out = L;
    return GLQ_OK;
}

glq_status glq_moe_destroy(glq_moe layer) {
    if (!layer) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(layer->device);
    free_moe(layer);
    return GLQ_OK;
}

glq_status glq_moe_reserve(glq_moe layer, int64_t max_T) {
    if (!layer) return GLQ_ERR_INVALID_ARG;
    if (max_T < 0) return GLQ_ERR_SHAPE;
    if (max_T == 0) return GLQ_OK;
    DeviceGuard guard(layer->device);
    size_t need[glq::FP8_WS_COUNT] = {};
    moe_need(layer, max_T, need);
    void *buf[glq::FP8_WS_COUNT];
    return glq::fp8_workspace(layer->device, need, 0, buf);
}

glq_status glq_moe_forward(glq_moe L, const void *x_dev, glq_dtype x_dtype, const void *logits_dev,
                           glq_dtype logits_dtype, void *y_dev, glq_dtype y_dtype, int64_t T, void *stream) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    if (T < 0) return GLQ_ERR_SHAPE;
    if (x_dtype != GLQ_F16 && x_dtype != GLQ_BF16) return GLQ_ERR_DTYPE;
    if (y_dtype != x_dtype && y_dtype != GLQ_F32) return GLQ_ERR_DTYPE;
    if (logits_dtype != x_dtype && logits_dtype != GLQ_F32) return GLQ_ERR_DTYPE;
    if (T == 0) return GLQ_OK;
    if (!x_dev || !y_dev || !logits_dev || !aligned(x_dev, 16) || !aligned(y_dev, 16) ||
        !aligned(logits_dev, logits_dtype == GLQ_F32 ? 4 : 2))
        return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    size_t need[glq::FP8_WS_COUNT] = {};
    moe_need(L, T, need);
    void *buf[glq::FP8_WS_COUNT];
    const glq_status st = glq::fp8_workspace(L->device, need, s, buf);
    if (st != GLQ_OK) return st;
    const size_t ye = y_dtype == GLQ_F32 ? 4 : 2, le = logits_dtype == GLQ_F32 ? 4 : 2;
    for (int64_t t = 0; t < T; t += glq::MOE_MAX_T) {
        glq::MoeParams p = moe_params(L, (int)std::min<int64_t>(glq::MOE_MAX_T, T - t));
        p.x = static_cast<const char *>(x_dev) + (size_t)t * L->d * 2;
        p.logits = static_cast<const char *>(logits_dev) + (size_t)t * L->experts * le;
        p.y = static_cast<char *>(y_dev) + (size_t)t * L->d * ye;
        p.x_dtype = (int)x_dtype;
        p.logits_dtype = (int)logits_dtype;
        p.y_dtype = (int)y_dtype;
        moe_workspace(L, p, static_cast<uint8_t *>(buf[glq::FP8_WS_MOE]));
        const glq_status e = launched(glq::launch_moe(p, L->num_sms, s));
        if (e != GLQ_OK) return e;
    }
    return GLQ_OK;
}

glq_status glq_moe_check(glq_moe L, void *stream) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    // a call that gave up may have left the grid barrier half way
    return glq::take_error(L->d_err, static_cast<cudaStream_t>(stream), L->d_bar);
}

glq_status glq_moe_selftest_wait(glq_moe L, int arrivals, int64_t limit, void *stream) {
    if (!L || arrivals < 1 || arrivals > 2 || limit <= 0) return GLQ_ERR_INVALID_ARG;
    DeviceGuard guard(L->device);
    return launched(glq::launch_moe_wait_selftest(L->d_bar, L->d_err, L->num_sms, arrivals == 2, (unsigned long long)limit,
                                                  static_cast<cudaStream_t>(stream)));
}

glq_status glq_moe_info(glq_moe L, glq_moe_config *config, size_t *device_bytes) {
    if (!L) return GLQ_ERR_INVALID_ARG;
    if (config)
        *config = glq_moe_config{L->experts, L->d, L->inter, L->topk, L->scoring, L->renormalize, L->routed_scale};
    if (device_bytes) *device_bytes = L->device_bytes;
    return GLQ_OK;
}

}  // extern "C"
