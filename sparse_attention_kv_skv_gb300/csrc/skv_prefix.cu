// A prefix that a whole batch shares (a text that all its requests start with, kept
// once in device memory): attention over it, the join with other attention results,
// the weight its tokens receive, and the eviction of the lightest.
//
// For unit (b, l) with `heads` query heads, rows k_j (576 bf16) of layer l, j < n:
//   s_hj = scale * q_h . k_j;   out_h = sum_j softmax_j(s_h) k_j[0..512);   lse_h = log sum_j exp s_hj
// Units that share a layer read the same rows, so their heads are rows of one product.

#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "skv_ctx.cuh"

namespace skv {
namespace {

constexpr int kDim = 576, kVDim = 512, kRowBytes = kDim * 2;
constexpr int kMaxHeads = 128;   // of a unit
constexpr int kMaxParts = 8;     // of a join
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

// The prefix and the call's units.
struct PrefixShape {
    const uint8_t* rows;
    int64_t layer_stride, row_stride;
    int n, B, heads, layers, layer0;  // layers of the call; layer0: the first of them
    __device__ __forceinline__ const uint4* row(int l, int j) const
    {
        return reinterpret_cast<const uint4*>(rows + (layer0 + l) * layer_stride + j * row_stride);
    }
    // A layer's query rows, entries and their heads in order: where row i lies among all [B][layers][heads].
    __device__ __forceinline__ int64_t q_row(int l, int64_t i) const
    {
        const int64_t b = i / heads;
        return (b * layers + l) * heads + (i - b * heads);
    }
};

// ---------------------------------------------------------------------------
// Sixteen query rows a CTA, the keys in blocks of 32; fp32 products on the cores.
constexpr int kQRows = 16, kKeys = 32, kThreads = 256;
constexpr size_t kTileSmem = (size_t)kQRows * kDim * 4 + (size_t)kKeys * kRowBytes;

__device__ __forceinline__ void load_keys(const PrefixShape& p, int l, int j0, uint4* sk)
{
    for (int i = threadIdx.x; i < kKeys * (kRowBytes / 16); i += kThreads) {
        const int j = i / (kRowBytes / 16), c = i % (kRowBytes / 16);
        sk[i] = j0 + j < p.n ? p.row(l, j0 + j)[c] : make_uint4(0, 0, 0, 0);
    }
}
__device__ __forceinline__ void load_queries(const PrefixShape& p, int l, int64_t i0, const uint16_t* q, float* sq)
{
    const int64_t rows = (int64_t)p.B * p.heads;
    for (int i = threadIdx.x; i < kQRows * kDim; i += kThreads) {
        const int64_t r = i0 + i / kDim;
        sq[i] = r < rows ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(q)[p.q_row(l, r) * kDim + i % kDim]) : 0.0f;
    }
}
__device__ __forceinline__ float dot(const float* a, const __nv_bfloat16* b)
{
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int d = 0; d < kDim; d += 4)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] = fmaf(a[d + x], __bfloat162float(b[d + x]), s[x]);
    return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ void __launch_bounds__(kThreads) attend_tile_kernel(PrefixShape p, const uint16_t* __restrict__ q,
                                                               uint16_t* __restrict__ out, float* __restrict__ lse, float scale_log2)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float sp[kQRows][kKeys + 1];
    float* sq = reinterpret_cast<float*>(smem);
    uint4* sk = reinterpret_cast<uint4*>(smem + (size_t)kQRows * kDim * 4);
    const __nv_bfloat16* kb = reinterpret_cast<const __nv_bfloat16*>(sk);
    const int l = blockIdx.y, r = threadIdx.x / 16, t = threadIdx.x % 16;
    const int64_t i0 = (int64_t)blockIdx.x * kQRows, rows = (int64_t)p.B * p.heads;
    load_queries(p, l, i0, q, sq);
    float acc[32] = {}, m = -INFINITY, total = 0.0f;
    for (int j0 = 0; j0 < p.n; j0 += kKeys) {
        __syncthreads();
        load_keys(p, l, j0, sk);
        __syncthreads();
        float s[2], mb = -INFINITY;
        for (int x = 0; x < 2; ++x) {
            const int j = t + 16 * x;
            s[x] = j0 + j < p.n ? dot(sq + r * kDim, kb + j * kDim) * scale_log2 : -INFINITY;
            mb = fmaxf(mb, s[x]);
        }
        for (int o = 1; o < 16; o <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, o));
        const float m2 = fmaxf(m, mb), base = m2 == -INFINITY ? 0.0f : m2, fix = exp2f(m - base);
        float ps = 0.0f;
        for (int x = 0; x < 2; ++x) {
            const float e = exp2f(s[x] - base);
            sp[r][t + 16 * x] = e;
            ps += e;
        }
        for (int o = 1; o < 16; o <<= 1) ps += __shfl_xor_sync(0xFFFFFFFFu, ps, o);
        total = total * fix + ps;
        m = m2;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 32; ++c) acc[c] *= fix;
        for (int j = 0; j < kKeys; ++j) {
            const float e = sp[r][j];
#pragma unroll
            for (int c = 0; c < 32; ++c) acc[c] = fmaf(e, __bfloat162float(kb[j * kDim + t + 16 * c]), acc[c]);
        }
    }
    if (i0 + r >= rows) return;
    const int64_t at = p.q_row(l, i0 + r);
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    for (int c = 0; c < 32; ++c)
        reinterpret_cast<__nv_bfloat16*>(out)[at * kVDim + t + 16 * c] = __float2bfloat16_rn(acc[c] * inv);
    if (t == 0 && lse) lse[at] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2;
}

// Thirty-two tokens a CTA, all query rows of the layer in groups of 16.
__global__ void __launch_bounds__(kThreads) weigh_tile_kernel(PrefixShape p, const uint16_t* __restrict__ q,
                                                              const float* __restrict__ lse, const float* weights,
                                                              int64_t weights_stride, float* out, int64_t out_stride,
                                                              float scale_log2, float gain)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float part[kQRows][kKeys];
    float* sq = reinterpret_cast<float*>(smem);
    uint4* sk = reinterpret_cast<uint4*>(smem + (size_t)kQRows * kDim * 4);
    const __nv_bfloat16* kb = reinterpret_cast<const __nv_bfloat16*>(sk);
    const int l = blockIdx.y, j0 = blockIdx.x * kKeys, r = threadIdx.x / 16, t = threadIdx.x % 16;
    const int64_t rows = (int64_t)p.B * p.heads;
    load_keys(p, l, j0, sk);
    float sum[2] = {0.0f, 0.0f};
    for (int64_t i0 = 0; i0 < rows; i0 += kQRows) {
        __syncthreads();
        load_queries(p, l, i0, q, sq);
        __syncthreads();
        const float e = i0 + r < rows ? lse[p.q_row(l, i0 + r)] : -INFINITY;
        if (e == -INFINITY) continue;
        for (int x = 0; x < 2; ++x) sum[x] += exp2f(fmaf(dot(sq + r * kDim, kb + (t + 16 * x) * kDim), scale_log2, -e * kLog2e));
    }
    for (int x = 0; x < 2; ++x) part[r][t + 16 * x] = sum[x];
    __syncthreads();
    const int j = j0 + threadIdx.x;
    if (threadIdx.x < kKeys && j < p.n) {
        float w = 0.0f;
        for (int x = 0; x < kQRows; ++x) w += part[x][threadIdx.x];
        const float before = weights ? weights[(p.layer0 + l) * weights_stride + j] : 0.0f;
        out[(p.layer0 + l) * out_stride + j] = fmaf(gain, w, before);
    }
}

// ---------------------------------------------------------------------------
struct JoinParts {
    const uint4* out[kMaxParts];
    const float* lse[kMaxParts];
};

__device__ __forceinline__ uint32_t bf2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A warp a row, 16 columns a lane.  All of a row is read before any of it is written, so the result may
// take a part's place.
template <int kParts>
__global__ void __launch_bounds__(256) join_kernel(JoinParts parts, int64_t rows, uint4* out, float* lse)
{
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows; r += step) {
        float e[kParts], top = -INFINITY;
        uint4 v[kParts][2];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            e[i] = parts.lse[i][r];
            v[i][0] = parts.out[i][r * 64 + lane];
            v[i][1] = parts.out[i][r * 64 + 32 + lane];
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) top = fmaxf(top, e[i]);
        const float base = top == -INFINITY ? 0.0f : top;
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < kParts; ++i) total += expf(e[i] - base);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        float acc[16] = {};
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (e[i] == -INFINITY) continue;
            const float w = expf(e[i] - base) * inv;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[8 * h + 2 * c] = fmaf(w, __uint_as_float(x[c] << 16), acc[8 * h + 2 * c]);
                    acc[8 * h + 2 * c + 1] = fmaf(w, __uint_as_float(x[c] & 0xFFFF0000u), acc[8 * h + 2 * c + 1]);
                }
            }
        }
        __syncwarp();  // every lane has read the row's lse
#pragma unroll
        for (int h = 0; h < 2; ++h)
            out[r * 64 + 32 * h + lane] = make_uint4(bf2(acc[8 * h], acc[8 * h + 1]), bf2(acc[8 * h + 2], acc[8 * h + 3]),
                                                     bf2(acc[8 * h + 4], acc[8 * h + 5]), bf2(acc[8 * h + 6], acc[8 * h + 7]));
        if (lane == 0 && lse) lse[r] = total == 0.0f ? -INFINITY : base + logf(total);
    }
}

// ---------------------------------------------------------------------------
// The tokens that stay (kept, ascending, -1 behind the last): their rows and weights moved together.  A warp
// moves four rows, nine 16-byte pieces a lane.
__global__ void __launch_bounds__(256) keep_kernel(PrefixShape p, const float* weights, int64_t weights_stride, int keep,
                                                   const int32_t* kept, uint4* rows_out, float* weights_out)
{
    constexpr int kPieces = kRowBytes / 16, kRowsAWarp = 4, kEach = kPieces * kRowsAWarp / 32;
    const int l = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8 * kRowsAWarp;
    kept += (int64_t)l * keep;
    for (int64_t i0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kRowsAWarp; i0 < keep; i0 += step) {
        const int32_t token = lane < kRowsAWarp && i0 + lane < keep ? kept[i0 + lane] : -1;
        if (rows_out) {
            uint4 v[kEach];
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int at = 32 * x + lane;
                const int32_t t = __shfl_sync(0xFFFFFFFFu, token, at / kPieces);
                if (t >= 0) v[x] = p.row(l, t)[at % kPieces];
            }
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int at = 32 * x + lane;
                if (__shfl_sync(0xFFFFFFFFu, token, at / kPieces) >= 0) rows_out[((int64_t)l * keep + i0) * kPieces + at] = v[x];
            }
        }
        if (weights_out && token >= 0) weights_out[(int64_t)l * keep + i0 + lane] = weights[(p.layer0 + l) * weights_stride + token];
    }
}

int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

}  // namespace

cudaError_t prepare_prefix()
{
    cudaError_t e = cudaFuncSetAttribute(attend_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTileSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(weigh_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTileSmem);
    return e;
}

}  // namespace skv

namespace {
using skv::PrefixShape;

// Runs f on the context's device and turns its result into a status.
template <typename F>
skv_status on_device(const skv_ctx* ctx, const char* what, F f)
{
    int prev = -1;
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != ctx->cfg.device && cudaSetDevice(ctx->cfg.device) != cudaSuccess) return SKV_ERR_CUDA;
    const cudaError_t e = f();
    if (prev >= 0 && prev != ctx->cfg.device) cudaSetDevice(prev);
    if (e == cudaSuccess) return SKV_OK;
    skv::set_last_error_message((std::string(what) + ": " + cudaGetErrorString(e)).c_str());
    return SKV_ERR_CUDA;
}

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// What the calls and their workspace queries check alike.
bool shape_ok(const skv_ctx* ctx, const skv_prefix* x, int32_t layer)
{
    return ctx && x && x->n >= 0 && x->n <= skv::kMaxSelectTokens && layer >= -1 && layer < ctx->cfg.num_layers;
}
bool batch_ok(const skv_ctx* ctx, int32_t B, int32_t heads)
{
    return B >= 0 && B <= ctx->cfg.max_batch && heads >= 1 && heads <= skv::kMaxHeads;
}
bool rows_ok(const skv_ctx* ctx, const skv_prefix& x)
{
    auto stride_ok = [](int64_t s, int64_t entries) {  // used only where the axis has more than one entry
        return entries <= 1 || (s > 0 && s % 16 == 0 && s < ((int64_t)1 << 40));
    };
    return x.n == 0 || (x.rows && aligned(x.rows, 16) && stride_ok(x.row_stride, x.n) &&
                        (x.n == 1 || x.row_stride >= skv::kRowBytes) && stride_ok(x.layer_stride, ctx->cfg.num_layers));
}
PrefixShape shape_of(const skv_ctx* ctx, const skv_prefix& x, int32_t B, int32_t heads, int32_t layer)
{
    return PrefixShape{static_cast<const uint8_t*>(x.rows), x.layer_stride, x.row_stride, (int)x.n, B, heads,
                       layer < 0 ? ctx->cfg.num_layers : 1, layer < 0 ? 0 : layer};
}
int64_t evict_bytes(const skv_ctx* ctx, const skv_prefix& x, int32_t layer)
{
    // a word a token, and the lengths
    const int64_t layers = layer < 0 ? ctx->cfg.num_layers : 1;
    return layers * skv::select_stride(x.n, 1) * 4 + layers * 4;
}
}  // namespace

extern "C" {

skv_status skv_attend_prefix_workspace(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                                       int64_t* bytes)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !bytes) return SKV_ERR_INVALID_ARG;
    *bytes = 16;
    return SKV_OK;
}

skv_status skv_attend_prefix(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                             const void* q_dev, void* out_dev, float* lse_dev, float sm_scale, void* workspace_dev,
                             int64_t workspace_bytes, skv_stream_t stream)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale))
        return SKV_ERR_INVALID_ARG;
    if (B == 0) return SKV_OK;
    int64_t need = 0;
    skv_attend_prefix_workspace(ctx, prefix, B, heads, layer, &need);
    if (!rows_ok(ctx, *prefix) || !q_dev || !out_dev || !workspace_dev || workspace_bytes < need || !aligned(q_dev, 16) ||
        !aligned(out_dev, 16) || !aligned(lse_dev, 4) || !aligned(workspace_dev, 16))
        return SKV_ERR_INVALID_ARG;
    const PrefixShape p = shape_of(ctx, *prefix, B, heads, layer);
    return on_device(ctx, "skv_attend_prefix", [&] {
        const int64_t groups = ((int64_t)B * heads + skv::kQRows - 1) / skv::kQRows;
        skv::attend_tile_kernel<<<dim3((unsigned)groups, (unsigned)p.layers), skv::kThreads, skv::kTileSmem, stream>>>(
            p, static_cast<const uint16_t*>(q_dev), static_cast<uint16_t*>(out_dev), lse_dev, sm_scale * skv::kLog2e);
        return cudaGetLastError();
    });
}

skv_status skv_join(skv_ctx* ctx, int32_t parts, const void* const* outs, const float* const* lses, int64_t rows,
                    void* out_dev, float* lse_dev, skv_stream_t stream)
{
    if (!ctx || parts < 1 || parts > skv::kMaxParts || rows < 0 || rows > (int64_t)1 << 32) return SKV_ERR_INVALID_ARG;
    if (rows == 0) return SKV_OK;
    if (!outs || !lses || !out_dev || !aligned(out_dev, 16) || !aligned(lse_dev, 4)) return SKV_ERR_INVALID_ARG;
    skv::JoinParts jp{};
    for (int i = 0; i < parts; ++i) {
        if (!outs[i] || !lses[i] || !aligned(outs[i], 16) || !aligned(lses[i], 4)) return SKV_ERR_INVALID_ARG;
        jp.out[i] = static_cast<const uint4*>(outs[i]);
        jp.lse[i] = lses[i];
    }
    return on_device(ctx, "skv_join", [&] {
        void (*const kernels[])(skv::JoinParts, int64_t, uint4*, float*) = {
            skv::join_kernel<1>, skv::join_kernel<2>, skv::join_kernel<3>, skv::join_kernel<4>,
            skv::join_kernel<5>, skv::join_kernel<6>, skv::join_kernel<7>, skv::join_kernel<8>};
        const unsigned grid = (unsigned)std::min<int64_t>((rows + 7) / 8, 1 << 20);
        kernels[parts - 1]<<<grid, 256, 0, stream>>>(jp, rows, static_cast<uint4*>(out_dev), lse_dev);
        return cudaGetLastError();
    });
}

skv_status skv_weigh_prefix_workspace(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                                      int64_t* bytes)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !bytes) return SKV_ERR_INVALID_ARG;
    *bytes = 16;
    return SKV_OK;
}

skv_status skv_weigh_prefix(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                            const void* q_dev, const float* lse_dev, const float* weights_dev, int64_t weights_stride,
                            float* out_dev, int64_t out_stride, float sm_scale, float gain, void* workspace_dev,
                            int64_t workspace_bytes, skv_stream_t stream)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale) ||
        !std::isfinite(gain))
        return SKV_ERR_INVALID_ARG;
    if (B == 0 || prefix->n == 0) return SKV_OK;
    int64_t need = 0;
    skv_weigh_prefix_workspace(ctx, prefix, B, heads, layer, &need);
    const bool many = ctx->cfg.num_layers > 1;
    if (!rows_ok(ctx, *prefix) || !q_dev || !lse_dev || !out_dev || !workspace_dev || workspace_bytes < need ||
        !aligned(q_dev, 16) || !aligned(workspace_dev, 16) || !aligned(lse_dev, 4) || !aligned(weights_dev, 4) ||
        !aligned(out_dev, 4) || (many && (out_stride < prefix->n || (weights_dev && weights_stride < prefix->n))) ||
        out_stride >= (int64_t)1 << 40 || weights_stride >= (int64_t)1 << 40)
        return SKV_ERR_INVALID_ARG;
    const PrefixShape p = shape_of(ctx, *prefix, B, heads, layer);
    return on_device(ctx, "skv_weigh_prefix", [&] {
        skv::weigh_tile_kernel<<<dim3((unsigned)((p.n + skv::kKeys - 1) / skv::kKeys), (unsigned)p.layers), skv::kThreads, skv::kTileSmem, stream>>>(
            p, static_cast<const uint16_t*>(q_dev), lse_dev, weights_dev, weights_stride, out_dev, out_stride,
            sm_scale * skv::kLog2e, gain);
        return cudaGetLastError();
    });
}

skv_status skv_evict_prefix_workspace(skv_ctx* ctx, const skv_prefix* prefix, int32_t layer, int64_t* bytes)
{
    if (!shape_ok(ctx, prefix, layer) || !bytes) return SKV_ERR_INVALID_ARG;
    *bytes = evict_bytes(ctx, *prefix, layer);
    return SKV_OK;
}

skv_status skv_evict_prefix(skv_ctx* ctx, const skv_prefix* prefix, int32_t layer, const float* weights_dev,
                            int64_t weights_stride, int32_t keep, int32_t first, int32_t last, int32_t* kept_dev,
                            void* rows_out_dev, float* weights_out_dev, void* workspace_dev, int64_t workspace_bytes,
                            skv_stream_t stream)
{
    if (!shape_ok(ctx, prefix, layer) || keep < 1 || keep > skv::kMaxSelectTokens || first < 0 || last < 0 ||
        (int64_t)first + last > keep)
        return SKV_ERR_INVALID_ARG;
    if (!rows_ok(ctx, *prefix) || !kept_dev || !workspace_dev || (prefix->n > 0 && !weights_dev) ||
        workspace_bytes < evict_bytes(ctx, *prefix, layer) || !aligned(workspace_dev, 16) || !aligned(rows_out_dev, 16) ||
        !aligned(kept_dev, 4) || !aligned(weights_dev, 4) || !aligned(weights_out_dev, 4) ||
        (ctx->cfg.num_layers > 1 && weights_stride < prefix->n) || weights_stride >= (int64_t)1 << 40)
        return SKV_ERR_INVALID_ARG;
    const PrefixShape p = shape_of(ctx, *prefix, 1, 1, layer);
    return on_device(ctx, "skv_evict_prefix", [&] {
        cudaError_t e = skv::launch_heaviest(ctx->d, weights_dev + p.layer0 * weights_stride, weights_stride, p.layers, p.n,
                                             keep, first, last, kept_dev, workspace_dev, ctx->device_sms, stream);
        if (e != cudaSuccess || (!rows_out_dev && !weights_out_dev) || p.n == 0) return e;
        const int64_t groups = ((int64_t)keep + 31) / 32;
        skv::keep_kernel<<<dim3((unsigned)std::min<int64_t>(groups, 1 << 20), (unsigned)p.layers), 256, 0, stream>>>(
            p, weights_dev, weights_stride, keep, kept_dev, static_cast<uint4*>(rows_out_dev), weights_out_dev);
        return cudaGetLastError();
    });
}

}  // extern "C"
