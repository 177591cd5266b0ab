// A prefix that a whole batch shares (a text that all its requests start with, kept
// once in device memory): attention over it, the join with other attention results,
// the weight its tokens receive, and the eviction of the lightest.
//
// For unit (b, l) with `heads` query heads, rows k_j (576 bf16) of layer l, j < n:
//   s_hj = scale * q_h . k_j;   out_h = sum_j softmax_j(s_h) k_j[0..512);   lse_h = log sum_j exp s_hj
// Units that share a layer read the same rows, so their heads are rows of one product.
//
// Times in this file are of calls replayed from a CUDA graph one after the other, in bursts of some milliseconds at 2.07 GHz,
// unless said otherwise.  "Among others": a program's call through the Python binding, with others around it.  The difference is
// the host's and, for products of hundreds of microseconds, the power limit, under which a large library product falls from 1.95
// PFLOP/s to 1.71.

#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "f32x2.cuh"
#include "skv_ctx.cuh"
#include "tcgen05.cuh"

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
    int n, B, heads, layers, layer0;  // layers of the launch; layer0: the first of them
    int unit_layers;                  // layers of the call: an entry has that many units
    int map_x, map_z;                 // where layer l of the launch begins in the rows' tensor map: column l * map_x, plane l * map_z
    __device__ __forceinline__ const uint4* row(int l, int j) const
    {
        return reinterpret_cast<const uint4*>(rows + (layer0 + l) * layer_stride + j * row_stride);
    }
};

// ---------------------------------------------------------------------------
// The kernels on the tensor cores run as clusters of two CTAs that multiply as one
// (cta_group::2).  Query rows go in tiles of 128: the heads of 128 / heads entries
// of a layer, in order; rows that are left over are zeros.
constexpr uint32_t kMaxSleepPolls = 1u << 20;  // bound of a wait whose polls may each sleep (4 s, measured; the longest, for a whole item, is some 3 s with rows that fill the GPU's memory)
constexpr int kTileRows = 128;
constexpr int kBoxes = kDim / 64;              // 64-dim columns of a row, 128 bytes wide
constexpr uint32_t kTileBox = kTileRows * 128; // such a column of a tile of 128 rows
constexpr uint32_t kSmemLimit = 227 * 1024;    // dynamic shared memory a CTA may have

__host__ __device__ __forceinline__ int entries_a_tile(int heads) { return kTileRows / heads; }

__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort)
{
    const uint32_t a = tc::smem_u32(bar);
#pragma unroll 1
    for (uint32_t i = 0; i < kMaxSleepPolls; ++i) {
        if (tc::mbar_test(a, parity)) return true;
        if ((i & 7u) == 7u && *abort) return false;
    }
    return false;
}
__device__ __forceinline__ void give_up(uint32_t* abort, uint32_t* err)
{
    if (!*(volatile uint32_t*)abort) {
        *(volatile uint32_t*)abort = 1u;
        atomicOr(err, DEVERR_TIMEOUT);
    }
}

// The end of a kernel of a CTA pair, by all threads of both; rank 0 has committed `fin` behind its last product.  What other
// pairs of the cluster commit to a CTA it has waited for before it comes here.
// `owner`: the warp that holds the tensor memory.
__device__ __forceinline__ void pair_exit(uint64_t* fin, uint32_t* abort, uint32_t* err, uint32_t tbase, bool owner, uint32_t cols)
{
    tc::fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0) {
        // no product of the pair, and no arrival of one, is left when either CTA leaves
        if (!tc::mbar_wait(fin, 0, 1u << 22)) give_up(abort, err);
        if (*(volatile uint32_t*)abort)  // copies of a call that gave up may still be landing: they take microseconds
            for (int i = 0; i < 256; ++i) __nanosleep(1000);
    }
    __syncthreads();
    tc::cluster_sync();  // neither CTA leaves while the other's products or copies may still reach it
    if (owner) {
        tc::fence_after_sync();
        tc::tmem2_dealloc(tbase, cols);
    }
}

// The query row that lies in row r of tile `tile`: its unit's first head's row plus its head, or -1.  (Of a launch on one of
// several layers, counted from that layer's first unit.)
__device__ __forceinline__ int64_t tile_row(const PrefixShape& p, int l, int tile, int r)
{
    const int per = entries_a_tile(p.heads), e = r / p.heads, b = tile * per + e;
    return e < per && b < p.B ? ((int64_t)b * p.unit_layers + l) * p.heads + (r - e * p.heads) : -1;
}

// ---------------------------------------------------------------------------
// Weights.  S^T = K Q^T with the keys as the product's rows (128 a CTA, 256 a
// pair) and 256 query rows as its columns (a tile of 128 from either CTA), so a thread of the
// epilogue owns a key and sums its query rows alone, without any exchange:
//   sum_i exp2(s_ij scale log2 e - lse_i log2 e)
// A piece of the work is 256 keys of a layer by a share of its query rows; the
// keys stay in shared memory (147 KB a CTA) while the queries stream past them through a ring of
// 64-dim columns.  Shares are summed in their order by a second kernel.
// What bounds it: the products, 128 cycles each of 256 x 256 x 16, 4608 a pair of tiles; beside them go 32 bytes a cycle
// from L2 and 96 of the 128 bytes a cycle that shared memory gives (with a CTA by itself, not a pair, 192 would), and an
// epilogue of 256 exponentials a thread, 2048 cycles.
// Measured: 447 us at 192 x 2 units of 128 heads over 16K tokens, 2.07 PFLOP/s (among others 491, 1.89); 9.1 us (9.5)
// at 4 units over 4096 tokens, 11.5 (13.8) at 5 x 3 of 40 heads over 10007: launch, set-up, 147 KB of keys a CTA, one or two products.
// (-lse log2 e and the scale in two floats each: 453 us for 443 and the same error, which is the tensor core's own.)
constexpr int kWRing = 4;                      // query columns in flight (16 KB each)
constexpr int kWEpilogue = 128, kWLoadWarp = 4, kWMmaWarp = 5, kWThreads = 192;
constexpr uint32_t kWTmemCols = 512;           // two products of 256 columns
struct alignas(16) WeighCtl {
    uint64_t a_full[kBoxes], a_free[kBoxes];   // key columns (full: in rank 0, the bytes of both CTAs)
    uint64_t b_full[kWRing], b_free[kWRing];   // query columns
    uint64_t d_full[2], d_free[2];             // products (free: in rank 0, a warp of either CTA's epilogue)
    uint64_t fin;                              // every product has completed
    alignas(16) float neg[2][2 * kTileRows];   // -lse log2 e of a product's query rows
    uint32_t tmem_base, abort;
};
constexpr uint32_t kWOffRing = kBoxes * kTileBox, kWOffCtl = kWOffRing + kWRing * kTileBox, kWSmem = kWOffCtl + sizeof(WeighCtl);
static_assert(kWSmem <= kSmemLimit, "shared memory of weigh_kernel");

struct WeighPlan {
    int tiles;     // of 256 keys, a layer
    int pairs;     // of tiles of query rows
    int shares;    // of the query rows
    int pieces;    // tiles * layers * shares, in this order (the tile fastest)
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWThreads, 1)
    weigh_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap q_map, PrefixShape p,
                 WeighPlan plan, const float* lse, const float* weights, int64_t weights_stride, float* out, int64_t out_stride,
                 float* part, float scale_log2, float gain, uint32_t* err, int withhold)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    WeighCtl& c = *reinterpret_cast<WeighCtl*>(smem + kWOffCtl);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;  // (the compiler sees that a warp stays together)
    const int cl = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    const uint32_t rank = blockIdx.x & 1u;
    const int per = entries_a_tile(p.heads);
    volatile uint32_t* abort = &c.abort;

    chain_next();
    if (tid == 0) {
        for (int i = 0; i < kBoxes; ++i) {
            tc::mbar_init(&c.a_full[i], 1);
            tc::mbar_init(&c.a_free[i], 1);
        }
        for (int i = 0; i < kWRing; ++i) {
            tc::mbar_init(&c.b_full[i], 1);
            tc::mbar_init(&c.b_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&c.d_full[i], 1);
            tc::mbar_init(&c.d_free[i], 2 * kWEpilogue / 32);
        }
        tc::mbar_init(&c.fin, 1);
        c.abort = 0u;
    }
    // query rows behind the last of a tile are zeros for good (a copy writes whole entries only)
    for (uint32_t i = tid; i < kWRing * kTileBox / 16; i += kWThreads)
        reinterpret_cast<uint4*>(smem + kWOffRing)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_smem_async();
    if (warp == kWMmaWarp) tc::tmem2_alloc(&c.tmem_base, kWTmemCols);
    tc::fence_before_sync();
    tc::cluster_sync();  // both CTAs' barriers exist
    tc::fence_after_sync();
    const uint32_t tbase = c.tmem_base;
    chain_wait();
    lse = behind_wait(lse);
    const float* before = weights ? behind_wait(weights) : nullptr;

    auto first_pair = [&](int share) { return (int)((int64_t)share * plan.pairs / plan.shares); };
    auto piece_of = [&](int i, int& l, int& tile, int& p0, int& p1) {
        tile = i % plan.tiles;
        const int rest = i / plan.tiles, share = rest / p.layers;
        l = rest - share * p.layers;
        p0 = first_pair(share);
        p1 = first_pair(share + 1);
        return share;
    };

    if (warp == kWLoadWarp) {
        if (lane == 0 && !withhold) {
            // rank 0's barriers count the bytes of both CTAs
            const uint32_t af = tc::map_to_rank(tc::smem_u32(&c.a_full[0]), 0), bf = tc::map_to_rank(tc::smem_u32(&c.b_full[0]), 0);
            const uint32_t q_bytes = (uint32_t)(per * p.heads) * 128u;
            bool ok = true;
            int g = 0, n = 0;  // query columns, pieces
            for (int i = cl; ok && i < plan.pieces; i += ncl, ++n) {
                int l, tile, p0, p1;
                piece_of(i, l, tile, p0, p1);
                for (int pr = p0; ok && pr < p1; ++pr)
                    for (int x = 0; x < kBoxes; ++x, ++g) {
                        if (pr == p0) {
                            if (n > 0 && !(ok = wait_phase(&c.a_free[x], (n - 1) & 1, abort))) break;
                            if (rank == 0) tc::mbar_arrive_expect_tx(&c.a_full[x], 2 * kTileBox);
                            tc::tma2_load3(tc::smem_u32(smem) + x * kTileBox, &key_map, 64 * x + l * p.map_x, 256 * tile + 128 * (int)rank,
                                           l * p.map_z, af + 8 * x);
                        }
                        const int st = g % kWRing;
                        if (g >= kWRing && !(ok = wait_phase(&c.b_free[st], ((g / kWRing) - 1) & 1, abort))) break;
                        if (rank == 0) tc::mbar_arrive_expect_tx(&c.b_full[st], 2 * q_bytes);
                        tc::tma2_load4(tc::smem_u32(smem) + kWOffRing + st * kTileBox, &q_map, 64 * x, 0, l, (2 * pr + (int)rank) * per,
                                       bf + 8 * st);
                    }
            }
            if (!ok) give_up(&c.abort, err);
        }
        __syncwarp();
    } else if (warp == kWMmaWarp) {
        if (rank == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(256, 256, 0), tb = __shfl_sync(0xFFFFFFFFu, tbase, 0);
            const uint64_t da = tc::sw128_kmajor_desc(tc::smem_u32(smem)), db = tc::sw128_kmajor_desc(tc::smem_u32(smem) + kWOffRing);
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, abort)); };
            bool ok = true;
            int g = 0, n = 0, it = 0;
            for (int i = cl; ok && i < plan.pieces; i += ncl, ++n) {
                int l, tile, p0, p1;
                piece_of(i, l, tile, p0, p1);
                for (int pr = p0; ok && pr < p1; ++pr, ++it) {
                    const int d = it & 1;
                    if (it >= 2 && !(ok = wait(&c.d_free[d], ((it >> 1) - 1) & 1))) break;
                    for (int x = 0; x < kBoxes; ++x, ++g) {
                        const int st = g % kWRing;
                        if (pr == p0 && !(ok = wait(&c.a_full[x], n & 1))) break;
                        if (!(ok = wait(&c.b_full[st], (g / kWRing) & 1))) break;
                        tc::fence_after_sync();
                        tc::mma2_bf16_x4_warp<2, 2>(tb + 256 * d, da + ((x * kTileBox) >> 4), db + ((st * kTileBox) >> 4), idesc,
                                                    x > 0 ? 1u : 0u);
                        tc::mma2_commit_warp(&c.b_free[st], 3);
                        if (pr + 1 == p1) tc::mma2_commit_warp(&c.a_free[x], 3);
                    }
                    if (ok) tc::mma2_commit_warp(&c.d_full[d], 3);
                }
            }
            if (!ok && lane == 0) give_up(&c.abort, err);
            tc::mma2_commit_warp(&c.fin, 3);
        }
    } else {
        const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
        const uint32_t df = tc::map_to_rank(tc::smem_u32(&c.d_free[0]), 0);
        auto neg_of = [&](int l, int tile) {
            const int64_t r = tile_row(p, l, tile, tid);
            const float e = r >= 0 ? lse[r] : -INFINITY;
            return e == -INFINITY ? -INFINITY : -e * kLog2e;  // a row that is none, or attended to nothing, adds nothing
        };
        bool ok = true;
        int it = 0;
        for (int i = cl; i < plan.pieces; i += ncl) {
            int l, tile, p0, p1;
            const int share = piece_of(i, l, tile, p0, p1);
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int pr = p0; pr < p1; ++pr, ++it) {
                const int d = it & 1;
                float* neg = c.neg[d];
                const float n0 = neg_of(l, 2 * pr), n1 = neg_of(l, 2 * pr + 1);
                neg[tid] = n0;
                neg[kTileRows + tid] = n1;
                const bool gaps = tc::named_sync_or(1, kWEpilogue, n0 == -INFINITY || n1 == -INFINITY);
                // a give-up must not leave the other threads at a barrier
                ok = ok && wait_phase(&c.d_full[d], (it >> 1) & 1, abort);
                if (__all_sync(0xFFFFFFFFu, ok)) {
                    tc::fence_after_sync();
                    // A row that adds nothing may have a NaN score (a key that holds an infinity, by a zero), so where there are
                    // such rows they are left out one by one (443 us at 192 x 2 units over 16K tokens, 473 with it).
                    auto sum_columns = [&](auto with_gaps) {
#pragma unroll 1
                        for (int c0 = 0; c0 < 2 * kTileRows; c0 += 32) {
                            float v[32];
                            tc::tmem_ld32(tl + 256 * d + c0, v);
#pragma unroll
                            for (int x = 0; x < 32; x += 4) {
                                const float4 f4 = *reinterpret_cast<const float4*>(neg + c0 + x);
                                const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const float e = ex2(fmaf(v[x + y], scale_log2, f[y]));
                                    acc[y] += decltype(with_gaps)::value && f[y] == -INFINITY ? 0.0f : e;
                                }
                            }
                        }
                    };
                    if (gaps)
                        sum_columns(std::true_type{});
                    else
                        sum_columns(std::false_type{});
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive_at(df + 8 * d);
                }
            }
            const int j = 256 * tile + 128 * (int)rank + tid;
            const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            if (ok && j < p.n) {
                if (plan.shares > 1)
                    part[((int64_t)share * p.layers + l) * p.n + j] = sum;
                else
                    out[(p.layer0 + l) * out_stride + j] =
                        fmaf(gain, sum, before ? before[(p.layer0 + l) * weights_stride + j] : 0.0f);
            }
        }
        if (!ok) give_up(&c.abort, err);
    }
    pair_exit(&c.fin, &c.abort, err, tbase, warp == kWMmaWarp, kWTmemCols);
}

__global__ void __launch_bounds__(256) weigh_sum_kernel(PrefixShape p, int shares, const float* part, const float* weights,
                                                        int64_t weights_stride, float* out, int64_t out_stride, float gain)
{
    chain_next();
    chain_wait();
    part = behind_wait(part);
    const int l = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
    if (j >= p.n) return;
    float sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < shares; ++i) sum += part[((int64_t)i * p.layers + l) * p.n + j];
    const float before = weights ? behind_wait(weights)[(p.layer0 + l) * weights_stride + j] : 0.0f;
    out[(p.layer0 + l) * out_stride + j] = fmaf(gain, sum, before);
}

// Shares of the query rows such that the clusters' last round is full: rounds * (a share's products + reading the keys,
// which takes as long as one product).
WeighPlan weigh_plan(int64_t n, int B, int heads, int layers, int device_sms)
{
    const int ncl = std::max(1, device_sms / 2);
    const int64_t tiles = (n + 255) / 256, rows = ((int64_t)B + entries_a_tile(heads) - 1) / entries_a_tile(heads), pairs = (rows + 1) / 2;
    WeighPlan best{(int)tiles, (int)pairs, 1, (int)(tiles * layers)};
    int64_t least = INT64_MAX;
    for (int64_t s = 1; s <= std::min<int64_t>(pairs, 32); ++s) {
        const int64_t rounds = (tiles * layers * s + ncl - 1) / ncl, cost = rounds * ((pairs + s - 1) / s + 1) + (s > 1 ? 1 : 0);
        if (cost < least && tiles * layers * s <= INT32_MAX) {
            least = cost;
            best.shares = (int)s;
            best.pieces = (int)(tiles * layers * s);
        }
    }
    return best;
}

// How a tensor map holds the rows of a launch's layers.  Every stride of a map has to be a multiple of the one before it, so
// planes [layers][n][576] where a layer's stride is a multiple of a row's; where the layers lie side by side within a row's
// stride (a cache [n][layers][576]) columns of one plane; else (layers padded by a part of a row) a launch takes one layer.
enum class RowsMap { kPlanes, kColumns, kOneLayer };
int64_t columns_bytes(const PrefixShape& p) { return (p.layers - 1) * p.layer_stride + kRowBytes; }
RowsMap rows_map(const PrefixShape& p)
{
    const int64_t row = p.row_stride, layer = p.layer_stride;
    if (p.layers == 1 || p.n == 0) return RowsMap::kPlanes;
    if (p.n == 1) return layer >= kRowBytes ? RowsMap::kPlanes : RowsMap::kOneLayer;
    if (row < kRowBytes || layer % row == 0) return RowsMap::kPlanes;  // (fewer bytes a row are refused where the rows are read)
    // (a column's number has 32 bits)
    const bool beside = layer >= kRowBytes && layer <= INT32_MAX && row >= columns_bytes(p) && columns_bytes(p) <= INT32_MAX;
    return beside ? RowsMap::kColumns : RowsMap::kOneLayer;
}
int launch_layers(const PrefixShape& p) { return rows_map(p) == RowsMap::kOneLayer ? 1 : p.layers; }

// Calls f(the shape of a launch, units before its first one) for each launch on a tensor map that the call takes.
template <typename F>
cudaError_t for_each_launch(PrefixShape p, F f)
{
    if (launch_layers(p) == p.layers) {
        p.map_x = rows_map(p) == RowsMap::kColumns ? (int)(p.layer_stride / 2) : 0;
        p.map_z = p.map_x ? 0 : 1;
        return f(p, (int64_t)0);
    }
    cudaError_t e = cudaSuccess;
    const int layer0 = p.layer0, layers = p.layers;
    p.layers = 1;
    p.map_x = p.map_z = 0;
    for (int l = 0; l < layers && e == cudaSuccess; ++l) {
        p.layer0 = layer0 + l;
        e = f(p, (int64_t)l);
    }
    return e;
}

// The rows of a launch's layers, box `box` rows by 64 columns; the queries as [B][layers][heads][576], box the
// entries of a tile by 64 columns.  128-byte swizzle; what lies outside reads as zeros.
cudaError_t encode_rows(const PrefixShape& p, int box, CUtensorMap* map)
{
    TensorMapEncoder encode = nullptr;
    const cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess) return e;
    const bool columns = p.map_x != 0;
    const cuuint64_t dims[3] = {(cuuint64_t)(columns ? columns_bytes(p) / 2 : kDim), (cuuint64_t)p.n, (cuuint64_t)(columns ? 1 : p.layers)};
    // the stride of an axis with one entry is never used: the next one's, or the one's before
    const int64_t row = p.n > 1 ? p.row_stride : p.layers > 1 ? p.layer_stride : kRowBytes;
    const cuuint64_t strides[2] = {(cuuint64_t)row, (cuuint64_t)(columns || p.layers == 1 ? row : p.layer_stride)};
    const cuuint32_t boxes[3] = {64, (cuuint32_t)box, 1}, ones[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t*>(p.rows) + p.layer0 * p.layer_stride, dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}
cudaError_t encode_queries(const PrefixShape& p, const void* q, CUtensorMap* map)
{
    TensorMapEncoder encode = nullptr;
    const cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[4] = {kDim, (cuuint64_t)p.heads, (cuuint64_t)p.layers, (cuuint64_t)p.B};
    const cuuint64_t strides[3] = {kRowBytes, (cuuint64_t)kRowBytes * p.heads, (cuuint64_t)kRowBytes * p.heads * p.unit_layers};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)p.heads, 1, (cuuint32_t)entries_a_tile(p.heads)}, ones[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, boxes, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

dim3 weigh_sum_grid(const PrefixShape& p) { return dim3((unsigned)((p.n + 255) / 256), (unsigned)p.layers); }
// The weights as they are (an empty batch).
cudaError_t launch_weigh_nothing(const PrefixShape& p, const float* weights, int64_t weights_stride, float* out, int64_t out_stride,
                                 cudaStream_t st)
{
    return launch_chained(weigh_sum_kernel, weigh_sum_grid(p), 256, 0, st, p, 0, static_cast<const float*>(nullptr), weights, weights_stride,
                          out, out_stride, 0.0f);
}

cudaError_t launch_weigh(const PrefixShape& p, const void* q, const float* lse, const float* weights,
                         int64_t weights_stride, float* out, int64_t out_stride, float sm_scale, float gain, float* part,
                         uint32_t* err, int device_sms, cudaStream_t st, bool withhold = false)
{
    const WeighPlan plan = weigh_plan(p.n, p.B, p.heads, p.layers, device_sms);
    CUtensorMap key_map, q_map;
    cudaError_t e = encode_rows(p, kTileRows, &key_map);
    if (e == cudaSuccess) e = encode_queries(p, q, &q_map);
    if (e != cudaSuccess) return e;
    const unsigned grid = 2u * (unsigned)std::min(plan.pieces, std::max(1, device_sms / 2));
    e = launch_chained(weigh_kernel, dim3(grid), kWThreads, kWSmem, st, key_map, q_map, p, plan, lse, weights, weights_stride, out,
                       out_stride, part, sm_scale * kLog2e, gain, err, withhold ? 1 : 0);
    if (e != cudaSuccess || plan.shares == 1) return e;
    return launch_chained(weigh_sum_kernel, weigh_sum_grid(p), 256, 0, st, p, plan.shares,
                          static_cast<const float*>(part), weights, weights_stride, out, out_stride, gain);
}

// ---------------------------------------------------------------------------
// Attention.  Tensor memory holds half of a tile's 128 x 512 output beside the scores, so
// a cluster of four CTAs, two pairs that multiply as one each, takes an item of the work: a pair
// of query tiles (256 rows of a product).  CTA (h, r), of pair h and row tile r, owns the value dims
// [256h, 256h + 256) of tile r, and of every block of 128 keys its pair scores the keys [64h, 64h + 64):
//   S = Q K^T   256 rows, the pair's 64 keys (32 from either CTA), 576 dims in columns of 64
//   O += P V    256 rows, 128 keys, the pair's 256 value dims (128 from either CTA)
// so nothing is multiplied twice.  The CTAs (0, r) and (1, r) swap their row maxima (both take the same reference
// maximum) and their halves of P, and at an item's end their shares of the sums.
// The softmax has a query row a thread (the row's tensor-memory lane).  It takes the exponentials with the
// reference there is while the maxima travel, and again if it has risen.  P is rounded to bf16, which is what the tensor cores take at full
// rate; the output is divided by the sum of the rounded values.  With the output's own rounding it is all that the result is off by: 1.7e-3 to
// 1.9e-3 of its size against 64 bits, 1.65e-3 to 1.7e-3 with P in fp32.  P goes into shared memory, by
// a bulk copy into the other pair's as well.
// Items that do not fill the clusters evenly are split along the keys; combine_prefix_kernel joins their parts.
// An item's queries are its products' first operand, 384 of their 576 dims in tensor memory; those come by way of the P and V tiles,
// which nothing has used yet (or has finished with: item_done), and the values are loaded once they have been taken.
// PV(g) is issued once S(g + 1) is (s_issued), so that the two streams of products take turns and the softmax of g + 1 starts early.
// What bounds it: the products, 2176 cycles a block (36 of 256 x 64 x 16, 8 of 256 x 256 x 16), beside which shared memory
// moves 265 KB (2070 cycles); from S to P there are an exchange of maxima, 64 exponentials a thread and the copy of P, some 2500 cycles, which
// the products of the next scores cover.  Measured: 913 to 933 us at 192 x 2 units over 16K tokens, 1.88 to 1.92 PFLOP/s in a burst of 2 ms
// (970 to 996 in one of 15 ms; among others 1046, 1.68); 174 us at 8 units over 128K, 1.68 (among others 189, 1.55); 12.9 us (14.2) at 2 over
// 1000, 17.9 (18.7) at 7 x 3 of 16 heads over 5003, where a
// launch, the queries' way into tensor memory (2 us), one block's chain, the parts' way out (2 us) and the joining kernel (3 us) are all there is.
// On the way here, at 192 x 2 units: a pair for each half of the value dims, both taking all scores, 1539 us; this decomposition
// with one warp for both streams of products 1075; waits and arrivals at cluster scope and the scores' columns in stages of their
// own 2151.  The code has to stay small: with 112 KB of it instead of 60 the instruction caches, which GPCs share, were what
// bounded it (1628 us; GPCs with three clusters were done in 249 us where those with five took 340).
// With the queries read into tensor memory by plain loads and the products in the order they come: 932, 171, 13.6 and 18.5; waiting for the
// next P tile as soon as one is sent, ahead of the next scores, 994.
// Scores double-buffered, with more of Q in shared memory: 1118; P by st.async instead of bulk copies: 1079 (against 1050).
constexpr int kBlk = 128, kHalfBlk = 64;       // keys of a block, and those that a pair scores
constexpr int kKRing = 2, kVRing = 2;          // key stages (32 keys, 36 KB), value stages (64 keys x 128 dims, 16 KB)
constexpr uint32_t kKBox = 32 * 128, kKStage = kBoxes * kKBox, kVBox = 64 * 128, kVStage = 2 * kVBox;
constexpr uint32_t kPBox = kTileRows * 128, kPTile = 2 * kPBox;  // P: 128 rows x 64 keys of a pair, both pairs' (two tiles)
constexpr int kVHalf = kVDim / 2;
constexpr int kQtBoxes = 6, kQsBoxes = kBoxes - kQtBoxes;  // query columns in tensor memory, in shared memory
constexpr uint32_t kColO = 0, kColS = 256, kColQ = 320;    // tensor memory: O 256 columns, S 64, Q 192
constexpr int kQWarp0 = 4, kAKeyWarp = 8, kAValueWarp = 9, kAScoreWarp = 10, kAValueMmaWarp = 11, kAThreads = 384;
constexpr float kRescaleLog2 = 8.0f;           // the reference maximum is raised when a score passes it by 2^8
struct alignas(16) AttendCtl {
    // "leader": the barrier of the pair's first CTA, which multiplies
    uint64_t q_full, q_tm, q_free;             // queries in shared memory (leader, bytes of both CTAs), in tensor memory
                                               // (leader, a warp of either CTA); the item's scores are done (both)
    uint64_t q_way, way_free;                  // queries on their way to tensor memory have arrived; have been taken (a warp each)
    uint64_t k_full[kKRing], k_free[kKRing];   // key stages (leader, bytes of both CTAs; both)
    uint64_t v_full[kVRing], v_free[kVRing];   // value stages
    uint64_t s_full, s_free;                   // a block's scores are complete (both); have been read (leader, a warp of either)
    uint64_t s_issued[4];                      // a block's scores are on their way (in the first CTA; they may be three blocks ahead)
    uint64_t m_full[2];                        // the other pair's maxima of a block have arrived (512 bytes)
    uint64_t x_full[2];                        // the other pair's half of a P tile has arrived (16 KB)
    uint64_t p_full[2];                        // a P tile is complete (leader: a warp of either CTA, and the second CTA once x_full)
    uint64_t pv_done[2];                       // O += P V of a block has completed in both pairs (all four CTAs)
    uint64_t item_done;                        // the last of an item's, as well, where another item follows (a waiter that does not follow the blocks)
    uint64_t l_full;                           // the other pair's shares of the sums have arrived (1024 bytes)
    uint64_t o_free;                           // an item's output has been read (leader, a warp of either CTA)
    uint64_t fin;                              // every product of the pair has completed (both streams)
    float mx[2][kTileRows], lx[kTileRows], rx[kTileRows];  // the other pair's maxima and sums
    uint32_t tmem_base, abort;
};
constexpr uint32_t kAOffP = kQsBoxes * kTileBox, kAOffK = kAOffP + 2 * kPTile, kAOffV = kAOffK + kKRing * kKStage,
                   kAOffCtl = kAOffV + kVRing * kVStage, kASmem = kAOffCtl + sizeof(AttendCtl);
static_assert(kASmem <= kSmemLimit && kAOffV % 1024 == 0, "shared memory of attend_prefix_kernel");
static_assert(2 * kPTile == 4 * kTileBox && kVRing * kVStage == 2 * kTileBox && kQtBoxes == 6, "the queries' way");
static_assert(kColQ + kQtBoxes * 32 <= 512, "tensor memory of attend_prefix_kernel");

struct AttendPlan {
    int pairs;            // of query tiles, a layer
    int direct, rest;     // items that clusters do whole, and those that are split
    int splits, blocks;   // of one of the latter; key blocks a split
    int all_blocks;       // key blocks of the prefix
    float* o;             // results of the splits: [rest * splits * 4 CTAs][256 / 4][128 rows][4], normalised
    float* lse;           // [rest * splits * 2 tiles][128], log2
    __host__ __device__ int pieces() const { return direct + rest * splits; }
    // Pieces: the whole items, then the first splits of the others, then their second ones (so that neighbours read the same keys).
    __device__ int item(int piece) const { return piece < direct ? piece : direct + (piece - direct) % rest; }
    __device__ int split(int piece) const { return piece < direct ? 0 : (piece - direct) / rest; }
};

__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kAThreads, 1)
    attend_prefix_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap value_map,
                         const __grid_constant__ CUtensorMap q_map, PrefixShape p, AttendPlan plan,
                         uint16_t* out, float* lse, float scale_log2, uint32_t* err, int withhold)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    AttendCtl& c = *reinterpret_cast<AttendCtl*>(smem + kAOffCtl);
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;  // (the compiler sees that a warp stays together)
    const int cl = blockIdx.x >> 2, ncl = gridDim.x >> 2;
    const uint32_t rank = blockIdx.x & 3u, half = rank >> 1, r = rank & 1u, leader = rank & 2u, peer = rank ^ 2u;
    const int per = entries_a_tile(p.heads), pieces = plan.pieces();
    volatile uint32_t* abort = &c.abort;

    chain_next();
    if (tid == 0) {
        tc::mbar_init(&c.q_full, 1);
        tc::mbar_init(&c.q_tm, 8);
        tc::mbar_init(&c.q_free, 1);
        tc::mbar_init(&c.q_way, 1);
        tc::mbar_init(&c.way_free, 4);
        for (int i = 0; i < kKRing; ++i) {
            tc::mbar_init(&c.k_full[i], 1);
            tc::mbar_init(&c.k_free[i], 1);
        }
        for (int i = 0; i < kVRing; ++i) {
            tc::mbar_init(&c.v_full[i], 1);
            tc::mbar_init(&c.v_free[i], 1);
        }
        tc::mbar_init(&c.s_full, 1);
        for (int i = 0; i < 4; ++i) tc::mbar_init(&c.s_issued[i], 1);
        tc::mbar_init(&c.s_free, 8);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&c.m_full[i], 1);
            tc::mbar_init(&c.x_full[i], 1);
            tc::mbar_init(&c.p_full[i], 9);
            tc::mbar_init(&c.pv_done[i], 2);
        }
        tc::mbar_init(&c.item_done, 2);
        tc::mbar_init(&c.l_full, 1);
        tc::mbar_init(&c.o_free, 8);
        tc::mbar_init(&c.fin, 2);
        c.abort = 0u;
    }
    if (per * p.heads < kTileRows) {  // query rows behind the last of a tile are zeros for good (a copy writes whole entries only)
        for (uint32_t i = tid; i < kQsBoxes * kTileBox / 16; i += kAThreads)
            reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
        tc::fence_smem_async();
    }
    if (warp == kAScoreWarp) tc::tmem2_alloc(&c.tmem_base, 512);
    tc::fence_before_sync();
    tc::cluster_sync();  // all CTAs' barriers exist
    tc::fence_after_sync();
    const uint32_t tbase = c.tmem_base;
    chain_wait();

    // a piece of the work: layer, pair of query tiles, key blocks [b0, b1)
    struct Piece {
        int l, pair, b0, b1;
    };
    auto piece_of = [&](int i) {
        const int item = plan.item(i);
        Piece w;
        w.l = item / plan.pairs;
        w.pair = item - w.l * plan.pairs;
        w.b0 = i < plan.direct ? 0 : plan.split(i) * plan.blocks;
        w.b1 = i < plan.direct ? plan.all_blocks : min(plan.all_blocks, w.b0 + plan.blocks);
        return w;
    };
    // where column x of the queries passes on its way to tensor memory
    auto way_of = [&](int x) -> uint32_t { return x < 4 ? kAOffP + x * kTileBox : kAOffV + (x - 4) * kTileBox; };
    auto at_leader = [&](uint64_t* bar) { return tc::map_to_rank(tc::smem_u32(bar), leader); };

    if (warp == kAKeyWarp) {
        if (lane == 0 && !withhold) {
            const uint32_t qf = at_leader(&c.q_full), qw = tc::map_to_rank(tc::smem_u32(&c.q_way), rank);
            const uint32_t kf = at_leader(&c.k_full[0]), q_bytes = (uint32_t)(per * p.heads) * 128u;
            bool ok = true;
            int g = 0, n = 0;  // blocks, pieces
            for (int i = cl; ok && i < pieces; i += ncl, ++n) {
                const Piece w = piece_of(i);
                for (int b = w.b0; b < w.b1; ++b, ++g) {
                    const int st = g % kKRing;
                    if (g >= kKRing && !(ok = wait_phase(&c.k_free[st], ((g / kKRing) - 1) & 1, abort))) break;
                    if (r == 0) tc::mbar_arrive_expect_tx(&c.k_full[st], 2 * kKStage);
#pragma unroll 1
                    for (int x = 0; x < kBoxes; ++x)
                        tc::tma2_load3(tc::smem_u32(smem) + kAOffK + st * kKStage + x * kKBox, &key_map, 64 * x + w.l * p.map_x,
                                       kBlk * b + kHalfBlk * (int)half + 32 * (int)r, w.l * p.map_z, kf + 8 * st);
                    if (b == w.b0) {  // the item's queries: most of them by way of the P and V tiles, once those are free
                        if (n > 0 && !(ok = wait_phase(&c.q_free, (n - 1) & 1, abort) &&
                                            wait_phase(&c.item_done, (n - 1) & 1, abort)))
                            break;
                        tc::mbar_arrive_expect_tx(&c.q_way, kQtBoxes * q_bytes);
                        if (r == 0) tc::mbar_arrive_expect_tx(&c.q_full, 2 * kQsBoxes * q_bytes);
#pragma unroll 1
                        for (int x = 0; x < kBoxes; ++x)
                            tc::tma2_load4(tc::smem_u32(smem) + (x < kQtBoxes ? way_of(x) : (x - kQtBoxes) * kTileBox), &q_map, 64 * x,
                                           0, w.l, (2 * w.pair + (int)r) * per, x < kQtBoxes ? qw : qf);
                    }
                }
            }
            if (!ok) give_up(&c.abort, err);
        }
        __syncwarp();
    } else if (warp == kAValueWarp) {
        if (lane == 0 && !withhold) {
            const uint32_t vf = at_leader(&c.v_full[0]);
            bool ok = true;
            int g = 0, n = 0;  // value stages, pieces
            for (int i = cl; ok && i < pieces; i += ncl, ++n) {
                const Piece w = piece_of(i);
                if (!(ok = wait_phase(&c.way_free, n & 1, abort))) break;
                for (int b = 2 * w.b0; b < 2 * w.b1; ++b, ++g) {
                    const int st = g % kVRing;
                    if (g >= kVRing && !(ok = wait_phase(&c.v_free[st], ((g / kVRing) - 1) & 1, abort))) break;
                    if (r == 0) tc::mbar_arrive_expect_tx(&c.v_full[st], 2 * kVStage);
#pragma unroll 1
                    for (int x = 0; x < 2; ++x)
                        tc::tma2_load3(tc::smem_u32(smem) + kAOffV + st * kVStage + x * kVBox, &value_map,
                                       kVHalf * (int)half + 128 * (int)r + 64 * x + w.l * p.map_x, 64 * b, w.l * p.map_z, vf + 8 * st);
                }
            }
            if (!ok) give_up(&c.abort, err);
        }
        __syncwarp();
    } else if (warp == kAScoreWarp) {
        // The two streams of products have a warp each: the tensor pipe takes few products ahead, and what a warp spends on
        // its waits and commits the other's products fill.
        if (r == 0) {
            const uint32_t idesc = tc::idesc_bf16_f32(256, kHalfBlk, 0);
            const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0), base = tc::smem_u32(smem);
            const uint32_t mine = 3u << __shfl_sync(0xFFFFFFFFu, leader, 0);  // the CTAs of this pair
            const uint64_t dq = tc::sw128_kmajor_desc(base), dk = tc::sw128_kmajor_desc(base + kAOffK);
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, abort)); };
            bool ok = true;
            int n = 0, g = 0;  // pieces, blocks
            for (int i = cl; ok && i < pieces; i += ncl, ++n) {
                const Piece w = piece_of(i);
                if (!(ok = wait(&c.q_tm, n & 1) && wait(&c.q_full, n & 1))) break;
                for (int b = w.b0; b < w.b1; ++b, ++g) {
                    const int st = g % kKRing;
                    if (!(ok = wait(&c.k_full[st], (g / kKRing) & 1))) break;
                    if (g > 0 && !(ok = wait(&c.s_free, (g - 1) & 1))) break;
                    tc::fence_after_sync();
                    const uint64_t ds = dk + ((st * kKStage) >> 4);
#pragma unroll 1
                    for (int x = 0; x < kQtBoxes; ++x)
                        tc::mma2_bf16_ta_x4_warp<8, 2>(tb + kColS, tb + kColQ + 32 * x, ds + ((x * kKBox) >> 4), idesc, x > 0 ? 1u : 0u);
#pragma unroll 1
                    for (int x = kQtBoxes; x < kBoxes; ++x)
                        tc::mma2_bf16_x4_warp<2, 2>(tb + kColS, dq + (((x - kQtBoxes) * kTileBox) >> 4), ds + ((x * kKBox) >> 4), idesc, 1u);
                    if (lane == 0) tc::mbar_arrive(&c.s_issued[g & 3]);
                    __syncwarp();
                    tc::mma2_commit_warp(&c.s_full, mine);
                    tc::mma2_commit_warp(&c.k_free[st], mine);
                    if (b + 1 == w.b1) tc::mma2_commit_warp(&c.q_free, mine);
                }
            }
            if (!ok && lane == 0) give_up(&c.abort, err);
            tc::mma2_commit_warp(&c.fin, mine);
        }
    } else if (warp == kAValueMmaWarp) {
        const uint32_t pf = at_leader(&c.p_full[0]);
        const uint32_t idesc = tc::idesc_bf16_f32(256, kVHalf, 1);
        const uint32_t tb = __shfl_sync(0xFFFFFFFFu, tbase, 0), base = tc::smem_u32(smem);
        const uint32_t mine = 3u << __shfl_sync(0xFFFFFFFFu, leader, 0);
        const uint64_t dp = tc::sw128_kmajor_desc(base + kAOffP), dv = tc::sw128_mnmajor_desc(base + kAOffV, kVBox);
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, abort)); };
        bool ok = true;
        int gv = 0, n = 0, g = 0;  // value stages, pieces, blocks
        for (int i = cl; ok && i < pieces; i += ncl, ++n) {
            const Piece w = piece_of(i);
            for (int b = w.b0; b < w.b1; ++b, ++g) {
                // the other pair's half of P
                if (lane == 0) tc::mbar_arrive_expect_tx(&c.x_full[g & 1], kPBox);
                __syncwarp();
                if (!(ok = wait(&c.x_full[g & 1], (g >> 1) & 1))) break;
                tc::fence_smem_async();
                if (r == 1) {  // this CTA's part of it is there
                    if (lane == 0) tc::mbar_arrive_at(pf + 8 * (g & 1));
                    __syncwarp();
                    continue;
                }
                if (!(ok = wait(&c.p_full[g & 1], (g >> 1) & 1))) break;
                if (b == w.b0 && n > 0 && !(ok = wait(&c.o_free, (n - 1) & 1))) break;  // the item before has read its O
                // behind the next block's scores, which the softmax waits for
                if (b + 1 < w.b1 && !(ok = wait(&c.s_issued[(g + 1) & 3], ((g + 1) >> 2) & 1))) break;
#pragma unroll 1
                for (int h = 0; h < 2; ++h, ++gv) {
                    const int st = gv % kVRing;
                    if (!(ok = wait(&c.v_full[st], (gv / kVRing) & 1))) break;
                    tc::fence_after_sync();
                    tc::mma2_bf16_x4_warp<2, 128>(tb + kColO, dp + (((g & 1) * kPTile + h * kPBox) >> 4), dv + ((st * kVStage) >> 4),
                                                  idesc, b > w.b0 || h > 0 ? 1u : 0u);
                    tc::mma2_commit_warp(&c.v_free[st], mine);
                }
                if (!ok) break;
                tc::mma2_commit_warp(&c.pv_done[g & 1], 15);
                // only where its waiter comes: an arrival that nobody waits for could reach a CTA that has left
                if (b + 1 == w.b1 && i + ncl < pieces) tc::mma2_commit_warp(&c.item_done, 15);
            }
        }
        if (!ok && lane == 0) give_up(&c.abort, err);
        if (r == 0) tc::mma2_commit_warp(&c.fin, mine);
    } else if (warp >= kQWarp0) {
        // the first 384 dims of the item's queries into tensor memory, a row a thread (by plain loads of the rows, which lie 1152
        // bytes apart, it took a microsecond more)
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16) + kColQ, qt = at_leader(&c.q_tm);
        const int row = tid - 32 * kQWarp0;
        const bool is = row < per * p.heads;
        bool ok = true;
        int n = 0;
        for (int i = cl; i < pieces; i += ncl, ++n) {
            if (!(ok = __all_sync(0xFFFFFFFFu, wait_phase(&c.q_way, n & 1, abort)))) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int x = 0; x < kQtBoxes; ++x) {
                const uint8_t* at = smem + way_of(x) + row * 128;
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const uint4 lo = is ? *reinterpret_cast<const uint4*>(at + ((j ^ (row & 7)) << 4)) : make_uint4(0, 0, 0, 0);
                    const uint4 hi = is ? *reinterpret_cast<const uint4*>(at + (((j + 1) ^ (row & 7)) << 4)) : make_uint4(0, 0, 0, 0);
                    const uint32_t a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    tc::tmem_st8_async(tl + 32 * x + 4 * j, a);
                }
            }
            tc::tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&c.way_free);
                tc::mbar_arrive_at(qt);
            }
        }
        if (!ok) give_up(&c.abort, err);
    } else {
        const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
        const uint32_t sf = at_leader(&c.s_free), pf = at_leader(&c.p_full[0]), of = at_leader(&c.o_free);
        const uint32_t mx_peer = tc::map_to_rank(tc::smem_u32(&c.mx[0][tid]), peer), mf_peer = tc::map_to_rank(tc::smem_u32(&c.m_full[0]), peer);
        const uint32_t lx_peer = tc::map_to_rank(tc::smem_u32(&c.lx[tid]), peer), rx_peer = tc::map_to_rank(tc::smem_u32(&c.rx[tid]), peer);
        const uint32_t lf_peer = tc::map_to_rank(tc::smem_u32(&c.l_full), peer), xf_peer = tc::map_to_rank(tc::smem_u32(&c.x_full[0]), peer);
        // this warp's rows of this pair's half of P tile 0, here and at the other pair's CTA of the same rows
        const uint32_t p_at = kAOffP + half * kPBox + (uint32_t)warp * 4096u;
        const uint32_t p_mine = tc::smem_u32(smem) + p_at, p_peer = tc::map_to_rank(p_mine, peer);
        bool ok = true;
        int g = 0, n = 0;
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, abort)); };
        for (int i = cl; ok && i < pieces; i += ncl, ++n) {
            const Piece w = piece_of(i);
            float m_ref = -INFINITY;  // reference maximum (log2) that the exponentials use; the same in both pairs
            float l_run = 0.0f;       // the sum of P over this pair's keys
            float r_run = 0.0f;       // of P as rounded to bf16, which the output is divided by
            for (int b = w.b0; b < w.b1; ++b, ++g) {
                const int bb = g & 1, left = p.n - kBlk * b - kHalfBlk * (int)half;  // keys of this pair's half that exist
                if (!(ok = wait(&c.s_full, g & 1))) break;
                tc::fence_after_sync();
                float v[kHalfBlk];
                tc::tmem_ld32(tl + kColS, *reinterpret_cast<float(*)[32]>(v));
                tc::tmem_ld32(tl + kColS + 32, *reinterpret_cast<float(*)[32]>(v + 32));
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_at(sf);
                if (left < kHalfBlk) {
#pragma unroll
                    for (int j = 0; j < kHalfBlk; ++j) v[j] = j < left ? v[j] : -INFINITY;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < kHalfBlk; ++j) mx[j & 3] = fmaxf(mx[j & 3], v[j]);
                const float mloc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (tid == 0) tc::mbar_arrive_expect_tx(&c.m_full[bb], kTileRows * 4);
                tc::st_async4(mx_peer + bb * kTileRows * 4, mloc, mf_peer + 8 * bb);
                // P tile bb is free, here and there, once both pairs have multiplied block g - 2 by it
                if (g >= 2 && !(ok = wait(&c.pv_done[bb], ((g >> 1) - 1) & 1))) break;
                uint32_t pk[kHalfBlk / 2];
                uint64_t ls, rs;
                float factor = 1.0f;
                for (bool settled = false;; settled = true) {
                    const float neg_m = m_ref == -INFINITY ? 0.0f : -m_ref;  // (only keys that are masked, or NaN)
                    const uint64_t scale2 = pair(scale_log2, scale_log2), neg2 = pair(neg_m, neg_m);
                    uint64_t sums[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < kHalfBlk / 2; ++j) {
                        float p0, p1;
                        split(fma2(pair(v[2 * j], v[2 * j + 1]), scale2, neg2), p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        pk[j] = bf2(p0, p1);
                        sums[j & 1] = add2(sums[j & 1], pair(p0, p1));
                        sums[2 + (j & 1)] = add2(sums[2 + (j & 1)], pair(__uint_as_float(pk[j] << 16), __uint_as_float(pk[j] & 0xFFFF0000u)));
                    }
                    ls = add2(sums[0], sums[1]);
                    rs = add2(sums[2], sums[3]);
                    if (settled) break;
                    if (!(ok = wait(&c.m_full[bb], (g >> 1) & 1))) break;
                    const float mb = fmaxf(mloc, c.mx[bb][tid]) * scale_log2;
                    if (mb > m_ref + kRescaleLog2) {
                        factor = ex2(m_ref - mb);  // (0 from -inf)
                        m_ref = mb;
                        l_run *= factor;
                        r_run *= factor;
                    }
                    if (!__any_sync(0xFFFFFFFFu, factor != 1.0f)) break;
                }
                if (!ok) break;
                if (b > w.b0 && __any_sync(0xFFFFFFFFu, factor != 1.0f)) {  // rescale this warp's rows of O
                    if (!(ok = wait(&c.pv_done[bb ^ 1], ((g - 1) >> 1) & 1))) break;
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int c0 = 0; c0 < kVHalf; c0 += 32) {
                        float ov[32];
                        tc::tmem_ld32(tl + kColO + c0, ov);
#pragma unroll
                        for (int j = 0; j < 32; ++j) ov[j] *= factor;
                        tc::tmem_st32(tl + kColO + c0, ov);
                    }
                    tc::fence_before_sync();
                }
                float s0, s1;
                split(ls, s0, s1);
                l_run += s0 + s1;
                split(rs, s0, s1);
                r_run += s0 + s1;
                uint8_t* row = smem + p_at + bb * kPTile + lane * 128;
#pragma unroll
                for (int j = 0; j < kHalfBlk / 8; ++j)  // 16-byte pieces where the swizzle puts them
                    *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
                tc::fence_smem_async();
                __syncwarp();
                if (lane == 0) {
                    tc::bulk_to_peer(p_peer + bb * kPTile, p_mine + bb * kPTile, 4096, xf_peer + 8 * bb);
                    tc::mbar_arrive_at(pf + 8 * bb);
                }
            }
            if (!ok) break;
            // the sums: pair 0's share + pair 1's, in that order in both
            if (tid == 0) tc::mbar_arrive_expect_tx(&c.l_full, kTileRows * 8);
            tc::st_async4(lx_peer, l_run, lf_peer);
            tc::st_async4(rx_peer, r_run, lf_peer);
            if (!(ok = wait(&c.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1) && wait(&c.l_full, n & 1))) break;
            tc::fence_after_sync();
            const float l_all = half == 0 ? l_run + c.lx[tid] : c.lx[tid] + l_run;
            const float r_all = half == 0 ? r_run + c.rx[tid] : c.rx[tid] + r_run;
            const float inv = r_all == 0.0f ? 0.0f : 1.0f / r_all, lse2 = m_ref + log2f(l_all);  // (0: scores of -inf alone)
            if (i < plan.direct) {
                const int64_t at = tile_row(p, w.l, 2 * w.pair + (int)r, tid);
                uint16_t* o = out + at * kVDim + kVHalf * (int)half;
#pragma unroll 1
                for (int c0 = 0; c0 < kVHalf; c0 += 32) {
                    float ov[32];
                    tc::tmem_ld32(tl + kColO + c0, ov);
                    if (at >= 0) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
                            *reinterpret_cast<uint4*>(o + c0 + j) =
                                make_uint4(bf2(ov[j] * inv, ov[j + 1] * inv), bf2(ov[j + 2] * inv, ov[j + 3] * inv),
                                           bf2(ov[j + 4] * inv, ov[j + 5] * inv), bf2(ov[j + 6] * inv, ov[j + 7] * inv));
                    }
                }
                if (half == 0 && lse && at >= 0) lse[at] = lse2 * kLn2;
            } else {
                const int64_t slot = (int64_t)(plan.item(i) - plan.direct) * plan.splits + plan.split(i);
                float4* o = reinterpret_cast<float4*>(plan.o) + (4 * slot + rank) * (kVHalf / 4) * kTileRows + tid;
                const bool mine = tile_row(p, w.l, 2 * w.pair + (int)r, tid) >= 0;  // (nobody reads the others)
                if (__any_sync(0xFFFFFFFFu, mine))
#pragma unroll 1
                for (int c0 = 0; c0 < kVHalf; c0 += 32) {
                    float ov[32];
                    tc::tmem_ld32(tl + kColO + c0, ov);
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            o[(c0 + j) / 4 * kTileRows] = make_float4(ov[j] * inv, ov[j + 1] * inv, ov[j + 2] * inv, ov[j + 3] * inv);
                    }
                }
                if (half == 0) plan.lse[(2 * slot + r) * kTileRows + tid] = lse2;
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_at(of);
        }
        if (!ok) give_up(&c.abort, err);
    }
    pair_exit(&c.fin, &c.abort, err, tbase, warp == kAScoreWarp, 512);
}

// The splits of an item joined: with lse_i their log2 sums and M the largest, out = sum 2^(lse_i - M) o_i / sum 2^(lse_i - M).
// A thread a row and four columns; kAtOnce splits' numbers are in flight together (19.2 us instead of 21.3 for a call of 10 splits).
template <int kAtOnce>
__global__ void __launch_bounds__(512) combine_prefix_kernel(PrefixShape p, AttendPlan plan, uint16_t* out, float* lse)
{
    chain_next();
    chain_wait();
    const int row = threadIdx.x % kTileRows, col4 = blockIdx.x * 4 + threadIdx.x / kTileRows;
    const int rank = blockIdx.y & 3, half = rank >> 1, r = rank & 1, item = plan.direct + (int)(blockIdx.y >> 2);
    const int l = item / plan.pairs, pair = item - l * plan.pairs;
    const int64_t at = tile_row(p, l, 2 * pair + r, row), slot0 = (int64_t)(item - plan.direct) * plan.splits;
    if (at < 0) return;
    const float* ls = behind_wait(plan.lse) + (2 * slot0 + r) * kTileRows + row;
    const float4* po = reinterpret_cast<const float4*>(behind_wait(plan.o)) + ((4 * slot0 + rank) * (kVHalf / 4) + col4) * kTileRows + row;
    float m = -INFINITY, acc[4] = {}, total = 0.0f;
    for (int i0 = 0; i0 < plan.splits; i0 += kAtOnce) {
        float li[kAtOnce], top = m;
        float4 o[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const bool is = i0 + i < plan.splits;
            li[i] = is ? ls[(int64_t)(i0 + i) * 2 * kTileRows] : -INFINITY;
            o[i] = is ? po[(int64_t)(i0 + i) * kVHalf * kTileRows] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, li[i]);
        const float base = top == -INFINITY ? 0.0f : top, fix = ex2(m - base);  // (only NaN, or scores of -inf)
        total *= fix;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] *= fix;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const float w = ex2(li[i] - base);
            total += w;
            acc[0] = fmaf(w, o[i].x, acc[0]);
            acc[1] = fmaf(w, o[i].y, acc[1]);
            acc[2] = fmaf(w, o[i].z, acc[2]);
            acc[3] = fmaf(w, o[i].w, acc[3]);
        }
        m = top;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    *reinterpret_cast<uint2*>(out + at * kVDim + kVHalf * half + 4 * col4) =
        make_uint2(bf2(acc[0] * inv, acc[1] * inv), bf2(acc[2] * inv, acc[3] * inv));
    if (col4 == 0 && half == 0 && lse) lse[at] = (base + log2f(total)) * kLn2;
}

// What an attention over an empty prefix returns.
__global__ void __launch_bounds__(256) nothing_kernel(int64_t rows, uint4* out, float* lse)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * (kVDim / 8); i += (int64_t)gridDim.x * 256) {
        out[i] = make_uint4(0, 0, 0, 0);
        if (lse && i < rows) lse[i] = -INFINITY;
    }
}

// Whole items for full rounds of the clusters; the rest in splits such that its rounds are short.  In units of a block's time
// (1.25 us): rounds * (blocks + 2.5 for what a piece costs besides) and, for the joining of the parts, 2, what their bytes
// take (0.5 MB a split, written and read) and 0.8 for every 12 splits after the first 12.  Swept over the splits, the choice was
// the fastest or within 0.2 us of it at 2 x 1000 (12.9 us with 8 splits, 18.5 with one), 1 x 3000 (14.1 with 12, 15.7 with 24),
// 1 x 10000, 1 x 20000 (21.8 with 32, 23.3 with 23) and 1 x 100000, 2 x 2 x 3000 and 9000, 6 x 3000 and 20000, 2 x 8 x 2000 and 20000,
// 7 x 3 x 5003 of 16 heads (18.1 with 10, 20.3 with 8), 64 x 2000 (31.6 with one, 47.8 with 2) and 80 x 2000 tokens (46.0 with 8, 55.2 with one).
AttendPlan attend_plan(int64_t n, int B, int heads, int layers, int ncl)
{
    const int nblk = (int)((n + kBlk - 1) / kBlk);
    const int64_t tiles = ((int64_t)B + entries_a_tile(heads) - 1) / entries_a_tile(heads), pairs = (tiles + 1) / 2, items = pairs * layers;
    AttendPlan a{(int)pairs, (int)(items / ncl * ncl), (int)(items % ncl), 1, nblk, nblk, nullptr, nullptr};
    if (a.rest == 0) return a;
    double least = 1e30;
    for (int k = 1; k <= std::min(nblk, 64); ++k) {
        const int blocks = (nblk + k - 1) / k;
        if ((nblk + blocks - 1) / blocks != k) continue;  // the last splits would be empty
        const double cost = (double)((a.rest * (int64_t)k + ncl - 1) / ncl) * (blocks + 2.5) + (k > 1 ? 2.0 + 0.07 * k * a.rest + 0.8 * ((k - 1) / 12) : 0.0);
        if (cost < least) {
            least = cost;
            a.splits = k;
            a.blocks = blocks;
        }
    }
    if (a.splits == 1) {
        a.direct += a.rest;
        a.rest = 0;
    }
    return a;
}
int64_t attend_bytes(const AttendPlan& a) { return (int64_t)a.rest * a.splits * 2 * kTileRows * (kVDim + 1) * 4; }

cudaError_t launch_attend_nothing(const PrefixShape& p, void* out, float* lse, cudaStream_t st)
{
    const int64_t rows = (int64_t)p.B * p.layers * p.heads;
    nothing_kernel<<<(unsigned)std::min<int64_t>((rows * (kVDim / 8) + 255) / 256, 1 << 16), 256, 0, st>>>(rows, static_cast<uint4*>(out), lse);
    return cudaGetLastError();
}

cudaError_t launch_attend_prefix(const PrefixShape& p, const void* q, void* out, float* lse, float sm_scale,
                                 void* workspace, uint32_t* err, int clusters, cudaStream_t st, bool withhold = false)
{
    AttendPlan plan = attend_plan(p.n, p.B, p.heads, p.layers, clusters);
    plan.o = static_cast<float*>(workspace);
    plan.lse = plan.o + (int64_t)plan.rest * plan.splits * 2 * kTileRows * kVDim;
    CUtensorMap key_map, value_map, q_map;
    cudaError_t e = encode_rows(p, 32, &key_map);
    if (e == cudaSuccess) e = encode_rows(p, 64, &value_map);
    if (e == cudaSuccess) e = encode_queries(p, q, &q_map);
    if (e != cudaSuccess) return e;
    e = launch_chained(attend_prefix_kernel, dim3(4u * (unsigned)std::min(plan.pieces(), clusters)), kAThreads, kASmem, st, key_map, value_map,
                       q_map, p, plan, static_cast<uint16_t*>(out), lse, sm_scale * kLog2e, err, withhold ? 1 : 0);
    if (e != cudaSuccess || plan.rest == 0) return e;
    return launch_chained(plan.splits <= 8 ? combine_prefix_kernel<8> : combine_prefix_kernel<12>, dim3(kVHalf / 16, 4u * (unsigned)plan.rest),
                          512, 0, st, p, plan, static_cast<uint16_t*>(out), lse);
}

// ---------------------------------------------------------------------------
struct JoinParts {
    const uint4* out[kMaxParts];
    const float* lse[kMaxParts];
};

// A warp a row, 16 columns a lane.  All of a row is read before any of it is written, so the result may
// take a part's place.  Bound by HBM: 90 us at two parts of 192 x 8 units of 128 heads (606 MB, 6.7 TB/s, a copy's
// rate); at 21 units 2.4 us (among others 7.4), a launch and a row's latency.
template <int kParts>
__global__ void __launch_bounds__(256) join_kernel(JoinParts parts, int64_t rows, uint4* out, float* lse)
{
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    chain_next();
    chain_wait();
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        parts.out[i] = behind_wait(parts.out[i]);
        parts.lse[i] = behind_wait(parts.lse[i]);
    }
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
// Eviction.  Weights are compared as unsigned words of the same order; tokens
// that always stay have the largest word, which no weight has.  The threshold tv is
// the word of the last token that stays: what is above it stays, and of those equal to it the
// first `ties`.  With the threshold known a scan gives every token that stays its place, so
// nothing is sorted, and ties go to the lower token.
struct Heaviest {
    const float* weights;
    int64_t stride;           // floats between layers
    int n, keep, first, last;
    const uint32_t* err;      // the error word
    // of token j, whose weight is x
    __device__ __forceinline__ uint32_t word(float x, int j) const
    {
        const uint32_t u = __float_as_uint(x + 0.0f);  // -0 as +0
        const uint32_t v = x != x ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;  // a NaN below everything
        return j < first || j >= n - last ? 0xFFFFFFFFu : v;
    }
    // kEach weights, `step` tokens apart: all reads in flight together
    template <int kEach>
    __device__ __forceinline__ void read(const float* w, int j0, int step, float (&x)[kEach]) const
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) x[i] = j0 + i * step < n ? w[j0 + i * step] : 0.0f;
    }
};
constexpr uint32_t kNoWord = 0xFFFFFFFEu;  // above every weight, below the tokens that always stay

// Inclusive sum over a CTA of kWarps warps, in thread order; *all receives the total.  (a __syncthreads inside)
template <int kWarps>
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t* warp_sum, uint32_t* all)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    const uint32_t w = lane < kWarps ? warp_sum[lane] : 0u;
    *all = __reduce_add_sync(0xFFFFFFFFu, w);
    return v + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u);
}

// Everything stays (or, with the error word set, nothing is said to).
__global__ void __launch_bounds__(256) keep_all_kernel(Heaviest h, int32_t* kept)
{
    chain_next();
    chain_wait();
    const bool none = *behind_wait(h.err) != 0u;
    kept += (int64_t)blockIdx.y * h.keep;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < h.keep; i += (int64_t)gridDim.x * 256) kept[i] = !none && i < h.n ? (int32_t)i : -1;
}

// Short rows: a CTA a layer, its words in shared memory.  The range of the words is narrowed by histograms of 2048
// equal parts until the part that holds the threshold has few enough to be ranked directly; the first range is that of the
// words themselves, so mostly the first histogram is the only one.  Bound by latency: some ten barriers; 5 us at 4096 tokens,
// 10 at 8 x 16001.  Short is what shared memory holds; the passes for long rows, swept over 1 to 61 layers: 15 to 24 us
// where this takes 10 (16001 tokens), 16 to 27 where it takes 13 (24000), 17 to 29 where it takes 16 to 17 (32768).  With the rows moved as
// well that is within 6 % from 24000 tokens on, either way.
constexpr int kShort = 32768, kShortThreads = 1024, kBins = 2048, kFew = 256;
__global__ void __launch_bounds__(kShortThreads) heaviest_short_kernel(Heaviest h, int32_t* kept)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    uint32_t* words = reinterpret_cast<uint32_t*>(smem);
    __shared__ uint32_t hist[kBins], few[kFew], above[kShort / 32], equal[kShort / 32], warp_sum[32];
    __shared__ uint32_t s_lo, s_hi, s_bin, s_before, s_count, s_few, s_tv, s_ties;
    const int tid = threadIdx.x, lane = tid & 31, n = h.n;
    if (tid == 0) {
        s_lo = 0xFFFFFFFFu;
        s_hi = 0u;
    }
    chain_next();
    chain_wait();
    const float* w = behind_wait(h.weights) + blockIdx.x * h.stride;
    kept += (int64_t)blockIdx.x * h.keep;
    const bool stop = __syncthreads_or(tid == 0 && *behind_wait(h.err) != 0u);
    if (stop) {
        for (int i = tid; i < h.keep; i += kShortThreads) kept[i] = -1;
        return;
    }
    uint32_t lo = 0xFFFFFFFFu, hi = 0u;
    for (int j0 = tid; j0 < n; j0 += 8 * kShortThreads) {
        float x[8];
        h.read(w, j0, kShortThreads, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i * kShortThreads;
            const uint32_t v = h.word(x[i], j);
            if (j < n) words[j] = v;
            if (j < n && v != 0xFFFFFFFFu) {
                lo = min(lo, v);
                hi = max(hi, v);
            }
        }
    }
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) {
        atomicMin(&s_lo, lo);
        atomicMax(&s_hi, hi);
    }
    __syncthreads();
    lo = s_lo;
    hi = s_hi;
    uint32_t need = (uint32_t)(h.keep - h.first - h.last);  // to take from [lo, hi]; every word above hi stays
    uint32_t tv = kNoWord, ties = 0u;
    while (need > 0u) {
        if (lo == hi) {
            tv = lo;
            ties = need;
            break;
        }
        const uint32_t span = hi - lo;
        const int bits = 32 - __clz(span), shift = bits > 11 ? bits - 11 : 0;
        hist[tid] = hist[tid + kShortThreads] = 0u;
        if (tid == 0) s_few = 0u;
        __syncthreads();
#pragma unroll 4
        for (int j = tid; j < n; j += kShortThreads) {
            const uint32_t x = words[j] - lo;
            if (x <= span) atomicAdd(&hist[x >> shift], 1u);
        }
        __syncthreads();
        const int top = kBins - 1 - 2 * tid;
        const uint32_t h1 = hist[top], h0 = hist[top - 1];
        uint32_t all;
        const uint32_t before = cta_scan<32>(h1 + h0, warp_sum, &all) - h1 - h0;
        if (before < need && need <= before + h1 + h0) {
            const bool first = need <= before + h1;
            s_bin = first ? top : top - 1;
            s_before = first ? before : before + h1;
            s_count = first ? h1 : h0;
        }
        __syncthreads();
        lo += s_bin << shift;
        hi = min(hi - lo, (1u << shift) - 1u) + lo;
        need -= s_before;
        const uint32_t in = s_count;
        if (in == need) {  // all of it
            tv = lo;
            ties = 0xFFFFFFFFu;
            break;
        }
        if (in <= kFew) {
            const uint32_t range = hi - lo;
#pragma unroll 4
            for (int j = tid; j < n; j += kShortThreads)
                if (words[j] - lo <= range) few[atomicAdd(&s_few, 1u)] = words[j];
            __syncthreads();
            if (tid < in) {
                const uint32_t mine = few[tid];
                uint32_t more = 0, same = 0;
                for (uint32_t i = 0; i < in; ++i) {
                    more += few[i] > mine;
                    same += few[i] == mine;
                }
                if (more < need && need <= more + same) {  // (equal words write the same)
                    s_tv = mine;
                    s_ties = need - more;
                }
            }
            __syncthreads();
            tv = s_tv;
            ties = s_ties;
            break;
        }
    }
    // a bit a token, a word of bits a thread
    for (int j0 = tid - lane; j0 < n; j0 += kShortThreads) {
        const uint32_t v = j0 + lane < n ? words[j0 + lane] : 0u;
        const uint32_t a = __ballot_sync(0xFFFFFFFFu, j0 + lane < n && v > tv), e = __ballot_sync(0xFFFFFFFFu, j0 + lane < n && v == tv);
        if (lane == 0) {
            above[j0 / 32] = a;
            equal[j0 / 32] = e;
        }
    }
    __syncthreads();
    const uint32_t a = 32 * tid < n ? above[tid] : 0u, e = 32 * tid < n ? equal[tid] : 0u;
    uint32_t all;
    const uint32_t upto = cta_scan<32>(__popc(a) | (uint32_t)__popc(e) << 16, warp_sum, &all);  // (at most 2^15 each)
    // what a word keeps: all above, and of the equal ones the first that are left; the word's first place beside it
    const uint32_t ab = (upto & 0xFFFFu) - __popc(a), eb = (upto >> 16) - __popc(e);
    uint32_t stay = a | e;
    if (eb + __popc(e) > ties) {
        uint32_t some = 0u, left = e;
        for (uint32_t i = eb; i < ties; ++i) {
            some |= left & (0u - left);
            left &= left - 1u;
        }
        stay = a | some;
    }
    above[tid] = stay;
    equal[tid] = ab + min(eb, ties);
    __syncthreads();
    for (int i = tid >> 5; 32 * i < n; i += kShortThreads / 32) {  // a word a warp, so that the writes are together
        const uint32_t m = above[i];
        if (m >> lane & 1u) kept[equal[i] + __popc(m & ((1u << lane) - 1u))] = 32 * i + lane;
    }
}

// Long rows: chunks of 4096 tokens, a CTA each, over the whole GPU.  Three passes find the threshold's digits (11, 11 and
// 10 bits, from the top) by histograms of the words that share the digits found so far; the last CTA of a layer to finish a pass
// picks the digit.  A fourth pass counts, a fifth writes.  Each pass reads the weights once, from L2 after the first: 29 us in all at
// 2 x 1M tokens (chunks of 8192 32, of 2048 38; one team of CTAs a layer 96).
constexpr int kChunk = 4096, kLongThreads = 512, kEachLong = kChunk / kLongThreads;
struct LongState {  // of a layer; zeros before the first pass
    uint32_t hist[3][kBins];
    uint32_t done[3];
    uint32_t digits;  // found so far; at last tv
    uint32_t need;    // to take from the words that share them; at last ties
    uint32_t err;     // the error word as the first pass saw it
    uint32_t pad[2];
};
static_assert(sizeof(LongState) % 16 == 0, "a layer's state");

template <int kPass>
__global__ void __launch_bounds__(kLongThreads) digit_kernel(Heaviest h, LongState* states)
{
    constexpr int kDigitBits = kPass < 2 ? 11 : 10, kShift = kPass == 0 ? 21 : kPass == 1 ? 10 : 0, kDigits = 1 << kDigitBits;
    __shared__ uint32_t hist[kBins], warp_sum[32], s_last, s_digit, s_before;
    const int tid = threadIdx.x;
    for (int i = tid; i < kBins; i += kLongThreads) hist[i] = 0u;
    chain_next();
    chain_wait();
    LongState& st = behind_wait(states)[blockIdx.y];
    const float* w = behind_wait(h.weights) + blockIdx.y * h.stride;
    const uint32_t digits = kPass ? __ldcg(&st.digits) : 0u;
    __syncthreads();
    float x[kChunk / kLongThreads];
    const int j0 = blockIdx.x * kChunk + tid;
    h.read(w, j0, kLongThreads, x);
#pragma unroll
    for (int i = 0; i < kChunk / kLongThreads; ++i) {
        const int j = j0 + i * kLongThreads;
        if (j < h.n) {
            const uint32_t v = h.word(x[i], j);
            if (v != 0xFFFFFFFFu && (kPass == 0 || v >> ((kShift + kDigitBits) & 31) == digits)) atomicAdd(&hist[(v >> kShift) & (kDigits - 1)], 1u);
        }
    }
    __syncthreads();
    for (int i = tid; i < kDigits; i += kLongThreads)
        if (hist[i]) atomicAdd(&st.hist[kPass][i], hist[i]);
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&st.done[kPass], 1u) == gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last CTA of the layer: kDigits / kLongThreads digits a thread, from the top
    constexpr int kEach = kDigits / kLongThreads;
    const uint32_t need = kPass ? __ldcg(&st.need) : (uint32_t)(h.keep - h.first - h.last);
    uint32_t c[kEach], sum = 0, all;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        c[i] = __ldcg(&st.hist[kPass][kDigits - 1 - kEach * tid - i]);
        sum += c[i];
    }
    uint32_t before = cta_scan<kLongThreads / 32>(sum, warp_sum, &all) - sum;
    if (tid == 0) {  // none needed: the word above all weights
        s_digit = (kNoWord >> kShift) & (kDigits - 1);
        s_before = 0u;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (before < need && need <= before + c[i]) {
            s_digit = kDigits - 1 - kEach * tid - i;
            s_before = before;
        }
        before += c[i];
    }
    __syncthreads();
    if (tid == 0) {
        st.digits = digits << kDigitBits | s_digit;
        st.need = need - s_before;
        if (kPass == 0) st.err = *behind_wait(h.err);
    }
}

__device__ __forceinline__ void chunk_bits(const Heaviest& h, const float* w, uint32_t tv, uint32_t (&a)[kEachLong], uint32_t (&e)[kEachLong], uint32_t& na, uint32_t& ne)
{
    // a warp has consecutive tokens of the chunk
    const int lane = threadIdx.x & 31, j0 = blockIdx.x * kChunk + (threadIdx.x >> 5) * (kChunk / (kLongThreads / 32)) + lane;
    float x[kEachLong];
    h.read(w, j0, 32, x);
    na = ne = 0u;
#pragma unroll
    for (int i = 0; i < kEachLong; ++i) {
        const uint32_t v = h.word(x[i], j0 + 32 * i);
        a[i] = __ballot_sync(0xFFFFFFFFu, j0 + 32 * i < h.n && v > tv);
        e[i] = __ballot_sync(0xFFFFFFFFu, j0 + 32 * i < h.n && v == tv);
        na += __popc(a[i]);
        ne += __popc(e[i]);
    }
}

__global__ void __launch_bounds__(kLongThreads) count_kernel(Heaviest h, const LongState* states, uint2* counts)
{
    __shared__ uint32_t sa, se;
    if (threadIdx.x == 0) sa = se = 0u;
    chain_next();
    chain_wait();
    const LongState& st = behind_wait(states)[blockIdx.y];
    uint32_t a[kEachLong], e[kEachLong], na, ne;
    chunk_bits(h, behind_wait(h.weights) + blockIdx.y * h.stride, st.digits, a, e, na, ne);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        atomicAdd(&sa, na);
        atomicAdd(&se, ne);
    }
    __syncthreads();
    if (threadIdx.x == 0) counts[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = make_uint2(sa, se);
}

__global__ void __launch_bounds__(kLongThreads) place_kernel(Heaviest h, const LongState* states, const uint2* counts, int32_t* kept)
{
    __shared__ uint32_t wa[kLongThreads / 32], we[kLongThreads / 32], sa, se;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) sa = se = 0u;
    chain_next();
    chain_wait();
    const LongState& st = behind_wait(states)[blockIdx.y];
    counts = behind_wait(counts) + (int64_t)blockIdx.y * gridDim.x;
    kept += (int64_t)blockIdx.y * h.keep;
    const uint32_t tv = st.digits, ties = st.need;
    if (st.err) {
        for (int64_t i = (int64_t)blockIdx.x * kLongThreads + tid; i < h.keep; i += (int64_t)gridDim.x * kLongThreads) kept[i] = -1;
        return;
    }
    uint32_t a[kEachLong], e[kEachLong], na, ne, ca = 0, ce = 0;
    chunk_bits(h, behind_wait(h.weights) + blockIdx.y * h.stride, tv, a, e, na, ne);
    if (lane == 0) {
        wa[warp] = na;
        we[warp] = ne;
    }
    for (int i = tid; i < (int)blockIdx.x; i += kLongThreads) {  // the chunks before this one
        const uint2 c = counts[i];
        ca += c.x;
        ce += c.y;
    }
    ca = __reduce_add_sync(0xFFFFFFFFu, ca);
    ce = __reduce_add_sync(0xFFFFFFFFu, ce);
    __syncthreads();
    if (lane == 0 && (ca | ce)) {
        atomicAdd(&sa, ca);
        atomicAdd(&se, ce);
    }
    __syncthreads();
    uint32_t ab = sa, eb = se;  // before this warp's tokens
    for (int i = 0; i < warp; ++i) {
        ab += wa[i];
        eb += we[i];
    }
    const uint32_t below = (1u << lane) - 1u;
    const int j0 = blockIdx.x * kChunk + warp * (kChunk / (kLongThreads / 32)) + lane;
#pragma unroll
    for (int i = 0; i < kEachLong; ++i) {
        const uint32_t er = eb + __popc(e[i] & below), ar = ab + __popc(a[i] & below);
        if (a[i] >> lane & 1u || (e[i] >> lane & 1u && er < ties)) kept[ar + min(er, ties)] = j0 + 32 * i;
        ab += __popc(a[i]);
        eb += __popc(e[i]);
    }
}

// The tokens that stay (kept, ascending, -1 behind the last): their rows and weights moved together.  A warp
// moves four rows, nine 16-byte pieces a lane.  Bound by HBM: 181 us at 2 x 262144 rows (1.21 GB, 6.7 TB/s, a copy's rate; 192 with
// a CTA for every 32 rows, 224 with streaming stores or loads that pass L1 by, 200 in pieces of 32 bytes).
constexpr int kKeepCtas = 24;  // CTAs a layer for every SM, at most
__global__ void __launch_bounds__(256) keep_kernel(PrefixShape p, const float* weights, int64_t weights_stride, int keep,
                                                   const int32_t* kept, uint4* rows_out, float* weights_out)
{
    constexpr int kPieces = kRowBytes / 16, kRowsAWarp = 4, kEach = kPieces * kRowsAWarp / 32;
    chain_next();
    chain_wait();
    const int l = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8 * kRowsAWarp;
    kept = behind_wait(kept) + (int64_t)l * keep;
    weights = behind_wait(weights);
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

// Workspace of an eviction: the layers' states and the chunks' counts (long rows only).
int64_t evict_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }
int64_t evict_bytes(int64_t n, int layers) { return n <= kShort ? 16 : layers * ((int64_t)sizeof(LongState) + evict_chunks(n) * (int64_t)sizeof(uint2)); }

cudaError_t launch_evict(const PrefixShape& p, const float* weights, int64_t weights_stride, int keep, int first, int last,
                         int32_t* kept, void* rows_out, float* weights_out, void* workspace, const uint32_t* err, int device_sms, cudaStream_t st)
{
    const Heaviest h{p.n ? weights + p.layer0 * weights_stride : nullptr, weights_stride, p.n, keep, first, last, err};
    const unsigned layers = (unsigned)p.layers;
    cudaError_t e = cudaSuccess;
    if (p.n <= keep) {
        e = launch_chained(keep_all_kernel, dim3((unsigned)std::min(1 << 16, (keep + 255) / 256), layers), 256, 0, st, h, kept);
    } else if (p.n <= kShort) {
        e = launch_chained(heaviest_short_kernel, dim3(layers), kShortThreads, (size_t)(p.n + 31) / 32 * 128, st, h, kept);
    } else {
        LongState* states = static_cast<LongState*>(workspace);
        uint2* counts = reinterpret_cast<uint2*>(states + layers);
        const dim3 grid((unsigned)evict_chunks(p.n), layers);
        e = cudaMemsetAsync(states, 0, layers * sizeof(LongState), st);
        if (e == cudaSuccess) e = launch_chained(digit_kernel<0>, grid, kLongThreads, 0, st, h, states);
        if (e == cudaSuccess) e = launch_chained(digit_kernel<1>, grid, kLongThreads, 0, st, h, states);
        if (e == cudaSuccess) e = launch_chained(digit_kernel<2>, grid, kLongThreads, 0, st, h, states);
        if (e == cudaSuccess) e = launch_chained(count_kernel, grid, kLongThreads, 0, st, h, static_cast<const LongState*>(states), counts);
        if (e == cudaSuccess)
            e = launch_chained(place_kernel, grid, kLongThreads, 0, st, h, static_cast<const LongState*>(states), static_cast<const uint2*>(counts), kept);
    }
    if (e != cudaSuccess || (!rows_out && !weights_out) || p.n == 0) return e;
    return launch_chained(keep_kernel, dim3((unsigned)std::min<int64_t>(((int64_t)keep + 31) / 32, kKeepCtas * device_sms), layers), 256, 0, st, p, weights,
                          weights_stride, keep, static_cast<const int32_t*>(kept), static_cast<uint4*>(rows_out), weights_out);
}

int64_t align16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

}  // namespace

cudaError_t prepare_prefix(int* clusters)
{
    cudaError_t e = cudaFuncSetAttribute(attend_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kASmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(weigh_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kWSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(heaviest_short_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShort * 4);
    if (e != cudaSuccess) return e;
    // clusters of four that are on the chip at once (its processors come in groups that are no multiple of four)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(4);
    cfg.blockDim = dim3(kAThreads);
    cfg.dynamicSmemBytes = kASmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(clusters, attend_prefix_kernel, &cfg);
    if (*clusters < 1) *clusters = 1;
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
    cudaError_t e = prev != ctx->cfg.device ? cudaSetDevice(ctx->cfg.device) : cudaSuccess;
    if (e == cudaSuccess) e = f();
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
// Clusters of skv_attend_prefix within skv_set_attend_sms's budget.
int attend_clusters(const skv_ctx* ctx)
{
    return ctx->attend_sms > 0 ? std::max(1, std::min(ctx->prefix_clusters, ctx->attend_sms / 4)) : ctx->prefix_clusters;
}
int call_layers(const skv_ctx* ctx, int32_t layer) { return layer < 0 ? ctx->cfg.num_layers : 1; }
PrefixShape shape_of(const skv_ctx* ctx, const skv_prefix& x, int32_t B, int32_t heads, int32_t layer)
{
    const int layers = call_layers(ctx, layer);
    return PrefixShape{static_cast<const uint8_t*>(x.rows), x.layer_stride, x.row_stride, (int)x.n, B, heads,
                       layers, layer < 0 ? 0 : layer, layers, 0, 1};
}
int64_t attend_workspace(const skv_ctx* ctx, const skv_prefix& x, int32_t B, int32_t heads, int32_t layer)
{
    if (B == 0 || x.n == 0) return 16;
    const int layers = skv::launch_layers(shape_of(ctx, x, B, heads, layer));
    return std::max<int64_t>(16, skv::attend_bytes(skv::attend_plan(x.n, B, heads, layers, attend_clusters(ctx))));
}
int64_t weigh_workspace(const skv_ctx* ctx, const skv_prefix& x, int32_t B, int32_t heads, int32_t layer)
{
    if (B == 0 || x.n == 0) return 16;
    const int layers = skv::launch_layers(shape_of(ctx, x, B, heads, layer)), shares = skv::weigh_plan(x.n, B, heads, layers, ctx->device_sms).shares;
    return shares > 1 ? skv::align16((int64_t)shares * layers * x.n * 4) : 16;
}

skv_status attend_impl(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                       const void* q_dev, void* out_dev, float* lse_dev, float sm_scale, void* workspace_dev,
                       int64_t workspace_bytes, skv_stream_t stream, bool withhold)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale))
        return SKV_ERR_INVALID_ARG;
    if (B == 0) return SKV_OK;
    if (!rows_ok(ctx, *prefix) || !q_dev || !out_dev || !workspace_dev || workspace_bytes < attend_workspace(ctx, *prefix, B, heads, layer) || !aligned(q_dev, 16) ||
        !aligned(out_dev, 16) || !aligned(lse_dev, 4) || !aligned(workspace_dev, 16))
        return SKV_ERR_INVALID_ARG;
    const PrefixShape p = shape_of(ctx, *prefix, B, heads, layer);
    return on_device(ctx, "skv_attend_prefix", [&] {
        if (p.n == 0) return skv::launch_attend_nothing(p, out_dev, lse_dev, stream);
        return skv::for_each_launch(p, [&](const PrefixShape& part, int64_t units) {
            const int64_t row = units * heads;
            return skv::launch_attend_prefix(part, static_cast<const uint8_t*>(q_dev) + row * skv::kRowBytes,
                                             static_cast<uint16_t*>(out_dev) + row * skv::kVDim, lse_dev ? lse_dev + row : nullptr, sm_scale,
                                             workspace_dev, &ctx->d.ctl[skv::CTL_ERR], attend_clusters(ctx), stream, withhold);
        });
    });
}

// A layer's new weights may take its old ones' place, and lie on nothing else that the call reads.
bool in_place_ok(const float* weights, int64_t weights_stride, const float* out, int64_t out_stride, int64_t n, int64_t layer0, int64_t layers)
{
    if (!weights || (weights == out && weights_stride == out_stride)) return true;
    const int64_t last = layer0 + layers - 1, bytes = 4 * n;
    auto read = [&](int64_t l) { return (int64_t)(reinterpret_cast<uintptr_t>(weights) + (uint64_t)(4 * l * weights_stride)); };
    auto written = [&](int64_t l) { return (int64_t)(reinterpret_cast<uintptr_t>(out) + (uint64_t)(4 * l * out_stride)); };
    if (read(last) + bytes <= written(layer0) || written(last) + bytes <= read(layer0)) return true;
    for (int64_t l = layer0; l <= last; ++l)
        for (int64_t o = layer0; o <= last; ++o)
            if (read(l) < written(o) + bytes && written(o) < read(l) + bytes && !(l == o && read(l) == written(o))) return false;
    return true;
}

skv_status weigh_impl(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                      const void* q_dev, const float* lse_dev, const float* weights_dev, int64_t weights_stride,
                      float* out_dev, int64_t out_stride, float sm_scale, float gain, void* workspace_dev,
                      int64_t workspace_bytes, skv_stream_t stream, bool withhold)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !(sm_scale > 0.0f) || !std::isfinite(sm_scale) ||
        !std::isfinite(gain))
        return SKV_ERR_INVALID_ARG;
    if (prefix->n == 0) return SKV_OK;
    const bool many = ctx->cfg.num_layers > 1;
    if (!rows_ok(ctx, *prefix) || !out_dev || !aligned(weights_dev, 4) || !aligned(out_dev, 4) ||
        (many && (out_stride < prefix->n || (weights_dev && weights_stride < prefix->n))) || out_stride >= (int64_t)1 << 40 ||
        weights_stride >= (int64_t)1 << 40)
        return SKV_ERR_INVALID_ARG;
    if (!in_place_ok(weights_dev, weights_stride, out_dev, out_stride, prefix->n, layer < 0 ? 0 : layer, call_layers(ctx, layer)))
        return SKV_ERR_INVALID_ARG;
    if (B > 0 && (!q_dev || !lse_dev || !workspace_dev || workspace_bytes < weigh_workspace(ctx, *prefix, B, heads, layer) ||
                  !aligned(q_dev, 16) || !aligned(workspace_dev, 16) || !aligned(lse_dev, 4)))
        return SKV_ERR_INVALID_ARG;
    const PrefixShape p = shape_of(ctx, *prefix, B, heads, layer);
    return on_device(ctx, "skv_weigh_prefix", [&] {
        if (B == 0) return skv::launch_weigh_nothing(p, weights_dev, weights_stride, out_dev, out_stride, stream);
        return skv::for_each_launch(p, [&](const PrefixShape& part, int64_t units) {
            const int64_t row = units * heads;
            return skv::launch_weigh(part, static_cast<const uint8_t*>(q_dev) + row * skv::kRowBytes, lse_dev + row, weights_dev,
                                     weights_stride, out_dev, out_stride, sm_scale, gain, static_cast<float*>(workspace_dev),
                                     &ctx->d.ctl[skv::CTL_ERR], ctx->device_sms, stream, withhold);
        });
    });
}
}  // namespace

extern "C" {

skv_status skv_attend_prefix_workspace(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                                       int64_t* bytes)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !bytes) return SKV_ERR_INVALID_ARG;
    *bytes = attend_workspace(ctx, *prefix, B, heads, layer);
    return SKV_OK;
}

skv_status skv_attend_prefix(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                             const void* q_dev, void* out_dev, float* lse_dev, float sm_scale, void* workspace_dev,
                             int64_t workspace_bytes, skv_stream_t stream)
{
    return attend_impl(ctx, prefix, B, heads, layer, q_dev, out_dev, lse_dev, sm_scale, workspace_dev, workspace_bytes, stream, false);
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
        return skv::launch_chained(kernels[parts - 1], dim3(grid), 256, 0, stream, jp, rows, static_cast<uint4*>(out_dev), lse_dev);
    });
}

skv_status skv_weigh_prefix_workspace(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                                      int64_t* bytes)
{
    if (!shape_ok(ctx, prefix, layer) || !batch_ok(ctx, B, heads) || !bytes) return SKV_ERR_INVALID_ARG;
    *bytes = weigh_workspace(ctx, *prefix, B, heads, layer);
    return SKV_OK;
}

skv_status skv_weigh_prefix(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, int32_t layer,
                            const void* q_dev, const float* lse_dev, const float* weights_dev, int64_t weights_stride,
                            float* out_dev, int64_t out_stride, float sm_scale, float gain, void* workspace_dev,
                            int64_t workspace_bytes, skv_stream_t stream)
{
    return weigh_impl(ctx, prefix, B, heads, layer, q_dev, lse_dev, weights_dev, weights_stride, out_dev, out_stride, sm_scale, gain,
                      workspace_dev, workspace_bytes, stream, false);
}

skv_status skv_selftest_prefix_timeout(skv_ctx* ctx, const skv_prefix* prefix, int32_t B, int32_t heads, const void* q_dev,
                                       const float* lse_dev, void* out_dev, float* weights_dev, int64_t weights_stride,
                                       void* workspace_dev, int64_t workspace_bytes, skv_stream_t stream)
{
    if (out_dev) return attend_impl(ctx, prefix, B, heads, -1, q_dev, out_dev, nullptr, 1.0f, workspace_dev, workspace_bytes, stream, true);
    return weigh_impl(ctx, prefix, B, heads, -1, q_dev, lse_dev, nullptr, 0, weights_dev, weights_stride, 1.0f, 1.0f, workspace_dev,
                      workspace_bytes, stream, true);
}

skv_status skv_evict_prefix_workspace(skv_ctx* ctx, const skv_prefix* prefix, int32_t layer, int64_t* bytes)
{
    if (!shape_ok(ctx, prefix, layer) || !bytes) return SKV_ERR_INVALID_ARG;
    *bytes = skv::evict_bytes(prefix->n, call_layers(ctx, layer));
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
        workspace_bytes < skv::evict_bytes(prefix->n, call_layers(ctx, layer)) || !aligned(workspace_dev, 16) || !aligned(rows_out_dev, 16) ||
        !aligned(kept_dev, 4) || !aligned(weights_dev, 4) || !aligned(weights_out_dev, 4) ||
        (ctx->cfg.num_layers > 1 && weights_stride < prefix->n) || weights_stride >= (int64_t)1 << 40)
        return SKV_ERR_INVALID_ARG;
    const PrefixShape p = shape_of(ctx, *prefix, 1, 1, layer);
    return on_device(ctx, "skv_evict_prefix", [&] {
        return skv::launch_evict(p, weights_dev, weights_stride, keep, first, last, kept_dev, rows_out_dev, weights_out_dev, workspace_dev,
                                 &ctx->d.ctl[skv::CTL_ERR], ctx->device_sms, stream);
    });
}

}  // extern "C"
