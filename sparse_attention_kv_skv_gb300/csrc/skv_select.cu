// The producer of the Top-k: a cheap score of every index key for the step's
// query, and the selection of the k best tokens ("SGLang и Tair представили
// иерархичную Sparse Attention ...", paragraph 2: DSA selects first and
// computes attention over the selection; "XM-Sparse: Netpreme X-Mem ...", section
// "为何稀疏注意力需要快速高容量内存层": the indexer's keys stay in HBM).
//
// For unit (b, l), index query heads q_h and weights w_h, and key j of the
// request, which stands for the tokens [j * block, (j + 1) * block):
//   score_j = sum_h w_h * max(0, q_h . k_j)         (without the max if relu is 0)
// The blocks with the k / block largest scores are taken, the lowest index first
// among equals, and their tokens written in ascending order.
//
// Two kernels.  score_kernel reads every key once and is bound by that: 2 * dim
// bytes a key at HBM rate.  pick_kernel finds each unit's threshold among its
// scores and writes the tokens.

#include <cuda.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "skv_ctx.cuh"
#include "tcgen05.cuh"

namespace skv {
namespace {

constexpr uint32_t kMaxSleepPolls = 1u << 20;  // bound of a wait whose polls may each sleep (about 2 s)
constexpr int kTileKeys = 128;                 // keys of a tile: the M of the product, one tensor-memory lane each
constexpr int kMaxHeads = 64;                  // its N
constexpr int kGroups = 2;                     // warpgroups that take scores out of tensor memory, a tile each in turn
constexpr int kLoadWarp = 4 * kGroups, kMmaWarp = kLoadWarp + 1;
constexpr int kScoreThreads = 32 * (kMmaWarp + 1);
constexpr int kDepth = 4;                      // products in tensor memory (64 columns each)
constexpr uint32_t kTmemCols = kDepth * kMaxHeads;
constexpr uint32_t kScoreSmem = 227 * 1024;    // dynamic shared memory of score_kernel, at most

// What both kernels need to know of a call.
struct SelectShape {
    int B, layers;         // units b * layers + l (layers: L, or 1 for a call on one layer)
    int heads, npad;       // npad: heads rounded up to the MMA's multiple of 16
    int block, first, last;
    int64_t stride;        // scores a unit has room for
};

__device__ __forceinline__ int keys_of(const Dev& d, int32_t r, int block)
{
    return (int)((d.len[r] + block - 1) / block);
}

struct alignas(16) ScoreCtl {
    uint64_t full[8], empty[8];            // key stages
    uint64_t q_full[2], q_empty[2];        // query buffers
    uint64_t d_full[kDepth], d_empty[kDepth];  // products
    float w[kGroups][kMaxHeads];           // a warpgroup's copy of its unit's weights
    long long sums[kScoreThreads / 32];
    int start[3];                          // first batch entry, layer and tile of this CTA
    uint32_t tmem_base, abort;
};

struct ScoreLayout {
    int stages;
    uint32_t off_q, off_ctl, bytes;
};
__host__ __device__ inline ScoreLayout score_layout(int dim, int npad)
{
    ScoreLayout a;
    const uint32_t stage = kTileKeys * dim * 2, q = 2u * npad * dim * 2;
    a.stages = (int)((kScoreSmem - q - sizeof(ScoreCtl)) / stage);
    if (a.stages > 8) a.stages = 8;
    a.off_q = a.stages * stage;
    a.off_ctl = a.off_q + q;
    a.bytes = a.off_ctl + (uint32_t)sizeof(ScoreCtl);
    return a;
}

__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort)
{
    const uint32_t a = tc::smem_u32(bar);
    for (uint32_t i = 0; i < kMaxSleepPolls; ++i) {
        if (tc::mbar_test(a, parity)) return true;
        if ((i & 7u) == 7u && *abort) return false;
    }
    return false;
}

__device__ __forceinline__ void give_up(ScoreCtl& c, uint32_t* err)
{
    if (!c.abort) {
        c.abort = 1u;
        atomicOr(err, DEVERR_TIMEOUT);
    }
}

// A CTA's walk over its tiles, in the order (batch entry, layer, tile).  Every
// role makes the same walk.  The entries of a call were checked before.
struct Walk {
    const Dev& d;
    const SelectShape& sh;
    const int32_t* req_ids;
    int b, l, tile, keys = 0, tiles = 0;
    int32_t r = 0;
    bool fresh = true;  // first tile of a unit (in this walk)
    __device__ Walk(const Dev& d_, const SelectShape& sh_, const int32_t* ids, const int* start)
        : d(d_), sh(sh_), req_ids(ids), b(start[0]), l(start[1]), tile(start[2])
    {
        enter();
    }
    __device__ void enter()
    {
        r = req_ids[b];
        keys = keys_of(d, r, sh.block);
        tiles = (keys + kTileKeys - 1) / kTileKeys;
    }
    __device__ int unit() const { return b * sh.layers + l; }
    __device__ bool last_of_unit() const { return tile + 1 == tiles; }
    // only called while tiles are left
    __device__ void next()
    {
        fresh = false;
        if (++tile < tiles) return;
        tile = 0;
        fresh = true;
        if (++l < sh.layers) return;
        l = 0;
        do {
            ++b;
            enter();
        } while (tiles == 0);
    }
};

// Scores as unsigned words of the same order: a NaN below everything, -0 as +0.
__device__ __forceinline__ uint32_t order_word(float s)
{
    const uint32_t u = __float_as_uint(s + 0.0f);
    return s != s ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A persistent grid, one CTA a SM; the call's tiles of 128 keys are dealt out
// evenly and in order, so a CTA stays on a unit as long as it can.  One thread
// loads key tiles (TMA, 128-byte swizzle) into a ring of stages and, when a unit
// begins, its query; one thread issues the products (keys x heads: the keys are
// the rows, so each thread of the epilogue owns a key and sums its heads without
// any exchange); two warpgroups in turn take a product out of tensor memory,
// weigh and sum it, and write one word a key.
// What bounds it: the keys' bytes.  128 keys of 128 dims are 32 KB, 0.73 us of
// this SM's share of HBM; the product takes 128 x 64 x 128 multiply-adds, a fifth of
// that, and the epilogue 64 max and fma a key.  So tiles need no reuse, only
// enough stages in flight (5 to 6 of 32 KB).
template <int kDim, bool kRelu>
__global__ void __launch_bounds__(kScoreThreads, 1)
    score_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap q_map, Dev d,
                 const int32_t* __restrict__ req_ids, const float* __restrict__ w, SelectShape sh, ScoreLayout lay,
                 uint32_t* __restrict__ scores)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    ScoreCtl& c = *reinterpret_cast<ScoreCtl*>(smem + lay.off_ctl);
    constexpr int kBoxes = kDim / 64;  // 64-dim columns of a key tile, 128 bytes wide
    constexpr uint32_t kBoxBytes = kTileKeys * 128, kStageBytes = kBoxes * kBoxBytes;
    const uint32_t q_box = sh.npad * 128u, q_bytes = kBoxes * q_box;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // pick_kernel, which waits for this kernel's end
    // the call's entries: every id an active request; how many tiles each has
    const int per = (sh.B + kScoreThreads - 1) / kScoreThreads;
    const int b0 = min(sh.B, tid * per), b1 = min(sh.B, b0 + per);
    bool bad = false, stop = tid == 0 && d.ctl[CTL_ERR] != 0u;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int32_t r = req_ids[b];
        if (r < 0 || r >= d.R || !d.active[r])
            bad = true;
        else
            mine += (keys_of(d, r, sh.block) + kTileKeys - 1) / kTileKeys;
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) c.sums[warp] = upto;
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && tid == 0) atomicOr(&d.ctl[CTL_ERR], DEVERR_BAD_REQUEST);
    if (__syncthreads_or(stop || bad)) return;  // pick_kernel sees the error word
    long long before = upto - mine, total = 0;
    for (int i = 0; i < kScoreThreads / 32; ++i) {
        if (i < warp) before += c.sums[i];
        total += c.sums[i];
    }
    const long long begin = total * sh.layers * blockIdx.x / gridDim.x;
    const int count = (int)(total * sh.layers * (blockIdx.x + 1) / gridDim.x - begin);
    if (count == 0) return;
    if (begin >= before * sh.layers && begin < (before + mine) * sh.layers) {  // this thread's entries hold it
        long long at = before * sh.layers;
        for (int b = b0; b < b1; ++b) {
            const long long t = (keys_of(d, req_ids[b], sh.block) + kTileKeys - 1) / kTileKeys;
            if (begin < at + t * sh.layers) {
                c.start[0] = b;
                c.start[1] = (int)((begin - at) / t);
                c.start[2] = (int)((begin - at) % t);
                break;
            }
            at += t * sh.layers;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < 8; ++s) {
            tc::mbar_init(&c.full[s], 1);
            tc::mbar_init(&c.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&c.q_full[i], 1);
            tc::mbar_init(&c.q_empty[i], 1);
        }
        for (int i = 0; i < kDepth; ++i) {
            tc::mbar_init(&c.d_full[i], 1);
            tc::mbar_init(&c.d_empty[i], 128);
        }
        c.abort = 0u;
    }
    // query rows behind the last head are zeros for good (a copy writes `heads` rows)
    for (uint32_t i = tid; i < 2 * q_bytes / 16; i += kScoreThreads)
        reinterpret_cast<uint4*>(smem + lay.off_q)[i] = make_uint4(0, 0, 0, 0);
    if (warp == kMmaWarp) tc::tmem_alloc(&c.tmem_base, kTmemCols);
    tc::fence_smem_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = c.tmem_base;
    const volatile uint32_t* abort = &c.abort;
    const int nst = lay.stages;

    if (warp == kLoadWarp) {
        if (lane == 0) {
            Walk k(d, sh, req_ids, c.start);
            bool ok = true;
            int units = 0, it = 0;
            for (; it < count; ++it) {
                if (k.fresh) {  // the unit's query, into the buffer the unit before the last one had
                    const int qb = units & 1;
                    if (units >= 2 && !(ok = wait_phase(&c.q_empty[qb], ((units >> 1) - 1) & 1, abort))) break;
                    tc::mbar_arrive_expect_tx(&c.q_full[qb], (uint32_t)sh.heads * kDim * 2);
#pragma unroll
                    for (int x = 0; x < kBoxes; ++x)
                        tc::tma_load3(tc::smem_u32(smem + lay.off_q) + qb * q_bytes + x * q_box, &q_map, 64 * x, 0, k.unit(),
                                      &c.q_full[qb]);
                    ++units;
                }
                const int s = it % nst;
                if (it >= nst && !(ok = wait_phase(&c.empty[s], ((it / nst) - 1) & 1, abort))) break;
                tc::mbar_arrive_expect_tx(&c.full[s], kStageBytes);
#pragma unroll
                for (int x = 0; x < kBoxes; ++x)
                    tc::tma_load4(tc::smem_u32(smem) + s * kStageBytes + x * kBoxBytes, &key_map, 64 * x, k.tile * kTileKeys,
                                  d.layer_sel >= 0 ? d.layer_sel : k.l, k.r, &c.full[s]);
                if (it + 1 < count) k.next();
            }
            if (!ok) {
                give_up(c, &d.ctl[CTL_ERR]);
                // no copy may still be landing when the CTA leaves
                for (int i = max(0, it - nst); i < it; ++i) tc::mbar_wait(&c.full[i % nst], (uint32_t)(i / nst) & 1u, 1u << 22);
                for (int i = max(0, units - 2); i < units; ++i) tc::mbar_wait(&c.q_full[i & 1], (uint32_t)(i >> 1) & 1u, 1u << 22);
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            Walk k(d, sh, req_ids, c.start);
            const uint32_t idesc = tc::idesc_bf16_f32(kTileKeys, sh.npad, 0);
            bool ok = true;
            int units = 0;
            for (int it = 0; it < count; ++it) {
                if (k.fresh) {
                    if (!(ok = wait_phase(&c.q_full[units & 1], (units >> 1) & 1, abort))) break;
                    ++units;
                }
                const int s = it % nst, p = it % kDepth, qb = (units - 1) & 1;
                if (it >= kDepth && !(ok = wait_phase(&c.d_empty[p], ((it / kDepth) - 1) & 1, abort))) break;
                if (!(ok = wait_phase(&c.full[s], (it / nst) & 1, abort))) break;
                tc::fence_after_sync();
                const uint32_t ka = tc::smem_u32(smem) + s * kStageBytes, qa = tc::smem_u32(smem + lay.off_q) + qb * q_bytes;
#pragma unroll
                for (int st = 0; st < kDim / 16; ++st)
                    tc::mma_bf16(tbase + p * kMaxHeads, tc::sw128_kmajor_desc(ka + (st >> 2) * kBoxBytes + (st & 3) * 32),
                                 tc::sw128_kmajor_desc(qa + (st >> 2) * q_box + (st & 3) * 32), idesc, st > 0 ? 1u : 0u);
                tc::mma_commit(&c.empty[s]);
                tc::mma_commit(&c.d_full[p]);
                if (k.last_of_unit()) tc::mma_commit(&c.q_empty[qb]);
                if (it + 1 < count) k.next();
            }
            if (!ok) give_up(c, &d.ctl[CTL_ERR]);
        }
    } else {
        const int grp = warp >> 2, t = tid & 127;
        const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
        Walk k(d, sh, req_ids, c.start);
        int weights_of = -1;  // the unit whose weights c.w[grp] holds
        bool ok = true;
        for (int it = 0; it < count; ++it) {
            if (it % kGroups == grp) {
                if (weights_of != k.unit()) {
                    weights_of = k.unit();
                    tc::named_sync(1 + grp, 128);  // the previous unit's are no longer read
                    if (t < kMaxHeads) c.w[grp][t] = t < sh.heads ? w[(size_t)weights_of * sh.heads + t] : 0.0f;
                    tc::named_sync(1 + grp, 128);
                }
                const int p = it % kDepth;
                // a give-up must not leave the other threads of the group at a barrier
                ok = ok && wait_phase(&c.d_full[p], (it / kDepth) & 1, abort);
                float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (__all_sync(0xFFFFFFFFu, ok)) {
                    tc::fence_after_sync();
                    const float4* ws = reinterpret_cast<const float4*>(c.w[grp]);
#pragma unroll
                    for (int c0 = 0; c0 < kMaxHeads; c0 += 32) {
                        if (c0 < sh.npad) {
                            float v[32];
                            tc::tmem_ld32(tl + p * kMaxHeads + c0, v);
                            if (c0 + 32 >= sh.npad) {  // all of it is in registers: the next product may come
                                tc::fence_before_sync();
                                tc::mbar_arrive(&c.d_empty[p]);
                            }
#pragma unroll
                            for (int x = 0; x < 32; x += 4) {
                                if (c0 + (x & ~15) < sh.npad) {  // columns behind npad hold no product
                                    const float4 f = ws[(c0 + x) / 4];
                                    float y[4];
#pragma unroll
                                    for (int j = 0; j < 4; ++j) {
                                        // a padding head's product is 0, but a NaN where the key holds an
                                        // infinity: the max drops it, else it is left out here
                                        y[j] = kRelu ? fmaxf(v[x + j], 0.0f) : c0 + x + j < sh.heads ? v[x + j] : 0.0f;
                                    }
                                    acc[0] = fmaf(f.x, y[0], acc[0]);
                                    acc[1] = fmaf(f.y, y[1], acc[1]);
                                    acc[2] = fmaf(f.z, y[2], acc[2]);
                                    acc[3] = fmaf(f.w, y[3], acc[3]);
                                }
                            }
                        }
                    }
                    const int j = k.tile * kTileKeys + t;
                    if (j < k.keys) {
                        const bool taken = j < sh.first || j >= k.keys - sh.last;
                        scores[(size_t)k.unit() * sh.stride + j] =
                            taken ? 0xFFFFFFFFu : order_word((acc[0] + acc[1]) + (acc[2] + acc[3]));
                    }
                }
            }
            if (it + 1 < count) k.next();
        }
        if (!ok) give_up(c, &d.ctl[CTL_ERR]);
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tbase, kTmemCols);
    }
}

// ---------------------------------------------------------------------------
constexpr int kPickThreads = 1024;
constexpr int kBins = 2048;            // two a thread
constexpr int kStagedKeys = 20480;     // scores a CTA keeps in shared memory (80 KB: two CTAs a SM)
constexpr int kWindowKeys = 262144;    // scores whose bits fit the same room when the scores stay in L2
constexpr int kFew = 1024;             // scores that are ranked directly
// Dynamic shared memory: the scores and two bits each, or the bits of a window alone.
constexpr size_t kPickSmem = (size_t)kStagedKeys * 4 + kStagedKeys / 4;
static_assert(kWindowKeys / 4 <= (int)kPickSmem, "a window's bits fit");
constexpr int kSample = 8;             // scores a thread samples of a long context

struct PickCtl {
    uint32_t hist[kBins];
    uint32_t few[kFew];                // the scores of the threshold's bin: this CTA's,
    uint32_t pool[kFew];               // and the team's
    uint32_t few_n;
    uint32_t lo, hi;                   // this CTA's range of scores
    uint32_t bin, need, count;         // the threshold's bin, what is still to take from it, what it holds
    uint32_t edge[2];                  // a bracket of the threshold, from a sample
    uint32_t above, ties;              // this CTA's scores above the threshold, and at it
    uint32_t warp_a[32], warp_b[32];
};

__device__ __forceinline__ uint32_t peer_load(const uint32_t* p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::map_to_rank(tc::smem_u32(p), rank)) : "memory");
    return v;
}
template <int kC>
__device__ __forceinline__ void team_sync()
{
    if constexpr (kC > 1)
        tc::cluster_sync();
    else
        __syncthreads();
}
template <int kC>
__device__ __forceinline__ uint32_t team_load(const uint32_t* p, uint32_t rank)
{
    if constexpr (kC > 1)
        return peer_load(p, rank);
    else
        return *p;
}

// f(score) for the m scores at s, four a thread at a time.
template <typename F>
__device__ __forceinline__ void each_score(const uint32_t* s, int m, F f)
{
    const int m4 = m >> 2;
#pragma unroll 4
    for (int i = threadIdx.x; i < m4; i += kPickThreads) {
        const uint4 v = reinterpret_cast<const uint4*>(s)[i];
        f(v.x);
        f(v.y);
        f(v.z);
        f(v.w);
    }
    const int i = 4 * m4 + threadIdx.x;
    if (i < m) f(s[i]);
}

// Inclusive sum over the CTA's threads, in thread order; `all` receives the total.
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
    const uint32_t w = warp_sum[lane];
    if (all) *all = __reduce_add_sync(0xFFFFFFFFu, w);
    return v + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u);
}

// One team (a CTA, or a cluster of kC that share the scores of a long context)
// a unit.  The threshold -- the score of the last block taken -- is found by
// narrowing its range: histogram 2048 equal parts of the range, find the part in
// which the count from above passes k / block, and go on inside it until it holds so few
// scores that they are ranked directly.  The first range is that of the scores
// themselves, so they spread over the bins and few atomics meet, and the first
// histogram is mostly the only one.  A context too long for shared memory is
// read from L2 in each pass; there the first range is a bracket of the threshold
// taken from a sample, so no pass is spent on the extremes and only the
// scores inside the bracket are counted (a bracket that misses is noticed by its
// counts and replaced by the whole range).  With the threshold known, one bit a
// score says what is taken, a scan of the words' counts gives each word its place,
// and the tokens come out ascending without a sort.
template <int kC>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(Dev d, const int32_t* __restrict__ req_ids, SelectShape sh,
                                                            const uint32_t* __restrict__ scores, int staged,
                                                            int32_t* __restrict__ topk)
{
    extern __shared__ __align__(16) uint32_t kept[];
    __shared__ PickCtl c;
    const int tid = threadIdx.x, lane = tid & 31;
    const int u = blockIdx.x / kC, rank = blockIdx.x % kC;
    int32_t* out = topk + (size_t)u * d.k;
    const int32_t r = req_ids[u / sh.layers];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores (and the error word) are complete
    if (d.ctl[CTL_ERR] != 0u) {  // the same for every CTA: nothing writes the word during this kernel
        for (int i = rank * kPickThreads + tid; i < d.k; i += kC * kPickThreads) out[i] = -1;
        return;
    }
    const int len = (int)d.len[r], n = keys_of(d, r, sh.block), nb = d.k / sh.block;
    if (n <= nb) {  // everything there is
        for (int i = rank * kPickThreads + tid; i < d.k; i += kC * kPickThreads) out[i] = i < len ? i : -1;
        return;
    }
    const int chunk = ((n + kC - 1) / kC + 127) & ~127;
    const int c0 = min(n, rank * chunk), m = min(n, c0 + chunk) - c0;
    const uint32_t* s = scores + (size_t)u * sh.stride + c0;
    if (tid == 0) {
        c.lo = 0xFFFFFFFFu;
        c.hi = 0u;
        c.above = c.ties = 0u;
    }
    for (int i = tid; i < kBins; i += kPickThreads) c.hist[i] = 0u;
    __syncthreads();

    // the first range
    uint32_t lo = 0xFFFFFFFFu, hi = 0u, seen[kSample];
    const bool on_chip = chunk <= staged;
    // a bit a score: above the threshold; at it (where not all of those are taken)
    uint32_t* taken = on_chip ? kept + chunk : kept;
    uint32_t* equal = taken + (on_chip ? chunk : kWindowKeys) / 32;
    if (on_chip) {
        const int m4 = m >> 2;
#pragma unroll 4
        for (int i = tid; i < m4; i += kPickThreads) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4*>(s) + i);
            reinterpret_cast<uint4*>(kept)[i] = v;
            lo = min(min(lo, v.x), min(v.y, min(v.z, v.w)));
            hi = max(max(hi, v.x), max(v.y, max(v.z, v.w)));
        }
        const int i = 4 * m4 + tid;
        if (i < m) {
            const uint32_t v = s[i];
            kept[i] = v;
            lo = min(lo, v);
            hi = max(hi, v);
        }
        s = kept;
    } else {  // evenly spaced scores of different keys (each CTA of the team has more than kSample * kPickThreads)
        const int step = m / (kSample * kPickThreads);
#pragma unroll
        for (int j = 0; j < kSample; ++j) {
            seen[j] = s[(size_t)(j * kPickThreads + tid) * step];
            lo = min(lo, seen[j]);
            hi = max(hi, seen[j]);
        }
    }
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if (lane == 0) {
        atomicMin(&c.lo, lo);
        atomicMax(&c.hi, hi);
    }
    team_sync<kC>();
    lo = 0xFFFFFFFFu;
    hi = 0u;
    for (int p = 0; p < kC; ++p) {
        lo = min(lo, team_load<kC>(&c.lo, p));
        hi = max(hi, team_load<kC>(&c.hi, p));
    }
    // thread t looks after the bins 2047 - 2t and 2046 - 2t: counts of the team, and a running count from the top
    uint32_t h1, h0, before, total;
    const int top = kBins - 1 - 2 * tid;
    auto count_bins = [&]() {
        team_sync<kC>();
        h1 = h0 = 0;
        for (int p = 0; p < kC; ++p) {
            h1 += team_load<kC>(&c.hist[top], p);
            h0 += team_load<kC>(&c.hist[top - 1], p);
        }
        before = cta_scan(h1 + h0, c.warp_a, &total) - h1 - h0;
    };
    auto clear_bins = [&]() {
        team_sync<kC>();  // the peers have read this histogram, too
        c.hist[top] = c.hist[top - 1] = 0u;
        __syncthreads();
    };
    auto shift_of = [](uint32_t span) {
        const int bits = 32 - __clz(span);
        return bits > 11 ? bits - 11 : 0;
    };
    uint32_t need = (uint32_t)nb;  // blocks still to take from [lo, hi]; every score above hi is taken
    bool bracket = false;
    if (!on_chip) {
        // ranks of the threshold in the sample, six standard deviations either way
        const int shift = shift_of(hi - lo);
#pragma unroll
        for (int j = 0; j < kSample; ++j) atomicAdd(&c.hist[(seen[j] - lo) >> shift], 1u);
        count_bins();
        const float share = (float)nb / (float)n * (float)total, dev = 6.0f * sqrtf(share) + 6.0f;
        const uint32_t upper = share > dev ? (uint32_t)(share - dev) : 0u, lower = (uint32_t)(share + dev);
        if (tid == 0) {
            c.edge[0] = 0u;            // no bin that low: open
            c.edge[1] = 0xFFFFFFFFu;
        }
        __syncthreads();
        if (before <= lower && lower < before + h1 + h0) c.edge[0] = lo + ((uint32_t)(top - 1) << shift);
        if (upper > 0u && before <= upper && upper < before + h1 + h0)
            c.edge[1] = min(hi - lo, ((uint32_t)(top + 1) << shift) - 1u) + lo;
        clear_bins();
        lo = c.edge[0];
        hi = max(c.edge[1], lo);
        bracket = true;
    }
    uint32_t above = 0;  // this thread's scores above the bracket
    bool all = false, exact = false;  // the whole range is taken; lo == hi is the threshold
    while (lo != hi || bracket) {
        const int shift = shift_of(hi - lo);
        each_score(s, m, [&](uint32_t v) {
            if (v >= lo && v <= hi) atomicAdd(&c.hist[(v - lo) >> shift], 1u);
            if (bracket) above += v > hi;
        });
        if (bracket) {
            above = __reduce_add_sync(0xFFFFFFFFu, above);
            if (lane == 0 && above) atomicAdd(&c.above, above);
        }
        count_bins();
        if (bracket) {
            uint32_t over = 0;
            for (int p = 0; p < kC; ++p) over += team_load<kC>(&c.above, p);
            bracket = false;
            if (over >= need || over + total < need) {  // the threshold is not in it
                clear_bins();
                lo = 0u;
                hi = 0xFFFFFFFFu;
                continue;
            }
            need -= over;
        }
        if (before < need && need <= before + h1) {
            c.bin = top;
            c.need = need - before;
            c.count = h1;
        } else if (before + h1 < need && need <= before + h1 + h0) {
            c.bin = top - 1;
            c.need = need - before - h1;
            c.count = h0;
        }
        clear_bins();
        lo += c.bin << shift;
        hi = min(hi - lo, (1u << shift) - 1u) + lo;  // (lo + 2^shift may pass 32 bits)
        need = c.need;
        const uint32_t in = c.count;
        all = need == in;
        if (all || lo == hi) break;
        if (in <= kFew) {
            // rank them: the threshold is the score with less than `need` above it and no less up to it
            if (tid == 0) c.few_n = 0u;
            __syncthreads();
            each_score(s, m, [&](uint32_t v) {
                if (v >= lo && v <= hi) c.few[atomicAdd(&c.few_n, 1u)] = v;
            });
            team_sync<kC>();
            uint32_t at = 0;
            for (int p = 0; p < kC; ++p) {
                const uint32_t np = team_load<kC>(&c.few_n, p);
                if (tid < np) c.pool[at + tid] = team_load<kC>(&c.few[tid], p);
                at += np;
            }
            __syncthreads();
            if (tid < in) {
                const uint32_t mine = c.pool[tid];
                uint32_t more = 0, same = 0;
                for (uint32_t i = 0; i < in; ++i) {
                    more += c.pool[i] > mine;
                    same += c.pool[i] == mine;
                }
                if (more < need && need <= more + same) {  // every thread with this score writes the same
                    c.lo = mine;
                    c.need = need - more;
                    c.count = same;
                }
            }
            __syncthreads();
            lo = hi = c.lo;
            need = c.need;
            all = need == c.count;
            break;
        }
        __syncthreads();  // c.bin, c.need and c.count have been read
    }
    exact = !all;  // then lo == hi, and of the scores equal to it the first `need` are taken
    // taken: above hi, or not below lo if the whole range is
    auto is_taken = [&](uint32_t v) { return v > hi || (all && v >= lo); };

    // one window of this CTA's scores: bits, the words' counts, places
    const int windows = (m + kWindowKeys - 1) / kWindowKeys;
    auto mark = [&](int w0, int wm) {
        const uint32_t* sw = s + w0;
        for (int i = 4 * tid; i < ((wm + 127) & ~127); i += 4 * kPickThreads) {
            uint32_t v[4];
            if (i + 4 <= wm) {
                const uint4 x = *reinterpret_cast<const uint4*>(sw + i);
                v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = i + j < wm ? sw[i + j] : 0u;
            }
            uint32_t a = 0, e = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = i + j < wm, t = in && is_taken(v[j]);
                a |= (uint32_t)t << j;
                e |= (uint32_t)(exact && in && !t && v[j] == lo) << j;
            }
            // eight lanes make a word of 32 keys
            uint32_t both = a | e << 4;
            a = both & 15u, e = both >> 4;
            a <<= 4 * (lane & 7);
            e <<= 4 * (lane & 7);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                a |= __shfl_xor_sync(0xFFFFFFFFu, a, o);
                e |= __shfl_xor_sync(0xFFFFFFFFu, e, o);
            }
            if ((lane & 7) == 0) {
                taken[i >> 5] = a;
                equal[i >> 5] = e;
            }
        }
    };
    if (tid == 0) c.above = 0u;
    team_sync<kC>();  // the peers have read c.above and the lists
    uint32_t na = 0, nt = 0;
    if (windows == 1) {
        mark(0, m);
        __syncthreads();
        for (int i = tid; i < (m + 31) / 32; i += kPickThreads) {
            na += __popc(taken[i]);
            nt += __popc(equal[i]);
        }
    } else {
        each_score(s, m, [&](uint32_t v) {
            const bool t = is_taken(v);
            na += t;
            nt += exact && !t && v == lo;
        });
    }
    uint32_t pa = 0, pt = 0;  // taken and equal in the CTAs before this one
    if constexpr (kC > 1) {
        na = __reduce_add_sync(0xFFFFFFFFu, na);
        nt = __reduce_add_sync(0xFFFFFFFFu, nt);
        if (lane == 0 && na) atomicAdd(&c.above, na);
        if (lane == 0 && nt) atomicAdd(&c.ties, nt);
        team_sync<kC>();
        for (int p = 0; p < rank; ++p) {
            pa += team_load<kC>(&c.above, p);
            pt += team_load<kC>(&c.ties, p);
        }
    }
    for (int w = 0; w < windows; ++w) {
        const int w0 = w * kWindowKeys, wm = min(m - w0, kWindowKeys);
        if (windows > 1) {
            __syncthreads();  // the window before has been written out
            mark(w0, wm);
            __syncthreads();
        }
        const int words = (wm + 31) / 32;
        for (int i0 = 0; i0 < words; i0 += kPickThreads) {
            const int i = i0 + tid;
            uint32_t a = i < words ? taken[i] : 0u, e = i < words ? equal[i] : 0u;
            const uint32_t ca = __popc(a), ce = __popc(e);
            uint32_t sum, sum_e;
            const uint32_t qa = pa + cta_scan(ca, c.warp_a, &sum) - ca;
            const uint32_t qe = exact ? pt + cta_scan(ce, c.warp_b, &sum_e) - ce : 0u;
            if (exact) {  // the first need - qe of the word's equal scores
                uint32_t left = need > qe ? need - qe : 0u;
                uint32_t kept_e = 0;
                while (e != 0u && left > 0u) {
                    kept_e |= e & (0u - e);
                    e &= e - 1u;
                    --left;
                }
                a |= kept_e;
                pt += sum_e;
            }
            uint32_t at = qa + min(qe, need);
            while (a != 0u) {
                const int key = c0 + w0 + 32 * i + __ffs(a) - 1;
                a &= a - 1u;
                if (sh.block == 1) {
                    out[at] = key;
                } else {
                    for (int x = 0; x < sh.block; ++x) {
                        const int token = key * sh.block + x;
                        out[(size_t)at * sh.block + x] = token < len ? token : -1;
                    }
                }
                ++at;
            }
            pa += sum;
            __syncthreads();  // the sums have been read
        }
    }
    if constexpr (kC > 1) tc::cluster_sync();  // the peers may still be reading this CTA's counts
}

}  // namespace

int64_t select_stride(int64_t max_context, int block) { return ((max_context + block - 1) / block + 127) / 128 * 128; }

cudaError_t prepare_select()
{
    cudaError_t e = cudaSuccess;
    auto set = [&](auto f, int bytes) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    set(score_kernel<64, false>, kScoreSmem);
    set(score_kernel<64, true>, kScoreSmem);
    set(score_kernel<128, false>, kScoreSmem);
    set(score_kernel<128, true>, kScoreSmem);
    set(pick_kernel<1>, (int)kPickSmem);
    set(pick_kernel<2>, (int)kPickSmem);
    set(pick_kernel<4>, (int)kPickSmem);
    set(pick_kernel<8>, (int)kPickSmem);
    return e;
}

cudaError_t launch_select(const Dev& d, const skv_index& ix, const int32_t* req_ids, int B, const void* q, const float* w,
                          int32_t* topk, void* workspace, int device_sms, cudaStream_t st)
{
    const int64_t max_keys = (d.T_max + ix.block - 1) / ix.block;
    TensorMapEncoder encode = nullptr;
    cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess) return e;
    SelectShape sh;
    sh.B = B;
    sh.layers = d.layer_sel >= 0 ? 1 : d.L;
    sh.heads = ix.heads;
    sh.npad = (ix.heads + 15) / 16 * 16;
    sh.block = ix.block;
    sh.first = ix.first;
    sh.last = ix.last;
    sh.stride = select_stride(d.T_max, ix.block);
    const int64_t units = (int64_t)B * sh.layers;

    CUtensorMap key_map, q_map;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    {
        const cuuint64_t dims[4] = {(cuuint64_t)ix.dim, (cuuint64_t)max_keys, (cuuint64_t)d.L, (cuuint64_t)d.R};
        // the stride of an axis with one entry is never used
        const cuuint64_t strides[3] = {(cuuint64_t)(max_keys > 1 ? ix.key_stride : 2 * ix.dim),
                                       (cuuint64_t)(d.L > 1 ? ix.layer_stride : 2 * ix.dim),
                                       (cuuint64_t)(d.R > 1 ? ix.request_stride : 2 * ix.dim)};
        const cuuint32_t box[4] = {64, kTileKeys, 1, 1};
        if (encode(&key_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ix.keys), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    {
        const cuuint64_t dims[3] = {(cuuint64_t)ix.dim, (cuuint64_t)ix.heads, (cuuint64_t)units};
        const cuuint64_t strides[2] = {(cuuint64_t)(2 * ix.dim), (cuuint64_t)(2 * ix.dim) * ix.heads};
        const cuuint32_t box[3] = {64, (cuuint32_t)ix.heads, 1};
        if (encode(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    uint32_t* scores = static_cast<uint32_t*>(workspace);
    const ScoreLayout lay = score_layout(ix.dim, sh.npad);
    const int64_t tiles = units * ((max_keys + kTileKeys - 1) / kTileKeys);  // at most
    const unsigned grid = (unsigned)std::min<int64_t>(device_sms, tiles);
    auto score = ix.dim == 64 ? (ix.relu ? score_kernel<64, true> : score_kernel<64, false>)
                              : (ix.relu ? score_kernel<128, true> : score_kernel<128, false>);
    score<<<grid, kScoreThreads, lay.bytes, st>>>(key_map, q_map, d, req_ids, w, sh, lay, scores);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    // A unit's scores go to one CTA while they fit its shared memory and units fill the SMs; else a
    // cluster shares them (never fewer than 2048 scores a CTA).
    int team = 1;
    while (team < 8 && max_keys / (2 * team) >= 2048 && (max_keys / team > kStagedKeys || units * team * 2 <= device_sms)) team *= 2;
    const int64_t chunk = ((max_keys + team - 1) / team + 127) & ~(int64_t)127;
    const int staged = (int)std::min<int64_t>(chunk, kStagedKeys);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * team));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = chunk <= staged ? (size_t)staged * 4 + staged / 4 : kPickSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = team;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // takes the SMs that score_kernel leaves, and waits
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto pick = team == 1 ? pick_kernel<1> : team == 2 ? pick_kernel<2> : team == 4 ? pick_kernel<4> : pick_kernel<8>;
    return cudaLaunchKernelEx(&cfg, pick, d, req_ids, sh, static_cast<const uint32_t*>(scores), staged, topk);
}

}  // namespace skv
