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
    int withhold_keys;     // the timeout self-test: no load is issued, so the first wait for one runs out
    int64_t stride;        // scores a unit has room for
};

// (Lengths are at most 2^30.  A 64-bit division costs 0.2 us, which a call of few keys notices.)
__device__ __forceinline__ int keys_of_len(int32_t len, int block) { return (int)(((uint32_t)len + block - 1u) / (uint32_t)block); }
__device__ __forceinline__ int keys_of(const Dev& d, int32_t r, int block) { return keys_of_len((int32_t)d.len[r], block); }
__device__ __forceinline__ uint64_t divide(uint64_t a, uint32_t b) { return a >> 32 ? a / b : (uint32_t)a / b; }

struct alignas(16) ScoreCtl {
    uint64_t full[8], empty[8];            // key stages
    uint64_t q_full[2], q_empty[2];        // query buffers
    uint64_t d_full[kDepth], d_empty[kDepth];  // products
    uint64_t fin;                          // every MMA this CTA issued has completed
    alignas(16) float w[kGroups][kMaxHeads];  // a warpgroup's copy of its unit's weights, read as float4
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
// enough stages in flight (6 of 32 KB at 64 heads), and the products issued at the
// tensor pipe's rate: from a single lane, with operands that have to be moved to uniform registers
// one by one, they were what held it back (986 us at 192 x 8 units of 16K keys).
// Measured: 895 us there (6.17 GB, 6.9 TB/s, a copy's rate), 625 us at 16
// units of 1M (4.29 GB, 6.9 TB/s); 7.6 us at 4 units of 4K, where the set-up and one
// tile's way through the roles are all there is.
template <int kDim, bool kRelu>
__global__ void __launch_bounds__(kScoreThreads, 1)
    score_kernel(const __grid_constant__ CUtensorMap key_map, const __grid_constant__ CUtensorMap q_map, Dev d,
                 const int32_t* req_ids, const float* w, SelectShape sh, ScoreLayout lay,
                 uint32_t* __restrict__ scores, int32_t* __restrict__ lens)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    ScoreCtl& c = *reinterpret_cast<ScoreCtl*>(smem + lay.off_ctl);
    constexpr int kBoxes = kDim / 64;  // 64-dim columns of a key tile, 128 bytes wide
    constexpr uint32_t kBoxBytes = kTileKeys * 128, kStageBytes = kBoxes * kBoxBytes;
    const uint32_t q_box = sh.npad * 128u, q_bytes = kBoxes * q_box;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    chain_next();
    chain_wait();
    req_ids = behind_wait(req_ids);
    w = behind_wait(w);

    // the call's entries: every id an active request; how many tiles each has
    const int per = (sh.B + kScoreThreads - 1) / kScoreThreads;
    const int b0 = min(sh.B, tid * per), b1 = min(sh.B, b0 + per);
    bool bad = false, stop = tid == 0 && d.ctl[CTL_ERR] != 0u;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
        const int32_t r = req_ids[b];
        int32_t len = 0;
        if (r < 0 || r >= d.R || !d.active[r]) {
            bad = true;
        } else {
            len = (int32_t)d.len[r];
            mine += (keys_of_len(len, sh.block) + kTileKeys - 1) / kTileKeys;
        }
        if (blockIdx.x == 0) lens[b] = len;  // for pick_kernel, which has it one read sooner
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
    stop = __syncthreads_or(stop || bad);  // pick_kernel sees the error word
    long long before = upto - mine, total = 0;
    for (int i = 0; i < kScoreThreads / 32; ++i) {
        if (i < warp) before += c.sums[i];
        total += c.sums[i];
    }
    const uint64_t all = stop ? 0 : (uint64_t)total * sh.layers, share = divide(all, gridDim.x);
    const uint32_t extra = (uint32_t)(all - share * gridDim.x);  // CTAs with one tile more
    const uint64_t begin = share * blockIdx.x + min(blockIdx.x, extra);
    const int count = (int)share + (blockIdx.x < extra ? 1 : 0);
    if (count > 0 && begin >= (uint64_t)before * sh.layers && begin < (uint64_t)(before + mine) * sh.layers) {  // this thread's entries hold it
        uint64_t at = (uint64_t)before * sh.layers;
        for (int b = b0; b < b1; ++b) {
            const uint32_t t = per == 1 ? (uint32_t)mine : (keys_of(d, req_ids[b], sh.block) + kTileKeys - 1) / kTileKeys;
            if (begin < at + (uint64_t)t * sh.layers) {
                const uint64_t l = divide(begin - at, t);
                c.start[0] = b;
                c.start[1] = (int)l;
                c.start[2] = (int)(begin - at - l * t);
                break;
            }
            at += (uint64_t)t * sh.layers;
        }
    }
    // (The set-up stays behind the wait: with it in front, all CTAs begin to stream in the same moment, which costs
    // 1 % of the bandwidth at 192 x 8 units of 16K keys and gains nothing at 4 of 4K.)
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
        tc::mbar_init(&c.fin, 1);
        c.abort = 0u;
    }
    // query rows behind the last head are zeros for good (a copy writes `heads` rows)
    for (uint32_t i = tid; i < 2 * q_bytes / 16; i += kScoreThreads)
        reinterpret_cast<uint4*>(smem + lay.off_q)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_smem_async();
    if (warp == kMmaWarp) tc::tmem_alloc(&c.tmem_base, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = c.tmem_base;
    const volatile uint32_t* abort = &c.abort;
    const int nst = lay.stages;

    if (count == 0) {
        // no tile for this CTA
    } else if (warp == kLoadWarp) {
        if (lane == 0 && !sh.withhold_keys) {
            Walk k(d, sh, req_ids, c.start);
            const uint64_t stream_once = tc::evict_first_policy();  // keys pass L2 by; the scores stay for pick_kernel
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
                                  d.layer_sel >= 0 ? d.layer_sel : k.l, k.r, &c.full[s], stream_once);
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
        // the whole warp walks, and a lane that is elected issues (see mma_bf16_warp)
        Walk k(d, sh, req_ids, c.start);
        const uint32_t idesc = tc::idesc_bf16_f32(kTileKeys, sh.npad, 0), tb = __shfl_sync(0xFFFFFFFFu, tbase, 0);
        const int all = __shfl_sync(0xFFFFFFFFu, count, 0);
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, abort)); };
        bool ok = true;
        int units = 0;
        for (int it = 0; it < all; ++it) {
            if (__all_sync(0xFFFFFFFFu, k.fresh)) {
                if (!(ok = wait(&c.q_full[units & 1], (units >> 1) & 1))) break;
                ++units;
            }
            const int s = it % nst, p = it % kDepth, qb = (units - 1) & 1;
            if (it >= kDepth && !(ok = wait(&c.d_empty[p], ((it / kDepth) - 1) & 1))) break;
            if (!(ok = wait(&c.full[s], (it / nst) & 1))) break;
            tc::fence_after_sync();
            const uint32_t ka = tc::smem_u32(smem) + s * kStageBytes, qa = tc::smem_u32(smem + lay.off_q) + qb * q_bytes;
#pragma unroll
            for (int st = 0; st < kDim / 16; ++st)
                tc::mma_bf16_warp(tb + p * kMaxHeads, tc::sw128_kmajor_desc(ka + (st >> 2) * kBoxBytes + (st & 3) * 32),
                                  tc::sw128_kmajor_desc(qa + (st >> 2) * q_box + (st & 3) * 32), idesc, st > 0 ? 1u : 0u);
            tc::mma_commit_warp(&c.empty[s]);
            tc::mma_commit_warp(&c.d_full[p]);
            if (__all_sync(0xFFFFFFFFu, k.last_of_unit())) tc::mma_commit_warp(&c.q_empty[qb]);
            if (it + 1 < all) k.next();
        }
        if (!ok) give_up(c, &d.ctl[CTL_ERR]);
        tc::mma_commit_warp(&c.fin);  // no product, and no arrival of one, is left when the CTA leaves
        if (!tc::mbar_wait(&c.fin, 0, 1u << 22)) give_up(c, &d.ctl[CTL_ERR]);
        __syncwarp();
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
constexpr int kPickThreads = 512;
constexpr int kBinBits = 10;
constexpr int kBins = 1 << kBinBits;   // two a thread
constexpr int kStagedKeys = 20480;     // scores a CTA keeps in shared memory (80 KB: two CTAs a SM; three up to 64 KB)
constexpr int kWindowKeys = 524288;    // scores whose bits fit the same room when the scores stay in L2
constexpr int kFew = 512;              // scores that are ranked directly
constexpr int kSample = 4;             // scores a thread samples of a long context
// Dynamic shared memory: the scores and a bit each, or the bits of a window alone.
constexpr size_t kPickSmem = (size_t)kStagedKeys * 4 + kStagedKeys / 8;
static_assert(kWindowKeys / 8 + kMaxTopk / 2 * 4 <= (int)kPickSmem, "a window's bits fit, and the blocks behind them");

template <int kC>
struct PickCtl {
    uint32_t hist[kBins];
    uint2 few[kFew];                   // (score, key) in the threshold's bin: this CTA's,
    uint2 pool[kC > 1 ? kFew : 1];     // and the team's
    uint32_t few_n;
    uint32_t lo, hi;                   // this CTA's range of scores
    uint32_t bin, need, count;         // the threshold's bin, what is still to take from it, what it holds
    uint32_t edge[2];                  // a bracket of the threshold, from a sample
    uint32_t over;                     // this CTA's scores above the bracket
    uint32_t taken;                    // what this CTA takes
    uint2 last;                        // (score, key) of the last block taken
    uint32_t err;                      // the error word, read by one thread
    uint32_t warp_sum[32];
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

// 16-byte reads a thread has in flight (longer contexts are read from L2 in every pass)
template <int kC>
constexpr int kAtOnce = kC > 1 ? 8 : 4;

__device__ __forceinline__ uint32_t largest(uint4 v) { return max(max(v.x, v.y), max(v.z, v.w)); }

// f(score, index) for those of the m scores at s that are at least `least`, and perhaps for others.  Four a thread at a
// time; mostly all four are below.
template <int kReads, typename F>
__device__ __forceinline__ void each_score(const uint32_t* s, int m, uint32_t least, F f)
{
    const int m4 = m >> 2;
    const uint4* s4 = reinterpret_cast<const uint4*>(s);
    int i = threadIdx.x;
    for (; i + (kReads - 1) * kPickThreads < m4; i += kReads * kPickThreads) {
        uint4 v[kReads];  // read before f may write shared memory, so that the reads are in flight together
#pragma unroll
        for (int x = 0; x < kReads; ++x) v[x] = s4[i + x * kPickThreads];
#pragma unroll
        for (int x = 0; x < kReads; ++x) {
            const int at = 4 * (i + x * kPickThreads);
            if (largest(v[x]) >= least) {
                f(v[x].x, at);
                f(v[x].y, at + 1);
                f(v[x].z, at + 2);
                f(v[x].w, at + 3);
            }
        }
    }
    for (; i < m4; i += kPickThreads) {
        const uint4 v = s4[i];
        if (largest(v) >= least) {
            f(v.x, 4 * i);
            f(v.y, 4 * i + 1);
            f(v.z, 4 * i + 2);
            f(v.w, 4 * i + 3);
        }
    }
    i = 4 * m4 + threadIdx.x;
    if (i < m) f(s[i], i);
}

// Inclusive sum over the CTA's threads, in thread order; *all receives the total.
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
    const uint32_t w = lane < kPickThreads / 32 ? warp_sum[lane] : 0u;
    *all = __reduce_add_sync(0xFFFFFFFFu, w);
    return v + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u);
}

// One team (a CTA, or a cluster of kC that share the scores of a long context)
// a unit.  Taken are the k / block first in the order (score descending, key
// ascending); the last of them is the threshold, and a key is taken if it is not
// behind it.  The threshold is found by narrowing its range: histogram 1024 equal
// parts of the range, find the part in which the count from above passes k / block, and
// go on inside it until it holds so few scores that they are ranked directly.
// The first range is that of the scores themselves, so they spread over the bins
// and few atomics meet, and the first histogram is mostly the only one.  (More
// scores equal to the threshold than can be ranked: their keys are narrowed down in the
// same way.)  A context too long for shared memory is read from L2 in each
// pass; there the first range is a bracket of the threshold taken from a sample,
// so no pass is spent on the extremes and only the scores inside the bracket are
// counted (a bracket that misses shows in its counts and is replaced by the
// whole range).  With the threshold known, one bit a score says what is taken, a
// scan of the words' counts gives each word its place, and the tokens come out
// ascending without a sort.
// Bound by latency: a unit is a chain of some twelve barriers, and three CTAs a SM (teams of eight
// for long contexts, two CTAs a SM, so that 16 teams are on the chip at once: with one they were not, 20 us more)
// only hide part of it.  Measured by itself: 63 us at 192 x 8 units of 16K scores (101 MB, just written), of a
// call 60; of a call of 16 units of 1M (67 MB read from L2 two to three times) 65; 7.7 us at 4 units of 4K.
template <int kC>
__global__ void __launch_bounds__(kPickThreads, kC == 1 ? 3 : 2) pick_kernel(Dev d, const int32_t* lens, SelectShape sh,
                                                            const uint32_t* scores, int staged,
                                                            int32_t* __restrict__ topk)
{
    extern __shared__ __align__(16) uint32_t kept[];
    __shared__ PickCtl<kC> c;
    constexpr int kReads = kAtOnce<kC>;
    const int tid = threadIdx.x, lane = tid & 31;
    const int u = blockIdx.x / kC, rank = blockIdx.x % kC;
    int32_t* out = topk + (size_t)u * d.k;
    chain_next();
    if (tid == 0) {
        c.lo = 0xFFFFFFFFu;
        c.hi = 0u;
        c.over = c.taken = 0u;
    }
    for (int i = tid; i < kBins; i += kPickThreads) c.hist[i] = 0u;
    chain_wait();  // the scores (and the error word) are complete
    lens = behind_wait(lens);
    scores = behind_wait(scores);
    const int len = __ldcg(lens + u / sh.layers);
    // One read a CTA, and the team goes by all of them: a call on another stream may set the word meanwhile.
    if (tid == 0) c.err = d.ctl[CTL_ERR];
    auto team_error = [&]() {  // behind a team_sync
        uint32_t e = 0;
        for (int p = 0; p < kC; ++p) e |= team_load<kC>(&c.err, p);
        return e != 0u;
    };
    auto fill = [&](bool nothing) {  // -1, or everything there is
        for (int i = rank * kPickThreads + tid; i < d.k; i += kC * kPickThreads) out[i] = !nothing && i < len ? i : -1;
        if constexpr (kC > 1) tc::cluster_sync();  // the peers may still be reading this CTA's memory
    };
    // A thread's first scores, read before it is known how many there are (a unit's room is a multiple of 128).
    uint4 first = make_uint4(0, 0, 0, 0);
    if (kC == 1 && 4 * tid < sh.stride) first = __ldcg(reinterpret_cast<const uint4*>(scores + (size_t)u * sh.stride) + tid);
    const int n = keys_of_len(len, sh.block), nb = d.k / sh.block;
    if (n <= nb) {
        team_sync<kC>();
        fill(team_error());
        return;
    }
    const int chunk = ((n + kC - 1) / kC + 127) & ~127;
    const int c0 = min(n, rank * chunk), m = min(n, c0 + chunk) - c0;
    const uint32_t* s = scores + (size_t)u * sh.stride + c0;
    const bool on_chip = chunk <= staged;
    uint32_t* bits = on_chip ? kept + chunk : kept;
    __syncthreads();

    // the first range
    uint32_t lo = 0xFFFFFFFFu, hi = 0u, seen[kSample];
    if (on_chip) {
        const int m4 = m >> 2;
        auto keep = [&](uint4 v, int i) {
            reinterpret_cast<uint4*>(kept)[i] = v;
            lo = min(min(lo, v.x), min(v.y, min(v.z, v.w)));
            hi = max(max(hi, v.x), max(v.y, max(v.z, v.w)));
        };
        if (kC == 1 && tid < m4) keep(first, tid);
#pragma unroll 8
        for (int i = kC == 1 ? tid + kPickThreads : tid; i < m4; i += kPickThreads) keep(__ldcg(reinterpret_cast<const uint4*>(s) + i), i);
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
    if (team_error()) {  // (the scores may never have been written)
        fill(true);
        return;
    }
    lo = c.lo;
    hi = c.hi;
    if constexpr (kC > 1) {
        for (int p = 0; p < kC; ++p) {
            lo = min(lo, team_load<kC>(&c.lo, p));
            hi = max(hi, team_load<kC>(&c.hi, p));
        }
    }
    // thread t looks after the bins kBins - 1 - 2t and kBins - 2 - 2t: counts of the team, and a running
    // count from the top
    static_assert(kBins == 2 * kPickThreads, "two bins a thread");
    uint32_t h1, h0, before, total;
    const int top = kBins - 1 - 2 * tid;
    auto count_bins = [&]() {
        team_sync<kC>();
        h1 = h0 = 0;
        for (int p = 0; p < kC; ++p) {
            h1 += team_load<kC>(&c.hist[top], p);
            h0 += team_load<kC>(&c.hist[top - 1], p);
        }
        before = cta_scan(h1 + h0, c.warp_sum, &total) - h1 - h0;
    };
    auto clear_bins = [&]() {
        team_sync<kC>();  // every thread of the team has read what it needs
        c.hist[top] = c.hist[top - 1] = 0u;
        __syncthreads();
    };
    auto shift_of = [](uint32_t span) {
        const int bits = 32 - __clz(span);
        return bits > kBinBits ? bits - kBinBits : 0;
    };
    uint32_t need = (uint32_t)nb;  // blocks still to take from [lo, hi]; every score above hi is taken
    bool bracket = false, open = false;
    if (!on_chip) {
        // ranks of the threshold in the sample, six standard deviations either way
        const int shift = shift_of(hi - lo);
#pragma unroll
        for (int j = 0; j < kSample; ++j) atomicAdd(&c.hist[(seen[j] - lo) >> shift], 1u);
        count_bins();
        const float share = (float)nb / (float)n * (float)total, dev = 6.0f * sqrtf(share) + 6.0f;
        const uint32_t upper = share > dev ? (uint32_t)(share - dev) : 0u, lower = (uint32_t)(share + dev);
        open = upper == 0u;  // then the last bin takes whatever lies above the sample, too
        if (tid == 0) {
            c.edge[0] = 0u;  // no bin that low
            c.edge[1] = hi;
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

    // Narrow the scores, then, if need be, the keys of the scores equal to the threshold (as ~key: the lower key is
    // the larger).  [lo, hi] is the range of either.
    bool keys = false, marked = false;
    uint32_t tv = 0, ti = 0;  // the threshold: score and key
    auto is_taken = [&](uint32_t v, uint32_t key) { return v > tv || (v == tv && key <= ti); };
    // One window of this CTA's scores: a bit each for f(score, key), which is false below `least`.  A lane has four
    // consecutive keys, eight lanes make a word.
    const int windows = (m + kWindowKeys - 1) / kWindowKeys;
    auto mark = [&](int w0, int wm, uint32_t least, auto f) {
        const uint32_t* sw = s + w0;
        const int end = (wm + 127) & ~127;  // whole warps
        for (int i0 = 4 * tid; i0 < end; i0 += 4 * kPickThreads * kReads) {
            uint4 v[kReads];
#pragma unroll
            for (int x = 0; x < kReads; ++x) {
                const int i = i0 + 4 * kPickThreads * x;
                v[x] = make_uint4(0, 0, 0, 0);
                if (i + 4 <= wm) {
                    v[x] = *reinterpret_cast<const uint4*>(sw + i);
                } else if (i < wm) {
                    v[x].x = sw[i];
                    if (i + 1 < wm) v[x].y = sw[i + 1];
                    if (i + 2 < wm) v[x].z = sw[i + 2];
                }
            }
#pragma unroll
            for (int x = 0; x < kReads; ++x) {
                const int i = i0 + 4 * kPickThreads * x;
                if (i < end) {  // the same for a warp
                    uint32_t a = 0u;
                    if (__any_sync(0xFFFFFFFFu, largest(v[x]) >= least)) {
                        const uint32_t key = (uint32_t)(c0 + w0 + i);
                        if (i + 4 <= wm)
                            a = (f(v[x].x, key) ? 1u : 0u) | (f(v[x].y, key + 1) ? 2u : 0u) |
                                (f(v[x].z, key + 2) ? 4u : 0u) | (f(v[x].w, key + 3) ? 8u : 0u);
                        else if (i < wm)
                            a = (f(v[x].x, key) ? 1u : 0u) | (i + 1 < wm && f(v[x].y, key + 1) ? 2u : 0u) |
                                (i + 2 < wm && f(v[x].z, key + 2) ? 4u : 0u);
                        a <<= 4 * (lane & 7);
                        a |= __shfl_xor_sync(0xFFFFFFFFu, a, 1);
                        a |= __shfl_xor_sync(0xFFFFFFFFu, a, 2);
                        a |= __shfl_xor_sync(0xFFFFFFFFu, a, 4);
                    }
                    if ((lane & 7) == 0) bits[i >> 5] = a;
                }
            }
        }
    };
    for (;;) {
        if (lo == hi && !bracket) {
            if (keys) {  // a single key
                ti = ~lo;
                break;
            }
            tv = lo;  // equal scores, more of them than needed
            keys = true;
            lo = ~(uint32_t)(n - 1);
            hi = 0xFFFFFFFFu;
        }
        const int shift = shift_of(hi - lo);
        uint32_t over = 0;
        const uint32_t span = hi - lo;
        if (keys)
            each_score<kReads>(s, m, tv, [&](uint32_t v, int i) {
                const uint32_t x = ~(uint32_t)(c0 + i) - lo;
                if (v == tv && x <= span) atomicAdd(&c.hist[x >> shift], 1u);
            });
        else if (bracket)
            each_score<kReads>(s, m, lo, [&](uint32_t v, int) {
                if (v > hi && !open)
                    ++over;
                else if (v >= lo)
                    atomicAdd(&c.hist[min((v - lo) >> shift, (uint32_t)kBins - 1u)], 1u);
            });
        else
            each_score<kReads>(s, m, lo, [&](uint32_t v, int) {
                if (v - lo <= span) atomicAdd(&c.hist[(v - lo) >> shift], 1u);
            });
        if (bracket) {
            over = __reduce_add_sync(0xFFFFFFFFu, over);
            if (lane == 0 && over) atomicAdd(&c.over, over);
        }
        count_bins();
        if (bracket) {
            over = 0;
            for (int p = 0; p < kC; ++p) over += team_load<kC>(&c.over, p);
            bracket = false;
            if (over >= need || over + total < need) {  // the threshold is not in it
                clear_bins();
                lo = 0u;
                hi = 0xFFFFFFFFu;
                continue;
            }
            need -= over;
            if (open) hi = 0xFFFFFFFFu;
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
        __syncthreads();
        lo += c.bin << shift;
        if (!open || c.bin != kBins - 1) hi = min(hi - lo, (1u << shift) - 1u) + lo;  // (lo + 2^shift may pass 32 bits)
        open = false;
        need = c.need;
        const uint32_t in = c.count;
        if (need == in) {  // all of the range
            if (!keys) {
                tv = lo;  // every score from lo on, whatever its key
                ti = 0xFFFFFFFFu;
            } else {
                ti = ~lo;
            }
            break;
        }
        if (in <= kFew) {
            // rank them in the order of taking: the threshold is the one with need - 1 before it
            if (tid == 0) c.few_n = 0u;
            __syncthreads();
            const uint32_t span = hi - lo;
            marked = windows == 1 && !keys;
            if (marked)  // the bits of what is above the range in the same pass
                mark(0, m, lo, [&](uint32_t v, uint32_t key) {
                    if (v - lo <= span) c.few[atomicAdd(&c.few_n, 1u)] = make_uint2(v, key);
                    return v > hi;
                });
            else
                each_score<kReads>(s, m, keys ? tv : lo, [&](uint32_t v, int i) {
                    const uint32_t key = (uint32_t)(c0 + i);
                    if ((keys ? ~key : v) - lo <= span && (!keys || v == tv)) c.few[atomicAdd(&c.few_n, 1u)] = make_uint2(v, key);
                });
            team_sync<kC>();
            const uint2* list = c.few;
            if constexpr (kC > 1) {
                uint32_t at = 0;
                for (int p = 0; p < kC; ++p) {
                    const uint32_t np = team_load<kC>(&c.few_n, p);
                    if (tid < np) c.pool[at + tid] = make_uint2(team_load<kC>(&c.few[tid].x, p), team_load<kC>(&c.few[tid].y, p));
                    at += np;
                }
                __syncthreads();
                list = c.pool;
            }
            if (tid < in) {
                const uint2 mine = list[tid];
                uint32_t first = 0;
                for (uint32_t i = 0; i < in; ++i) {
                    const uint2 o = list[i];
                    first += o.x > mine.x || (o.x == mine.x && o.y < mine.y);
                }
                if (first + 1 == need) c.last = mine;
            }
            __syncthreads();
            tv = c.last.x;
            ti = c.last.y;
            if (marked && tid < c.few_n && is_taken(c.few[tid].x, c.few[tid].y))
                atomicOr(&bits[(c.few[tid].y - c0) >> 5], 1u << ((c.few[tid].y - c0) & 31u));
            break;
        }
        clear_bins();
    }
    if (!marked && windows == 1) mark(0, m, tv, is_taken);
    uint32_t base = 0;  // taken in the CTAs before this one
    if constexpr (kC > 1) {
        uint32_t mine = 0;
        if (windows == 1) {
            __syncthreads();
            for (int i = tid; i < (m + 31) / 32; i += kPickThreads) mine += __popc(bits[i]);
        } else {
            each_score<kReads>(s, m, tv, [&](uint32_t v, int i) { mine += is_taken(v, (uint32_t)(c0 + i)); });
        }
        mine = __reduce_add_sync(0xFFFFFFFFu, mine);
        if (lane == 0 && mine) atomicAdd(&c.taken, mine);
        team_sync<kC>();
        for (int p = 0; p < rank; ++p) base += team_load<kC>(&c.taken, p);
    }
    const uint32_t base0 = base;
    // the blocks taken, by place: where the scores were (more of them than blocks), or behind the window's bits
    uint32_t* blocks = (on_chip ? kept : kept + kWindowKeys / 32) - base0;
    for (int w = 0; w < windows; ++w) {
        const int w0 = w * kWindowKeys, wm = min(m - w0, kWindowKeys);
        __syncthreads();  // the bits are written, or the window before has been written out
        if (windows > 1) {
            mark(w0, wm, tv, is_taken);
            __syncthreads();
        }
        const int words = (wm + 31) / 32;
        for (int i0 = 0; i0 < words; i0 += kPickThreads) {
            const int i = i0 + tid;
            uint32_t a = i < words ? bits[i] : 0u, sum;
            uint32_t at = base + cta_scan(__popc(a), c.warp_sum, &sum) - __popc(a);
            while (a != 0u) {
                const int key = c0 + w0 + 32 * i + __ffs(a) - 1;
                a &= a - 1u;
                if (sh.block == 1)
                    out[at] = key;
                else
                    blocks[at] = (uint32_t)key;
                ++at;
            }
            base += sum;
            if (i0 + kPickThreads < words) __syncthreads();  // the sums have been read
        }
    }
    if (sh.block > 1) {  // the blocks' tokens, by all threads
        __syncthreads();
        for (int i = (int)base0 * sh.block + tid; i < (int)base * sh.block; i += kPickThreads) {
            const int at = i / sh.block, token = (int)blocks[at] * sh.block + (i - at * sh.block);
            out[i] = token < len ? token : -1;
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
                          int32_t* topk, void* workspace, int device_sms, cudaStream_t st, bool withhold_keys)
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
    sh.withhold_keys = withhold_keys ? 1 : 0;
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
    int32_t* lens = reinterpret_cast<int32_t*>(scores + units * sh.stride);
    const ScoreLayout lay = score_layout(ix.dim, sh.npad);
    const int64_t tiles = units * ((max_keys + kTileKeys - 1) / kTileKeys);  // at most
    const unsigned grid = (unsigned)std::min<int64_t>(device_sms, tiles);
    auto score = ix.dim == 64 ? (ix.relu ? score_kernel<64, true> : score_kernel<64, false>)
                              : (ix.relu ? score_kernel<128, true> : score_kernel<128, false>);
    e = launch_chained(score, dim3(grid), kScoreThreads, lay.bytes, st, key_map, q_map, d, req_ids, w, sh, lay, scores, lens);
    if (e != cudaSuccess) return e;

    // A unit's scores go to one CTA while they fit its shared memory and units fill the SMs; else a
    // cluster shares them (never fewer than 8192 scores a CTA: the cluster's barriers cost more than they save).
    int team = 1;
    while (team < 8 && max_keys / (2 * team) >= 8192 && (max_keys / team > kStagedKeys || units * team * 2 <= device_sms)) team *= 2;
    const int64_t chunk = ((max_keys + team - 1) / team + 127) & ~(int64_t)127;
    const int staged = (int)std::min<int64_t>(chunk, kStagedKeys);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(units * team));
    cfg.blockDim = dim3(kPickThreads);
    cfg.dynamicSmemBytes = chunk <= staged ? (size_t)staged * 4 + staged / 8 : kPickSmem;
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
    return cudaLaunchKernelEx(&cfg, pick, d, static_cast<const int32_t*>(lens), sh, static_cast<const uint32_t*>(scores), staged, topk);
}

}  // namespace skv
