// Rounding KV rows to 4 bits and back (the packed row of q4.cuh).  A cache of
// packed rows moves 336 bytes a token over the host link instead of 1152, and
// the link is what bounds a decode step's assembly ("Sparse Attention-Driven
// KVCache Management for Domestic AI Supernodes", agenda item 3: the overhead
// of on-demand data movement).  Measured, 2048 tokens a unit of which 20 % are
// new: a step of 192 x 8 units of 16K tokens 1.008 ms instead of 2.92 (521 instead of
// 180 M rows/s, 175 instead of 207 GB/s), of 32 x 4 units of 128K 113 us instead of 297,
// of 4 x 4 units of 1M 30 us instead of 52.
//
// For a row x, groups g of 16 values:
//   a_g = max |x| over the group (0 for a group that holds a NaN or an infinity);
//   e   = the least integer with 2688 * 2^e >= max a_g, kept in [-100, 116]
//         (2688 = 448 * 6, the largest e4m3 times the largest e2m1);
//   s_g = a_g * 2^-e / 6 rounded to e4m3 (a NaN for a group with a NaN or an infinity);
//   c_i = x_i * 2^-e / s_g rounded to e2m1 (0 where s_g = 0).
// Roundings are to nearest, ties to even, saturating.

#include <cstdint>
#include <string>

#include "q4.cuh"
#include "skv_ctx.cuh"

namespace skv {
namespace {

// 32 bytes at a time: one access if everything is 32-byte aligned (kWide), else two.
template <bool kWide>
__device__ __forceinline__ void load32(const uint8_t* p, uint4& a, uint4& b)
{
    if constexpr (kWide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                     : "l"(p));
    } else {
        a = reinterpret_cast<const uint4*>(p)[0];
        b = reinterpret_cast<const uint4*>(p)[1];
    }
}
template <bool kWide>
__device__ __forceinline__ void store32(uint8_t* p, uint4 a, uint4 b)
{
    if constexpr (kWide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                     "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = a;
        reinterpret_cast<uint4*>(p)[1] = b;
    }
}

constexpr int kPackThreads = 128;
constexpr int kLanesPerRow = 4;                              // 9 groups of 16 values a lane
constexpr int kLaneGroups = q4::kGroups / kLanesPerRow;
constexpr int kPackRows = kPackThreads / kLanesPerRow;       // rows a CTA packs
static_assert(kLaneGroups * kLanesPerRow == q4::kGroups, "groups divide over the lanes of a row");

// s_g of a group as an e4m3 byte; t = a_g * 2^-e, at most 2688 save in rows at the end of bf16's range.
__device__ __forceinline__ uint32_t scale_code(float t)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(__fdiv_rn(t, 6.0f)));
    return r & 0xFFu;
}

// Two values to two codes (lo in the low half of the byte); y = x * 2^-e / s.
// y comes from a multiplication with the reciprocal, so it is off by up to
// 2^-22, and a tie between two codes must stay one.  x has 8 significant bits
// and a tie m * s has 3 + 4, which is 8 bits too: an x that is not the tie is
// at least 2^-8 away from it.  Rounding y to 12 bits therefore restores every
// tie and makes no other value one.
__device__ __forceinline__ uint32_t code_pair(float lo, float hi)
{
    const float l = __uint_as_float((__float_as_uint(lo) + 0x800u) & 0xFFFFF000u);
    const float h = __uint_as_float((__float_as_uint(hi) + 0x800u) & 0xFFFFF000u);
    uint32_t r;
    asm("{\n .reg .b8 b, z;\n .reg .b16 w;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n mov.b16 w, {b, 0};\n"
        " cvt.u32.u16 %0, w;\n}\n"
        : "=r"(r)
        : "f"(h), "f"(l));
    return r;
}

// Four neighbouring lanes hold a row: lane t of them the groups t, t + 4, ...,
// so a warp's loads and stores run along 128-byte pieces of 8 rows, and the
// row's maximum is two shuffles away.  The whole row stays in registers
// between the maximum and the rounding (one read of the input), 288 bytes a
// lane, all requested at once.  Bound by HBM: 131072 rows with values, 346 MB, in
// 53.4 us, 6.5 TB/s (16-byte accesses and streaming hints: 58.8 us); without
// values, 195 MB, in 34.3 us, 5.7 TB/s.
template <bool kWide>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const uint8_t* rows, int64_t stride, int64_t n,
                                                            uint8_t* __restrict__ packed, uint8_t* __restrict__ values)
{
    chain_next();
    chain_wait();
    rows = behind_wait(rows);
    const int64_t row = (int64_t)blockIdx.x * kPackRows + threadIdx.x / kLanesPerRow;
    const int t = threadIdx.x % kLanesPerRow;
    const bool real = row < n;
    const uint8_t* src = rows + (real ? row : n - 1) * stride;
    uint4 x[kLaneGroups][2];
#pragma unroll
    for (int i = 0; i < kLaneGroups; ++i) load32<kWide>(src + 32 * (t + kLanesPerRow * i), x[i][0], x[i][1]);
    // sizes of bf16 values order like their bits; 0x7F80 and above is an infinity or a NaN
    uint32_t top[kLaneGroups], row_top = 0;
#pragma unroll
    for (int i = 0; i < kLaneGroups; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {x[i][c].x, x[i][c].y, x[i][c].z, x[i][c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
        }
        top[i] = max(m & 0xFFFFu, m >> 16);
        if (top[i] < 0x7F80u) row_top = max(row_top, top[i]);
    }
    row_top = max(row_top, __shfl_xor_sync(0xFFFFFFFFu, row_top, 1));
    row_top = max(row_top, __shfl_xor_sync(0xFFFFFFFFu, row_top, 2));
    // row_top = m * 2^E with m in [1, 2): 2688 = 1.3125 * 2^11, and 1.3125 is fraction 40 of 128
    const int e = min(116, max(-100, (int)(row_top >> 7) - 127 - 11 + ((row_top & 127u) > 40u ? 1 : 0)));
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e
    const uint32_t eb = (uint32_t)(e + 127);

    uint32_t tail[12];  // the row's last 48 bytes: 9 words of scales, the exponent, zeros
#pragma unroll
    for (int i = 0; i < kLaneGroups; ++i) {
        const bool bad = top[i] >= 0x7F80u;
        const uint32_t sc = bad ? 0x7Fu : scale_code(__uint_as_float(top[i] << 16) * down);
        const float s = q4::scale_value(sc);
        const float f = bad || sc == 0u ? 0.0f : __frcp_rn(s) * down;
        uint32_t code[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t w[4] = {x[i][c].x, x[i][c].y, x[i][c].z, x[i][c].w};
            code[c] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                code[c] |= code_pair(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xFFFF0000u) * f) << (8 * j);
            if (f == 0.0f) code[c] = 0u;  // nothing to round (and 0 * infinity is not 0)
        }
        const int g = t + kLanesPerRow * i;
        if (real) {
            *reinterpret_cast<uint2*>(packed + row * q4::kRowBytes + 8 * g) = make_uint2(code[0], code[1]);
            if (values) {
                const uint32_t factor = q4::group_factor(sc, eb);
                store32<kWide>(values + row * (2 * q4::kDim) + 32 * g, q4::decode8(code[0], factor), q4::decode8(code[1], factor));
            }
        }
        uint32_t word = sc << (8 * t);  // scales of the groups 4i .. 4i + 3
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
        tail[i] = word | __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    }
    tail[9] = eb;
    tail[10] = tail[11] = 0u;
    if (real && t < 3) {
        uint4 w = make_uint4(tail[0], tail[1], tail[2], tail[3]);
        if (t == 1) w = make_uint4(tail[4], tail[5], tail[6], tail[7]);
        if (t == 2) w = make_uint4(tail[8], tail[9], tail[10], tail[11]);
        reinterpret_cast<uint4*>(packed + row * q4::kRowBytes + q4::kScalesAt)[t] = w;
    }
}

constexpr int kUnpackThreads = 256;

// One thread per group of 16 values: 8 bytes of codes in, 32 bytes out, both
// contiguous across a warp; the exponent comes out of L1.  Bound by HBM: 131072
// rows, 195 MB, in 29.1 us, 6.7 TB/s (8 values a thread and 16-byte stores: 34.2 us;
// two or four groups a thread: 29.8 and 31.0).
template <bool kWide>
__global__ void __launch_bounds__(kUnpackThreads) unpack_kernel(const uint8_t* packed, int64_t n,
                                                                uint8_t* __restrict__ values)
{
    chain_next();
    chain_wait();
    packed = behind_wait(packed);
    const int64_t at = (int64_t)blockIdx.x * kUnpackThreads + threadIdx.x;
    if (at >= n * q4::kGroups) return;
    const int64_t row = at / q4::kGroups;
    const int g = (int)(at - row * q4::kGroups);
    const uint8_t* p = packed + row * q4::kRowBytes;
    const uint2 code = *reinterpret_cast<const uint2*>(p + 8 * g);
    const uint32_t factor = q4::group_factor(p[q4::kScalesAt + g], p[q4::kExpAt]);
    store32<kWide>(values + at * 32, q4::decode8(code.x, factor), q4::decode8(code.y, factor));
}

}  // namespace

// Whether 32-byte accesses are aligned.
static bool wide(const void* a, const void* b, int64_t stride)
{
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | (uintptr_t)stride) & 31u) == 0;
}

cudaError_t launch_pack_rows(const void* rows, int64_t stride, int64_t n, void* packed, void* values, cudaStream_t st)
{
    return launch_chained(wide(rows, values, stride) ? pack_kernel<true> : pack_kernel<false>,
                          dim3((unsigned)((n + kPackRows - 1) / kPackRows)), kPackThreads, 0, st,
                          static_cast<const uint8_t*>(rows), stride, n, static_cast<uint8_t*>(packed),
                          static_cast<uint8_t*>(values));
}

cudaError_t launch_unpack_rows(const void* packed, int64_t n, void* values, cudaStream_t st)
{
    return launch_chained(wide(nullptr, values, 0) ? unpack_kernel<true> : unpack_kernel<false>,
                          dim3((unsigned)((n * q4::kGroups + kUnpackThreads - 1) / kUnpackThreads)), kUnpackThreads, 0, st,
                          static_cast<const uint8_t*>(packed), n, static_cast<uint8_t*>(values));
}

}  // namespace skv
