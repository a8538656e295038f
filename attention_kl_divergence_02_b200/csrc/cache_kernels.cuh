// cache_kernels.cuh -- rows written to a paged key-value cache, and read back.
//
// e4m3 row: with a = max_i |x_i| over the finite elements, the scale is 2^e, e the least integer of
// at least -96 with a <= 448 * 2^e; the codes are x_i * 2^-e rounded to nearest even, infinities
// at +-448, NaN kept (at e = 120, the largest, codes end at 240: 256 * 2^120 is no bf16 number).
// A power of two makes the scaling exact in both directions and costs one byte;
// against a free scale it wastes less than one bit of e4m3's exponent range and none of its
// mantissa.  2^-96 keeps scale, inverse and every code's value normal in fp32 and bf16.
// Reading back is exact: 4 significant bits fit bf16.
//
// Bound: memory.  Of the rows that a warp holds at a time, one half are keys and the other half the same
// tokens' values, so the pool rows are looked up once for both, by one lane per token, before the loads; a warp
// does kCacheTurns such turns, all of whose loads are in flight together.  A lane takes 16 contiguous
// bytes of the side that is written: 16 elements of a row to be quantised, 8 of one to be read back
// (there, 16 elements would be two stores of half a sector each: 81 us instead of 69 for 32 heads of
// 16384 rows of d = 128; quantising them takes 66, 93 % of measured HBM, and 63 with read-only loads, which
// an early launch rules out: see wait_for_stream).
#pragma once

#include "paged.cuh"

namespace skl {

constexpr int kCacheThreads = 128;
constexpr int kCacheTurns = 4;

template <int D, int ELEMS>
struct CacheCfg {
    static constexpr int kElems = ELEMS;                  // of a lane
    static constexpr int kLoads = kElems / 8;             // 16-byte loads of its dense part
    static constexpr int kLanes = D / kElems;             // of a row
    static constexpr int kGroups = 32 / kLanes;           // rows at a time
    static constexpr int kTokens = kGroups / 2 * kCacheTurns;   // of a warp
    static_assert(kLanes >= kCacheTurns, "a row's lanes keep the exponents of their turns");
};

struct CacheParams {
    uint8_t* rows[2];              // key and value pages
    uint8_t* exps[2];              // nullptr for bf16
    uint16_t* dense[2];            // [B, Hkv, NT, d]
    const int* table;              // [B, width]
    const int* start;              // [B] or nullptr: 0
    const int* count;              // [B] or nullptr: NT
    int B, Hkv, NT, width, pages, page_size, page_shift;
};

// The pool row of token i of sequence b, head h; -1 where there is nothing to do (behind the count)
// or nothing that exists (recorded).
__device__ __forceinline__ int cache_row(const CacheParams& p, int b, int h, int i) {
    const int n = p.count ? p.count[b] : p.NT, s = p.start ? p.start[b] : 0;
    if (i >= n || i >= p.NT) return -1;
    const unsigned pos = (unsigned)s + (unsigned)i;       // s, i < 2^31: no wrap for s >= 0
    if (s >= 0 && pos < (unsigned)p.width * (unsigned)p.page_size) {
        const int page = p.table[(size_t)b * p.width + (pos >> p.page_shift)];
        if ((unsigned)page < (unsigned)p.pages) return (page * p.Hkv + h) * p.page_size + (pos & (p.page_size - 1));
    }
    g_page_status = 5;
    return -1;
}

// The exponent byte of a row whose largest finite magnitude has these bf16 bits: a = f * 2^x,
// 448 = 1.75 * 2^8.  A subnormal a has exponent field 0, below the floor all the same.
__device__ __forceinline__ uint32_t row_exponent(uint32_t bits) {
    const int e = (int)(bits >> 7) - 8 + ((bits & 0x7fu) > 0x60u ? 1 : 0);
    return (uint32_t)max(e, 127 - 96);
}

// Two fp32 to two e4m3 codes (lo in the low byte), to nearest even, beyond 448 at 448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}

// The larger magnitude of two bf16, as bits, infinities and NaN as 0 where FINITE.
template <bool FINITE>
__device__ __forceinline__ uint32_t top_bits(uint32_t x) {
    uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
    if (FINITE) {
        lo = lo >= 0x7f80u ? 0u : lo;
        hi = hi >= 0x7f80u ? 0u : hi;
    }
    return max(lo, hi);
}

template <bool FINITE>
__device__ __forceinline__ uint32_t top_bits4(uint4 x) {
    return max(max(top_bits<FINITE>(x.x), top_bits<FINITE>(x.y)), max(top_bits<FINITE>(x.z), top_bits<FINITE>(x.w)));
}

template <int D, bool F8>
__global__ void __launch_bounds__(kCacheThreads) streamkl_cache_append_kernel(const CacheParams p) {
    using C = CacheCfg<D, F8 ? 16 : 8>;
    const int lane = threadIdx.x & 31, c = lane % C::kLanes, pool = (lane / C::kLanes) & 1, sub = lane / C::kLanes / 2;
    const int groups = (p.NT + C::kTokens - 1) / C::kTokens;
    const unsigned w = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
    const int bh = w / (unsigned)groups, i0 = (w % (unsigned)groups) * C::kTokens;
    wait_for_stream();
    if (bh >= p.B * p.Hkv) return;
    const int mine = lane < C::kTokens ? cache_row(p, bh / p.Hkv, bh % p.Hkv, i0 + lane) : -1;
    const uint16_t* dense = (pool ? p.dense[1] : p.dense[0]) + ((size_t)bh * p.NT + i0) * D + c * C::kElems;
    uint8_t* rows = pool ? p.rows[1] : p.rows[0];
    int row[kCacheTurns];
    uint4 x[kCacheTurns][C::kLoads];
#pragma unroll
    for (int r = 0; r < kCacheTurns; ++r) {
        const int i = r * (C::kGroups / 2) + sub;
        row[r] = __shfl_sync(0xffffffffu, mine, i);
#pragma unroll
        for (int k = 0; k < C::kLoads; ++k) {
            x[r][k] = make_uint4(0, 0, 0, 0);
            if (row[r] >= 0) x[r][k] = reinterpret_cast<const uint4*>(dense + (size_t)i * D)[k];
        }
    }
    if (!F8) {
#pragma unroll
        for (int r = 0; r < kCacheTurns; ++r)
            if (row[r] >= 0) *reinterpret_cast<uint4*>(rows + (size_t)row[r] * D * 2 + c * 16) = x[r][0];
        return;
    }
    uint32_t exponent = 0;                                // lane c keeps that of turn c
    int exponent_row = -1;
#pragma unroll
    for (int r = 0; r < kCacheTurns; ++r) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < C::kLoads; ++k) top = max(top, top_bits4<false>(x[r][k]));
#pragma unroll
        for (int d = C::kLanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        if (__any_sync(0xffffffffu, top >= 0x7f80u)) {
            top = 0;
#pragma unroll
            for (int k = 0; k < C::kLoads; ++k) top = max(top, top_bits4<true>(x[r][k]));
#pragma unroll
            for (int d = C::kLanes / 2; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        }
        const uint32_t e = row_exponent(top);
        const float inv = exp_scale(254u - e);            // 2^-(e - 127)
        uint32_t y[2 * C::kLoads];
#pragma unroll
        for (int k = 0; k < C::kLoads; ++k) {
            const uint32_t v[4] = {x[r][k].x, x[r][k].y, x[r][k].z, x[r][k].w};
            uint32_t z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo = bf16_lo(v[i]) * inv, hi = bf16_hi(v[i]) * inv;
                if (e == 247) {          // 256 * 2^120 would be infinite: the last scale ends at 240
                    if (fabsf(lo) > 240.f) lo = copysignf(240.f, lo);
                    if (fabsf(hi) > 240.f) hi = copysignf(240.f, hi);
                }
                z[i] = e4m3x2(lo, hi);
            }
            y[2 * k] = z[0] | z[1] << 16;
            y[2 * k + 1] = z[2] | z[3] << 16;
        }
        if (row[r] >= 0) *reinterpret_cast<uint4*>(rows + (size_t)row[r] * D + c * 16) = make_uint4(y[0], y[1], y[C::kLoads], y[2 * C::kLoads - 1]);
        if (c == r) {
            exponent = e;
            exponent_row = row[r];
        }
    }
    if (exponent_row >= 0) (pool ? p.exps[1] : p.exps[0])[exponent_row] = (uint8_t)exponent;
}

template <int D, bool F8>
__global__ void __launch_bounds__(kCacheThreads) streamkl_cache_gather_kernel(const CacheParams p) {
    using C = CacheCfg<D, 8>;
    const int lane = threadIdx.x & 31, c = lane % C::kLanes, pool = (lane / C::kLanes) & 1, sub = lane / C::kLanes / 2;
    const int groups = (p.NT + C::kTokens - 1) / C::kTokens;
    const unsigned w = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
    const int bh = w / (unsigned)groups, i0 = (w % (unsigned)groups) * C::kTokens;
    wait_for_stream();
    if (bh >= p.B * p.Hkv) return;
    const int mine = lane < C::kTokens ? cache_row(p, bh / p.Hkv, bh % p.Hkv, i0 + lane) : -1;
    uint16_t* dense = (pool ? p.dense[1] : p.dense[0]) + ((size_t)bh * p.NT + i0) * D + c * C::kElems;
    const uint8_t* rows = pool ? p.rows[1] : p.rows[0];
    int row[kCacheTurns];
    uint4 x[kCacheTurns];
    uint32_t exponent = 0;
#pragma unroll
    for (int r = 0; r < kCacheTurns; ++r) {
        row[r] = __shfl_sync(0xffffffffu, mine, r * (C::kGroups / 2) + sub);
        x[r] = make_uint4(0, 0, 0, 0);
        if (row[r] < 0) continue;
        if (F8) {
            const uint2 v = *reinterpret_cast<const uint2*>(rows + (size_t)row[r] * D + c * 8);
            x[r].x = v.x;
            x[r].y = v.y;
            if (c == r) exponent = (pool ? p.exps[1] : p.exps[0])[row[r]];
        } else {
            x[r] = *reinterpret_cast<const uint4*>(rows + (size_t)row[r] * D * 2 + c * 16);
        }
    }
#pragma unroll
    for (int r = 0; r < kCacheTurns; ++r) {
        uint4 y = x[r];
        if (F8) {
            const float s = exp_scale(__shfl_sync(0xffffffffu, exponent, r, C::kLanes));
            uint32_t h[4];
            e4m3x4_half2(x[r].x, h[0], h[1]);
            e4m3x4_half2(x[r].y, h[2], h[3]);
            const float2 v0 = half2_floats(h[0]), v1 = half2_floats(h[1]), v2 = half2_floats(h[2]), v3 = half2_floats(h[3]);
            y = make_uint4(bf16_pair(v0.x * s, v0.y * s), bf16_pair(v1.x * s, v1.y * s), bf16_pair(v2.x * s, v2.y * s),
                           bf16_pair(v3.x * s, v3.y * s));
        }
        if (row[r] >= 0) *reinterpret_cast<uint4*>(dense + (size_t)(r * (C::kGroups / 2) + sub) * D) = y;
    }
}

}  // namespace skl
