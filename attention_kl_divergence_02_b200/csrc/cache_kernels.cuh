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
// Bound: memory.  Half a warp takes a key row and the other half the same token's value row (16
// lanes x 8 elements at d = 128), so both share the page lookup; each warp takes 4 tokens of one
// head at once, whose loads are independent.
#pragma once

#include "paged.cuh"

namespace skl {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 4;      // tokens of a warp

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
__device__ __forceinline__ long long cache_row(const CacheParams& p, int b, int h, int i) {
    if (p.count && i >= p.count[b]) return -1;
    const int s = p.start ? p.start[b] : 0;
    const long long pos = (long long)s + i;
    if (s >= 0 && pos < (long long)p.width * p.page_size) {
        const int page = p.table[(size_t)b * p.width + (pos >> p.page_shift)];
        if ((unsigned)page < (unsigned)p.pages)
            return ((long long)page * p.Hkv + h) * p.page_size + (pos & (p.page_size - 1));
    }
    g_page_status = 5;
    return -1;
}

// The exponent byte of a row whose largest finite magnitude is a.
__device__ __forceinline__ uint32_t row_exponent(float a) {
    const uint32_t bits = __float_as_uint(a);
    // a = f * 2^x; 448 = 1.75 * 2^8.  A subnormal a has x = -127 here, below the floor all the same.
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(max(e, -96) + 127);
}

// Two fp32 to two e4m3 codes (lo in the low byte), to nearest even, beyond 448 at 448, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}

template <int D, bool F8>
__global__ void __launch_bounds__(kCacheThreads) streamkl_cache_append_kernel(const CacheParams p) {
    constexpr int kElems = D / 16;                        // of a lane: 8 or 4
    constexpr int kWords = kElems / 2;
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    const int groups = (p.NT + kCacheRows - 1) / kCacheRows;
    const long long all = (long long)p.B * p.Hkv * groups;
    const long long step = (long long)gridDim.x * (kCacheThreads / 32);
    for (long long w = (long long)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5); w < all; w += step) {
        const int bh = (int)(w / groups), i0 = (int)(w % groups) * kCacheRows;
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        long long row[kCacheRows];
        uint32_t x[kCacheRows][kWords];
#pragma unroll
        for (int r = 0; r < kCacheRows; ++r) {
            row[r] = i0 + r < p.NT ? cache_row(p, b, h, i0 + r) : -1;
            const uint16_t* from = p.dense[half] + ((size_t)bh * p.NT + i0 + r) * D + c * kElems;
#pragma unroll
            for (int k = 0; k < kWords; ++k) x[r][k] = 0;
            if (row[r] >= 0) {
                if (kWords == 4) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
                    x[r][0] = v.x; x[r][1] = v.y; x[r][kWords - 2] = v.z; x[r][kWords - 1] = v.w;
                } else {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(from));
                    x[r][0] = v.x; x[r][1] = v.y;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kCacheRows; ++r) {
            if (row[r] < 0) continue;                     // the same in every lane
            if (!F8) {
                uint8_t* to = p.rows[half] + (size_t)row[r] * D * 2 + c * kElems * 2;
                if (kWords == 4)
                    *reinterpret_cast<uint4*>(to) = make_uint4(x[r][0], x[r][1], x[r][kWords - 2], x[r][kWords - 1]);
                else
                    *reinterpret_cast<uint2*>(to) = make_uint2(x[r][0], x[r][1]);
                continue;
            }
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < kWords; ++k) top = fmaxf(top, fmaxf(finite_abs(x[r][k]), finite_abs(x[r][k] >> 16)));
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const uint32_t e = row_exponent(top);
            const float inv = exp_scale(254u - e);        // 2^-(e - 127)
            uint32_t y[kWords];
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                float lo = bf16_lo(x[r][k]) * inv, hi = bf16_hi(x[r][k]) * inv;
                if (e == 247) {          // 256 * 2^120 would be infinite: the last scale ends at 240
                    if (fabsf(lo) > 240.f) lo = copysignf(240.f, lo);
                    if (fabsf(hi) > 240.f) hi = copysignf(240.f, hi);
                }
                y[k] = e4m3x2(lo, hi);
            }
            uint8_t* to = p.rows[half] + (size_t)row[r] * D + c * kElems;
            if (kWords == 4)
                *reinterpret_cast<uint2*>(to) = make_uint2(y[0] | y[1] << 16, y[kWords - 2] | y[kWords - 1] << 16);
            else
                *reinterpret_cast<uint32_t*>(to) = y[0] | y[1] << 16;
            if (c == 0) p.exps[half][row[r]] = (uint8_t)e;
        }
    }
}

template <int D, bool F8>
__global__ void __launch_bounds__(kCacheThreads) streamkl_cache_gather_kernel(const CacheParams p) {
    constexpr int kElems = D / 16;
    constexpr int kWords = kElems / 2;
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    const int groups = (p.NT + kCacheRows - 1) / kCacheRows;
    const long long all = (long long)p.B * p.Hkv * groups;
    const long long step = (long long)gridDim.x * (kCacheThreads / 32);
    for (long long w = (long long)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5); w < all; w += step) {
        const int bh = (int)(w / groups), i0 = (int)(w % groups) * kCacheRows;
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        long long row[kCacheRows];
        uint32_t x[kCacheRows][kWords], e[kCacheRows];
#pragma unroll
        for (int r = 0; r < kCacheRows; ++r) {
            row[r] = i0 + r < p.NT ? cache_row(p, b, h, i0 + r) : -1;
            if (row[r] < 0) continue;
            const uint8_t* from = p.rows[half] + (size_t)row[r] * D * (F8 ? 1 : 2) + c * kElems * (F8 ? 1 : 2);
            if (F8) {
                e[r] = p.exps[half][row[r]];
                if (kWords == 4) {
                    const uint2 v = *reinterpret_cast<const uint2*>(from);
                    x[r][0] = v.x; x[r][1] = v.y;
                } else {
                    x[r][0] = *reinterpret_cast<const uint32_t*>(from);
                }
            } else if (kWords == 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(from);
                x[r][0] = v.x; x[r][1] = v.y; x[r][kWords - 2] = v.z; x[r][kWords - 1] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(from);
                x[r][0] = v.x; x[r][1] = v.y;
            }
        }
#pragma unroll
        for (int r = 0; r < kCacheRows; ++r) {
            if (row[r] < 0) continue;
            uint32_t y[kWords];
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                if (F8) {
                    const float s = exp_scale(e[r]);
                    const float2 v = half2_floats(e4m3x2_half2(x[r][k >> 1] >> (16 * (k & 1))));
                    y[k] = bf16_pair(v.x * s, v.y * s);
                } else {
                    y[k] = x[r][k];
                }
            }
            uint16_t* to = p.dense[half] + ((size_t)bh * p.NT + i0 + r) * D + c * kElems;
            if (kWords == 4)
                *reinterpret_cast<uint4*>(to) = make_uint4(y[0], y[1], y[kWords - 2], y[kWords - 1]);
            else
                *reinterpret_cast<uint2*>(to) = make_uint2(y[0], y[1]);
        }
    }
}

}  // namespace skl
