// paged_attn_kernel.cuh -- attention of a few new tokens over a paged key-value cache.
//
//     s_j = scale <q, k_j>,   o = sum_j exp(s_j - lse) v_j,   lse = log sum_j exp(s_j)
//
// over the keys j that the row sees, in one pass: running maximum m, sum l and weighted sum o are
// rescaled by 2^(m_old - m_new) when the maximum grows.
//
// Bound: every cached byte is read once and used for 2 flops per query row and element, so with the
// few rows of a KV head (Hq / Hkv * NQ) the floor is cache bytes / HBM bandwidth.  Everything here
// serves the loads: each warp streams its own 16-key tiles through a ring of cp.async stages that
// only it touches (see KeyTile), so no barrier stands between a load and the next.
//
// Per tile a warp computes S^T = K Q^T (16 keys x 8 rows per product), takes the maxima over the
// lanes that share a row, and turns P^T around with movmatrix into the B operand of
// O^T = V^T P^T (M: 16 columns of d, N: 8 rows, K: 16 keys).  V^T's fragments need two keys'
// values of one column in a register: the lane copies the same 16 bytes of four keys and joins
// them with byte permutes.
//
// bf16 cache: P is split into two bf16 terms (hi + lo, 16 bits of it), because one bf16 rounding of P
// (up to 2^-9 of each weight) would add as much error as the output's own rounding; the tensor pipe
// has room for the second product.
// e4m3 cache: values are met as fp16 (exact) without their scales 2^e_j; those go into the weights,
// P'_j = 2^(s_j + e_j - m'), with a running maximum m' of s_j + e_j, so that P' <= 1 whatever the
// scales are; fp16 keeps 11 bits of it (error 2^-12), which is below the output's rounding.  l keeps its
// own maximum m of s_j.
#pragma once

#include "paged.cuh"

namespace skl {

template <int D, bool F8>
struct ValueTile {
    static constexpr int kRow = D * (F8 ? 1 : 2);
    static constexpr int kLane = kRow / 8;                      // bytes of a row per lane
    static constexpr int kCopy = kLane < 16 ? kLane : 16;       // bytes of one copy
    static constexpr int kChunks = kLane / kCopy;
    static constexpr int kElems = kCopy / (F8 ? 1 : 2);         // elements of a copy
    static constexpr int kBytes = kTileKeys * kRow;

    // lane (g, t): chunk g (and g + 8 where a row has 16) of keys 2t, 2t+1, 2t+8, 2t+9
    __device__ static __forceinline__ int key(int j, int t) { return 2 * t + (j & 1) + 8 * (j >> 1); }

    __device__ static __forceinline__ void copy(uint32_t dst, const uint8_t* rows, int valid, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = key(j, t) < valid;
#pragma unroll
            for (int u = 0; u < kChunks; ++u) {
                const uint32_t to = dst + (j * kChunks + u) * 32 * kCopy + lane * kCopy;
                const uint8_t* from = rows + key(j, t) * kRow + (u * 8 + g) * kCopy;
                if (kCopy == 16) cp_async16(to, from, in ? 16 : 0);
                else cp_async8(to, from, in ? 8 : 0);
            }
        }
    }
    // the lane's words (4 bytes) of key j, chunk u
    __device__ static __forceinline__ void load(uint32_t src, int j, int u, int lane, uint32_t* w) {
        const uint32_t from = src + (j * kChunks + u) * 32 * kCopy + lane * kCopy;
        if (kCopy == 16) {
            const uint4 v = lds128(from);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
            const uint2 v = lds64(from);
            w[0] = v.x; w[1] = v.y;
        }
    }
};

template <int D, bool F8, int NT>
struct AttnCfg {
    using K = KeyTile<D, F8>;
    using V = ValueTile<D, F8>;
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = D / 16;
    static constexpr int kExps = F8 ? 32 : 0;                          // 16 key, 16 value exponents
    static constexpr int kStage = K::kBytes + V::kBytes + kExps;
    static constexpr int kStages = (D == 128 && !F8) ? 3 : (D == 64 && F8) ? 8 : 6;
    static constexpr int kWarp = kStage * kStages;
    static constexpr int kStride = D + 4;                              // floats of a row's state
    static constexpr bool kSharedQ = NT > 2;                           // query fragments in shared memory
    static constexpr int kQ = kPagedWarps * kWarp;
    static constexpr int kFactor = kQ + (kSharedQ ? NT * kSteps * 32 * 8 : 0);
    static constexpr int kStats = kFactor + (kSharedQ ? NT * 32 * 4 : 0);   // [warp][3][kRows]
    static constexpr int kRed = kStats + kPagedWarps * 3 * kRows * 4;
    static constexpr int kSmem = kRed + 64;
    static constexpr int kPart = kRows * kStride;                      // floats of a partial state
    static_assert(kWarp >= kRows * kStride * 4, "a warp's state is joined in its stages");
};

// Four columns of a finished row: o / l, rounded once to bf16, and the row's lse.  Weights that refer to
// m' = MV come back to m = M by 2^(MV - M), after the division so that nothing overflows
// that the result does not.  A row without keys (l = 0): zeros and -inf.
template <int D>
__device__ __forceinline__ void attn_finish(const PagedParams& p, size_t row, int c, float4 acc, float M, float MV, float L) {
    const bool none = L == 0.f;
    const float inv = none ? 0.f : 1.f / L, f = none ? 0.f : exp2f(MV - M);
    uint2 y;
    y.x = none ? 0u : bf16_pair(acc.x * inv * f, acc.y * inv * f);
    y.y = none ? 0u : bf16_pair(acc.z * inv * f, acc.w * inv * f);
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * c) = y;
    if (c == 0) p.lse1[row] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <int D, bool F8, int NT>
__global__ void __launch_bounds__(kPagedThreads, 2) streamkl_paged_attn_kernel(const PagedParams p) {
    using C = AttnCfg<D, F8, NT>;
    using K = typename C::K;
    using V = typename C::V;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t sb = smem_u32(smem);
    const uint32_t stage0 = sb + warp * C::kWarp;
    float* stats = reinterpret_cast<float*>(smem + C::kStats);
    int* red = reinterpret_cast<int*>(smem + C::kRed);
    const int head_stride = p.page_size * K::kRow;       // bytes of one page of one head

    // sequences without keys: zeros and -inf
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (threadIdx.x == 0 && (p.lengths[b] < 0 || p.lengths[b] > p.width * p.page_size)) g_page_status = 5;
        if (seq_len(p, b) > 0) continue;
        const size_t r0 = (size_t)b * p.Hkv * p.rows, n = (size_t)p.Hkv * p.rows;
        for (size_t i = threadIdx.x; i < n * (D / 8); i += kPagedThreads)
            reinterpret_cast<uint4*>(p.out + r0 * D)[i] = make_uint4(0, 0, 0, 0);
        for (size_t i = threadIdx.x; i < n; i += kPagedThreads) p.lse1[r0 + i] = -INFINITY;
    }

    const int total = plan_total(p, red);
    const int share = plan_share(p, total);
    const long long first = (long long)blockIdx.x * share;
    if (first >= total) return;
    const int g0 = (int)first, g1 = (int)min((long long)total, first + share);
    int b, base;
    plan_locate(p, g0, red, b, base);
    int len = seq_len(p, b), units = (len + kUnitKeys - 1) / kUnitKeys;

    for (int pos = g0; pos < g1;) {
        const int off = pos - base, seg = off / units, u0 = off - seg * units;
        const int n = min(units - u0, g1 - pos);          // units, hence tiles of a warp
        const int h = seg / p.rblocks, rb = seg - h * p.rblocks;
        const int row0 = rb * C::kRows;
        const size_t qrow = ((size_t)b * p.Hkv + h) * p.rows;
        const int* table = p.table + (size_t)b * p.width;
        const int key00 = u0 * kUnitKeys + warp * kTileKeys;
        uint32_t bad = 0;                                 // stages whose page does not exist

        auto issue = [&](int i, int s) {
            const int key0 = key00 + i * kUnitKeys;
            const uint32_t dst = stage0 + s * C::kStage;
            bad &= ~(1u << s);
            if (key0 < len) {
                const int page = __ldg(table + (key0 >> p.page_shift));
                if ((unsigned)page < (unsigned)p.pages) {
                    const size_t row = ((size_t)page * p.Hkv + h) * p.page_size + (key0 & (p.page_size - 1));
                    const int valid = len - key0;
                    K::copy(dst, p.a.rows + row * K::kRow, valid, lane);
                    V::copy(dst + K::kBytes, p.b.rows + row * V::kRow, valid, lane);
                    if (F8 && lane < 2)
                        cp_async16(dst + K::kBytes + V::kBytes + lane * 16, (lane ? p.b.exps : p.a.exps) + row, 16);
                } else {
                    bad |= 1u << s;
                    if (lane == 0) g_page_status = 5;
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int s = 0; s < C::kStages - 1; ++s) {
            if (s < n) issue(s, s);
            else cp_commit();
        }

        // queries of this segment, as B fragments
        uint2 qf[C::kSharedQ ? 1 : NT * C::kSteps];
        float fac[NT][2];
        if (C::kSharedQ) {
            uint2 f[C::kSteps];
            float one;
            load_queries<D, F8>(p.q1 + qrow * D, row0 + 8 * warp, p.rows, p.sl2, f, one);
            if (warp < NT) {
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s)
                    reinterpret_cast<uint2*>(smem + C::kQ)[(warp * C::kSteps + s) * 32 + lane] = f[s];
                if (t == 0) reinterpret_cast<float*>(smem + C::kFactor)[warp * 8 + g] = one;
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                fac[nt][0] = reinterpret_cast<float*>(smem + C::kFactor)[nt * 8 + 2 * t];
                fac[nt][1] = reinterpret_cast<float*>(smem + C::kFactor)[nt * 8 + 2 * t + 1];
            }
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float one;
                load_queries<D, F8>(p.q1 + qrow * D, row0 + 8 * nt, p.rows, p.sl2, qf + nt * C::kSteps, one);
                fac[nt][0] = __shfl_sync(0xffffffffu, one, 8 * t);
                fac[nt][1] = __shfl_sync(0xffffffffu, one, 8 * t + 4);
            }
        }
        // first key that a row does not see; the least over all rows
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                lim[nt][j] = p.causal ? len - (p.NQ - 1) + (row0 + nt * 8 + 2 * t + j) % p.NQ : len;
        const int least = p.causal ? len - (p.NQ - 1) : len;

        float o[D / 16][NT][4], m[NT][2], mv[NT][2], l[NT][2];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = mv[nt][j] = kNoMax;
                l[nt][j] = 0.f;
            }

        int st = 0;
        for (int i = 0; i < n; ++i, st = st + 1 == C::kStages ? 0 : st + 1) {
            __syncwarp();       // every lane is done with the stage that is filled next
            if (i + C::kStages - 1 < n) issue(i + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
            else cp_commit();
            cp_wait<C::kStages - 1>();
            __syncwarp();       // the exponents were copied by lanes 0 and 1
            const int key0 = key00 + i * kUnitKeys;
            if (key0 >= len || ((bad >> st) & 1u)) continue;
            const uint32_t ks = stage0 + st * C::kStage, vs = ks + K::kBytes, es = vs + V::kBytes;

            // S^T
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
            for (int u = 0; u < K::kChunks; ++u) {
                const uint4 x = lds128(ks + u * 512 + lane * 16), y = lds128(ks + (K::kChunks + u) * 512 + lane * 16);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int w = 0; w < K::kSteps; ++w) {
                    uint32_t a0, a1, a2, a3;
                    if (F8) {
                        a0 = e4m3x2_half2(xw[w]);
                        a1 = e4m3x2_half2(yw[w]);
                        a2 = e4m3x2_half2(xw[w] >> 16);
                        a3 = e4m3x2_half2(yw[w] >> 16);
                    } else {
                        a0 = xw[(2 * w) & 3];
                        a1 = yw[(2 * w) & 3];
                        a2 = xw[(2 * w + 1) & 3];
                        a3 = yw[(2 * w + 1) & 3];
                    }
                    const int step = u * K::kSteps + w;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint2 q = C::kSharedQ ? lds64(sb + C::kQ + ((nt * C::kSteps + step) * 32 + lane) * 8)
                                                    : qf[C::kSharedQ ? 0 : nt * C::kSteps + step];
                        mma16816<F8>(s[nt], a0, a1, a2, a3, q.x, q.y);
                    }
                }
            }
            // scores in base 2; ev: exponents of the values' scales
            float ev[2] = {0.f, 0.f};
            if (F8) {
                const float k0 = exp_scale(lds8(es + g)), k1 = exp_scale(lds8(es + 8 + g));
                ev[0] = (float)((int)lds8(es + 16 + g) - 127);
                ev[1] = (float)((int)lds8(es + 24 + g) - 127);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    s[nt][0] = s[nt][0] * fac[nt][0] * k0;
                    s[nt][1] = s[nt][1] * fac[nt][1] * k0;
                    s[nt][2] = s[nt][2] * fac[nt][0] * k1;
                    s[nt][3] = s[nt][3] * fac[nt][1] * k1;
                }
            } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[nt][c] *= fac[nt][c & 1];
            }
            const bool edge = key0 + kTileKeys > least;
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (key0 + g + 8 * (c >> 1) >= lim[nt][c & 1]) s[nt][c] = -INFINITY;
            }
            // maxima over the tile's keys (the 8 lanes with this t), rescaling, weights
            uint32_t ph[NT][2], pl[NT][2];      // B fragments of P^T: hi and lo (bf16), or P' (fp16)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = fmaxf(s[nt][j], s[nt][j + 2]);
                    float topv = F8 ? fmaxf(s[nt][j] + ev[0], s[nt][j + 2] + ev[1]) : 0.f;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                        if (F8) topv = fmaxf(topv, __shfl_xor_sync(0xffffffffu, topv, d));
                    }
                    const float mn = fmaxf(m[nt][j], top);
                    const float a = ex2(m[nt][j] - mn);
                    m[nt][j] = mn;
                    const float p0 = ex2(s[nt][j] - mn), p1 = ex2(s[nt][j + 2] - mn);
                    l[nt][j] = fmaf(l[nt][j], a, p0 + p1);
                    float av = a;
                    if (F8) {
                        const float vn = fmaxf(mv[nt][j], topv);
                        av = ex2(mv[nt][j] - vn);
                        mv[nt][j] = vn;
                        w[j] = ex2(s[nt][j] + ev[0] - vn);
                        w[j + 2] = ex2(s[nt][j + 2] + ev[1] - vn);
                    } else {
                        w[j] = p0;
                        w[j + 2] = p1;
                    }
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        o[k][nt][j] *= av;
                        o[k][nt][j + 2] *= av;
                    }
                }
                if (F8) {
                    ph[nt][0] = movmatrix(pack_half(w[0], w[1]));
                    ph[nt][1] = movmatrix(pack_half(w[2], w[3]));
                } else {
                    const uint32_t h0 = bf16_pair(w[0], w[1]), h1 = bf16_pair(w[2], w[3]);
                    ph[nt][0] = movmatrix(h0);
                    ph[nt][1] = movmatrix(h1);
                    pl[nt][0] = movmatrix(bf16_pair(w[0] - bf16_lo(h0), w[1] - bf16_hi(h0)));
                    pl[nt][1] = movmatrix(bf16_pair(w[2] - bf16_lo(h1), w[3] - bf16_hi(h1)));
                }
            }
            // O^T += V^T P^T
            uint32_t v[V::kChunks][4][4];
#pragma unroll
            for (int u = 0; u < V::kChunks; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) V::load(vs, j, u, lane, v[u][j]);
            // A row that does not see a key must not meet its values even with weight 0 (0 * inf and
            // 0 * NaN are NaN): where such a tile holds values that are not finite, each query
            // position is done by itself with the keys behind its limit cleared.
            bool slow = false;
            if (edge && least < len) {
                bool odd = false;
#pragma unroll
                for (int u = 0; u < V::kChunks; ++u)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int w = 0; w < V::kCopy / 4; ++w)
#pragma unroll
                            for (int e = 0; e < 32; e += F8 ? 8 : 16)
                                odd |= F8 ? ((v[u][j][w] >> e) & 0x7fu) == 0x7fu
                                          : ((v[u][j][w] >> e) & 0x7f80u) == 0x7f80u;
                slow = __any_sync(0xffffffffu, odd);
            }
            auto fragment = [&](int mt, uint32_t* a, const uint32_t* mask) {
                // m-tile mt: columns 2x, 2x + 1 of the lane's elements of chunk u
                const int u = mt / (V::kElems / 2), x = mt % (V::kElems / 2);
                const int w = F8 ? x >> 1 : x;
                const uint32_t k0 = v[u][0][w] & mask[0], k1 = v[u][1][w] & mask[1];
                const uint32_t k2 = v[u][2][w] & mask[2], k3 = v[u][3][w] & mask[3];
                if (F8) {
                    const uint32_t sel = (x & 1) ? 0x7362u : 0x5140u;
                    const uint32_t lo = __byte_perm(k0, k1, sel), hi = __byte_perm(k2, k3, sel);
                    a[0] = e4m3x2_half2(lo);
                    a[1] = e4m3x2_half2(lo >> 16);
                    a[2] = e4m3x2_half2(hi);
                    a[3] = e4m3x2_half2(hi >> 16);
                } else {
                    a[0] = __byte_perm(k0, k1, 0x5410);
                    a[1] = __byte_perm(k0, k1, 0x7632);
                    a[2] = __byte_perm(k2, k3, 0x5410);
                    a[3] = __byte_perm(k2, k3, 0x7632);
                }
            };
            if (!slow) {
                const uint32_t all[4] = {~0u, ~0u, ~0u, ~0u};
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    uint32_t a[4];
                    fragment(mt, a, all);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816<F8>(o[mt][nt], a[0], a[1], a[2], a[3], ph[nt][0], ph[nt][1]);
                        if (!F8) mma16816<F8>(o[mt][nt], a[0], a[1], a[2], a[3], pl[nt][0], pl[nt][1]);
                    }
                }
            } else {
#pragma unroll 1
                for (int i0 = 0; i0 < p.NQ; ++i0) {
                    uint32_t mask[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) mask[j] = key0 + V::key(j, t) < least + i0 ? ~0u : 0u;
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        uint32_t a[4];
                        fragment(mt, a, mask);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float c[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816<F8>(c, a[0], a[1], a[2], a[3], ph[nt][0], ph[nt][1]);
                            if (!F8) mma16816<F8>(c, a[0], a[1], a[2], a[3], pl[nt][0], pl[nt][1]);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (lim[nt][k & 1] == least + i0) o[mt][nt][k] += c[k];
                        }
                    }
                }
            }
        }
        cp_wait<0>();
        __syncwarp();

        // the warps' states, joined in their stages
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x = l[nt][j];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                if (g == 0) {
                    float* e = stats + warp * 3 * C::kRows + nt * 8 + 2 * t + j;
                    e[0] = m[nt][j];
                    e[C::kRows] = F8 ? mv[nt][j] : m[nt][j];
                    e[2 * C::kRows] = x;
                }
            }
        float* mine = reinterpret_cast<float*>(smem + warp * C::kWarp);
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            const int u = mt / (V::kElems / 2), x = mt % (V::kElems / 2);
            const int d = u * 8 * V::kElems + g * V::kElems + 2 * x;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<float2*>(mine + (nt * 8 + 2 * t + j) * C::kStride + d) =
                        make_float2(o[mt][nt][j], o[mt][nt][j + 2]);
        }
        __syncthreads();
        const bool whole = n == units;
        float* part = p.part + ((size_t)blockIdx.x * 2 + (pos == g0 ? 0 : 1)) * C::kPart;
        const int rows = min(C::kRows, p.rows - row0);
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kPagedThreads) {
            const int r = idx / (D / 4), c = idx % (D / 4);
            float M = kNoMax, MV = kNoMax, L = 0.f;
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w) {
                M = fmaxf(M, stats[(w * 3) * C::kRows + r]);
                MV = fmaxf(MV, stats[(w * 3 + 1) * C::kRows + r]);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w) {
                const float f = ex2(stats[(w * 3) * C::kRows + r] - M), fv = ex2(stats[(w * 3 + 1) * C::kRows + r] - MV);
                L = fmaf(stats[(w * 3 + 2) * C::kRows + r], f, L);
                const float4 x = *reinterpret_cast<const float4*>(smem + w * C::kWarp + (r * C::kStride + 4 * c) * 4);
                acc.x = fmaf(x.x, fv, acc.x);
                acc.y = fmaf(x.y, fv, acc.y);
                acc.z = fmaf(x.z, fv, acc.z);
                acc.w = fmaf(x.w, fv, acc.w);
            }
            if (whole) {
                attn_finish<D>(p, qrow + row0 + r, c, acc, M, MV, L);
            } else {
                float* to = part + r * C::kStride;
                *reinterpret_cast<float4*>(to + 4 * c) = acc;
                if (c == 0) *reinterpret_cast<float4*>(to + D) = make_float4(M, MV, L, 0.f);
            }
        }
        __syncthreads();

        pos += n;
        if (pos < g1 && pos - base == units * p.Hkv * p.rblocks) {
            base = pos;
            do {
                len = seq_len(p, ++b);
            } while (len == 0);
            units = (len + kUnitKeys - 1) / kUnitKeys;
        }
    }
}

// Joins the partial states of the segments that were cut.  Block x looks at the boundary
// between the shares of CTAs x and x + 1 and takes the segment that is cut there for the first
// time; blockIdx.y and gridDim.y deal out its rows.  The four warps take every fourth state.
template <int D, int NT>
__global__ void __launch_bounds__(kPagedThreads) streamkl_paged_attn_join_kernel(const PagedParams p) {
    constexpr int kRows = 8 * NT, kStride = D + 4, kPart = kRows * kStride;
    __shared__ int red[8];
    __shared__ float st[kPagedWarps][4];
    __shared__ float4 ac[kPagedWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int total = plan_total(p, red);
    const int share = plan_share(p, total);
    const long long cut = (long long)(blockIdx.x + 1) * share;
    int b = 0, base = 0;
    const bool in = cut < total;
    if (in) plan_locate(p, (int)cut, red, b, base);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!in) return;
    const int units = seq_units(p, b);
    const int seg = ((int)cut - base) / units, s0 = base + seg * units;
    if (s0 == (int)cut || s0 / share != (int)blockIdx.x) return;   // not cut here, or cut before
    const int c0 = s0 / share, c1 = (s0 + units - 1) / share;
    const int h = seg / p.rblocks, rb = seg - h * p.rblocks, row0 = rb * kRows;
    const size_t qrow = ((size_t)b * p.Hkv + h) * p.rows;
    const int rows = min(kRows, p.rows - row0);
    const int first_slot = 2 * c0 + (s0 == c0 * share ? 0 : 1);
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float M = kNoMax, MV = kNoMax, L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = c0 + warp; c <= c1; c += kPagedWarps) {
            const float* from = p.part + (size_t)(c == c0 ? first_slot : 2 * c) * kPart + r * kStride;
            const float4 s = *reinterpret_cast<const float4*>(from + D);
            const float4 x = lane < D / 4 ? *reinterpret_cast<const float4*>(from + 4 * lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float Mn = fmaxf(M, s.x), Vn = fmaxf(MV, s.y);
            L = L * ex2(M - Mn) + s.z * ex2(s.x - Mn);
            const float f0 = ex2(MV - Vn), f1 = ex2(s.y - Vn);
            acc.x = acc.x * f0 + x.x * f1;
            acc.y = acc.y * f0 + x.y * f1;
            acc.z = acc.z * f0 + x.z * f1;
            acc.w = acc.w * f0 + x.w * f1;
            M = Mn;
            MV = Vn;
        }
        __syncthreads();
        if (lane == 0) {
            st[warp][0] = M;
            st[warp][1] = MV;
            st[warp][2] = L;
        }
        ac[warp][lane] = acc;
        __syncthreads();
        if (warp == 0 && lane < D / 4) {
            M = fmaxf(fmaxf(st[0][0], st[1][0]), fmaxf(st[2][0], st[3][0]));
            MV = fmaxf(fmaxf(st[0][1], st[1][1]), fmaxf(st[2][1], st[3][1]));
            L = 0.f;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w) {
                const float f = ex2(st[w][0] - M), fv = ex2(st[w][1] - MV);
                const float4 x = ac[w][lane];
                L = fmaf(st[w][2], f, L);
                acc.x = fmaf(x.x, fv, acc.x);
                acc.y = fmaf(x.y, fv, acc.y);
                acc.z = fmaf(x.z, fv, acc.z);
                acc.w = fmaf(x.w, fv, acc.w);
            }
            attn_finish<D>(p, qrow + row0 + r, lane, acc, M, MV, L);
        }
    }
}

}  // namespace skl
