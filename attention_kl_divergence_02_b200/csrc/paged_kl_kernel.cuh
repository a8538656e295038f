// paged_kl_kernel.cuh -- KL divergence of two attentions over paged key caches, a few new tokens.
//
// The forward's recurrence (StreamKL technical summary, gist.science, Portuguese, "1. Formulação
// Online (Passagem Forward)") over pages and a ragged batch: per query row the five running
// scalars m1, l1, m2, l2, acc = sum_j 2^(u1_j - m1) (u1_j - u2_j), u the scores in base 2, and
//
//     KL = ln 2 * (acc / l1 + m2 - m1 + log2(l2 / l1)).
//
// The two caches may be of different types (a student over a quantised cache against its teacher
// over the unquantised one), or one cache serves both (each key is read once).
//
// Bound: key bytes / HBM bandwidth, as in paged_attn_kernel.cuh, whose tiles, copies and division of
// the work this shares.  There is no weighted sum of values, so every lane keeps scalars of its own
// over the keys that it sees and no maximum crosses lanes until the segment ends.
//
// The last line is evaluated in fp64 (a few hundred rows): acc / l1 and the difference of the log
// sums are each as large as the scores' spread and may cancel to a small divergence.
#pragma once

#include "paged.cuh"

namespace skl {

// F1, F2: e4m3 (else bf16) keys of either cache; SHARED: one cache (F1 == F2).
template <int D, bool F1, bool F2, bool SHARED, int NT>
struct KlCfg {
    using K1 = KeyTile<D, F1>;
    using K2 = KeyTile<D, F2>;
    static constexpr int kUnit = kPagedWarps * kTileKeys;
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = D / 16;
    static constexpr int kOff2 = K1::kBytes;
    static constexpr int kExp1 = kOff2 + (SHARED ? 0 : K2::kBytes);
    static constexpr int kExp2 = kExp1 + (F1 ? 16 : 0);
    static constexpr int kStage = kExp2 + (F2 && !SHARED ? 16 : 0);
    static constexpr int kMax = 24 * 1024 / kStage;
    static constexpr int kStages = kMax > 8 ? 8 : kMax;
    static constexpr int kWarp = kStage * kStages;
    static constexpr bool kSharedQ = NT > 2;
    static constexpr int kQ = kPagedWarps * kWarp;                         // [2][NT][steps][lane]
    static constexpr int kFactor = kQ + (kSharedQ ? 2 * NT * kSteps * 32 * 8 : 0);   // [2][NT][8]
    static constexpr int kStats = kFactor + (kSharedQ ? 2 * NT * 8 * 4 : 0);         // [warp][5][kRows]
    static constexpr int kRed = kStats + kPagedWarps * 5 * kRows * 4;
    static constexpr int kSmem = kRed + 64;
    static constexpr int kPart = kRows * 5;
};

// Joins state b (of other keys) to state a: m1, l1, m2, l2, acc.
__device__ __forceinline__ void kl_join(float* a, const float* b) {
    const float M1 = fmaxf(a[0], b[0]), M2 = fmaxf(a[2], b[2]);
    const float ea = ex2(a[0] - M1), eb = ex2(b[0] - M1);
    a[1] = a[1] * ea + b[1] * eb;
    a[4] = a[4] * ea + b[4] * eb;
    a[3] = a[3] * ex2(a[2] - M2) + b[3] * ex2(b[2] - M2);
    a[0] = M1;
    a[2] = M2;
}

// A finished row.  No key seen: divergence 0, both lse -inf.
__device__ __forceinline__ void kl_finish(const PagedParams& p, size_t row, const float* a) {
    if (a[1] == 0.f) {
        p.kl[row] = 0.f;
        p.lse1[row] = p.lse2[row] = -INFINITY;
        return;
    }
    const double ln2 = 0.693147180559945309417;
    const double g1 = log2((double)a[1]), g2 = log2((double)a[3]);
    p.lse1[row] = (float)(ln2 * ((double)a[0] + g1));
    p.lse2[row] = (float)(ln2 * ((double)a[2] + g2));
    p.kl[row] = (float)(ln2 * ((double)a[4] / (double)a[1] + ((double)a[2] - (double)a[0]) + (g2 - g1)));
}

// S^T of one tile: c[nt] += K Q^T for every block of 8 query rows.
template <int D, bool F8, int NT, bool SHARED_Q>
__device__ __forceinline__ void tile_scores(uint32_t ks, int lane, const uint2* qf, uint32_t qs, float (*c)[4]) {
    using K = KeyTile<D, F8>;
    constexpr int kSteps = D / 16;
#pragma unroll
    for (int u = 0; u < K::kChunks; ++u) {
        const uint4 x = K::load(ks, 0, u, lane), y = K::load(ks, 1, u, lane);
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
                const uint2 q = SHARED_Q ? lds64(qs + ((nt * kSteps + step) * 32 + lane) * 8)
                                         : qf[SHARED_Q ? 0 : nt * kSteps + step];
                mma16816<F8>(c[nt], a0, a1, a2, a3, q.x, q.y);
            }
        }
    }
}

template <int D, bool F1, bool F2, bool SHARED, int NT>
__global__ void __launch_bounds__(kPagedThreads, 2) streamkl_paged_kl_kernel(const PagedParams p) {
    using C = KlCfg<D, F1, F2, SHARED, NT>;
    using K1 = typename C::K1;
    using K2 = typename C::K2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t sb = smem_u32(smem);
    const uint32_t stage0 = sb + warp * C::kWarp;
    float* stats = reinterpret_cast<float*>(smem + C::kStats);
    int* red = reinterpret_cast<int*>(smem + C::kRed);

    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (threadIdx.x == 0 && (p.lengths[b] < 0 || p.lengths[b] > p.width * p.page_size)) g_page_status = 5;
        if (seq_len(p, b) > 0) continue;
        const size_t r0 = (size_t)b * p.Hkv * p.rows, n = (size_t)p.Hkv * p.rows;
        for (size_t i = threadIdx.x; i < n; i += kPagedThreads) {
            p.kl[r0 + i] = 0.f;
            p.lse1[r0 + i] = p.lse2[r0 + i] = -INFINITY;
        }
    }

    const int total = plan_total<C::kUnit>(p, red);
    const int share = plan_share(p, total);
    const long long first = (long long)blockIdx.x * share;
    if (first >= total) return;
    const int g0 = (int)first, g1 = (int)min((long long)total, first + share);
    int b, base;
    plan_locate<C::kUnit>(p, g0, red, b, base);
    int len = seq_len(p, b), units = (len + C::kUnit - 1) / C::kUnit;

    for (int pos = g0; pos < g1;) {
        const int off = pos - base, seg = off / units, u0 = off - seg * units;
        const int n = min(units - u0, g1 - pos);
        const int h = seg / p.rblocks, rb = seg - h * p.rblocks;
        const int row0 = rb * C::kRows;
        const size_t qrow = ((size_t)b * p.Hkv + h) * p.rows;
        const int* table = p.table + (size_t)b * p.width;
        const int key00 = u0 * C::kUnit + warp * kTileKeys;
        uint32_t bad = 0;

        auto issue = [&](int i, int s) {
            const int key0 = key00 + i * C::kUnit;
            const uint32_t dst = stage0 + s * C::kStage;
            bad &= ~(1u << s);
            if (key0 < len) {
                const int page = __ldg(table + (key0 >> p.page_shift));
                if ((unsigned)page < (unsigned)p.pages) {
                    const size_t row = ((size_t)page * p.Hkv + h) * p.page_size + (key0 & (p.page_size - 1));
                    const int valid = len - key0;
                    K1::copy(dst, p.a.rows + row * K1::kRow, valid, lane);
                    if (!SHARED) K2::copy(dst + C::kOff2, p.b.rows + row * K2::kRow, valid, lane);
                    if (F1 && lane == 0) cp_async16(dst + C::kExp1, p.a.exps + row, 16);
                    if (F2 && !SHARED && lane == 1) cp_async16(dst + C::kExp2, p.b.exps + row, 16);
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

        uint2 qf1[C::kSharedQ ? 1 : NT * C::kSteps], qf2[C::kSharedQ ? 1 : NT * C::kSteps];
        float fac1[NT][2], fac2[NT][2];
        if (C::kSharedQ) {
            uint2 f[C::kSteps];
            float one;
            float* fs = reinterpret_cast<float*>(smem + C::kFactor);
            uint2* qs = reinterpret_cast<uint2*>(smem + C::kQ);
            load_queries<D, F1>(p.q1 + qrow * D, row0 + 8 * warp, p.rows, p.sl2, f, one);
            if (warp < NT) {
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s) qs[(warp * C::kSteps + s) * 32 + lane] = f[s];
                if (t == 0) fs[warp * 8 + g] = one;
            }
            load_queries<D, F2>(p.q2 + qrow * D, row0 + 8 * warp, p.rows, p.sl2, f, one);
            if (warp < NT) {
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s) qs[((NT + warp) * C::kSteps + s) * 32 + lane] = f[s];
                if (t == 0) fs[(NT + warp) * 8 + g] = one;
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    fac1[nt][j] = fs[nt * 8 + 2 * t + j];
                    fac2[nt][j] = fs[(NT + nt) * 8 + 2 * t + j];
                }
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float one;
                load_queries<D, F1>(p.q1 + qrow * D, row0 + 8 * nt, p.rows, p.sl2, qf1 + nt * C::kSteps, one);
                fac1[nt][0] = __shfl_sync(0xffffffffu, one, 8 * t);
                fac1[nt][1] = __shfl_sync(0xffffffffu, one, 8 * t + 4);
                load_queries<D, F2>(p.q2 + qrow * D, row0 + 8 * nt, p.rows, p.sl2, qf2 + nt * C::kSteps, one);
                fac2[nt][0] = __shfl_sync(0xffffffffu, one, 8 * t);
                fac2[nt][1] = __shfl_sync(0xffffffffu, one, 8 * t + 4);
            }
        }
        int lim[NT][2];
        float a[NT][2][5];      // m1, l1, m2, l2, acc of this lane's keys
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                lim[nt][j] = p.causal ? len - (p.NQ - 1) + (row0 + nt * 8 + 2 * t + j) % p.NQ : len;
                a[nt][j][0] = a[nt][j][2] = kNoMax;
                a[nt][j][1] = a[nt][j][3] = a[nt][j][4] = 0.f;
            }
        const int least = p.causal ? len - (p.NQ - 1) : len;

        int st = 0;
        for (int i = 0; i < n; ++i, st = st + 1 == C::kStages ? 0 : st + 1) {
            __syncwarp();
            if (i + C::kStages - 1 < n) issue(i + C::kStages - 1, st == 0 ? C::kStages - 1 : st - 1);
            else cp_commit();
            cp_wait<C::kStages - 1>();
            __syncwarp();
            const int key0 = key00 + i * C::kUnit;
            if (key0 >= len || ((bad >> st) & 1u)) continue;
            const uint32_t ks = stage0 + st * C::kStage;

            float s1[NT][4], s2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s1[nt][c] = s2[nt][c] = 0.f;
            tile_scores<D, F1, NT, C::kSharedQ>(ks, lane, qf1, sb + C::kQ, s1);
            tile_scores<D, F2, NT, C::kSharedQ>(SHARED ? ks : ks + C::kOff2, lane, qf2, sb + C::kQ + NT * C::kSteps * 256, s2);
            float k1[2] = {1.f, 1.f}, k2[2] = {1.f, 1.f};
            if (F1) {
                k1[0] = exp_scale(lds8(ks + C::kExp1 + g));
                k1[1] = exp_scale(lds8(ks + C::kExp1 + 8 + g));
            }
            if (F2) {
                k2[0] = SHARED ? k1[0] : exp_scale(lds8(ks + C::kExp2 + g));
                k2[1] = SHARED ? k1[1] : exp_scale(lds8(ks + C::kExp2 + 8 + g));
            }
            const bool edge = key0 + kTileKeys > least;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float u[2], v[2], d[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        u[k] = s1[nt][j + 2 * k] * fac1[nt][j];
                        v[k] = s2[nt][j + 2 * k] * fac2[nt][j];
                        if (F1) u[k] *= k1[k];
                        if (F2) v[k] *= k2[k];
                        d[k] = u[k] - v[k];
                        if (edge && key0 + g + 8 * k >= lim[nt][j]) {
                            u[k] = v[k] = -INFINITY;
                            d[k] = 0.f;
                        }
                    }
                    float* x = a[nt][j];
                    const float n1 = fmaxf(x[0], fmaxf(u[0], u[1])), n2 = fmaxf(x[2], fmaxf(v[0], v[1]));
                    const float r1 = ex2(x[0] - n1), r2 = ex2(x[2] - n2);
                    const float e0 = ex2(u[0] - n1), e1 = ex2(u[1] - n1);
                    x[1] = fmaf(x[1], r1, e0 + e1);
                    x[4] = fmaf(x[4], r1, fmaf(e0, d[0], e1 * d[1]));
                    x[3] = fmaf(x[3], r2, ex2(v[0] - n2) + ex2(v[1] - n2));
                    x[0] = n1;
                    x[2] = n2;
                }
        }
        cp_wait<0>();

#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    float y[5];
#pragma unroll
                    for (int k = 0; k < 5; ++k) y[k] = __shfl_xor_sync(0xffffffffu, a[nt][j][k], d);
                    kl_join(a[nt][j], y);
                }
                if (g == 0)
#pragma unroll
                    for (int k = 0; k < 5; ++k) stats[(warp * 5 + k) * C::kRows + nt * 8 + 2 * t + j] = a[nt][j][k];
            }
        __syncthreads();
        const int r = threadIdx.x;
        if (r < min(C::kRows, p.rows - row0)) {
            float x[5], y[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) x[k] = stats[k * C::kRows + r];
#pragma unroll
            for (int w = 1; w < kPagedWarps; ++w) {
#pragma unroll
                for (int k = 0; k < 5; ++k) y[k] = stats[(w * 5 + k) * C::kRows + r];
                kl_join(x, y);
            }
            if (n == units) {
                kl_finish(p, qrow + row0 + r, x);
            } else {
                float* to = p.part + ((size_t)blockIdx.x * 2 + (pos == g0 ? 0 : 1)) * C::kPart + r;
#pragma unroll
                for (int k = 0; k < 5; ++k) to[k * C::kRows] = x[k];
            }
        }
        __syncthreads();

        pos += n;
        if (pos < g1 && pos - base == units * p.Hkv * p.rblocks) {
            base = pos;
            do {
                len = seq_len(p, ++b);
            } while (len == 0);
            units = (len + C::kUnit - 1) / C::kUnit;
        }
    }
}

// Joins the partial states of the segments that were cut; see streamkl_paged_attn_join_kernel.
// A warp takes a row and its lanes the states.
template <int NT, int UNIT>
__global__ void __launch_bounds__(kPagedThreads) streamkl_paged_kl_join_kernel(const PagedParams p) {
    constexpr int kRows = 8 * NT, kPart = kRows * 5;
    __shared__ int red[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int total = plan_total<UNIT>(p, red);
    const int share = plan_share(p, total);
    const long long cut = (long long)(blockIdx.x + 1) * share;
    int b = 0, base = 0;
    const bool in = cut < total;
    if (in) plan_locate<UNIT>(p, (int)cut, red, b, base);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!in) return;
    const int units = seq_units<UNIT>(p, b);
    const int seg = ((int)cut - base) / units, s0 = base + seg * units;
    if (s0 == (int)cut || s0 / share != (int)blockIdx.x) return;
    const int c0 = s0 / share, c1 = (s0 + units - 1) / share;
    const int h = seg / p.rblocks, rb = seg - h * p.rblocks, row0 = rb * kRows;
    const size_t qrow = ((size_t)b * p.Hkv + h) * p.rows;
    const int first_slot = 2 * c0 + (s0 == c0 * share ? 0 : 1);
    for (int r = warp; r < min(kRows, p.rows - row0); r += kPagedWarps) {
        float x[5] = {kNoMax, 0.f, kNoMax, 0.f, 0.f}, y[5];
        for (int c = c0 + lane; c <= c1; c += 32) {
            const float* from = p.part + (size_t)(c == c0 ? first_slot : 2 * c) * kPart + r;
#pragma unroll
            for (int k = 0; k < 5; ++k) y[k] = from[k * kRows];
            kl_join(x, y);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
            for (int k = 0; k < 5; ++k) y[k] = __shfl_xor_sync(0xffffffffu, x[k], d);
            kl_join(x, y);
        }
        if (lane == 0) kl_finish(p, qrow + row0 + r, x);
    }
}

}  // namespace skl
