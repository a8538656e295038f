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
// The last line is summed in fp64: its terms are as large as the scores' spread and may cancel to a small
// divergence.
#pragma once

#include "paged.cuh"

namespace skl {

// F1, F2: e4m3 (else bf16) keys of either cache; SHARED: one cache (F1 == F2).  A warp folds H 16-key
// tiles of either cache at a time: two where three stages of them fit its share of shared memory.
template <int D, bool F1, bool F2, bool SHARED, int NT>
struct KlCfg {
    using K1 = KeyTile<D, F1>;
    using K2 = KeyTile<D, F2>;
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = D / 16;
    static constexpr int kCtas = NT == 1 ? 3 : 2;                          // on an SM
    static constexpr int kShare = (kCtas == 3 ? 18 : 26) * 1024;           // of a warp
    static constexpr int kTiles = K1::kBytes + (SHARED ? 0 : K2::kBytes);  // one tile of each cache
    static constexpr int H = kTiles <= 3072 ? 2 : 1;
    static constexpr int kKeys = H * kTileKeys;
    static constexpr int kUnit = kPagedWarps * kKeys;
    static constexpr int kStart = 4;                                   // see PagedPlan
    static constexpr int kOff2 = H * K1::kBytes;
    static constexpr int kExp1 = H * kTiles;
    static constexpr int kExp2 = SHARED ? kExp1 : kExp1 + (F1 ? kKeys : 0);
    static constexpr int kStage = (kExp2 + (F2 ? kKeys : 0) + 127) / 128 * 128;
    static constexpr int kFit = kShare / kStage;
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kWarp = kStage * kStages;
    static constexpr int kStats = kPagedWarps * kWarp;                     // [warp][5][kRows]
    static constexpr int kSmem = kStats + kPagedWarps * 5 * kRows * 4;
    static constexpr int kPart = kRows * 5;
    static_assert(kStages >= 2, "ring");
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
    p.lse1[row] = (float)ln2 * (a[0] + log2f(a[1]));
    p.lse2[row] = (float)ln2 * (a[2] + log2f(a[3]));
    p.kl[row] = (float)(ln2 * ((double)(a[4] / a[1]) + ((double)a[2] - (double)a[0]) + (double)log2f(a[3] / a[1])));
}

// S^T of one tile: c[nt] += K Q^T for every block of 8 query rows; BOTH: also c2 from qf2 with the same keys.
// at: the lane's load offsets.
template <int D, bool F8, int NT, bool BOTH>
__device__ __forceinline__ void tile_scores(uint32_t ks, const uint32_t* at, const uint2* qf, float (*c)[4], const uint2* qf2,
                                            float (*c2)[4]) {
    using K = KeyTile<D, F8>;
    constexpr int kSteps = D / 16;
#pragma unroll
    for (int u = 0; u < K::kChunks; ++u) {
        const uint4 x = lds128(ks + at[u & 1] + K::load_step(0, u)), y = lds128(ks + at[u & 1] + K::load_step(1, u));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int w = 0; w < K::kSteps; ++w) {
            uint32_t a0, a1, a2, a3;
            if (F8) {
                e4m3x4_half2(xw[w], a0, a2);
                e4m3x4_half2(yw[w], a1, a3);
            } else {
                a0 = xw[(2 * w) & 3];
                a1 = yw[(2 * w) & 3];
                a2 = xw[(2 * w + 1) & 3];
                a3 = yw[(2 * w + 1) & 3];
            }
            const int step = u * K::kSteps + w;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint2 q = qf[nt * kSteps + step];
                mma16816<F8>(c[nt], a0, a1, a2, a3, q.x, q.y);
                if (BOTH) {
                    const uint2 r = qf2[nt * kSteps + step];
                    mma16816<F8>(c2[nt], a0, a1, a2, a3, r.x, r.y);
                }
            }
        }
    }
}

template <int D, bool F1, bool F2, bool SHARED, int NT>
__global__ void __launch_bounds__(kPagedThreads, KlCfg<D, F1, F2, SHARED, NT>::kCtas) streamkl_paged_kl_kernel(const PagedParams p) {
    using C = KlCfg<D, F1, F2, SHARED, NT>;
    using K1 = typename C::K1;
    using K2 = typename C::K2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t sb = smem_u32(smem);
    const uint32_t ring = sb + warp * C::kWarp;
    float* stats = reinterpret_cast<float*>(smem + C::kStats);
    constexpr int H = C::H;
    // where this lane copies from and to, and loads from, in every tile
    const uint8_t *keys1 = p.a.rows + lane * 16, *keys2 = p.b.rows + lane * 16;
    const uint32_t to1 = K1::copy_offset(lane), to2 = K2::copy_offset(lane);
    const uint32_t at1[2] = {(uint32_t)K1::load_offset(lane, 0), (uint32_t)K1::load_offset(lane, K1::kChunks > 1)};
    const uint32_t at2[2] = {(uint32_t)K2::load_offset(lane, 0), (uint32_t)K2::load_offset(lane, K2::kChunks > 1)};

    wait_for_stream();
    PagedWalk<C::kUnit, C::kStart> walk;
    for (bool more = walk.start(p); more; more = walk.next(p)) {
        const int n = walk.n, len = walk.len;                   // units, hence turns of a warp; keys
        const int h = walk.seg / p.rblocks, rb = walk.seg - h * p.rblocks;
        const int row0 = rb * C::kRows;
        const size_t qrow = ((size_t)walk.b * p.Hkv + h) * p.rows;
        const int* table = p.table + (size_t)walk.b * p.width;
        const int key00 = walk.u0 * C::kUnit + warp * C::kKeys;
        Queries<D, F1> raw1[NT];
        Queries<D, F2> raw2[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            raw1[nt].load(p.q1 + qrow * D, row0 + 8 * nt, p.rows);
            raw2[nt].load(p.q2 + qrow * D, row0 + 8 * nt, p.rows);
        }
        uint32_t bad = 0;         // bit (turn % 16) * 2 + tile: no such page
        PageAhead<H> pages;
        pages.start(p, table, key00, C::kUnit, len, n);
        auto request = [&](int i, uint32_t dst) {
            if (i < n) {
                bad &= ~(3u << ((i & 15) * 2));
                pages.turn(i);
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    const int key = key00 + i * C::kUnit + x * kTileKeys, page = pages.page(i, x);
                    const bool there = (unsigned)page < (unsigned)p.pages;
                    const int valid = there ? len - key : 0;
                    const int row = there && key < len ? (page * p.Hkv + h) * p.page_size + (key & (p.page_size - 1)) : 0;
                    if (!there) {
                        bad |= 1u << ((i & 15) * 2 + x);
                        if (lane == 0) g_page_status = 5;
                    }
                    K1::copy(dst + x * K1::kBytes + to1, keys1 + (size_t)row * K1::kRow, valid, lane);
                    if (!SHARED) K2::copy(dst + C::kOff2 + x * K2::kBytes + to2, keys2 + (size_t)row * K2::kRow, valid, lane);
                    if (F1 && lane == x) cp_async16(dst + C::kExp1 + x * kTileKeys, p.a.exps + row);
                    if (F2 && !SHARED && lane == H + x) cp_async16(dst + C::kExp2 + x * kTileKeys, p.b.exps + row);
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) request(i, ring + i * C::kStage);

        uint2 qf1[NT * C::kSteps], qf2[NT * C::kSteps];
        int e1[NT][2], e2[NT][2];             // of query 2t + j
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int f1 = raw1[nt].fragments(qf1 + nt * C::kSteps), f2 = raw2[nt].fragments(qf2 + nt * C::kSteps);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                e1[nt][j] = __shfl_sync(0xffffffffu, f1, 8 * t + 4 * j);
                e2[nt][j] = __shfl_sync(0xffffffffu, f2, 8 * t + 4 * j);
            }
        }
        ScoreScale scale1, scale2;
        float fac1[NT][2], fac2[NT][2];
        if (F1) scale1.start<NT>(p, e1);
        if (F2) scale2.start<NT>(p, e2);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (F1) fac1[nt][j] = scale1.row(e1[nt][j]);
                if (F2) fac2[nt][j] = scale2.row(e2[nt][j]);
            }
        // first key that a row does not see (of query 2t + j of block nt); the least over all rows
        auto limit = [&](int nt, int j) {
            return p.causal ? len - (p.NQ - 1) + (row0 + nt * 8 + 2 * t + j) % p.NQ : len;
        };
        float a[NT][2][5];      // m1, l1, m2, l2, acc of this lane's keys
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                a[nt][j][0] = a[nt][j][2] = kNoMax;
                a[nt][j][1] = a[nt][j][3] = a[nt][j][4] = 0.f;
            }
        const int least = p.causal ? len - (p.NQ - 1) : len;

        uint32_t ks = ring, last = ring + (C::kStages - 1) * C::kStage;     // stages of this turn and the one before
#pragma unroll 1
        for (int i = 0; i < n; ++i, last = ks, ks = ks == ring + (C::kStages - 1) * C::kStage ? ring : ks + C::kStage) {
            __syncwarp();       // every lane is done with the stage that is refilled
            request(i + C::kStages - 1, last);
            cp_wait<C::kStages - 1>();
            __syncwarp();       // what other lanes copied
            const int key0 = key00 + i * C::kUnit;
            if (key0 >= len) continue;

            // scores in base 2, each rounded once (and never fused into a later difference), their difference, and
            // whether a lane's references have to move
            float u[H][NT][2][2], v[H][NT][2][2], d[H][NT][2][2];
            bool grew = false;
#pragma unroll
            for (int x = 0; x < H; ++x) {
                float s1[NT][4], s2[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s1[nt][c] = s2[nt][c] = 0.f;
                tile_scores<D, F1, NT, SHARED>(ks + x * K1::kBytes, at1, qf1, s1, qf2, s2);
                if (!SHARED) tile_scores<D, F2, NT, false>(ks + C::kOff2 + x * K2::kBytes, at2, qf2, s2, nullptr, nullptr);
                float k1[2] = {p.sl2, p.sl2}, k2[2] = {p.sl2, p.sl2};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float of1 = F1 ? exp_scale(lds8(ks + C::kExp1 + x * 16 + 8 * k + g)) : 1.f;
                    if (F1) k1[k] = scale1.key * of1;
                    if (F2) k2[k] = scale2.key * (SHARED ? of1 : exp_scale(lds8(ks + C::kExp2 + x * 16 + 8 * k + g)));
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float y = __fmul_rn(s1[nt][j + 2 * k], k1[k]), z = __fmul_rn(s2[nt][j + 2 * k], k2[k]);
                            if (F1) y = __fmul_rn(y, fac1[nt][j]);
                            if (F2) z = __fmul_rn(z, fac2[nt][j]);
                            u[x][nt][j][k] = y;
                            v[x][nt][j][k] = z;
                            d[x][nt][j][k] = y - z;
                        }
            }
            if (key0 + C::kKeys > least || ((bad >> ((i & 15) * 2)) & 3u)) {
#pragma unroll
                for (int x = 0; x < H; ++x)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
                                if (key0 + x * kTileKeys + g + 8 * k >= limit(nt, j) || ((bad >> ((i & 15) * 2 + x)) & 1u)) {
                                    u[x][nt][j][k] = v[x][nt][j][k] = -INFINITY;
                                    d[x][nt][j][k] = 0.f;
                                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float n1 = fmaxf(u[0][nt][j][0], u[0][nt][j][1]), n2 = fmaxf(v[0][nt][j][0], v[0][nt][j][1]);
                    if (H == 2) {
                        n1 = fmaxf(n1, fmaxf(u[H - 1][nt][j][0], u[H - 1][nt][j][1]));
                        n2 = fmaxf(n2, fmaxf(v[H - 1][nt][j][0], v[H - 1][nt][j][1]));
                    }
                    grew |= n1 > a[nt][j][0] + kSlack;
                    grew |= n2 > a[nt][j][2] + kSlack;
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float* x = a[nt][j];
                        float n1 = x[0], n2 = x[2];
#pragma unroll
                        for (int y = 0; y < H; ++y) {
                            n1 = fmaxf(n1, fmaxf(u[y][nt][j][0], u[y][nt][j][1]));
                            n2 = fmaxf(n2, fmaxf(v[y][nt][j][0], v[y][nt][j][1]));
                        }
                        const float r1 = ex2(x[0] - n1);
                        x[1] *= r1;
                        x[4] *= r1;
                        x[3] *= ex2(x[2] - n2);
                        x[0] = n1;
                        x[2] = n2;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float* x = a[nt][j];
#pragma unroll
                    for (int y = 0; y < H; ++y) {
                        const float e0 = ex2(u[y][nt][j][0] - x[0]), e1 = ex2(u[y][nt][j][1] - x[0]);
                        x[1] += e0 + e1;
                        x[4] = fmaf(e0, d[y][nt][j][0], fmaf(e1, d[y][nt][j][1], x[4]));
                        x[3] += ex2(v[y][nt][j][0] - x[2]) + ex2(v[y][nt][j][1] - x[2]);
                    }
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
        const int r = threadIdx.x, rows = min(C::kRows, p.rows - row0);
        if (r < rows) {
            float x[5], y[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) x[k] = stats[k * C::kRows + r];
#pragma unroll
            for (int w = 1; w < kPagedWarps; ++w) {
#pragma unroll
                for (int k = 0; k < 5; ++k) y[k] = stats[(w * 5 + k) * C::kRows + r];
                kl_join(x, y);
            }
            if (walk.complete()) {
                kl_finish(p, qrow + row0 + r, x);
            } else {
                float* to = p.part + (size_t)walk.slot() * C::kPart + r;
#pragma unroll
                for (int k = 0; k < 5; ++k) to[k * C::kRows] = x[k];
            }
        }
        if (!walk.complete()) {
            const int c0 = walk.c0(), c1 = walk.c1();
            if (arrive_last(p.arrived + c0, c1 - c0 + 1, reinterpret_cast<int*>(smem))) {
                // a power of two of lanes to a row, every such state each
                constexpr int kLanes = NT == 1 ? 16 : 8;
                const int jr = threadIdx.x / kLanes, sub = threadIdx.x % kLanes, first_slot = walk.first_slot();
                float x[5] = {kNoMax, 0.f, kNoMax, 0.f, 0.f}, y[5];
                if (jr < rows) {
#pragma unroll 4
                    for (int c = c0 + sub; c <= c1; c += kLanes) {
                        const float* from = p.part + (size_t)(c == c0 ? first_slot : 2 * c) * C::kPart + jr;
#pragma unroll
                        for (int k = 0; k < 5; ++k) y[k] = __ldcg(from + k * C::kRows);
                        kl_join(x, y);
                    }
                }
#pragma unroll
                for (int d = kLanes / 2; d > 0; d >>= 1) {
#pragma unroll
                    for (int k = 0; k < 5; ++k) y[k] = __shfl_xor_sync(0xffffffffu, x[k], d);
                    kl_join(x, y);
                }
                if (sub == 0 && jr < rows) kl_finish(p, qrow + row0 + jr, x);
            }
        }
        __syncthreads();
    }

    // sequences without keys
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (threadIdx.x == 0 && (p.lengths[b] < 0 || p.lengths[b] > p.width * p.page_size)) g_page_status = 5;
        if (seq_len(p, b) > 0) continue;
        const size_t r0 = (size_t)b * p.Hkv * p.rows, n = (size_t)p.Hkv * p.rows;
        for (size_t i = threadIdx.x; i < n; i += kPagedThreads) {
            p.kl[r0 + i] = 0.f;
            p.lse1[r0 + i] = p.lse2[r0 + i] = -INFINITY;
        }
    }
}

}  // namespace skl
