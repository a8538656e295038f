// paged_attn_kernel.cuh -- attention of a few new tokens over a paged key-value cache.
//
//     s_j = scale <q, k_j>,   o = sum_j exp(s_j - lse) v_j,   lse = log sum_j exp(s_j)
//
// over the keys j that the row sees, in one pass: sum l and weighted sum o refer to a running
// maximum m and are rescaled by 2^(m_old - m_new) when it moves (see kSlack).  A score in base 2 is rounded once,
// and that one value is what m is a maximum of and what m is subtracted from: were the weight's exponent
// a fused s * factor - m of any factor, the largest key's would be its product's rounding error, 2^(E - 24) for
// a score near 2^E, and from 2^30 on weights would all vanish or overflow.  So a bf16 cache's products are
// multiplied by the scale first; an e4m3 cache's by scale times key scale, and what is left, the query row's
// power of two, may be fused, because that product is exact (see ScoreScale).
//
// Bound: every cached byte is read once and used for 2 flops per query row and element, so with the
// few rows of a KV head (Hq / Hkv * NQ) the floor is cache bytes / HBM bandwidth.  Everything here
// serves the loads: each warp streams its own tiles through a ring of cp.async slots that only it
// touches (see RowTile), so no barrier of the CTA stands between a load and the next.
//
// Per tile a warp computes S^T = K Q^T (16 keys x 8 rows per product) and the weights, and turns P^T around
// with movmatrix into the B operand of O^T = V^T P^T (M: 16 columns of d, N: 8 rows, K: 16 keys).  V^T's
// fragments need two keys' values of one column in a register: the lane loads the same bytes of four
// keys and joins them with byte permutes.  The m16n8k16 products suffice: the tensor pipe is 14 to 19 %
// busy, and without any one of the three steps the kernel takes as long (64 uneven sequences: 106 us
// against 106 when that was measured); without the copies it takes 78.
//
// bf16 cache: P is split into two bf16 terms (hi + lo, off by 2^-16 of a weight), because one bf16 rounding
// of P (2^-8) would add as much error as the output's own rounding; the tensor pipe has room for the
// second product.  hi is the largest bf16 number below P, so that lo is above 0 wherever P is: times an infinite
// value both are that infinity (a lo of either sign, or 0, would make NaN of it).  What needs 8 bits is kept exactly.
// e4m3 cache: values are met as fp16 (exact) without their scales 2^e_j; those go into the weights,
// P'_j = 2^(s_j - m + e_j - x), where m + x follows the running maximum of s_j + e_j, so that P' stays within
// fp16 whatever the scales are; its rounding (2^-11) is an eighth of the output's.  l keeps to m alone.  x is kept
// instead of the sum m + x, in which scores beyond 2^24 would leave no bits for it.
// Where a turn's scales lie within 2^kNear of each other (and all so far within 2^-40 .. 2^40), P' is
// the sum's weight times two factors and m + x moves by the bound max s + max e, which is at most kNear too
// high; elsewhere both are taken key by key, with a second exponential.
// fp16 ends at 2^-24, and weights that vanish there still count in l: many of them would pull the output
// towards 0 (2^20 keys 25 octaves below a sink: up to 9.7 % with the reference at the maximum).  So m + x moves
// kDrop below the maximum, which with the slack uses fp16 up to 2^15: what is lost of a weight is at most 2^-32
// of the warp's largest P', 2^-28 with the bound.
#pragma once

#include "paged.cuh"

namespace skl {

// The terms of two weights of 0 or more, as bf16 pairs (hi of 0 is 0).
__device__ __forceinline__ void weight_terms(float w0, float w1, uint32_t& hi, uint32_t& lo) {
    const int x0 = max(__float_as_int(w0) - 1, 0), x1 = max(__float_as_int(w1) - 1, 0);
    hi = __byte_perm(x0, x1, 0x7632);
    lo = bf16_pair(w0 - __uint_as_float(x0 & 0xffff0000u), w1 - __uint_as_float(x1 & 0xffff0000u));
}

constexpr int kNear = 4;      // octaves, see above
constexpr float kDrop = 7.f;  // the same; 2^(kDrop + kSlack) is below fp16's largest, 65504

// Values: lane (g, t) of V^T's fragments holds columns of keys 2t, 2t + 1, 2t + 8 and 2t + 9, and takes
// kElems contiguous ones of each: chunk g (and g + 8 where a row has 16), or half a chunk where it has
// four.  The lanes of a load phase meet rows 2t of all t.
template <int D, bool F8>
struct ValueTile : RowTile<D, F8> {
    using R = RowTile<D, F8>;
    static constexpr int kLane = R::kRow / 8;                   // bytes of a row per lane
    static constexpr int kLoad = kLane < 16 ? kLane : 16;       // bytes of one load
    static constexpr int kChunks = kLane / kLoad;
    static constexpr int kElems = kLoad / (F8 ? 1 : 2);         // elements of a load

    __device__ static __forceinline__ int key(int j, int t) { return 2 * t + (j & 1) + 8 * (j >> 1); }

    __device__ static __forceinline__ int place(int row, int chunk) {
        if (R::kRow >= 128) return row * R::kRow + (chunk ^ (row & 6)) * 16;
        return ((row & 1) + (row >> 2) * 2) * 128 + ((row >> 1) & 1) * 64 + (chunk ^ (((row >> 2) & 1) * 2)) * 16;
    }
    __device__ static __forceinline__ int copy_offset(int lane) { return place(R::copy_row(lane), lane % R::kRowChunks); }
    // as KeyTile::copy; the tile is 128-byte aligned, so a row's swizzle flips bits of the address
    __device__ static __forceinline__ void copy(uint32_t dst, const uint8_t* from, int valid, int lane) {
        if (valid >= kTileKeys) {
#pragma unroll
            for (int i = 0; i < R::kCopies; ++i) cp_async16((dst ^ flip(i)) + i * 512, from + i * 512);
        } else {
#pragma unroll
            for (int i = 0; i < R::kCopies; ++i)
                cp_async16((dst ^ flip(i)) + i * 512, from + i * 512, i * R::kStep + R::copy_row(lane) < valid ? 16 : 0);
        }
    }
    __device__ static constexpr uint32_t flip(int i) { return R::kRow >= 128 ? ((i * R::kStep) & 6) * 16 : 0; }
    // load u of key(j, t) lies at load_offset(lane) + load_step(j, u)
    __device__ static __forceinline__ int load_offset(int lane) {
        const int g = lane >> 2;
        return kLoad == 16 ? place(key(0, lane & 3), g) : place(key(0, lane & 3), g >> 1) + (g & 1) * 8;
    }
    __device__ static constexpr int load_step(int j, int u) {
        return R::kRow >= 128 ? ((j & 1) + 8 * (j >> 1)) * R::kRow + u * 128 : (j & 1) * 128 + (j >> 1) * 512;
    }
    // the lane's words (4 bytes) there
    __device__ static __forceinline__ void load(uint32_t src, uint32_t* w) {
        if (kLoad == 16) {
            const uint4 v = lds128(src);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
            const uint2 v = lds64(src);
            w[0] = v.x; w[1] = v.y;
        }
    }
};

// NT: blocks of 8 query rows; a warp folds H 16-key tiles at a time.  Two tiles halve the waits and the
// bookkeeping per key and give the products two independent chains (20 rows over e4m3 keys: 38.4 us with
// one, 36.2 with two); the registers do not hold them with 32 rows, nor a warp's shared memory three
// slots of them with bf16 rows of d = 128 (and 166 us are near the floor of 164 there).  With 32 rows of
// d = 128 they do not hold one tile's either: 80 (bf16) and 88 bytes (e4m3) of a thread are spilled, 62 and
// 59 us for 64 x 8192 keys, where 24 rows take 55 and 43.
template <int D, bool F8, int NT>
struct AttnCfg {
    using K = KeyTile<D, F8>;
    using V = ValueTile<D, F8>;
    static constexpr int H = NT == 4 || (NT == 3 && !F8) || (D == 128 && !F8) ? 1 : 2;
    // Resident CTAs per SM, registers permitting.  At most 8 rows, 131072 bf16 keys of 16 heads / 64 uneven e4m3
    // sequences: 2: 170 / 125 us, 3: 169 / 109, 4 (128 registers, spills): 178 / 108.
    static constexpr int kCtas = NT == 1 ? 3 : 2;
    static constexpr int kKeys = H * kTileKeys;                        // of a warp at a time
    static constexpr int kUnit = kPagedWarps * kKeys;
    static constexpr int kStart = NT == 1 ? 4 : 6;                     // see PagedPlan
    static constexpr int kRows = 8 * NT;
    static constexpr int kSteps = D / 16;
    // A slot holds the keys or the values of kKeys tokens, and their exponents.  The slots form a ring,
    // keys and values in turn; their number is odd, so that the slot refilled after a key (value) slot
    // is used again takes keys (values).
    static constexpr int kExps = H * K::kBytes;
    static constexpr int kSlot = H * K::kBytes + (F8 ? 128 : 0);
    static constexpr int kFit = (kCtas == 3 ? 17 : 26) * 1024 / kSlot;   // a warp's share of shared memory
    static constexpr int kSlots = kFit >= 9 ? 9 : (kFit % 2 ? kFit : kFit - 1);
    static constexpr int kAhead = (kSlots - 1) / 2;                    // tiles in flight
    static constexpr int kWarp = kSlot * kSlots;
    static constexpr int kStride = D + 4;                              // floats of a row's state
    static constexpr bool kSharedQ = NT > 2;                           // query fragments in shared memory
    static constexpr int kQ = kPagedWarps * kWarp;
    static constexpr int kFactor = kQ + (kSharedQ ? NT * kSteps * 32 * 8 : 0);
    static constexpr int kStats = kFactor + (kSharedQ ? NT * 32 * 4 : 0);   // [warp][3][kRows]
    static constexpr int kSmem = kStats + kPagedWarps * 3 * kRows * 4;
    static constexpr int kPart = kRows * kStride;                      // floats of a partial state
    static_assert(kSlots >= 3 && kSlots % 2 == 1, "ring");
    static_assert(kWarp >= kRows * kStride * 4, "a warp's state is joined in its slots");
    static_assert(K::kBytes == V::kBytes, "one slot size");
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "resident CTAs");
};

// Four columns of a finished row: o / l, rounded once to bf16, and the row's lse.  Weights that refer to
// M + X come back to M by 2^X, after the division so that this step overflows nothing
// that the result does not.  A row that sees no key (l = 0): zeros and -inf.  No other row has l = 0: M is kSlack
// above one of the rounded scores (rounded itself, by at most as much again), whose weight is therefore 2^-16 or more.
template <int D>
__device__ __forceinline__ void attn_finish(const PagedParams& p, size_t row, int c, float4 acc, float M, float X, float L) {
    const bool none = L == 0.f;
    const float inv = none ? 0.f : 1.f / L, f = none ? 0.f : exp2f(X);
    uint2 y;
    y.x = none ? 0u : bf16_pair(acc.x * inv * f, acc.y * inv * f);
    y.y = none ? 0u : bf16_pair(acc.z * inv * f, acc.w * inv * f);
    *reinterpret_cast<uint2*>(p.out + row * D + 4 * c) = y;
    if (c == 0) p.lse1[row] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// Joins the partial states of CTAs c0 .. c1 (first_slot, then 2c) into rows [row, row + rows), of which
// this is one of `shares` CTAs.  `each` of the WARPS warps take ROWS rows together, every each-th state in order,
// kBatch loaded together, and meet in shared memory (WARPS * ROWS * 33 float4).  Two rows together where
// there may be more than 8 keep twice the loads in flight: 7 uneven sequences, 20 rows over e4m3 keys, 34.7 -> 32.8 us
// (33.5 with scores rounded once), 4 x 32768 keys of bf16, 32 rows, 66.1 -> 60.8; up to 8 rows have a warp or more a row anyway.
constexpr int kBatch = 8;

struct RowState {
    float m = kNoMax, x = 0.f, l = 0.f;       // reference of the sum; the weighted sum's, less that; sum
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);

    // references m1 >= m and m1 + x1 >= m + x
    __device__ __forceinline__ void move(float m1, float x1) {
        const float f = ex2((m - m1) + x - x1);
        l *= ex2(m - m1);
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
        m = m1;
        x = x1;
    }
    // a state (m, x, l of q; its weighted sum y) whose references are not above this one's
    __device__ __forceinline__ void add(float4 q, float4 y) {
        const float f = ex2((q.x - m) + q.y - x);
        l = fmaf(q.z, ex2(q.x - m), l);
        acc.x = fmaf(y.x, f, acc.x);
        acc.y = fmaf(y.y, f, acc.y);
        acc.z = fmaf(y.z, f, acc.z);
        acc.w = fmaf(y.w, f, acc.w);
    }
};

template <int D, int PART, int WARPS, int ROWS>
__device__ __forceinline__ void attn_join(const PagedParams& p, int c0, int c1, int first_slot, size_t row, int rows, int mine,
                                          int shares, float4* scratch) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int states = c1 - c0 + 1;
    int each = 1;
    while (each < WARPS && (each * kBatch * 4 < states || (each * kBatch < states && each * rows < WARPS * ROWS * shares))) each *= 2;
    const int part = warp & (each - 1), group = warp / each, groups = WARPS / each;
    for (int r0 = mine * groups * ROWS; r0 < rows; r0 += shares * groups * ROWS) {
        const int r = r0 + group * ROWS;
        RowState to[ROWS];
        for (int c = c0 + part; c <= c1 && r < rows; c += kBatch * each) {
            float4 q[ROWS][kBatch], x[ROWS][kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int ck = c + k * each;
                const float* from = p.part + (size_t)(ck == c0 ? first_slot : 2 * ck) * PART + r * (D + 4);
#pragma unroll
                for (int i = 0; i < ROWS; ++i) {
                    q[i][k] = make_float4(kNoMax, 0.f, 0.f, 0.f);
                    x[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (ck <= c1 && r + i < rows) {
                        q[i][k] = __ldcg(reinterpret_cast<const float4*>(from + i * (D + 4) + D));
                        x[i][k] = __ldcg(reinterpret_cast<const float4*>(from + i * (D + 4) + 4 * (lane % (D / 4))));
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                float m1 = to[i].m;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) m1 = fmaxf(m1, q[i][k].x);
                float x1 = (to[i].m - m1) + to[i].x;
#pragma unroll
                for (int k = 0; k < kBatch; ++k) x1 = fmaxf(x1, (q[i][k].x - m1) + q[i][k].y);
                to[i].move(m1, x1);
#pragma unroll
                for (int k = 0; k < kBatch; ++k) to[i].add(q[i][k], x[i][k]);
            }
        }
        if (each > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                scratch[(warp * ROWS + i) * 33 + lane] = to[i].acc;
                if (lane == 0) scratch[(warp * ROWS + i) * 33 + 32] = make_float4(to[i].m, to[i].x, to[i].l, 0.f);
            }
            __syncthreads();
            if (part == 0)
                for (int w = warp + 1; w < warp + each; ++w)
#pragma unroll
                    for (int i = 0; i < ROWS; ++i) {
                        const float4 q = scratch[(w * ROWS + i) * 33 + 32];
                        const float m1 = fmaxf(to[i].m, q.x);
                        to[i].move(m1, fmaxf((to[i].m - m1) + to[i].x, (q.x - m1) + q.y));
                        to[i].add(q, scratch[(w * ROWS + i) * 33 + lane]);
                    }
        }
        if (part == 0 && lane < D / 4)
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                if (r + i < rows) attn_finish<D>(p, row + r + i, lane, to[i].acc, to[i].m, to[i].x, to[i].l);
    }
}

template <int D, bool F8, int NT>
__global__ void __launch_bounds__(kPagedThreads, AttnCfg<D, F8, NT>::kCtas) streamkl_paged_attn_kernel(const PagedParams p) {
    using C = AttnCfg<D, F8, NT>;
    using K = typename C::K;
    using V = typename C::V;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t sb = smem_u32(smem);
    const uint32_t ring = sb + warp * C::kWarp;
    constexpr int H = C::H;
    // where this lane copies from and to, and loads from, in every tile
    const uint8_t *keys = p.a.rows + lane * 16, *values = p.b.rows + lane * 16;
    const uint32_t key_to = K::copy_offset(lane), value_to = V::copy_offset(lane);
    const uint32_t key_at[2] = {(uint32_t)K::load_offset(lane, 0), (uint32_t)K::load_offset(lane, K::kChunks > 1)};
    const uint32_t value_at = V::load_offset(lane);
    float* stats = reinterpret_cast<float*>(smem + C::kStats);

    wait_for_stream();
    PagedWalk<C::kUnit, C::kStart> walk;
    for (bool more = walk.start(p); more; more = walk.next(p)) {
        const int n = walk.n, len = walk.len;                   // units, hence turns of a warp; keys
        const int h = walk.seg / p.rblocks, rb = walk.seg - h * p.rblocks;
        const int row0 = rb * C::kRows;
        const size_t qrow = ((size_t)walk.b * p.Hkv + h) * p.rows;
        const int* table = p.table + (size_t)walk.b * p.width;
        const int key00 = walk.u0 * C::kUnit + warp * C::kKeys;

        Queries<D, F8> raw[C::kSharedQ ? 1 : NT];
        if (C::kSharedQ) {
            raw[0].load(p.q1 + qrow * D, row0 + 8 * warp, p.rows);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) raw[C::kSharedQ ? 0 : nt].load(p.q1 + qrow * D, row0 + 8 * nt, p.rows);
        }

        // The turn whose rows are requested next: pool rows and number of existing keys of each tile.
        int row[H], valid[H];
        uint32_t bad = 0;                                 // bit (turn % 16) * 2 + tile: no such page
        PageAhead<H> pages;
        pages.start(p, table, key00, C::kUnit, len, n);
        auto request_keys = [&](int i, uint32_t dst) {
            if (i < n) {
                bad &= ~(3u << ((i & 15) * 2));
                pages.turn(i);
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    const int key = key00 + i * C::kUnit + x * kTileKeys, page = pages.page(i, x);
                    const bool there = (unsigned)page < (unsigned)p.pages;
                    valid[x] = there ? len - key : 0;
                    row[x] = there && key < len ? (page * p.Hkv + h) * p.page_size + (key & (p.page_size - 1)) : 0;
                    if (!there) {
                        bad |= 1u << ((i & 15) * 2 + x);
                        if (lane == 0) g_page_status = 5;
                    }
                    K::copy(dst + x * K::kBytes + key_to, keys + (size_t)row[x] * K::kRow, valid[x], lane);
                    if (F8 && lane == x) cp_async16(dst + C::kExps + x * kTileKeys, p.a.exps + row[x]);
                }
            }
            cp_commit();
        };
        auto request_values = [&](int i, uint32_t dst) {
            if (i < n) {
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    V::copy(dst + x * V::kBytes + value_to, values + (size_t)row[x] * V::kRow, valid[x], lane);
                    if (F8 && lane == x) cp_async16(dst + C::kExps + x * kTileKeys, p.b.exps + row[x]);
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < C::kAhead; ++i) {
            request_keys(i, ring + 2 * i * C::kSlot);
            request_values(i, ring + (2 * i + 1) * C::kSlot);
        }

        // queries of this segment, as B fragments
        uint2 qf[C::kSharedQ ? 1 : NT * C::kSteps];
        int qe[NT][2];
        if (C::kSharedQ) {
            uint2 f[C::kSteps];
            const int one = raw[0].fragments(f);
            if (warp < NT) {
#pragma unroll
                for (int s = 0; s < C::kSteps; ++s)
                    reinterpret_cast<uint2*>(smem + C::kQ)[(warp * C::kSteps + s) * 32 + lane] = f[s];
                if (t == 0) reinterpret_cast<int*>(smem + C::kFactor)[warp * 8 + g] = one;
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                qe[nt][0] = reinterpret_cast<int*>(smem + C::kFactor)[nt * 8 + 2 * t];
                qe[nt][1] = reinterpret_cast<int*>(smem + C::kFactor)[nt * 8 + 2 * t + 1];
            }
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int one = raw[C::kSharedQ ? 0 : nt].fragments(qf + (C::kSharedQ ? 0 : nt * C::kSteps));
                qe[nt][0] = __shfl_sync(0xffffffffu, one, 8 * t);
                qe[nt][1] = __shfl_sync(0xffffffffu, one, 8 * t + 4);
            }
        }
        ScoreScale scale;
        float fac[NT][2];
        if (F8) {
            scale.start<NT>(p, qe);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) fac[nt][j] = scale.row(qe[nt][j]);
        }
        // first key that a row does not see (of query 2t + j of block nt); the least over all rows
        auto limit = [&](int nt, int j) {
            return p.causal ? len - (p.NQ - 1) + (row0 + nt * 8 + 2 * t + j) % p.NQ : len;
        };
        const int least = p.causal ? len - (p.NQ - 1) : len;

        // m: reference of the sum, up to kSlack above the scores' maximum; m + x: of the weights (bf16: x = 0), kDrop below
        // what it follows; mx: 2^-x; l: sum
        float o[D / 16][NT][4], m[NT][2], x[NT][2], mx[NT][2], l[NT][2];
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
                m[nt][j] = kNoMax;
                x[nt][j] = l[nt][j] = 0.f;
                mx[nt][j] = 1.f;
            }
        bool tame = true;       // e4m3: every value scale so far within 2^-40 .. 2^40

        uint32_t cur = ring, last = ring + (C::kSlots - 1) * C::kSlot;   // slots of this item and the one before
        auto advance = [&]() {
            last = cur;
            cur = cur == ring + (C::kSlots - 1) * C::kSlot ? ring : cur + C::kSlot;
        };
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int key0 = key00 + i * C::kUnit;
            __syncwarp();       // every lane is done with the slot that is refilled
            request_keys(i + C::kAhead, last);
            cp_wait<C::kSlots - 1>();
            __syncwarp();       // the exponents were copied by single lanes
            const bool some = key0 < len;
            const bool edge = key0 + C::kKeys > least || ((bad >> ((i & 15) * 2)) & 3u);
            auto seen = [&](int x, int k, int nt, int j) {     // key g + 8k of tile x, query 2t + j of block nt
                return key0 + x * kTileKeys + g + 8 * k < limit(nt, j) && !((bad >> ((i & 15) * 2 + x)) & 1u);
            };

            // S^T, scores in base 2 but for the row's power of two fac (e4m3)
            float s[H][NT][4];
            if (some) {
#pragma unroll
                for (int x = 0; x < H; ++x)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) s[x][nt][0] = s[x][nt][1] = s[x][nt][2] = s[x][nt][3] = 0.f;
#pragma unroll
                for (int u = 0; u < K::kChunks; ++u) {
                    uint4 y[H][2];
#pragma unroll
                    for (int x = 0; x < H; ++x)
#pragma unroll
                        for (int k = 0; k < 2; ++k) y[x][k] = lds128(cur + x * K::kBytes + key_at[u & 1] + K::load_step(k, u));
#pragma unroll
                    for (int w = 0; w < K::kSteps; ++w) {
                        uint32_t a[H][4];
#pragma unroll
                        for (int x = 0; x < H; ++x) {
                            const uint32_t w0[4] = {y[x][0].x, y[x][0].y, y[x][0].z, y[x][0].w};
                            const uint32_t w1[4] = {y[x][1].x, y[x][1].y, y[x][1].z, y[x][1].w};
                            if (F8) {
                                e4m3x4_half2(w0[w], a[x][0], a[x][2]);
                                e4m3x4_half2(w1[w], a[x][1], a[x][3]);
                            } else {
                                a[x][0] = w0[(2 * w) & 3];
                                a[x][1] = w1[(2 * w) & 3];
                                a[x][2] = w0[(2 * w + 1) & 3];
                                a[x][3] = w1[(2 * w + 1) & 3];
                            }
                        }
                        const int step = u * K::kSteps + w;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 q = C::kSharedQ ? lds64(sb + C::kQ + ((nt * C::kSteps + step) * 32 + lane) * 8)
                                                        : qf[C::kSharedQ ? 0 : nt * C::kSteps + step];
#pragma unroll
                            for (int x = 0; x < H; ++x) mma16816<F8>(s[x][nt], a[x][0], a[x][1], a[x][2], a[x][3], q.x, q.y);
                        }
                    }
                }
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    float k[2] = {p.sl2, p.sl2};
                    if (F8) {
                        k[0] = scale.key * exp_scale(lds8(cur + C::kExps + x * 16 + g));
                        k[1] = scale.key * exp_scale(lds8(cur + C::kExps + x * 16 + 8 + g));
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[x][nt][c] = __fmul_rn(s[x][nt][c], k[c >> 1]);
                }
                if (edge) {
#pragma unroll
                    for (int x = 0; x < H; ++x)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (!seen(x, c >> 1, nt, c & 1)) s[x][nt][c] = -INFINITY;
                }
            }
            advance();

            __syncwarp();
            request_values(i + C::kAhead, last);
            cp_wait<C::kSlots - 1>();
            __syncwarp();
            if (some) {
                // e4m3: the exponents' range over the turn's keys
                int e_max = 0;
                bool near = true;
                if (F8) {
                    const int at = lane & (C::kKeys - 1);
                    const uint32_t e = lds8(cur + C::kExps + at);
                    const bool in = !edge || (key0 + at < len && !((bad >> ((i & 15) * 2 + (at >> 4))) & 1u));
                    e_max = (int)__reduce_max_sync(0xffffffffu, in ? e : 0u);
                    const int e_min = (int)__reduce_min_sync(0xffffffffu, in ? e : 255u);
                    tame = tame && e_min >= 127 - 40 && e_max <= 127 + 40;
                    near = tame && e_max - e_min <= kNear;
                    e_max -= 127;
                }
                // exponent byte of value key g + 8k of tile x; 127 where there is no such key
                auto value_exp = [&](int x, int k) {
                    const uint32_t e = lds8(cur + C::kExps + x * 16 + 8 * k + g);
                    return edge && !(key0 + x * 16 + 8 * k + g < len && !((bad >> ((i & 15) * 2 + x)) & 1u)) ? 127u : e;
                };
                // The lane's own maxima lm of the scores, and lm + hi of the scores times the values' scales (near:
                // its bound), against the references: only where one lies beyond them do the 8 lanes with
                // this t exchange maxima and the sums move.
                float lm[NT][2], hi[NT][2];
                bool grew = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
                        if (H == 2) top = fmaxf(top, fmaxf(s[H - 1][nt][j], s[H - 1][nt][j + 2]));
                        lm[nt][j] = F8 ? top * fac[nt][j] : top;
                        hi[nt][j] = (float)e_max;
                        grew |= lm[nt][j] > m[nt][j];
                    }
                if (F8) {
                    if (!near) {
                        float ev[H][2];
#pragma unroll
                        for (int y = 0; y < H; ++y)
#pragma unroll
                            for (int k = 0; k < 2; ++k) ev[y][k] = (float)((int)value_exp(y, k) - 127);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                hi[nt][j] = kNoMax;      // stays where the lane's keys are all masked (lm = -inf)
#pragma unroll
                                for (int y = 0; y < H; ++y)
#pragma unroll
                                    for (int k = 0; k < 2; ++k)
                                        hi[nt][j] = fmaxf(hi[nt][j], fmaf(s[y][nt][j + 2 * k], fac[nt][j], -lm[nt][j]) + ev[y][k]);
                            }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) grew |= (lm[nt][j] - m[nt][j]) + hi[nt][j] > x[nt][j] + (kSlack + kDrop);
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float top = lm[nt][j];
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            top = fmaxf(m[nt][j], top + kSlack);
                            const float by = m[nt][j] - top;
                            float a = ex2(by);
                            l[nt][j] *= a;
                            if (F8) {
                                float ref = (lm[nt][j] - top) + hi[nt][j];
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, d));
                                ref = fmaxf(by + x[nt][j], ref - kDrop);
                                a = ex2(by + x[nt][j] - ref);
                                x[nt][j] = ref;
                                mx[nt][j] = ex2(-ref);
                            }
                            m[nt][j] = top;
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                o[k][nt][j] *= a;
                                o[k][nt][j + 2] *= a;
                            }
                        }
                }
                // weights, in place of the scores
                uint32_t ph[H][NT][2], pl[H][NT][2];    // B fragments of P^T: hi and lo (bf16), or P' (fp16)
                if (F8 && !near) {
#pragma unroll
                    for (int y = 0; y < H; ++y) {
                        const float ev[2] = {(float)((int)value_exp(y, 0) - 127), (float)((int)value_exp(y, 1) - 127)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float q = fmaf(s[y][nt][c], fac[nt][c & 1], -m[nt][c & 1]);
                                s[y][nt][c] = ex2(q + (ev[c >> 1] - x[nt][c & 1]));
                                l[nt][c & 1] += ex2(q);
                            }
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float sum = 0.f;
#pragma unroll
                            for (int y = 0; y < H; ++y)
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float z = s[y][nt][j + 2 * k];
                                    const float q = ex2(F8 ? fmaf(z, fac[nt][j], -m[nt][j]) : __fsub_rn(z, m[nt][j]));
                                    sum += q;
                                    s[y][nt][j + 2 * k] = q;
                                }
                            l[nt][j] += sum;
                        }
                    if (F8) {
                        float kv[H][2];
#pragma unroll
                        for (int y = 0; y < H; ++y)
#pragma unroll
                            for (int k = 0; k < 2; ++k) kv[y][k] = exp_scale(value_exp(y, k));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
#pragma unroll
                                for (int y = 0; y < H; ++y)
#pragma unroll
                                    for (int k = 0; k < 2; ++k) s[y][nt][j + 2 * k] *= mx[nt][j] * kv[y][k];
                            }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < H; ++x) {
                        const float* w = s[x][nt];
                        if (F8) {
                            ph[x][nt][0] = movmatrix(pack_half(w[0], w[1]));
                            ph[x][nt][1] = movmatrix(pack_half(w[2], w[3]));
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                uint32_t hi, lo;
                                weight_terms(w[2 * k], w[2 * k + 1], hi, lo);
                                ph[x][nt][k] = movmatrix(hi);
                                pl[x][nt][k] = movmatrix(lo);
                            }
                        }
                    }
                // O^T += V^T P^T
#pragma unroll
                for (int x = 0; x < H; ++x) {
                    const uint32_t at = cur + x * V::kBytes + value_at;
                    const int keyx = key0 + x * kTileKeys;
                    uint32_t v[V::kChunks][4][4];
#pragma unroll
                    for (int u = 0; u < V::kChunks; ++u)
#pragma unroll
                        for (int j = 0; j < 4; ++j) V::load(at + V::load_step(j, u), v[u][j]);
                    // A row that does not see a key must not meet its values even with weight 0 (0 * inf
                    // and 0 * NaN are NaN): where such a tile holds values that are not finite, each query
                    // position is done by itself with the keys behind its limit cleared.
                    bool slow = false;
                    if (edge && least < len) {
                        bool odd = false;
#pragma unroll
                        for (int u = 0; u < V::kChunks; ++u)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
#pragma unroll
                                for (int w = 0; w < V::kLoad / 4; ++w)
#pragma unroll
                                    for (int e = 0; e < 32; e += F8 ? 8 : 16)
                                        odd |= F8 ? ((v[u][j][w] >> e) & 0x7fu) == 0x7fu
                                                  : ((v[u][j][w] >> e) & 0x7f80u) == 0x7f80u;
                        slow = __any_sync(0xffffffffu, odd);
                    }
                    auto fragment = [&](int mt, uint32_t* a, const uint32_t* mask) {
                        // m-tile mt: columns 2y, 2y + 1 of the lane's elements of chunk u
                        const int u = mt / (V::kElems / 2), y = mt % (V::kElems / 2);
                        const int w = F8 ? y >> 1 : y;
                        uint32_t k0 = v[u][0][w], k1 = v[u][1][w], k2 = v[u][2][w], k3 = v[u][3][w];
                        if (mask) {
                            k0 &= mask[0];
                            k1 &= mask[1];
                            k2 &= mask[2];
                            k3 &= mask[3];
                        }
                        if (F8) {
                            const uint32_t sel = (y & 1) ? 0x7362u : 0x5140u;
                            const uint32_t lo = __byte_perm(k0, k1, sel), hi = __byte_perm(k2, k3, sel);
                            e4m3x4_half2(lo, a[0], a[1]);
                            e4m3x4_half2(hi, a[2], a[3]);
                        } else {
                            a[0] = __byte_perm(k0, k1, 0x5410);
                            a[1] = __byte_perm(k0, k1, 0x7632);
                            a[2] = __byte_perm(k2, k3, 0x5410);
                            a[3] = __byte_perm(k2, k3, 0x7632);
                        }
                    };
                    if (!slow) {
#pragma unroll
                        for (int mt = 0; mt < D / 16; ++mt) {
                            uint32_t a[4];
                            fragment(mt, a, nullptr);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<F8>(o[mt][nt], a[0], a[1], a[2], a[3], ph[x][nt][0], ph[x][nt][1]);
                                if (!F8) mma16816<F8>(o[mt][nt], a[0], a[1], a[2], a[3], pl[x][nt][0], pl[x][nt][1]);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (int y = 0; y < min(p.NQ, C::kRows); ++y) {
                            const int i0 = (row0 + y) % p.NQ;      // the positions of this block's rows
                            uint32_t mask[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) mask[j] = keyx + V::key(j, t) < least + i0 ? ~0u : 0u;
#pragma unroll
                            for (int mt = 0; mt < D / 16; ++mt) {
                                uint32_t a[4];
                                fragment(mt, a, mask);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float c[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma16816<F8>(c, a[0], a[1], a[2], a[3], ph[x][nt][0], ph[x][nt][1]);
                                    if (!F8) mma16816<F8>(c, a[0], a[1], a[2], a[3], pl[x][nt][0], pl[x][nt][1]);
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        if (limit(nt, k & 1) == least + i0) o[mt][nt][k] += c[k];
                                }
                            }
                        }
                    }
                }
            }
            advance();
        }
        cp_wait<0>();
        __syncwarp();

        // the warps' states, joined in their slots
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float sum = l[nt][j];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (g == 0) {
                    float* e = stats + warp * 3 * C::kRows + nt * 8 + 2 * t + j;
                    e[0] = m[nt][j];
                    e[C::kRows] = F8 ? x[nt][j] : 0.f;
                    e[2 * C::kRows] = sum;
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
        const bool whole = walk.complete();
        float* part = p.part + (size_t)walk.slot() * C::kPart;
        const int rows = min(C::kRows, p.rows - row0);
        for (int idx = threadIdx.x; idx < rows * (D / 4); idx += kPagedThreads) {
            const int i = idx / (D / 4), c = idx % (D / 4);
            float M = kNoMax, X = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, stats[(w * 3) * C::kRows + i]);
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w)
                X = fmaxf(X, (stats[(w * 3) * C::kRows + i] - M) + stats[(w * 3 + 1) * C::kRows + i]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kPagedWarps; ++w) {
                const float by = stats[(w * 3) * C::kRows + i] - M, fv = ex2(by + stats[(w * 3 + 1) * C::kRows + i] - X);
                L = fmaf(stats[(w * 3 + 2) * C::kRows + i], ex2(by), L);
                const float4 y = *reinterpret_cast<const float4*>(smem + w * C::kWarp + (i * C::kStride + 4 * c) * 4);
                acc.x = fmaf(y.x, fv, acc.x);
                acc.y = fmaf(y.y, fv, acc.y);
                acc.z = fmaf(y.z, fv, acc.z);
                acc.w = fmaf(y.w, fv, acc.w);
            }
            if (whole) {
                attn_finish<D>(p, qrow + row0 + i, c, acc, M, X, L);
            } else {
                float* to = part + i * C::kStride;
                *reinterpret_cast<float4*>(to + 4 * c) = acc;
                if (c == 0) *reinterpret_cast<float4*>(to + D) = make_float4(M, X, L, 0.f);
            }
        }
        if (!whole && p.arrived) {
            const int c0 = walk.c0(), c1 = walk.c1();
            if (arrive_last(p.arrived + c0, c1 - c0 + 1, reinterpret_cast<int*>(stats)))
                attn_join<D, C::kPart, kPagedWarps, NT == 1 ? 1 : 2>(p, c0, c1, walk.first_slot(), qrow + row0, rows, 0, 1, reinterpret_cast<float4*>(smem));
        }
        __syncthreads();
    }
    // sequences without keys: zeros and -inf
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (threadIdx.x == 0 && (p.lengths[b] < 0 || p.lengths[b] > p.width * p.page_size)) g_page_status = 5;
        if (seq_len(p, b) > 0) continue;
        const size_t r0 = (size_t)b * p.Hkv * p.rows, n = (size_t)p.Hkv * p.rows;
        for (size_t i = threadIdx.x; i < n * (D / 8); i += kPagedThreads)
            reinterpret_cast<uint4*>(p.out + r0 * D)[i] = make_uint4(0, 0, 0, 0);
        for (size_t i = threadIdx.x; i < n; i += kPagedThreads) p.lse1[r0 + i] = -INFINITY;
    }
}

// The join in a kernel of its own, for segments with so many states and rows that one CTA would be long at it.
// Block x looks at the boundary between the shares of CTAs x and x + 1 and takes the segment that is cut
// there for the first time; blockIdx.y and gridDim.y deal out its rows.
constexpr int kJoinThreads = 256;

template <int D, int NT, int UNIT, int START>
__global__ void __launch_bounds__(kJoinThreads) streamkl_paged_attn_join_kernel(const PagedParams p) {
    constexpr int kRows = 8 * NT, kPart = kRows * (D + 4);
    __shared__ float4 scratch[kJoinThreads / 32 * 33];
    wait_for_stream();      // the main kernel is complete
    PagedCut<UNIT, START> cut;
    if (!cut.find(p, blockIdx.x)) return;
    const int h = cut.seg / p.rblocks, rb = cut.seg - h * p.rblocks, row0 = rb * kRows;
    const size_t qrow = ((size_t)cut.b * p.Hkv + h) * p.rows;
    attn_join<D, kPart, kJoinThreads / 32, 1>(p, cut.c0, cut.c1, cut.first_slot, qrow + row0, min(kRows, p.rows - row0), blockIdx.y,
                                           gridDim.y, scratch);
}

}  // namespace skl
