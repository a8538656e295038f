// paged.cuh -- what the kernels over a paged key-value cache share: the cache's view, the
// division of the work among a persistent grid, and the warp-level pieces (asynchronous copies
// into shared memory, the m16n8k16 product, e4m3 rows).
//
// A cache pool holds pages of one kind of row (keys or values), [pages, Hkv, page_size, d],
// bf16 or e4m3; an e4m3 row has one power-of-two scale, kept as the byte exponent + 127 in
// [pages, Hkv, page_size].  Sequence b's token j lies in page table[b][j / page_size].
//
// Work division.  A segment is one (sequence, KV head, block of query rows); its keys are cut
// into units (of 64 or 128 keys).  All segments' units in a row, T of them, are dealt out in equal contiguous
// shares of P = ceil(T / grid): lengths are read on the device, so a ragged batch loads every
// SM alike and the host needs no lengths.  A share may begin or end inside a segment; such a
// CTA stores a partial state, and the CTA that comes last joins the segment's states in the
// order of their CTAs (whichever comes last: the same inputs give the same bits).  A CTA has at most two
// partial segments, its first (slot 2c) and its last (slot 2c + 1), so the workspace depends on
// the grid alone and not on the lengths.  Where the page table is so narrow that every segment is short,
// segments are dealt out whole, and there is nothing to join.
#pragma once

#include "sm100.cuh"

namespace skl {

// A page table entry or a length that points outside the cache (STREAMKL_ERR_PAGE, 5).  A word of
// its own: the pipelined kernels give up their waits when g_status is set.
__device__ int g_page_status = 0;

constexpr int kPagedThreads = 128;     // 4 warps, each with its own tiles and copies
constexpr int kPagedWarps = kPagedThreads / 32;
constexpr int kTileKeys = 16;          // keys of a product (its M)
constexpr float kNoMax = -3.402823466e38f;   // running maximum before any key
// Running sums refer to 2^m with m within kSlack (log2 units) of the running maximum, and are rescaled only
// when it grows beyond that, which costs fp32 sums and the weights' 16-bit types (relative rounding, fp16 up to
// 2^15) nothing: the rescaling, in almost every turn of a short sequence with many rows otherwise, all but
// vanishes.  Attention moves m to kSlack above the maximum, so that no weight exceeds 1 and the sums of weights
// times values overflow no sooner than they must; the divergence, without values, moves it to the maximum.
constexpr float kSlack = 8.f;

struct PagedPool {
    const uint8_t* rows;
    const uint8_t* exps;   // nullptr for bf16
};

struct PagedParams {
    PagedPool a, b;        // attention: keys, values; divergence: keys 1, keys 2
    const int* table;      // [B, width]
    const int* lengths;    // [B]
    const uint16_t* q1;    // [B, Hq, NQ, d]: the rows of one KV head are contiguous
    const uint16_t* q2;
    int B, Hkv, NQ;
    int rows;              // query rows of one KV head: Hq / Hkv * NQ
    int rblocks;           // blocks of query rows
    int width, pages, page_size, page_shift;
    int causal;
    int whole;             // segments are not cut: no partial states
    int grid;              // CTAs of the main kernel
    float sl2;             // scale * log2(e)
    float mant;            // the same as mant * 2^exp, mant in [1, 2)
    int exp;
    uint16_t* out;         // attention
    float* lse1;
    float* lse2;           // divergence
    float* kl;
    unsigned* arrived;     // [CTAs]: partial states of the segment first cut behind a CTA; all 0 between calls
    float* part;           // partial states, slot-major
};

__device__ __forceinline__ int seq_len(const PagedParams& p, int b) {
    const int n = p.lengths[b];
    const int cap = p.width * p.page_size;
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// UNIT: keys of a unit, all warps' tiles once.  START: units' worth of time that a CTA spends on beginning and
// ending a segment; shares are equal in units plus START per segment, or a CTA with two segments would
// end late by that much (64 uneven sequences, e4m3: 100 -> 94 us; a unit weighs 8 to 32 KB of keys and values, and the
// constant was not measured for each).  On the line of all segments, each is START + units long.
template <int UNIT, int START>
struct PagedPlan {
    // of sequence b's segments
    __device__ static __forceinline__ int units(int len) { return (len + UNIT - 1) / UNIT; }
    __device__ static __forceinline__ int length(const PagedParams& p, int b) {
        const int n = units(seq_len(p, b));
        return n ? n + START : 0;
    }

    // Length of the whole line.  Each warp computes it by itself, as the rest of the plan: 32 sequences at a
    // time, without a barrier.  head: of sequence `lane`, which most batches need not read again.
    __device__ static __forceinline__ int total(const PagedParams& p, int& head) {
        const int lane = threadIdx.x & 31;
        int n = head = lane < p.B ? length(p, lane) : 0;
        for (int b = lane + 32; b < p.B; b += 32) n += length(p, b);
        return __reduce_add_sync(0xffffffffu, n) * p.Hkv * p.rblocks;
    }

    // The share of a CTA.
    __device__ static __forceinline__ int share(const PagedParams& p, int total) { return max((total + p.grid - 1) / p.grid, 1); }

    // The sequence at position g of the line, and where it begins.
    __device__ static __forceinline__ void locate(const PagedParams& p, int g, int head, int& b, int& base) {
        const int lane = threadIdx.x & 31, per = p.Hkv * p.rblocks;
        int before = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int x = (b0 == 0 ? head : b0 + lane < p.B ? length(p, b0 + lane) : 0) * per;
            int upto = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const unsigned behind = __ballot_sync(0xffffffffu, g < before + upto);
            if (behind) {
                const int at = __ffs(behind) - 1;
                b = b0 + at;
                base = before + __shfl_sync(0xffffffffu, upto - x, at);
                return;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
        b = base = 0;      // not reached for g < total
    }
};

// A CTA's walk over its work: whole segments in turn where all are short (p.whole), else its share of the
// line, cut where it begins and ends.
template <int UNIT, int START>
struct PagedWalk {
    using Plan = PagedPlan<UNIT, START>;
    int b, len, seg, units, u0, n;     // sequence, its keys, segment in it, its units, first unit and number of them to do
    int pos, base, end, first, share;  // position on the line, where the sequence begins, end and begin of the share

    __device__ __forceinline__ bool start(const PagedParams& p) {
        first = 0;
        if (p.whole) {
            pos = (int)blockIdx.x;
            end = p.B * p.Hkv * p.rblocks;
            return find_whole(p);
        }
        int head;
        const int total = Plan::total(p, head);
        share = Plan::share(p, total);
        const long long at = (long long)blockIdx.x * share;
        if (at >= total) return false;
        first = pos = (int)at;
        end = (int)min((long long)total, at + share);
        Plan::locate(p, pos, head, b, base);
        len = seq_len(p, b);
        units = Plan::units(len);
        return cut() || next(p);
    }
    __device__ __forceinline__ bool next(const PagedParams& p) {
        if (p.whole) {
            pos += gridDim.x;
            return find_whole(p);
        }
        do {
            pos = base + (seg + 1) * (START + units);
            if (pos >= end) return false;
            if (seg + 1 == p.Hkv * p.rblocks) {
                base = pos;
                do {
                    if (++b >= p.B) return false;      // not met while the lengths stay as they are
                    len = seq_len(p, b);
                } while (len == 0);
                units = Plan::units(len);
            }
        } while (!cut());
        return true;
    }
    __device__ __forceinline__ bool complete() const { return n == units; }
    // Where this CTA's partial state of the segment goes, and the segment's CTAs; their states are the first's
    // at first_slot() and the others' at 2c.
    __device__ __forceinline__ int slot() const { return 2 * blockIdx.x + (pos == first ? 0 : 1); }
    __device__ __forceinline__ int c0() const { return (begin() + START) / share; }
    __device__ __forceinline__ int c1() const { return (begin() + START + units - 1) / share; }
    __device__ __forceinline__ int first_slot() const { return 2 * c0() + (begin() > c0() * share ? 1 : 0); }

private:
    __device__ __forceinline__ int begin() const { return base + seg * (START + units); }
    // the units at pos; false where the share ends before the segment's first
    __device__ __forceinline__ bool cut() {
        seg = (pos - base) / (START + units);
        const int unit0 = begin() + START;      // of unit 0 on the line
        u0 = max(pos - unit0, 0);
        n = min(end - unit0, units) - u0;
        return n > 0;
    }
    __device__ __forceinline__ bool find_whole(const PagedParams& p) {
        const int per = p.Hkv * p.rblocks;
        for (; pos < end; pos += gridDim.x) {
            b = pos / per;
            seg = pos - b * per;
            len = seq_len(p, b);
            if (len > 0) {
                n = units = Plan::units(len);
                u0 = 0;
                return true;
            }
        }
        return false;
    }
};

// Called by all threads of a CTA once its partial state of a segment is written: true in the one that
// comes last of `states`, which then may read them all (past L1, __ldcg).  The counter wraps back
// to 0 with the last.  One thread's release carries the writes that the barrier put before it, and its
// acquire, behind the second barrier, lets the others read.  flag: a word of shared memory.
__device__ __forceinline__ bool arrive_last(unsigned* counter, int states, int* flag) {
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned before;
        asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(before) : "l"(counter), "r"((unsigned)states - 1u) : "memory");
        *flag = before == (unsigned)states - 1u;
    }
    __syncthreads();
    return *flag != 0;
}

// The segment whose units begin in CTA `block`'s share and end in a later one's, for a join in a kernel of
// its own.
template <int UNIT, int START>
struct PagedCut {
    using Plan = PagedPlan<UNIT, START>;
    int b, seg, c0, c1, first_slot;

    __device__ __forceinline__ bool find(const PagedParams& p, int block) {
        int head;
        const int total = Plan::total(p, head), share = Plan::share(p, total);
        const long long cut = (long long)(block + 1) * share;
        if (cut >= total) return false;
        int base;
        Plan::locate(p, (int)cut, head, b, base);
        const int units = Plan::units(seq_len(p, b));
        seg = ((int)cut - base) / (START + units);
        const int begin = base + seg * (START + units);
        c0 = (begin + START) / share;
        c1 = (begin + START + units - 1) / share;
        first_slot = 2 * c0 + (begin > c0 * share ? 1 : 0);
        return c0 == block && c1 > block;
    }
};

// Every kernel here is launched as a programmatic dependent of whatever ran before on its stream: its launch
// overlaps that kernel's end (2.0 to 2.4 us a call between short kernels: 64 single tokens written and read
// back 8.2 -> 5.7 us, one short sequence's attention 8.2 -> 5.8, 131072 keys 167.5 -> 165.6), and its
// threads begin here, where they wait until that kernel is complete and its writes are visible.  What they read
// may have been written while they were already running, so all of it takes plain loads, behind the wait: a
// read-only load (ld.global.nc) would promise data that is constant for the kernel's whole duration.  Letting
// the next kernel come before this one's last CTA is done (launch_dependents) was no better: 6.0 and 7.6 us where
// 5.8 and 5.8 are without.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The pages of a warp's tiles, H a turn: every lane holds one entry, looked up a batch of 32 / H turns
// ahead, so that no request waits for the table.
template <int H>
struct PageAhead {
    static constexpr int kTurns = 32 / H;
    const int* table;
    int key, step, len, shift, now, then;      // key: of this lane's tile in turn 0

    __device__ __forceinline__ void start(const PagedParams& p, const int* row, int key00, int unit, int n_keys, int turns) {
        const int lane = threadIdx.x & 31;
        table = row;
        key = key00 + (lane / H) * unit + (lane % H) * kTileKeys;
        step = kTurns * unit;
        len = n_keys;
        shift = p.page_shift;
        now = look_up(0);
        then = turns > kTurns ? look_up(1) : 0;
    }
    __device__ __forceinline__ int look_up(int batch) const {
        const int at = key + batch * step;
        return at >= 0 && at < len ? table[at >> shift] : 0;
    }
    // before the first page of turn i
    __device__ __forceinline__ void turn(int i) {
        if (i % kTurns == 0 && i > 0) {
            now = then;
            then = look_up(i / kTurns + 1);
        }
    }
    __device__ __forceinline__ int page(int i, int x) const { return __shfl_sync(0xffffffffu, now, (i % kTurns) * H + x); }
};

// ------------------------------------------------------------------ warp-level pieces
// 16 bytes from global into shared memory, `bytes` of them read, zeros behind.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// c += A (16 x 16) B (16 x 8), fp32 sums.  HALF: fp16 operands, else bf16.
template <bool HALF>
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    if (HALF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four e4m3 values as two pairs of fp16 values, exactly (NaN stays NaN).
__device__ __forceinline__ void e4m3x4_half2(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(x));
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ float2 half2_floats(uint32_t x) {
    float2 y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(y.x), "=f"(y.y) : "r"(x));
    return y;
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// A 16-row tile of keys or values in shared memory.  A warp copies its own tiles with coalesced
// 16-byte copies (consecutive lanes, consecutive chunks: the tile is contiguous in its page) and
// reads them back as fragments; `place` is where a row's 16-byte chunk lies, such that both the copies
// and the fragment loads touch every bank once.  (Copying straight into fragment order instead,
// lane by lane, costs the value tiles four sectors of four different lines per quarter-warp:
// 219 against 168 us for 131072 keys of 16 heads.)
//
// Keys: the product is S^T = K Q^T: 16 keys are the M rows, 8 query rows the N columns.  Lane (g, t)
// = (lane / 4, lane % 4) of an A fragment holds columns of keys g and g + 8; which columns of d the
// 16 slots of a k-step stand for is free as long as K and Q agree, so the lane takes 16
// contiguous bytes of a key row (chunk u: bytes [64u + 16t, +16)) as its slots of 2 (bf16) or 4
// (e4m3) k-steps.  The 8 lanes of a load phase meet chunks t of two neighbouring rows.
// Where a lane's chunk lies splits into a lane's constant, computed once per kernel, and compile-time
// offsets; `place` states the layout, and the static functions below follow it.
template <int D, bool F8>
struct RowTile {
    static constexpr int kRow = D * (F8 ? 1 : 2);     // bytes of a row
    static constexpr int kRowChunks = kRow / 16;
    static constexpr int kBytes = kTileKeys * kRow;   // of a tile
    static constexpr int kCopies = kBytes / 512;      // of a lane: copy i is 512 / kRow rows further
    static constexpr int kStep = 512 / kRow;

    __device__ static __forceinline__ int copy_row(int lane) { return lane / kRowChunks; }
};

template <int D, bool F8>
struct KeyTile : RowTile<D, F8> {
    using R = RowTile<D, F8>;
    static constexpr int kChunks = R::kRow / 64;      // 16-byte chunks of a row per lane
    static constexpr int kElems = F8 ? 16 : 8;        // elements of a chunk
    static constexpr int kSteps = kElems / 4;         // k-steps of a chunk

    __device__ static __forceinline__ int place(int row, int chunk) {
        return row * R::kRow + ((R::kRow >= 128 ? chunk ^ ((row & 1) * 4) : chunk) * 16);
    }
    __device__ static __forceinline__ int copy_offset(int lane) { return place(R::copy_row(lane), lane % R::kRowChunks); }
    // dst: the tile + copy_offset; from: the tile's first row + lane * 16; valid: rows that exist (zeros behind)
    __device__ static __forceinline__ void copy(uint32_t dst, const uint8_t* from, int valid, int lane) {
        if (valid >= kTileKeys) {
#pragma unroll
            for (int i = 0; i < R::kCopies; ++i) cp_async16(dst + i * 512, from + i * 512);
        } else {
#pragma unroll
            for (int i = 0; i < R::kCopies; ++i)
                cp_async16(dst + i * 512, from + i * 512, i * R::kStep + R::copy_row(lane) < valid ? 16 : 0);
        }
    }
    // chunk u of key g + 8h lies at load_offset(lane, u & 1) + load_step(h, u)
    __device__ static __forceinline__ int load_offset(int lane, int odd) { return place(lane >> 2, (lane & 3) + 4 * odd); }
    __device__ static constexpr int load_step(int h, int u) { return h * 8 * R::kRow + (u >> 1) * 128; }
};

// Power of two that brings a query row's largest magnitude into [2^14, 2^15): e4m3 keys meet
// the query in fp16 (the type that holds e4m3 exactly), and a row scaled so keeps every bf16
// bit of elements down to 2^-29 of its largest and loses at most 2^-40 of it below.
// top: largest finite magnitude of the row, 2^(e-127) <= top < 2^(e-126).  The exponent is kept at
// -110 or more so that both the scale and its inverse are normal numbers.
__device__ __forceinline__ int query_exponent(float top) {
    const int e = (int)(__float_as_uint(top) >> 23) - 127 - 14;
    return top > 0.f ? max(e, -110) : 0;
}

// 2^e for an exponent byte e + 127 of 1..254.
__device__ __forceinline__ float exp_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// 2^n for any n up to 127, by way of the subnormal numbers and never 0.
__device__ __forceinline__ float pow2_down(int n) { return n >= -126 ? pow2(n) : __uint_as_float(1u << max(n + 149, 0)); }

// How an e4m3 key's product with a stretched query row becomes a score in base 2: times
// (mant * 2^c * the key's scale), which is rounded, times 2^(e + exp - c), the row's, which is exact.
// c = -24 keeps the first factor in range for any row: a product is below 2^31, so with scales of
// 2^-96 to 2^120 neither it nor its factor overflows or loses bits, and a score is right however large its
// key and small its query are, or the other way round.  Only where a row of the block exceeds 2^118 or so, c
// is higher, for the row's factor to exist.
struct ScoreScale {
    float key;       // to be multiplied by the key's scale
    int shift;       // of a row's e

    // e: exponents (Queries::fragments) of the lane's rows 2t + j of every block; all lanes call
    template <int NT>
    __device__ __forceinline__ void start(const PagedParams& p, const int (*e)[2]) {
        int top = e[0][0];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top = max(top, max(e[nt][0], e[nt][1]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int c = max(-24, top + p.exp - 127);
        key = p.mant * pow2(c);
        shift = p.exp - c;
    }
    __device__ __forceinline__ float row(int e) const { return pow2_down(e + shift); }
};

__device__ __forceinline__ float finite_abs(uint32_t bf16_bits) {   // 0 for infinities and NaN
    const uint32_t x = bf16_bits & 0x7fffu;
    return x >= 0x7f80u ? 0.f : __uint_as_float(x << 16);
}

// 8 query rows as B fragments for KeyTile<D, F8>, in two steps: the loads are issued before a segment's first
// keys are requested, or they would queue behind the megabytes that all CTAs request at once (measured:
// 5 us instead of under 1), and turned into fragments after.
template <int D, bool F8>
struct Queries {
    static constexpr int kLoads = D / 32;      // 16-byte loads of a row per lane
    uint4 v[kLoads];

    // rows row0 .. row0 + 7 of the KV head's contiguous rows q; rows past `rows` are zeros
    __device__ __forceinline__ void load(const uint16_t* q, int row0, int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const bool have = row0 + g < rows;
        const uint16_t* src = q + (size_t)(row0 + g) * D;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            // bf16 keys: chunk u covers columns [32u + 8t, +8); e4m3: [64(u/2) + 16t + 8(u%2), +8)
            const int col = F8 ? (u >> 1) * 64 + t * 16 + (u & 1) * 8 : u * 32 + t * 8;
            v[u] = have ? *reinterpret_cast<const uint4*>(src + col) : make_uint4(0, 0, 0, 0);
        }
    }
    // frag[s] of every k-step; returns the exponent e of the power of two by which the products of row lane / 4
    // are to be multiplied (e4m3 keys)
    __device__ __forceinline__ int fragments(uint2* frag) const {
        if (!F8) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
                frag[2 * u] = make_uint2(v[u].x, v[u].y);
                frag[2 * u + 1] = make_uint2(v[u].z, v[u].w);
            }
            return 0;
        }
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(finite_abs(w[i]), finite_abs(w[i] >> 16)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = query_exponent(top);
        const float inv = pow2(-e);
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = pack_half(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
            frag[2 * u] = make_uint2(h[0], h[1]);
            frag[2 * u + 1] = make_uint2(h[2], h[3]);
        }
        return e;
    }
};

}  // namespace skl
