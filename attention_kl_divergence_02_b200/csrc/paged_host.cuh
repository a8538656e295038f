// paged_host.cuh -- host side of the paged-cache entry points: argument checks and launches.
// Included once, at the end of streamkl.cu.
#pragma once

namespace {

constexpr int kWholeFew = 3, kWholeMany = 8;      // units
constexpr int kJoinApart = 256;      // states * rows of a segment beyond which the join is a kernel of its own
constexpr int kPagedMaxCtas = 4;     // most resident CTAs per SM of any variant

int page_shift_of(int n) {
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

// Query rows are folded in blocks of 8 n.  Attention: n = 1 to 4, the fewest blocks that hold a KV head's rows (beyond
// 32 rows, blocks of 32 and a rest in one of 32 too).
// Divergence: 1 or 2; more rows are several blocks, which read the keys again, from L2, since the CTAs
// that do the blocks of one head run side by side (32 rows over 64 x 8192 bf16 keys of d = 128: 52 us, and
// 65 with one block of 32, whose query fragments do not fit the registers).
int paged_row_tiles(long long rows, bool divergence) {
    const int most = divergence ? 2 : 4;
    return (int)std::min<long long>((rows + 7) / 8, most);
}

// The counters at the head of a workspace, one per CTA: a fixed size, so that every call keeps them in one
// place; a GPU has at most kPagedMaxSms SMs here.
constexpr int kPagedMaxSms = (int)(STREAMKL_PAGED_COUNTER_BYTES / sizeof(unsigned)) / kPagedMaxCtas;
int paged_sms() { return std::min(num_sms(), kPagedMaxSms); }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// As a programmatic dependent of what ran before on the stream: see wait_for_stream.
template <typename P>
cudaError_t launch_after(void (*kernel)(P), dim3 grid, int threads, int smem, const P& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess) cudaGetLastError();      // it is returned here and must not meet a later check
    return e;
}

// Launches a kernel whose shared memory needs an attribute that lasts as long as the device's context.  These
// calls are made per token, so it is set once per kernel and device (`done`, a bit per device) and
// again where a launch fails without it (after a cudaDeviceReset).
template <typename K>
int launch_main(K kernel, int smem, const skl::PagedParams& p, cudaStream_t st, std::atomic<unsigned long long>& done,
                const char* what) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    for (bool set = (done.load(std::memory_order_relaxed) & bit) == 0;; set = true) {
        if (set) {
            const int rc = set_smem(kernel, smem);
            if (rc) return rc;
            done.fetch_or(bit, std::memory_order_relaxed);
        }
        e = launch_after(kernel, dim3((unsigned)p.grid), skl::kPagedThreads, smem, p, st);
        if (e == cudaSuccess) return STREAMKL_OK;
        if (set) return cuda_fail(e, what);
    }
}

// The grid, and whether segments are dealt out whole instead of in equal shares: where all are short, since a
// whole segment needs no plan, partial state or join.  Measured, 8 KV heads, d = 128, attention over
// bf16 (e4m3), whole against shares, us: one sequence of 128 keys 4.1 against 5.8, 256 keys 5.4 against 5.9
// (5.9 against 7.1), 512 keys 8.1 against 6.3 (8.1 against 7.1); 32 sequences of 512 keys 14.0 against 17.1
// (9.7 against 12.7).  Units are 64 (128) keys.  With enough segments to fill half the grid, eight units
// bound what uneven lengths can cost.  The host knows the table's width and not the lengths: behind a table that is
// kept wider than the batch needs, as in a captured step, short sequences take the shares.
template <int UNIT>
void paged_grid(skl::PagedParams* p, int ctas) {
    const long long units = ((long long)p->width * p->page_size + UNIT - 1) / UNIT;
    const long long segments = (long long)p->B * p->Hkv * p->rblocks;
    p->grid = ctas * paged_sms();
    p->whole = units <= (2 * segments >= p->grid ? kWholeMany : kWholeFew) ? 1 : 0;
    if (p->whole) p->grid = (int)std::min<long long>(p->grid, segments);
}

int check_cache(const streamkl_cache* c, bool values) {
    if (!c || !c->k || (values && !c->v)) return STREAMKL_ERR_INVALID_ARG;
    if (c->type != STREAMKL_CACHE_BF16 && c->type != STREAMKL_CACHE_E4M3) return STREAMKL_ERR_INVALID_ARG;
    if (c->pages < 1 || c->page_size < 1 || c->Hkv < 1 || c->d < 1) return STREAMKL_ERR_INVALID_ARG;
    if (c->type == STREAMKL_CACHE_E4M3 && (!c->k_exp || (values && !c->v_exp))) return STREAMKL_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return STREAMKL_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return STREAMKL_ERR_UNSUPPORTED;
    if ((double)c->pages * c->Hkv * c->page_size >= 2147483648.0) return STREAMKL_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->k_exp) || (values && (!aligned16(c->v) || !aligned16(c->v_exp))))
        return STREAMKL_ERR_UNSUPPORTED;
    return STREAMKL_OK;
}

int check_table(const streamkl_cache* c, const int* table, int width, int B) {
    if (!table || width < 1 || B < 1) return STREAMKL_ERR_INVALID_ARG;
    if ((long long)width * c->page_size > (1ll << 30)) return STREAMKL_ERR_UNSUPPORTED;
    return STREAMKL_OK;
}

int cache_move(const streamkl_cache* c, const uint16_t* k, const uint16_t* v, const int* table, int width,
               const int* start, const int* count, int B, int NT, bool append, void* stream) {
    int rc = check_cache(c, true);
    if (rc) return rc;
    if ((rc = check_table(c, table, width, B))) return rc;
    if (!k || !v || NT < 1) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return STREAMKL_ERR_UNSUPPORTED;
    if ((long long)B * c->Hkv * NT >= (1ll << 31)) return STREAMKL_ERR_UNSUPPORTED;
    skl::CacheParams p;
    p.rows[0] = static_cast<uint8_t*>(c->k);
    p.rows[1] = static_cast<uint8_t*>(c->v);
    p.exps[0] = c->k_exp;
    p.exps[1] = c->v_exp;
    p.dense[0] = const_cast<uint16_t*>(k);
    p.dense[1] = const_cast<uint16_t*>(v);
    p.table = table;
    p.start = start;
    p.count = count;
    p.B = B; p.Hkv = c->Hkv; p.NT = NT; p.width = width; p.pages = c->pages;
    p.page_size = c->page_size;
    p.page_shift = page_shift_of(c->page_size);
    const bool f8 = c->type == STREAMKL_CACHE_E4M3;
    // an append to an e4m3 cache takes 16 elements a lane, everything else 8
    const int tokens = c->d == 128 ? (append && f8 ? skl::CacheCfg<128, 16>::kTokens : skl::CacheCfg<128, 8>::kTokens)
                                   : (append && f8 ? skl::CacheCfg<64, 16>::kTokens : skl::CacheCfg<64, 8>::kTokens);
    const long long warps = (long long)B * c->Hkv * ((NT + tokens - 1) / tokens);
    const int per = skl::kCacheThreads / 32;
    const int grid = (int)((warps + per - 1) / per);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    auto kernel = c->d == 128 ? (f8 ? (append ? skl::streamkl_cache_append_kernel<128, true> : skl::streamkl_cache_gather_kernel<128, true>)
                                    : (append ? skl::streamkl_cache_append_kernel<128, false> : skl::streamkl_cache_gather_kernel<128, false>))
                              : (f8 ? (append ? skl::streamkl_cache_append_kernel<64, true> : skl::streamkl_cache_gather_kernel<64, true>)
                                    : (append ? skl::streamkl_cache_append_kernel<64, false> : skl::streamkl_cache_gather_kernel<64, false>));
    const cudaError_t e = launch_after(kernel, dim3((unsigned)grid), skl::kCacheThreads, 0, p, st);
    if (e != cudaSuccess) return cuda_fail(e, append ? "streamkl_cache_append launch" : "streamkl_cache_gather launch");
    return STREAMKL_OK;
}

// Checks and fills what attention and divergence share.
int paged_params(const streamkl_cache* c, const int* table, int width, const int* lengths, int B, int Hq, int NQ,
                 float scale, int causal, bool divergence, void* workspace, size_t workspace_bytes,
                 skl::PagedParams* p) {
    int rc = check_table(c, table, width, B);
    if (rc) return rc;
    if (!lengths || Hq < 1 || NQ < 1) return STREAMKL_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale)) return STREAMKL_ERR_UNSUPPORTED;
    if (Hq % c->Hkv != 0) return STREAMKL_ERR_UNSUPPORTED;
    if ((long long)B * Hq * NQ >= (1ll << 31)) return STREAMKL_ERR_UNSUPPORTED;
    const long long rows = (long long)(Hq / c->Hkv) * NQ;
    const int nt = paged_row_tiles(rows, divergence);
    const long long rblocks = (rows + 8 * nt - 1) / (8 * nt);
    const long long most = ((long long)width * c->page_size + 63) / 64 + 16;   // the smallest unit; PagedPlan's START
    if ((double)B * c->Hkv * (double)rblocks * (double)most >= 2147483648.0) return STREAMKL_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < streamkl_paged_workspace_bytes(B, Hq, c->Hkv, NQ, c->d))
        return STREAMKL_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return STREAMKL_ERR_UNSUPPORTED;
    p->table = table;
    p->lengths = lengths;
    p->B = B; p->Hkv = c->Hkv; p->NQ = NQ;
    p->rows = (int)rows;
    p->rblocks = (int)rblocks;
    p->width = width;
    p->pages = c->pages;
    p->page_size = c->page_size;
    p->page_shift = page_shift_of(c->page_size);
    p->causal = causal ? 1 : 0;
    p->sl2 = scale * 1.4426950408889634f;
    if (!std::isfinite(p->sl2)) return STREAMKL_ERR_UNSUPPORTED;
    p->mant = 2.f * std::frexp(p->sl2, &p->exp);
    p->exp -= 1;
    p->arrived = static_cast<unsigned*>(workspace);
    p->part = reinterpret_cast<float*>(static_cast<char*>(workspace) + STREAMKL_PAGED_COUNTER_BYTES);
    return STREAMKL_OK;
}

template <int D, bool F8, int NT>
int launch_paged_attn(skl::PagedParams p, cudaStream_t st) {
    using C = skl::AttnCfg<D, F8, NT>;
    static_assert(C::kCtas <= kPagedMaxCtas, "workspace");
    static std::atomic<unsigned long long> done{0};
    paged_grid<C::kUnit>(&p, C::kCtas);
    const long long segments = (long long)p.B * p.Hkv * p.rblocks;
    const long long states = (p.grid + segments - 1) / segments + 1;      // of a segment, about
    const int rows = std::min(p.rows, 8 * NT);
    const bool apart = !p.whole && states * rows > kJoinApart;
    if (apart) p.arrived = nullptr;
    const int rc = launch_main(skl::streamkl_paged_attn_kernel<D, F8, NT>, C::kSmem, p, st, done, "streamkl_paged_attn launch");
    if (rc || !apart) return rc;
    // where a segment has many states, each of its rows gets a CTA
    const int gy = states > 16 ? rows : NT;
    const cudaError_t e = launch_after(skl::streamkl_paged_attn_join_kernel<D, NT, C::kUnit, C::kStart>,
                                       dim3((unsigned)(p.grid - 1), (unsigned)gy), skl::kJoinThreads, 0, p, st);
    return e == cudaSuccess ? STREAMKL_OK : cuda_fail(e, "streamkl_paged_attn join launch");
}

template <int D, bool F8>
int launch_paged_attn_rows(const skl::PagedParams& p, cudaStream_t st) {
    switch (paged_row_tiles(p.rows, false)) {
        case 1: return launch_paged_attn<D, F8, 1>(p, st);
        case 2: return launch_paged_attn<D, F8, 2>(p, st);
        case 3: return launch_paged_attn<D, F8, 3>(p, st);
        default: return launch_paged_attn<D, F8, 4>(p, st);
    }
}

template <int D, bool F1, bool F2, bool SHARED, int NT>
int launch_paged_kl(skl::PagedParams p, cudaStream_t st) {
    using C = skl::KlCfg<D, F1, F2, SHARED, NT>;
    static_assert(C::kCtas <= kPagedMaxCtas, "workspace");
    static std::atomic<unsigned long long> done{0};
    paged_grid<C::kUnit>(&p, C::kCtas);
    return launch_main(skl::streamkl_paged_kl_kernel<D, F1, F2, SHARED, NT>, C::kSmem, p, st, done, "streamkl_paged_kl launch");
}

template <int D, bool F1, bool F2, bool SHARED>
int launch_paged_kl_rows(const skl::PagedParams& p, cudaStream_t st) {
    return paged_row_tiles(p.rows, true) == 1 ? launch_paged_kl<D, F1, F2, SHARED, 1>(p, st)
                                              : launch_paged_kl<D, F1, F2, SHARED, 2>(p, st);
}

template <int D>
int launch_paged_kl_types(const skl::PagedParams& p, bool f1, bool f2, bool shared, cudaStream_t st) {
    if (shared) return f1 ? launch_paged_kl_rows<D, true, true, true>(p, st) : launch_paged_kl_rows<D, false, false, true>(p, st);
    if (f1) return f2 ? launch_paged_kl_rows<D, true, true, false>(p, st) : launch_paged_kl_rows<D, true, false, false>(p, st);
    return f2 ? launch_paged_kl_rows<D, false, true, false>(p, st) : launch_paged_kl_rows<D, false, false, false>(p, st);
}

}  // namespace

extern "C" {

int streamkl_cache_append(const streamkl_cache* cache, const uint16_t* k, const uint16_t* v, const int* table,
                          int width, const int* start, const int* count, int B, int NT, void* stream) {
    return cache_move(cache, k, v, table, width, start, count, B, NT, true, stream);
}

int streamkl_cache_gather(const streamkl_cache* cache, const int* table, int width, const int* start,
                          const int* count, int B, int NT, uint16_t* k, uint16_t* v, void* stream) {
    return cache_move(cache, k, v, table, width, start, count, B, NT, false, stream);
}

size_t streamkl_paged_workspace_bytes(int B, int Hq, int Hkv, int NQ, int d) {
    if (B < 1 || Hq < 1 || Hkv < 1 || NQ < 1 || Hq % Hkv || (d != 64 && d != 128)) return 0;
    const long long rows = (long long)(Hq / Hkv) * NQ;
    return STREAMKL_PAGED_COUNTER_BYTES + (size_t)kPagedMaxCtas * paged_sms() * 2 * 8 * paged_row_tiles(rows, false) * (d + 4) * sizeof(float);
}

int streamkl_paged_attn(const streamkl_cache* cache, const uint16_t* q, const int* table, int width,
                        const int* lengths, int B, int Hq, int NQ, float scale, int causal, uint16_t* out,
                        float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !out || !lse) return STREAMKL_ERR_INVALID_ARG;
    int rc = check_cache(cache, true);
    if (rc) return rc;
    if (!aligned16(q) || !aligned16(out) || !aligned4(lse)) return STREAMKL_ERR_UNSUPPORTED;
    skl::PagedParams p = {};
    if ((rc = paged_params(cache, table, width, lengths, B, Hq, NQ, scale, causal, false, workspace, workspace_bytes, &p)))
        return rc;
    p.a = {static_cast<const uint8_t*>(cache->k), cache->k_exp};
    p.b = {static_cast<const uint8_t*>(cache->v), cache->v_exp};
    p.q1 = q;
    p.out = out;
    p.lse1 = lse;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f8 = cache->type == STREAMKL_CACHE_E4M3;
    if (cache->d == 128) return f8 ? launch_paged_attn_rows<128, true>(p, st) : launch_paged_attn_rows<128, false>(p, st);
    return f8 ? launch_paged_attn_rows<64, true>(p, st) : launch_paged_attn_rows<64, false>(p, st);
}

int streamkl_paged_kl(const streamkl_cache* cache1, const uint16_t* q1, const streamkl_cache* cache2,
                      const uint16_t* q2, const int* table, int width, const int* lengths, int B, int Hq, int NQ,
                      float scale, int causal, float* kl, float* lse1, float* lse2, void* workspace,
                      size_t workspace_bytes, void* stream) {
    if (!q1 || !q2 || !kl || !lse1 || !lse2) return STREAMKL_ERR_INVALID_ARG;
    int rc = check_cache(cache1, false);
    if (rc) return rc;
    if ((rc = check_cache(cache2, false))) return rc;
    if (cache1->pages != cache2->pages || cache1->page_size != cache2->page_size || cache1->Hkv != cache2->Hkv ||
        cache1->d != cache2->d)
        return STREAMKL_ERR_UNSUPPORTED;
    const bool shared = cache1->k == cache2->k;
    if (shared && (cache1->type != cache2->type || cache1->k_exp != cache2->k_exp)) return STREAMKL_ERR_INVALID_ARG;
    if (!aligned16(q1) || !aligned16(q2) || !aligned4(kl) || !aligned4(lse1) || !aligned4(lse2))
        return STREAMKL_ERR_UNSUPPORTED;
    skl::PagedParams p = {};
    if ((rc = paged_params(cache1, table, width, lengths, B, Hq, NQ, scale, causal, true, workspace, workspace_bytes, &p)))
        return rc;
    p.a = {static_cast<const uint8_t*>(cache1->k), cache1->k_exp};
    p.b = {static_cast<const uint8_t*>(cache2->k), cache2->k_exp};
    p.q1 = q1;
    p.q2 = q2;
    p.kl = kl;
    p.lse1 = lse1;
    p.lse2 = lse2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f1 = cache1->type == STREAMKL_CACHE_E4M3, f2 = cache2->type == STREAMKL_CACHE_E4M3;
    return cache1->d == 128 ? launch_paged_kl_types<128>(p, f1, f2, shared, st)
                            : launch_paged_kl_types<64>(p, f1, f2, shared, st);
}

}  // extern "C"
