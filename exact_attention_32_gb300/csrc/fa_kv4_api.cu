// C ABI of the 4-bit KV cache and of fa_key_weights: argument validation and
// dispatch, in the order of fa_api.cu (sizes, then device, pointers, overlaps).
// The operations and every argument are documented in include/fa.h.
#include <math.h>
#include <stdint.h>

#include "fa.h"
#include "fa_internal.h"

namespace {

// Tokens of a sequence: positions, and what loops over them step beyond (up to 2^18), fit 31 bits.
constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (1 << 20);

int check_cache_sizes(const fa_kv4_cache *c)
{
    if (c == nullptr || c->n_pages < 1 || c->Hkv < 1 || c->d < 1) return FA_ERR_INVALID_ARG;
    if (c->n_pages > 0x7fffffffLL || c->Hkv > (int64_t(1) << 20)) return FA_ERR_INVALID_ARG;
    const int64_t P = c->page_size;
    if (P < 16 || P > 1024 || (P & (P - 1)) != 0) return FA_ERR_INVALID_ARG;
    if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
    if (c->n_pages * c->Hkv > (int64_t(1) << 44) / (P * c->d)) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

// B sequences over a page table of max_pages columns: every position fits 31 bits.
int check_table_sizes(const fa_kv4_cache *c, int64_t B, int64_t max_pages)
{
    if (B < 1 || max_pages < 1 || B > (int64_t(1) << 31) / c->Hkv) return FA_ERR_INVALID_ARG;
    if (max_pages > kMaxTokens / c->page_size) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

Kv4Cache view(const fa_kv4_cache *c)
{
    Kv4Cache v;
    v.k = static_cast<uint8_t *>(c->k);
    v.v = static_cast<uint8_t *>(c->v);
    v.k_scale = static_cast<uint8_t *>(c->k_scale);
    v.v_scale = static_cast<uint8_t *>(c->v_scale);
    v.weights = c->weights;
    v.n_pages = static_cast<int>(c->n_pages);
    v.heads = static_cast<int>(c->Hkv);
    v.log2_page = 0;
    while ((int64_t(1) << v.log2_page) < c->page_size) ++v.log2_page;
    v.d = static_cast<int>(c->d);
    return v;
}

struct Range {
    const void *p;
    uint64_t bytes;
};

// The cache's arrays (the weights last, null bytes without them).
void cache_ranges(const fa_kv4_cache *c, Range (&r)[5])
{
    const uint64_t rows = static_cast<uint64_t>(c->n_pages * c->Hkv * c->page_size);
    const uint64_t d = static_cast<uint64_t>(c->d);
    r[0] = {c->k, rows * d / 2};
    r[1] = {c->v, rows * d / 2};
    r[2] = {c->k_scale, rows * d / 32};
    r[3] = {c->v_scale, rows};
    r[4] = {c->weights, c->weights != nullptr ? rows * 4 : 0};
}

int check_cache_pointers(const fa_kv4_cache *c, int dev)
{
    int st;
    for (const void *p : {static_cast<const void *>(c->k), static_cast<const void *>(c->v)})
        if ((st = fa_check_device_pointer(p, dev, 32)) != FA_OK) return st;  // what a TMA of 4-bit values asks for
    for (const void *p : {static_cast<const void *>(c->k_scale), static_cast<const void *>(c->v_scale)})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    if (c->weights != nullptr) return fa_check_device_pointer(c->weights, dev, 16);
    return FA_OK;
}

bool meet(const Range &a, const Range &b) { return a.bytes != 0 && b.bytes != 0 && fa_ranges_overlap(a.p, a.bytes, b.p, b.bytes); }

// No output meets an input or another output.
template <int NO, int NI>
bool outputs_clear(const Range (&out)[NO], const Range (&in)[NI])
{
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < NI; ++j)
            if (meet(out[i], in[j])) return false;
        for (int j = i + 1; j < NO; ++j)
            if (meet(out[i], out[j])) return false;
    }
    return true;
}

uint64_t bytes(int64_t n) { return static_cast<uint64_t>(n); }

}  // namespace

extern "C" int fa_kv4_append(const fa_kv4_cache *cache, const void *k_new, const void *v_new, const float *w_new,
                             const int32_t *n_new, const int32_t *lens, const int32_t *page_table, int64_t B,
                             int64_t S, int64_t max_pages, void *stream)
{
    int st = check_cache_sizes(cache);
    if (st != FA_OK || (st = check_table_sizes(cache, B, max_pages)) != FA_OK) return st;
    if (S < 1 || S > kMaxTokens || B * cache->Hkv > (int64_t(1) << 40) / (S * cache->d)) return FA_ERR_INVALID_ARG;
    if (w_new != nullptr && cache->weights == nullptr) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = check_cache_pointers(cache, dev)) != FA_OK) return st;
    for (const void *p : {k_new, v_new})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(lens), static_cast<const void *>(page_table)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(w_new), static_cast<const void *>(n_new)})
        if (p != nullptr && (st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    Range out[5];
    cache_ranges(cache, out);
    const int64_t rows = B * cache->Hkv * S;
    const Range in[6] = {{k_new, bytes(rows * cache->d * 2)},       {v_new, bytes(rows * cache->d * 2)},
                         {w_new, w_new ? bytes(rows * 4) : 0},      {n_new, n_new ? bytes(B * 4) : 0},
                         {lens, bytes(B * 4)},                      {page_table, bytes(B * max_pages * 4)}};
    if (!outputs_clear(out, in)) return FA_ERR_INVALID_ARG;
    return fa_launch_kv4_append(view(cache), k_new, v_new, w_new, n_new, lens, page_table, B, S, max_pages, sm_count,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK
               : FA_ERR_LAUNCH;
}

extern "C" int fa_kv4_read(const fa_kv4_cache *cache, const int32_t *first, const int32_t *lens,
                           const int32_t *page_table, int64_t B, int64_t max_pages, int64_t T, void *k_out,
                           void *v_out, void *stream)
{
    int st = check_cache_sizes(cache);
    if (st != FA_OK || (st = check_table_sizes(cache, B, max_pages)) != FA_OK) return st;
    if (T < 1 || T > kMaxTokens || B * cache->Hkv > (int64_t(1) << 40) / (T * cache->d)) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = check_cache_pointers(cache, dev)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(k_out), static_cast<const void *>(v_out)})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(lens), static_cast<const void *>(page_table)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    if (first != nullptr && (st = fa_check_device_pointer(first, dev, 4)) != FA_OK) return st;
    Range c[5];
    cache_ranges(cache, c);
    const int64_t ob = B * cache->Hkv * T * cache->d * 2;
    const Range out[2] = {{k_out, bytes(ob)}, {v_out, bytes(ob)}};
    const Range in[7] = {c[0], c[1], c[2], c[3], {first, first ? bytes(B * 4) : 0}, {lens, bytes(B * 4)},
                         {page_table, bytes(B * max_pages * 4)}};
    if (!outputs_clear(out, in)) return FA_ERR_INVALID_ARG;
    return fa_launch_kv4_read(view(cache), first, lens, page_table, B, max_pages, T, k_out, v_out, sm_count,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK
               : FA_ERR_LAUNCH;
}

namespace {

int check_decode_sizes(int64_t B, int64_t H, int64_t Hkv, int64_t n_q, int64_t d, int64_t max_tokens, int accumulate)
{
    if (B < 1 || H < 1 || Hkv < 1 || n_q < 1 || d < 1 || max_tokens < 1) return FA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
    if (Hkv > (int64_t(1) << 20) || H % Hkv != 0 || n_q > 64 || H / Hkv > 1024 / n_q) return FA_ERR_INVALID_ARG;
    if (max_tokens > kMaxTokens || (accumulate != 0 && accumulate != 1)) return FA_ERR_INVALID_ARG;
    if (B > (int64_t(1) << 31) / (H * n_q) || B * H * n_q > (int64_t(1) << 40) / max_tokens) return FA_ERR_INVALID_ARG;
    return FA_OK;
}

}  // namespace

extern "C" int64_t fa_fwd_kv4_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t n_q, int64_t d,
                                              int64_t max_tokens, int accumulate)
{
    if (check_decode_sizes(B, H, Hkv, n_q, d, max_tokens, accumulate) != FA_OK) return -1;
    return fa_kv4_decode_workspace(B, H, Hkv, n_q, d, max_tokens, accumulate, false);
}

extern "C" int64_t fa_fwd_kv4_tree_workspace_bytes(int64_t B, int64_t H, int64_t Hkv, int64_t n_q, int64_t d, int64_t max_tokens)
{
    if (check_decode_sizes(B, H, Hkv, n_q, d, max_tokens, 0) != FA_OK) return -1;
    return fa_kv4_decode_workspace(B, H, Hkv, n_q, d, max_tokens, 0, true);
}

namespace {

// fa_fwd_kv4, and with masks fa_fwd_kv4_tree.
int attend(const void *q, const fa_kv4_cache *cache, const int32_t *lens, const int32_t *page_table, const uint64_t *tree,
           const int32_t *n_new, void *o, float *lse, int64_t B, int64_t H, int64_t n_q, int64_t max_pages, float scale,
           int accumulate, void *workspace, int64_t workspace_bytes, void *stream)
{
    int st = check_cache_sizes(cache);
    if (st != FA_OK || (st = check_table_sizes(cache, B, max_pages)) != FA_OK) return st;
    const int64_t max_tokens = max_pages * cache->page_size;
    if ((st = check_decode_sizes(B, H, cache->Hkv, n_q, cache->d, max_tokens, accumulate)) != FA_OK) return st;
    if (!(scale > 0.f) || !isfinite(scale)) return FA_ERR_INVALID_ARG;
    if (accumulate && cache->weights == nullptr) return FA_ERR_INVALID_ARG;
    const int64_t need = fa_kv4_decode_workspace(B, H, cache->Hkv, n_q, cache->d, max_tokens, accumulate, tree != nullptr);
    if (workspace_bytes < need) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = check_cache_pointers(cache, dev)) != FA_OK) return st;
    for (const void *p : {q, static_cast<const void *>(o), static_cast<const void *>(workspace)})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(lse), static_cast<const void *>(lens),
                          static_cast<const void *>(page_table)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    if (tree != nullptr && (st = fa_check_device_pointer(tree, dev, 8)) != FA_OK) return st;
    if (n_new != nullptr && (st = fa_check_device_pointer(n_new, dev, 4)) != FA_OK) return st;
    Range c[5];
    cache_ranges(cache, c);
    const int64_t rows = B * H * n_q;
    const Range out[4] = {{o, bytes(rows * cache->d * 2)}, {lse, bytes(rows * 4)}, {workspace, bytes(need)},
                          {c[4].p, accumulate ? c[4].bytes : 0}};
    const Range in[9] = {{q, bytes(rows * cache->d * 2)}, c[0], c[1], c[2], c[3], {lens, bytes(B * 4)},
                         {page_table, bytes(B * max_pages * 4)}, {tree, tree ? bytes(B * n_q * 8) : 0},
                         {n_new, n_new ? bytes(B * 4) : 0}};
    if (!outputs_clear(out, in)) return FA_ERR_INVALID_ARG;
    Kv4DecodeProblem p;
    p.cache = view(cache);
    p.q = q;
    p.lens = lens;
    p.table = page_table;
    p.o = o;
    p.lse = lse;
    p.B = B;
    p.H = H;
    p.n_q = n_q;
    p.max_pages = max_pages;
    p.scale = scale;
    p.accumulate = accumulate;
    p.tree = tree;
    p.n_new = n_new;
    return fa_launch_kv4_decode(p, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

// Two caches of one layout: the same pool, or arrays apart.
int check_same_layout(const fa_kv4_cache *a, const fa_kv4_cache *b)
{
    return a->Hkv == b->Hkv && a->page_size == b->page_size && a->d == b->d ? FA_OK : FA_ERR_INVALID_ARG;
}
bool one_pool_or_two(const Range (&a)[5], const Range (&b)[5])
{
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < 5; ++j)
            if (meet(a[i], b[j]) && !(i == j && a[i].p == b[j].p)) return false;
    return true;
}

}  // namespace

extern "C" int fa_fwd_kv4(const void *q, const fa_kv4_cache *cache, const int32_t *lens, const int32_t *page_table,
                          void *o, float *lse, int64_t B, int64_t H, int64_t n_q, int64_t max_pages, float scale,
                          int accumulate, void *workspace, int64_t workspace_bytes, void *stream)
{
    return attend(q, cache, lens, page_table, nullptr, nullptr, o, lse, B, H, n_q, max_pages, scale, accumulate, workspace,
                  workspace_bytes, stream);
}

extern "C" int fa_fwd_kv4_tree(const void *q, const fa_kv4_cache *cache, const int32_t *lens, const int32_t *page_table,
                               const uint64_t *tree, const int32_t *n_new, void *o, float *lse, int64_t B, int64_t H,
                               int64_t n_q, int64_t max_pages, float scale, void *workspace, int64_t workspace_bytes,
                               void *stream)
{
    if (tree == nullptr) return FA_ERR_INVALID_ARG;
    return attend(q, cache, lens, page_table, tree, n_new, o, lse, B, H, n_q, max_pages, scale, 0, workspace, workspace_bytes, stream);
}

extern "C" int fa_kv4_keep(const fa_kv4_cache *cache, const int32_t *lens, const int32_t *page_table, int64_t max_pages,
                           const int32_t *path, const int32_t *n_path, const int32_t *n_new, int64_t B, int64_t n_draft,
                           int32_t *new_lens, void *stream)
{
    int st = check_cache_sizes(cache);
    if (st != FA_OK || (st = check_table_sizes(cache, B, max_pages)) != FA_OK) return st;
    if (n_draft < 1 || n_draft > 64) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = check_cache_pointers(cache, dev)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(lens), static_cast<const void *>(page_table), static_cast<const void *>(path),
                          static_cast<const void *>(n_path), static_cast<const void *>(new_lens)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    if (n_new != nullptr && (st = fa_check_device_pointer(n_new, dev, 4)) != FA_OK) return st;
    Range c[5];
    cache_ranges(cache, c);
    const Range out[6] = {c[0], c[1], c[2], c[3], c[4], {new_lens, bytes(B * 4)}};
    const Range in[5] = {{lens, bytes(B * 4)}, {page_table, bytes(B * max_pages * 4)}, {path, bytes(B * n_draft * 4)},
                         {n_path, bytes(B * 4)}, {n_new, n_new ? bytes(B * 4) : 0}};
    if (!outputs_clear(out, in)) return FA_ERR_INVALID_ARG;
    Kv4KeepProblem p;
    p.cache = view(cache);
    p.lens = lens;
    p.table = page_table;
    p.path = path;
    p.n_path = n_path;
    p.n_new = n_new;
    p.new_lens = new_lens;
    p.B = B;
    p.max_pages = max_pages;
    p.n_draft = static_cast<int>(n_draft);
    return fa_launch_kv4_keep(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

extern "C" int fa_kv4_copy_pages(const fa_kv4_cache *from, const int32_t *pages, const fa_kv4_cache *to, const int32_t *to_pages,
                                 int64_t n, void *stream)
{
    int st = check_cache_sizes(from);
    if (st != FA_OK || (st = check_cache_sizes(to)) != FA_OK || (st = check_same_layout(from, to)) != FA_OK) return st;
    if (n < 1 || n > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    // a page's pieces are counted in 31 bits
    if (from->Hkv * from->page_size > (int64_t(1) << 28) / from->d) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = check_cache_pointers(from, dev)) != FA_OK ||
        (st = check_cache_pointers(to, dev)) != FA_OK)
        return st;
    for (const void *p : {static_cast<const void *>(pages), static_cast<const void *>(to_pages)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    Range cf[5], out[5];
    cache_ranges(from, cf);
    cache_ranges(to, out);
    const Range in[2] = {{pages, bytes(n * 4)}, {to_pages, bytes(n * 4)}};
    if (!outputs_clear(out, in) || !one_pool_or_two(cf, out)) return FA_ERR_INVALID_ARG;
    return fa_launch_kv4_copy(view(from), pages, view(to), to_pages, n, sm_count, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? FA_OK
               : FA_ERR_LAUNCH;
}

extern "C" int fa_kv4_evict(const fa_kv4_cache *from, const int32_t *lens, const int32_t *page_table,
                            int64_t max_pages, const fa_kv4_cache *to, const int32_t *to_table, int64_t to_max_pages,
                            int64_t B, int64_t keep, int64_t recent, int32_t *kept, int32_t *new_lens, void *stream)
{
    int st = check_cache_sizes(from);
    if (st != FA_OK || (st = check_cache_sizes(to)) != FA_OK) return st;
    if ((st = check_table_sizes(from, B, max_pages)) != FA_OK || (st = check_table_sizes(to, B, to_max_pages)) != FA_OK)
        return st;
    if ((st = check_same_layout(from, to)) != FA_OK) return st;
    if (from->weights == nullptr || to->weights == nullptr) return FA_ERR_INVALID_ARG;
    if (keep < 1 || recent < 0 || recent > keep || keep > to_max_pages * to->page_size) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK || (st = check_cache_pointers(from, dev)) != FA_OK ||
        (st = check_cache_pointers(to, dev)) != FA_OK)
        return st;
    for (const void *p : {static_cast<const void *>(lens), static_cast<const void *>(page_table),
                          static_cast<const void *>(to_table), static_cast<const void *>(kept),
                          static_cast<const void *>(new_lens)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    // the two caches may be one pool; the index arrays may not lie in either
    Range cf[5], ct[5];
    cache_ranges(from, cf);
    cache_ranges(to, ct);
    const Range out[7] = {ct[0], ct[1], ct[2], ct[3], ct[4], {kept, bytes(B * from->Hkv * keep * 4)},
                          {new_lens, bytes(B * 4)}};
    const Range in[3] = {{lens, bytes(B * 4)}, {page_table, bytes(B * max_pages * 4)},
                         {to_table, bytes(B * to_max_pages * 4)}};
    if (!outputs_clear(out, in)) return FA_ERR_INVALID_ARG;
    for (int i = 5; i < 7; ++i)
        for (const Range &r : cf)
            if (meet(out[i], r)) return FA_ERR_INVALID_ARG;
    if (!one_pool_or_two(cf, ct)) return FA_ERR_INVALID_ARG;
    Kv4EvictProblem p;
    p.from = view(from);
    p.to = view(to);
    p.lens = lens;
    p.table = page_table;
    p.to_table = to_table;
    p.kept = kept;
    p.new_lens = new_lens;
    p.B = B;
    p.max_pages = max_pages;
    p.to_max_pages = to_max_pages;
    p.keep = keep;
    p.recent = recent;
    p.sm_count = sm_count;
    return fa_launch_kv4_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}

extern "C" int fa_key_weights(const void *q, const void *k, const float *lse, float *weights, int64_t B, int64_t H,
                              int64_t Hkv, int64_t N, int64_t d, float scale, int causal, int64_t first_query,
                              void *stream)
{
    int st = fa_check_sizes(B, H, N, d);
    if (st != FA_OK) return st;
    if (Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
    if ((causal != 0 && causal != 1) || !(scale > 0.f) || !isfinite(scale)) return FA_ERR_INVALID_ARG;
    if (first_query < 0 || first_query >= N) return FA_ERR_INVALID_ARG;
    int dev = 0, sm_count = 0;
    if ((st = fa_current_device(&dev, &sm_count)) != FA_OK) return st;
    for (const void *p : {q, k})
        if ((st = fa_check_device_pointer(p, dev, 16)) != FA_OK) return st;
    for (const void *p : {static_cast<const void *>(lse), static_cast<const void *>(weights)})
        if ((st = fa_check_device_pointer(p, dev, 4)) != FA_OK) return st;
    const Range out[1] = {{weights, bytes(B * Hkv * N * 4)}};
    const Range in[3] = {{q, bytes(B * H * N * d * 2)}, {k, bytes(B * Hkv * N * d * 2)}, {lse, bytes(B * H * N * 4)}};
    if (!outputs_clear(out, in)) return FA_ERR_INVALID_ARG;
    FaKeyWeightsProblem p;
    p.q = q;
    p.k = k;
    p.lse = lse;
    p.weights = weights;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.N = N;
    p.first_query = first_query;
    p.d = static_cast<int>(d);
    p.scale = scale;
    p.causal = causal;
    p.sm_count = sm_count;
    return fa_launch_key_weights(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_LAUNCH;
}
