// kda_cache_api.cu -- the C ABI of the cache calls: argument validation, launch and error
// mapping.  Declarations and semantics: include/kda.h.

#include "kda_api_util.cuh"
#include "kda_cache.cuh"

namespace {

using kda::Cache;
using kda::conflict;
using kda::Heads;
using kda::Pages;
using kda::Span;

bool misaligned(const void *p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
bool bad(const int32_t *p) { return !p || misaligned(p, 4); }

kda_status check_cache(const kda_cache_dims *c, int32_t N, int32_t *refs, int32_t *table, int32_t *lens, Cache &C) {
    if (!c || c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1 || N < 0) return KDA_ERR_INVALID_ARGUMENT;
    const int32_t p = c->page_size;
    if (p < 8 || p > 1024 || (p & (p - 1))) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)c->max_pages * p > INT32_MAX / 2 || (int64_t)N * c->max_pages > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    C = Cache{};
    C.N = N;
    C.P = c->num_pages;
    C.wide = c->max_pages;
    while ((1 << C.shift) < p) ++C.shift;
    C.refs = refs;
    C.table = table;
    C.lens = lens;
    return KDA_OK;
}
Span refs_of(const Cache &C) { return {C.refs, (size_t)C.P * 4}; }
Span table_of(const Cache &C) { return {C.table, (size_t)C.N * C.wide * 4}; }
Span lens_of(const Cache &C) { return {C.lens, (size_t)C.N * 4}; }

kda_status check_heads_dims(int32_t heads, int32_t d, Cache &C) {
    if (heads < 1 || d < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (d % 8 || d > 1024 || (int64_t)heads * d > (1 << 20)) return KDA_ERR_UNSUPPORTED;
    C.H = heads;
    C.d = d;
    return KDA_OK;
}
constexpr int64_t kMostStride = (int64_t)1 << 38;
bool bad_strides(std::initializer_list<int64_t> all) {
    for (int64_t s : all)
        if (s < 0 || s % 8 || s > kMostStride) return true;
    return false;
}
bool bad_rows(const kda_heads *x, int64_t T, const Cache &C) {
    if (!x || !x->data || misaligned(x->data, 16) || bad_strides({x->token_stride, x->head_stride})) return true;
    return (C.H > 1 && x->head_stride < C.d) || (T > 1 && x->token_stride < C.d);
}
bool bad_pages(const kda_pages *x, const Cache &C) {
    if (!x || !x->data || misaligned(x->data, 16) || bad_strides({x->page_stride, x->token_stride, x->head_stride})) return true;
    // every element of its own: the strides in order of size each past what the smaller ones span
    int64_t s[3] = {x->page_stride, x->token_stride, x->head_stride}, n[3] = {C.P, (int64_t)1 << C.shift, C.H};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                int64_t t = s[i];
                s[i] = s[j], s[j] = t;
                t = n[i], n[i] = n[j], n[j] = t;
            }
    int64_t span = C.d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < span) return true;
        span += (n[i] - 1) * s[i];
    }
    return false;
}
Span span_of(const kda_heads *x, int64_t T, const Cache &C) {
    return {x->data, (size_t)((T - 1) * x->token_stride + (C.H - 1) * x->head_stride + C.d) * 2};
}
Span span_of(const kda_pages *x, const Cache &C) {
    return {x->data, (size_t)((C.P - 1) * x->page_stride + (((int64_t)1 << C.shift) - 1) * x->token_stride +
                              (C.H - 1) * x->head_stride + C.d) * 2};
}
Heads heads_at(const kda_heads *x) { return {(const uint16_t *)x->data, x->token_stride, x->head_stride}; }
Pages pages_at(const kda_pages *x) {
    return {(uint16_t *)const_cast<void *>(x->data), x->page_stride, x->token_stride, x->head_stride};
}

kda_status done(cudaError_t e, const char *where) { return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, where); }

}  // namespace

extern "C" {

int64_t kda_cache_workspace(const kda_cache_dims *cache) {
    Cache C;
    if (check_cache(cache, 0, nullptr, nullptr, nullptr, C) != KDA_OK) return -1;
    return (int64_t)C.P * 4 + 16;
}

kda_status kda_cache_reserve(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs, int32_t *page_table,
                             int32_t *kv_lens, const int32_t *new_lens, int32_t *src, int32_t *dst, int32_t *missing,
                             void *workspace, int64_t workspace_bytes, kda_stream_t stream) {
    return kda_cache_reserve_granted(cache, num_seqs, page_refs, page_table, kv_lens, new_lens, src, dst, missing, nullptr,
                                     workspace, workspace_bytes, stream);
}

kda_status kda_cache_reserve_granted(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs, int32_t *page_table,
                                     int32_t *kv_lens, const int32_t *new_lens, int32_t *src, int32_t *dst, int32_t *missing,
                                     int32_t *granted, void *workspace, int64_t workspace_bytes, kda_stream_t stream) {
    Cache C;
    const kda_status st = check_cache(cache, num_seqs, page_refs, page_table, kv_lens, C);
    if (st != KDA_OK) return st;
    const int64_t need = (int64_t)C.P * 4 + 16;
    if (bad(page_refs) || (C.N > 0 && (bad(page_table) || bad(kv_lens) || bad(new_lens))) || misaligned(missing, 4) ||
        (src == nullptr) != (dst == nullptr) || misaligned(src, 4) || misaligned(dst, 4) || misaligned(granted, 4) || !workspace ||
        workspace_bytes < need || misaligned(workspace, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    if (conflict({refs_of(C), table_of(C), lens_of(C), {src, (size_t)C.N * 4}, {dst, (size_t)C.N * 4}, {missing, 4},
                  {granted, (size_t)C.N * 4}, {workspace, (size_t)need}},
                 {{new_lens, (size_t)C.N * 4}}))
        return KDA_ERR_INVALID_ARGUMENT;
    if (C.N == 0 && !missing) return KDA_OK;
    return done(kda_launch_cache_reserve(C, new_lens, src, dst, missing, granted, (int32_t *)workspace, (cudaStream_t)stream),
                "kda_cache_reserve");
}

kda_status kda_cache_append(const kda_cache_dims *cache, int32_t num_seqs, int32_t total_tokens, int32_t kv_heads,
                            int32_t head_dim, const kda_heads *k, const kda_heads *v, const kda_pages *k_pages,
                            const kda_pages *v_pages, const int32_t *page_table, const int32_t *kv_lens,
                            const int32_t *cu_seqlens, kda_stream_t stream) {
    return kda_cache_append_granted(cache, num_seqs, total_tokens, kv_heads, head_dim, k, v, k_pages, v_pages, page_table,
                                    kv_lens, cu_seqlens, nullptr, stream);
}

kda_status kda_cache_append_granted(const kda_cache_dims *cache, int32_t num_seqs, int32_t total_tokens, int32_t kv_heads,
                                    int32_t head_dim, const kda_heads *k, const kda_heads *v, const kda_pages *k_pages,
                                    const kda_pages *v_pages, const int32_t *page_table, const int32_t *kv_lens,
                                    const int32_t *cu_seqlens, const int32_t *granted, kda_stream_t stream) {
    Cache C;
    kda_status st = check_cache(cache, num_seqs, nullptr, const_cast<int32_t *>(page_table), const_cast<int32_t *>(kv_lens), C);
    if (st == KDA_OK) st = check_heads_dims(kv_heads, head_dim, C);
    if (st != KDA_OK) return st;
    const int64_t T = total_tokens;
    if (T < 0 || misaligned(cu_seqlens, 4) || misaligned(granted, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (!cu_seqlens && (C.N == 0 ? T != 0 : T % C.N != 0)) return KDA_ERR_INVALID_ARGUMENT;
    if (T == 0 || C.N == 0) return KDA_OK;
    if (bad_rows(k, T, C) || bad_rows(v, T, C) || bad_pages(k_pages, C) || bad_pages(v_pages, C) || bad(page_table) ||
        bad(kv_lens))
        return KDA_ERR_INVALID_ARGUMENT;
    // (the two caches may be parts of one tensor: their spans may interleave)
    const Span reads[6] = {span_of(k, T, C), span_of(v, T, C), table_of(C), lens_of(C),
                           {cu_seqlens, cu_seqlens ? (size_t)(C.N + 1) * 4 : 0}, {granted, (size_t)C.N * 4}};
    for (const Span &r : reads)
        if (conflict({span_of(k_pages, C)}, {r}) || conflict({span_of(v_pages, C)}, {r})) return KDA_ERR_INVALID_ARGUMENT;
    if (k_pages->data == v_pages->data) return KDA_ERR_INVALID_ARGUMENT;
    return done(kda_launch_cache_append(C, heads_at(k), heads_at(v), pages_at(k_pages), pages_at(v_pages), cu_seqlens, T,
                                        cu_seqlens ? 0 : T / C.N, granted, (cudaStream_t)stream),
                "kda_cache_append");
}

kda_status kda_cache_free(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs, int32_t *page_table,
                          int32_t *kv_lens, int32_t count, const int32_t *seqs, const int32_t *keep, kda_stream_t stream) {
    Cache C;
    const kda_status st = check_cache(cache, num_seqs, page_refs, page_table, kv_lens, C);
    if (st != KDA_OK) return st;
    if (count < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (count == 0) return KDA_OK;
    if (bad(page_refs) || (C.N > 0 && (bad(page_table) || bad(kv_lens))) || bad(seqs) || misaligned(keep, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    if (conflict({refs_of(C), table_of(C), lens_of(C)}, {{seqs, (size_t)count * 4}, {keep, keep ? (size_t)count * 4 : 0}}))
        return KDA_ERR_INVALID_ARGUMENT;
    return done(kda_launch_cache_free(C, count, seqs, keep, (cudaStream_t)stream), "kda_cache_free");
}

kda_status kda_cache_fork(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs, int32_t *page_table,
                          int32_t *kv_lens, int32_t count, const int32_t *parents, const int32_t *children, int32_t *src,
                          int32_t *dst, int32_t *missing, void *workspace, int64_t workspace_bytes, kda_stream_t stream) {
    Cache C;
    const kda_status st = check_cache(cache, num_seqs, page_refs, page_table, kv_lens, C);
    if (st != KDA_OK) return st;
    if (count < 0 || misaligned(missing, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (count == 0)   // nothing was lacking
        return missing ? done(cudaMemsetAsync(missing, 0, 4, (cudaStream_t)stream), "kda_cache_fork") : KDA_OK;
    const int64_t need = (int64_t)C.P * 4 + 16;
    if (bad(page_refs) || (C.N > 0 && (bad(page_table) || bad(kv_lens))) || bad(parents) || bad(children) || bad(src) || bad(dst) ||
        !workspace || workspace_bytes < need || misaligned(workspace, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t list = (size_t)count * 4;
    if (conflict({refs_of(C), table_of(C), lens_of(C), {src, list}, {dst, list}, {missing, 4}, {workspace, (size_t)need}},
                 {{parents, list}, {children, list}}))
        return KDA_ERR_INVALID_ARGUMENT;
    return done(kda_launch_cache_fork(C, count, parents, children, src, dst, missing, (int32_t *)workspace,
                                      (cudaStream_t)stream),
                "kda_cache_fork");
}

kda_status kda_cache_compact(const kda_cache_dims *cache, int32_t num_seqs, const int32_t *page_refs,
                             const int32_t *page_table, const int32_t *kv_lens, int32_t *refs_out, int32_t *table_out,
                             int32_t *src, int32_t *dst, void *workspace, int64_t workspace_bytes, kda_stream_t stream) {
    Cache C;
    const kda_status st = check_cache(cache, num_seqs, const_cast<int32_t *>(page_refs), const_cast<int32_t *>(page_table),
                                      const_cast<int32_t *>(kv_lens), C);
    if (st != KDA_OK) return st;
    const int64_t need = (int64_t)C.P * 4 + 16;
    if (bad(page_refs) || bad(refs_out) || bad(src) || bad(dst) || !workspace || workspace_bytes < need ||
        misaligned(workspace, 16) || (C.N > 0 && (bad(page_table) || bad(table_out) || bad(kv_lens))))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t refs = (size_t)C.P * 4, table = (size_t)C.N * C.wide * 4;
    if (conflict({{refs_out, refs}, {table_out, table}, {src, refs}, {dst, refs}, {workspace, (size_t)need}},
                 {lens_of(C), {page_refs == refs_out ? nullptr : page_refs, refs},
                  {page_table == table_out ? nullptr : page_table, table}}))
        return KDA_ERR_INVALID_ARGUMENT;
    return done(kda_launch_cache_compact(C, refs_out, table_out, src, dst, (int32_t *)workspace, (cudaStream_t)stream),
                "kda_cache_compact");
}

kda_status kda_cache_copy(const kda_cache_dims *cache, int32_t kv_heads, int32_t head_dim, const kda_pages *k_pages,
                          const kda_pages *v_pages, int32_t count, const int32_t *src, const int32_t *dst,
                          kda_stream_t stream) {
    Cache C;
    kda_status st = check_cache(cache, 0, nullptr, nullptr, nullptr, C);
    if (st == KDA_OK) st = check_heads_dims(kv_heads, head_dim, C);
    if (st != KDA_OK) return st;
    if (count < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (count == 0) return KDA_OK;
    if (bad_pages(k_pages, C) || bad_pages(v_pages, C) || bad(src) || bad(dst)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t list = (size_t)count * 4;
    for (const Span &r : {Span{src, list}, Span{dst, list}})
        if (conflict({span_of(k_pages, C)}, {r}) || conflict({span_of(v_pages, C)}, {r})) return KDA_ERR_INVALID_ARGUMENT;
    if (k_pages->data == v_pages->data) return KDA_ERR_INVALID_ARGUMENT;
    return done(kda_launch_cache_copy(C, pages_at(k_pages), pages_at(v_pages), count, src, dst, (cudaStream_t)stream),
                "kda_cache_copy");
}

}  // extern "C"
