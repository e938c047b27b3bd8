// kda_attn_api.cu -- the C ABI of the softmax attention calls: argument validation,
// launch and error mapping.  Declarations and semantics: include/kda.h.

#include "kda_api_util.cuh"
#include "kda_attn_common.cuh"

namespace {

using kda::Attn;
using kda::conflict;
using kda::Span;

bool misaligned(const void *p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
bool sixteen(int32_t t) { return t == KDA_DTYPE_BF16 || t == KDA_DTYPE_F16; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

kda_status check_dims(const kda_attn_dims *d, Attn &A) {
    if (!d) return KDA_ERR_INVALID_ARGUMENT;
    if (d->num_seqs < 0 || d->total_tokens < 0 || d->q_heads < 1 || d->kv_heads < 1 || d->head_dim < 1)
        return KDA_ERR_INVALID_ARGUMENT;
    if (!sixteen(d->in_dtype) && d->in_dtype != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (!sixteen(d->out_dtype) && d->out_dtype != KDA_DTYPE_F32) return KDA_ERR_INVALID_ARGUMENT;
    if (d->q_heads % d->kv_heads != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (!(d->scale > 0.f) || d->scale > 1e30f) return KDA_ERR_INVALID_ARGUMENT;
    if (!sixteen(d->in_dtype) || (d->out_dtype != d->in_dtype && d->out_dtype != KDA_DTYPE_F32))
        return KDA_ERR_UNSUPPORTED;
    if (d->head_dim != 64 && d->head_dim != 128) return KDA_ERR_UNSUPPORTED;
    // rows (token, query head) and blocks are counted in 32 bits
    if ((int64_t)d->total_tokens * d->q_heads > INT32_MAX / 2 ||
        (int64_t)d->num_seqs * d->q_heads > INT32_MAX / 4)
        return KDA_ERR_UNSUPPORTED;
    A = Attn{};
    A.N = d->num_seqs;
    A.T = d->total_tokens;
    A.Hq = d->q_heads;
    A.Hkv = d->kv_heads;
    A.G = d->q_heads / d->kv_heads;
    A.d = d->head_dim;
    A.in_dtype = d->in_dtype;
    A.out_dtype = d->out_dtype;
    A.scale = d->scale;
    A.scale_log2 = (float)((double)d->scale * 1.4426950408889634);
    return KDA_OK;
}

kda_status check_lengths(Attn &A, const int32_t *cu) {
    A.cu = cu;
    if (cu) return misaligned(cu, 4) ? KDA_ERR_INVALID_ARGUMENT : KDA_OK;
    if (A.N == 0 ? A.T != 0 : A.T % A.N != 0) return KDA_ERR_INVALID_ARGUMENT;
    A.seq_len = A.N ? A.T / A.N : 0;
    return KDA_OK;
}

// [T, heads, d] with strides: 16-byte pieces must be readable, and no two elements the same.
bool bad_heads(const kda_heads *x, int64_t T, int64_t heads, int d) {
    if (!x || !x->data || misaligned(x->data, 16)) return true;
    if (x->token_stride % 8 || x->head_stride % 8) return true;
    const int64_t most = (int64_t)1 << 38;
    if (x->token_stride < 0 || x->head_stride < 0 || x->token_stride > most || x->head_stride > most) return true;
    return (heads > 1 && x->head_stride < d) || (T > 1 && x->token_stride < d);
}
Span span_of(const kda_heads *x, int64_t T, int64_t heads, int d) {
    return {x->data, (size_t)((T - 1) * x->token_stride + (heads - 1) * x->head_stride + d) * 2};
}
bool bad_pages(const kda_pages *x, int64_t P, int64_t page, int64_t heads, int d) {
    if (!x || !x->data || misaligned(x->data, 16)) return true;
    const int64_t most = (int64_t)1 << 38;
    for (int64_t s : {x->page_stride, x->token_stride, x->head_stride})
        if (s % 8 || s < 0 || s > most) return true;
    return (heads > 1 && x->head_stride < d) || (page > 1 && x->token_stride < d) || (P > 1 && x->page_stride < d);
}
Span span_of(const kda_pages *x, int64_t P, int64_t page, int64_t heads, int d) {
    return {x->data, (size_t)((P - 1) * x->page_stride + (page - 1) * x->token_stride + (heads - 1) * x->head_stride + d) * 2};
}
size_t osize(const Attn &A) { return A.out_dtype == KDA_DTYPE_F32 ? 4 : 2; }
size_t cu_bytes(const Attn &A) { return A.cu ? (size_t)(A.N + 1) * 4 : 0; }

}  // namespace

bool kda_make_attn_map(CUtensorMap *m, const void *base, bool bf16, int d, int64_t heads, int64_t rows, int64_t pages,
                       int64_t s_head, int64_t s_row, int64_t s_page, int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    // the stride of a dimension of one is never used, but has to be a legal one
    const auto stride = [d](int64_t s, int64_t n) { return (cuuint64_t)(n > 1 ? s : (int64_t)d) * 2; };
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows, (cuuint64_t)pages};
    const cuuint64_t strides[3] = {stride(s_head, heads), stride(s_row, rows), stride(s_page, pages)};
    const cuuint32_t boxes[4] = {64, 1, (cuuint32_t)box, 1}, step[4] = {1, 1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base),
              dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

extern "C" {

kda_status kda_attn_prefill(const kda_attn_dims *dims, const kda_heads *q, const kda_heads *k, const kda_heads *v,
                            const int32_t *cu_seqlens, void *out, float *lse, kda_stream_t stream) {
    Attn A;
    kda_status st = check_dims(dims, A);
    if (st == KDA_OK) st = check_lengths(A, cu_seqlens);
    if (st != KDA_OK) return st;
    if (A.T == 0 || A.N == 0) return KDA_OK;
    if (bad_heads(q, A.T, A.Hq, A.d) || bad_heads(k, A.T, A.Hkv, A.d) || bad_heads(v, A.T, A.Hkv, A.d) || !out ||
        misaligned(out, 16) || misaligned(lse, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t rows = (size_t)A.T * A.Hq;
    if (conflict({{out, rows * A.d * osize(A)}, {lse, rows * 4}},
                 {span_of(q, A.T, A.Hq, A.d), span_of(k, A.T, A.Hkv, A.d), span_of(v, A.T, A.Hkv, A.d),
                  {cu_seqlens, cu_bytes(A)}}))
        return KDA_ERR_INVALID_ARGUMENT;
    A.q = q->data, A.q_t = q->token_stride, A.q_h = q->head_stride;
    A.k = k->data, A.k_t = k->token_stride, A.k_h = k->head_stride;
    A.v = v->data, A.v_t = v->token_stride, A.v_h = v->head_stride;
    A.out = out;
    A.lse = lse;
    cudaError_t e = kda_launch_attn_prefill(A, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_attn_prefill");
}

int64_t kda_attn_backward_workspace(const kda_attn_dims *dims) {
    Attn A;
    if (check_dims(dims, A) != KDA_OK) return -1;
    return kda_attn_backward_ws(A);
}

kda_status kda_attn_backward(const kda_attn_dims *dims, const kda_heads *q, const kda_heads *k, const kda_heads *v,
                             const kda_heads *out, const float *lse, const kda_heads *d_out, const int32_t *cu_seqlens,
                             void *dq, void *dk, void *dv, void *workspace, int64_t workspace_bytes,
                             kda_stream_t stream) {
    Attn A;
    kda_status st = check_dims(dims, A);
    if (st == KDA_OK) st = check_lengths(A, cu_seqlens);
    if (st != KDA_OK) return st;
    if (A.T == 0 || A.N == 0) return KDA_OK;
    if (bad_heads(q, A.T, A.Hq, A.d) || bad_heads(k, A.T, A.Hkv, A.d) || bad_heads(v, A.T, A.Hkv, A.d) ||
        bad_heads(out, A.T, A.Hq, A.d) || bad_heads(d_out, A.T, A.Hq, A.d) || !lse || misaligned(lse, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    for (const void *p : {(const void *)dq, (const void *)dk, (const void *)dv})
        if (!p || misaligned(p, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t need = kda_attn_backward_ws(A);
    if (workspace_bytes < need || !workspace || misaligned(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t rows = (size_t)A.T * A.Hq, nq = rows * A.d * osize(A), nk = (size_t)A.T * A.Hkv * A.d * osize(A);
    if (conflict({{dq, nq}, {dk, nk}, {dv, nk}, {workspace, (size_t)need}},
                 {span_of(q, A.T, A.Hq, A.d), span_of(k, A.T, A.Hkv, A.d), span_of(v, A.T, A.Hkv, A.d),
                  span_of(out, A.T, A.Hq, A.d), span_of(d_out, A.T, A.Hq, A.d), {lse, rows * 4},
                  {cu_seqlens, cu_bytes(A)}}))
        return KDA_ERR_INVALID_ARGUMENT;
    A.q = q->data, A.q_t = q->token_stride, A.q_h = q->head_stride;
    A.k = k->data, A.k_t = k->token_stride, A.k_h = k->head_stride;
    A.v = v->data, A.v_t = v->token_stride, A.v_h = v->head_stride;
    A.lse = const_cast<float *>(lse);
    const kda::AttnGrads X{out->data, d_out->data, out->token_stride, out->head_stride, d_out->token_stride,
                           d_out->head_stride, dq, dk, dv};
    cudaError_t e = kda_launch_attn_backward(A, X, (float *)workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_attn_backward");
}

static kda_status check_paged(const kda_attn_dims *dims, const kda_cache_dims *cache, const int32_t *cu_seqlens, Attn &A) {
    kda_status st = check_dims(dims, A);
    if (st == KDA_OK) st = check_lengths(A, cu_seqlens);
    if (st != KDA_OK) return st;
    if (!cache || cache->num_pages < 1 || cache->page_size < 1 || cache->max_pages < 1) return KDA_ERR_INVALID_ARGUMENT;
    const int32_t p = cache->page_size;
    if (p < 8 || p > 1024 || (p & (p - 1))) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)cache->max_pages * p > INT32_MAX / 2) return KDA_ERR_UNSUPPORTED;
    A.P = cache->num_pages;
    A.page = p;
    A.wide = cache->max_pages;
    return KDA_OK;
}

int64_t kda_attn_paged_workspace(const kda_attn_dims *dims, const kda_cache_dims *cache, const int32_t *cu_seqlens) {
    Attn A;
    if (check_paged(dims, cache, cu_seqlens, A) != KDA_OK) return -1;
    return kda_attn_paged_ws(A);
}

kda_status kda_attn_paged(const kda_attn_dims *dims, const kda_cache_dims *cache, const kda_heads *q,
                          const kda_pages *k_pages, const kda_pages *v_pages, const int32_t *page_table,
                          const int32_t *kv_lens, const int32_t *cu_seqlens, void *out, float *lse, void *workspace,
                          int64_t workspace_bytes, kda_stream_t stream) {
    return kda_attn_paged_granted(dims, cache, q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, nullptr, out, lse, workspace,
                                  workspace_bytes, stream);
}

kda_status kda_attn_paged_granted(const kda_attn_dims *dims, const kda_cache_dims *cache, const kda_heads *q,
                                  const kda_pages *k_pages, const kda_pages *v_pages, const int32_t *page_table,
                                  const int32_t *kv_lens, const int32_t *cu_seqlens, const int32_t *granted, void *out,
                                  float *lse, void *workspace, int64_t workspace_bytes, kda_stream_t stream) {
    Attn A;
    kda_status st = check_paged(dims, cache, cu_seqlens, A);
    if (st != KDA_OK) return st;
    if (A.T == 0 || A.N == 0) return KDA_OK;
    if (bad_heads(q, A.T, A.Hq, A.d) || bad_pages(k_pages, A.P, A.page, A.Hkv, A.d) ||
        bad_pages(v_pages, A.P, A.page, A.Hkv, A.d) || !page_table || misaligned(page_table, 4) || !kv_lens ||
        misaligned(kv_lens, 4) || misaligned(granted, 4) || !out || misaligned(out, 16) || misaligned(lse, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t need = kda_attn_paged_ws(A);
    if (workspace_bytes < need || (need > 0 && !workspace) || misaligned(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t rows = (size_t)A.T * A.Hq;
    if (conflict({{out, rows * A.d * osize(A)}, {lse, rows * 4}, {workspace, (size_t)need}},
                 {span_of(q, A.T, A.Hq, A.d), span_of(k_pages, A.P, A.page, A.Hkv, A.d),
                  span_of(v_pages, A.P, A.page, A.Hkv, A.d), {page_table, (size_t)A.N * A.wide * 4},
                  {kv_lens, (size_t)A.N * 4}, {cu_seqlens, cu_bytes(A)}, {granted, (size_t)A.N * 4}}))
        return KDA_ERR_INVALID_ARGUMENT;
    A.q = q->data, A.q_t = q->token_stride, A.q_h = q->head_stride;
    A.k = k_pages->data, A.k_p = k_pages->page_stride, A.k_t = k_pages->token_stride, A.k_h = k_pages->head_stride;
    A.v = v_pages->data, A.v_p = v_pages->page_stride, A.v_t = v_pages->token_stride, A.v_h = v_pages->head_stride;
    A.table = page_table;
    A.lens = kv_lens;
    A.granted = granted;
    A.out = out;
    A.lse = lse;
    cudaError_t e = kda_launch_attn_paged(A, workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_attn_paged");
}

}  // extern "C"
