// kda_ssm_api.cu -- the C ABI of the state space layer calls and the 8-bit
// packing: argument validation, launch and error mapping.  Declarations and
// semantics: include/kda.h.

#include "kda_api_util.cuh"
#include "kda_ssm_common.cuh"

namespace {

using kda::conflict;
using kda::esize;
using kda::Rows;
using kda::Span;
using kda::SsmProblem;
using kda::valid_dtype;

constexpr int kMaxStates = 64, kMinTaps = 2, kMaxTaps = 4;

bool misaligned(const void *p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }

kda_status check_dims(const kda_ssm_dims *d, bool conv, SsmProblem &P) {
    if (!d) return KDA_ERR_INVALID_ARGUMENT;
    if (d->num_seqs < 0 || d->total_tokens < 0 || d->channels < 1 || d->state_size < 1) return KDA_ERR_INVALID_ARGUMENT;
    if (!valid_dtype(d->in_dtype) || !valid_dtype(d->out_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    if (conv ? d->state_size < kMinTaps || d->state_size > kMaxTaps : d->state_size > kMaxStates)
        return KDA_ERR_UNSUPPORTED;
    // every grid is below one block per 32 (token, channel) pairs, per 8 (sequence,
    // channel) pairs or per 4 tokens; one grid holds 2^31 - 1 blocks
    const int64_t per_token = (int64_t)d->total_tokens * ((d->channels + 31) / 32 + 8);
    const int64_t per_seq = (int64_t)d->num_seqs * ((d->channels + 7) / 8);
    if (per_token > INT32_MAX || per_seq > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    P = SsmProblem{};
    P.N = d->num_seqs;
    P.T = d->total_tokens;
    P.D = d->channels;
    P.S = d->state_size;
    P.in_dtype = d->in_dtype;
    P.out_dtype = d->out_dtype;
    return KDA_OK;
}

kda_status check_lengths(SsmProblem &P, const int32_t *cu) {
    P.cu = cu;
    if (!cu) {
        if (P.N == 0 ? P.T != 0 : P.T % P.N != 0) return KDA_ERR_INVALID_ARGUMENT;
        P.seq_len = P.N ? P.T / P.N : 0;
    } else if (misaligned(cu, 4)) {
        return KDA_ERR_INVALID_ARGUMENT;
    }
    return KDA_OK;
}

// One activation: checked, its byte range, and whether pieces of `piece` bytes
// may be read.
struct Checked {
    kda_status st;
    Rows r;
    Span data, scales;
};
Checked check_rows(const kda_rows *x, int64_t T, int64_t width, size_t es, bool codes_allowed, size_t piece) {
    Checked c{KDA_OK, {}, {nullptr, 0}, {nullptr, 0}};
    if (T == 0) return c;
    if (!x || !x->data || (x->stride < width && T > 1) || x->stride < 0) {
        c.st = KDA_ERR_INVALID_ARGUMENT;
        return c;
    }
    c.r.p = x->data;
    c.r.stride = x->stride;
    if (x->scales) {
        es = 1;
        c.r.scales = x->scales;
        c.r.ngroups = (int32_t)((width + KDA_PACK_GROUP - 1) / KDA_PACK_GROUP);
        c.scales = {x->scales, (size_t)T * c.r.ngroups * 4};
        if (!codes_allowed || x->stride != width || misaligned(x->scales, 4)) c.st = KDA_ERR_INVALID_ARGUMENT;
    }
    if (misaligned(x->data, es) || x->stride > ((int64_t)1 << 40)) c.st = KDA_ERR_INVALID_ARGUMENT;
    c.data = {x->data, ((size_t)(T - 1) * x->stride + width) * es};
    c.r.vec = !misaligned(x->data, piece) && (x->stride * es) % piece == 0;
    return c;
}

size_t cu_bytes(const SsmProblem &P) { return P.cu ? (size_t)(P.N + 1) * 4 : 0; }

// Pieces that the scan kernels read of a row: a thread's share of a block's
// channels, at most 16 bytes.
size_t scan_piece(int S, size_t es) {
    const int ln = S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16;
    const size_t b = 32 / ln * es;
    return b > 16 ? 16 : b;
}

// The inputs of a scan, their checks and spans (filled into `reads`, 13 of them).
kda_status check_inputs(const kda_ssm_inputs *in, bool codes, SsmProblem &P, Span (&reads)[13]) {
    if (!in) return KDA_ERR_INVALID_ARGUMENT;
    kda_status st = check_lengths(P, in->cu_seqlens);
    if (st != KDA_OK) return st;
    const size_t es = esize(P.in_dtype);
    const bool has_z = in->z.data != nullptr;
    const bool x8 = in->u.scales != nullptr;
    const size_t xp = scan_piece(P.S, x8 ? 1 : es);
    const Checked u = check_rows(&in->u, P.T, P.D, es, codes, xp);
    const Checked dt = check_rows(&in->dt, P.T, P.D, es, false, scan_piece(P.S, es));
    const Checked B = check_rows(&in->B, P.T, P.S, es, false, 4 * es);
    const Checked C = check_rows(&in->C, P.T, P.S, es, false, 4 * es);
    Checked z{KDA_OK, {}, {nullptr, 0}, {nullptr, 0}};
    if (has_z) {
        z = check_rows(&in->z, P.T, P.D, es, codes, xp);
        if (P.T > 0 && (in->z.scales != nullptr) != x8) return KDA_ERR_INVALID_ARGUMENT;
    }
    for (kda_status each : {u.st, dt.st, B.st, C.st, z.st})
        if (each != KDA_OK) return each;
    if (!in->A || misaligned(in->A, 4) || misaligned(in->D, 4) || misaligned(in->dt_bias, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    P.u = u.r;
    P.dt = dt.r;
    P.B = B.r;
    P.C = C.r;
    P.z = z.r;
    P.A = in->A;
    P.skip = in->D;
    P.dt_bias = in->dt_bias;
    P.softplus = in->delta_softplus != 0;
    const size_t d4 = (size_t)P.D * 4;
    const Span all[13] = {u.data, u.scales, dt.data, B.data, C.data, z.data, z.scales,
                          {in->A, d4 * P.S}, {in->D, in->D ? d4 : 0}, {in->dt_bias, in->dt_bias ? d4 : 0},
                          {in->cu_seqlens, cu_bytes(P)}, {nullptr, 0}, {nullptr, 0}};
    for (int i = 0; i < 13; ++i) reads[i] = all[i];
    return KDA_OK;
}

bool any_conflict(std::initializer_list<Span> writes, const Span (&reads)[13], std::initializer_list<Span> more) {
    if (conflict(writes, more)) return true;
    for (const Span &r : reads)
        for (const Span &w : writes)
            if (kda::overlaps(w.p, w.n, r.p, r.n)) return true;
    return false;
}

}  // namespace

extern "C" {

kda_status kda_act_pack8(int32_t rows, int32_t channels, int32_t in_dtype, const kda_rows *x, int8_t *codes,
                         float *scales, kda_stream_t stream) {
    if (rows < 0 || channels < 1 || !valid_dtype(in_dtype)) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t ng = ((int64_t)channels + KDA_PACK_GROUP - 1) / KDA_PACK_GROUP;
    if (rows * ng / 256 + 1 > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (rows == 0) return KDA_OK;
    const Checked c = check_rows(x, rows, channels, esize(in_dtype), false, 16);
    if (c.st != KDA_OK) return c.st;
    if (!codes || !scales || misaligned(scales, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (conflict({{codes, (size_t)rows * channels}, {scales, (size_t)rows * ng * 4}}, {c.data}))
        return KDA_ERR_INVALID_ARGUMENT;
    cudaError_t e = kda_launch_act_pack8(rows, channels, in_dtype, c.r, codes, scales, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_act_pack8");
}

kda_status kda_ssm_conv(const kda_ssm_dims *dims, const kda_rows *x, const float *weight, const float *bias,
                        const float *conv_state_in, const int32_t *cu_seqlens, int32_t swish, void *out,
                        float *conv_state_out, kda_stream_t stream) {
    SsmProblem P;
    kda_status st = check_dims(dims, true, P);
    if (st == KDA_OK) st = check_lengths(P, cu_seqlens);
    if (st != KDA_OK) return st;
    if (P.N == 0) return KDA_OK;
    const Checked c = check_rows(x, P.T, P.D, esize(P.in_dtype), false, 4 * esize(P.in_dtype));
    if (c.st != KDA_OK) return c.st;
    if (!weight || misaligned(weight, 4) || misaligned(bias, 4) || misaligned(conv_state_in, 4) ||
        misaligned(conv_state_out, 4) || (P.T > 0 && !out) || misaligned(out, esize(P.out_dtype)))
        return KDA_ERR_INVALID_ARGUMENT;
    const size_t sb = (size_t)P.N * (P.S - 1) * P.D * 4;
    const float *cin_read = conv_state_in == conv_state_out ? nullptr : conv_state_in;
    if (conflict({{out, (size_t)P.T * P.D * esize(P.out_dtype)}, {conv_state_out, sb}},
                 {c.data, {weight, (size_t)P.D * P.S * 4}, {bias, (size_t)P.D * 4}, {cin_read, sb},
                  {cu_seqlens, cu_bytes(P)}}))
        return KDA_ERR_INVALID_ARGUMENT;
    P.u = c.r;
    cudaError_t e = kda_launch_ssm_conv(P, weight, bias, conv_state_in, swish != 0, out, conv_state_out,
                                        (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_ssm_conv");
}

int64_t kda_ssm_conv_backward_workspace(const kda_ssm_dims *dims) {
    SsmProblem P;
    if (check_dims(dims, true, P) != KDA_OK) return -1;
    int tile;
    return kda_ssm_conv_backward_tiles(P, &tile) * (P.S + 1) * P.D * (int64_t)sizeof(float);
}

kda_status kda_ssm_conv_backward(const kda_ssm_dims *dims, const kda_rows *x, const float *weight, const float *bias,
                                 const float *conv_state_in, const int32_t *cu_seqlens, int32_t swish,
                                 const kda_rows *d_out, const float *d_conv_state_out, void *dx, float *dweight,
                                 float *dbias, float *d_conv_state_in, void *workspace, int64_t workspace_bytes,
                                 kda_stream_t stream) {
    SsmProblem P;
    kda_status st = check_dims(dims, true, P);
    if (st == KDA_OK) st = check_lengths(P, cu_seqlens);
    if (st != KDA_OK) return st;
    const size_t es = esize(P.in_dtype);
    const Checked c = check_rows(x, P.T, P.D, es, true, x && x->scales ? 4 : 4 * es);
    const Checked y = check_rows(d_out, P.T, P.D, es, false, 4 * es);
    if (c.st != KDA_OK) return c.st;
    if (y.st != KDA_OK) return y.st;
    const int64_t need = kda_ssm_conv_backward_workspace(dims);
    if (!weight || !dweight || (P.T > 0 && !dx) || misaligned(dx, esize(P.out_dtype)) || workspace_bytes < need ||
        (need > 0 && !workspace) || misaligned(workspace, 16))
        return KDA_ERR_INVALID_ARGUMENT;
    for (const void *p : {(const void *)weight, (const void *)bias, (const void *)conv_state_in,
                          (const void *)d_conv_state_out, (const void *)dweight, (const void *)dbias,
                          (const void *)d_conv_state_in})
        if (misaligned(p, 4)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t sb = (size_t)P.N * (P.S - 1) * P.D * 4, wb = (size_t)P.D * P.S * 4, db = (size_t)P.D * 4;
    if (conflict({{dx, (size_t)P.T * P.D * esize(P.out_dtype)}, {dweight, wb}, {dbias, db}, {d_conv_state_in, sb},
                  {workspace, (size_t)need}},
                 {c.data, c.scales, y.data, {weight, wb}, {bias, db}, {conv_state_in, sb}, {d_conv_state_out, sb},
                  {cu_seqlens, cu_bytes(P)}}))
        return KDA_ERR_INVALID_ARGUMENT;
    P.u = c.r;
    P.dy = y.r;
    cudaError_t e = kda_launch_ssm_conv_backward(P, weight, bias, conv_state_in, d_conv_state_out, swish != 0, dx,
                                                 dweight, dbias, d_conv_state_in, (float *)workspace,
                                                 (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_ssm_conv_backward");
}

int64_t kda_ssm_scan_workspace(const kda_ssm_dims *dims) {
    SsmProblem P;
    if (check_dims(dims, false, P) != KDA_OK) return -1;
    return kda_ssm_scan_ws(P);
}

kda_status kda_ssm_scan(const kda_ssm_dims *dims, const kda_ssm_inputs *in, const float *init_state, void *out,
                        float *final_state, float *chunk_states, int64_t chunk_capacity, void *workspace,
                        int64_t workspace_bytes, kda_stream_t stream) {
    SsmProblem P;
    Span reads[13];
    kda_status st = check_dims(dims, false, P);
    if (st == KDA_OK) st = check_inputs(in, false, P, reads);
    if (st != KDA_OK) return st;
    if (chunk_capacity < 0 || (chunk_capacity > 0 && !chunk_states) || (P.T > 0 && !out) ||
        misaligned(out, esize(P.out_dtype)) || misaligned(init_state, 4) || misaligned(final_state, 4) ||
        misaligned(chunk_states, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const int64_t need = kda_ssm_scan_ws(P);
    if (workspace_bytes < need || (need > 0 && !workspace) || misaligned(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    if (P.N == 0) return KDA_OK;
    const size_t row = (size_t)P.D * P.S * 4, sb = P.N * row;
    if (any_conflict({{out, (size_t)P.T * P.D * esize(P.out_dtype)}, {final_state, sb},
                      {chunk_states, (size_t)chunk_capacity * row}, {workspace, (size_t)need}},
                     reads, {{init_state == final_state ? nullptr : init_state, sb}}))
        return KDA_ERR_INVALID_ARGUMENT;
    P.svec = P.S % 4 == 0;
    for (const void *p : {(const void *)P.A, (const void *)init_state, (const void *)final_state, (const void *)chunk_states})
        if (misaligned(p, 16)) P.svec = false;
    cudaError_t e = kda_launch_ssm_scan(P, init_state, out, final_state, chunk_capacity > 0 ? chunk_states : nullptr,
                                        chunk_capacity, (float *)workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_ssm_scan");
}

kda_status kda_ssm_step(const kda_ssm_dims *dims, const kda_ssm_inputs *in, float *state, void *out,
                        kda_stream_t stream) {
    SsmProblem P;
    Span reads[13];
    kda_status st = check_dims(dims, false, P);
    if (st == KDA_OK) st = check_inputs(in, false, P, reads);
    if (st != KDA_OK) return st;
    if (P.T != P.N || P.cu) return KDA_ERR_INVALID_ARGUMENT;
    if (P.N == 0) return KDA_OK;
    if (!state || misaligned(state, 4) || !out || misaligned(out, esize(P.out_dtype))) return KDA_ERR_INVALID_ARGUMENT;
    if (any_conflict({{out, (size_t)P.N * P.D * esize(P.out_dtype)}, {state, (size_t)P.N * P.D * P.S * 4}}, reads, {}))
        return KDA_ERR_INVALID_ARGUMENT;
    P.svec = P.S % 4 == 0 && !misaligned(P.A, 16) && !misaligned(state, 16);
    cudaError_t e = kda_launch_ssm_step(P, state, out, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_ssm_step");
}

int64_t kda_ssm_scan_backward_workspace(const kda_ssm_dims *dims) {
    SsmProblem P;
    if (check_dims(dims, false, P) != KDA_OK) return -1;
    return kda_ssm_scan_backward_ws(P);
}

kda_status kda_ssm_scan_backward(const kda_ssm_dims *dims, const kda_ssm_inputs *in, const float *init_state,
                                 const float *chunk_states, int64_t chunk_capacity, const kda_rows *d_out,
                                 const float *d_final_state, const kda_ssm_grads *grads, void *workspace,
                                 int64_t workspace_bytes, kda_stream_t stream) {
    SsmProblem P;
    Span reads[13];
    kda_status st = check_dims(dims, false, P);
    if (st == KDA_OK) st = check_inputs(in, true, P, reads);
    if (st != KDA_OK) return st;
    if (!grads) return KDA_ERR_INVALID_ARGUMENT;
    const kda_ssm_grads &g = *grads;
    const size_t eo = esize(P.out_dtype);
    const Checked y = check_rows(d_out, P.T, P.D, esize(P.in_dtype), false, scan_piece(P.S, esize(P.in_dtype)));
    if (y.st != KDA_OK) return y.st;
    const bool has_z = P.z.p != nullptr;
    if (chunk_capacity < 0 || (chunk_capacity > 0 && !chunk_states))
        return KDA_ERR_INVALID_ARGUMENT;
    if (P.T > 0 && (!g.du || !g.ddt || !g.dB || !g.dC || (has_z && !g.dz))) return KDA_ERR_INVALID_ARGUMENT;
    if (!g.dA) return KDA_ERR_INVALID_ARGUMENT;
    for (const void *p : {(const void *)g.du, (const void *)g.ddt, (const void *)g.dB, (const void *)g.dC, (const void *)g.dz})
        if (misaligned(p, eo)) return KDA_ERR_INVALID_ARGUMENT;
    for (const void *p : {(const void *)g.dA, (const void *)g.dD, (const void *)g.ddt_bias, (const void *)g.d_init_state,
                          (const void *)init_state, (const void *)chunk_states, (const void *)d_final_state})
        if (misaligned(p, 4)) return KDA_ERR_INVALID_ARGUMENT;
    if (!P.cu && P.N > 0) {
        // equal lengths: the rows needed are known here, as in kda_backward
        const int64_t per = P.seq_len / KDA_CHUNK, nch = (P.seq_len + KDA_CHUNK - 1) / KDA_CHUNK;
        if (nch > 1 && chunk_capacity < (int64_t)(P.N - 1) * per + nch - 1) return KDA_ERR_INVALID_ARGUMENT;
    }
    const int64_t need = kda_ssm_scan_backward_ws(P);
    if (workspace_bytes < need || (need > 0 && !workspace) || misaligned(workspace, 16)) return KDA_ERR_INVALID_ARGUMENT;
    const size_t row = (size_t)P.D * P.S * 4, sb = P.N * row, td = (size_t)P.T * P.D * eo, ts = (size_t)P.T * P.S * eo;
    if (any_conflict({{g.du, td}, {g.ddt, td}, {has_z ? g.dz : nullptr, td}, {g.dB, ts}, {g.dC, ts}, {g.dA, row},
                      {g.dD, (size_t)P.D * 4}, {g.ddt_bias, (size_t)P.D * 4}, {g.d_init_state, sb},
                      {workspace, (size_t)need}},
                     reads, {y.data, {init_state, sb}, {d_final_state, sb}, {chunk_states, (size_t)chunk_capacity * row}}))
        return KDA_ERR_INVALID_ARGUMENT;
    P.dy = y.r;
    P.svec = P.S % 4 == 0;
    for (const void *p : {(const void *)P.A, (const void *)init_state, (const void *)chunk_states,
                          (const void *)d_final_state, (const void *)g.dA, (const void *)g.d_init_state})
        if (misaligned(p, 16)) P.svec = false;
    cudaError_t e = kda_launch_ssm_scan_backward(P, init_state, chunk_states, chunk_capacity, d_final_state, g.du, g.ddt,
                                                 g.dB, g.dC, g.dz, g.dA, g.dD, g.ddt_bias, g.d_init_state,
                                                 (float *)workspace, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : kda_cuda_fail(e, "kda_ssm_scan_backward");
}

}  // extern "C"
