/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention operator.
 *
 * The operator is the per-head gated delta-rule recurrence
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,
 *     o_t = S_t^T q_t,            alpha_t = exp(g_t)  (one factor per key channel)
 *
 * from "Understanding Kimi K3's Attention" (state-update and readout
 * equations, symbol table) and "Kimi K3.1 and the Road From Softmax Attention
 * to Kimi Delta Attention" (section "5. Kimi Delta Attention").  The readout
 * uses the state after the token's own write ("Kimi K3 course, lesson 2";
 * "Inside Kimi K3", section "Sequence mixing": the intra-chunk causal matrix
 * includes the diagonal).
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 *  - All tensors are row-major and contiguous, in DEVICE memory, owned by
 *    the caller.  The library allocates no device memory, with two
 *    exceptions: the KDA_PREFILL_TC_SPLIT prefill variant (its ring of chunk
 *    operands, about 0.28 MB per (sequence, head) it runs at once, at most
 *    27 MB) and the KDA_PREFILL_TC_2PASS variant (8 KB per chunk and head)
 *    take stream-ordered scratch from a memory pool of the library's own, and
 *    return it on the same stream when the call's work is done.
 *  - q, k  [T_tot, H, d_k];  v, out [T_tot, H, d_v];  g [T_tot, H, d_k] fp32
 *    (log-decay); beta [T_tot, H] fp32; states [N, H, d_k, d_v] fp32 with row
 *    i = key channel i (the decay scales rows: "Hybrid Attention", section
 *    "Forgetting can be selective, too").
 *  - No scaling, normalisation or gating is applied: q and k arrive already
 *    L2-normalised, the 1/sqrt(d) readout scale and the output gate belong to
 *    the caller ("Understanding Kimi K3's Attention", symbol table and output
 *    equation).
 *  - Preconditions that are documented but not checked on the device (they
 *    would need a read of device memory): g in [-5, 0] (the log-decay bound
 *    g_t = g_min Sigmoid(e^A z_t), g_min = -5) and beta in [0, 1].  Inputs
 *    outside them give finite but unspecified results; they never fault.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream).  KDA_OK means "enqueued".  Arguments are validated on
 *    the host before anything is launched; an error return launches nothing.
 *  - Supported head sizes: d_k == d_v, either 64 or 128.  Anything else
 *    returns KDA_ERR_UNSUPPORTED.
 */
#ifndef KDA_H
#define KDA_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARGUMENT = 1, /* null pointer, negative size, bad dtype */
    KDA_ERR_UNSUPPORTED = 2,      /* valid but not implemented (head size, dtype combo) */
    KDA_ERR_CUDA = 3,             /* a CUDA runtime call or launch failed */
    KDA_ERR_TIMEOUT = 4           /* a bounded device-side wait gave up */
} kda_status;

/* KDA_DTYPE_F16 is taken by the softmax attention and cache calls (kda_attn_*,
 * kda_cache_*) only. */
typedef enum { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1, KDA_DTYPE_F16 = 2 } kda_dtype;

/* Prefill kernel selection: a diagnostic and test selector, not a tuning
 * knob.  KDA_PREFILL_DEFAULT (what callers should pass) picks TC where it
 * supports the call, else FP32.  TC_SPLIT and TC_2PASS run only when named
 * (both are slower than TC on the 96-head layer).  The tensor-core kernels
 * take d_k = d_v = 128, bf16 q/k/v, and q, k, v, g (or z) and out 16-byte
 * aligned; TC_SPLIT also needs a device that supports cooperative launches.
 * TC_2PASS takes 8 KB of stream-ordered scratch per chunk and head (about
 * 0.2 GB for a 96-head, 8192-token layer) from a pool of the library's own.
 * Naming a variant that does not support the call returns
 * KDA_ERR_UNSUPPORTED. */
typedef enum {
    KDA_PREFILL_DEFAULT = 0,
    KDA_PREFILL_FP32 = 1,     /* CUDA-core fp32 chunked kernel (any supported shape) */
    KDA_PREFILL_TC = 2,       /* tcgen05 kernel, one CTA per (sequence, head) (d = 128) */
    KDA_PREFILL_TC_SPLIT = 3, /* tcgen05 kernel with the state recurrence and the intra-chunk
                                 work on different SMs, one cooperative launch (d = 128) */
    KDA_PREFILL_TC_2PASS = 4  /* tcgen05, two launches: the intra-chunk products of every
                                 chunk on every SM, then the state recurrence (d = 128) */
} kda_prefill_variant;

typedef void *kda_stream_t; /* a cudaStream_t */

typedef struct {
    int32_t num_seqs;     /* N >= 0 */
    int32_t total_tokens; /* T_tot >= 0 (decode: must equal num_seqs) */
    int32_t num_heads;    /* H >= 1 */
    int32_t d_k;          /* key/query head size */
    int32_t d_v;          /* value head size */
    int32_t in_dtype;     /* kda_dtype of q, k, v */
    int32_t out_dtype;    /* kda_dtype of out */
    int32_t variant;      /* kda_prefill_variant (ignored by decode) */
} kda_dims;

/*
 * kda_prefill -- chunk-parallel prefill over a packed variable-length batch.
 *
 * Evaluates the recurrence for every sequence n and head h over tokens
 * [cu_seqlens[n], cu_seqlens[n+1]), starting from init_state[n,h] (zeros if
 * init_state is NULL), writes o_t for every token into `out` and, if
 * final_state is non-NULL, the state after the last token of each sequence.
 * Tokens inside a chunk are evaluated together and the state is carried
 * from chunk to chunk ("Inside Kimi K3", section "Sequence mixing";
 * "Hybrid Attention", section "But isn't a recurrent update sequential?");
 * the result equals the token-by-token recurrence up to rounding, for any
 * sequence length (no divisibility requirement).
 *
 *   q, k, v     device, in_dtype, layouts above.
 *   g, beta     device, fp32.
 *   init_state  device fp32 [N, H, d_k, d_v] or NULL.
 *   cu_seqlens  device int32 [N+1] or NULL.  If NULL, T_tot must be a
 *               multiple of N and sequence n covers [n T, (n+1) T) with
 *               T = T_tot / N.  Otherwise cu[0] = 0, non-decreasing,
 *               cu[N] = T_tot; entries outside [0, T_tot] are clamped on the
 *               device and a decreasing pair is read as an empty sequence, so
 *               a malformed array can never cause an out-of-bounds access.
 *               An empty sequence copies init_state (or zeros) to final_state.
 *   out         device, out_dtype [T_tot, H, d_v].
 *   final_state device fp32 [N, H, d_k, d_v] or NULL.  May alias init_state
 *               exactly (each slice is read before it is written).
 *
 * No output (out, final_state, and the checkpoints of the calls below) may
 * share a byte with an input or with another output, except final_state ==
 * init_state: the kernels read later chunks' inputs while they write earlier
 * outputs.  KDA_ERR_INVALID_ARGUMENT if one does.
 *
 * Accumulation is fp32; a bf16 `out` is the round-to-nearest-even of the
 * value an fp32 `out` would hold.
 */
kda_status kda_prefill(const kda_dims *dims, const void *q, const void *k, const void *v,
                       const float *g, const float *beta, const float *init_state,
                       const int32_t *cu_seqlens, void *out, float *final_state,
                       kda_stream_t stream);

/*
 * kda_prefill_noalloc -- kda_prefill that allocates nothing.
 *
 * The pages have no counterpart of this call: it is an interface addition for
 * callers that may not allocate device memory during a call -- hosts whose own
 * caching allocator owns all of the GPU's memory from start-up (an allocation
 * outside it can fail or fragment it) and latency-bound services that keep
 * allocation off their serving path.
 *
 * Same arguments, layouts, semantics and errors as kda_prefill; dims->variant
 * is ignored.  It always runs the KDA_PREFILL_TC_SPLIT kernel, with that
 * kernel's scratch (ring of chunk operands, hand-off words, step table) in a
 * fixed array of the library (about 5 MB, which every device that loads the
 * library keeps until the process exits) instead of pool memory.  That array
 * limits a call to at most 16 chains of at most 4096 (sequence, head) pairs
 * each and at most 65536 sequences; a batch beyond that, or one the split
 * kernel does not take (d_k = d_v != 128, fp32 inputs, q/k/v/g/out not
 * 16-byte aligned, a device without cooperative launches), returns
 * KDA_ERR_UNSUPPORTED and launches nothing.
 *
 * The first call on a device looks up the device address of the array
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture on the device.  Every call shares the one array
 * and clears the parts that must start at zero itself; calls that overlap on
 * the GPU (on different streams or from different host threads) race on it
 * and must be serialised by the caller.
 */
kda_status kda_prefill_noalloc(const kda_dims *dims, const void *q, const void *k, const void *v,
                               const float *g, const float *beta, const float *init_state,
                               const int32_t *cu_seqlens, void *out, float *final_state,
                               kda_stream_t stream);

/* Chunk length of the prefill kernels; checkpoint intervals are multiples of it. */
#define KDA_CHUNK 32

/*
 * kda_prefill_checkpointed -- kda_prefill that also writes state checkpoints.
 *
 * Prefix reuse restores the recurrent state at a token boundary from sparse
 * state checkpoints ("Inside Kimi K3", section "Sequence mixing: fixed-state
 * KDA alongside global MLA").  Besides everything kda_prefill does, this call
 * writes the state of every sequence after each `interval` tokens:
 * checkpoint j (j = 1 .. floor(len_n / interval)) of sequence n is the state
 * after its first j * interval tokens, i.e. the final_state a prefill over
 * that prefix alone would return.
 *
 *   checkpoints device fp32 [capacity, H, d_k, d_v], 4-byte aligned.  Sequence n
 *               uses rows base_n .. base_n + floor(len_n / interval) - 1 with
 *               base_n = sum over m < n of floor(len_m / interval).  Rows at
 *               or beyond `capacity` are not written; checkpoints may be NULL
 *               only with capacity 0 (then this is kda_prefill).
 *   interval    tokens between checkpoints: a positive multiple of KDA_CHUNK.
 *   capacity    number of rows the caller allocated (>= 0).
 *
 * Every other argument, and every other error, is as in kda_prefill;
 * KDA_ERR_INVALID_ARGUMENT if interval is not a positive multiple of
 * KDA_CHUNK, capacity < 0, or checkpoints is NULL or misaligned while
 * capacity > 0.  The checkpoint stores add 4 d_k d_v bytes per checkpoint
 * and head to the prefill's traffic.
 */
kda_status kda_prefill_checkpointed(const kda_dims *dims, const void *q, const void *k,
                                    const void *v, const float *g, const float *beta,
                                    const float *init_state, const int32_t *cu_seqlens,
                                    void *out, float *final_state, float *checkpoints,
                                    int64_t interval, int64_t capacity, kda_stream_t stream);

/*
 * kda_prefill_gated -- kda_prefill with the gate prologue fused into the load
 * stage: the call takes the decay logits and the write-strength logits and
 * forms, per token t, head h and key channel c,
 *
 *   g[t,h,c] = g_min Sigmoid(e^{A_h} z[t,h,c]),  g_min = -5,
 *   beta[t,h] = Sigmoid(beta_logit[t,h])
 *
 * ("Understanding Kimi K3's Attention": the log-decay bound equation, and the
 * symbol table for z_t, A_h and beta_t), then evaluates the same recurrence
 * as kda_prefill.  g never goes through memory; z costs 2 bytes per channel
 * in bf16 where g costs 4.
 *
 *   z           device, in_dtype, [T_tot, H, d_k]: the decay logits (an input:
 *               must not overlap `out`).
 *   a_log       device fp32 [H]: the per-head log-scales A_h.
 *   beta_logit  device fp32 [T_tot, H].
 *
 * Every other argument, and every other error, is as in kda_prefill;
 * KDA_ERR_INVALID_ARGUMENT if there are tokens and z or a_log is NULL.
 */
kda_status kda_prefill_gated(const kda_dims *dims, const void *q, const void *k, const void *v,
                             const void *z, const float *a_log, const float *beta_logit,
                             const float *init_state, const int32_t *cu_seqlens, void *out,
                             float *final_state, kda_stream_t stream);

/*
 * kda_prefill_output_gated -- kda_prefill followed by the layer's output gate,
 * fused into the store of the output where the kernel allows:
 *
 *   y[t,h,j] = Sigmoid(gate_logit[t,h,j]) * o~[t,h,j] / sqrt(ms + eps) * w[j],
 *   ms = (1/d_v) sum_j o~[t,h,j]^2
 *
 * with o~ the ungated readout that kda_prefill would write.  The pages give
 * the layer output as W_o [Sigmoid(W_g x_t) . RMSNorm(o~_t)] ("Inside Kimi
 * K3", section "Sequence mixing: fixed-state KDA alongside global MLA"); this
 * call forms the bracket.  The pages do not define the norm further; here it
 * is the root-mean-square over one head's d_v channels with eps inside the
 * root and an optional per-channel weight.  The projections W_g, W_o stay
 * with the caller.
 *
 *   gate_logit  device, in_dtype, [T_tot, H, d_v]: W_g x_t per head (an input:
 *               must not overlap `out`).
 *   norm_weight device fp32 [d_v], 4-byte aligned, or NULL (weight 1).
 *   eps         finite, > 0.
 *
 * The tensor-core kernel applies the gate before its store when out is bf16
 * and gate_logit is 16-byte aligned; otherwise the prefill writes o~ and a
 * second kernel gates `out` in place (with a bf16 `out`, o~ is then rounded
 * to bf16 once before the norm).  Every other argument, and every other
 * error, is as in kda_prefill; KDA_ERR_INVALID_ARGUMENT if there are tokens
 * and gate_logit is NULL or equals out, or eps is not a positive finite
 * number, or norm_weight is misaligned.
 */
kda_status kda_prefill_output_gated(const kda_dims *dims, const void *q, const void *k,
                                    const void *v, const float *g, const float *beta,
                                    const void *gate_logit, const float *norm_weight, float eps,
                                    const float *init_state, const int32_t *cu_seqlens,
                                    void *out, float *final_state, kda_stream_t stream);

/*
 * kda_output_gate -- the output gate alone, in place: for every row (token t,
 * head h) of `out`,
 *
 *   out[t,h,j] <- Sigmoid(gate_logit[t,h,j]) * out[t,h,j] / sqrt(ms + eps) * w[j],
 *   ms = (1/d_v) sum_j out[t,h,j]^2,
 *
 * the same gate as kda_prefill_output_gated, for outputs that another call
 * wrote: kda_prefill_gated's, or kda_decode's (dims->total_tokens rows).
 *
 *   out          device, out_dtype, [T_tot, H, d_v], read and overwritten.
 *   gate_logit   device, in_dtype, [T_tot, H, d_v]; must not overlap out.
 *   norm_weight  device fp32 [d_v], 4-byte aligned, or NULL (weight 1).
 *   eps          finite, > 0.
 *
 * dims->num_seqs and dims->variant are not used; d_k must equal d_v as
 * everywhere.  KDA_ERR_INVALID_ARGUMENT for a bad dims, a NULL or misaligned
 * pointer while there are rows, out overlapping gate_logit or norm_weight,
 * or a bad eps.
 */
kda_status kda_output_gate(const kda_dims *dims, void *out, const void *gate_logit,
                           const float *norm_weight, float eps, kda_stream_t stream);

/*
 * kda_qkv_prologue -- q, k and v from their projections: for every stream
 * (q, k, v), token t, head h and channel j,
 *
 *   c[t,h,j] = sum_{i=0..3} w[s,h,j,3-i] * x_s[t-i,h,j]
 *   y        = c * Sigmoid(c)                                  (Swish)
 *   q, k     = y / sqrt(sum_j y[t,h,j]^2 + eps)                 v = y
 *
 * The pages define q, k = L2Norm(Swish(ShortConv(W x))) and v =
 * Swish(ShortConv(W_v x)) ("Understanding Kimi K3's Attention", symbol
 * table), with a convolution of width 4 ("Inside Kimi K3", section "Sequence
 * mixing: fixed-state KDA alongside global MLA") that is causal ("Hybrid
 * Attention", section "KDA: don't write the same information twice").
 * Here it is a per-channel convolution over the tokens of one sequence, with
 * no bias, and L2Norm is taken over one head's d channels with eps inside
 * the root.  The projections W x stay with the caller.
 *
 *   dims        num_seqs N, total_tokens T, num_heads H, d_k = d_v = d (64 or
 *               128); in_dtype is the type of x_*, out_dtype that of q, k, v;
 *               variant is not used.
 *   x_q, x_k, x_v  device, in_dtype, [T, H, d]: the projections.
 *   conv_weight device fp32 [3, H, d, 4], 16-byte aligned: streams q, k, v;
 *               tap 3 multiplies the current token, tap 3-i the token i places
 *               earlier.
 *   conv_state_in  device fp32 [N, 3, 3, H, d] or NULL (zeros): for each
 *               sequence and stream, the three inputs before its first token,
 *               entry 0 the oldest.  Aligned to d/32 floats.
 *   cu_seqlens  device int32 [N+1] as in kda_prefill, or NULL (N equal
 *               sequences).  The convolution restarts at every sequence start.
 *               With N = 0 the call does nothing and returns KDA_OK.
 *   q, k, v     device, out_dtype, [T, H, d]: written.
 *   conv_state_out device fp32 [N, 3, 3, H, d] or NULL: the last three inputs
 *               of each sequence, entry 0 the oldest (taken from
 *               conv_state_in, or 0, where a sequence is shorter than three).
 *               This is the conv_state_in of the next segment: a decode step
 *               is a call with one token per sequence.
 *   eps         finite, > 0.
 *
 * x_* and q, k, v must be aligned to d/32 elements.  No output may overlap an
 * input or another output (the two conv states included); alternate two state
 * buffers between calls.  KDA_ERR_INVALID_ARGUMENT for a bad dims, a bad eps,
 * a NULL or misaligned pointer that is needed, or an overlap;
 * KDA_ERR_UNSUPPORTED for d other than 64 or 128, or sizes beyond one grid.
 */
kda_status kda_qkv_prologue(const kda_dims *dims, const void *x_q, const void *x_k,
                            const void *x_v, const float *conv_weight,
                            const float *conv_state_in, const int32_t *cu_seqlens, void *q,
                            void *k, void *v, float *conv_state_out, float eps,
                            kda_stream_t stream);

/*
 * kda_prefill_scalar_decay -- the same chunked prefill for the two special
 * cases of the recurrence the pages build KDA from ("Kimi K3.1 and the Road
 * From Softmax Attention to Kimi Delta Attention", sections "3. The delta
 * rule" and "4. Gating"):
 *
 *   Gated DeltaNet: S_t = (I - beta_t k_t k_t^T) alpha_t S_{t-1} + beta_t k_t v_t^T
 *                   with one decay alpha_t = exp(g_head[t,h]) per head and step;
 *   delta rule:     g_head == NULL, alpha_t = 1.
 *
 * A scalar decay is the channel-wise decay with one value repeated over the
 * key channels, so the result equals kda_prefill with g[t,h,c] = g_head[t,h]
 * (the kernels form the same running sums from it, and the same output).
 * The per-channel decay tensor is not read: 4 bytes per (token, head)
 * replace 4 d_k.
 *
 *   g_head  device fp32 [T_tot, H], 4-byte aligned, values in [-5, 0]; or
 *           NULL (no decay).
 *
 * Every other argument, and every other error, is as in kda_prefill.
 */
kda_status kda_prefill_scalar_decay(const kda_dims *dims, const void *q, const void *k,
                                    const void *v, const float *g_head, const float *beta,
                                    const float *init_state, const int32_t *cu_seqlens,
                                    void *out, float *final_state, kda_stream_t stream);

/*
 * kda_backward -- gradients of kda_prefill.  Given the upstream gradients
 * d_out = dL/d out and d_final_state = dL/d final_state (NULL => 0), writes
 * dL/dq, dL/dk, dL/dv, dL/dg, dL/dbeta and dL/d init_state for the same packed
 * batch.  The pages train the chunked computation and check its gradients
 * against the recurrent version ("Hybrid Attention", section "But isn't a
 * recurrent update sequential?"); this call computes them chunk by chunk,
 * walking each sequence's chunks in reverse and carrying the adjoint of the
 * state, from the forward's state at the start of every chunk.
 *
 *   chunk_states   device fp32 [chunk_capacity, H, d_k, d_v]: the checkpoints
 *                  kda_prefill_checkpointed writes with interval = KDA_CHUNK
 *                  for the same inputs (row layout as there).  It may be NULL
 *                  only if T_tot <= KDA_CHUNK (then no sequence has a second
 *                  chunk).  Rows at or past chunk_capacity are never read.  With
 *                  cu_seqlens NULL a capacity below the rows the batch needs
 *                  returns KDA_ERR_INVALID_ARGUMENT; with cu_seqlens (lengths
 *                  known only on the device) a needed row past the capacity is
 *                  recorded in the device status word, which
 *                  kda_get_last_device_error then reports as
 *                  KDA_ERR_INVALID_ARGUMENT (those gradients are not valid).
 *   d_out          device, in_dtype, [T_tot, H, d_v].
 *   d_final_state  device fp32 [N, H, d_k, d_v] or NULL.
 *   dq, dk, dv     device, out_dtype: [T_tot, H, d_k], [T_tot, H, d_k], [T_tot, H, d_v].
 *   dg             device fp32 [T_tot, H, d_k];  dbeta  device fp32 [T_tot, H].
 *   d_init_state   device fp32 [N, H, d_k, d_v] or NULL (not written).
 *
 * No gradient may share a byte with an input or with another gradient.
 * Arithmetic: with bf16 inputs at d_k = d_v = 128 (16-byte aligned q, k, v, g
 * and d_out) the products run on the tensor cores with tf32 operands and fp32
 * accumulation; otherwise (fp32 inputs, d = 64) everything is fp32 on the CUDA
 * cores.
 * Every other argument (q, k, v, g, beta, init_state, cu_seqlens, dims) and
 * every other error is as in kda_prefill; KDA_ERR_INVALID_ARGUMENT also if
 * chunk_capacity < 0, chunk_states is NULL or misaligned where it is needed,
 * or a gradient overlaps an input or another gradient.
 */
kda_status kda_backward(const kda_dims *dims, const void *q, const void *k, const void *v,
                        const float *g, const float *beta, const float *init_state,
                        const int32_t *cu_seqlens, const float *chunk_states,
                        int64_t chunk_capacity, const void *d_out, const float *d_final_state,
                        void *dq, void *dk, void *dv, float *dg, float *dbeta,
                        float *d_init_state, kda_stream_t stream);

/*
 * kda_decode -- one single-token update of N independent fixed-size states.
 *
 * For each sequence n and head h: M = Diag(exp g) S, u = beta (v - M^T k),
 * S <- M + k u^T (in place), o = S^T q -- the delta form of the recurrence
 * ("Understanding Kimi K3's Attention", rewritten update; "Hybrid
 * Attention", recurrent implementation).  Each fp32 state is read once and
 * written once.
 *
 *   dims        total_tokens must equal num_seqs (one token per sequence).
 *   q, k, v     device, in_dtype, [N, H, d]; g device fp32 [N, H, d_k];
 *               beta device fp32 [N, H].
 *   state_inout device fp32 [N, H, d_k, d_v], updated in place.
 *   out         device, out_dtype [N, H, d_v].
 *
 * Neither out nor the state may share a byte with an input or with each
 * other (KDA_ERR_INVALID_ARGUMENT).
 */
kda_status kda_decode(const kda_dims *dims, const void *q, const void *k, const void *v,
                      const float *g, const float *beta, float *state_inout, void *out,
                      kda_stream_t stream);

/* ---------------------------------------------------------------------------
 * State space layers and 8-bit activations
 * ---------------------------------------------------------------------------
 * The calls below are the sequence mixing of a selective state space layer: the
 * same family of recurrences without the erase term, with a decay of its own for
 * every state entry.  For channel d, state entry n and the tokens t of a sequence,
 *
 *   Delta_t[d] = softplus(dt_t[d] + dt_bias[d])
 *   h_t[d,n]   = exp(Delta_t[d] A[d,n]) h_{t-1}[d,n] + Delta_t[d] u_t[d] B_t[n]
 *   y_t[d]     = (sum_n C_t[n] h_t[d,n] + D[d] u_t[d]) * z_t[d] Sigmoid(z_t[d])
 *
 * where u comes from a short causal convolution.  The pages have no counterpart;
 * these are additions for models that mix such layers with KDA layers.
 *
 * Conventions: as above, except that the activations are given as rows
 * (kda_rows) whose stride the caller chooses, so that slices of a projection's
 * output need no copy.  Inputs are fp32 or bf16 (one type a call); A, D,
 * dt_bias, weights and states are fp32; all arithmetic is fp32, and a bf16
 * output is rounded once.  Masked or absent work has no special value: an
 * infinity or a NaN in an input reaches the outputs that depend on it and no
 * other sequence or channel (the gradients of B, C and the parameters are sums
 * over channels or tokens).  Rows of an output that belong to no sequence (tokens
 * before cu_seqlens[0] or from cu_seqlens[N] on) are left as they were, those of
 * gradients too; with N == 0 that is every row, and the parameters' gradients are 0.
 * A malformed cu_seqlens never causes an access out of bounds; what a call then
 * writes to the outputs is unspecified.
 * The calls allocate nothing: a call that needs scratch takes a workspace, whose
 * size another function gives.  Results do not depend on timing: repeated calls
 * give the same bits.  Calls on different streams may overlap as long as they
 * share no written buffer (workspace included); every call may be captured into
 * a CUDA graph, whose replays use the buffers named at the capture.
 */

/* Tokens [T, channels] of an activation: row t starts at data + t * stride
 * elements.  With scales == NULL data holds the call's input type.  Where a call
 * says so, scales != NULL makes data int8 codes as kda_act_pack8 writes them
 * (stride == channels) with scales fp32 [T, ceil(channels / KDA_PACK_GROUP)].
 * data must be aligned to its element; vector accesses are used where address and
 * stride allow. */
typedef struct {
    const void *data;
    int64_t stride;
    const float *scales;
} kda_rows;

typedef struct {
    int32_t num_seqs;     /* N >= 0 */
    int32_t total_tokens; /* T >= 0 (kda_ssm_step: must equal num_seqs) */
    int32_t channels;     /* D >= 1 */
    int32_t state_size;   /* scan: S, 1..64; convolution: taps W, 2..4 */
    int32_t in_dtype;     /* kda_dtype of the activations read */
    int32_t out_dtype;    /* kda_dtype of the activations (or their gradients) written */
} kda_ssm_dims;

/* What every scan call reads. */
typedef struct {
    kda_rows u, dt, B, C, z;   /* [T, D], [T, D], [T, S], [T, S]; z [T, D], or data NULL: no gate */
    const float *A;            /* [D, S]; finite */
    const float *D;            /* [D] or NULL (0) */
    const float *dt_bias;      /* [D] or NULL (0) */
    const int32_t *cu_seqlens; /* [N+1] or NULL (N equal sequences), as in kda_prefill */
    int32_t delta_softplus;    /* 1: Delta = softplus(dt + dt_bias); 0: Delta = dt + dt_bias */
} kda_ssm_inputs;

/* Channels that share a scale in the 8-bit packing. */
#define KDA_PACK_GROUP 32

/*
 * kda_act_pack8 -- an activation in 8 bits, to be kept for a gradient.
 *
 * Per token, each group of KDA_PACK_GROUP neighbouring channels (the last may be
 * partial) has m = max |x|, scale = m / 127 and codes round(x * (127 / m)), half
 * to even; code * scale is off x by at most half a scale.  A group with m below
 * 2^-120 has scale 0 and codes 0; one that holds an infinity or a NaN has scale NaN
 * (the rest of its codes are unspecified).
 *
 *   x       device, in_dtype rows [rows, channels].
 *   codes   device int8 [rows, channels];  scales  device fp32 [rows, ceil(channels / 32)].
 */
kda_status kda_act_pack8(int32_t rows, int32_t channels, int32_t in_dtype, const kda_rows *x,
                         int8_t *codes, float *scales, kda_stream_t stream);

/*
 * kda_ssm_conv -- causal per-channel convolution of W taps over each sequence, and
 * Swish:  c_t = bias + sum_k weight[k] x_{t-(W-1-k)},  out = c_t Sigmoid(c_t)
 * (or c_t with swish == 0).
 *
 *   x              in_dtype rows [T, D].
 *   weight         device fp32 [D, W] (entry W-1 on the current token);  bias  fp32 [D] or NULL.
 *   conv_state_in  device fp32 [N, W-1, D] or NULL (zeros): the W-1 inputs before each
 *                  sequence's first token, oldest first.
 *   out            device, out_dtype [T, D].
 *   conv_state_out device fp32 [N, W-1, D] or NULL: the last W-1 inputs of each sequence
 *                  (from conv_state_in where it is shorter).  May be conv_state_in itself.
 *
 * One token per sequence (cu_seqlens NULL, T == N) is the decode step: one launch
 * that writes the output and moves the state.
 */
kda_status kda_ssm_conv(const kda_ssm_dims *dims, const kda_rows *x, const float *weight,
                        const float *bias, const float *conv_state_in, const int32_t *cu_seqlens,
                        int32_t swish, void *out, float *conv_state_out, kda_stream_t stream);

/*
 * kda_ssm_conv_backward -- gradients of kda_ssm_conv for d_out (in_dtype rows
 * [T, D]) and d_conv_state_out (fp32 [N, W-1, D] or NULL: zero).
 *
 *   x              as in the forward call, or its 8-bit codes and scales: the gradients
 *                  are then those at the values the codes stand for.
 *   dx             device, out_dtype [T, D];  dweight  fp32 [D, W];  dbias  fp32 [D] or NULL;
 *   d_conv_state_in  fp32 [N, W-1, D] or NULL.
 *   workspace      kda_ssm_conv_backward_workspace(dims) bytes, 16-byte aligned: W + 1 rows of
 *                  D floats a run of tokens (6 MB for 8192 tokens of 8192 channels, W = 4).
 */
int64_t kda_ssm_conv_backward_workspace(const kda_ssm_dims *dims);
kda_status kda_ssm_conv_backward(const kda_ssm_dims *dims, const kda_rows *x, const float *weight,
                                 const float *bias, const float *conv_state_in,
                                 const int32_t *cu_seqlens, int32_t swish, const kda_rows *d_out,
                                 const float *d_conv_state_out, void *dx, float *dweight,
                                 float *dbias, float *d_conv_state_in, void *workspace,
                                 int64_t workspace_bytes, kda_stream_t stream);

/*
 * kda_ssm_scan -- the scan over a packed batch of prompts.
 *
 *   init_state   device fp32 [N, D, S] or NULL (zeros).
 *   out          device, out_dtype [T, D].
 *   final_state  device fp32 [N, D, S] or NULL.  May be init_state itself, with the same results.
 *   chunk_states device fp32 [chunk_capacity, D, S] or NULL (with chunk_capacity 0): the
 *                state after every KDA_CHUNK tokens of each sequence, rows as in
 *                kda_prefill_checkpointed with interval KDA_CHUNK; what the gradients need.
 *   workspace    kda_ssm_scan_workspace(dims) bytes (0 for batches that need none), 16-byte
 *                aligned: 2 S + 1 floats a channel for each place where a sequence is cut (3 MB
 *                for 8192 tokens of 4096 channels with 16 states).
 */
int64_t kda_ssm_scan_workspace(const kda_ssm_dims *dims);
kda_status kda_ssm_scan(const kda_ssm_dims *dims, const kda_ssm_inputs *in, const float *init_state,
                        void *out, float *final_state, float *chunk_states, int64_t chunk_capacity,
                        void *workspace, int64_t workspace_bytes, kda_stream_t stream);

/*
 * kda_ssm_step -- one token for each of N sequences: state (device fp32 [N, D, S],
 * updated in place) and out (out_dtype [N, D]).  in->cu_seqlens must be NULL.
 */
kda_status kda_ssm_step(const kda_ssm_dims *dims, const kda_ssm_inputs *in, float *state, void *out,
                        kda_stream_t stream);

/* What kda_ssm_scan_backward writes: du, ddt, dz (out_dtype [T, D]; dz is needed
 * with z), dB, dC (out_dtype [T, S]), dA (fp32 [D, S]), dD and ddt_bias (fp32 [D]
 * or NULL), d_init_state (fp32 [N, D, S] or NULL). */
typedef struct {
    void *du, *ddt, *dB, *dC, *dz;
    float *dA, *dD, *ddt_bias, *d_init_state;
} kda_ssm_grads;

/*
 * kda_ssm_scan_backward -- gradients of kda_ssm_scan for d_out (in_dtype rows
 * [T, D]) and d_final_state (fp32 [N, D, S] or NULL: zero).
 *
 *   in           as in the forward call; u and z may both be 8-bit codes and scales
 *                (dt, B, C and d_out stay in_dtype): the gradients are then those at the
 *                values the codes stand for, with the states run on from chunk_states.
 *   chunk_states the forward's, chunk_capacity rows (NULL with 0 rows).  Where a row that is
 *                needed is missing: as in kda_backward (an error where lengths are known on
 *                the host, else the device status word).
 *   workspace    kda_ssm_scan_backward_workspace(dims) bytes, 16-byte aligned.  Most of it are
 *                shares of dB and dC: 2 s floats a token for every 1024 / s channels, s = 8, 16,
 *                32 or 64 the first not below S (8192 tokens of 4096 channels: 74 MB with 16
 *                states, 1.0 GB with 64).
 */
int64_t kda_ssm_scan_backward_workspace(const kda_ssm_dims *dims);
kda_status kda_ssm_scan_backward(const kda_ssm_dims *dims, const kda_ssm_inputs *in,
                                 const float *init_state, const float *chunk_states,
                                 int64_t chunk_capacity, const kda_rows *d_out,
                                 const float *d_final_state, const kda_ssm_grads *grads,
                                 void *workspace, int64_t workspace_bytes, kda_stream_t stream);

/* In all of these: no output may share a byte with an input or another output
 * except where a call allows it.  KDA_ERR_INVALID_ARGUMENT for a NULL or misaligned
 * pointer that is needed, a negative size, a stride below the row's length (one
 * row excepted), an overlap, or a workspace too small; KDA_ERR_UNSUPPORTED for S
 * outside 1..64, W outside 2..4, or sizes beyond one grid.  The workspace
 * functions return -1 for dims that the call refuses. */

/* ---------------------------------------------------------------------------
 * Softmax attention and its paged cache
 * ---------------------------------------------------------------------------
 * A hybrid stack keeps a softmax attention layer after every few KDA layers ("The
 * Kimi K3 Architecture", hybrid backbone).  The pages use a compressed form of it; the calls
 * below are the plain one with grouped heads.  For query head h, key head h / G of
 * H_kv = H_q / G, token i of a sequence of L tokens whose last n are the call's, and
 * scores s_ij = scale q_i . k_j over the keys j <= L - n + i:
 *
 *   lse_i = log sum_j e^(s_ij),   out_i = sum_j e^(s_ij - lse_i) v_j
 *
 * A token that sees no key (L < n) has out 0 and lse -inf.
 *
 * Conventions: activations are 16-bit (bf16 or fp16, one type a call), products are
 * accumulated in fp32 on the tensor cores, maxima, sums and log-sums are fp32, and
 * the weights e^(s - max) are rounded to the 16-bit type for the product with v (fp16: times 2^11, so
 * that weights down to 2^-25 of a row's largest keep all bits).  In kda_attn_paged those of sequences of
 * up to 16 rows, that is tokens times H_q / H_kv, keep twice the bits of the type.  Heads are
 * given with strides (kda_heads), so that parts of a projection's rows need no copy.  Keys
 * and values that a row may not see never reach it, whatever they hold, as long as
 * they belong to another sequence or lie behind the cache's length; inside a sequence an
 * infinity or a NaN in k or v reaches the tokens that see it, and one in v may reach up to 127
 * tokens before it (in kda_attn_paged up to 382: the row tiles of a chunk end anywhere in a key tile, and
 * the two of a block may share their walk over the keys).  Rows of an output that belong to no sequence are left as they were.
 * A malformed cu_seqlens, length or page table never causes an access out of bounds; what
 * a call then writes to its outputs is unspecified.
 * The calls allocate nothing and give the same bits every time; calls on different streams
 * may overlap as long as they share no written buffer (workspace included); every call
 * may be captured into a CUDA graph, whose replays use the buffers named at the capture.
 * Errors, before any launch: KDA_ERR_INVALID_ARGUMENT for a NULL or misaligned pointer that is
 * needed, a negative size, strides that are no multiple of 8 or fall below what they step over, an
 * overlap of an output with anything else, or a workspace too small; KDA_ERR_UNSUPPORTED for
 * other types, head dims and page sizes than named here, T H_q from 2^30 on, N H_q from 2^29 on,
 * max_pages page_size from 2^30 on, or (kda_cache_*) N max_pages from 2^31 on.
 */

/* [T, H, head_dim] activations: head h of token t starts at data + t * token_stride +
 * h * head_stride elements.  data 16-byte aligned, strides multiples of 8. */
typedef struct {
    const void *data;
    int64_t token_stride, head_stride;
} kda_heads;

/* The same of a cache [num_pages, page_size, H_kv, head_dim]. */
typedef struct {
    const void *data;
    int64_t page_stride, token_stride, head_stride;
} kda_pages;

typedef struct {
    int32_t num_seqs;     /* N >= 0 */
    int32_t total_tokens; /* T >= 0 */
    int32_t q_heads;      /* H_q, a multiple of H_kv */
    int32_t kv_heads;     /* H_kv >= 1 */
    int32_t head_dim;     /* 64 or 128 */
    int32_t in_dtype;     /* KDA_DTYPE_BF16 or KDA_DTYPE_F16 */
    int32_t out_dtype;    /* in_dtype or KDA_DTYPE_F32 */
    float scale;          /* > 0 */
} kda_attn_dims;

typedef struct {
    int32_t num_pages;    /* P >= 1 */
    int32_t page_size;    /* tokens of a page: 8, 16, 32, ... 1024 */
    int32_t max_pages;    /* pages of a sequence: the row length of the page table */
} kda_cache_dims;

/*
 * kda_attn_prefill -- causal attention over the whole prompts of a packed batch.
 *
 *   q         heads [T, H_q, d];  k, v  heads [T, H_kv, d].
 *   cu_seqlens device int32 [N+1], or NULL (N equal sequences), as in kda_prefill.
 *   out       device, out_dtype [T, H_q, d], contiguous, 16-byte aligned.
 *   lse       device fp32 [T, H_q] or NULL: what the gradients need.
 */
kda_status kda_attn_prefill(const kda_attn_dims *dims, const kda_heads *q, const kda_heads *k,
                            const kda_heads *v, const int32_t *cu_seqlens, void *out, float *lse,
                            kda_stream_t stream);

/*
 * kda_attn_backward -- gradients of kda_attn_prefill for d_out = dL/d out: with
 * P = e^(s - lse), delta_i = d_out_i . out_i and dS_ij = P_ij (d_out_i . v_j - delta_i) for
 * the keys j that token i sees (0 for the others),
 *
 *   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij d_out_i
 *
 * (the sums of dk and dv over the query heads of the group too).  P and dS are rounded to the
 * 16-bit type for the products (in sequences of up to 128 tokens what that leaves is a second
 * operand: twice the bits), sums are fp32, and none depends on timing.  In fp16, which has few powers of
 * two, both are rounded behind a power of two: P down to 2^-29 and dS down to 2^-27 of the largest
 * |d_out_i| |v_j| of the row (dq) or of the rows that see the key (dk) keep all bits of the type, however
 * large or small d_out and v are.  An infinity or a
 * NaN in a sequence may reach gradients of that sequence up to 127 tokens to either side of
 * where the formulas have it, and no other sequence's.
 *
 *   out, lse   the forward's (out in in_dtype, heads [T, H_q, d]; lse fp32 [T, H_q]).
 *   d_out      in_dtype, heads [T, H_q, d].
 *   dq, dk, dv device, out_dtype, contiguous [T, H_q, d], [T, H_kv, d], [T, H_kv, d], 16-byte
 *              aligned.
 *   workspace  kda_attn_backward_workspace(dims) bytes, 16-byte aligned: two floats a token
 *              and query head (fp16: three, and one a token and key head).
 */
int64_t kda_attn_backward_workspace(const kda_attn_dims *dims);
kda_status kda_attn_backward(const kda_attn_dims *dims, const kda_heads *q, const kda_heads *k,
                             const kda_heads *v, const kda_heads *out, const float *lse,
                             const kda_heads *d_out, const int32_t *cu_seqlens, void *dq, void *dk,
                             void *dv, void *workspace, int64_t workspace_bytes,
                             kda_stream_t stream);

/*
 * kda_attn_paged -- attention of each sequence's new tokens over its pages of a cache, in
 * which the new tokens' keys and values are already (kda_cache_append).  One token a
 * sequence is the decode step; pieces of prompts and single tokens may be mixed.
 *
 *   q          heads [T, H_q, d] of the new tokens.
 *   k_pages, v_pages  [P, page_size, H_kv, d].
 *   page_table device int32 [N, max_pages]: page j of sequence n holds its tokens
 *              j page_size ...; entries behind a sequence's last page are not read.  A
 *              page number outside [0, P), or a length past the table, is recorded in the
 *              device status word (kda_get_last_device_error then returns
 *              KDA_ERR_INVALID_ARGUMENT); such keys and values read as zeros.
 *   kv_lens    device int32 [N]: tokens in the cache, the new ones among them.
 *   cu_seqlens device int32 [N+1] of the new tokens, or NULL (T / N each).
 *   out, lse   as in kda_attn_prefill.
 *   workspace  kda_attn_paged_workspace(dims, cache, cu_seqlens) bytes, 16-byte aligned
 *              (of cu_seqlens it matters only whether it is NULL): shares of rows whose
 *              keys are split over blocks (d = 128: 2.5 MB for one token, 40 MB for a chunk, up
 *              to 81 MB for a large batch that may hold both).
 */
int64_t kda_attn_paged_workspace(const kda_attn_dims *dims, const kda_cache_dims *cache,
                                 const int32_t *cu_seqlens);
kda_status kda_attn_paged(const kda_attn_dims *dims, const kda_cache_dims *cache,
                          const kda_heads *q, const kda_pages *k_pages, const kda_pages *v_pages,
                          const int32_t *page_table, const int32_t *kv_lens,
                          const int32_t *cu_seqlens, void *out, float *lse, void *workspace,
                          int64_t workspace_bytes, kda_stream_t stream);

/*
 * kda_attn_paged_granted -- the same behind a reservation that may have refused sequences.
 *
 *   granted    device int32 [N] or NULL, as kda_cache_reserve_granted wrote it: the tokens of a
 *              sequence that was granted fewer than it has in this call see nothing (out 0, lse -inf).
 */
kda_status kda_attn_paged_granted(const kda_attn_dims *dims, const kda_cache_dims *cache,
                                  const kda_heads *q, const kda_pages *k_pages,
                                  const kda_pages *v_pages, const int32_t *page_table,
                                  const int32_t *kv_lens, const int32_t *cu_seqlens,
                                  const int32_t *granted, void *out, float *lse, void *workspace,
                                  int64_t workspace_bytes, kda_stream_t stream);

/* ---------------------------------------------------------------------------
 * The pages of a cache
 * ---------------------------------------------------------------------------
 * A cache is, on the device: pages of keys and values (one pair of tensors a layer), and
 * for all layers together
 *
 *   page_refs  int32 [P]: how many table entries name a page; 0: it is free.
 *   page_table int32 [N, max_pages]: the pages of each sequence, -1 behind the last.
 *   kv_lens    int32 [N]: tokens of each sequence (0: the row is empty).
 *
 * An empty cache is page_refs 0, page_table -1, kv_lens 0.  The calls keep this state; none
 * waits for the host, and what they decide follows from the state alone: free pages are
 * given out lowest number first, to the sequences (or children) in their order.  A last
 * page that is not full and grows belongs to one sequence only (kda_cache_fork copies it, and
 * kda_cache_reserve one that a sequence was shortened into), so that kda_cache_append never
 * writes into a shared page where every sequence got its pages.  Where a reservation may refuse one,
 * take kda_cache_reserve_granted and hand what it granted to kda_cache_append_granted and
 * kda_attn_paged_granted: the length of a refused sequence does not count its new tokens, and
 * without that word they would be written over the last ones that it has.  A sequence or page number out of range
 * is passed by and recorded in the device status word (kda_get_last_device_error then
 * returns KDA_ERR_INVALID_ARGUMENT).  Conventions as in the softmax attention calls.
 */

/* Bytes of the workspace of kda_cache_reserve, kda_cache_fork and kda_cache_compact (16-byte
 * aligned): a number a page.  -1 for dims that the calls refuse. */
int64_t kda_cache_workspace(const kda_cache_dims *cache);

/*
 * kda_cache_reserve -- pages for new tokens: kv_lens[n] grows by new_lens[n] (int32 [N], < 0
 * counts as 0) and the table by the pages that the new length needs.  A sequence gets all
 * of its pages or none: once they run out, those in front have theirs and every later
 * one that needs a page keeps its old length, as does one whose row in the table is too
 * short.
 *
 *   src, dst   int32 [N], or both NULL.  A sequence that grows from the middle of a page that
 *              others share (kda_cache_fork, then kda_cache_free with keep) gets a page of its
 *              own in its place: for every layer, page src[n] is to be copied to dst[n]
 *              (kda_cache_copy) before anything else takes pages; -1 where there is nothing to
 *              copy.  Without the lists such a sequence keeps its old length, and the device
 *              status word records it.
 *   missing    int32 [1] or NULL: pages that were lacking (short rows are not counted).
 *
 * kda_cache_reserve_granted also says who was served:
 *
 *   granted    int32 [N] or NULL: the new tokens of each sequence that have a place: new_lens[n]
 *              (0 for what is below 0), or 0 where the sequence kept its old length.
 *
 * Without both missing and granted a refusal is recorded in the device status word
 * (KDA_ERR_INVALID_ARGUMENT).
 */
kda_status kda_cache_reserve(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs,
                             int32_t *page_table, int32_t *kv_lens, const int32_t *new_lens,
                             int32_t *src, int32_t *dst, int32_t *missing, void *workspace,
                             int64_t workspace_bytes, kda_stream_t stream);
kda_status kda_cache_reserve_granted(const kda_cache_dims *cache, int32_t num_seqs,
                                     int32_t *page_refs, int32_t *page_table, int32_t *kv_lens,
                                     const int32_t *new_lens, int32_t *src, int32_t *dst,
                                     int32_t *missing, int32_t *granted, void *workspace,
                                     int64_t workspace_bytes, kda_stream_t stream);

/*
 * kda_cache_append -- writes the new tokens' keys and values into one layer's pages: of the
 * n new tokens of a sequence, token i goes to place kv_lens - n + i (kv_lens counts them
 * already; places below 0 are passed by).
 *
 *   k, v       heads [T, H_kv, d], bf16 or fp16 (16-bit elements are moved as they are);
 *              head_dim a multiple of 8.
 *   k_pages, v_pages  [P, page_size, H_kv, d], each element of its own.
 *   cu_seqlens int32 [N+1] of the new tokens, or NULL (T / N each).
 *   granted    (kda_cache_append_granted) int32 [N] or NULL, as kda_cache_reserve_granted wrote it:
 *              a sequence that was granted fewer than it has new tokens here is passed by.
 */
kda_status kda_cache_append(const kda_cache_dims *cache, int32_t num_seqs, int32_t total_tokens,
                            int32_t kv_heads, int32_t head_dim, const kda_heads *k,
                            const kda_heads *v, const kda_pages *k_pages, const kda_pages *v_pages,
                            const int32_t *page_table, const int32_t *kv_lens,
                            const int32_t *cu_seqlens, kda_stream_t stream);
kda_status kda_cache_append_granted(const kda_cache_dims *cache, int32_t num_seqs,
                                    int32_t total_tokens, int32_t kv_heads, int32_t head_dim,
                                    const kda_heads *k, const kda_heads *v, const kda_pages *k_pages,
                                    const kda_pages *v_pages, const int32_t *page_table,
                                    const int32_t *kv_lens, const int32_t *cu_seqlens,
                                    const int32_t *granted, kda_stream_t stream);

/*
 * kda_cache_free -- gives pages back: of each of `count` sequences (seqs, int32) the first
 * keep tokens stay (int32 [count], < 0 counts as 0; NULL: none), its length becomes that if it was
 * more, and the pages behind are freed unless another sequence shares them.  A sequence may be
 * listed more than once: the smallest keep holds.
 */
kda_status kda_cache_free(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs,
                          int32_t *page_table, int32_t *kv_lens, int32_t count,
                          const int32_t *seqs, const int32_t *keep, kda_stream_t stream);

/*
 * kda_cache_fork -- children[i] becomes a continuation of parents[i], i < count: it shares the
 * parent's full pages, and has a page of its own where the last is not full.  The children
 * are empty rows, all different, and none of them a parent; a parent may have many.  A
 * child for which no page is left stays empty, as does every later one that needs a page.  A
 * child that has pages is passed by and recorded in the device status word.
 *
 *   src, dst   int32 [count]: for every layer, page src[i] is to be copied to dst[i]
 *              (kda_cache_copy); -1 where there is nothing to copy.
 *   missing    int32 [1] or NULL: pages that were lacking.
 */
kda_status kda_cache_fork(const kda_cache_dims *cache, int32_t num_seqs, int32_t *page_refs,
                          int32_t *page_table, int32_t *kv_lens, int32_t count,
                          const int32_t *parents, const int32_t *children, int32_t *src,
                          int32_t *dst, int32_t *missing, void *workspace, int64_t workspace_bytes,
                          kda_stream_t stream);

/*
 * kda_cache_compact -- renumbers the pages so that the L in use are 0 .. L-1: those from L on
 * move, lowest first, to the free numbers below L, lowest first.
 *
 *   refs_out, table_out  as page_refs and page_table; may be page_refs and page_table themselves.
 *   src, dst   int32 [P]: for every layer, page src[i] is to be copied to dst[i]
 *              (kda_cache_copy); -1 from the number of moved pages on.
 */
kda_status kda_cache_compact(const kda_cache_dims *cache, int32_t num_seqs,
                             const int32_t *page_refs, const int32_t *page_table,
                             const int32_t *kv_lens, int32_t *refs_out, int32_t *table_out,
                             int32_t *src, int32_t *dst, void *workspace, int64_t workspace_bytes,
                             kda_stream_t stream);

/*
 * kda_cache_copy -- page dst[i] of one layer's keys and values becomes a copy of page src[i]
 * (int32 [count]; an entry with a number below 0 is passed by).  No page may be both copied
 * from and to, or be copied to twice, in one call: what such a page then holds is unspecified.
 * The lists of kda_cache_fork and kda_cache_compact keep to that.
 */
kda_status kda_cache_copy(const kda_cache_dims *cache, int32_t kv_heads, int32_t head_dim,
                          const kda_pages *k_pages, const kda_pages *v_pages, int32_t count,
                          const int32_t *src, const int32_t *dst, kda_stream_t stream);

/*
 * kda_get_last_device_error -- report, then clear, the device-side status.
 *
 * The tensor-core prefill kernels wait on their own asynchronous copies,
 * tensor-core operations and (the split kernel) on each other's CTAs with
 * bounded waits; a wait that gives up makes the kernel stop early (outputs of
 * the affected sequences are then incomplete) and records a status word on
 * the device instead of trapping.  kda_backward records a device-side
 * argument check there too (a needed chunk-state row past chunk_capacity).
 * This call synchronises `stream` and, since the previous call, returns
 * KDA_ERR_INVALID_ARGUMENT if the backward's check failed, else
 * KDA_ERR_TIMEOUT if any wait gave up, else KDA_OK; then it resets the
 * words.  KDA_ERR_CUDA if the synchronisation itself fails.
 */
kda_status kda_get_last_device_error(kda_stream_t stream);

/*
 * kda_selftest_timeout -- diagnostic of the bounded-wait path (not part of
 * the method).  Enqueues a one-warp kernel on `stream` that waits, with the
 * same bounded wait the prefill kernel uses, on a barrier nothing arrives on;
 * the wait gives up after a few milliseconds and records the device status
 * word, so that the next kda_get_last_device_error() returns KDA_ERR_TIMEOUT.
 * Nothing traps or hangs and the CUDA context stays usable.
 */
kda_status kda_selftest_timeout(kda_stream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char *kda_status_string(kda_status status);

/* Text of the most recent CUDA error seen by this thread's calls into the
 * library ("" if none).  Static storage per thread; valid until the next call. */
const char *kda_last_cuda_error(void);

/* Library version as 10000*major + 100*minor + patch. */
int32_t kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
