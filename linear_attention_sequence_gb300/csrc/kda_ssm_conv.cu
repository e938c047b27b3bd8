// kda_ssm_conv.cu -- the short causal convolution of a state space layer, its
// Swish, and their gradients, over a packed batch.
//
//   c_t = bias + sum_k w[k] x_{t-(W-1-k)},   y_t = c_t Sigmoid(c_t)   (or c_t)
//   dc_t = dy_t (s + c_t s (1 - s)),  s = Sigmoid(c_t)               (or dy_t)
//   dx_t = sum_k w[k] dc_{t+(W-1-k)},  dw[k] = sum_t dc_t x_{t-(W-1-k)},  dbias = sum_t dc_t
//
// with the inputs before a sequence's first token taken from its carried state.
// HBM-bound: a thread takes V neighbouring channels (16 bytes of a bf16 row) and
// walks a run of tokens with the W - 1 last inputs in registers, so that each
// input is read once, but for the W - 1 rows that a run reads of its neighbour.
// The gradient walks forward too: with dc_t known, dx of token t - (W-1) is
// complete.  A run's share of dw and dbias goes to a workspace, and a second
// kernel adds the runs up in their order, so the sums do not depend on timing.

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kThreads = 128;

struct ConvArgs {
    SsmProblem P;             // P.S: taps
    const float *w, *bias, *cin;
    bool swish, ovec;
    void *out;
    float *cout;
    // gradients
    const float *dcout;
    float *dcin, *part;
    int tile;
};

template <int V>
__device__ __forceinline__ void load_cols(const float *p, float (&v)[V], int have) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (p && i < have) ? p[i] : 0.f;
}

// The W taps of V channels.
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c0, int have, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = i < have ? a.w[(int64_t)(c0 + i) * W + k] : 0.f;
    load_cols<V>(a.bias ? a.bias + c0 : nullptr, b, have);
}

// The W - 1 inputs before token t of sequence n = [sa, sb).
template <typename IN, int V, int W>
__device__ __forceinline__ void load_window(const ConvArgs &a, int n, int64_t sa, int64_t t, int c0, int have,
                                            float (&x)[W][V]) {
    const SsmProblem &P = a.P;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t u = t - (W - 1) + k;
        if (u >= sa) {
            Raw<IN, V> r;
            r.load((const IN *)P.u.p + u * P.u.stride + c0, have, P.u.vec);
            if constexpr (sizeof(IN) == 1) {
                const float sc = P.u.scales[u * P.u.ngroups + c0 / kPackGroup];
#pragma unroll
                for (int i = 0; i < V; ++i) x[k][i] = r.get(i) * sc;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[k][i] = r.get(i);
            }
        } else {
            // u - sa + W - 1 is in 0 .. W - 2
            load_cols<V>(a.cin ? a.cin + ((int64_t)n * (W - 1) + (u - sa + W - 1)) * P.D + c0 : nullptr, x[k], have);
        }
    }
}

template <int V, int W>
__device__ __forceinline__ void shift(float (&x)[W][V]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) x[k][i] = x[k + 1][i];
}

template <typename IN, typename OUT, int V, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_kernel(const ConvArgs a) {
    constexpr int PB = 8;                      // rows in flight
    const SsmProblem &P = a.P;
    const int nvb = (P.D + V * kThreads - 1) / (V * kThreads);
    const int c0 = ((int)(blockIdx.x % nvb) * kThreads + threadIdx.x) * V;
    const int64_t t0 = (int64_t)(blockIdx.x / nvb) * a.tile, t1 = min(t0 + a.tile, (int64_t)P.T);
    const int have = P.D - c0;
    if (have <= 0) return;
    float w[W][V], b[V], x[W][V];
    load_taps<V, W>(a, c0, have, w, b);
    int n = 0;
    int64_t sa = 0, sb = 0, t = t0;
    while (t < t1) {
        if (!find_seq(P.cu, P.N, P.T, P.seq_len, t, n, sa, sb)) {
            t = sa;                            // rows outside every sequence stay as they are
            continue;
        }
        load_window<IN, V, W>(a, n, sa, t, c0, have, x);
        const int64_t end = min(sb, t1);
        for (; t < end; t += PB) {
            Raw<IN, V> r[PB];
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                r[i].clear();
                if (t + i < end) r[i].load((const IN *)P.u.p + (t + i) * P.u.stride + c0, have, P.u.vec);
            }
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                if (t + i < end) {
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        x[W - 1][j] = r[i].get(j);
                        float c = b[j];
#pragma unroll
                        for (int k = 0; k < W; ++k) c = fmaf(w[k][j], x[k][j], c);
                        o[j] = a.swish ? c * sigmoid_fast(c) : c;
                    }
                    store_row<OUT, V>((OUT *)a.out + (t + i) * P.D + c0, o, have, a.ovec);
                    shift<V, W>(x);
                }
            }
        }
        t = end;
    }
}

// The last W - 1 inputs of every sequence.  A thread owns one channel of one
// sequence and reads before it writes: cout may be cin.
template <typename IN, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_state_kernel(const ConvArgs a) {
    const SsmProblem &P = a.P;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)P.N * P.D) return;
    const int n = (int)(i / P.D);
    const int64_t c = i - (int64_t)n * P.D;
    int64_t sa, sb;
    seq_bounds(P.cu, n, P.T, P.seq_len, sa, sb);
    float v[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t u = sb - (W - 1) + k;
        if (u >= sa) v[k] = ld_elem((const IN *)P.u.p + u * P.u.stride + c);
        else v[k] = a.cin ? a.cin[((int64_t)n * (W - 1) + (u - sa + W - 1)) * P.D + c] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) a.cout[((int64_t)n * (W - 1) + k) * P.D + c] = v[k];
}

// One token a sequence: output and new state in one pass.
template <typename IN, typename OUT, int V, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_token_kernel(const ConvArgs a) {
    const SsmProblem &P = a.P;
    const int nv = (P.D + V - 1) / V;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t n = i / nv;
    if (n >= P.N) return;
    const int c0 = (int)(i - n * nv) * V, have = P.D - c0;
    float w[W][V], b[V], x[W][V];
    load_window<IN, V, W>(a, (int)n, n, n, c0, have, x);
    Raw<IN, V> r;
    r.load((const IN *)P.u.p + n * P.u.stride + c0, have, P.u.vec);
    load_taps<V, W>(a, c0, have, w, b);
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        x[W - 1][j] = r.get(j);
        float c = b[j];
#pragma unroll
        for (int k = 0; k < W; ++k) c = fmaf(w[k][j], x[k][j], c);
        o[j] = a.swish ? c * sigmoid_fast(c) : c;
    }
    store_row<OUT, V>((OUT *)a.out + n * P.D + c0, o, have, a.ovec);
    if (a.cout) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < have) a.cout[(n * (W - 1) + k) * P.D + c0 + j] = x[k + 1][j];
    }
}

template <typename IN, typename DY, typename OUT, int V, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_backward_kernel(const ConvArgs a) {
    constexpr int PB = 4;
    const SsmProblem &P = a.P;
    const int nvb = (P.D + V * kThreads - 1) / (V * kThreads);
    const int c0 = ((int)(blockIdx.x % nvb) * kThreads + threadIdx.x) * V;
    const int64_t tile = blockIdx.x / nvb;
    const int64_t t0 = tile * a.tile, t1 = min(t0 + a.tile, (int64_t)P.T);
    const int have = P.D - c0;
    if (have <= 0) return;
    float w[W][V], b[V], x[W][V], dw[W][V], db[V], dc[W][V];
    load_taps<V, W>(a, c0, have, w, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = 0.f;
    }
    int n = 0;
    int64_t sa = 0, sb = 0, t = t0;
    while (t < t1) {
        if (!find_seq(P.cu, P.N, P.T, P.seq_len, t, n, sa, sb)) {
            t = sa;
            continue;
        }
        const int64_t s0 = t, s1 = min(sb, t1);          // the tokens of this run in this sequence
        const int64_t last = min(sb, s1 + W - 1);        // dc is needed up to here
        load_window<IN, V, W>(a, n, sa, t, c0, have, x);
#pragma unroll
        for (int k = 0; k < W; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) dc[k][i] = 0.f;
        // step t gives dc_t and completes position t - (W-1); past the end dc = 0
        for (; t < s1 + W - 1; t += PB) {
            Raw<IN, V> rx[PB];
            Raw<DY, V> ry[PB];
            float sc[PB];
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                rx[i].clear();
                ry[i].clear();
                sc[i] = 0.f;
                if (t + i < last) {
                    rx[i].load((const IN *)P.u.p + (t + i) * P.u.stride + c0, have, P.u.vec);
                    ry[i].load((const DY *)P.dy.p + (t + i) * P.dy.stride + c0, have, P.dy.vec);
                    if constexpr (sizeof(IN) == 1) sc[i] = P.u.scales[(t + i) * P.u.ngroups + c0 / kPackGroup];
                }
            }
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int64_t ti = t + i;
                if (ti >= s1 + W - 1) break;
                const bool own = ti < s1;                 // counted by this run; later ones by the next
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    x[W - 1][j] = sizeof(IN) == 1 ? rx[i].get(j) * sc[i] : rx[i].get(j);
                    float d = ry[i].get(j);               // 0 past the end
                    if (a.swish) {
                        float c = b[j];
#pragma unroll
                        for (int k = 0; k < W; ++k) c = fmaf(w[k][j], x[k][j], c);
                        const float s = sigmoid_fast(c);
                        d *= fmaf(c * s, 1.f - s, s);
                    }
                    if (ti >= last) d = 0.f;
                    dc[W - 1][j] = d;
                    if (own) {
                        db[j] += d;
#pragma unroll
                        for (int k = 0; k < W; ++k) dw[k][j] = fmaf(d, x[k][j], dw[k][j]);
                    }
                }
                const int64_t p = ti - (W - 1);           // the position whose gradient is complete
                if (p >= s0 || s0 == sa) {                // p < s0 = sa: the carried state
                    float o[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float v = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k) v = fmaf(w[W - 1 - k][j], dc[k][j], v);
                        o[j] = v;
                    }
                    // the carried state out holds the last W - 1 positions
                    const int64_t back = p - (sb - (W - 1));
                    if (a.dcout && back >= 0) {
                        float e[V];
                        load_cols<V>(a.dcout + ((int64_t)n * (W - 1) + back) * P.D + c0, e, have);
#pragma unroll
                        for (int j = 0; j < V; ++j) o[j] += e[j];
                    }
                    if (p >= sa) {
                        store_row<OUT, V>((OUT *)a.out + p * P.D + c0, o, have, a.ovec);
                    } else if (a.dcin) {
                        float *q = a.dcin + ((int64_t)n * (W - 1) + (p - sa + W - 1)) * P.D + c0;
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (j < have) q[j] = o[j];
                    }
                }
                shift<V, W>(x);
                shift<V, W>(dc);
            }
        }
        t = s1;
    }
    float *part = a.part + tile * (W + 1) * P.D + c0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if (j < have) {
#pragma unroll
            for (int k = 0; k < W; ++k) part[(int64_t)k * P.D + j] = dw[k][j];
            part[(int64_t)W * P.D + j] = db[j];
        }
    }
}

// dw and dbias: the runs' shares, added in their order.  A warp takes 32
// channels of one row of the shares; its kRuns warps add every kRuns-th run and
// join through shared memory.
constexpr int kRuns = 8;
__global__ void __launch_bounds__(32 * kRuns)
kda_ssm_conv_reduce_kernel(const float *__restrict__ part, int64_t tiles, int D, int W, float *dw, float *dbias) {
    __shared__ float s[kRuns][32];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int nb = (D + 31) / 32;
    const int k = blockIdx.x / nb, c = (blockIdx.x % nb) * 32 + lane;
    float v = 0.f;
    if (c < D)
        for (int64_t i = y; i < tiles; i += kRuns) v += part[(i * (W + 1) + k) * D + c];
    s[y][lane] = v;
    __syncthreads();
    if (y == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < kRuns; ++i) v += s[i][lane];
        if (k < W) {
            if (dw) dw[(int64_t)c * W + k] = v;
        } else if (dbias) {
            dbias[c] = v;
        }
    }
}

// A sequence without tokens hands its state on: so does its gradient.
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_empty_kernel(const ConvArgs a) {
    const SsmProblem &P = a.P;
    const int W = P.S;
    const int64_t per = (int64_t)(W - 1) * P.D, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= per * P.N) return;
    int64_t sa, sb;
    seq_bounds(P.cu, (int)(i / per), P.T, P.seq_len, sa, sb);
    if (sa == sb) a.dcin[i] = a.dcout ? a.dcout[i] : 0.f;
}

// Tokens of a run: 64 (32 without gradients), fewer where that would leave the
// GPU without work: at least a warp a scheduler is wanted, and 16 tokens keep the
// rows that two runs read within a fifth.
int run_length(int64_t T, int32_t D, int V, int most) {
    const int64_t columns = (D + (int64_t)V * 32 - 1) / (V * 32);   // warps across
    int tile = most;
    while (tile > 16 && (T + tile - 1) / tile * columns < 152 * 16) tile /= 2;
    return tile;
}

template <typename IN, typename OUT, int W>
cudaError_t forward(ConvArgs &a, cudaStream_t stream) {
    constexpr int V = sizeof(IN) == 2 ? 8 : 4;
    const SsmProblem &P = a.P;
    if (!P.cu && P.seq_len == 1) {
        const int64_t n = (int64_t)P.N * ((P.D + V - 1) / V);
        kda_ssm_conv_token_kernel<IN, OUT, V, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    if (P.T > 0) {
        a.tile = run_length(P.T, P.D, V, 32);
        const int64_t blocks = (P.T + a.tile - 1) / a.tile * ((P.D + V * kThreads - 1) / (V * kThreads));
        kda_ssm_conv_kernel<IN, OUT, V, W><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.cout) {
        const int64_t n = (int64_t)P.N * P.D;
        kda_ssm_conv_state_kernel<IN, W><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

template <typename IN, typename OUT>
cudaError_t forward_taps(ConvArgs &a, cudaStream_t s) {
    if (a.P.S == 2) return forward<IN, OUT, 2>(a, s);
    if (a.P.S == 3) return forward<IN, OUT, 3>(a, s);
    return forward<IN, OUT, 4>(a, s);
}

constexpr int kBackV = 4;

template <typename IN, typename DY, typename OUT, int W>
cudaError_t backward(ConvArgs &a, float *dw, float *dbias, cudaStream_t stream) {
    constexpr int V = kBackV;
    const SsmProblem &P = a.P;
    const int64_t tiles = kda_ssm_conv_backward_tiles(P, &a.tile);
    if (tiles > 0) {
        const int64_t blocks = tiles * ((P.D + V * kThreads - 1) / (V * kThreads));
        kda_ssm_conv_backward_kernel<IN, DY, OUT, V, W><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (dw || dbias) {
        const unsigned blocks = (unsigned)((W + 1) * ((P.D + 31) / 32));
        kda_ssm_conv_reduce_kernel<<<blocks, 32 * kRuns, 0, stream>>>(a.part, tiles, P.D, W, dw, dbias);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.dcin && (P.cu || P.seq_len == 0)) {
        const int64_t n = (int64_t)P.N * (W - 1) * P.D;
        kda_ssm_conv_empty_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

template <typename IN, typename DY, typename OUT>
cudaError_t backward_taps(ConvArgs &a, float *dw, float *dbias, cudaStream_t s) {
    if (a.P.S == 2) return backward<IN, DY, OUT, 2>(a, dw, dbias, s);
    if (a.P.S == 3) return backward<IN, DY, OUT, 3>(a, dw, dbias, s);
    return backward<IN, DY, OUT, 4>(a, dw, dbias, s);
}

template <typename DY, typename OUT>
cudaError_t backward_input(ConvArgs &a, float *dw, float *dbias, cudaStream_t s) {
    if (a.P.u.scales) return backward_taps<int8_t, DY, OUT>(a, dw, dbias, s);
    return backward_taps<DY, DY, OUT>(a, dw, dbias, s);
}

bool out_vec(const void *p, const SsmProblem &P) {
    const int es = P.out_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    return ((uintptr_t)p & 15u) == 0 && (int64_t)P.D * es % 16 == 0;
}

}  // namespace

cudaError_t kda_launch_ssm_conv(const SsmProblem &P, const float *w, const float *bias, const float *cin, bool swish,
                                void *out, float *cout, cudaStream_t stream) {
    ConvArgs a{};
    a.P = P;
    a.w = w;
    a.bias = bias;
    a.cin = cin;
    a.swish = swish;
    a.out = out;
    a.cout = cout;
    a.ovec = out_vec(out, P);
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return forward_taps<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (ib) return forward_taps<__nv_bfloat16, float>(a, stream);
    if (ob) return forward_taps<float, __nv_bfloat16>(a, stream);
    return forward_taps<float, float>(a, stream);
}

int64_t kda_ssm_conv_backward_tiles(const SsmProblem &P, int *tile) {
    *tile = run_length(P.T, P.D, kBackV, 64);
    return ((int64_t)P.T + *tile - 1) / *tile;
}

cudaError_t kda_launch_ssm_conv_backward(const SsmProblem &P, const float *w, const float *bias, const float *cin,
                                         const float *dcout, bool swish, void *dx, float *dw, float *dbias,
                                         float *dcin, float *workspace, cudaStream_t stream) {
    ConvArgs a{};
    a.P = P;
    a.w = w;
    a.bias = bias;
    a.cin = cin;
    a.dcout = dcout;
    a.swish = swish;
    a.out = dx;
    a.dcin = dcin;
    a.part = workspace;
    a.ovec = out_vec(dx, P);
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return backward_input<__nv_bfloat16, __nv_bfloat16>(a, dw, dbias, stream);
    if (ib) return backward_input<__nv_bfloat16, float>(a, dw, dbias, stream);
    if (ob) return backward_input<float, __nv_bfloat16>(a, dw, dbias, stream);
    return backward_input<float, float>(a, dw, dbias, stream);
}
