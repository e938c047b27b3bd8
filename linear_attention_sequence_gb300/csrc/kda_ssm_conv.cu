// kda_ssm_conv.cu -- the short causal convolution of a state space layer, its
// Swish, and their gradients, over a packed batch.
//
//   c_t = bias + sum_k w[k] x_{t-(W-1-k)},   y_t = c_t Sigmoid(c_t)   (or c_t)
//   dc_t = dy_t (s + c_t s (1 - s)),  s = Sigmoid(c_t)               (or dy_t)
//   dx_t = sum_k w[k] dc_{t+(W-1-k)},  dw[k] = sum_t dc_t x_{t-(W-1-k)},  dbias = sum_t dc_t
//
// with the inputs before a sequence's first token taken from its carried state.
// HBM-bound: a thread takes four neighbouring channels and walks a run of tokens
// with the W - 1 last inputs in registers, so that each input is read once, but
// for the W - 1 rows that a run reads of its neighbour.  The rows of one batch are
// loaded while the batch before is computed (kRows rows in flight a thread).  The
// arithmetic is on pairs of channels, one issue slot for two operations.
// The gradient walks forward too: with dc_t known, dx of token t - (W-1) is
// complete.  A run's share of dw and dbias goes to a workspace, and a second
// kernel adds the runs up in their order, so the sums do not depend on timing.
// 8192 x 8192 bf16: the convolution 48 us (5.6 TB/s) alone, 53 a call; the gradient
// from 8-bit x 92 us a call, bound by instruction issue at 14 warps an SM (two
// channels a thread at twice the warps took 111).  256 tokens of 12288 channels: 17.5 us.

#include <initializer_list>

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kThreads = 128;
constexpr int V = 4;          // channels of a thread
constexpr int NP = V / 2;     // pairs of them
constexpr int kRows = 8;      // rows loaded ahead

struct ConvArgs {
    SsmProblem P;             // P.S: taps
    const float *w, *bias, *cin;
    bool swish, ovec;
    bool fvec;                // four fp32 neighbours may be read and written at once (weights, bias, states, shares)
    void *out;
    float *cout;
    // gradients
    const float *dcout;
    float *dcin, *part;
    int tile;
    unsigned state_block;     // first block that moves states instead
};

// Four neighbouring fp32 values; those at or past `have`, and all of a NULL array, are 0.
// Ordinary loads: the one-token kernel may write a state where it has read it.
__device__ __forceinline__ void load4(const float *p, f2 (&v)[NP], int have, bool vec) {
    float x[V];
    if (!p) {
        v[0] = v[1] = 0;
        return;
    }
    if (vec && have >= V) {
        const float4 q = *reinterpret_cast<const float4 *>(p);
        v[0] = pack2(q.x, q.y);
        v[1] = pack2(q.z, q.w);
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < have ? p[i] : 0.f;
    v[0] = pack2(x[0], x[1]);
    v[1] = pack2(x[2], x[3]);
}
__device__ __forceinline__ void store4(float *p, const f2 (&v)[NP], int have, bool vec) {
    float x[V];
    unpack2(v[0], x[0], x[1]);
    unpack2(v[1], x[2], x[3]);
    store_row<float, V>(p, x, have, vec);
}

// The W taps of four channels, which are 4 W neighbours in memory.
template <int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int c0, int have, f2 (&w)[W][NP], f2 (&b)[NP]) {
    float x[V * W];
    const float *p = a.w + (int64_t)c0 * W;
    if (a.fvec && have >= V) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float4 q = __ldg(reinterpret_cast<const float4 *>(p) + i);
            x[4 * i] = q.x; x[4 * i + 1] = q.y; x[4 * i + 2] = q.z; x[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * W; ++i) x[i] = i < have * W ? p[i] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
        for (int j = 0; j < NP; ++j) w[k][j] = pack2(x[2 * j * W + k], x[(2 * j + 1) * W + k]);
    load4(a.bias ? a.bias + c0 : nullptr, b, have, a.fvec);
}

// A row as pairs; `scale`: what a code stands for.
template <typename IN>
__device__ __forceinline__ void to_pairs(const Raw<IN, V> &r, float scale, f2 (&x)[NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        x[j] = pack2(r.get(2 * j), r.get(2 * j + 1));
        if constexpr (sizeof(IN) == 1) x[j] = mul2(x[j], pack2(scale, scale));
    }
}
template <typename IN>
__device__ __forceinline__ float scale_of(const Rows &u, int64_t t, int c0) {
    if constexpr (sizeof(IN) == 1) return __ldg(u.scales + t * u.ngroups + c0 / kPackGroup);
    return 1.f;
}

// The W - 1 inputs before token t of sequence n = [sa, sb).
template <typename IN, int W>
__device__ __forceinline__ void load_window(const ConvArgs &a, int n, int64_t sa, int64_t t, int c0, int have,
                                            f2 (&x)[W][NP]) {
    const SsmProblem &P = a.P;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t u = t - (W - 1) + k;
        if (u >= sa) {
            Raw<IN, V> r;
            r.load((const IN *)P.u.p + u * P.u.stride + c0, have, P.u.vec);
            to_pairs<IN>(r, scale_of<IN>(P.u, u, c0), x[k]);
        } else {
            // u - sa + W - 1 is in 0 .. W - 2
            load4(a.cin ? a.cin + ((int64_t)n * (W - 1) + (u - sa + W - 1)) * P.D + c0 : nullptr, x[k], have, a.fvec);
        }
    }
}

template <int W>
__device__ __forceinline__ void shift(f2 (&x)[W][NP]) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int j = 0; j < NP; ++j) x[k][j] = x[k + 1][j];
}

// c_t of four channels from the window.
template <int W>
__device__ __forceinline__ void convolve(const f2 (&w)[W][NP], const f2 (&b)[NP], const f2 (&x)[W][NP], f2 (&c)[NP]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        c[j] = b[j];
#pragma unroll
        for (int k = 0; k < W; ++k) c[j] = fma2(w[k][j], x[k][j], c[j]);
    }
}

// Sigmoid of a pair.
__device__ __forceinline__ f2 sigmoid_pair(f2 c) {
    const f2 e = add2(exp2_pair(mul2(c, pack2(-kLog2e, -kLog2e))), pack2(1.f, 1.f));
    float x, y;
    unpack2(e, x, y);
    return pack2(rcp_fast(x), rcp_fast(y));
}

template <typename OUT, bool FULL>
__device__ __forceinline__ void store_pairs(OUT *p, const f2 (&v)[NP], int have, bool vec) {
    float x[V];
    unpack2(v[0], x[0], x[1]);
    unpack2(v[1], x[2], x[3]);
    store_row<OUT, V, FULL>(p, x, have, vec);
}

// Tokens [t, end) of one sequence.  FULL: every access may take four elements.
template <typename IN, typename OUT, int W, bool FULL>
__device__ __forceinline__ void conv_run(const ConvArgs &a, const f2 (&w)[W][NP], const f2 (&b)[NP], f2 (&x)[W][NP],
                                         int64_t t, int64_t end, int c0, int have) {
    const SsmProblem &P = a.P;
    const int64_t stride = P.u.stride, D = P.D;
    const IN *px = (const IN *)P.u.p + t * stride + c0;
    OUT *po = (OUT *)a.out + t * D + c0;
    auto token = [&](const Raw<IN, V> &r) {
        f2 c[NP];
        to_pairs<IN>(r, 1.f, x[W - 1]);
        convolve<W>(w, b, x, c);
        if (a.swish) {
#pragma unroll
            for (int j = 0; j < NP; ++j) c[j] = mul2(c[j], sigmoid_pair(c[j]));
        }
        store_pairs<OUT, FULL>(po, c, have, a.ovec);
        shift<W>(x);
        po += D;
    };
    int left = (int)(end - t);
    if (left >= kRows) {
        Raw<IN, V> next[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i, px += stride) next[i].template load<FULL>(px, have, P.u.vec);
        for (; left >= kRows; left -= kRows) {
            Raw<IN, V> r[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) r[i] = next[i];
            if (left >= 2 * kRows) {
#pragma unroll
                for (int i = 0; i < kRows; ++i, px += stride) next[i].template load<FULL>(px, have, P.u.vec);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) token(r[i]);
        }
    }
    for (; left > 0; --left, px += stride) {
        Raw<IN, V> r;
        r.template load<FULL>(px, have, P.u.vec);
        token(r);
    }
}

// The last W - 1 inputs of every sequence.  A thread owns one channel of one
// sequence and reads before it writes: cout may be cin.
template <typename IN, int W>
__device__ __forceinline__ void conv_state(const ConvArgs &a, int64_t i) {
    const SsmProblem &P = a.P;
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
template <typename IN, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_state_kernel(const __grid_constant__ ConvArgs a) {
    conv_state<IN, W>(a, (int64_t)blockIdx.x * kThreads + threadIdx.x);
}

template <typename IN, typename OUT, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_kernel(const __grid_constant__ ConvArgs a) {
    const SsmProblem &P = a.P;
    if (blockIdx.x >= a.state_block) {         // the blocks behind: the state
        conv_state<IN, W>(a, (int64_t)(blockIdx.x - a.state_block) * kThreads + threadIdx.x);
        return;
    }
    const int nvb = (P.D + V * kThreads - 1) / (V * kThreads);
    const int c0 = ((int)(blockIdx.x % nvb) * kThreads + threadIdx.x) * V;
    const int64_t t0 = (int64_t)(blockIdx.x / nvb) * a.tile, t1 = min(t0 + a.tile, (int64_t)P.T);
    const int have = P.D - c0;
    if (have <= 0) return;
    const bool full = P.u.vec && a.ovec && have >= V;
    f2 w[W][NP], b[NP], x[W][NP];
    int n = 0;
    int64_t sa = 0, sb = 0, t = t0;
    load_taps<W>(a, c0, have, w, b);
    while (t < t1) {
        if (!find_seq(P.cu, P.N, P.T, P.seq_len, t, n, sa, sb)) {
            t = sa;                            // rows outside every sequence stay as they are
            continue;
        }
        const int64_t end = min(sb, t1);
        load_window<IN, W>(a, n, sa, t, c0, have, x);
        if (full) conv_run<IN, OUT, W, true>(a, w, b, x, t, end, c0, have);
        else conv_run<IN, OUT, W, false>(a, w, b, x, t, end, c0, have);
        t = end;
    }
}

// One token a sequence: output and new state in one pass (cout may be cin: a thread
// reads what it writes).
template <typename IN, typename OUT, int W>
__global__ void __launch_bounds__(kThreads) kda_ssm_conv_token_kernel(const __grid_constant__ ConvArgs a) {
    const SsmProblem &P = a.P;
    const int nv = (P.D + V * kThreads - 1) / (V * kThreads);
    const int64_t n = blockIdx.x / nv;
    const int c0 = ((int)(blockIdx.x % nv) * kThreads + threadIdx.x) * V, have = P.D - c0;
    if (have <= 0) return;
    f2 w[W][NP], b[NP], x[W][NP], c[NP];
    Raw<IN, V> r;
    r.load((const IN *)P.u.p + n * P.u.stride + c0, have, P.u.vec);
    load_window<IN, W>(a, (int)n, n, n, c0, have, x);
    load_taps<W>(a, c0, have, w, b);
    to_pairs<IN>(r, 1.f, x[W - 1]);
    convolve<W>(w, b, x, c);
    if (a.swish) {
#pragma unroll
        for (int j = 0; j < NP; ++j) c[j] = mul2(c[j], sigmoid_pair(c[j]));
    }
    store_pairs<OUT, false>((OUT *)a.out + n * P.D + c0, c, have, a.ovec);
    if (a.cout) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) store4(a.cout + (n * (W - 1) + k) * P.D + c0, x[k + 1], have, a.fvec);
    }
}

// What a run gathers.
template <int W>
struct Back {
    f2 w[W][NP], b[NP], x[W][NP], dc[W][NP], dw[W][NP], db[NP];

    // One step: token t's row r and gradient y.  `own`: counted by this run.
    template <typename IN, typename DY, bool OWN>
    __device__ __forceinline__ void step(const Raw<IN, V> &r, const Raw<DY, V> &y, float scale, bool swish) {
        to_pairs<IN>(r, scale, x[W - 1]);
        to_pairs<DY>(y, 1.f, dc[W - 1]);
        if (swish) {
            f2 c[NP];
            convolve<W>(w, b, x, c);
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                // s + c s (1 - s) = s (1 + c (1 - s))
                const f2 s = sigmoid_pair(c[j]);
                const f2 e = fma2(mul2(c[j], pack2(-1.f, -1.f)), s, c[j]);
                dc[W - 1][j] = mul2(dc[W - 1][j], fma2(s, e, s));
            }
        }
        if (OWN) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                db[j] = add2(db[j], dc[W - 1][j]);
#pragma unroll
                for (int k = 0; k < W; ++k) dw[k][j] = fma2(dc[W - 1][j], x[k][j], dw[k][j]);
            }
        }
    }
    // The gradient of the position W - 1 tokens back, now complete.
    __device__ __forceinline__ void complete(f2 (&o)[NP]) const {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
            o[j] = mul2(w[W - 1][j], dc[0][j]);
#pragma unroll
            for (int k = 1; k < W; ++k) o[j] = fma2(w[W - 1 - k][j], dc[k][j], o[j]);
        }
    }
    __device__ __forceinline__ void move() {
        shift<W>(x);
        shift<W>(dc);
    }
};

// Steps [t, end) whose positions t - (W-1) are plain tokens of this run: no state in
// or out, no end of the sequence among them.
template <typename IN, typename DY, typename OUT, int W, bool FULL>
__device__ __forceinline__ void back_run(const ConvArgs &a, Back<W> &k, int64_t t, int64_t end, int c0, int have) {
    constexpr int PB = 4;                      // rows (of x and of d_out) loaded ahead
    const SsmProblem &P = a.P;
    const int64_t sx = P.u.stride, sy = P.dy.stride, D = P.D;
    const IN *px = (const IN *)P.u.p + t * sx + c0;
    const DY *py = (const DY *)P.dy.p + t * sy + c0;
    const float *ps = P.u.scales + t * P.u.ngroups + c0 / kPackGroup;
    OUT *po = (OUT *)a.out + (t - (W - 1)) * D + c0;
    int left = (int)(end - t);
    Raw<IN, V> nx[PB];
    Raw<DY, V> ny[PB];
    float ns[PB];
    auto fetch = [&](int i) {
        nx[i].template load<FULL>(px, have, P.u.vec);
        ny[i].template load<FULL>(py, have, P.dy.vec);
        ns[i] = 1.f;
        if constexpr (sizeof(IN) == 1) {
            ns[i] = __ldg(ps);
            ps += P.u.ngroups;
        }
        px += sx;
        py += sy;
    };
    auto token = [&](const Raw<IN, V> &x, const Raw<DY, V> &y, float s) {
        f2 o[NP];
        k.template step<IN, DY, true>(x, y, s, a.swish);
        k.complete(o);
        store_pairs<OUT, FULL>(po, o, have, a.ovec);
        po += D;
        k.move();
    };
    if (left >= PB) {
#pragma unroll
        for (int i = 0; i < PB; ++i) fetch(i);
        for (; left >= PB; left -= PB) {
            Raw<IN, V> rx[PB];
            Raw<DY, V> ry[PB];
            float rs[PB];
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                rx[i] = nx[i];
                ry[i] = ny[i];
                rs[i] = ns[i];
            }
            if (left >= 2 * PB) {
#pragma unroll
                for (int i = 0; i < PB; ++i) fetch(i);
            }
#pragma unroll
            for (int i = 0; i < PB; ++i) token(rx[i], ry[i], rs[i]);
        }
    }
    for (; left > 0; --left) {
        fetch(0);
        token(nx[0], ny[0], ns[0]);
    }
}

template <typename IN, typename DY, typename OUT, int W>
__global__ void __launch_bounds__(kThreads, 4) kda_ssm_conv_backward_kernel(const __grid_constant__ ConvArgs a) {
    let_next();
    const SsmProblem &P = a.P;
    const int nvb = (P.D + V * kThreads - 1) / (V * kThreads);
    const int c0 = ((int)(blockIdx.x % nvb) * kThreads + threadIdx.x) * V;
    const int64_t tile = blockIdx.x / nvb;
    const int64_t t0 = tile * a.tile, t1 = min(t0 + a.tile, (int64_t)P.T);
    const int have = P.D - c0;
    if (have <= 0) return;
    const bool full = P.u.vec && P.dy.vec && a.ovec && have >= V;
    Back<W> k;
    load_taps<W>(a, c0, have, k.w, k.b);
#pragma unroll
    for (int j = 0; j < NP; ++j) {
        k.db[j] = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) k.dw[i][j] = 0;
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
        load_window<IN, W>(a, n, sa, t, c0, have, k.x);
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) k.dc[i][j] = 0;
        // step t gives dc_t and completes position t - (W-1); past the end dc = 0.  The
        // first W - 1 steps and those from s1 on are the careful ones.
        while (t < s1 + W - 1) {
            if (t == s0 + W - 1 && t < s1 && !(a.dcout && s1 > sb - (W - 1))) {
                if (full) back_run<IN, DY, OUT, W, true>(a, k, t, s1, c0, have);
                else back_run<IN, DY, OUT, W, false>(a, k, t, s1, c0, have);
                t = s1;
                continue;
            }
            Raw<IN, V> r;
            Raw<DY, V> y;
            r.clear();
            y.clear();
            float scale = 0.f;
            if (t < last) {
                r.load((const IN *)P.u.p + t * P.u.stride + c0, have, P.u.vec);
                y.load((const DY *)P.dy.p + t * P.dy.stride + c0, have, P.dy.vec);
                scale = scale_of<IN>(P.u, t, c0);
            }
            if (t < s1) k.template step<IN, DY, true>(r, y, scale, a.swish);
            else k.template step<IN, DY, false>(r, y, scale, a.swish && t < last);
            const int64_t p = t - (W - 1);                // the position whose gradient is complete
            if (p >= s0 || s0 == sa) {                    // p < s0 = sa: the carried state
                f2 o[NP];
                k.complete(o);
                // the carried state out holds the last W - 1 positions
                const int64_t back = p - (sb - (W - 1));
                if (a.dcout && back >= 0) {
                    f2 e[NP];
                    load4(a.dcout + ((int64_t)n * (W - 1) + back) * P.D + c0, e, have, a.fvec);
#pragma unroll
                    for (int j = 0; j < NP; ++j) o[j] = add2(o[j], e[j]);
                }
                if (p >= sa) {
                    store_pairs<OUT, false>((OUT *)a.out + p * P.D + c0, o, have, a.ovec);
                } else if (a.dcin) {
                    store4(a.dcin + ((int64_t)n * (W - 1) + (p - sa + W - 1)) * P.D + c0, o, have, a.fvec);
                }
            }
            k.move();
            ++t;
        }
        t = s1;
    }
    float *part = a.part + tile * (W + 1) * P.D + c0;
#pragma unroll
    for (int i = 0; i < W; ++i) store4(part + (int64_t)i * P.D, k.dw[i], have, a.fvec);
    store4(part + (int64_t)W * P.D, k.db, have, a.fvec);
}

// dw and dbias: the runs' shares, added in their order.  A warp takes 32
// channels of one row of the shares; its kRuns warps add every kRuns-th run and
// join through shared memory.  The blocks behind hand the gradient of the state
// of sequences without tokens on, as those hand on their state.
constexpr int kRuns = 8;
__global__ void __launch_bounds__(32 * kRuns)
kda_ssm_conv_reduce_kernel(const __grid_constant__ ConvArgs a, int64_t tiles, unsigned blocks, float *dw, float *dbias) {
    wait_before();
    const SsmProblem &P = a.P;
    const int D = P.D, W = P.S;
    if (blockIdx.x >= blocks) {
        const int64_t per = (int64_t)(W - 1) * D, i = (int64_t)(blockIdx.x - blocks) * (32 * kRuns) + threadIdx.x;
        if (i >= per * P.N) return;
        int64_t sa, sb;
        seq_bounds(P.cu, (int)(i / per), P.T, P.seq_len, sa, sb);
        if (sa == sb) a.dcin[i] = a.dcout ? a.dcout[i] : 0.f;
        return;
    }
    __shared__ float s[kRuns][32];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int nb = (D + 31) / 32;
    const int k = blockIdx.x / nb, c = (blockIdx.x % nb) * 32 + lane;
    float v = 0.f;
    if (c < D) {
        const float *p = a.part + (int64_t)k * D + c;
        const int64_t step = (int64_t)(W + 1) * D;
#pragma unroll 8
        for (int64_t i = y; i < tiles; i += kRuns) v += p[i * step];
    }
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

// Tokens of a run: as many as make the blocks fill the GPU's places (`per_sm` an SM)
// a whole number of times, with at most `most` tokens a run; at least 16, which keeps the
// rows that two runs read within a fifth.  (8192 x 8192, gradient from 8 bits, the kernel
// alone under a profiler: runs of 128, which fill 1.7 times the places, 93 us, of 216,
// once, 88.)
int run_length(int64_t T, int32_t D, int per_sm, int most) {
    const int64_t work = T * ((D + V * kThreads - 1) / (V * kThreads)), places = 152 * (int64_t)per_sm;
    int64_t rounds = (work + places * most - 1) / (places * most);
    if (rounds < 1) rounds = 1;
    const int64_t tile = (work + places * rounds - 1) / (places * rounds);
    return tile < 16 ? 16 : (int)tile;
}

template <typename IN, typename OUT, int W>
cudaError_t forward(ConvArgs &a, cudaStream_t stream) {
    const SsmProblem &P = a.P;
    const int64_t across = (P.D + V * kThreads - 1) / (V * kThreads);
    if (!P.cu && P.seq_len == 1) {
        kda_ssm_conv_token_kernel<IN, OUT, W><<<(unsigned)(P.N * across), kThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    const unsigned state_blocks = a.cout ? (unsigned)(((int64_t)P.N * P.D + kThreads - 1) / kThreads) : 0;
    // a state in place is written only behind the kernel that reads it
    const bool apart = a.cout == a.cin || P.T == 0;
    if (P.T > 0) {
        a.tile = run_length(P.T, P.D, sizeof(IN) == 2 ? 5 : 4, 200);
        a.state_block = (unsigned)((P.T + a.tile - 1) / a.tile * across);
        kda_ssm_conv_kernel<IN, OUT, W><<<a.state_block + (apart ? 0 : state_blocks), kThreads, 0, stream>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (state_blocks && apart) {
        kda_ssm_conv_state_kernel<IN, W><<<state_blocks, kThreads, 0, stream>>>(a);
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

template <typename IN, typename DY, typename OUT, int W>
cudaError_t backward(ConvArgs &a, float *dw, float *dbias, cudaStream_t stream) {
    const SsmProblem &P = a.P;
    const int64_t tiles = kda_ssm_conv_backward_tiles(P, &a.tile);
    if (tiles > 0) {
        const int64_t blocks = tiles * ((P.D + V * kThreads - 1) / (V * kThreads));
        kda_ssm_conv_backward_kernel<IN, DY, OUT, W><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const unsigned blocks = dw || dbias ? (unsigned)((W + 1) * ((P.D + 31) / 32)) : 0;
    const int64_t n = a.dcin && (P.cu || P.seq_len == 0) ? (int64_t)P.N * (W - 1) * P.D : 0;
    const unsigned more = (unsigned)((n + 32 * kRuns - 1) / (32 * kRuns));
    if (blocks + more == 0) return cudaSuccess;
    return launch_behind(tiles > 0, kda_ssm_conv_reduce_kernel, blocks + more, 32 * kRuns, 0, stream, a, tiles, blocks, dw, dbias);
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
    return ((uintptr_t)p & 15u) == 0 && (int64_t)P.D * es % (V * es) == 0;
}
bool all_aligned(const SsmProblem &P, std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p & 15u) return false;
    return P.D % V == 0;
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
    a.fvec = all_aligned(P, {w, bias, cin, cout});
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return forward_taps<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (ib) return forward_taps<__nv_bfloat16, float>(a, stream);
    if (ob) return forward_taps<float, __nv_bfloat16>(a, stream);
    return forward_taps<float, float>(a, stream);
}

int64_t kda_ssm_conv_backward_tiles(const SsmProblem &P, int *tile) {
    *tile = run_length(P.T, P.D, 4, 256);
    return P.N == 0 ? 0 : ((int64_t)P.T + *tile - 1) / *tile;   // (rows without a sequence belong to no run)
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
    a.fvec = all_aligned(P, {w, bias, cin, dcout, dcin, workspace});
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return backward_input<__nv_bfloat16, __nv_bfloat16>(a, dw, dbias, stream);
    if (ib) return backward_input<__nv_bfloat16, float>(a, dw, dbias, stream);
    if (ob) return backward_input<float, __nv_bfloat16>(a, dw, dbias, stream);
    return backward_input<float, float>(a, dw, dbias, stream);
}
