// kda_ssm_backward.cu -- gradients of the selective scan.
//
// With a_t = exp(Delta_t A), h_t = a_t h_{t-1} + Delta_t u_t B_t, and the
// gradient dyp_t = dy_t z_t Sigmoid(z_t) of the ungated output, the adjoint of
// the state runs back through each sequence:
//
//   g_t = C_t dyp_t + a_{t+1} g_{t+1}            (g after the last token: d_final)
//   dC_t[n] = sum_d dyp_t h_t          dB_t[n] = sum_d g_t Delta_t u_t
//   p_t = sum_n g_t B_t                r_t = sum_n g_t a_t h_{t-1} A
//   du_t = Delta_t p_t + D dyp_t       dDelta_t = u_t p_t + r_t
//   dA = sum_t g_t a_t h_{t-1} Delta_t dD = sum_t dyp_t u_t
//   ddt = dDelta Sigmoid(dt + bias)    dz_t = dy_t y_t (s + z s (1 - s)), s = Sigmoid(z_t)
//   d_init = a_1 g_1
//
// The states come again from the forward's states at the chunk starts (every 32
// tokens).  Lanes hold states as in the scan (four of one channel).  A tile is
// one chunk, taken in two halves of 16 tokens whose states stay in registers:
// the second half's start is run up to first, so a decay is formed 2.5 times, and no
// state goes through memory.  Sums over a channel's states are exchanges between
// its LN lanes; sums over channels (dB, dC) are exchanges between the lanes of
// a warp, then shared memory between the warps, then a workspace row per block
// that a second kernel adds up in order.

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int TT = kSsmTile;
constexpr int HT = TT / 2;
constexpr float kLn2 = 0.6931471805599453f;

__device__ unsigned g_ssm_status = 0;

struct BackArgs {
    SsmProblem P;
    const float *init, *chunks, *d_final;
    int64_t chunk_capacity;
    void *du, *ddt, *dz;
    float *dA, *dskip, *dbias, *d_init;   // per sequence: [N, D, S], [N, D], [N, D] (the results themselves for N = 1)
    float *part;                          // [blocks across D][T][2 SP]
    bool ovec, obf;
};

template <int LN>
struct Layout {
    static constexpr int CW = 32 / LN, CB = kWarps * CW, SP = 4 * LN, E = CB / 4;
    static constexpr int YS = CB + 8;
    static constexpr int BI = (TT * LN + kThreads - 1) / kThreads;
    struct Smem {
        float4 d[TT][CB];                  // Delta, Delta u, dyp, u
        float4 b[TT][LN], c[TT][LN];
        float p[TT][YS], r[TT][YS], y[TT][YS];
        float part[kWarps][TT][2 * SP];    // dC, dB
    };
};

template <int E>
__device__ __forceinline__ void store_grad(void *p, int64_t at, const float (&v)[E], int have, bool vec, bool bf) {
    if (bf) store_row<__nv_bfloat16, E>((__nv_bfloat16 *)p + at, v, have, vec);
    else store_row<float, E>((float *)p + at, v, have, vec);
}

// X: type of u and z (int8 codes or IN); IN: type of dt, B, C and d_out.
template <typename X, typename IN, int LN>
__global__ void __launch_bounds__(kThreads)
kda_ssm_scan_backward_kernel(const BackArgs a) {
    using L = Layout<LN>;
    constexpr int CW = L::CW, CB = L::CB, E = L::E, SP = L::SP;
    constexpr bool kCodes = sizeof(X) == 1;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename L::Smem &sm = *reinterpret_cast<typename L::Smem *>(smem_raw);
    __shared__ int s_seq;

    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB, cb = blockIdx.x % ncb;
    const int n = longest_first(P.cu, P.N, P.T, P.seq_len, blockIdx.x / ncb, &s_seq);
    const int ch0 = cb * CB;
    int64_t sa, sb;
    seq_bounds(P.cu, n, P.T, P.seq_len, sa, sb);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wc = warp * CW + lane / LN, ch = ch0 + wc;
    const int q = lane % LN, n0 = 4 * q;
    const bool live = ch < P.D;

    f2 A01 = 0, A23 = 0, g01 = 0, g23 = 0, dA01 = 0, dA23 = 0;
    if (live) {
        const float4 A = load_states(P.A + (int64_t)ch * P.S, n0, P.S, P.svec);
        A01 = pack2(A.x * kLog2e, A.y * kLog2e);
        A23 = pack2(A.z * kLog2e, A.w * kLog2e);
        if (a.d_final) {
            const float4 g = load_states(a.d_final + ((int64_t)n * P.D + ch) * P.S, n0, P.S, P.svec);
            g01 = pack2(g.x, g.y);
            g23 = pack2(g.z, g.w);
        }
    }

    const int srow = tid >> 2, sc = (tid & 3) * E;
    const int have = P.D - (ch0 + sc);
    float bias[E], skip[E], sum_skip[E], sum_bias[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = (P.dt_bias && i < have) ? P.dt_bias[ch0 + sc + i] : 0.f;
        skip[i] = (P.skip && i < have) ? P.skip[ch0 + sc + i] : 0.f;
        sum_skip[i] = sum_bias[i] = 0.f;
    }
    constexpr int kScales = E <= kPackGroup ? 1 : E / kPackGroup;
    Raw<X, E> ru, rz;
    Raw<IN, E> rd, ry;
    Raw<IN, 4> rb[L::BI], rc[L::BI];
    float su[kScales], sz[kScales];
    float4 rh;                                   // the tile's start state
    const int64_t row0 = ckpt_first_row(P.cu, n, P.T, P.seq_len, TT);
    auto fetch = [&](int64_t tile) {
        const int64_t t0 = sa + tile * TT, t = t0 + srow;
        ru.clear();
        rz.clear();
        rd.clear();
        ry.clear();
#pragma unroll
        for (int i = 0; i < kScales; ++i) su[i] = sz[i] = 0.f;
        if (t < sb && have > 0) {
            ru.load((const X *)P.u.p + t * P.u.stride + ch0 + sc, have, P.u.vec);
            if (P.z.p) rz.load((const X *)P.z.p + t * P.z.stride + ch0 + sc, have, P.z.vec);
            rd.load((const IN *)P.dt.p + t * P.dt.stride + ch0 + sc, have, P.dt.vec);
            ry.load((const IN *)P.dy.p + t * P.dy.stride + ch0 + sc, have, P.dy.vec);
            if constexpr (kCodes) {
#pragma unroll
                for (int i = 0; i < kScales; ++i) {
                    const int64_t g = t * P.u.ngroups + (ch0 + sc) / kPackGroup + i;
                    su[i] = P.u.scales[g];
                    if (P.z.p) sz[i] = P.z.scales[g];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < L::BI; ++k) {
            const int i = tid + k * kThreads;
            const int64_t tb = t0 + i / LN;
            const int nb = 4 * (i % LN);
            rb[k].clear();
            rc[k].clear();
            if (i < TT * LN && tb < sb && nb < P.S) {
                rb[k].load((const IN *)P.B.p + tb * P.B.stride + nb, P.S - nb, P.B.vec);
                rc[k].load((const IN *)P.C.p + tb * P.C.stride + nb, P.S - nb, P.C.vec);
            }
        }
        rh = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) {
            if (tile == 0) {
                if (a.init) rh = load_states(a.init + ((int64_t)n * P.D + ch) * P.S, n0, P.S, P.svec);
            } else {
                const int64_t row = row0 + tile - 1;
                if (row < a.chunk_capacity)
                    rh = load_states(a.chunks + (row * P.D + ch) * P.S, n0, P.S, P.svec);
                else
                    atomicOr(&g_ssm_status, kBwdMissingState);
            }
        }
    };
    const int64_t tiles = (sb - sa + TT - 1) / TT;
    if (tiles > 0) fetch(tiles - 1);

#pragma unroll 1
    for (int64_t tile = tiles - 1; tile >= 0; --tile) {
        const int64_t t0 = sa + tile * TT;
        const bool mine = t0 + srow < sb && have > 0;
        const f2 h0_01 = pack2(rh.x, rh.y), h0_23 = pack2(rh.z, rh.w);
        float zz[E], dyv[E], raw[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            float u = ru.get(i), z = rz.get(i);
            if constexpr (kCodes) {
                u *= su[i / kPackGroup];
                z *= sz[i / kPackGroup];
            }
            zz[i] = z;
            dyv[i] = ry.get(i);
            raw[i] = rd.get(i) + bias[i];
            const float dl = mine ? (P.softplus ? softplus_fast(raw[i]) : raw[i]) : 0.f;
            const float dyp = P.z.p ? dyv[i] * (z * sigmoid_fast(z)) : dyv[i];
            sm.d[srow][sc + i] = make_float4(dl, dl * u, dyp, u);
        }
#pragma unroll
        for (int k = 0; k < L::BI; ++k) {
            const int i = tid + k * kThreads;
            if (i < TT * LN) {
                sm.b[i / LN][i % LN] = make_float4(rb[k].get(0), rb[k].get(1), rb[k].get(2), rb[k].get(3));
                sm.c[i / LN][i % LN] = make_float4(rc[k].get(0), rc[k].get(1), rc[k].get(2), rc[k].get(3));
            }
        }
        if (tile > 0) fetch(tile - 1);
        __syncthreads();

#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
            f2 s01 = h0_01, s23 = h0_23;
            if (half) {
#pragma unroll 4
                for (int t = 0; t < HT; ++t) {
                    const float4 d = sm.d[t][wc];
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(&sm.b[t][q]);
                    const f2 dd = pack2(d.x, d.x), du = pack2(d.y, d.y);
                    s01 = fma2(exp2_pair(mul2(dd, A01)), s01, mul2(du, b.x));
                    s23 = fma2(exp2_pair(mul2(dd, A23)), s23, mul2(du, b.y));
                }
            }
            const int tb = half * HT;
            f2 H01[HT + 1], H23[HT + 1];
            H01[0] = s01;
            H23[0] = s23;
#pragma unroll
            for (int i = 0; i < HT; ++i) {
                const float4 d = sm.d[tb + i][wc];
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(&sm.b[tb + i][q]);
                const f2 dd = pack2(d.x, d.x), du = pack2(d.y, d.y);
                H01[i + 1] = fma2(exp2_pair(mul2(dd, A01)), H01[i], mul2(du, b.x));
                H23[i + 1] = fma2(exp2_pair(mul2(dd, A23)), H23[i], mul2(du, b.y));
            }
            constexpr int G = LN < 4 ? 4 : LN;
#pragma unroll
            for (int j = HT - G; j >= 0; j -= G) {
                float vp[G], vr[G], vy[G];
#pragma unroll
                for (int i = G - 1; i >= 0; --i) {
                    const int t = tb + j + i;
                    const float4 d = sm.d[t][wc];
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(&sm.b[t][q]);
                    const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(&sm.c[t][q]);
                    const f2 dd = pack2(d.x, d.x), du = pack2(d.y, d.y), dyp = pack2(d.z, d.z);
                    g01 = fma2(dyp, c.x, g01);
                    g23 = fma2(dyp, c.y, g23);
                    vy[i] = sum2(fma2(c.x, H01[j + i + 1], mul2(c.y, H23[j + i + 1])));
                    vp[i] = sum2(fma2(b.x, g01, mul2(b.y, g23)));
                    float v[8];
                    unpack2(mul2(dyp, H01[j + i + 1]), v[0], v[1]);
                    unpack2(mul2(dyp, H23[j + i + 1]), v[2], v[3]);
                    unpack2(mul2(du, g01), v[4], v[5]);
                    unpack2(mul2(du, g23), v[6], v[7]);
                    g01 = mul2(g01, exp2_pair(mul2(dd, A01)));
                    g23 = mul2(g23, exp2_pair(mul2(dd, A23)));
                    const f2 x01 = mul2(g01, H01[j + i]), x23 = mul2(g23, H23[j + i]);
                    vr[i] = sum2(fma2(x01, A01, mul2(x23, A23)));
                    dA01 = fma2(x01, dd, dA01);
                    dA23 = fma2(x23, dd, dA23);
                    // over the channels of the warp
                    constexpr int CL = CW < 8 ? CW : 8;
                    reduce_scatter<CL, LN, 8>(v);
#pragma unroll
                    for (int off = CL; off < CW; off *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off * LN);
                    if (lane / LN < CL) {
#pragma unroll
                        for (int k = 0; k < 8 / CL; ++k) {
                            const int vi = (lane / LN) * (8 / CL) + k;
                            sm.part[warp][t][(vi >> 2) * SP + n0 + (vi & 3)] = v[k];
                        }
                    }
                }
                // over the states of a channel
                reduce_scatter<LN, 1, G>(vp);
                reduce_scatter<LN, 1, G>(vr);
                reduce_scatter<LN, 1, G>(vy);
#pragma unroll
                for (int i = 0; i < G / LN; ++i) {
                    const int t = tb + j + q * (G / LN) + i;
                    sm.p[t][wc] = vp[i];
                    sm.r[t][wc] = vr[i];
                    sm.y[t][wc] = vy[i];
                }
            }
        }
        __syncthreads();
        // dB and dC of this block's channels
        for (int i = tid; i < TT * 2 * SP / 4; i += kThreads) {
            const int t = i / (2 * SP / 4), k = i % (2 * SP / 4);
            if (t0 + t < sb) {
                float4 s = *reinterpret_cast<const float4 *>(&sm.part[0][t][4 * k]);
#pragma unroll
                for (int w = 1; w < kWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.part[w][t][4 * k]);
                    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
                }
                *reinterpret_cast<float4 *>(a.part + ((int64_t)cb * P.T + t0 + t) * (2 * SP) + 4 * k) = s;
            }
        }
        if (mine) {
            float o1[E], o2[E], o3[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float4 d = sm.d[srow][sc + i];       // written by this thread
                const float p = sm.p[srow][sc + i], r = sm.r[srow][sc + i] * kLn2;
                o1[i] = fmaf(d.x, p, skip[i] * d.z);
                float x = fmaf(d.w, p, r);
                if (P.softplus) x *= sigmoid_fast(raw[i]);
                o2[i] = x;
                sum_bias[i] += x;
                sum_skip[i] = fmaf(d.z, d.w, sum_skip[i]);
                const float y = fmaf(skip[i], d.w, sm.y[srow][sc + i]), s = sigmoid_fast(zz[i]);
                o3[i] = dyv[i] * y * fmaf(zz[i] * s, 1.f - s, s);
            }
            const int64_t at = (t0 + srow) * P.D + ch0 + sc;
            store_grad<E>(a.du, at, o1, have, a.ovec, a.obf);
            store_grad<E>(a.ddt, at, o2, have, a.ovec, a.obf);
            if (P.z.p) store_grad<E>(a.dz, at, o3, have, a.ovec, a.obf);
        }
    }
    const int64_t at = ((int64_t)n * P.D + ch) * P.S;
    if (live) {
        float4 v;
        unpack2(dA01, v.x, v.y);
        unpack2(dA23, v.z, v.w);
        store_states(a.dA + at, v, n0, P.S, P.svec);
        if (a.d_init) {
            unpack2(g01, v.x, v.y);
            unpack2(g23, v.z, v.w);
            store_states(a.d_init + at, v, n0, P.S, P.svec);
        }
    }
    // dD and ddt_bias: over the 32 rows of threads
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; ++i) {
        sm.p[srow][sc + i] = sum_skip[i];
        sm.r[srow][sc + i] = sum_bias[i];
    }
    __syncthreads();
    for (int c = tid; c < CB; c += kThreads) {
        if (ch0 + c < P.D) {
            float x = 0.f, y = 0.f;
            for (int t = 0; t < TT; ++t) {
                x += sm.p[t][c];
                y += sm.r[t][c];
            }
            if (a.dskip) a.dskip[(int64_t)n * P.D + ch0 + c] = x;
            if (a.dbias) a.dbias[(int64_t)n * P.D + ch0 + c] = y;
        }
    }
}

// dB and dC: the blocks' shares, added in their order.  Tokens outside every
// sequence are left as they are.
template <typename OUT>
__global__ void __launch_bounds__(256)
kda_ssm_reduce_bc_kernel(const SsmProblem P, const float *__restrict__ part, int ncb, int SP, OUT *dB, OUT *dC) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / (2 * SP);
    if (t >= P.T) return;
    const int k = (int)(i - t * (2 * SP)), n = k % SP;
    if (n >= P.S) return;
    if (P.cu) {
        int m;
        int64_t sa, sb;
        if (!find_seq(P.cu, P.N, P.T, P.seq_len, t, m, sa, sb)) return;
    }
    float v = 0.f;
    const float *p = part + i;
    const int64_t step = (int64_t)P.T * 2 * SP;
#pragma unroll 8
    for (int c = 0; c < ncb; ++c) v += p[c * step];
    st_elem((k < SP ? dC : dB) + t * P.S + n, v);
}

// Sums over the sequences of [N, M] into [M].
__global__ void __launch_bounds__(256) kda_ssm_reduce_seq_kernel(const float *__restrict__ part, int N, int64_t M, float *out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= M) return;
    float v = 0.f;
#pragma unroll 4
    for (int n = 0; n < N; ++n) v += part[n * M + i];
    out[i] = v;
}

int lanes_of(int S) { return S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16; }
int blocks_across(const SsmProblem &P) {
    const int CB = kWarps * 32 / lanes_of(P.S);
    return (P.D + CB - 1) / CB;
}
int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

template <typename X, typename IN, int LN>
cudaError_t launch(const BackArgs &a, cudaStream_t stream) {
    using L = Layout<LN>;
    const int smem = (int)sizeof(typename L::Smem);
    cudaError_t e = cudaFuncSetAttribute(kda_ssm_scan_backward_kernel<X, IN, LN>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (int64_t)a.P.N * blocks_across(a.P);
    kda_ssm_scan_backward_kernel<X, IN, LN><<<(unsigned)blocks, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename X, typename IN>
cudaError_t by_states(const BackArgs &a, cudaStream_t s) {
    switch (lanes_of(a.P.S)) {
        case 2: return launch<X, IN, 2>(a, s);
        case 4: return launch<X, IN, 4>(a, s);
        case 8: return launch<X, IN, 8>(a, s);
        default: return launch<X, IN, 16>(a, s);
    }
}

}  // namespace

cudaError_t kda_ssm_read_status(unsigned *status) {
    unsigned w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_ssm_status, sizeof(w));
    if (e == cudaSuccess && w) {
        *status |= w;
        w = 0;
        e = cudaMemcpyToSymbol(g_ssm_status, &w, sizeof(w));
    }
    return e;
}

int64_t kda_ssm_scan_backward_ws(const SsmProblem &P) {
    const int SP = 4 * lanes_of(P.S);
    int64_t n = (int64_t)blocks_across(P) * P.T * 2 * SP;
    if (P.N != 1) n += up4((int64_t)P.N * P.D * P.S) + 2 * up4((int64_t)P.N * P.D);
    return n * (int64_t)sizeof(float);
}

cudaError_t kda_launch_ssm_scan_backward(const SsmProblem &P, const float *init, const float *chunk_states,
                                         int64_t chunk_capacity, const float *d_final, void *du, void *ddt, void *dB,
                                         void *dC, void *dz, float *dA, float *dskip, float *dbias, float *d_init,
                                         float *workspace, cudaStream_t stream) {
    BackArgs a{};
    a.P = P;
    a.init = init;
    a.chunks = chunk_states;
    a.chunk_capacity = chunk_states ? chunk_capacity : 0;
    a.d_final = d_final;
    a.du = du;
    a.ddt = ddt;
    a.dz = dz;
    a.d_init = d_init;
    a.obf = P.out_dtype == KDA_DTYPE_BF16;
    a.ovec = (int64_t)P.D * (a.obf ? 2 : 4) % 16 == 0;
    for (const void *p : {(const void *)du, (const void *)ddt, (const void *)dz})
        if ((uintptr_t)p & 15u) a.ovec = false;
    const int SP = 4 * lanes_of(P.S), ncb = blocks_across(P);
    a.part = workspace;
    float *more = workspace + (int64_t)ncb * P.T * 2 * SP;
    const int64_t nA = (int64_t)P.D * P.S;
    const bool direct = P.N == 1;
    a.dA = direct ? dA : more;
    a.dskip = !dskip ? nullptr : direct ? dskip : more + up4(P.N * nA);
    a.dbias = !dbias ? nullptr : direct ? dbias : more + up4(P.N * nA) + up4((int64_t)P.N * P.D);
    cudaError_t e = cudaSuccess;
    if (P.N > 0) {
        const bool bf = P.in_dtype == KDA_DTYPE_BF16;
        if (P.u.scales) e = bf ? by_states<int8_t, __nv_bfloat16>(a, stream) : by_states<int8_t, float>(a, stream);
        else e = bf ? by_states<__nv_bfloat16, __nv_bfloat16>(a, stream) : by_states<float, float>(a, stream);
        if (e != cudaSuccess) return e;
    }
    if (P.T > 0 && P.N > 0) {
        const int64_t n = (int64_t)P.T * 2 * SP;
        const unsigned blocks = (unsigned)((n + 255) / 256);
        if (a.obf)
            kda_ssm_reduce_bc_kernel<__nv_bfloat16><<<blocks, 256, 0, stream>>>(P, a.part, ncb, SP, (__nv_bfloat16 *)dB, (__nv_bfloat16 *)dC);
        else
            kda_ssm_reduce_bc_kernel<float><<<blocks, 256, 0, stream>>>(P, a.part, ncb, SP, (float *)dB, (float *)dC);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (!direct) {
        kda_ssm_reduce_seq_kernel<<<(unsigned)((nA + 255) / 256), 256, 0, stream>>>(a.dA, P.N, nA, dA);
        if (dskip) kda_ssm_reduce_seq_kernel<<<(unsigned)((P.D + 255) / 256), 256, 0, stream>>>(a.dskip, P.N, P.D, dskip);
        if (dbias) kda_ssm_reduce_seq_kernel<<<(unsigned)((P.D + 255) / 256), 256, 0, stream>>>(a.dbias, P.N, P.D, dbias);
        e = cudaGetLastError();
    }
    return e;
}
