// kda_ssm_scan.cu -- the selective scan over a packed batch.
//
//   Delta = softplus(dt + dt_bias)                       (or dt + dt_bias itself)
//   h_t[d,n] = exp(Delta_t[d] A[d,n]) h_{t-1}[d,n] + Delta_t[d] u_t[d] B_t[n]
//   y_t[d]   = (sum_n C_t[n] h_t[d,n] + D[d] u_t[d]) z_t[d] Sigmoid(z_t[d])
//
// Every state entry is a recurrence of its own.  One lane holds four states of
// one channel, LN >= S / 4 lanes (2, 4, 8 or 16) hold a channel, a block of four
// warps 128 / LN channels of one sequence, and walks the sequence in
// tiles of 32 tokens: the block stages Delta, Delta u, B and C of a tile in
// shared memory as fp32 while the next tile's loads are in flight, each warp
// runs its recurrences over the tile, and the block writes the tile's outputs.
// Tokens past the sequence's end are staged as Delta = 0, which leaves a state as
// it is.

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int TT = kSsmTile;

struct ScanArgs {
    SsmProblem P;
    const float *init;
    void *out;
    float *fin;
    float *chunks;
    int64_t chunk_capacity;
    bool ovec;
};

template <int LN>
struct Layout {
    static constexpr int CW = 32 / LN;         // channels of a warp
    static constexpr int CB = kWarps * CW;     // channels of a block
    static constexpr int E = CB / 4;           // elements of a row that one thread stages (4 threads a row)
    static constexpr int YS = CB + 8;          // row of the output tile: the 4 tokens a warp writes at once take different banks
    static constexpr int BI = (TT * LN + kThreads - 1) / kThreads;   // 4-element pieces of B (and C) that a thread stages
    struct Smem {
        float2 d[2][TT][CB];                   // Delta, Delta u
        float4 b[2][TT][LN], c[2][TT][LN];
        float y[TT][YS];
    };
};

template <typename IN, typename OUT, int LN>
__global__ void __launch_bounds__(kThreads)
kda_ssm_scan_kernel(const ScanArgs a) {
    using L = Layout<LN>;
    constexpr int CW = L::CW, CB = L::CB, E = L::E;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename L::Smem &sm = *reinterpret_cast<typename L::Smem *>(smem_raw);
    __shared__ int s_seq;

    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB;
    const int n = longest_first(P.cu, P.N, P.T, P.seq_len, blockIdx.x / ncb, &s_seq);
    const int ch0 = (blockIdx.x % ncb) * CB;
    int64_t sa, sb;
    seq_bounds(P.cu, n, P.T, P.seq_len, sa, sb);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // this lane's states
    const int wc = warp * CW + lane / LN;      // channel within the block
    const int ch = ch0 + wc;
    const int q = lane % LN, n0 = 4 * q;
    const bool live = ch < P.D;
    f2 A01 = 0, A23 = 0, h01 = 0, h23 = 0;
    if (live) {
        const float4 A = load_states(P.A + (int64_t)ch * P.S, n0, P.S, P.svec);
        A01 = pack2(A.x * kLog2e, A.y * kLog2e);
        A23 = pack2(A.z * kLog2e, A.w * kLog2e);
        if (a.init) {
            const float4 h = load_states(a.init + ((int64_t)n * P.D + ch) * P.S, n0, P.S, P.svec);
            h01 = pack2(h.x, h.y);
            h23 = pack2(h.z, h.w);
        }
    }

    // this thread's part of the staging: row tid / 4, E channels
    const int srow = tid >> 2, sc = (tid & 3) * E;
    const int have = P.D - (ch0 + sc);         // channels that exist (may be <= 0)
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = (P.dt_bias && i < have) ? P.dt_bias[ch0 + sc + i] : 0.f;
        skip[i] = (P.skip && i < have) ? P.skip[ch0 + sc + i] : 0.f;
    }
    Raw<IN, E> ru, rd, rz;
    Raw<IN, 4> rb[L::BI], rc[L::BI];
    auto fetch = [&](int64_t t0) {
        const int64_t t = t0 + srow;
        ru.clear();
        rd.clear();
        rz.clear();
        if (t < sb && have > 0) {
            ru.load((const IN *)P.u.p + t * P.u.stride + ch0 + sc, have, P.u.vec);
            rd.load((const IN *)P.dt.p + t * P.dt.stride + ch0 + sc, have, P.dt.vec);
            if (P.z.p) rz.load((const IN *)P.z.p + t * P.z.stride + ch0 + sc, have, P.z.vec);
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
    };
    fetch(sa);
    const int64_t row0 = a.chunks ? ckpt_first_row(P.cu, n, P.T, P.seq_len, TT) : 0;

    for (int64_t t0 = sa, tile = 0; t0 < sb; t0 += TT, ++tile) {
        const int buf = (int)(tile & 1);
        // stage: tokens past the end have Delta = 0
        {
            const bool in = t0 + srow < sb;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = rd.get(i) + bias[i];
                const float dl = in ? (P.softplus ? softplus_fast(x) : x) : 0.f;
                sm.d[buf][srow][sc + i] = make_float2(dl, dl * ru.get(i));
            }
#pragma unroll
            for (int k = 0; k < L::BI; ++k) {
                const int i = tid + k * kThreads;
                if (i < TT * LN) {
                    sm.b[buf][i / LN][i % LN] = make_float4(rb[k].get(0), rb[k].get(1), rb[k].get(2), rb[k].get(3));
                    sm.c[buf][i / LN][i % LN] = make_float4(rc[k].get(0), rc[k].get(1), rc[k].get(2), rc[k].get(3));
                }
            }
        }
        const Raw<IN, E> cu_u = ru, cu_z = rz;
        if (t0 + TT < sb) fetch(t0 + TT);
        __syncthreads();

        constexpr int G = LN < 4 ? 4 : LN;     // tokens between two reductions
#pragma unroll 1
        for (int g = 0; g < TT; g += G) {
            float y[G];
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const float2 d = sm.d[buf][g + i][wc];
                const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(&sm.b[buf][g + i][q]);
                const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(&sm.c[buf][g + i][q]);
                const f2 dd = pack2(d.x, d.x), du = pack2(d.y, d.y);
                h01 = fma2(exp2_pair(mul2(dd, A01)), h01, mul2(du, b.x));
                h23 = fma2(exp2_pair(mul2(dd, A23)), h23, mul2(du, b.y));
                y[i] = sum2(fma2(c.x, h01, mul2(c.y, h23)));
            }
            reduce_scatter<LN, 1, G>(y);
#pragma unroll
            for (int i = 0; i < G / LN; ++i) sm.y[g + q * (G / LN) + i][wc] = y[i];
        }
        if (a.chunks && t0 + TT <= sb && live) {
            const int64_t row = row0 + tile;
            if (row < a.chunk_capacity) {
                float4 h;
                unpack2(h01, h.x, h.y);
                unpack2(h23, h.z, h.w);
                store_states(a.chunks + (row * P.D + ch) * P.S, h, n0, P.S, P.svec);
            }
        }
        __syncthreads();
        if (t0 + srow < sb && have > 0) {
            float o[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float v = fmaf(skip[i], cu_u.get(i), sm.y[srow][sc + i]);
                if (P.z.p) {
                    const float z = cu_z.get(i);
                    v *= z * sigmoid_fast(z);
                }
                o[i] = v;
            }
            store_row<OUT, E>((OUT *)a.out + (t0 + srow) * P.D + ch0 + sc, o, have, a.ovec);
        }
    }
    if (a.fin && live) {
        float4 h;
        unpack2(h01, h.x, h.y);
        unpack2(h23, h.z, h.w);
        store_states(a.fin + ((int64_t)n * P.D + ch) * P.S, h, n0, P.S, P.svec);
    }
}

template <typename IN, typename OUT, int LN>
cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    using L = Layout<LN>;
    const int64_t blocks = (int64_t)a.P.N * ((a.P.D + L::CB - 1) / L::CB);
    const int smem = (int)sizeof(typename L::Smem);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kda_ssm_scan_kernel<IN, OUT, LN>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    kda_ssm_scan_kernel<IN, OUT, LN><<<(unsigned)blocks, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename IN, typename OUT>
cudaError_t by_states(const ScanArgs &a, cudaStream_t s) {
    if (a.P.S <= 8) return launch<IN, OUT, 2>(a, s);
    if (a.P.S <= 16) return launch<IN, OUT, 4>(a, s);
    if (a.P.S <= 32) return launch<IN, OUT, 8>(a, s);
    return launch<IN, OUT, 16>(a, s);
}

}  // namespace

cudaError_t kda_launch_ssm_scan(const SsmProblem &P, const float *init, void *out, float *final_state,
                                float *chunk_states, int64_t chunk_capacity, cudaStream_t stream) {
    ScanArgs a{P, init, out, final_state, chunk_states, chunk_capacity, false};
    const int es = P.out_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    a.ovec = ((uintptr_t)out & 15u) == 0 && (int64_t)P.D * es % 16 == 0;
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return by_states<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (ib) return by_states<__nv_bfloat16, float>(a, stream);
    if (ob) return by_states<float, __nv_bfloat16>(a, stream);
    return by_states<float, float>(a, stream);
}
