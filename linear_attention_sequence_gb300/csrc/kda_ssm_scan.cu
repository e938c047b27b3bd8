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

constexpr int kWarps = 4;                 // warps that scan
constexpr int kScanners = 32 * kWarps;
constexpr int kStagers = 256;             // threads that stage
constexpr int kThreads = kScanners + kStagers;
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
    static constexpr int TR = CB >= 16 ? 8 : 4;   // threads that stage a row
    static constexpr int E = CB / TR;          // its elements that each of them stages
    static constexpr int BI = (TT * LN + kStagers - 1) / kStagers;   // 4-element pieces of B (and C) that a thread stages
    struct Smem {
        float2 d[2][TT][CB];                   // Delta, Delta u; channel pairs permuted (column())
        float4 b[2][TT][LN], c[2][TT][LN];
        float y[2][TT][CB][LN];                // the lanes' shares of C_t h_t
    };
    // Where channel c lies in a row of d: the 16-byte pieces that eight staging threads
    // write at once take different banks, and the channels of a warp stay together.
    static __device__ __forceinline__ int column(int c) { return c ^ (((c >> 4) & 3) << 1); }
};

// The staging warps: load a tile, form Delta and Delta u, and finish the outputs of
// an earlier tile.
template <typename IN, typename OUT, int LN>
struct Stager {
    using L = Layout<LN>;
    static constexpr int E = L::E;
    const ScanArgs &a;
    typename L::Smem &sm;
    int64_t sb;
    int tid, srow, sc, ch0, have;
    float bias[E], skip[E];
    Raw<IN, E> ru, rd, rz;                     // the tile being fetched
    Raw<IN, E> u0, z0, u1, z1;                 // of the tile staged last, and of the one before
    Raw<IN, 4> rb[L::BI], rc[L::BI];

    __device__ __forceinline__ Stager(const ScanArgs &a_, typename L::Smem &sm_, int64_t sb_, int ch0_)
        : a(a_), sm(sm_), sb(sb_), ch0(ch0_) {
        tid = threadIdx.x - kScanners;
        srow = tid / L::TR;
        sc = tid % L::TR * E;
        have = srow < TT ? a.P.D - (ch0 + sc) : 0;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            bias[i] = (a.P.dt_bias && i < have) ? a.P.dt_bias[ch0 + sc + i] : 0.f;
            skip[i] = (a.P.skip && i < have) ? a.P.skip[ch0 + sc + i] : 0.f;
        }
        u0.clear();
        z0.clear();
    }
    __device__ __forceinline__ void fetch(int64_t t0) {
        const SsmProblem &P = a.P;
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
            const int i = tid + k * kStagers;
            const int64_t tb = t0 + i / LN;
            const int nb = 4 * (i % LN);
            rb[k].clear();
            rc[k].clear();
            if (i < TT * LN && tb < sb && nb < P.S) {
                rb[k].load((const IN *)P.B.p + tb * P.B.stride + nb, P.S - nb, P.B.vec);
                rc[k].load((const IN *)P.C.p + tb * P.C.stride + nb, P.S - nb, P.C.vec);
            }
        }
    }
    // The fetched tile, which starts at t0, into buffer `buf`; tokens past the end
    // have Delta = 0.
    __device__ __forceinline__ void stage(int64_t t0, int buf) {
        const bool in = t0 + srow < sb;
        if (srow < TT) {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            float4 v;
            const float x = rd.get(i) + bias[i], y = rd.get(i + 1) + bias[i + 1];
            v.x = in ? (a.P.softplus ? softplus_fast(x) : x) : 0.f;
            v.z = in ? (a.P.softplus ? softplus_fast(y) : y) : 0.f;
            v.y = v.x * ru.get(i);
            v.w = v.z * ru.get(i + 1);
            *reinterpret_cast<float4 *>(&sm.d[buf][srow][L::column(sc + i)]) = v;
        }
        }
#pragma unroll
        for (int k = 0; k < L::BI; ++k) {
            const int i = tid + k * kStagers;
            if (i < TT * LN) {
                sm.b[buf][i / LN][i % LN] = make_float4(rb[k].get(0), rb[k].get(1), rb[k].get(2), rb[k].get(3));
                sm.c[buf][i / LN][i % LN] = make_float4(rc[k].get(0), rc[k].get(1), rc[k].get(2), rc[k].get(3));
            }
        }
        u1 = u0;
        z1 = z0;
        u0 = ru;
        z0 = rz;
    }
    // The outputs of the tile that starts at t0.
    __device__ __forceinline__ void finish(int64_t t0, int buf, const Raw<IN, E> &u, const Raw<IN, E> &z) {
        if (t0 + srow >= sb || have <= 0) return;
        float o[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float *p = sm.y[buf][srow][sc + i];
            float v = 0.f;
            if constexpr (LN == 2) {
                const float2 y = *reinterpret_cast<const float2 *>(p);
                v = y.x + y.y;
            } else {
#pragma unroll
                for (int k = 0; k < LN; k += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(p + k);
                    v += (y.x + y.y) + (y.z + y.w);
                }
            }
            v = fmaf(skip[i], u.get(i), v);
            if (a.P.z.p) {
                const float g = z.get(i);
                v *= g * sigmoid_fast(g);
            }
            o[i] = v;
        }
        store_row<OUT, E>((OUT *)a.out + (t0 + srow) * a.P.D + ch0 + sc, o, have, a.ovec);
    }
};

template <typename IN, typename OUT, int LN>
__global__ void __launch_bounds__(kThreads)
kda_ssm_scan_kernel(const ScanArgs a) {
    using L = Layout<LN>;
    constexpr int CW = L::CW, CB = L::CB;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename L::Smem &sm = *reinterpret_cast<typename L::Smem *>(smem_raw);
    __shared__ int s_seq;

    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB;
    const int n = longest_first(P.cu, P.N, P.T, P.seq_len, blockIdx.x / ncb, &s_seq);
    const int ch0 = (blockIdx.x % ncb) * CB;
    int64_t sa, sb;
    seq_bounds(P.cu, n, P.T, P.seq_len, sa, sb);
    const int64_t tiles = (sb - sa + TT - 1) / TT;

    if (threadIdx.x >= kScanners) {
        // Between barriers k and k + 1 the scanning warps run over tile k; these
        // warps stage tile k + 1 and finish tile k - 1.
        Stager<IN, OUT, LN> st(a, sm, sb, ch0);
        if (tiles > 0) {
            st.fetch(sa);
            st.stage(sa, 0);
        }
        if (tiles > 1) st.fetch(sa + TT);
        __syncthreads();
        for (int64_t k = 0; k < tiles; ++k) {
            const int64_t t0 = sa + k * TT;
            if (k + 1 < tiles) {
                st.stage(t0 + TT, (int)(k + 1) & 1);
                if (k + 2 < tiles) st.fetch(t0 + 2 * TT);
            } else {
                st.u1 = st.u0;
                st.z1 = st.z0;
            }
            __syncthreads();
            st.finish(t0, (int)k & 1, st.u1, st.z1);
        }
        return;
    }

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    const int64_t row0 = a.chunks ? ckpt_first_row(P.cu, n, P.T, P.seq_len, TT) : 0;
    const int col = L::column(wc);
    __syncthreads();
    for (int64_t k = 0; k < tiles; ++k) {
        const int buf = (int)k & 1;
        // Groups of G tokens.  While one group's recurrence (a chain of fused
        // multiply-adds) runs, the next group's decays and inputs are formed and the
        // operands of the one behind it are read.
        constexpr int G = 4;
        float *ys = sm.y[buf][0][wc] + q;
        float2 d[G];
        ulonglong2 b[G], c[2][G];
        f2 a01[2][G], a23[2][G], x01[2][G], x23[2][G];
        auto read = [&](int g) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                d[i] = sm.d[buf][g * G + i][col];
                b[i] = *reinterpret_cast<const ulonglong2 *>(&sm.b[buf][g * G + i][q]);
            }
        };
        auto form = [&](int g) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const f2 dd = pack2(d[i].x, d[i].x), du = pack2(d[i].y, d[i].y);
                a01[g & 1][i] = exp2_pair(mul2(dd, A01));
                a23[g & 1][i] = exp2_pair(mul2(dd, A23));
                x01[g & 1][i] = mul2(du, b[i].x);
                x23[g & 1][i] = mul2(du, b[i].y);
                c[g & 1][i] = *reinterpret_cast<const ulonglong2 *>(&sm.c[buf][g * G + i][q]);
            }
        };
        read(0);
        form(0);
        read(1);
#pragma unroll
        for (int g = 0; g < TT / G; ++g) {
            if (g + 1 < TT / G) form(g + 1);
            if (g + 2 < TT / G) read(g + 2);
#pragma unroll
            for (int i = 0; i < G; ++i) {
                h01 = fma2(a01[g & 1][i], h01, x01[g & 1][i]);
                h23 = fma2(a23[g & 1][i], h23, x23[g & 1][i]);
                ys[(g * G + i) * CB * LN] = sum2(fma2(c[g & 1][i].x, h01, mul2(c[g & 1][i].y, h23)));
            }
        }
        if (a.chunks && sa + (k + 1) * TT <= sb && live) {
            const int64_t row = row0 + k;
            if (row < a.chunk_capacity) {
                float4 h;
                unpack2(h01, h.x, h.y);
                unpack2(h23, h.z, h.w);
                store_states(a.chunks + (row * P.D + ch) * P.S, h, n0, P.S, P.svec);
            }
        }
        __syncthreads();
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
