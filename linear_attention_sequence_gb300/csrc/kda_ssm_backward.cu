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
// tokens).  A lane holds four states of two neighbouring channels, as in the scan.
// Chunks are taken from the last to the first, each in two halves of 16 tokens and
// four quarters of 8: the states at the quarters' starts are run up to first, then a
// quarter's states are formed again, kept in registers, and its gradients follow
// back through it.  A decay is formed 2.75 times; no state goes through memory.
// Sums over a channel's states are exchanges between its LN lanes.  Sums over
// channels (dB, dC) are exchanges between the lanes of a warp, then shared
// memory between the warps, then a workspace row per block that a second kernel
// adds up in order.
//
// Four warps do that; four more stage the activations (step size, gate, values of the
// codes) a chunk ahead and finish the gradients of the half before, as in the
// scan.  The two kinds need very different numbers of registers: 160 and 96 of the
// 128 a thread that two blocks an SM allow.
//
// Sequences are cut into parts as in the scan: a first kernel runs the adjoint
// alone back through every part but the first from zero, g_in' = g_part +
// exp(A sum Delta) g_in carries it on, and the gradients proper run every part from its
// own g_in.
//
// 8192 tokens of 4096 channels with 16 states, bf16, u and z in 8 bits: 770 us, of which
// 121 for the adjoint alone and 14 for the sums across blocks.  Bound by instruction
// issue: about 120 instructions per 128 state entries, 0.58 a cycle.

#include <type_traits>

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kScanners = 128, kStagers = 128;
constexpr int kThreads = kScanners + kStagers;
constexpr int TT = kSsmTile;
constexpr int HT = TT / 2;       // tokens of a half
constexpr int QT = 8;            // tokens of a quarter
constexpr float kLn2 = 0.6931471805599453f;

__device__ unsigned g_ssm_status = 0;

struct BackArgs {
    SsmProblem P;
    const float *init, *chunks, *d_final;
    int64_t chunk_capacity;
    void *du, *ddt, *dz;
    float *dA, *dskip, *dbias;   // per part: [D, S], [D], [D] (the results themselves where there is one part)
    float *d_init;
    float *share;                // [blocks across D][T][2 SP]
    bool ovec, obf;
    Parts parts;
    float *carry, *sums;         // as in the scan, from part to the one before it
};

template <typename IN, int LN>
struct Layout {
    static constexpr int CW = 64 / LN, CB = 4 * CW, SP = 4 * LN;
    static constexpr int TR = 8, E = CB / TR;            // threads that stage a row, channels of each
    static constexpr bool kBf = sizeof(IN) == 2;
    static constexpr int YS = CB == 128 ? 144 : CB == 64 ? 72 : CB == 32 ? 36 : 20;
    struct Smem {
        float2 d[2][TT][CB];                 // Delta, Delta u (column())
        float dyp[2][TT][CB];                // (swz())
        uint4 bc[2][TT][LN][kBf ? 1 : 2];
        float h[2][CB][SP];                  // state at the chunk's start
        float out[2][3][HT][YS];             // p, r, y of a half
        float share[2][4][HT][2 * SP];       // the warps' shares of dC, dB
        float bias[CB], skip[CB];            // (swz())
        float sums[2][HT][CB];               // of dyp u and of ddt, by row of staging threads (swz())
    };
    static constexpr int kBlocks = sizeof(Smem) <= 113 * 1024 ? 2 : 1;   // an SM
    static __device__ __forceinline__ int column(int c) { return c ^ (((c >> 4) & 7) << 1); }
    static __device__ __forceinline__ int ycol(int c) { return c + 4 * (c >> 5); }
    // The same for rows of floats that staging threads read and write four at a time.
    static __device__ __forceinline__ int swz(int c) { return c ^ (((c >> 5) & 3) << 2); }
};

// E consecutive floats, from channel c on, of a row laid out by swz().
template <typename L, int E>
__device__ __forceinline__ void read_swz(const float *row, int c, float (&v)[E]) {
    if constexpr (E == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(row + L::swz(c));
        v[0] = x.x; v[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(row + L::swz(c + i));
            v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
        }
    }
}
template <typename L, int E>
__device__ __forceinline__ void write_swz(float *row, int c, const float (&v)[E]) {
    if constexpr (E == 2) {
        *reinterpret_cast<float2 *>(row + L::swz(c)) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4)
            *reinterpret_cast<float4 *>(row + L::swz(c + i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

// E gradients.  WIDE: their type is known (BF) and they may be written at once; a
// branch around each store would keep the steps of several channels from overlapping.
template <bool WIDE, bool BF, int E>
__device__ __forceinline__ void store_grad(void *p, int64_t at, const float (&v)[E], int have, bool vec, bool bf) {
    if constexpr (WIDE) {
        if constexpr (BF) store_row<__nv_bfloat16, E, true>((__nv_bfloat16 *)p + at, v, have, true);
        else store_row<float, E, true>((float *)p + at, v, have, true);
    } else {
        if (bf) store_row<__nv_bfloat16, E>((__nv_bfloat16 *)p + at, v, have, vec);
        else store_row<float, E>((float *)p + at, v, have, vec);
    }
}

// E values of a row of codes or plain values.
template <typename X, int E>
struct Vals {
    Raw<X, E> r;
    float s[E > kPackGroup ? E / kPackGroup : 1];
    // The row of token t from channel c on, or zeros if !ok.  FAST: all channels or
    // none exist, at an address that allows wide accesses.
    template <bool FAST>
    __device__ __forceinline__ void load(const Rows &x, int t, int c, int have, bool ok) {
        const X *p = (const X *)x.p + (int64_t)t * x.stride + c;
        if constexpr (FAST) {
            r.load_if(p, ok);
        } else {
            if (ok) r.load(p, have, x.vec);
            else r.clear();
        }
        if constexpr (sizeof(X) == 1) {
            uint32_t w = 0;
            ahead4(w, x.scales + (int64_t)t * x.ngroups + c / kPackGroup, ok);
            s[0] = __uint_as_float(w);
        }
    }
    __device__ __forceinline__ void clear() {
        r.clear();
        s[0] = 0.f;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(X) == 1) return r.get(i) * s[0];
        return r.get(i);
    }
};

// Four states of B and C of each of N tokens that a thread stages (one of ROWS in
// all); tokens past the end, and states past S, are 0.
template <typename IN, int LN, int ROWS>
struct RawBC {
    static constexpr int N = (ROWS * LN + kStagers - 1) / kStagers;
    Raw<IN, 4> b[N], c[N];
    template <bool BOTH, bool FAST>
    __device__ __forceinline__ void load(const SsmProblem &P, int t0, int end, int tid, bool live) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = tid + k * kStagers, n0 = 4 * (i % LN);
            const int t = t0 + i / LN;
            const IN *pb = (const IN *)P.B.p + (int64_t)t * P.B.stride + n0, *pc = (const IN *)P.C.p + (int64_t)t * P.C.stride + n0;
            const bool ok = i < ROWS * LN && live && t < end && n0 < P.S;
            if constexpr (FAST) {
                if (BOTH) b[k].load_if(pb, ok);
                c[k].load_if(pc, ok);
            } else {
                if (BOTH) b[k].clear();
                c[k].clear();
                if (ok) {
                    if (BOTH) b[k].load(pb, P.S - n0, P.B.vec);
                    c[k].load(pc, P.S - n0, P.C.vec);
                }
            }
        }
    }
    // `to`: [ROWS][LN][1 or 2] pieces
    template <bool BOTH>
    __device__ __forceinline__ void put(uint4 *to, int tid) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = tid + k * kStagers;
            if (i < ROWS * LN) {
                if constexpr (sizeof(IN) == 2) {
                    to[i] = make_uint4(BOTH ? b[k].w[0] : 0u, BOTH ? b[k].w[1] : 0u, c[k].w[0], c[k].w[1]);
                } else {
                    if (BOTH) to[2 * i] = make_uint4(b[k].w[0], b[k].w[1], b[k].w[2], b[k].w[3]);
                    to[2 * i + 1] = make_uint4(c[k].w[0], c[k].w[1], c[k].w[2], c[k].w[3]);
                }
            }
        }
    }
};

// Whether a thread's E channels, and four states, all exist or none do, and may be
// read at once.
template <int E>
__device__ __forceinline__ bool all_wide(const SsmProblem &P, bool u) {
    return P.D % E == 0 && P.S % 4 == 0 && P.dt.vec && P.dy.vec && P.B.vec && P.C.vec && (!u || P.u.vec) && (!P.z.p || P.z.vec);
}

// Sixteen bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// E consecutive floats of shared memory (aligned to 16 bytes, or 8 for E = 2).
template <int E>
__device__ __forceinline__ void read_row(const float *p, float (&v)[E]) {
    if constexpr (E == 2) {
        const float2 x = *reinterpret_cast<const float2 *>(p);
        v[0] = x.x; v[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p + i);
            v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
        }
    }
}

template <typename IN>
__device__ __forceinline__ void read_b(const uint4 *p, f2 &b01, f2 &b23) {
    if constexpr (sizeof(IN) == 2) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        b01 = pack2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
        b23 = pack2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    } else {
        b01 = pack2(__uint_as_float(p[0].x), __uint_as_float(p[0].y));
        b23 = pack2(__uint_as_float(p[0].z), __uint_as_float(p[0].w));
    }
}
template <typename IN>
__device__ __forceinline__ void read_c(const uint4 *p, f2 &c01, f2 &c23) {
    if constexpr (sizeof(IN) == 2) {
        read_b<IN>(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint2 *>(p) + 1), c01, c23);
    } else {
        read_b<IN>(p + 1, c01, c23);
    }
}

// What a part of a sequence is to a block.
struct Place {
    int n, part, count;
    int sa, pa, pb;                          // (token numbers are below 2^31)
    int row;                                 // of the carry: between this part and the next
};
__device__ __forceinline__ bool place_of(const BackArgs &a, const Part &p, Place &w) {
    w.n = p.n;
    w.part = p.k;
    w.count = p.count;
    w.row = p.row;
    if (p.n < 0) return false;
    int64_t sa, sb;
    seq_bounds(a.P.cu, p.n, a.P.T, a.P.seq_len, sa, sb);
    const int64_t pa = sa + p.k * a.parts.len;
    w.sa = (int)sa;
    w.pa = (int)pa;
    w.pb = (int)(p.k == p.count - 1 ? sb : pa + a.parts.len);
    // as in the scan: overlapping sequences could need more rows than there are
    return p.count == 1 || p.row + (p.k < p.count - 1) <= a.parts.rows;
}

// The staging warps.
template <typename X, typename IN, int LN, bool FAST, bool BF>
struct Stager {
    using L = Layout<IN, LN>;
    static constexpr int E = L::E, CB = L::CB, SP = L::SP;
    const BackArgs &a;
    typename L::Smem &sm;
    const int pa, pb;
    int tid, srow, sc, ch0, cb, have;
    int64_t row0;                             // of the chunk states: the part's first chunk's start, in sequences' numbering
    Vals<X, E> u, z;                          // of the half to stage next
    Vals<IN, E> dt, dy;
    Vals<X, E> fu, fz;                        // of the half to finish next
    Vals<IN, E> fdt, fdy;
    RawBC<IN, LN, HT> bc;
    int first;                                // the sequence, where the part is its first; else -1

    __device__ __forceinline__ Stager(const BackArgs &a_, typename L::Smem &sm_, const Place &w, int ch0_, int cb_)
        : a(a_), sm(sm_), pa(w.pa), pb(w.pb), ch0(ch0_), cb(cb_) {
        const SsmProblem &P = a.P;
        tid = threadIdx.x - kScanners;
        srow = tid / L::TR;
        sc = tid % L::TR * E;
        have = P.D - (ch0 + sc);
        z.clear();                            // (where there is no gate, its values are formed and left out)
        fz.clear();
        // chunk k of the part starts with row row0 + k; the sequence's first chunk with its initial state
        row0 = ckpt_first_row(P.cu, w.n, P.T, P.seq_len, TT) + (w.pa - w.sa) / TT - 1;
        first = w.pa == w.sa ? w.n : -1;
#pragma unroll
        for (int i = 0; i < E; ++i) sm.sums[0][srow][L::swz(sc + i)] = sm.sums[1][srow][L::swz(sc + i)] = 0.f;
        for (int c = tid; c < CB; c += kStagers) {
            sm.bias[L::swz(c)] = P.dt_bias && ch0 + c < P.D ? P.dt_bias[ch0 + c] : 0.f;
            sm.skip[L::swz(c)] = P.skip && ch0 + c < P.D ? P.skip[ch0 + c] : 0.f;
        }
        asm volatile("bar.sync 1, %0;" ::"r"(kStagers) : "memory");
    }
    __device__ __forceinline__ void fetch(int j, Vals<X, E> &vu, Vals<X, E> &vz, Vals<IN, E> &vdt, Vals<IN, E> &vdy) {
        const SsmProblem &P = a.P;
        const int t = pa + j * HT + srow, c = ch0 + sc;
        const bool ok = j >= 0 && t < pb && have > 0;
        vu.template load<FAST>(P.u, t, c, have, ok);
        if (P.z.p) vz.template load<FAST>(P.z, t, c, have, ok);
        vdt.template load<FAST>(P.dt, t, c, have, ok);
        vdy.template load<FAST>(P.dy, t, c, have, ok);
    }
    __device__ __forceinline__ void fetch_next(int j) {
        fetch(j, u, z, dt, dy);
        bc.template load<true, FAST>(a.P, pa + j * HT, pb, tid, j >= 0);
    }
    // Half j into shared memory; with the second half of a chunk, its start state.
    __device__ __forceinline__ void stage(int j) {
        const SsmProblem &P = a.P;
        const int buf = (j >> 1) & 1, row = (j & 1) * HT + srow;
        const int t0 = pa + j * HT;
        if (j & 1) {
            const int64_t row = row0 + (j >> 1);
            const float *from = nullptr;
            if (j == 1 && first >= 0) {
                if (a.init) from = a.init + (int64_t)first * P.D * P.S;
            } else if (row < a.chunk_capacity) {
                from = a.chunks + row * P.D * P.S;
            } else if (tid == 0) {
                atomicOr(&g_ssm_status, kBwdMissingState);
            }
            for (int i = tid; i < CB * LN; i += kStagers) {
                const int c = i / LN, n0 = 4 * (i % LN);
                float4 *to = reinterpret_cast<float4 *>(&sm.h[buf][c][n0]);
                if (from && ch0 + c < P.D && P.svec && n0 < P.S)
                    copy16(to, from + (int64_t)(ch0 + c) * P.S + n0);   // waited for before the barrier
                else if (from && ch0 + c < P.D)
                    *to = load_states(from + (int64_t)(ch0 + c) * P.S, n0, P.S, P.svec);
                else
                    *to = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        bc.template put<true>(sm.bc[buf][(j & 1) * HT][0], tid);
        const bool in = t0 + srow < pb && have > 0;
        constexpr int VE = E < 4 ? E : 4;      // at a time
#pragma unroll
        for (int i0 = 0; i0 < E; i0 += VE) {
            float dl[VE], dyp[VE];
            read_swz<L, VE>(sm.bias, sc + i0, dl);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                dl[i] += dt.get(i0 + i);
                dyp[i] = dy.get(i0 + i);
            }
            float sp[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                sp[i] = dl[i];
                const float g = z.get(i0 + i), f = g * sigmoid_fast(g);
                dyp[i] *= P.z.p ? f : 1.f;
            }
            softplus_all(sp);
#pragma unroll
            for (int i = 0; i < VE; ++i) dl[i] = P.softplus ? sp[i] : dl[i];
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
                float4 v;
                v.x = in ? dl[i] : 0.f;
                v.z = in ? dl[i + 1] : 0.f;
                v.y = v.x * u.get(i0 + i);
                v.w = v.z * u.get(i0 + i + 1);
                *reinterpret_cast<float4 *>(&sm.d[buf][row][L::column(sc + i0 + i)]) = v;
            }
            write_swz<L, VE>(sm.dyp[buf][row], sc + i0, dyp);
        }
    }
    // The gradients of half j.
    __device__ __forceinline__ void finish(int j) {
        const SsmProblem &P = a.P;
        const int buf = (j >> 1) & 1, row = (j & 1) * HT + srow, ob = j & 1;
        const int t0 = pa + j * HT;
        for (int i = tid; i < HT * 2 * SP / 4; i += kStagers) {
            const int t = i / (2 * SP / 4), k = i % (2 * SP / 4);
            if (t0 + t < pb) {
                float4 s = *reinterpret_cast<const float4 *>(&sm.share[ob][0][t][4 * k]);
#pragma unroll
                for (int v = 1; v < 4; ++v) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sm.share[ob][v][t][4 * k]);
                    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
                }
                *reinterpret_cast<float4 *>(a.share + ((int64_t)cb * P.T + t0 + t) * (2 * SP) + 4 * k) = s;
            }
        }
        if (t0 + srow >= pb || have <= 0) return;
        // a few channels at a time, to keep few values alive; Delta and dyp were written by this thread
        constexpr int VE = E < 4 ? E : 4;
        const int64_t row_at = (int64_t)(t0 + srow) * P.D + ch0 + sc;
        if (P.z.p) {
#pragma unroll
            for (int k = 0; k < E; k += VE) {
                float o[VE], v[VE];
                read_swz<L, VE>(sm.skip, sc + k, v);
                read_row<VE>(&sm.out[ob][2][srow][L::ycol(sc + k)], o);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float g = fz.get(k + i), s = sigmoid_fast(g);
                    o[i] = fdy.get(k + i) * fmaf(v[i], fu.get(k + i), o[i]) * fmaf(g * s, 1.f - s, s);
                }
                store_grad<FAST, BF, VE>(a.dz, row_at + k, o, have - k, a.ovec, a.obf);
            }
        }
#pragma unroll
        for (int k = 0; k < E; k += VE) {
            const int c = sc + k, yc = L::ycol(c);
            float o[VE], x[VE], dyp[VE], v[VE];
            read_swz<L, VE>(sm.skip, c, v);
            read_row<VE>(&sm.out[ob][0][srow][yc], o);
            read_row<VE>(&sm.out[ob][1][srow][yc], x);
            read_swz<L, VE>(sm.dyp[buf][row], c, dyp);
#pragma unroll
            for (int i = 0; i < VE; i += 2) {
                const float4 d = *reinterpret_cast<const float4 *>(&sm.d[buf][row][L::column(c + i)]);
                x[i] = fmaf(fu.get(k + i), o[i], x[i] * kLn2);
                x[i + 1] = fmaf(fu.get(k + i + 1), o[i + 1], x[i + 1] * kLn2);
                o[i] = fmaf(d.x, o[i], v[i] * dyp[i]);
                o[i + 1] = fmaf(d.z, o[i + 1], v[i + 1] * dyp[i + 1]);
            }
            store_grad<FAST, BF, VE>(a.du, row_at + k, o, have - k, a.ovec, a.obf);
            read_swz<L, VE>(sm.bias, c, v);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float s = sigmoid_fast(fdt.get(k + i) + v[i]);
                x[i] *= P.softplus ? s : 1.f;
            }
            store_grad<FAST, BF, VE>(a.ddt, row_at + k, x, have - k, a.ovec, a.obf);
            read_swz<L, VE>(sm.sums[0][srow], c, v);
            read_swz<L, VE>(sm.sums[1][srow], c, o);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                v[i] = fmaf(dyp[i], fu.get(k + i), v[i]);
                o[i] += x[i];
            }
            write_swz<L, VE>(sm.sums[0][srow], c, v);
            write_swz<L, VE>(sm.sums[1][srow], c, o);
        }
    }
};

// What the staging warps do for a part.
template <typename X, typename IN, int LN, bool FAST, bool BF>
__device__ __forceinline__ void stage_part(const BackArgs &a, typename Layout<IN, LN>::Smem &sm, const Place &w, int ch0,
                                           int cb, int tiles) {
    // While the other warps work through half j, these stage half j - 2 (the
    // whole chunk before j's is in place when j is its second half) and finish half
    // j + 1.
    Stager<X, IN, LN, FAST, BF> st(a, sm, w, ch0, cb);
    const int last = 2 * tiles - 1;
    if (tiles > 0) {
        st.fetch_next(last);
        st.stage(last);
        st.fetch_next(last - 1);
        st.stage(last - 1);
        st.fetch_next(last - 2);
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();
    
    for (int j = last; j >= 0; --j) {
        if (j < last) st.finish(j + 1);
        if (j >= 2) {
            st.stage(j - 2);
            st.fetch_next(j - 3);
        }
        st.fetch(j, st.fu, st.fz, st.fdt, st.fdy);
        // a chunk's start state is needed two steps after it was asked for
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
    }
    if (tiles > 0) st.finish(0);
}

// X: type of u and z (int8 codes or IN); IN: type of dt, B, C and d_out.
template <typename X, typename IN, int LN>
__global__ void __launch_bounds__(kThreads, (Layout<IN, LN>::kBlocks))
kda_ssm_scan_backward_kernel(const __grid_constant__ BackArgs a) {
    using L = Layout<IN, LN>;
    constexpr int CW = L::CW, CB = L::CB, SP = L::SP;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename L::Smem &sm = *reinterpret_cast<typename L::Smem *>(smem_raw);
    __shared__ Part s_part;

    let_next();
    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB, cb = (int)(blockIdx.x % ncb), slot = (int)(blockIdx.x / ncb);
    const int ch0 = cb * CB;
    Place w;
    const bool some = place_of(a, longest_part(a.parts, P.cu, P.N, P.T, P.seq_len, slot, &s_part), w);
    // the shares of dA, dD and ddt_bias: by part, in the sequences' order where it keeps them
    const int64_t at = some && w.row + w.n < a.parts.most ? w.row + w.n : slot;
    if (!some) {
        // a part that the batch does not have: its shares are 0
        for (int64_t i = threadIdx.x; i < (int64_t)min(CB, P.D - ch0) * P.S; i += kThreads)
            a.dA[(at * P.D + ch0) * P.S + i] = 0.f;
        for (int i = threadIdx.x; i < min(CB, P.D - ch0); i += kThreads) {
            if (a.dskip) a.dskip[at * P.D + ch0 + i] = 0.f;
            if (a.dbias) a.dbias[at * P.D + ch0 + i] = 0.f;
        }
        return;
    }
    const int tiles = (int)((w.pb - w.pa + TT - 1) / TT);

    if (threadIdx.x >= kScanners) {
        if constexpr (L::kBlocks == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (!all_wide<L::E>(P, true) || !a.ovec) stage_part<X, IN, LN, false, false>(a, sm, w, ch0, cb, tiles);
        else if (a.obf) stage_part<X, IN, LN, true, true>(a, sm, w, ch0, cb, tiles);
        else stage_part<X, IN, LN, true, false>(a, sm, w, ch0, cb, tiles);
        // dD and ddt_bias: over the rows of threads
        asm volatile("bar.sync 1, %0;" ::"r"(kStagers) : "memory");
        for (int c = threadIdx.x - kScanners; c < CB; c += kStagers) {
            if (ch0 + c < P.D) {
                float x = 0.f, y = 0.f;
                for (int t = 0; t < HT; ++t) {
                    x += sm.sums[0][t][L::swz(c)];
                    y += sm.sums[1][t][L::swz(c)];
                }
                if (a.dskip) a.dskip[at * P.D + ch0 + c] = x;
                if (a.dbias) a.dbias[at * P.D + ch0 + c] = y;
            }
        }
        return;
    }

    if constexpr (L::kBlocks == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    wait_before();                           // the carry; the staging warps need nothing of it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wc = warp * CW + lane / LN * 2, ch = ch0 + wc;
    const int q = lane % LN, n0 = 4 * q;
    f2 A[2][2], g[2][2], dA[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (ch + c < P.D) {
            x = load_states(P.A + (int64_t)(ch + c) * P.S, n0, P.S, P.svec);
            const float *from = w.part < w.count - 1 ? a.carry + (int64_t)w.row * P.D * P.S
                                : a.d_final ? a.d_final + (int64_t)w.n * P.D * P.S : nullptr;
            if (from) y = load_states(from + (int64_t)(ch + c) * P.S, n0, P.S, P.svec);
        }
        A[c][0] = pack2(x.x * kLog2e, x.y * kLog2e);
        A[c][1] = pack2(x.z * kLog2e, x.w * kLog2e);
        g[c][0] = pack2(y.x, y.y);
        g[c][1] = pack2(y.z, y.w);
        dA[c][0] = dA[c][1] = 0;
    }
    const int col = L::column(wc), yc = L::ycol(wc);
    f2 eighth[2][2];                         // the states at the chunk's second quarter
    __syncthreads();
#pragma unroll 1
    for (int j = 2 * tiles - 1; j >= 0; --j) {
        const int buf = (j >> 1) & 1, ob = j & 1;
        auto forward = [&](int t, f2 (&h)[2][2]) {
            const float4 d = *reinterpret_cast<const float4 *>(&sm.d[buf][t][col]);
            f2 b01, b23;
            read_b<IN>(sm.bc[buf][t][q], b01, b23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float dl = c ? d.z : d.x, x = c ? d.w : d.y;
                const f2 dd = pack2(dl, dl), du = pack2(x, x);
                h[c][0] = fma2(exp2_pair(mul2(dd, A[c][0])), h[c][0], mul2(du, b01));
                h[c][1] = fma2(exp2_pair(mul2(dd, A[c][1])), h[c][1], mul2(du, b23));
            }
        };
        f2 third[2][2], s[2][2];             // the state at the half's second quarter; the quarter's start
        if (j & 1) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(&sm.h[buf][wc + c][n0]);
                s[c][0] = pack2(v.x, v.y);
                s[c][1] = pack2(v.z, v.w);
            }
#pragma unroll 1
            for (int k = 0; k < 3; ++k) {
#pragma unroll
                for (int t = 0; t < QT; ++t) forward(k * QT + t, s);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (k == 0) eighth[c][i] = s[c][i];
                        if (k == 1) third[c][i] = s[c][i];
                    }
            }
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                s[c][0] = eighth[c][0];
                s[c][1] = eighth[c][1];
                const float4 v = *reinterpret_cast<const float4 *>(&sm.h[buf][wc + c][n0]);
                third[c][0] = pack2(v.x, v.y);
                third[c][1] = pack2(v.z, v.w);
            }
        }
#pragma unroll 1
        for (int k = 1; k >= 0; --k) {       // the half's quarters, from the states s and third
            const int tb = (j & 1) * HT + k * QT;
            f2 H[QT + 1][2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) H[0][c][i] = k ? s[c][i] : third[c][i];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 2; ++i) H[t + 1][c][i] = H[t][c][i];
                forward(tb + t, H[t + 1]);
            }
#pragma unroll
            for (int t4 = QT - 4; t4 >= 0; t4 -= 4) {
                float vp[2][4], vr[2][4], vy[2][4];
#pragma unroll
                for (int i = 3; i >= 0; --i) {
                    const int t = t4 + i;
                    const float4 d = *reinterpret_cast<const float4 *>(&sm.d[buf][tb + t][col]);
                    const float2 e = *reinterpret_cast<const float2 *>(&sm.dyp[buf][tb + t][L::swz(wc)]);
                    f2 b01, b23, c01, c23, sC01 = 0, sC23 = 0, sB01 = 0, sB23 = 0;
                    read_b<IN>(sm.bc[buf][tb + t][q], b01, b23);
                    read_c<IN>(sm.bc[buf][tb + t][q], c01, c23);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float dl = c ? d.z : d.x, xu = c ? d.w : d.y, ey = c ? e.y : e.x;
                        const f2 dd = pack2(dl, dl), du = pack2(xu, xu), dyp = pack2(ey, ey);
                        const f2 h0 = H[t + 1][c][0], h1 = H[t + 1][c][1];
                        g[c][0] = fma2(dyp, c01, g[c][0]);
                        g[c][1] = fma2(dyp, c23, g[c][1]);
                        vy[c][i] = sum2(fma2(c01, h0, mul2(c23, h1)));
                        vp[c][i] = sum2(fma2(b01, g[c][0], mul2(b23, g[c][1])));
                        if (c == 0) {
                            sC01 = mul2(dyp, h0);
                            sC23 = mul2(dyp, h1);
                            sB01 = mul2(du, g[c][0]);
                            sB23 = mul2(du, g[c][1]);
                        } else {
                            sC01 = fma2(dyp, h0, sC01);
                            sC23 = fma2(dyp, h1, sC23);
                            sB01 = fma2(du, g[c][0], sB01);
                            sB23 = fma2(du, g[c][1], sB23);
                        }
                        g[c][0] = mul2(g[c][0], exp2_pair(mul2(dd, A[c][0])));
                        g[c][1] = mul2(g[c][1], exp2_pair(mul2(dd, A[c][1])));
                        const f2 x0 = mul2(g[c][0], H[t][c][0]), x1 = mul2(g[c][1], H[t][c][1]);
                        vr[c][i] = sum2(fma2(x0, A[c][0], mul2(x1, A[c][1])));
                        dA[c][0] = fma2(x0, dd, dA[c][0]);
                        dA[c][1] = fma2(x1, dd, dA[c][1]);
                    }
                    // over the channels of the warp
                    float v[8];
                    unpack2(sC01, v[0], v[1]);
                    unpack2(sC23, v[2], v[3]);
                    unpack2(sB01, v[4], v[5]);
                    unpack2(sB23, v[6], v[7]);
                    constexpr int G = 32 / LN, CL = G < 8 ? G : 8;   // groups of lanes; values are spread over CL of them
                    reduce_scatter<CL, LN, 8>(v);
#pragma unroll
                    for (int off = CL; off < G; off *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off * LN);
                    if (lane / LN < CL) {
#pragma unroll
                        for (int m = 0; m < 8 / CL; ++m) {
                            const int vi = (lane / LN) * (8 / CL) + m;
                            sm.share[ob][warp][k * QT + t][(vi >> 2) * SP + n0 + (vi & 3)] = v[m];
                        }
                    }
                }
                // over the states of a channel; lane q ends with the sums of token q (LN = 2: of two)
                constexpr int QL = LN < 4 ? LN : 4;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    reduce_scatter<QL, 1, 4>(vp[c]);
                    reduce_scatter<QL, 1, 4>(vr[c]);
                    reduce_scatter<QL, 1, 4>(vy[c]);
#pragma unroll
                    for (int off = 4; off < LN; off *= 2) {
                        vp[c][0] += __shfl_xor_sync(0xffffffffu, vp[c][0], off);
                        vr[c][0] += __shfl_xor_sync(0xffffffffu, vr[c][0], off);
                        vy[c][0] += __shfl_xor_sync(0xffffffffu, vy[c][0], off);
                    }
                }
                if (q < QL) {
#pragma unroll
                    for (int i = 0; i < 4 / QL; ++i) {
                        const int t = k * QT + t4 + q * (4 / QL) + i;
                        *reinterpret_cast<float2 *>(&sm.out[ob][0][t][yc]) = make_float2(vp[0][i], vp[1][i]);
                        *reinterpret_cast<float2 *>(&sm.out[ob][1][t][yc]) = make_float2(vr[0][i], vr[1][i]);
                        *reinterpret_cast<float2 *>(&sm.out[ob][2][t][yc]) = make_float2(vy[0][i], vy[1][i]);
                    }
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (ch + c >= P.D) break;
        float4 v;
        unpack2(dA[c][0], v.x, v.y);
        unpack2(dA[c][1], v.z, v.w);
        store_states(a.dA + (at * P.D + ch + c) * P.S, v, n0, P.S, P.svec);
        if (a.d_init && w.part == 0) {
            unpack2(g[c][0], v.x, v.y);
            unpack2(g[c][1], v.z, v.w);
            store_states(a.d_init + ((int64_t)w.n * P.D + ch + c) * P.S, v, n0, P.S, P.svec);
        }
    }
}

// The adjoint alone, back through every part but a sequence's first, from 0: what it
// gives the part before, and the sum of Delta.
template <typename X, typename IN, int LN>
__global__ void __launch_bounds__(kThreads, 2)
kda_ssm_adjoint_kernel(const __grid_constant__ BackArgs a) {
    using L = Layout<IN, LN>;
    constexpr int CW = L::CW, CB = L::CB, E = L::E, HTB = kStagers / L::TR;
    static_assert(HTB == HT, "a thread stages one row of a half");
    struct Smem {
        float2 d[2][TT][CB];                 // Delta, dyp
        uint4 bc[2][TT][LN][L::kBf ? 1 : 2];
    };
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw);
    let_next();
    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB, ch0 = (int)(blockIdx.x % ncb) * CB;
    Part p = part_of_row<false>(a.parts, P.cu, P.N, P.T, P.seq_len, (int)(blockIdx.x / ncb));
    ++p.k;                                   // the part behind the row
    ++p.row;
    Place w;
    if (!place_of(a, p, w)) return;
    const int tiles = (int)((w.pb - w.pa + TT - 1) / TT);

    if (threadIdx.x >= kScanners) {
        const int tid = threadIdx.x - kScanners, srow = tid / L::TR, sc = tid % L::TR * E, have = P.D - (ch0 + sc);
        float bias[E];
        Vals<X, E> z[2];
        Vals<IN, E> dt[2], dy[2];
        RawBC<IN, LN, TT> bc;
#pragma unroll
        for (int i = 0; i < E; ++i) bias[i] = P.dt_bias && i < have ? P.dt_bias[ch0 + sc + i] : 0.f;
        auto fetch = [&](int k, auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            bc.template load<false, FAST>(P, w.pa + k * TT, w.pb, tid, k >= 0);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int t = w.pa + k * TT + r * HT + srow;
                const bool ok = k >= 0 && t < w.pb && have > 0;
                if (P.z.p) z[r].template load<FAST>(P.z, t, ch0 + sc, have, ok);
                dt[r].template load<FAST>(P.dt, t, ch0 + sc, have, ok);
                dy[r].template load<FAST>(P.dy, t, ch0 + sc, have, ok);
            }
        };
        auto stage = [&](int k) {
            const int buf = k & 1;
            const int t0 = w.pa + k * TT;
            bc.template put<false>(sm.bc[buf][0][0], tid);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r * HT + srow;
                const bool in = t0 + row < w.pb;
                float dl[E], e[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    dl[i] = dt[r].get(i) + bias[i];
                    e[i] = dy[r].get(i);
                }
                if (P.softplus) softplus_all(dl);
                if (P.z.p) {
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const float x = z[r].get(i);
                        e[i] *= x * sigmoid_fast(x);
                    }
                }
#pragma unroll
                for (int i = 0; i < E; i += 2)
                    *reinterpret_cast<float4 *>(&sm.d[buf][row][L::column(sc + i)]) =
                        make_float4(in ? dl[i] : 0.f, e[i], in ? dl[i + 1] : 0.f, e[i + 1]);
            }
        };
        auto run = [&](auto fast) {
            fetch(tiles - 1, fast);
            stage(tiles - 1);
            fetch(tiles - 2, fast);               // (nothing where there is no such tile)
            __syncthreads();
            for (int k = tiles - 1; k >= 0; --k) {
                if (k > 0) {
                    stage(k - 1);
                    fetch(k - 2, fast);
                }
                __syncthreads();
            }
        };
        if (all_wide<E>(P, false)) run(std::true_type());
        else run(std::false_type());
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wc = warp * CW + lane / LN * 2, ch = ch0 + wc, q = lane % LN, n0 = 4 * q;
    f2 A[2][2], g[2][2];
    float dsum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ch + c < P.D) x = load_states(P.A + (int64_t)(ch + c) * P.S, n0, P.S, P.svec);
        A[c][0] = pack2(x.x * kLog2e, x.y * kLog2e);
        A[c][1] = pack2(x.z * kLog2e, x.w * kLog2e);
        g[c][0] = g[c][1] = 0;
    }
    const int col = L::column(wc);
    __syncthreads();
    for (int k = tiles - 1; k >= 0; --k) {
        const int buf = k & 1;
        float ds[2] = {0.f, 0.f};
#pragma unroll 8
        for (int t = TT - 1; t >= 0; --t) {
            const float4 d = *reinterpret_cast<const float4 *>(&sm.d[buf][t][col]);
            f2 c01, c23;
            read_c<IN>(sm.bc[buf][t][q], c01, c23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float dl = c ? d.z : d.x, e = c ? d.w : d.y;
                const f2 dd = pack2(dl, dl), dyp = pack2(e, e);
                g[c][0] = mul2(fma2(dyp, c01, g[c][0]), exp2_pair(mul2(dd, A[c][0])));
                g[c][1] = mul2(fma2(dyp, c23, g[c][1]), exp2_pair(mul2(dd, A[c][1])));
                ds[c] += dl;
            }
        }
        dsum[0] += ds[0];
        dsum[1] += ds[1];
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (ch + c >= P.D) break;
        float4 v;
        unpack2(g[c][0], v.x, v.y);
        unpack2(g[c][1], v.z, v.w);
        store_states(a.carry + ((int64_t)(w.row - 1) * P.D + ch + c) * P.S, v, n0, P.S, P.svec);
        if (q == 0) a.sums[(int64_t)(w.row - 1) * P.D + ch + c] = dsum[c];
    }
}

// From what the parts give back to what the ones before them start with, in place.
__global__ void __launch_bounds__(256) kda_ssm_carry_back_kernel(const __grid_constant__ BackArgs a) {
    let_next();
    const SsmProblem &P = a.P;
    const int64_t M = (int64_t)P.D * P.S;
    const int per = (int)((M + 255) / 256), i = blockIdx.x / per;
    const Part w = part_of_row<true>(a.parts, P.cu, P.N, P.T, P.seq_len, i);
    const int64_t n = w.n, row = w.row;
    const int K = w.count - 1;
    if (n < 0 || row + K > a.parts.rows) return;
    wait_before();
    const int64_t m = (int64_t)(blockIdx.x - i * per) * 256 + threadIdx.x;
    if (m >= M) return;
    const float A = P.A[m] * kLog2e;
    float c = a.d_final ? a.d_final[n * M + m] : 0.f;
    float *p = a.carry + row * M + m;
    const float *s = a.sums + row * P.D + m / P.S;
    carry_on<true>(p, s, K, M, P.D, A, c);
}

// The sums that cross blocks, each in a fixed order: dB and dC over the blocks
// across the channels (`first` blocks; tokens outside every sequence are left as they
// are), then dA, dD and ddt_bias over the parts.
struct ReduceArgs {
    SsmProblem P;
    const float *share;          // [ncb][T][2 SP]: dC, dB
    int ncb, SP;
    unsigned first;
    int parts;
    const float *from[3];        // [parts][n[k]]
    float *to[3];                // [n[k]], or nullptr
    int64_t n[3];
    void *dB, *dC;
};
template <typename OUT>
__global__ void __launch_bounds__(256) kda_ssm_reduce_kernel(const __grid_constant__ ReduceArgs a) {
    const SsmProblem &P = a.P;
    wait_before();
    if (blockIdx.x < a.first) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const int64_t t = i / (2 * a.SP);
        if (t >= P.T) return;
        const int k = (int)(i - t * (2 * a.SP)), n = k % a.SP;
        if (n >= P.S) return;
        if (P.cu) {
            int m;
            int64_t sa, sb;
            if (!find_seq(P.cu, P.N, P.T, P.seq_len, t, m, sa, sb)) return;
        }
        float v = 0.f;
        const float *p = a.share + i;
        const int64_t step = (int64_t)P.T * 2 * a.SP;
#pragma unroll 8
        for (int c = 0; c < a.ncb; ++c) v += p[c * step];
        st_elem((OUT *)(k < a.SP ? a.dC : a.dB) + t * P.S + n, v);
        return;
    }
    int64_t i = (int64_t)(blockIdx.x - a.first) * 256 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (a.to[k]) {
            if (i < a.n[k]) {
                float v = 0.f;
#pragma unroll 8
                for (int p = 0; p < a.parts; ++p) v += a.from[k][p * a.n[k] + i];
                a.to[k][i] = v;
                return;
            }
            i -= a.n[k];
        }
    }
}

int lanes_of(int S) { return S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16; }
int blocks_across(const SsmProblem &P) {
    const int CB = 256 / lanes_of(P.S);
    return (P.D + CB - 1) / CB;
}
template <int LN>
int blocks_an_sm(bool bf) {
    return bf ? Layout<__nv_bfloat16, LN>::kBlocks : Layout<float, LN>::kBlocks;
}
// Cutting adds the adjoint's pass only, 0.19 of the kernel's own.  8192 tokens, S = 16,
// bf16, u and z in 8 bits, in 1 / 4 / 7 / 14 / 19 / 24 parts: 4096 channels 1768 / 864 /
// 780 / 773 / 768 / 764 us, 8192 channels 1804 / 1627 / 1453 / 1429 / 1473 / 1466.  One
// sequence of 512 tokens and 512 channels, bf16: whole 121 us, parts of four tiles 47, of one
// 29.  A ragged batch's parts cost the same whatever they were cut from, so that every
// sequence longer than a part is cut (3148 tokens in 13 sequences, 1000 channels: 98 us;
// from 1.5 parts' length on 115; from 2 134).
Parts back_parts(const SsmProblem &P, bool ragged) {
    const bool bf = P.in_dtype == KDA_DTYPE_BF16;
    int of = 1;
    switch (lanes_of(P.S)) {
        case 2: of = blocks_an_sm<2>(bf); break;
        case 4: of = blocks_an_sm<4>(bf); break;
        case 8: of = blocks_an_sm<8>(bf); break;
        default: of = blocks_an_sm<16>(bf); break;
    }
    return cut_parts(P, ragged, blocks_across(P), {of == 2 ? 1.45 : 2.0, 0.19, 0.7, 0.02, 1.0, 304});
}

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

template <typename X, typename IN, int LN>
cudaError_t launch(const BackArgs &a, cudaStream_t stream) {
    using L = Layout<IN, LN>;
    const int64_t across = blocks_across(a.P);
    cudaError_t e;
    if (a.parts.rows > 0) {
        const int smem = (int)(sizeof(float2) * 2 * TT * L::CB + sizeof(uint4) * 2 * TT * LN * (L::kBf ? 1 : 2));
        e = cudaFuncSetAttribute(kda_ssm_adjoint_kernel<X, IN, LN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kda_ssm_adjoint_kernel<X, IN, LN><<<(unsigned)(a.parts.rows * across), kThreads, smem, stream>>>(a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        const int64_t n = (int64_t)a.parts.cut * (((int64_t)a.P.D * a.P.S + 255) / 256);
        e = launch_behind(true, kda_ssm_carry_back_kernel, (unsigned)n, 256, 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    const int smem = (int)sizeof(typename L::Smem);
    e = cudaFuncSetAttribute(kda_ssm_scan_backward_kernel<X, IN, LN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_behind(a.parts.rows > 0, kda_ssm_scan_backward_kernel<X, IN, LN>, (unsigned)(a.parts.most * across), kThreads, smem,
                         stream, a);
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

// Places in the workspace, in floats.
struct Space {
    int64_t dA, dskip, dbias, carry, sums, all;
};
// (for a batch with cu_seqlens and one without, whichever takes more)
Space space_of(const SsmProblem &P) {
    const Parts x = back_parts(P, true), y = back_parts(P, false);
    const int64_t rows = x.rows > y.rows ? x.rows : y.rows, most = P.N + rows, row = (int64_t)P.D * P.S;
    Space s;
    s.dA = up4((int64_t)blocks_across(P) * P.T * 8 * lanes_of(P.S));
    s.dskip = s.dA + up4(most * row);
    s.dbias = s.dskip + up4(most * P.D);
    s.carry = s.dbias + up4(most * P.D);
    s.sums = s.carry + up4(rows * row);
    s.all = s.sums + up4(rows * P.D);
    return s;
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
    return space_of(P).all * (int64_t)sizeof(float);
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
    a.parts = back_parts(P, P.cu != nullptr);
    const Space sp = space_of(P);
    const int SP = 4 * lanes_of(P.S), ncb = blocks_across(P);
    const int64_t nA = (int64_t)P.D * P.S;
    const bool direct = a.parts.most == 1;
    a.share = workspace;
    a.dA = direct ? dA : workspace + sp.dA;
    a.dskip = !dskip ? nullptr : direct ? dskip : workspace + sp.dskip;
    a.dbias = !dbias ? nullptr : direct ? dbias : workspace + sp.dbias;
    a.carry = workspace + sp.carry;
    a.sums = workspace + sp.sums;
    cudaError_t e = cudaSuccess;
    if (P.N > 0) {
        const bool bf = P.in_dtype == KDA_DTYPE_BF16;
        if (P.u.scales) e = bf ? by_states<int8_t, __nv_bfloat16>(a, stream) : by_states<int8_t, float>(a, stream);
        else e = bf ? by_states<__nv_bfloat16, __nv_bfloat16>(a, stream) : by_states<float, float>(a, stream);
        if (e != cudaSuccess) return e;
    }
    ReduceArgs r{};
    r.P = P;
    r.share = a.share;
    r.ncb = ncb;
    r.SP = SP;
    r.first = P.N > 0 ? (unsigned)(((int64_t)P.T * 2 * SP + 255) / 256) : 0;
    r.parts = a.parts.most;
    r.dB = dB;
    r.dC = dC;
    int64_t n = 0;
    if (!direct) {
        const float *from[3] = {a.dA, a.dskip, a.dbias};
        float *to[3] = {dA, dskip, dbias};
        for (int k = 0; k < 3; ++k) {
            r.from[k] = from[k];
            r.to[k] = to[k];
            r.n[k] = k ? P.D : nA;
            if (to[k]) n += r.n[k];
        }
    }
    const unsigned blocks = r.first + (unsigned)((n + 255) / 256);
    if (blocks == 0) return cudaSuccess;
    return launch_behind(P.N > 0, a.obf ? kda_ssm_reduce_kernel<__nv_bfloat16> : kda_ssm_reduce_kernel<float>, blocks, 256, 0,
                         stream, r);
}
