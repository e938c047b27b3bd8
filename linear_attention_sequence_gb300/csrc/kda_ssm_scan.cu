// kda_ssm_scan.cu -- the selective scan over a packed batch.
//
//   Delta = softplus(dt + dt_bias)                       (or dt + dt_bias itself)
//   h_t[d,n] = exp(Delta_t[d] A[d,n]) h_{t-1}[d,n] + Delta_t[d] u_t[d] B_t[n]
//   y_t[d]   = (sum_n C_t[n] h_t[d,n] + D[d] u_t[d]) z_t[d] Sigmoid(z_t[d])
//
// Every state entry is a recurrence of its own.  A lane holds four states of each
// of two neighbouring channels, LN >= S / 4 lanes (2, 4, 8 or 16) hold a channel pair, a
// block of four scanning warps 256 / LN channels.  It walks its part of a sequence
// in tiles of 32 tokens.  Four more warps stage the tiles: they form Delta and Delta u
// in shared memory one tile ahead, and finish the outputs of the tile before
// (the lanes' shares of C_t h_t added up, the skip, the gate), so that the
// scanning warps hold nothing but recurrences.
//
// What bounds it.  A state entry costs one exponential and about six operations,
// its share of B and C read from shared memory, and of Delta.  Shared memory gives
// 128 bytes a cycle an SM whatever lanes share, and a lane that held one
// channel needed 11 bytes an entry (44 cycles for 128 entries a scheduler,
// against 16 of exponentials); two channels a lane and, for bf16, B and C kept as
// bf16 bring that to 5.  8192 tokens of 4096 channels with 16 states, bf16: 277 us (111 of
// them the first of the passes below, 166 the second), 0.6 instructions issued a cycle.
//
// Few channels.  A sequence is cut into parts where its channels alone would
// not fill the GPU: a first kernel runs all parts but the last from a zero state
// (no outputs), a second one carries the states from part to part, h_in' =
// h_part + exp(A sum Delta) h_in, and the scan proper runs every part from its own
// h_in.  Where the final state takes the initial state's place, the second kernel also
// copies the initial states that the third reads (no time that shows: 277 us with one
// buffer and with two).

#include <type_traits>

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kScanners = 128, kStagers = 128;
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
    Parts parts;
    // One row for every part but the last of its sequence; row (number of the part)
    // - (number of its sequence).
    float *carry;      // [D, S]: what the part ends with, then what the next one starts with
    float *sums;       // [D]: sum of Delta over the part
    // Where the final state takes the initial state's place, part 0 of a cut sequence could
    // read after its last part has written: it reads a copy, [D, S] at its row of the carry,
    // that the carry kernel takes.  nullptr: it reads init.
    float *first;
};

template <typename IN, int LN>
struct Layout {
    static constexpr int CW = 64 / LN;         // channels of a warp
    static constexpr int CB = 4 * CW;          // channels of a block
    static constexpr int TR = 8;               // threads that stage a row
    static constexpr int RP = kStagers / TR;   // rows staged at once
    static constexpr int NR = TT / RP;         // times a thread does that in a tile
    static constexpr int E = CB / TR;          // channels of a thread
    static constexpr bool kBf = sizeof(IN) == 2;
    static constexpr int BI = (TT * LN + kStagers - 1) / kStagers;   // four-state pieces of B (and C) a thread stages
    // Row of the lanes' shares.  Its length spreads a half-warp's stores over all
    // banks, and the gap after 32 channels the reads of eight staging threads.
    static constexpr int YS = CB == 128 ? 144 : CB == 64 ? 72 : CB == 32 ? 36 : 18;
    struct Smem {
        float2 d[2][TT][CB];                   // Delta, Delta u (column())
        uint4 bc[2][TT][LN][kBf ? 1 : 2];      // four states of B and C: bf16 both in one piece
        float y[2][TT][LN][YS];                // the lanes' shares of C_t h_t (ycol())
    };
    // Where channel c lies in a row of d: the 16-byte pieces that eight staging threads
    // write at once take different banks; a warp's channels stay together.
    static __device__ __forceinline__ int column(int c) { return c ^ (((c >> 4) & 7) << 1); }
    static __device__ __forceinline__ int ycol(int c) { return c + 4 * (c >> 5); }
};

// The staging warps.  STATES: only what the states need.  FAST: a thread's channels,
// and four states, all exist or none do, and may be read and written at once.
template <typename IN, typename OUT, int LN, bool STATES, bool FAST>
struct Stager {
    using L = Layout<IN, LN>;
    static constexpr int E = L::E, NR = L::NR, RP = L::RP, BI = L::BI;
    const ScanArgs &a;
    typename L::Smem &sm;
    const int64_t pb;
    int tid, srow, sc, have;
    const IN *pu, *pd, *pz, *pB, *pC;          // this thread's place in the tile to fetch
    const IN *fu, *fz;                         // and in the tile to finish
    OUT *po;
    float bias[E], skip[E];
    Raw<IN, E> ru[NR], rd[NR];
    Raw<IN, 4> rb[BI], rc[BI];
    Raw<IN, E> gu[NR], gz[NR];

    __device__ __forceinline__ Stager(const ScanArgs &a_, typename L::Smem &sm_, int64_t pa, int64_t pb_, int ch0)
        : a(a_), sm(sm_), pb(pb_) {
        const SsmProblem &P = a.P;
        tid = threadIdx.x - kScanners;
        srow = tid / L::TR;
        sc = tid % L::TR * E;
        have = P.D - (ch0 + sc);
        const int64_t t = pa + srow;
        pu = fu = (const IN *)P.u.p + t * P.u.stride + ch0 + sc;
        pd = (const IN *)P.dt.p + t * P.dt.stride + ch0 + sc;
        pz = fz = (const IN *)P.z.p + t * P.z.stride + ch0 + sc;
        po = (OUT *)a.out + t * P.D + ch0 + sc;
        pB = (const IN *)P.B.p + (pa + tid / LN) * P.B.stride + 4 * (tid % LN);
        pC = (const IN *)P.C.p + (pa + tid / LN) * P.C.stride + 4 * (tid % LN);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            bias[i] = (P.dt_bias && i < have) ? P.dt_bias[ch0 + sc + i] : 0.f;
            skip[i] = (P.skip && i < have) ? P.skip[ch0 + sc + i] : 0.f;
        }
    }
    static __device__ __forceinline__ void load(Raw<IN, E> &r, const IN *p, int have, bool vec, bool ok) {
        if constexpr (FAST) {
            r.load_if(p, ok);
        } else {
            if (ok) r.load(p, have, vec);
            else r.clear();
        }
    }
    // Loads the next tile, which starts at t0 (nothing if !live).
    __device__ __forceinline__ void fetch(int64_t t0, bool live) {
        const SsmProblem &P = a.P;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const bool ok = live && t0 + srow + r * RP < pb && have > 0;
            load(ru[r], pu + r * RP * P.u.stride, have, P.u.vec, ok);
            load(rd[r], pd + r * RP * P.dt.stride, have, P.dt.vec, ok);
        }
        pu += TT * P.u.stride;
        pd += TT * P.dt.stride;
#pragma unroll
        for (int k = 0; k < BI; ++k) {
            const int i = tid + k * kStagers, nb = 4 * (i % LN);
            const IN *qB = pB + k * (kStagers / LN) * P.B.stride, *qC = pC + k * (kStagers / LN) * P.C.stride;
            const bool ok = live && i < TT * LN && t0 + i / LN < pb && nb < P.S;
            if constexpr (FAST) {
                rb[k].load_if(qB, ok);
                if (!STATES) rc[k].load_if(qC, ok);
            } else {
                rb[k].clear();
                rc[k].clear();
                if (ok) {
                    rb[k].load(qB, P.S - nb, P.B.vec);
                    if (!STATES) rc[k].load(qC, P.S - nb, P.C.vec);
                }
            }
        }
        pB += TT * P.B.stride;
        pC += TT * P.C.stride;
    }
    // The fetched tile, which starts at t0, into buffer `buf`; tokens past the end
    // have Delta = 0, which leaves a state as it is.
    __device__ __forceinline__ void stage(int64_t t0, int buf) {
        // Many step sizes together: their chains of dependent operations overlap.  fp32
        // rows leave registers for one row's (all: 494, a row's: 464 us over 8192 tokens of
        // 4096 channels; bf16: 279 and 285).
        constexpr int RC = L::kBf ? NR : 1;
#pragma unroll
        for (int r0 = 0; r0 < NR; r0 += RC) {
            float dl[RC * E];
#pragma unroll
            for (int k = 0; k < RC * E; ++k) dl[k] = rd[r0 + k / E].get(k % E) + bias[k % E];
            if (a.P.softplus) softplus_all(dl);
#pragma unroll
            for (int r = r0; r < r0 + RC; ++r) {
                const int row = srow + r * RP;
                const bool in = t0 + row < pb;
#pragma unroll
                for (int i = 0; i < E; i += 2) {
                    float4 v;
                    v.x = in ? dl[(r - r0) * E + i] : 0.f;
                    v.z = in ? dl[(r - r0) * E + i + 1] : 0.f;
                    v.y = v.x * ru[r].get(i);
                    v.w = v.z * ru[r].get(i + 1);
                    *reinterpret_cast<float4 *>(&sm.d[buf][row][L::column(sc + i)]) = v;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < BI; ++k) {
            const int i = tid + k * kStagers;
            if (i < TT * LN) {
                uint4 *p = sm.bc[buf][i / LN][i % LN];
                if constexpr (L::kBf) {
                    p[0] = make_uint4(rb[k].w[0], rb[k].w[1], STATES ? 0u : rc[k].w[0], STATES ? 0u : rc[k].w[1]);
                } else {
                    p[0] = make_uint4(rb[k].w[0], rb[k].w[1], rb[k].w[2], rb[k].w[3]);
                    if (!STATES) p[1] = make_uint4(rc[k].w[0], rc[k].w[1], rc[k].w[2], rc[k].w[3]);
                }
            }
        }
    }
    // u and z again, of the tile to finish next, which starts at t0.
    __device__ __forceinline__ void fetch_again(int64_t t0, bool live) {
        const SsmProblem &P = a.P;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const bool ok = live && t0 + srow + r * RP < pb && have > 0;
            load(gu[r], fu + r * RP * P.u.stride, have, P.u.vec, ok);
            if (P.z.p) load(gz[r], fz + r * RP * P.z.stride, have, P.z.vec, ok);
        }
        fu += TT * P.u.stride;
        fz += TT * P.z.stride;
    }
    // The outputs of the tile that starts at t0.
    __device__ __forceinline__ void finish(int64_t t0, int buf) {
        const SsmProblem &P = a.P;
        constexpr int VE = E < 4 ? E : 4;
        float o[NR * E];
#pragma unroll
        for (int k = 0; k < NR * E; k += VE) {
            float s[VE] = {};
#pragma unroll
            for (int q = 0; q < LN; ++q) {
                const float *p = &sm.y[buf][srow + k / E * RP][q][L::ycol(sc + k % E)];
                if constexpr (VE == 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(p);
                    s[0] += y.x; s[1] += y.y; s[2] += y.z; s[3] += y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2 *>(p);
                    s[0] += y.x; s[1] += y.y;
                }
            }
#pragma unroll
            for (int i = 0; i < VE; ++i) o[k + i] = fmaf(skip[(k + i) % E], gu[k / E].get((k + i) % E), s[i]);
        }
        if (P.z.p) {
#pragma unroll
            for (int k = 0; k < NR * E; ++k) {
                const float z = gz[k / E].get(k % E);
                o[k] *= z * sigmoid_fast(z);
            }
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            OUT *p = po + r * RP * (int64_t)P.D;
            float v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] = o[r * E + i];
            if (t0 + srow + r * RP < pb && have > 0) store_row<OUT, E, FAST>(p, v, have, a.ovec);
        }
        po += TT * (int64_t)P.D;
    }
};

template <typename IN, typename OUT, int LN, bool STATES>
__global__ void __launch_bounds__(kThreads, LN == 2 ? 1 : 2)
kda_ssm_scan_kernel(const __grid_constant__ ScanArgs a) {
    using L = Layout<IN, LN>;
    constexpr int CW = L::CW, CB = L::CB;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    typename L::Smem &sm = *reinterpret_cast<typename L::Smem *>(smem_raw);
    __shared__ Part s_part;

    if (STATES) let_next();
    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB;
    const int ch0 = (int)(blockIdx.x % ncb) * CB, slot = (int)(blockIdx.x / ncb);
    const Part w = STATES ? part_of_row<false>(a.parts, P.cu, P.N, P.T, P.seq_len, slot)
                          : longest_part(a.parts, P.cu, P.N, P.T, P.seq_len, slot, &s_part);
    const int n = w.n, part = w.k, count = w.count;
    const int64_t row = w.row;                 // of the carry
    if (n < 0) return;
    int64_t sa, sb;
    seq_bounds(P.cu, n, P.T, P.seq_len, sa, sb);
    const int64_t pa = sa + part * a.parts.len, pb = part == count - 1 ? sb : pa + a.parts.len;
    // Sequences that overlap (a malformed cu_seqlens) could need more rows than
    // there are; their results are unspecified.
    if (count > 1 && row + (part < count - 1) > a.parts.rows) return;
    const int tiles = (int)((pb - pa + TT - 1) / TT);

    if (threadIdx.x >= kScanners) {
        // Between barriers k and k + 1 the scanning warps run over tile k; these
        // warps stage tile k + 1 and finish tile k - 1.
        if (tiles == 0) return;
        auto run = [&](auto fast) {
            Stager<IN, OUT, LN, STATES, decltype(fast)::value> st(a, sm, pa, pb, ch0);
            if (tiles > 0) {
                st.fetch(pa, true);
                st.stage(pa, 0);
                if (tiles > 1) st.fetch(pa + TT, true);
                __syncthreads();
                for (int k = 0; k <= tiles; ++k) {
                    const int64_t t0 = pa + (int64_t)k * TT;
                    if (k + 1 < tiles) {
                        st.stage(t0 + TT, (k + 1) & 1);
                        if (k + 2 < tiles) st.fetch(t0 + 2 * TT, true);
                    }
                    if (!STATES) {
                        if (k > 0) st.finish(t0 - TT, (k - 1) & 1);
                        if (k < tiles) st.fetch_again(t0, true);
                    }
                    if (k < tiles) __syncthreads();
                }
            }
        };
        if (P.D % L::E == 0 && P.S % 4 == 0 && P.u.vec && P.dt.vec && P.B.vec && P.C.vec && (STATES || !P.z.p || P.z.vec) &&
            (STATES || a.ovec))
            run(std::true_type());
        else
            run(std::false_type());
        return;
    }

    if (!STATES) wait_before();                // the carry; the staging warps need nothing of it
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wc = warp * CW + lane / LN * 2;  // the first of this lane's channels within the block
    const int ch = ch0 + wc;
    const int q = lane % LN, n0 = 4 * q;
    f2 A[2][2], h[2][2];                       // channel, pair of states
    float dsum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (ch + c < P.D) {
            x = load_states(P.A + (int64_t)(ch + c) * P.S, n0, P.S, P.svec);
            const float *from = STATES ? nullptr : part > 0 ? a.carry + (row - 1) * P.D * P.S
                                : a.first && count > 1 ? a.first + row * P.D * P.S
                                : a.init ? a.init + (int64_t)n * P.D * P.S : nullptr;
            if (from) y = load_states(from + (int64_t)(ch + c) * P.S, n0, P.S, P.svec);
        }
        A[c][0] = pack2(x.x * kLog2e, x.y * kLog2e);
        A[c][1] = pack2(x.z * kLog2e, x.w * kLog2e);
        h[c][0] = pack2(y.x, y.y);
        h[c][1] = pack2(y.z, y.w);
    }
    auto put = [&](float *p) {                 // the states, of [D, S] at p
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float4 v;
            unpack2(h[c][0], v.x, v.y);
            unpack2(h[c][1], v.z, v.w);
            if (ch + c < P.D) store_states(p + (int64_t)(ch + c) * P.S, v, n0, P.S, P.svec);
        }
    };
    const int64_t row0 = !STATES && a.chunks ? ckpt_first_row(P.cu, n, P.T, P.seq_len, TT) + (pa - sa) / TT : 0;
    const int col = L::column(wc), yc = L::ycol(wc);
    if (tiles > 0) __syncthreads();
    for (int k = 0; k < tiles; ++k) {
        const int buf = k & 1;
        // The operands of one group of tokens are read while the group before is
        // computed.
        constexpr int G = L::kBf ? 4 : 2;      // (fp32 operands take twice the registers)
        float4 d[2][G];
        uint4 bc[2][G][L::kBf ? 1 : 2];
        float ds[2] = {0.f, 0.f};
        auto read = [&](int g, int to) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                d[to][i] = *reinterpret_cast<const float4 *>(&sm.d[buf][g * G + i][col]);
                bc[to][i][0] = sm.bc[buf][g * G + i][q][0];
                if constexpr (!L::kBf && !STATES) bc[to][i][1] = sm.bc[buf][g * G + i][q][1];
            }
        };
        auto group = [&](int g, int from) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                f2 b01, b23, c01 = 0, c23 = 0;
                const uint4 w = bc[from][i][0];
                if constexpr (L::kBf) {
                    b01 = pack2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u));
                    b23 = pack2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
                    if constexpr (!STATES) {
                        c01 = pack2(__uint_as_float(w.z << 16), __uint_as_float(w.z & 0xffff0000u));
                        c23 = pack2(__uint_as_float(w.w << 16), __uint_as_float(w.w & 0xffff0000u));
                    }
                } else {
                    b01 = pack2(__uint_as_float(w.x), __uint_as_float(w.y));
                    b23 = pack2(__uint_as_float(w.z), __uint_as_float(w.w));
                    if constexpr (!STATES) {
                        const uint4 v = bc[from][i][1];
                        c01 = pack2(__uint_as_float(v.x), __uint_as_float(v.y));
                        c23 = pack2(__uint_as_float(v.z), __uint_as_float(v.w));
                    }
                }
                float2 y;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float dl = c ? d[from][i].z : d[from][i].x, xu = c ? d[from][i].w : d[from][i].y;
                    const f2 dd = pack2(dl, dl), du = pack2(xu, xu);
                    h[c][0] = fma2(exp2_pair(mul2(dd, A[c][0])), h[c][0], mul2(du, b01));
                    h[c][1] = fma2(exp2_pair(mul2(dd, A[c][1])), h[c][1], mul2(du, b23));
                    if constexpr (STATES) ds[c] += dl;
                    else (c ? y.y : y.x) = sum2(fma2(c01, h[c][0], mul2(c23, h[c][1])));
                }
                if constexpr (!STATES) *reinterpret_cast<float2 *>(&sm.y[buf][g * G + i][q][yc]) = y;
            }
        };
        read(0, 0);
#pragma unroll 1
        for (int g = 0; g < TT / G; g += 2) {
            read(g + 1, 1);
            group(g, 0);
            if (g + 2 < TT / G) read(g + 2, 0);
            group(g + 1, 1);
        }
        if (STATES) {
            dsum[0] += ds[0];
            dsum[1] += ds[1];
        } else if (a.chunks && pa + (int64_t)(k + 1) * TT <= sb) {
            if (row0 + k < a.chunk_capacity) put(a.chunks + (row0 + k) * P.D * P.S);
        }
        __syncthreads();
    }
    if (STATES) {
        put(a.carry + row * P.D * P.S);
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (q == 0 && ch + c < P.D) a.sums[row * P.D + ch + c] = dsum[c];
    } else if (a.fin && part == count - 1) {
        put(a.fin + (int64_t)n * P.D * P.S);
    }
}

// From what the parts end with to what the next ones start with, in place.
__global__ void __launch_bounds__(256) kda_ssm_carry_kernel(const __grid_constant__ ScanArgs a) {
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
    const int64_t d = m / P.S;
    const float A = P.A[m] * kLog2e;
    float c = a.init ? a.init[n * M + m] : 0.f;
    if (a.first) a.first[row * M + m] = c;
    float *p = a.carry + row * M + m;
    const float *s = a.sums + row * P.D + d;
    carry_on<false>(p, s, K, M, P.D, A, c);
}

template <typename IN, typename OUT, int LN, bool STATES>
cudaError_t launch_one(const ScanArgs &a, cudaStream_t stream) {
    using L = Layout<IN, LN>;
    const int smem = (int)sizeof(typename L::Smem);
    cudaError_t e = cudaFuncSetAttribute(kda_ssm_scan_kernel<IN, OUT, LN, STATES>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (STATES ? a.parts.rows : a.parts.most) * ((a.P.D + L::CB - 1) / L::CB);
    return launch_behind(!STATES && a.parts.rows > 0, kda_ssm_scan_kernel<IN, OUT, LN, STATES>, (unsigned)blocks, kThreads,
                         smem, stream, a);
}

template <typename IN, typename OUT, int LN>
cudaError_t launch(const ScanArgs &a, cudaStream_t stream) {
    if (a.parts.rows > 0) {
        // the output type plays no part in the states
        cudaError_t e = launch_one<IN, float, LN, true>(a, stream);
        if (e != cudaSuccess) return e;
        const int64_t blocks = (int64_t)a.parts.cut * (((int64_t)a.P.D * a.P.S + 255) / 256);
        e = launch_behind(true, kda_ssm_carry_kernel, (unsigned)blocks, 256, 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return launch_one<IN, OUT, LN, false>(a, stream);
}

template <typename IN, typename OUT>
cudaError_t by_states(const ScanArgs &a, cudaStream_t s) {
    if (a.P.S <= 8) return launch<IN, OUT, 2>(a, s);
    if (a.P.S <= 16) return launch<IN, OUT, 4>(a, s);
    if (a.P.S <= 32) return launch<IN, OUT, 8>(a, s);
    return launch<IN, OUT, 16>(a, s);
}

int64_t up4(int64_t n) { return (n + 3) / 4 * 4; }

// Cutting adds a pass over the states, 0.67 of the scan's own time.  8192 tokens, S = 16,
// bf16, whole against the best of 2 .. 64 parts: 4096 channels 425 and 277 us (7 parts; 4:
// 314, 19: 279), 2048: 422 and 152 (19), 1024: 414 and 84 (19), 512: 414 and 54 (37);
// 8192 channels: 432 and 513 (14).  One sequence of 256 tokens and 512 channels: whole 18.8 us, 8 parts 12.9.  fp32 rows
// of up to 16 states keep a block alone on its SM waiting for memory, so that a second one
// costs less (4096 channels: 396 us in 19 parts, 466 in the 7 of bf16; 8192: 700 in 2
// parts, 739 whole).  A ragged batch's sequence of up to 1.5 parts stays whole (28,000
// tokens in 8 sequences, 4096 channels: 655 us; with all longer ones cut 796).  Up to 8 states
// take a whole SM a block: 152 places are then 0.89 of the time of 304 (18 ragged batches).
Parts scan_parts(const SsmProblem &P, bool ragged) {
    const int LN = P.S <= 8 ? 2 : P.S <= 16 ? 4 : P.S <= 32 ? 8 : 16;
    const bool waits = P.in_dtype == KDA_DTYPE_F32 && LN <= 4;
    const double pair = LN == 2 ? 2.0 : waits ? 1.3 : 1.63, start = waits ? 1.8 : 3.0;
    return cut_parts(P, ragged, (P.D + 256 / LN - 1) / (256 / LN), {pair, 0.67, start, 0.1, 1.5, LN == 2 ? 152 : 304});
}

}  // namespace

// (for a batch with cu_seqlens and one without, whichever takes more)
int64_t kda_ssm_scan_ws(const SsmProblem &P) {
    const Parts x = scan_parts(P, true), y = scan_parts(P, false);
    const int64_t rows = x.rows > y.rows ? x.rows : y.rows;
    return (2 * up4(rows * P.D * P.S) + rows * P.D) * (int64_t)sizeof(float);
}

cudaError_t kda_launch_ssm_scan(const SsmProblem &P, const float *init, void *out, float *final_state,
                                float *chunk_states, int64_t chunk_capacity, float *workspace, cudaStream_t stream) {
    ScanArgs a{P, init, out, final_state, chunk_states, chunk_capacity, false, scan_parts(P, P.cu != nullptr), workspace, nullptr, nullptr};
    float *first = workspace + up4(a.parts.rows * P.D * P.S);
    a.sums = first + up4(a.parts.rows * P.D * P.S);
    if (init && init == final_state) a.first = first;
    const int es = P.out_dtype == KDA_DTYPE_BF16 ? 2 : 4;
    a.ovec = ((uintptr_t)out & 15u) == 0 && (int64_t)P.D * es % 16 == 0;
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return by_states<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (ib) return by_states<__nv_bfloat16, float>(a, stream);
    if (ob) return by_states<float, __nv_bfloat16>(a, stream);
    return by_states<float, float>(a, stream);
}
