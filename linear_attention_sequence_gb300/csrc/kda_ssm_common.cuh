// kda_ssm_common.cuh -- what the state space kernels share (sm_103a): packed
// fp32 arithmetic, the elementary functions, and loads of rows whose address
// or length may not allow vector accesses.
#pragma once

#include "kda_common.cuh"

namespace kda {

// Tokens of a scan tile, and the interval of the chunk states.
constexpr int kSsmTile = KDA_CHUNK;
// Channels that share one scale in the 8-bit packing.
constexpr int kPackGroup = KDA_PACK_GROUP;

// ---- kernels that follow one another
// A kernel launched by launch_behind() may start once every block of the one before
// it has started and called let_next(); it calls wait_before() ahead of its first read
// of what that one (and those before it) wrote.  The kernel in front of the first of
// such a chain is complete when the chain starts.  What the one before writes changes
// while the later kernel is on the GPU, so that it is read with ordinary loads; __ldg and
// ld.global.nc are for what no kernel of the chain writes.
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... Params, typename... Args>
cudaError_t launch_behind(bool behind, void (*kernel)(Params...), unsigned blocks, int threads, int smem, cudaStream_t stream,
                          const Args &...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = behind ? &attr : nullptr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- packed pairs of fp32 (one issue slot for two operations)
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f2 v) {
    float x, y;
    unpack2(v, x, y);
    return x + y;
}

// 2^x, relative error below 2^-22; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 exp2_pair(f2 v) {
    float x, y;
    unpack2(v, x, y);
    return pack2(exp2_fast(x), exp2_fast(y));
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// Sigmoid(x) = 1 / (1 + e^-x).  e^-x = inf gives 0, the limit.
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.f + exp2_fast(-kLog2e * x)); }

// softplus(x) = log(1 + e^x) = max(x, 0) + log1p(e^-|x|).  With w = e^-|x| in
// (0, 1] and r = w / (2 + w) <= 1/3, log1p(w) = 2 artanh(r) = r p(r^2), p(s) = 2 (1 +
// s/3 + s^2/5 + ...); p is a Chebyshev fit of degree 4 on [0, 1/9], off by less
// than 8e-9 of its value.  Small results keep their relative precision, which the
// logarithm of a rounded 1 + w would lose: step sizes of 1e-3 and less are ordinary.
__device__ __forceinline__ float softplus_fast(float x) {
    const float w = exp2_fast(-kLog2e * fabsf(x));
    const float r = w * rcp_fast(2.f + w);
    const float s = r * r;
    float p = 0.28174657f;
    p = fmaf(p, s, 0.27961419f);
    p = fmaf(p, s, 0.40024854f);
    p = fmaf(p, s, 0.66666316f);
    p = fmaf(p, s, 2.00000001f);
    return fmaf(p, r, fmaxf(x, 0.f));
}

// The same of many values at once, step by step, so that their chains of
// dependent operations overlap.
template <int N>
__device__ __forceinline__ void softplus_all(float (&x)[N]) {
    float w[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = exp2_fast(-kLog2e * fabsf(x[i]));
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = rcp_fast(2.f + w[i]);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const f2 q = mul2(pack2(w[i], w[i + 1]), pack2(r[i], r[i + 1])), s = mul2(q, q);
        f2 p = pack2(0.28174657f, 0.28174657f);
        p = fma2(p, s, pack2(0.27961419f, 0.27961419f));
        p = fma2(p, s, pack2(0.40024854f, 0.40024854f));
        p = fma2(p, s, pack2(0.66666316f, 0.66666316f));
        p = fma2(p, s, pack2(2.00000001f, 2.00000001f));
        p = fma2(p, q, pack2(fmaxf(x[i], 0.f), fmaxf(x[i + 1], 0.f)));
        unpack2(p, x[i], x[i + 1]);
    }
}

// ---- rows of activations as the kernels get them
struct Rows {
    const void *p;         // first element; nullptr: absent
    int64_t stride;        // elements from one token's row to the next
    const float *scales;   // != nullptr: int8 codes, [T, ngroups] scales
    int32_t ngroups;
    int32_t vec;           // rows may be read with 16-byte accesses
};

// Loads of inputs ahead of their use.  They stay where they are written (a plain
// read-only load may be moved by the compiler down to its first use, across
// barriers too), leave L1 to what is read again, and are predicated instead of
// branched around: a register that a load writes in one branch only is copied where
// the branches meet, and that copy waits for the load.  With !ok the value stays.
__device__ __forceinline__ void ahead16(uint32_t &x, uint32_t &y, uint32_t &z, uint32_t &w, const void *p, bool ok) {
    asm volatile("{ .reg .pred q; setp.ne.u32 q, %5, 0; @q ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4]; }"
                 : "+r"(x), "+r"(y), "+r"(z), "+r"(w) : "l"(p), "r"((uint32_t)ok));
}
__device__ __forceinline__ void ahead8(uint32_t &x, uint32_t &y, const void *p, bool ok) {
    asm volatile("{ .reg .pred q; setp.ne.u32 q, %3, 0; @q ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2]; }"
                 : "+r"(x), "+r"(y) : "l"(p), "r"((uint32_t)ok));
}
__device__ __forceinline__ void ahead4(uint32_t &x, const void *p, bool ok) {
    asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q ld.global.nc.L1::no_allocate.u32 %0, [%1]; }"
                 : "+r"(x) : "l"(p), "r"((uint32_t)ok));
}
__device__ __forceinline__ void ahead2(uint32_t &x, const void *p, bool ok) {
    asm volatile("{ .reg .pred q; .reg .u16 h; setp.ne.u32 q, %2, 0; mov.u16 h, 0; @q ld.global.nc.L1::no_allocate.u16 h, [%1]; "
                 "cvt.u32.u16 %0, h; }" : "+r"(x) : "l"(p), "r"((uint32_t)ok));
}

// E consecutive elements of a row, raw (as loaded) and as fp32.  Elements at or
// past `have` read as 0.
template <typename T, int E>
struct Raw {
    static constexpr int kBytes = E * (int)sizeof(T);
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    // All E elements, from an address aligned to min(16, kBytes) bytes; with !ok, zeros.
    __device__ __forceinline__ void load_if(const T *p, bool ok) {
        clear();
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                ahead16(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3], reinterpret_cast<const uint4 *>(p) + i, ok);
        } else if constexpr (kBytes % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 8; ++i) ahead8(w[2 * i], w[2 * i + 1], reinterpret_cast<const uint2 *>(p) + i, ok);
        } else if constexpr (kBytes % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) ahead4(w[i], reinterpret_cast<const uint32_t *>(p) + i, ok);
        } else {
            static_assert(kBytes == 2, "two, or a multiple of four bytes");
            ahead2(w[0], p, ok);
        }
    }
    // All E elements at once, for use soon.
    __device__ __forceinline__ void load_all(const T *p) {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
            }
        } else if constexpr (kBytes % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 8; ++i) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p) + i);
                w[2 * i] = v.x; w[2 * i + 1] = v.y;
            }
        } else if constexpr (kBytes % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
        } else {
            slow(p, E);
        }
    }
    // `vec`: p is aligned to min(16, kBytes) bytes; FULL: that, and all E elements exist
    template <bool FULL = false>
    __device__ __forceinline__ void load(const T *p, int have, bool vec) {
        if (FULL || (vec && have >= E)) load_all(p);
        else slow(p, have);
    }
    __device__ __forceinline__ void slow(const T *p, int have) {
        clear();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (i < have) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = __ldg(reinterpret_cast<const uint32_t *>(p) + i);
                } else if constexpr (sizeof(T) == 2) {
                    w[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(p) + i) << (16 * (i % 2));
                } else {
                    w[i / 4] |= (uint32_t)__ldg(reinterpret_cast<const unsigned char *>(p) + i) << (8 * (i % 4));
                }
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        if constexpr (sizeof(T) == 2) return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        // the byte, made 0 .. 255, as the last place of 2^23
        return __uint_as_float(__byte_perm(w[i / 4] ^ 0x80808080u, 0x4b000000u, 0x7440 + i % 4)) - 8388736.f;
    }
};

// E consecutive results of a row.  `vec`: the address is aligned to
// min(16, E * sizeof(T)) bytes; FULL: that, and all E exist.
template <typename T, int E, bool FULL = false>
__device__ __forceinline__ void store_row(T *p, const float (&v)[E], int have, bool vec) {
    constexpr int kBytes = E * (int)sizeof(T);
    if ((FULL || (vec && have >= E)) && kBytes % 4 == 0) {
        uint32_t w[(kBytes + 3) / 4];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&b);
            }
        }
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i)
                reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (kBytes % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kBytes / 8; ++i) reinterpret_cast<uint2 *>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < have) st_elem(p + i, v[i]);
    }
}

// Sums over groups of L lanes that are `STEP` lanes apart, K values at a time:
// each exchange keeps one half of the values and sends the other, so K values
// cost K - K/L exchanges where L <= K.  On return v[0 .. K/L - 1] holds the sums
// of values number (index of this lane in its group) * K/L + i.  L <= K.
template <int L, int STEP, int K>
__device__ __forceinline__ void reduce_scatter(float (&v)[K]) {
    static_assert(K % L == 0, "every lane ends with as many values");
    const int lane = threadIdx.x & 31;
    int n = K;
#pragma unroll
    for (int off = L / 2; off >= 1; off /= 2) {
        n /= 2;
        const bool up = lane & (off * STEP);
#pragma unroll
        for (int i = 0; i < K / 2; ++i) {
            if (i < n) {
                const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off * STEP);
            }
        }
    }
}

// Four states of one channel, n0 .. n0 + 3; those at or past S read as 0.
__device__ __forceinline__ float4 load_states(const float *p, int n0, int S, bool vec) {
    if (vec) return n0 < S ? *reinterpret_cast<const float4 *>(p + n0) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 r;
    r.x = n0 + 0 < S ? p[n0 + 0] : 0.f;
    r.y = n0 + 1 < S ? p[n0 + 1] : 0.f;
    r.z = n0 + 2 < S ? p[n0 + 2] : 0.f;
    r.w = n0 + 3 < S ? p[n0 + 3] : 0.f;
    return r;
}
__device__ __forceinline__ void store_states(float *p, float4 v, int n0, int S, bool vec) {
    if (vec) {
        if (n0 < S) *reinterpret_cast<float4 *>(p + n0) = v;
        return;
    }
    if (n0 + 0 < S) p[n0 + 0] = v.x;
    if (n0 + 1 < S) p[n0 + 1] = v.y;
    if (n0 + 2 < S) p[n0 + 2] = v.z;
    if (n0 + 3 < S) p[n0 + 3] = v.w;
}

// The sequence of token t in a packed batch: its number n and its bounds.  False
// if the token lies outside every sequence; then sa is the first token after t
// that may lie in one (total if there is none: no sequences, or malformed lengths), so
// that a walk which goes on there comes to an end.  t < total.
__host__ __device__ __forceinline__ bool find_seq(const int32_t *cu, int N, int64_t total, int64_t seq_len, int64_t t,
                                                  int &n, int64_t &sa, int64_t &sb) {
    if (!cu) {
        n = (int)(t / seq_len);   // t < total = N seq_len, so seq_len > 0
    } else {
        int lo = -1, hi = N;      // cu[lo] <= t < cu[hi], taking cu[-1] = -inf and cu[N] = inf
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (cu[m] <= t) lo = m; else hi = m;
        }
        n = lo;
        if (n < 0) {              // before the first sequence, or there is none
            const int64_t first = N > 0 ? cu[0] : total;
            sa = sb = first > t && first < total ? first : total;
            return false;
        }
    }
    seq_bounds(cu, n, total, seq_len, sa, sb);
    if (t >= sa && t < sb) return true;
    sa = sb = total;              // behind the last sequence (or a malformed array)
    return false;
}

// How sequences are cut into parts that run side by side: one of more than
// `whole` tokens into parts of `len` (the last may be shorter), any other stays one
// part (an empty one too).
struct Parts {
    int64_t len, whole;
    int32_t most;            // parts of the batch at most
    int64_t rows;            // parts that have one behind them, at most: rows of a carry
    int32_t cut;             // sequences that are cut, at most

    __host__ __device__ int of(int64_t n) const {
        return n > whole ? (int)(((unsigned)n + (unsigned)len - 1u) / (unsigned)len) : 1;
    }
};

// A part of a batch: its sequence (-1: there is none), its place in it, the sequence's
// number of parts, and the row of a carry between it and the part behind it (of a last
// part, the row past its sequence's).
struct Part {
    int n, k, count, row;
};

// The part of a batch in place p of the launch; places start in order, so the parts of
// long sequences come first and the short sequences fill in at the end (scan, 16 sequences
// of up to 1500 tokens, 2048 channels: 118 us, in their own order 234).  A thread looks at
// one sequence, as in longest_first(), and the one that p falls in answers through
// *answer; batches of more sequences than threads keep their order.  Every thread of the
// block must call it.
__device__ __forceinline__ Part longest_part(const Parts &parts, const int32_t *cu, int N, int64_t total, int64_t seq_len,
                                             int p, Part *answer) {
    Part w;
    w.n = -1;
    w.k = 0;
    w.count = 1;
    w.row = 0;
    if (!cu) {
        w.count = parts.of(seq_len);
        w.n = p / w.count;
        w.k = p - w.n * w.count;
        w.row = p - w.n;
        if (w.n >= N) w.n = -1;
        return w;
    }
    if (threadIdx.x == 0) *answer = w;
    __syncthreads();
    if (N <= (int)blockDim.x) {
        const int m = threadIdx.x;
        if (m < N) {
            int64_t a, b;
            seq_bounds(cu, m, total, seq_len, a, b);
            const int64_t n = b - a;
            int before = 0, rows = 0;
            for (int m2 = 0; m2 < N; ++m2) {
                seq_bounds(cu, m2, total, seq_len, a, b);
                const int c = parts.of(b - a);
                if (b - a > n || (b - a == n && m2 < m)) before += c;
                if (m2 < m) rows += c - 1;
            }
            w.count = parts.of(n);
            w.k = p - before;
            w.n = m;
            w.row = rows + w.k;
            if (w.k >= 0 && w.k < w.count) *answer = w;
        }
    } else if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int before = 0;
        for (int m0 = 0; m0 < N; m0 += 32) {
            int c = 0;
            if (m0 + lane < N) {
                int64_t a, b;
                seq_bounds(cu, m0 + lane, total, seq_len, a, b);
                c = parts.of(b - a);
            }
            int upto = c;
#pragma unroll
            for (int off = 1; off < 32; off *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
            }
            w.k = p - (before + upto - c);
            if (w.k >= 0 && w.k < c) {
                w.n = m0 + lane;
                w.count = c;
                w.row = p - w.n;
                *answer = w;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
            if (before > p) break;
        }
    }
    __syncthreads();
    return *answer;
}

// The part before row r of a carry (CUT: the first of the cut sequence number r).
// Every warp finds it by itself (all 32 lanes must call).
template <bool CUT>
__device__ __forceinline__ Part part_of_row(const Parts &parts, const int32_t *cu, int N, int64_t total, int64_t seq_len,
                                            int r) {
    Part w;
    w.n = -1;
    w.k = 0;
    w.count = 1;
    w.row = 0;
    if (!cu) {
        w.count = parts.of(seq_len);
        const int rows = w.count - 1;
        if (rows == 0) return w;
        w.n = CUT ? r : r / rows;
        w.k = CUT ? 0 : r - w.n * rows;
        w.row = CUT ? w.n * rows : r;
        if (w.n >= N) w.n = -1;
        return w;
    }
    const int lane = threadIdx.x & 31;
    int rows = 0, seen = 0;                    // of the sequences before: rows, and those that are cut
    for (int m0 = 0; m0 < N; m0 += 32) {
        int c = 0;
        if (m0 + lane < N) {
            int64_t a, b;
            seq_bounds(cu, m0 + lane, total, seq_len, a, b);
            c = parts.of(b - a) - 1;
        }
        const unsigned cut = __ballot_sync(0xffffffffu, c > 0);
        int upto = c;
#pragma unroll
        for (int off = 1; off < 32; off *= 2) {
            const int x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        const int k = r - (rows + upto - c);
        const bool mine = CUT ? c > 0 && seen + __popc(cut & ((1u << lane) - 1u)) == r : k >= 0 && k < c;
        const unsigned hit = __ballot_sync(0xffffffffu, mine);
        if (hit) {
            const int l = __ffs(hit) - 1;
            w.n = m0 + l;
            w.count = __shfl_sync(0xffffffffu, c, l) + 1;
            w.k = CUT ? 0 : __shfl_sync(0xffffffffu, k, l);
            w.row = CUT ? __shfl_sync(0xffffffffu, rows + upto - c, l) : r;
            return w;
        }
        rows += __shfl_sync(0xffffffffu, upto, 31);
        seen += __popc(cut);
    }
    return w;
}

// The rows of a carry in place: p[k M] becomes c' = p[k M] + exp2(A s[k D]) c, k = 0 .. K-1 or
// back (BACK).  Eight rows are read before the first of them is written, so that their
// loads overlap (18 rows of 4096 x 16: 13.2 -> 6.9 us).
template <bool BACK>
__device__ __forceinline__ void carry_on(float *p, const float *s, int K, int64_t M, int64_t D, float A, float c) {
    constexpr int R = 8;
    for (int k0 = 0; k0 < K; k0 += R) {
        float local[R], sum[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            const int i = min(k0 + j, K - 1), k = BACK ? K - 1 - i : i;
            local[j] = p[k * M];
            sum[j] = s[k * D];
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (k0 + j < K) {
                c = c != 0.f ? fmaf(exp2_fast(A * sum[j]), c, local[j]) : local[j];
                p[(BACK ? K - 1 - (k0 + j) : k0 + j) * M] = c;
            }
        }
    }
}

// Launch parameters of the state space kernels after validation.
struct SsmProblem {
    int32_t N, T, D, S;          // sequences, tokens, channels, states per channel (or taps)
    int32_t in_dtype, out_dtype;
    int64_t seq_len;             // tokens per sequence where cu is nullptr
    const int32_t *cu;
    Rows u, dt, B, C, z, dy;
    const float *A, *skip, *dt_bias;
    bool softplus;
    bool svec;                   // state rows may be read with 16-byte accesses
};

// What a kernel's run takes, in the time that a block alone on its SM takes for a tile.
struct PartCosts {
    double pair;             // two blocks that share an SM, each a tile (2: they do not share)
    double first;            // the pass that cutting adds, of the kernel's own
    double start;            // a round of blocks, before their first tile
    double part;             // a part in the carry
    double whole;            // a ragged batch's longest sequence that stays whole, in parts' lengths
    int places;              // parts that a ragged batch is cut into, at full length
};

// How a batch is cut, with `across` blocks side by side for a sequence: into the K
// parts of least cost, if n blocks run in rounds of 304, of which the last may find them
// alone (a little less than alone after others: the first to end make room early).
// Against the best of up to 20 K on batches of equal lengths (64 .. 8192 tokens, 64 ..
// 8192 channels, 8 .. 64 states) what it picks takes 1.00 to 1.09 of the time.  Where
// the lengths are known only on the device (`ragged`), a part is one place's share of the
// batch's work, which no sequence that stays whole outlasts by much (30 batches, S = 16: shares
// of one 380th, 456th and 608th take 1.02 to 1.12 of a 304th's time, one 152nd 1.0 to 1.4).
inline Parts cut_parts(const SsmProblem &P, bool ragged, int64_t across, const PartCosts &c) {
    if (P.N == 0) return {kSsmTile, INT32_MAX, 0, 0, 0};   // no parts, whatever rows there are
    const int64_t tokens = ragged ? P.T : P.T / P.N, b = ragged ? across : across * P.N;
    const int64_t tiles = (tokens + kSsmTile - 1) / kSsmTile;
    const auto cost = [&](int64_t n, int64_t t) {
        const int64_t full = n / 304, rest = n % 304;
        const double last = rest > 152 ? c.pair : rest == 0 ? 0.0 : full > 0 ? 0.9 : 1.0;
        return (c.pair * (double)full + last) * (double)t + c.start * (double)(full + (rest > 0));
    };
    Parts parts;
    parts.len = (tiles < 1 ? 1 : tiles) * kSsmTile;
    parts.whole = INT32_MAX;
    if (ragged) {
        const int64_t t = (tiles * across + c.places - 1) / c.places;
        if (t < tiles) {
            parts.len = t * kSsmTile;
            parts.whole = (int64_t)(c.whole * (double)parts.len);
        }
    } else {
        double least = cost(b, tiles);
        for (int64_t K = 2; K <= 64 && K <= tiles; ++K) {
            const int64_t t = (tiles + K - 1) / K, k = (tiles + t - 1) / t;
            if (k != K) continue;              // (as short as with fewer)
            const double x = c.first * cost(b * (k - 1), t) + cost(b * k, t) + c.part * (double)k;
            if (x < least) {
                least = x;
                parts.len = parts.whole = t * kSsmTile;
            }
        }
    }
    parts.rows = parts.whole == INT32_MAX ? 0 : ragged ? P.T / parts.len : (int64_t)P.N * (parts.of(tokens) - 1);
    parts.cut = ragged && parts.rows < P.N ? (int32_t)parts.rows : parts.rows ? P.N : 0;
    parts.most = P.N + (int32_t)parts.rows;
    return parts;
}

}  // namespace kda

// Launchers.
cudaError_t kda_launch_act_pack8(int64_t rows, int32_t D, int32_t in_dtype, const kda::Rows &x, int8_t *codes,
                                 float *scales, cudaStream_t stream);
cudaError_t kda_launch_ssm_scan(const kda::SsmProblem &P, const float *init, void *out, float *final_state,
                                float *chunk_states, int64_t chunk_capacity, float *workspace, cudaStream_t stream);
int64_t kda_ssm_scan_ws(const kda::SsmProblem &P);
cudaError_t kda_launch_ssm_conv(const kda::SsmProblem &P, const float *w, const float *bias, const float *cin,
                                bool swish, void *out, float *cout, cudaStream_t stream);
int64_t kda_ssm_conv_backward_tiles(const kda::SsmProblem &P, int *tile);
cudaError_t kda_launch_ssm_conv_backward(const kda::SsmProblem &P, const float *w, const float *bias,
                                         const float *cin, const float *dcout, bool swish, void *dx, float *dw,
                                         float *dbias, float *dcin, float *workspace, cudaStream_t stream);
int64_t kda_ssm_scan_backward_ws(const kda::SsmProblem &P);
cudaError_t kda_launch_ssm_scan_backward(const kda::SsmProblem &P, const float *init, const float *chunk_states,
                                         int64_t chunk_capacity, const float *d_final, void *du, void *ddt, void *dB,
                                         void *dC, void *dz, float *dA, float *dskip, float *dbias, float *d_init,
                                         float *workspace, cudaStream_t stream);
cudaError_t kda_ssm_read_status(unsigned *status);
cudaError_t kda_launch_ssm_step(const kda::SsmProblem &P, float *state, void *out, cudaStream_t stream);
