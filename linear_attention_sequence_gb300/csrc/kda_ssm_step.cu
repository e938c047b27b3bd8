// kda_ssm_step.cu -- one token of the selective scan for N independent
// sequences, the states updated in place.
//
// HBM-bound: a state entry is read once and written once, 8 bytes for about 7
// operations.  One lane holds four states of a channel (a 16-byte access),
// LN >= S / 4 lanes (2, 4, 8 or 16) a channel; the lanes of a warp cover
// neighbouring channels, so a warp moves whole lines.  NB sequences a lane keep
// NB state loads in flight and use the decay rates A (read once from DRAM, then
// from L2) NB times; a channel's lanes share out the step sizes and gates of
// the NB sequences between them.  256 sequences of 12288 channels with 16 states, bf16: 69 us,
// 6.2 TB/s (91 % of the measured copy rate); every lane computing its own step sizes: 118 us.

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kThreads = 128;

struct StepArgs {
    SsmProblem P;
    float *state;
    void *out;
};

// NB sequences a lane; lane q of a channel prepares and finishes OWN of them: numbers
// q OWN .. (where LN > NB, lanes from NB on none).  FULL: four states at a time.
template <typename IN, typename OUT, int LN, int NB, bool FULL>
__global__ void __launch_bounds__(kThreads) kda_ssm_step_kernel(const __grid_constant__ StepArgs a) {
    constexpr int CB = kThreads / LN;
    constexpr int OWN = NB >= LN ? NB / LN : 1;
    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB;
    const int64_t seq0 = (int64_t)(blockIdx.x / ncb) * NB;
    const int count = (int)min((int64_t)NB, P.N - seq0);
    const int chx = (int)(blockIdx.x % ncb) * CB + threadIdx.x / LN;
    const bool live = chx < P.D;
    const int ch = live ? chx : P.D - 1;        // lanes past the last channel run along on it
    const int q = threadIdx.x % LN, n0 = 4 * q;
    float4 h[NB];
    Raw<IN, 4> rb[NB], rc[NB];
    float *st = a.state + (seq0 * P.D + ch) * P.S + n0;
    const int64_t sstep = (int64_t)P.D * P.S;
    const IN *pb = (const IN *)P.B.p + seq0 * P.B.stride + n0, *pc = (const IN *)P.C.p + seq0 * P.C.stride + n0;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        h[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        rb[i].clear();
        rc[i].clear();
        if (i < count && n0 < P.S) {
            if (FULL) {
                h[i] = __ldcs(reinterpret_cast<const float4 *>(st + i * sstep));
            } else {
                h[i] = load_states(st + i * sstep, 0, P.S - n0, P.svec);
            }
            rb[i].template load<FULL>(pb + i * P.B.stride, P.S - n0, P.B.vec);
            rc[i].template load<FULL>(pc + i * P.C.stride, P.S - n0, P.C.vec);
        }
    }
    const int first = OWN * (LN > NB && q >= NB ? 0 : q);
    float dt[OWN], u[OWN], z[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int64_t n = seq0 + min(first + i, count - 1);
        dt[i] = ld_elem((const IN *)P.dt.p + n * P.dt.stride + ch);
        u[i] = ld_elem((const IN *)P.u.p + n * P.u.stride + ch);
        z[i] = P.z.p ? ld_elem((const IN *)P.z.p + n * P.z.stride + ch) : 0.f;
    }
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n0 < P.S) {
        const float *p = P.A + (int64_t)ch * P.S + n0;
        A = FULL ? *reinterpret_cast<const float4 *>(p) : load_states(p, 0, P.S - n0, P.svec);
    }
    A.x *= kLog2e; A.y *= kLog2e; A.z *= kLog2e; A.w *= kLog2e;
    const float bias = P.dt_bias ? P.dt_bias[ch] : 0.f, skip = P.skip ? P.skip[ch] : 0.f;
    float dl[OWN], du[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const float x = dt[i] + bias;
        dl[i] = P.softplus ? softplus_fast(x) : x;
        du[i] = dl[i] * u[i];
    }
    float y[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const float d = __shfl_sync(0xffffffffu, dl[i % OWN], i / OWN, LN), x = __shfl_sync(0xffffffffu, du[i % OWN], i / OWN, LN);
        h[i].x = fmaf(exp2_fast(d * A.x), h[i].x, x * rb[i].get(0));
        h[i].y = fmaf(exp2_fast(d * A.y), h[i].y, x * rb[i].get(1));
        h[i].z = fmaf(exp2_fast(d * A.z), h[i].z, x * rb[i].get(2));
        h[i].w = fmaf(exp2_fast(d * A.w), h[i].w, x * rb[i].get(3));
        y[i] = fmaf(rc[i].get(0), h[i].x, rc[i].get(1) * h[i].y) + fmaf(rc[i].get(2), h[i].z, rc[i].get(3) * h[i].w);
        if (i < count && live && n0 < P.S) {
            if (FULL) {
                __stcs(reinterpret_cast<float4 *>(st + i * sstep), h[i]);
            } else {
                store_states(st + i * sstep, h[i], 0, P.S - n0, P.svec);
            }
        }
    }
    if constexpr (LN > NB) {
        // lanes NB apart first, then as below
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int off = LN / 2; off >= NB; off /= 2) y[i] += __shfl_xor_sync(0xffffffffu, y[i], off);
        reduce_scatter<NB, 1, NB>(y);
    } else {
        reduce_scatter<LN, 1, NB>(y);
    }
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        if (live && q * OWN + i < count) {
            float v = fmaf(skip, u[i], y[i]);
            if (P.z.p) v *= z[i] * sigmoid_fast(z[i]);
            st_elem((OUT *)a.out + (seq0 + q * OWN + i) * P.D + ch, v);
        }
    }
}

template <typename IN, typename OUT, int LN, int NB>
cudaError_t launch_nb(const StepArgs &a, cudaStream_t stream) {
    const SsmProblem &P = a.P;
    const int64_t blocks = (P.D + kThreads / LN - 1) / (kThreads / LN) * (((int64_t)P.N + NB - 1) / NB);
    if (P.svec && P.B.vec && P.C.vec)
        kda_ssm_step_kernel<IN, OUT, LN, NB, true><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    else
        kda_ssm_step_kernel<IN, OUT, LN, NB, false><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename IN, typename OUT, int LN>
cudaError_t launch(const StepArgs &a, cudaStream_t stream) {
    const int64_t ncb = (a.P.D + kThreads / LN - 1) / (kThreads / LN);
    // four sequences a lane once that still leaves every SM several blocks
    if (ncb * a.P.N >= 4 * 152 * 8) return launch_nb<IN, OUT, LN, 4>(a, stream);
    return launch_nb<IN, OUT, LN, 1>(a, stream);
}

template <typename IN, typename OUT>
cudaError_t by_states(const StepArgs &a, cudaStream_t s) {
    if (a.P.S <= 8) return launch<IN, OUT, 2>(a, s);
    if (a.P.S <= 16) return launch<IN, OUT, 4>(a, s);
    if (a.P.S <= 32) return launch<IN, OUT, 8>(a, s);
    return launch<IN, OUT, 16>(a, s);
}

}  // namespace

cudaError_t kda_launch_ssm_step(const SsmProblem &P, float *state, void *out, cudaStream_t stream) {
    const StepArgs a{P, state, out};
    const bool ib = P.in_dtype == KDA_DTYPE_BF16, ob = P.out_dtype == KDA_DTYPE_BF16;
    if (ib && ob) return by_states<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (ib) return by_states<__nv_bfloat16, float>(a, stream);
    if (ob) return by_states<float, __nv_bfloat16>(a, stream);
    return by_states<float, float>(a, stream);
}
