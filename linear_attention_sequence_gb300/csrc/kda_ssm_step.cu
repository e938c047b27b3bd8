// kda_ssm_step.cu -- one token of the selective scan for N independent
// sequences, the states updated in place.
//
// HBM-bound: a state entry is read once and written once, 8 bytes for about 7
// operations.  One lane holds four states of a channel (a 16-byte access),
// LN = ceil(S / 4) lanes (a power of two) a channel; the lanes of a warp cover
// neighbouring channels, so a warp moves whole lines.  NB sequences a lane keep
// NB state loads in flight and use the decay rates A (read once from DRAM, then
// from L2) NB times.

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kThreads = 128;

struct StepArgs {
    SsmProblem P;
    float *state;
    void *out;
};

template <typename IN, typename OUT, int LN, int NB>
__global__ void __launch_bounds__(kThreads) kda_ssm_step_kernel(const StepArgs a) {
    constexpr int CB = kThreads / LN;
    const SsmProblem &P = a.P;
    const int ncb = (P.D + CB - 1) / CB;
    const int seq0 = (int)(blockIdx.x / ncb) * NB;
    const int ch = (int)(blockIdx.x % ncb) * CB + threadIdx.x / LN;
    const int q = threadIdx.x % LN, n0 = 4 * q;
    const bool live = ch < P.D;
    float4 h[NB];
    Raw<IN, 4> rb[NB], rc[NB];
    float dt[NB], u[NB], z[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t n = seq0 + i;
        h[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        rb[i].clear();
        rc[i].clear();
        dt[i] = u[i] = z[i] = 0.f;
        if (n < P.N && live) {
            const float *s = a.state + (n * P.D + ch) * P.S;
            if (P.svec) {
                if (n0 < P.S) h[i] = __ldcs(reinterpret_cast<const float4 *>(s + n0));
            } else {
                h[i] = load_states(s, n0, P.S, false);
            }
            if (n0 < P.S) {
                rb[i].load((const IN *)P.B.p + n * P.B.stride + n0, P.S - n0, P.B.vec);
                rc[i].load((const IN *)P.C.p + n * P.C.stride + n0, P.S - n0, P.C.vec);
            }
            dt[i] = ld_elem((const IN *)P.dt.p + n * P.dt.stride + ch);
            u[i] = ld_elem((const IN *)P.u.p + n * P.u.stride + ch);
            if (P.z.p) z[i] = ld_elem((const IN *)P.z.p + n * P.z.stride + ch);
        }
    }
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    float bias = 0.f, skip = 0.f;
    if (live) {
        A = load_states(P.A + (int64_t)ch * P.S, n0, P.S, P.svec);
        if (P.dt_bias) bias = P.dt_bias[ch];
        if (P.skip) skip = P.skip[ch];
    }
    A.x *= kLog2e; A.y *= kLog2e; A.z *= kLog2e; A.w *= kLog2e;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t n = seq0 + i;
        const float x = dt[i] + bias;
        const float dl = P.softplus ? softplus_fast(x) : x;
        const float du = dl * u[i];
        h[i].x = fmaf(exp2_fast(dl * A.x), h[i].x, du * rb[i].get(0));
        h[i].y = fmaf(exp2_fast(dl * A.y), h[i].y, du * rb[i].get(1));
        h[i].z = fmaf(exp2_fast(dl * A.z), h[i].z, du * rb[i].get(2));
        h[i].w = fmaf(exp2_fast(dl * A.w), h[i].w, du * rb[i].get(3));
        float y = fmaf(rc[i].get(0), h[i].x, rc[i].get(1) * h[i].y) + fmaf(rc[i].get(2), h[i].z, rc[i].get(3) * h[i].w);
#pragma unroll
        for (int off = LN / 2; off; off /= 2) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (n < P.N && live) {
            float *s = a.state + (n * P.D + ch) * P.S;
            if (P.svec) {
                if (n0 < P.S) __stcs(reinterpret_cast<float4 *>(s + n0), h[i]);
            } else {
                store_states(s, h[i], n0, P.S, false);
            }
            if (q == 0) {
                y = fmaf(skip, u[i], y);
                if (P.z.p) y *= z[i] * sigmoid_fast(z[i]);
                st_elem((OUT *)a.out + n * P.D + ch, y);
            }
        }
    }
}

template <typename IN, typename OUT, int LN>
cudaError_t launch(const StepArgs &a, cudaStream_t stream) {
    const int64_t ncb = (a.P.D + kThreads / LN - 1) / (kThreads / LN);
    // four sequences a lane once that still leaves every SM several blocks
    if (ncb * a.P.N >= 4 * 152 * 8) {
        kda_ssm_step_kernel<IN, OUT, LN, 4><<<(unsigned)(ncb * ((a.P.N + 3) / 4)), kThreads, 0, stream>>>(a);
    } else {
        kda_ssm_step_kernel<IN, OUT, LN, 1><<<(unsigned)(ncb * a.P.N), kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

template <typename IN, typename OUT>
cudaError_t by_states(const StepArgs &a, cudaStream_t s) {
    if (a.P.S <= 4) return launch<IN, OUT, 1>(a, s);
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
