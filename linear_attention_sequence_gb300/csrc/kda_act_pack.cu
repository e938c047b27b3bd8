// kda_act_pack.cu -- activations in 8 bits.
//
// 32 neighbouring channels of a token share one scale:
//   m = max |x|,  scale = m / 127,  code = round(x * (127 / m))   (half to even)
// and code * scale stands for x, off by at most half a scale.  m = 0 (or below
// 2^-120, where 127 / m would overflow) gives scale = 0 and codes 0; an infinity or a
// NaN in the group gives scale = NaN, so that what is read back says so.
//
// HBM-bound: each element is read once (2 or 4 bytes) and written once (1 byte,
// and 4 bytes a group).  Four lanes take a group, 8 channels each, so that a warp
// reads and writes whole sectors and the maximum costs two exchanges; a thread
// has kIlp groups in flight.

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kThreads = 256;
constexpr int kIlp = 4;
constexpr int kE = kPackGroup / 4;   // channels of a lane

struct PackArgs {
    Rows x;
    int64_t total;      // groups
    int32_t D, ng;
    bool cvec;          // codes may be written 8 bytes at a time
    int8_t *codes;
    float *scales;
};

template <typename IN>
__global__ void __launch_bounds__(kThreads) kda_act_pack8_kernel(const PackArgs a) {
    const int64_t first = (int64_t)blockIdx.x * (kThreads / 4 * kIlp) + threadIdx.x / 4;
    const int sub = (threadIdx.x & 3) * kE;
    Raw<IN, kE> r[kIlp];
    int64_t row[kIlp];
    int col[kIlp];
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
        const int64_t g = first + i * (kThreads / 4);
        if (a.total >> 31) {
            row[i] = g / a.ng;
        } else {
            row[i] = (uint32_t)g / (uint32_t)a.ng;
        }
        col[i] = (int)(g - row[i] * a.ng) * kPackGroup + sub;
        r[i].clear();
        if (g < a.total && col[i] < a.D)
            r[i].load((const IN *)a.x.p + row[i] * a.x.stride + col[i], a.D - col[i], a.x.vec);
    }
#pragma unroll
    for (int i = 0; i < kIlp; ++i) {
        const int64_t g = first + i * (kThreads / 4);
        // the bits of |x| order as |x| does, and those of a NaN above all
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < kE; ++k) m = max(m, __float_as_uint(r[i].get(k)) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float amax = __uint_as_float(m);
        float scale, inv;
        if (m >= 0x7f800000u) {
            scale = __uint_as_float(0x7fc00000u);
            inv = 0.f;
        } else if (amax < 0x1p-120f) {
            scale = inv = 0.f;
        } else {
            scale = __fdiv_rn(amax, 127.f);
            inv = __fdiv_rn(127.f, amax);
        }
        if (g >= a.total) continue;
        if (sub == 0) a.scales[g] = scale;
        int8_t *p = a.codes + row[i] * a.D + col[i];
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kE; ++k) {
            // inf * 0 and NaN * 0 convert to 0
            const int v = __float2int_rn(r[i].get(k) * inv);
            c[k / 4] |= (uint32_t)(v & 0xff) << (8 * (k % 4));
        }
        if (a.cvec) {
            if (col[i] < a.D) *reinterpret_cast<uint2 *>(p) = make_uint2(c[0], c[1]);
        } else {
#pragma unroll
            for (int k = 0; k < kE; ++k)
                if (col[i] + k < a.D) p[k] = (int8_t)(c[k / 4] >> (8 * (k % 4)));
        }
    }
}

}  // namespace

cudaError_t kda_launch_act_pack8(int64_t rows, int32_t D, int32_t in_dtype, const Rows &x, int8_t *codes,
                                 float *scales, cudaStream_t stream) {
    PackArgs a;
    a.x = x;
    a.D = D;
    a.ng = (D + kPackGroup - 1) / kPackGroup;
    a.total = rows * a.ng;
    a.codes = codes;
    a.scales = scales;
    a.cvec = D % kE == 0 && ((uintptr_t)codes & 7u) == 0;
    const int64_t per = kThreads / 4 * kIlp;
    const unsigned blocks = (unsigned)((a.total + per - 1) / per);
    if (in_dtype == KDA_DTYPE_BF16)
        kda_act_pack8_kernel<__nv_bfloat16><<<blocks, kThreads, 0, stream>>>(a);
    else
        kda_act_pack8_kernel<float><<<blocks, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}
