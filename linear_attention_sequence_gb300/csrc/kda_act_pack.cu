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
// has the same channels of four rows in flight.  8192 x 12288 bf16: 49 us, 6.4 TB/s
// (94 % of the measured copy rate).

#include "kda_ssm_common.cuh"

namespace {

using namespace kda;

constexpr int kThreads = 256;
constexpr int kRowsOf = 4;           // rows of a thread, all loaded before the first is used
constexpr int kE = kPackGroup / 4;   // channels of a lane

struct PackArgs {
    Rows x;
    int64_t rows, total;   // total: groups across x blocks of kRowsOf rows
    int32_t D, ng;
    bool cvec;             // codes may be written 8 bytes at a time
    int8_t *codes;
    float *scales;
};

// The largest |x| of a lane's channels, as bits: the bits of |x| order as |x|
// does, and those of a NaN above all.
__device__ __forceinline__ uint32_t abs_max(const Raw<float, kE> &r) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kE; ++k) m = max(m, r.w[k] & 0x7fffffffu);
    return m;
}
__device__ __forceinline__ uint32_t abs_max(const Raw<__nv_bfloat16, kE> &r) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kE / 2; ++k) m = __vmaxu2(m, r.w[k] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
}

template <typename IN, bool FULL>
__global__ void __launch_bounds__(kThreads) kda_act_pack8_kernel(const __grid_constant__ PackArgs a) {
    // four lanes to a group of channels, of kRowsOf rows
    const int64_t id = (int64_t)blockIdx.x * (kThreads / 4) + threadIdx.x / 4;
    const int64_t block = a.total >> 32 ? id / a.ng : (int64_t)((uint32_t)id / (uint32_t)a.ng);
    const int g = (int)(id - block * a.ng);
    const int col = g * kPackGroup + (threadIdx.x & 3) * kE;
    const int64_t row = block * kRowsOf;
    const int rows = (int)max((int64_t)0, min((int64_t)kRowsOf, a.rows - row));
    const int have = a.D - col;                 // <= 0: only the exchange
    const IN *x = (const IN *)a.x.p + row * a.x.stride + col;
    Raw<IN, kE> r[kRowsOf];
#pragma unroll
    for (int i = 0; i < kRowsOf; ++i, x += a.x.stride) {
        if (i < rows && (FULL || have > 0)) r[i].template load<FULL>(x, have, a.x.vec);
        else r[i].clear();
    }
    int8_t *codes = a.codes + row * a.D + col;
    float *scales = a.scales + row * a.ng + g;
#pragma unroll
    for (int i = 0; i < kRowsOf; ++i, codes += a.D, scales += a.ng) {
        uint32_t m = abs_max(r[i]);
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
        if (i >= rows) continue;
        if ((threadIdx.x & 3) == 0) *scales = scale;
        // 1.5 2^23 + v, whose last place is 1, rounds v to an integer (half to even) and
        // holds it in its low byte
        uint32_t b[kE], c[2];
#pragma unroll
        for (int k = 0; k < kE; ++k) b[k] = __float_as_uint(__fadd_rn(__fmul_rn(r[i].get(k), inv), 12582912.f));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            c[k] = __byte_perm(__byte_perm(b[4 * k], b[4 * k + 1], 0x0040), __byte_perm(b[4 * k + 2], b[4 * k + 3], 0x0040), 0x5410);
        if (FULL || (a.cvec && have >= kE)) {
            *reinterpret_cast<uint2 *>(codes) = make_uint2(c[0], c[1]);
        } else {
#pragma unroll
            for (int k = 0; k < kE; ++k)
                if (k < have) codes[k] = (int8_t)(c[k / 4] >> (8 * (k % 4)));
        }
    }
}

template <typename IN>
void launch(const PackArgs &a, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((a.total * 4 + kThreads - 1) / kThreads);
    // whole groups, and accesses as wide as a lane's share
    if (a.x.vec && a.cvec && a.D % kPackGroup == 0)
        kda_act_pack8_kernel<IN, true><<<blocks, kThreads, 0, stream>>>(a);
    else
        kda_act_pack8_kernel<IN, false><<<blocks, kThreads, 0, stream>>>(a);
}

}  // namespace

cudaError_t kda_launch_act_pack8(int64_t rows, int32_t D, int32_t in_dtype, const Rows &x, int8_t *codes,
                                 float *scales, cudaStream_t stream) {
    PackArgs a;
    a.x = x;
    a.D = D;
    a.ng = (D + kPackGroup - 1) / kPackGroup;
    a.rows = rows;
    a.total = (rows + kRowsOf - 1) / kRowsOf * a.ng;
    a.codes = codes;
    a.scales = scales;
    a.cvec = D % kE == 0 && ((uintptr_t)codes & 7u) == 0;
    if (in_dtype == KDA_DTYPE_BF16) launch<__nv_bfloat16>(a, stream);
    else launch<float>(a, stream);
    return cudaGetLastError();
}
