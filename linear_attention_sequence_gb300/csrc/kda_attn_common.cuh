// kda_attn_common.cuh -- what the softmax attention kernels share: the problem as
// validated by the host, the tensor-core and packed-arithmetic instructions that
// sm100_ptx.cuh does not have, and the way a batch is cut into pieces of work.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "kda_common.cuh"
#include "sm100_ptx.cuh"

namespace kda {

constexpr int kAttnKeys = 128;             // keys of a tile of the tensor-core kernels
constexpr unsigned kAttnTimeout = 1u;      // status: a bounded wait gave up

// A validated attention call.  Activations [T, H, d] have strides in elements.
struct Attn {
    int32_t N, T, Hq, Hkv, G, d;
    int32_t in_dtype, out_dtype;
    const int32_t *cu;        // [N+1] or nullptr: N sequences of seq_len tokens
    int64_t seq_len;
    float scale_log2;         // scale * log2(e)
    float scale;
    const void *q, *k, *v;    // k, v: [T, Hkv, d], or pages [P, page, Hkv, d]
    int64_t q_t, q_h, k_t, k_h, v_t, v_h;
    // the cache (kda_attn_paged)
    const int32_t *table;     // [N, wide]
    const int32_t *lens;      // [N]: tokens in the cache, the new ones among them
    const int32_t *granted;   // [N] or nullptr: new tokens that got a place (all of a sequence's, or its tokens see nothing)
    int32_t P, page, wide;
    int64_t k_p, v_p;         // strides of a page
    // results
    void *out;                // [T, Hq, d], contiguous
    float *lse;               // [T, Hq] or nullptr; the backward reads it
};

// What the backward reads and writes besides.
struct AttnGrads {
    const void *out, *d_out;  // [T, Hq, d], strides in elements
    int64_t o_t, o_h, do_t, do_h;
    void *dq, *dk, *dv;       // contiguous
};

// Sequence n of the call: its tokens [a, b) and the keys it has.
struct AttnSeq {
    int64_t a, b, keys;
};
template <bool PAGED>
__device__ __forceinline__ AttnSeq attn_seq(const Attn &A, int n) {
    AttnSeq s;
    seq_bounds(A.cu, n, A.T, A.seq_len, s.a, s.b);
    s.keys = s.b - s.a;
    if (PAGED) {
        const int64_t most = (int64_t)A.wide * A.page, len = A.lens[n];
        s.keys = len < 0 ? 0 : len > most ? most : len;
        if (A.granted && A.granted[n] < s.b - s.a) s.keys = 0;
    }
    return s;
}

// The warp's number, as a value the compiler knows to be the same in all lanes: the products'
// descriptors are then formed in uniform registers, where the tensor cores take them (8192
// tokens of the forward: 362 -> 340 us).
__device__ __forceinline__ int attn_warp() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// ---------------------------------------------------------------- small arithmetic
// 2^x to about 2 ulp of fp32 (0 for -inf); the attention weights are rounded to 16 bits
// behind it, their sum in fp32 is not.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two 32-bit values as a pair of the packed fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two fp32 values rounded to a pair of 16-bit ones (a in the low half).
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    uint32_t r;
    if (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <bool BF16>
__device__ __forceinline__ void unpack16(uint32_t r, float &a, float &b) {
    if (BF16) {
        a = __uint_as_float(r << 16);
        b = __uint_as_float(r & 0xffff0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r));
        a = f.x;
        b = f.y;
    }
}

// ---------------------------------------------------------------- 16-bit tensor-core products
// Instruction descriptor, kind::f16: D fp32; A and B bf16 or fp16; A K-major; B K-major,
// or with `mn` the other way (its N index contiguous).
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int M, int N, bool mn) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// A tile of R rows (keys or tokens) by d channels of 16 bits lies in d / 64 blocks, each R
// rows of 128 bytes in the 128-byte swizzle.  Read K-major (the channels are summed over)
// a step of 16 channels moves 32 bytes inside a block: sm100::sdesc_sw128.  Read the other
// way (the rows are summed over, the channels are the N index) the leading offset is the
// distance of two blocks, and a step of 16 rows moves 2048 bytes.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(block_bytes >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
// Called by all 32 lanes of a converged warp; one of them issues (see sm100_ptx.cuh).
__device__ __forceinline__ void mma16_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Row block product D[128, N] (+)= A B^T over d channels: both operands K-major tiles.
template <int D, bool BF16, int N>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t a_saddr, uint32_t b_saddr, uint32_t a_block,
                                         uint32_t b_block) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        const uint32_t at = (s & 3) * 32;
        mma16_ss(d_tmem, sm100::sdesc_sw128(a_saddr + (s >> 2) * a_block + at),
                 sm100::sdesc_sw128(b_saddr + (s >> 2) * b_block + at), idesc_16(BF16, 128, N, false), s > 0);
    }
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z,
                                            int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(sm100::smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(sm100::smem_u32(bar))
        : "memory");
}

// 32 columns of tensor memory without the wait; tmem_wait_ld() comes before any use.  The values
// leave as fp32 registers, so that nothing (not even a change of type) reads them before
// the wait.
__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]),
          "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]),
          "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]),
          "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// The registers in `v` pass through, so that no use of them moves before the wait.
template <int K>
__device__ __forceinline__ void tmem_wait_ld(float (&v)[K]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < K; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tmem_st16_raw(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// One channel row of a result: 16-bit, or fp32.
template <bool BF16>
__device__ __forceinline__ void store8(void *base, bool f32, int64_t at, const float *x) {
    if (f32) {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
        p[0] = make_float4(x[0], x[1], x[2], x[3]);
        p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
            make_uint4(pack16<BF16>(x[0], x[1]), pack16<BF16>(x[2], x[3]), pack16<BF16>(x[4], x[5]),
                       pack16<BF16>(x[6], x[7]));
    }
}

// ---------------------------------------------------------------- bounded waits
// Waits of one block's roles on one another's barriers, each called by a whole warp (all of
// its lanes see the phase complete, or all give up: what they wait for is one word).  A wait
// that gives up records the status word; the warp then leaves its loop, and so do, each by
// its own bounded wait, those that depend on it.
constexpr uint32_t kAttnPolls = 1u << 20;
constexpr uint32_t kAttnLongPolls = 1u << 24;   // for waits that last as long as a piece of work
// The thread is suspended until the phase completes, or for up to a microsecond a poll (a
// sleep between polls would wake too late: 100 cycles count here).
__device__ __forceinline__ bool attn_poll(uint64_t *bar, uint32_t parity, uint32_t polls) {
#pragma unroll 1
    for (uint32_t i = 0; i < polls; ++i)
        if (sm100::mbar_try_wait_suspend(bar, parity, 1000)) return true;
    return false;
}
__device__ __forceinline__ bool attn_wait(uint64_t *bar, uint32_t parity, unsigned *status, uint32_t polls = kAttnPolls) {
    if (attn_poll(bar, parity, polls)) return true;
    atomicOr(status, kAttnTimeout);
    return false;
}
__device__ __forceinline__ bool attn_wait_long(uint64_t *bar, uint32_t parity, unsigned *status) {
    return attn_wait(bar, parity, status, kAttnLongPolls);
}

}  // namespace kda

// Allows a kernel `bytes` of dynamic shared memory on the current device, once a device (the call
// costs as much as a third of a launch).
template <auto Kernel>
cudaError_t kda_allow_smem(int bytes) {
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = (uint64_t)1 << (dev & 63);
    if (dev < 64 && (allowed.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launchers (kda_attn_*.cu).
int64_t kda_attn_paged_ws(const kda::Attn &A);
cudaError_t kda_launch_attn_prefill(const kda::Attn &A, cudaStream_t stream);
int64_t kda_attn_backward_ws(const kda::Attn &A);
cudaError_t kda_launch_attn_backward(const kda::Attn &A, const kda::AttnGrads &X, float *workspace, cudaStream_t stream);
cudaError_t kda_launch_attn_paged(const kda::Attn &A, void *workspace, cudaStream_t stream);

// A TMA view of [pages, rows, heads, d] 16-bit elements with strides in elements; a box is
// 64 channels of `box` rows of one head.  False if the driver refuses it.
bool kda_make_attn_map(CUtensorMap *m, const void *base, bool bf16, int d, int64_t heads, int64_t rows, int64_t pages,
                       int64_t s_head, int64_t s_row, int64_t s_page, int box);
