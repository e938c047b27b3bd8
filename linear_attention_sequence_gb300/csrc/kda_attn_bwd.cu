// kda_attn_bwd.cu -- gradients of causal softmax attention over packed prompts
// (kda_attn_backward) on the tensor cores (sm_103a).
//
//   P = e^(scale Q K^T - lse),  dP = dO V^T,  delta = rowsum(dO O),  dS = P (dP - delta)
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
//
// P is formed again from the forward's log-sums; nothing of size T x T is kept.  dK and dV sum
// over the queries and over the heads of a group, dQ over the keys.  Two kinds of blocks
// share one launch, each with its sum in tensor memory from first to last, so that no sum
// depends on timing and nothing is added in global memory:
//
//   key blocks    128 keys of a key head against all query tiles that see them, head by head
//                 of the group.  The products are taken with the keys as rows (S^T = K Q^T, dP^T
//                 = V dO^T), so that P^T and dS^T stand in tensor memory as the A operands of
//                 dV and dK.  4 products a tile pair.
//   query blocks  128 queries of a head against the key tiles they see.  3 products.
//
// That is 7 products where a single pass with additions of dQ in global memory needs 5; the two
// more are the price of results that repeat bit by bit.  A key block walks the heads of its group one
// after another and is not cut, so that few key heads leave SMs idle: 8192 tokens of heads of 128 take 91 us
// with one head, 322 with 4 on one, 640 with 8 and 950 with 12 (32 on 8: 1,130 by themselves).
//
// In both, two threads a row: warps 0-3 have the first 64 columns of a score tile and warps 4-7
// the others.  P and dS are rounded to the inputs' 16-bit type because the tensor cores read
// them so; all sums are fp32.  A sequence of one tile (128 tokens) has few rows over which
// that rounding averages out, and time to spare: what it leaves follows as a second operand, in the
// columns of tensor memory that the 16-bit values leave free.
//
// fp16 has few powers of two: below 2^-14 its step is fixed, above 65504 it ends.  P and dS are therefore
// stored times powers of two that the epilogues take back.  P <= 1 is stored as 2^15 P (folded into
// lse log2 e).  |dS| <= 2 |d_out_i| max_j |v_j| (delta is d_out_i . out_i, and out_i a mean of values), so
// that 2^15 over that bound is safe whatever the inputs: for a query block's row with the row's own |d_out_i|, for
// a key block, whose sums run over the queries, with the largest |d_out_i| of the queries that see it.  The
// delta kernel leaves the norms, and each block looks for the maxima it needs before its first step: four
// bytes a token and head next to a step's 2,000 cycles.  (Maxima kept by atomics instead, and cleared by a
// memset: 90 us for the 13 packed prompts, which take 57.4 us like this and took 53.4 unscaled; 8192 tokens with 32 on 8
// heads of 128 take 1,183 us and took 1,154.)
#include <stddef.h>

#include "kda_attn_plan.cuh"

using namespace kda;

namespace {

__device__ unsigned g_attn_bwd_status;

constexpr int kThreads = 352;   // eight compute warps, products, loads, row statistics
constexpr int kProductWarp = 8, kLoadWarp = 9, kStatWarp = 10;
constexpr int kTile = 128;

struct Grads {
    const void *out, *d_out;
    int64_t o_t, o_h, do_t, do_h;
    void *dq, *dk, *dv;
    float *delta, *lse2;     // [Hq][T]; fp16: lse log2(e) - kPLog2
    float *y_norm, *v_norm;  // fp16: [Hq][T], |d_out|^2; [Hkv][T], |v|^2
    int64_t key_blocks;      // blocks below this one are key blocks
};

template <int D>
struct Lay {
    static constexpr int kBytes = kTile * D * 2;   // a tile of 128 rows
    static constexpr int kBlock = kTile * 128;     // 64 channels of it
    // Two rings of tiles.  A: queries (key blocks) or keys (query blocks), held from the scores to the
    // last product of a step; B: dO or values, held for less.
    static constexpr int kA = D == 128 ? 3 : 4, kB = D == 128 ? 2 : 4;
    static constexpr int kTiles = (2 + kA + kB) * kBytes;
};
constexpr int kStats = 2;   // steps of row statistics in flight
constexpr float kPLog2 = 15.f, kPScale = 32768.f;   // fp16: P is stored times 2^15

struct alignas(16) Control {
    uint64_t own_full, a_full[4], a_empty[4], b_full[4], b_empty[4], stat_full[kStats], stat_empty[kStats];
    uint64_t s_full[2], p_ready, dp_full, dp_free, ds_ready[2], done;
    uint32_t tmem;
    AttnPart part;
    int64_t scan[kThreads / 32];
    alignas(16) float stat[kStats][2][kTile];   // read as float4
    float most[2][8];   // fp16: each compute warp's largest |d_out|^2 and |v|^2
};
static_assert(offsetof(Control, stat) % 16 == 0 && alignof(Control) % 16 == 0, "vector reads of stat");

// fp16: the power of two that dS is stored times, from |d_out|^2 and the largest |v|^2: with x their product,
// 2 sqrt(x) times it is at most 2^15 (1 where there is nothing to scale, or an infinity or NaN, which stays one).
__device__ __forceinline__ float range_scale(float dd, float vv) {
    const float x = dd * vv;   // (2^-96 ... 2^79, or 0)
    if (!(x > 0.f && x < INFINITY)) return 1.f;
    const int half = ((int)(__float_as_uint(x) >> 23) - 127 + 2) >> 1;   // sqrt(x) < 2^half
    return __uint_as_float((uint32_t)(14 - half + 127) << 23);
}

// delta and lse log2(e), head-major.  16 (8) lanes a row.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) kda_attn_delta_kernel(const Attn A, const Grads B) {
    constexpr int LANES = D / 8;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
    const int c = threadIdx.x % LANES;
    const int64_t rows = (int64_t)A.T * A.Hq;
    float sum = 0.f, dd = 0.f, vv = 0.f;
    const int64_t t = row / A.Hq, h = row - t * A.Hq;
    if (row < rows) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(B.out) + t * B.o_t + h * B.o_h) + c);
        const uint4 y = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(B.d_out) + t * B.do_t + h * B.do_h) + c);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b, e, f;
            unpack16<BF16>(xs[i], a, b);
            unpack16<BF16>(ys[i], e, f);
            sum = fmaf(a, e, fmaf(b, f, sum));
            if (!BF16) dd = fmaf(e, e, fmaf(f, f, dd));
        }
        if (!BF16 && h % A.G == 0) {   // the key head's values once
            const uint4 z = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(A.v) + t * A.v_t + h / A.G * A.v_h) + c);
            const uint32_t zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, b;
                unpack16<BF16>(zs[i], a, b);
                vv = fmaf(a, a, fmaf(b, b, vv));
            }
        }
    }
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (!BF16) {
            dd += __shfl_xor_sync(0xffffffffu, dd, o);
            vv += __shfl_xor_sync(0xffffffffu, vv, o);
        }
    }
    if (!BF16 && row < rows && c == 0) {
        B.y_norm[h * A.T + t] = dd;
        if (h % A.G == 0) B.v_norm[h / A.G * A.T + t] = vv;
    }
    if (row < rows && c == 0) {
        B.delta[h * A.T + t] = sum;
        // a row that saw nothing has weights 0
        const float l = A.lse[row];
        B.lse2[h * A.T + t] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f - (BF16 ? 0.f : kPLog2);
    }
}

// Rows [from, 128) of a tile in shared memory cleared, by a warp: they belong to another
// sequence, and 0 * NaN is NaN.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int from) {
    for (int x = threadIdx.x & 31; x < (kTile - from) * (D / 8); x += 32)
        *reinterpret_cast<uint4 *>(tile + (x % (D / 8)) / 8 * Lay<D>::kBlock + (from + x / (D / 8)) * 128 + (x % 8) * 16) =
            make_uint4(0, 0, 0, 0);
    sm100::fence_proxy_async_smem();
    __syncwarp();
}

template <int D>
__device__ __forceinline__ void load_tile(uint8_t *to, const CUtensorMap *map, uint64_t *bar, int head, int64_t row) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_load_4d(to + b * Lay<D>::kBlock, map, bar, b * 64, head, (int)row, 0);
}

// D[128, d] += A B: A [128, 128] 16-bit in tensor memory (its halves of 64 columns at a_tmem and
// a_tmem + 64), B a tile of 128 rows.
template <int D, bool BF16>
__device__ __forceinline__ void mma_sum(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_saddr, bool more) {
#pragma unroll
    for (int s = 0; s < 8; ++s)
        mma16_ts(d_tmem, a_tmem + (s >> 2) * 64 + (s & 3) * 8, sdesc_mn(b_saddr + s * 2048, Lay<D>::kBlock),
                 idesc_16(BF16, 128, D, true), more || s > 0);
}

// dP - delta; fp16: times the scale in `by`, which `minus` has already.
template <bool BF16>
__device__ __forceinline__ uint64_t less_delta(uint64_t dp, uint64_t by, uint64_t minus) {
    return BF16 ? add2(dp, minus) : fma2(dp, by, minus);
}

// fp16: the largest norms, by the 256 threads of the compute warps.  An infinity or NaN counts for nothing: it reaches
// what it reaches without a scale.
__device__ __forceinline__ void look(const float *x, int n, float &most) {
    for (int i = threadIdx.x; i < n; i += 8 * 256) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = i + e * 256 < n ? x[i + e * 256] : 0.f;   // in flight together
#pragma unroll
        for (int e = 0; e < 8; ++e) most = fmaxf(most, v[e] < INFINITY ? v[e] : 0.f);
    }
}
__device__ __forceinline__ void leave(float most, float *place) {
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if ((threadIdx.x & 31) == 0) place[threadIdx.x >> 5] = most;
}
__device__ __forceinline__ float largest(const float *place) {
    float most = place[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) most = fmaxf(most, place[i]);
    return most;
}

// 64 fp32 columns of the thread's row.
__device__ __forceinline__ void load64(uint32_t at, float (&x)[64]) {
    tmem_ld32_nowait(at, x);
    tmem_ld32_nowait(at + 32, x + 32);
    tmem_wait_ld(x);
}
// 64 columns as 16-bit pairs into the 32 columns at `at`.
template <bool BF16>
__device__ __forceinline__ void store64(uint32_t at, const float (&x)[64]) {
    uint32_t p[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) p[i] = pack16<BF16>(x[2 * i], x[2 * i + 1]);
    tmem_st16_raw(at, p);
    tmem_st16_raw(at + 16, p + 16);
    sm100::tmem_wait_st();
    sm100::tc_fence_before();
}

// What that rounding leaves, into the 32 columns behind (store64 follows and waits).
template <bool BF16>
__device__ __forceinline__ void store64_rest(uint32_t at, const float (&x)[64]) {
    uint32_t p[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float a, b;
        unpack16<BF16>(pack16<BF16>(x[2 * i], x[2 * i + 1]), a, b);
        p[i] = pack16<BF16>(x[2 * i] - a, x[2 * i + 1] - b);
    }
    tmem_st16_raw(at + 32, p);
    tmem_st16_raw(at + 48, p + 16);
}

// A result row: COLS channels of tensor memory, scaled, to `at` elements into `to`.
template <int COLS, bool BF16>
__device__ __forceinline__ void write_row(void *to, bool f32, int64_t at, uint32_t tmem, float scale, bool live) {
#pragma unroll 1
    for (int x = 0; x < COLS; x += 32) {
        float v[32];
        tmem_ld32_nowait(tmem + x, v);
        tmem_wait_ld(v);
#pragma unroll
        for (int y = 0; y < 32; ++y) v[y] *= scale;
        if (live)
#pragma unroll
            for (int y = 0; y < 32; y += 8) store8<BF16>(to, f32, at + x + y, v + y);
    }
}

template <int D, bool BF16>
__device__ void key_block(const CUtensorMap *qm, const CUtensorMap *km, const CUtensorMap *vm, const CUtensorMap *om,
                          const Attn &A, const Grads &B, Control &ct, const AttnPart &part, uint8_t *base, const AttnSeq &sq, uint32_t tmem, int warp) {
    using L = Lay<D>;
    constexpr int NA = L::kA, NB = L::kB;
    const int lane = threadIdx.x & 31;
    uint8_t *Ks = base, *Vs = base + L::kBytes, *ra = base + 2 * L::kBytes, *rb = ra + NA * L::kBytes;   // queries, dO
    const int kt = part.tile, hk = part.head, G = A.G;
    const int len = (int)(sq.b - sq.a), tiles = (len + kTile - 1) / kTile;
    const int per = tiles - kt, n = per * G;   // step j: head j / per of the group, query tile kt + j % per
    const int tail = len - (tiles - 1) * kTile;   // rows of the last tile
    const bool rest = tiles == 1;                 // (see the top)
    constexpr uint32_t S = 0, DP = 128, DV = 256, DK = 256 + D;
    bool ok = true;
    auto wait = [&](uint64_t *bar, int phase) { return attn_wait(bar, phase & 1, &g_attn_bwd_status); };

    if (warp == kLoadWarp) {
        if (lane == 0) {
            sm100::mbar_arrive_expect_tx(&ct.own_full, 2 * L::kBytes);
            load_tile<D>(Ks, km, &ct.own_full, hk, sq.a + kt * kTile);
            load_tile<D>(Vs, vm, &ct.own_full, hk, sq.a + kt * kTile);
        }
        __syncwarp();
        int a = 0, b = 0;   // tiles issued
        for (int j = 0; j < n; ++j) {
            const int sa = j % NA, sb = j % NB, h = hk * G + j / per;
            const int64_t row = sq.a + (int64_t)(kt + j % per) * kTile;
            if (j >= NA) ok = wait(&ct.a_empty[sa], j / NA - 1);
            if (!ok) break;
            if (lane == 0) {
                sm100::mbar_arrive_expect_tx(&ct.a_full[sa], L::kBytes);
                load_tile<D>(ra + sa * L::kBytes, qm, &ct.a_full[sa], h, row);
            }
            __syncwarp();
            ++a;
            if (j >= NB) ok = wait(&ct.b_empty[sb], j / NB - 1);
            if (!ok) break;
            if (lane == 0) {
                sm100::mbar_arrive_expect_tx(&ct.b_full[sb], L::kBytes);
                load_tile<D>(rb + sb * L::kBytes, om, &ct.b_full[sb], h, row);
            }
            __syncwarp();
            ++b;
        }
        // no copy may land after the block's end
        attn_wait(&ct.own_full, 0, &g_attn_bwd_status);
        for (int j = max(0, a - NA); j < a; ++j) wait(&ct.a_full[j % NA], j / NA);
        for (int j = max(0, b - NB); j < b; ++j) wait(&ct.b_full[j % NB], j / NB);
    } else if (warp == kStatWarp) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernel in front writes delta and lse2
        float by = 1.f;   // what dP - delta is multiplied by: P comes times kPScale
        if (!BF16) {
            sm100::named_sync(1, 288);   // the compute warps have looked
            by = range_scale(largest(ct.most[0]), largest(ct.most[1])) / kPScale;
        }
        for (int j = 0; j < n; ++j) {
            const int st = j % kStats;
            const int64_t h = hk * G + j / per, at = h * A.T + sq.a, row = (int64_t)(kt + j % per) * kTile + lane * 4;
            float x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = row + i < len ? B.lse2[at + row + i] : INFINITY;
                y[i] = row + i < len ? B.delta[at + row + i] * by : 0.f;
            }
            if (j >= kStats) ok = wait(&ct.stat_empty[st], j / kStats - 1);
            if (!ok) break;
            *reinterpret_cast<float4 *>(&ct.stat[st][0][lane * 4]) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(&ct.stat[st][1][lane * 4]) = make_float4(y[0], y[1], y[2], y[3]);
            sm100::mbar_arrive(&ct.stat_full[st]);
        }
    } else if (warp == kProductWarp) {
        const uint32_t k_at = sm100::smem_u32(Ks), v_at = sm100::smem_u32(Vs), a_at = sm100::smem_u32(ra), b_at = sm100::smem_u32(rb);
        // the tiles of step j, their rows behind the sequence cleared
        auto arrived_a = [&](int j) {
            if (!wait(&ct.a_full[j % NA], j / NA)) return false;
            if (tail < kTile && j % per == per - 1) clear_rows<D>(ra + (j % NA) * L::kBytes, tail);
            return true;
        };
        auto arrived_b = [&](int j) {
            if (!wait(&ct.b_full[j % NB], j / NB)) return false;
            if (tail < kTile && j % per == per - 1) clear_rows<D>(rb + (j % NB) * L::kBytes, tail);
            return true;
        };
        auto scores = [&](int j) {
            sm100::tc_fence_after();
            mma_rows<D, BF16, 128>(tmem + S, k_at, a_at + (j % NA) * L::kBytes, L::kBlock, L::kBlock);
            sm100::mma_commit_el(&ct.s_full[0]);
        };
        auto dscores = [&](int j) {
            sm100::tc_fence_after();
            mma_rows<D, BF16, 128>(tmem + DP, v_at, b_at + (j % NB) * L::kBytes, L::kBlock, L::kBlock);
            sm100::mma_commit_el(&ct.dp_full);
        };
        ok = wait(&ct.own_full, 0) && arrived_a(0);
        if (ok) {
            scores(0);
            ok = arrived_b(0);
            if (ok) dscores(0);
        }
        for (int j = 0; j < n && ok; ++j) {
            ok = wait(&ct.p_ready, j);
            if (!ok) break;
            sm100::tc_fence_after();
            mma_sum<D, BF16>(tmem + DV, tmem + S, b_at + (j % NB) * L::kBytes, j > 0);
            if (rest) mma_sum<D, BF16>(tmem + DV, tmem + S + 32, b_at + (j % NB) * L::kBytes, true);
            sm100::mma_commit_el(&ct.b_empty[j % NB]);
            if (j + 1 < n) {
                ok = arrived_a(j + 1);
                if (!ok) break;
                scores(j + 1);
            }
            ok = wait(&ct.ds_ready[0], j);
            if (!ok) break;
            sm100::tc_fence_after();
            mma_sum<D, BF16>(tmem + DK, tmem + DP, a_at + (j % NA) * L::kBytes, j > 0);
            if (rest) mma_sum<D, BF16>(tmem + DK, tmem + DP + 32, a_at + (j % NA) * L::kBytes, true);
            sm100::mma_commit_el(&ct.a_empty[j % NA]);
            if (j + 1 < n) {
                ok = arrived_b(j + 1);
                if (!ok) break;
                dscores(j + 1);
            }
        }
        sm100::mma_commit_el(&ct.done);
        attn_wait(&ct.done, 0, &g_attn_bwd_status);
    } else {
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float c = A.scale_log2;
        float scale = 1.f;
        if (!BF16) {
            asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernel in front writes the norms
            float y = 0.f, v = 0.f;
            for (int g = 0; g < G; ++g) look(B.y_norm + (int64_t)(hk * G + g) * A.T + sq.a + kt * kTile, len - kt * kTile, y);
            look(B.v_norm + (int64_t)hk * A.T + sq.a, len, v);
            leave(y, ct.most[0]);
            leave(v, ct.most[1]);
            sm100::named_sync(1, 288);
            scale = range_scale(largest(ct.most[0]), largest(ct.most[1]));
        }
        const uint64_t by = pack2(scale / kPScale, scale / kPScale);
        for (int j = 0; j < n; ++j) {
            const int st = j % kStats, qt = kt + j % per;
            ok = wait(&ct.stat_full[st], j / kStats) && wait(&ct.s_full[0], j);
            if (!ok) break;
            sm100::tc_fence_after();
            float p[64];
            load64(lanes + S + half * 64, p);
            const float4 *l4 = reinterpret_cast<const float4 *>(&ct.stat[st][0][half * 64]);
            const uint64_t c2 = pack2(c, c);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const float4 l = l4[x];
                unpack2(fma2(pack2(p[4 * x], p[4 * x + 1]), c2, pack2(-l.x, -l.y)), p[4 * x], p[4 * x + 1]);
                unpack2(fma2(pack2(p[4 * x + 2], p[4 * x + 3]), c2, pack2(-l.z, -l.w)), p[4 * x + 2], p[4 * x + 3]);
#pragma unroll
                for (int y = 0; y < 4; ++y) p[4 * x + y] = ex2(p[4 * x + y]);
            }
            // query column x of this half: seen from key row r, and a token of the sequence
            const bool masked = qt == kt || (tail < kTile && qt == tiles - 1);
            const int lo = qt == kt ? r - half * 64 : 0, hi = len - qt * kTile - half * 64;
            if (masked) {
#pragma unroll
                for (int x = 0; x < 64; ++x) p[x] = x >= lo && x < hi ? p[x] : 0.f;
            }
            if (rest) store64_rest<BF16>(lanes + S + half * 64, p);
            store64<BF16>(lanes + S + half * 64, p);
            sm100::mbar_arrive(&ct.p_ready);
            ok = wait(&ct.dp_full, j);
            if (!ok) break;
            sm100::tc_fence_after();
            float dp[64];
            load64(lanes + DP + half * 64, dp);
            const float4 *d4 = reinterpret_cast<const float4 *>(&ct.stat[st][1][half * 64]);
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const float4 d = d4[x];
                unpack2(mul2(pack2(p[4 * x], p[4 * x + 1]),
                             less_delta<BF16>(pack2(dp[4 * x], dp[4 * x + 1]), by, pack2(-d.x, -d.y))),
                        dp[4 * x], dp[4 * x + 1]);
                unpack2(mul2(pack2(p[4 * x + 2], p[4 * x + 3]),
                             less_delta<BF16>(pack2(dp[4 * x + 2], dp[4 * x + 3]), by, pack2(-d.z, -d.w))),
                        dp[4 * x + 2], dp[4 * x + 3]);
            }
            if (masked) {
#pragma unroll
                for (int x = 0; x < 64; ++x) dp[x] = x >= lo && x < hi ? dp[x] : 0.f;
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(&ct.stat_empty[st]);
            if (rest) store64_rest<BF16>(lanes + DP + half * 64, dp);
            store64<BF16>(lanes + DP + half * 64, dp);
            sm100::mbar_arrive(&ct.ds_ready[0]);
        }
        ok = ok && wait(&ct.done, 0);
        if (ok) {
            sm100::tc_fence_after();
            const int64_t at = ((sq.a + kt * kTile + r) * A.Hkv + hk) * D;
            const bool live = kt * kTile + r < len, f32 = A.out_dtype == KDA_DTYPE_F32;
            if (half == 0)
                write_row<D, BF16>(B.dv, f32, at, lanes + DV, BF16 ? 1.f : 1.f / kPScale, live);
            else
                write_row<D, BF16>(B.dk, f32, at, lanes + DK, A.scale / scale, live);
        }
        sm100::tc_fence_before();
    }
}

template <int D, bool BF16>
__device__ void query_block(const CUtensorMap *qm, const CUtensorMap *km, const CUtensorMap *vm, const CUtensorMap *om,
                            const Attn &A, const Grads &B, Control &ct, const AttnPart &part, uint8_t *base, const AttnSeq &sq, uint32_t tmem, int warp) {
    using L = Lay<D>;
    constexpr int NA = L::kA, NB = L::kB;
    const int lane = threadIdx.x & 31;
    uint8_t *Qs = base, *Os = base + L::kBytes, *ra = base + 2 * L::kBytes, *rb = ra + NA * L::kBytes;   // keys, values
    const int qt = part.tile, h = part.head, hk = h / A.G;
    const int len = (int)(sq.b - sq.a), n = qt + 1;
    const int tail = len - qt * kTile;   // rows of the last key tile (the diagonal one), if below 128
    const bool rest = len <= kTile;      // (see the top)
    constexpr uint32_t S[2] = {0, 128}, DP = 256, DQ = 384;
    bool ok = true;
    auto wait = [&](uint64_t *bar, int phase) { return attn_wait(bar, phase & 1, &g_attn_bwd_status); };

    if (warp == kLoadWarp) {
        if (lane == 0) {
            sm100::mbar_arrive_expect_tx(&ct.own_full, 2 * L::kBytes);
            load_tile<D>(Qs, qm, &ct.own_full, h, sq.a + (int64_t)qt * kTile);
            load_tile<D>(Os, om, &ct.own_full, h, sq.a + (int64_t)qt * kTile);
        }
        __syncwarp();
        int a = 0, b = 0;
        for (int j = 0; j < n; ++j) {
            const int sa = j % NA, sb = j % NB;
            const int64_t row = sq.a + (int64_t)j * kTile;
            if (j >= NA) ok = wait(&ct.a_empty[sa], j / NA - 1);
            if (!ok) break;
            if (lane == 0) {
                sm100::mbar_arrive_expect_tx(&ct.a_full[sa], L::kBytes);
                load_tile<D>(ra + sa * L::kBytes, km, &ct.a_full[sa], hk, row);
            }
            __syncwarp();
            ++a;
            if (j >= NB) ok = wait(&ct.b_empty[sb], j / NB - 1);
            if (!ok) break;
            if (lane == 0) {
                sm100::mbar_arrive_expect_tx(&ct.b_full[sb], L::kBytes);
                load_tile<D>(rb + sb * L::kBytes, vm, &ct.b_full[sb], hk, row);
            }
            __syncwarp();
            ++b;
        }
        attn_wait(&ct.own_full, 0, &g_attn_bwd_status);
        for (int j = max(0, a - NA); j < a; ++j) wait(&ct.a_full[j % NA], j / NA);
        for (int j = max(0, b - NB); j < b; ++j) wait(&ct.b_full[j % NB], j / NB);
    } else if (warp == kProductWarp) {
        const uint32_t q_at = sm100::smem_u32(Qs), o_at = sm100::smem_u32(Os), a_at = sm100::smem_u32(ra), b_at = sm100::smem_u32(rb);
        auto scores = [&](int j) {
            if (!wait(&ct.a_full[j % NA], j / NA)) return false;
            if (j == n - 1 && tail < kTile) clear_rows<D>(ra + (j % NA) * L::kBytes, tail);
            sm100::tc_fence_after();
            mma_rows<D, BF16, 128>(tmem + S[j & 1], q_at, a_at + (j % NA) * L::kBytes, L::kBlock, L::kBlock);
            sm100::mma_commit_el(&ct.s_full[j & 1]);
            return true;
        };
        auto dscores = [&](int j) {
            if (!wait(&ct.b_full[j % NB], j / NB)) return false;
            sm100::tc_fence_after();
            mma_rows<D, BF16, 128>(tmem + DP, o_at, b_at + (j % NB) * L::kBytes, L::kBlock, L::kBlock);
            sm100::mma_commit_el(&ct.dp_full);
            sm100::mma_commit_el(&ct.b_empty[j % NB]);
            return true;
        };
        ok = wait(&ct.own_full, 0) && scores(0) && dscores(0);
        for (int j = 0; j < n && ok; ++j) {
            if (j + 1 < n) {
                ok = scores(j + 1) && wait(&ct.dp_free, j) && dscores(j + 1);
                if (!ok) break;
            }
            // (two barriers in turn: the compute warps may be through step j + 1, whose scores are
            // there already, before this wait is reached, but not through j + 2)
            ok = wait(&ct.ds_ready[j & 1], j >> 1);
            if (!ok) break;
            sm100::tc_fence_after();
            mma_sum<D, BF16>(tmem + DQ, tmem + S[j & 1], a_at + (j % NA) * L::kBytes, j > 0);
            if (rest) mma_sum<D, BF16>(tmem + DQ, tmem + S[j & 1] + 32, a_at + (j % NA) * L::kBytes, true);
            sm100::mma_commit_el(&ct.a_empty[j % NA]);
        }
        sm100::mma_commit_el(&ct.done);
        attn_wait(&ct.done, 0, &g_attn_bwd_status);
    } else if (warp < 8) {
        const int half = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool live = qt * kTile + r < len;
        const int64_t at = (int64_t)h * A.T + sq.a + qt * kTile + r;
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the kernel in front writes delta and lse2
        const float lse2 = live ? B.lse2[at] : INFINITY, delta = live ? B.delta[at] : 0.f;
        float scale = 1.f, by = 1.f;
        if (!BF16) {
            float v = 0.f;
            look(B.v_norm + (int64_t)hk * A.T + sq.a, min(len, n * kTile), v);
            leave(v, ct.most[1]);
            sm100::named_sync(1, 256);
            if (live) scale = range_scale(B.y_norm[at], largest(ct.most[1]));
            by = scale / kPScale;
        }
        const float c = A.scale_log2;
        const uint64_t c2 = pack2(c, c), l2 = pack2(-lse2, -lse2), d2 = pack2(-delta * by, -delta * by), by2 = pack2(by, by);
        for (int j = 0; j < n; ++j) {
            ok = wait(&ct.s_full[j & 1], j >> 1);
            if (!ok) break;
            sm100::tc_fence_after();
            float p[64];
            load64(lanes + S[j & 1] + half * 64, p);
#pragma unroll
            for (int x = 0; x < 64; x += 2) {
                float a, b;
                unpack2(fma2(pack2(p[x], p[x + 1]), c2, l2), a, b);
                p[x] = ex2(a);
                p[x + 1] = ex2(b);
            }
            ok = wait(&ct.dp_full, j);
            if (!ok) break;
            sm100::tc_fence_after();
            float dp[64];
            load64(lanes + DP + half * 64, dp);
            sm100::tc_fence_before();
            sm100::mbar_arrive(&ct.dp_free);
#pragma unroll
            for (int x = 0; x < 64; x += 2)
                unpack2(mul2(pack2(p[x], p[x + 1]), less_delta<BF16>(pack2(dp[x], dp[x + 1]), by2, d2)), dp[x], dp[x + 1]);
            if (j == n - 1) {
#pragma unroll
                for (int x = 0; x < 64; ++x) dp[x] = x + half * 64 <= r ? dp[x] : 0.f;
            }
            if (rest) store64_rest<BF16>(lanes + S[j & 1] + half * 64, dp);
            store64<BF16>(lanes + S[j & 1] + half * 64, dp);
            sm100::mbar_arrive(&ct.ds_ready[j & 1]);
        }
        ok = ok && wait(&ct.done, 0);
        if (ok) {
            sm100::tc_fence_after();
            write_row<D / 2, BF16>(B.dq, A.out_dtype == KDA_DTYPE_F32,
                                   ((sq.a + qt * kTile + r) * A.Hq + h) * D + half * (D / 2), lanes + DQ + half * (D / 2),
                                   A.scale / scale, live);
        }
        sm100::tc_fence_before();
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
kda_attn_backward_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap km,
                         const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap om, const Attn A,
                         const Grads B) {
    // the tiles, and behind them what the warps tell each other (there is no room for both and a gap)
    extern __shared__ __align__(1024) uint8_t base[];
    Control &ct = *reinterpret_cast<Control *>(base + Lay<D>::kTiles);
    if (sm100::smem_u32(base) & 1023) {   // the swizzled tiles need it
        if (threadIdx.x == 0) atomicOr(&g_attn_bwd_status, kAttnTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = attn_warp();
    const bool keys = blockIdx.x < B.key_blocks;
    if (tid == 0) {
        sm100::prefetch_tmap(&qm);
        sm100::prefetch_tmap(&km);
        sm100::prefetch_tmap(&vm);
        sm100::prefetch_tmap(&om);
        sm100::mbar_init(&ct.own_full, 1);
        for (int i = 0; i < 4; ++i) {
            sm100::mbar_init(&ct.a_full[i], 1);
            sm100::mbar_init(&ct.a_empty[i], 1);
            sm100::mbar_init(&ct.b_full[i], 1);
            sm100::mbar_init(&ct.b_empty[i], 1);
        }
        for (int i = 0; i < kStats; ++i) {
            sm100::mbar_init(&ct.stat_full[i], 32);
            sm100::mbar_init(&ct.stat_empty[i], 8);
        }
        sm100::mbar_init(&ct.s_full[0], 1);
        sm100::mbar_init(&ct.s_full[1], 1);
        sm100::mbar_init(&ct.dp_full, 1);
        sm100::mbar_init(&ct.done, 1);
        sm100::mbar_init(&ct.p_ready, 256);
        sm100::mbar_init(&ct.dp_free, 256);
        sm100::mbar_init(&ct.ds_ready[0], 256);
        sm100::mbar_init(&ct.ds_ready[1], 256);
        sm100::fence_mbar_init();
    }
    auto tiles = [&](int n) {
        const AttnSeq s = attn_seq<false>(A, n);
        return (s.b - s.a + kTile - 1) / kTile;
    };
    // the first key tiles are seen by the most queries, the last query tiles see the most keys:
    // those start first
    const int same = A.cu ? -1 : (int)((A.seq_len + kTile - 1) / kTile);
    AttnPart part;
    const bool some = attn_whole_part<kThreads>(A.N, keys ? A.Hkv : A.Hq, blockIdx.x - (keys ? 0u : (uint32_t)B.key_blocks),
                                                !keys, same, tiles, part, &ct.part, ct.scan);
    if (!some) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // no kernel ends before the one in front of it
        return;
    }
    const AttnSeq sq = attn_seq<false>(A, part.n);
    if (warp == kProductWarp) {
        sm100::tmem_alloc(&ct.tmem, 512);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = ct.tmem;
    if (keys)
        key_block<D, BF16>(&qm, &km, &vm, &om, A, B, ct, part, base, sq, tmem, warp);
    else
        query_block<D, BF16>(&qm, &km, &vm, &om, A, B, ct, part, base, sq, tmem, warp);
    __syncthreads();
    if (warp == kProductWarp) sm100::tmem_dealloc(tmem, 512);
}

template <int D, bool BF16>
cudaError_t backward(const Attn &A, Grads &B, cudaStream_t stream) {
    CUtensorMap qm, km, vm, om;
    if (!kda_make_attn_map(&qm, A.q, BF16, D, A.Hq, A.T, 1, A.q_h, A.q_t, 0, kTile) ||
        !kda_make_attn_map(&km, A.k, BF16, D, A.Hkv, A.T, 1, A.k_h, A.k_t, 0, kTile) ||
        !kda_make_attn_map(&vm, A.v, BF16, D, A.Hkv, A.T, 1, A.v_h, A.v_t, 0, kTile) ||
        !kda_make_attn_map(&om, B.d_out, BF16, D, A.Hq, A.T, 1, B.do_h, B.do_t, 0, kTile))
        return cudaErrorInvalidValue;
    const auto kernel = kda_attn_backward_kernel<D, BF16>;
    constexpr int smem = Lay<D>::kTiles + (int)sizeof(Control);
    static_assert(smem <= 232448, "shared memory of a block");
    cudaError_t e = kda_allow_smem<kda_attn_backward_kernel<D, BF16>>(smem);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)A.T * A.Hq;
    kda_attn_delta_kernel<D, BF16><<<(unsigned)((rows * (D / 8) + 255) / 256), 256, 0, stream>>>(A, B);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t tiles = A.cu ? (int64_t)A.T / kTile + A.N : (A.seq_len + kTile - 1) / kTile * A.N;
    B.key_blocks = tiles * A.Hkv;
    // The gradients' kernel may start once every block of delta's has started or ended (with many that is near
    // its end); what it reads but delta's results was there before that one started, and its results are
    // written after it has waited.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(B.key_blocks + tiles * A.Hq));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, qm, km, vm, om, A, B);
}

}  // namespace

int64_t kda_attn_backward_ws(const Attn &A) {
    const int64_t rows = (int64_t)A.T * A.Hq;
    return A.in_dtype == KDA_DTYPE_BF16 ? rows * 8 : rows * 12 + (int64_t)A.T * A.Hkv * 4;
}

cudaError_t kda_launch_attn_backward(const Attn &A, const AttnGrads &X, float *workspace, cudaStream_t stream) {
    Grads B{};
    B.out = X.out, B.o_t = X.o_t, B.o_h = X.o_h;
    B.d_out = X.d_out, B.do_t = X.do_t, B.do_h = X.do_h;
    B.dq = X.dq, B.dk = X.dk, B.dv = X.dv;
    B.delta = workspace;
    B.lse2 = workspace + (int64_t)A.T * A.Hq;
    B.y_norm = B.lse2 + (int64_t)A.T * A.Hq;
    B.v_norm = B.y_norm + (int64_t)A.T * A.Hq;
    const bool b = A.in_dtype == KDA_DTYPE_BF16;
    if (A.d == 128) return b ? backward<128, true>(A, B, stream) : backward<128, false>(A, B, stream);
    return b ? backward<64, true>(A, B, stream) : backward<64, false>(A, B, stream);
}

cudaError_t kda_attn_bwd_read_status(unsigned *status) {
    unsigned w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_attn_bwd_status, sizeof(w));
    if (e == cudaSuccess && w) {
        *status |= w;
        w = 0;
        e = cudaMemcpyToSymbol(g_attn_bwd_status, &w, sizeof(w));
    }
    return e;
}
