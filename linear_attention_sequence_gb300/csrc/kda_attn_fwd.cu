// kda_attn_fwd.cu -- causal softmax attention on the tensor cores (sm_103a): whole prompts
// of a packed batch (kda_attn_prefill) and chunks of new tokens over a paged cache
// (kda_attn_paged, sequences of more than kAttnFewRows query rows).
//
// A block takes 256 query rows of one key head.  A row is a (token, query head of the
// group) pair, token major, so that a group of any size fills the tiles and few tokens of a
// large group still make one.  The rows are two tiles of 128; keys and values pass
// through a ring of 128-key tiles in shared memory (TMA, 128-byte swizzle).  For each key
// tile and row tile
//
//   S = Q K^T               tcgen05, fp32 in tensor memory
//   P = 2^(c S - c m)       one thread a row: its 128 scores in registers, c = scale log2 e
//   O += P V                tcgen05, P 16 bits in tensor memory over the columns of S
//
// While one tile's softmax runs, the tensor cores work on the other's products.  m is the
// running maximum of the row.  O and the running sum are rescaled only when the maximum
// has grown by more than 2^8 (of the 16-bit types' range P then uses no more than it has,
// and the fp32 sums nothing): after the first tiles hardly ever, and it is the softmax threads
// themselves that do it, between the products.  P is rounded to 16 bits because the tensor
// cores read it so (half a step of P's own value); sums, maxima and O are fp32.
//
// Keys that a row may not see get the score -inf by a select, and value rows behind a
// sequence's last key are cleared in shared memory before the product (0 * NaN is NaN).
#include <mutex>

#include "kda_attn_plan.cuh"

using namespace kda;

namespace {

__device__ unsigned g_attn_status;

constexpr int kThreads = 320;      // two softmax warpgroups, the product warp, the load warp
constexpr int kProductWarp = 8, kLoadWarp = 9;
constexpr int kTileRows = 256;
constexpr float kGrowth = 8.f;     // log2 of the growth of a maximum that O is rescaled for

template <int D>
struct Lay {
    static constexpr int kTileBytes = kAttnKeys * D * 2;              // a tile of keys, values, or 128 queries
    static constexpr int kBlockBytes = kAttnKeys * 128;               // 64 channels of it
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kSmem = 1024 + (2 + kStages) * kTileBytes + 1024;
};

struct Control {
    uint64_t q_full, full[8], empty[8], s_full[2], p_ready[2], o_full[2], done;
    uint32_t tmem;
    AttnPart part;
    int64_t scan[kThreads / 32];
};

// Where the shares of split row tiles go, and what the joining kernel needs to know of them.
struct Shares {
    int32_t *count;   // [1] shares in all
    int32_t *rec;     // [slots][8]: n, tile, head, split, splits
    float *lse;       // [slots][rows]
    float *out;       // [slots][rows][d]
};

template <int D, bool BF16, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
kda_attn_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Attn A,
                   const Shares sh, const int box, const int few) {
    using L = Lay<D>;
    constexpr int NST = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *Qs = base, *ring = base + 2 * L::kTileBytes;
    __shared__ Control ct;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = A.G;

    if (tid == 0) {
        sm100::mbar_init(&ct.q_full, 256);
        for (int i = 0; i < NST; ++i) {
            sm100::mbar_init(&ct.full[i], 1);
            sm100::mbar_init(&ct.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&ct.s_full[i], 1);
            sm100::mbar_init(&ct.p_ready[i], 128);
            sm100::mbar_init(&ct.o_full[i], 1);
        }
        sm100::mbar_init(&ct.done, 1);
        sm100::fence_mbar_init();
    }
    // which part
    bool some;
    if (PAGED) {
        auto need = [&](int n) {
            const AttnSeq s = attn_seq<true>(A, n);
            const int64_t rows = (s.b - s.a) * G;
            return AttnNeed{rows > few ? (int32_t)((rows + kTileRows - 1) / kTileRows) : 0,
                            (int32_t)((s.keys + kAttnKeys - 1) / kAttnKeys)};
        };
        int64_t slots;
        some = attn_split_part<kThreads>(A.N, A.Hkv, blockIdx.x, 152, 3, 4, need, &ct.part, ct.scan, &slots);
        if (blockIdx.x == 0 && tid == 0) *sh.count = (int32_t)slots;
    } else {
        auto tiles = [&](int n) {
            const AttnSeq s = attn_seq<false>(A, n);
            return ((s.b - s.a) * G + kTileRows - 1) / kTileRows;
        };
        some = attn_whole_part<kThreads>(A.N, A.Hkv, blockIdx.x, true, tiles, &ct.part, ct.scan);
    }
    if (!some) return;
    const AttnPart part = ct.part;
    const AttnSeq sq = attn_seq<PAGED>(A, part.n);
    const int32_t tokens = (int32_t)(sq.b - sq.a), rows = tokens * G - part.tile * kTileRows;   // rows from this tile on
    const int32_t behind = (int32_t)sq.keys - tokens;   // key index that the first token sees last
    // of each row tile, the key tiles [j0, j0 + n[i]) that some row of it sees
    int32_t n_of[2], n = 0;
    const int32_t j0 = PAGED ? part.j0 : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int32_t last = min(rows, (i + 1) * 128) - 1;   // last row of the tile
        int32_t seen = 0;
        if (last >= i * 128) seen = behind + (part.tile * kTileRows + last) / G + 1;
        seen = max(0, min(seen, (int32_t)sq.keys));
        int32_t tiles = (seen + kAttnKeys - 1) / kAttnKeys;
        if (PAGED) tiles = min(tiles, part.j1);
        n_of[i] = max(0, tiles - j0);
        n = max(n, n_of[i]);
    }
    if (warp == kProductWarp) {
        sm100::tmem_alloc(&ct.tmem, 512);
        sm100::tmem_relinquish();
    }
    sm100::tc_fence_before();
    __syncthreads();
    sm100::tc_fence_after();
    const uint32_t tmem = ct.tmem;
    bool ok = true;
    int issued = 0;   // tiles asked for by the load warp

    if (warp == kLoadWarp) {
        // ------------------------------------------------ keys and values
        const int boxes = kAttnKeys / box;             // boxes of 64 channels that make a block
        const int mine = lane / boxes, which = lane % boxes;
        const bool issues = lane < boxes * (D / 64);
        const int loads = 2 * n;
        const int32_t *row = PAGED ? A.table + (int64_t)part.n * A.wide : nullptr;
        bool bad = false;
        for (int c = 0; c < loads && ok; ++c) {
            // order: K0, K1, V0, K2, V1, ...
            const bool values = c == loads - 1 || (c > 0 && (c & 1) == 0);
            const int j = j0 + (values ? (c == loads - 1 ? n - 1 : c / 2 - 1) : (c + 1) / 2);
            int page = 0, at;
            if (PAGED) {
                const int64_t first = (int64_t)j * kAttnKeys + which * box;
                page = A.P;   // past the cache: reads zeros
                at = (int)(first % A.page);
                if (issues && first < sq.keys) {
                    const int p = row[first / A.page];
                    if (p >= 0 && p < A.P) page = p; else bad = true;
                }
            } else {
                at = (int)(sq.a + (int64_t)j * kAttnKeys);
            }
            const int st = c % NST;
            if (c >= NST) ok = attn_wait(&ct.empty[st], (c / NST - 1) & 1, &g_attn_status);
            if (!ok) break;
            uint8_t *to = ring + st * L::kTileBytes;
            if (lane == 0) sm100::mbar_arrive_expect_tx(&ct.full[st], L::kTileBytes);
            __syncwarp();
            if (issues)
                tma_load_4d(to + mine * L::kBlockBytes + which * box * 128, values ? &vmap : &kmap, &ct.full[st],
                            mine * 64, part.head, at, page);
            ++issued;
        }
        if (bad) atomicOr(&g_attn_status, kCacheBadPage);
        __syncwarp();
    } else if (warp == kProductWarp) {
        // ------------------------------------------------ products
        const uint32_t q_at = sm100::smem_u32(Qs), ring_at = sm100::smem_u32(ring);
        constexpr uint32_t S[2] = {0, 128}, O[2] = {256, 256 + D};
        auto full = [&](int c) { return attn_wait(&ct.full[c % NST], (c / NST) & 1, &g_attn_status); };
        if (n > 0) {
            ok = attn_wait(&ct.q_full, 0, &g_attn_status) && full(0);
            if (ok) {
                sm100::tc_fence_after();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (n_of[i] == 0) continue;
                    mma_rows<D, BF16, 128>(tmem + S[i], q_at + i * L::kTileBytes, ring_at, L::kBlockBytes, L::kBlockBytes);
                    sm100::mma_commit_el(&ct.s_full[i]);
                }
                sm100::mma_commit_el(&ct.empty[0]);
            }
        }
        for (int j = 0; j < n && ok; ++j) {
            const bool more = j + 1 < n;
            const int ck = 2 * j + 1, cv = more ? 2 * j + 2 : 2 * j + 1;
            if (more) ok = full(ck);
            ok = ok && full(cv);
            if (!ok) break;
            const uint32_t k_at = ring_at + (ck % NST) * L::kTileBytes, v_at = ring_at + (cv % NST) * L::kTileBytes;
            const int32_t left = (int32_t)sq.keys - (j0 + j) * kAttnKeys;   // keys from this tile on
            if (left < kAttnKeys) {
                // value rows behind the last key hold anything
                uint8_t *v = ring + (cv % NST) * L::kTileBytes;
                for (int x = lane; x < (kAttnKeys - left) * (D / 8); x += 32)
                    *reinterpret_cast<uint4 *>(v + (x % (D / 64 * 8)) / 8 * L::kBlockBytes +
                                               (left + x / (D / 8)) * 128 + (x % 8) * 16) = make_uint4(0, 0, 0, 0);
                sm100::fence_proxy_async_smem();
                __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (j < n_of[i]) {
                    ok = ok && attn_wait(&ct.p_ready[i], j & 1, &g_attn_status);
                    if (!ok) break;
                    sm100::tc_fence_after();
#pragma unroll
                    for (int s = 0; s < kAttnKeys / 16; ++s)
                        mma16_ts(tmem + O[i], tmem + S[i] + s * 8, sdesc_mn(v_at + s * 2048, L::kBlockBytes),
                                 idesc_16(BF16, 128, D, true), j > 0 || s > 0);
                    if (j == n_of[i] - 1) sm100::mma_commit_el(&ct.o_full[i]);
                }
                if (j + 1 < n_of[i]) {
                    mma_rows<D, BF16, 128>(tmem + S[i], q_at + i * L::kTileBytes, k_at, L::kBlockBytes, L::kBlockBytes);
                    sm100::mma_commit_el(&ct.s_full[i]);
                }
            }
            sm100::mma_commit_el(&ct.empty[cv % NST]);
            if (more) sm100::mma_commit_el(&ct.empty[ck % NST]);
        }
        // whatever was issued is over before the block ends
        sm100::mma_commit_el(&ct.done);
        attn_wait(&ct.done, 0, &g_attn_status);
    } else {
        // ------------------------------------------------ softmax: one thread a row
        {
            const uint16_t *q = static_cast<const uint16_t *>(A.q);
            constexpr int CH = D / 8;   // 16-byte pieces of a row
            for (int x = tid; x < kTileRows * CH; x += 256) {
                const int r = x / CH, c = x % CH;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < rows) {
                    const int fr = part.tile * kTileRows + r, tok = fr / G;
                    v = __ldg(reinterpret_cast<const uint4 *>(q + (sq.a + tok) * A.q_t +
                                                              (int64_t)(part.head * G + fr - tok * G) * A.q_h + c * 8));
                }
                *reinterpret_cast<uint4 *>(Qs + (r >> 7) * L::kTileBytes + (c >> 3) * L::kBlockBytes + (r & 127) * 128 +
                                           (((c & 7) ^ (r & 7)) << 4)) = v;
            }
            sm100::fence_proxy_async_smem();
            sm100::mbar_arrive(&ct.q_full);
        }
        const int i = warp >> 2, r = tid;                    // row tile, row of the block
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t S = lanes + i * 128, O = lanes + 256 + i * D;
        const int fr = part.tile * kTileRows + r, tok = fr / G, g = fr - tok * G;
        const bool live = r < rows;
        const int32_t seen = live ? max(0, min(behind + tok + 1, (int32_t)sq.keys)) : 0;
        const float c = A.scale_log2;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < n_of[i]; ++j) {
            ok = attn_wait(&ct.s_full[i], j & 1, &g_attn_status);
            if (!ok) break;
            sm100::tc_fence_after();
            float s[128];
#pragma unroll
            for (int x = 0; x < 4; ++x) tmem_ld32_nowait(S + x * 32, s + x * 32);
            tmem_wait_ld(s);
            const int32_t vis = seen - (j0 + j) * kAttnKeys;
            if (__any_sync(0xffffffffu, vis < kAttnKeys)) {
#pragma unroll
                for (int x = 0; x < 128; ++x) s[x] = x < vis ? s[x] : -INFINITY;
            }
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int x = 4; x < 128; x += 4)
#pragma unroll
                for (int y = 0; y < 4; ++y) mx[y] = fmaxf(mx[y], s[x + y]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grown = top > m && (top - m) * c > kGrowth;   // also from -inf
            if (j > 0 && __any_sync(0xffffffffu, grown)) {
                // S of this tile is complete, and so, issued before it, is the product before
                const float f = grown ? ex2((m - top) * c) : 1.f;
                l *= f;
#pragma unroll 1
                for (int x = 0; x < D; x += 16) {
                    float o[16];
                    sm100::tmem_ld16(O + x, o);
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] *= f;
                    sm100::tmem_st16(O + x, o);
                }
                sm100::tmem_wait_st();
            }
            if (grown) m = top;
            const float shift = m == -INFINITY ? 0.f : -m * c;
            const uint64_t c2 = pack2(c, c), s2 = pack2(shift, shift);
            uint64_t sum[2] = {0, 0};
            uint32_t p[64];
#pragma unroll
            for (int x = 0; x < 64; ++x) {
                float a, b;
                unpack2(fma2(pack2(s[2 * x], s[2 * x + 1]), c2, s2), a, b);
                a = ex2(a);
                b = ex2(b);
                sum[x & 1] = add2(sum[x & 1], pack2(a, b));
                p[x] = pack16<BF16>(a, b);
                if ((x & 15) == 15) tmem_st16_raw(S + (x & ~15), p + (x & ~15));
            }
            float a, b;
            unpack2(add2(sum[0], sum[1]), a, b);
            l += a + b;
            sm100::tmem_wait_st();
            sm100::tc_fence_before();
            sm100::mbar_arrive(&ct.p_ready[i]);
        }
        if (n_of[i] > 0) {
            ok = ok && attn_wait(&ct.o_full[i], 0, &g_attn_status);
            sm100::tc_fence_after();
        }
        // ------------------------------------------------ results
        // With m still -inf the row has seen no key (or scores of -inf only): out 0.  A sum
        // that is NaN reaches the row through 1 / l.
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        const float lse = l > 0.f || l != l ? m * A.scale + logf(l) : -INFINITY;
        const bool share = PAGED && part.slot >= 0;
        const int64_t at = sq.a + tok;
        const int h = part.head * G + g;
        if (ok) {
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
                float o[32];
                if (n_of[i] > 0) {
                    tmem_ld32_nowait(O + x, o);
                    tmem_wait_ld(o);
                } else {
#pragma unroll
                    for (int y = 0; y < 32; ++y) o[y] = 0.f;
                }
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = inv == 0.f ? 0.f : o[y] * inv;
                if (!live) continue;
#pragma unroll
                for (int y = 0; y < 32; y += 8) {
                    if (share)
                        store8<BF16>(sh.out, true, ((int64_t)part.slot * kTileRows + r) * D + x + y, o + y);
                    else
                        store8<BF16>(A.out, A.out_dtype == KDA_DTYPE_F32, (at * A.Hq + h) * D + x + y, o + y);
                }
            }
            if (live) {
                if (share)
                    sh.lse[(int64_t)part.slot * kTileRows + r] = lse;
                else if (A.lse)
                    A.lse[at * A.Hq + h] = lse;
            }
        }
        if (PAGED && share && tid == 0) {
            int32_t *rec = sh.rec + (int64_t)part.slot * 8;
            rec[0] = part.n;
            rec[1] = part.tile;
            rec[2] = part.head;
            rec[3] = part.split;
            rec[4] = part.splits;
        }
        sm100::tc_fence_before();
    }
    if (warp == kLoadWarp) {
        // no copy may land after the block's end: the last ones of each stage
        for (int c = max(0, issued - NST); c < issued; ++c) attn_wait(&ct.full[c % NST], (c / NST) & 1, &g_attn_status);
    }
    __syncthreads();
    if (warp == kProductWarp) sm100::tmem_dealloc(tmem, 512);
}

// Joins the shares of split row tiles: out = sum_s w_s out_s with w_s = e^(lse_s - lse) in
// the order of the shares.  One warp a row, four channels a lane.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) kda_attn_join_kernel(const Attn A, const Shares sh, const int tile_rows) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int slot = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (slot >= *sh.count) return;
    const int32_t *rec = sh.rec + (int64_t)slot * 8;
    if (rec[3] != 0) return;
    const int n = rec[0], tile = rec[1], head = rec[2], splits = rec[4];
    int64_t a, b;
    seq_bounds(A.cu, n, A.T, A.seq_len, a, b);
    const int64_t rows = (b - a) * A.G - (int64_t)tile * tile_rows;
    for (int r = blockIdx.y * 4 + warp; r < tile_rows && r < rows; r += gridDim.y * 4) {
        const float *lse = sh.lse + (int64_t)slot * tile_rows + r;
        const float *out = sh.out + ((int64_t)slot * tile_rows + r) * D;
        float top = -INFINITY;
        for (int s = lane; s < splits; s += 32) top = fmaxf(top, lse[(int64_t)s * tile_rows]);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        for (int s = lane; s < splits; s += 32) sum += __expf(lse[(int64_t)s * tile_rows] - ref);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        constexpr int PER = D / 32;
        float acc[PER] = {};
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float w = __expf(lse[(int64_t)s * tile_rows] - ref);
            const float *o = out + (int64_t)s * tile_rows * D + lane * PER;
            float v[PER];
            if (PER == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(o);
                v[0] = x.x, v[1] = x.y, v[2 % PER] = x.z, v[3 % PER] = x.w;
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(o);
                v[0] = x.x, v[1] = x.y;
            }
#pragma unroll
            for (int y = 0; y < PER; ++y) acc[y] += w == 0.f ? 0.f : w * v[y];
        }
        const bool none = !(sum > 0.f) && sum == sum;   // no key seen anywhere
        const float inv = none ? 0.f : 1.f / sum;
        const int64_t fr = (int64_t)tile * tile_rows + r, tok = fr / A.G;
        const int64_t at = (a + tok) * A.Hq + head * A.G + (fr - tok * A.G);
        if (A.out_dtype == KDA_DTYPE_F32) {
#pragma unroll
            for (int y = 0; y < PER; ++y) static_cast<float *>(A.out)[at * D + lane * PER + y] = acc[y] * inv;
        } else {
#pragma unroll
            for (int y = 0; y < PER; y += 2)
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(A.out) + at * D + lane * PER + y) =
                    pack16<BF16>(acc[y] * inv, acc[y + 1] * inv);
        }
        if (lane == 0 && A.lse) A.lse[at] = none ? -INFINITY : top + logf(sum);
    }
}

// ---------------------------------------------------------------- few rows
// Sequences of at most kFewRows (token, query head) rows a key head, which is what a decode
// step has.  The keys are read once and each is used by 16 rows at most: HBM bounds it, and
// what matters is that loads never pause.  A block takes a run of keys of one head through a
// ring of 64-key stages; each of four warps takes 16 of them with the register products
// (m16n8k16; a tcgen05 product of 128 rows would be padding for the most part) and keeps
// its own maximum, sum and output, which are joined once at the end.
constexpr int kFewRows = 16, kFewKeys = 64, kFewThreads = 160;

template <int D>
struct FewLay {
    static constexpr int kTile = kFewKeys * D * 2;      // 64 keys, or their values
    static constexpr int kBlock = kFewKeys * 128;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kSmem = 1024 + kStages * 2 * kTile;
    static_assert(kStages * 2 * kTile >= 4 * 16 * D * 4, "the warps' outputs are joined in the ring");
};

struct FewControl {
    uint64_t full[6], empty[6];
    AttnPart part;
    int64_t scan[kFewThreads / 32];
    float m[4][16], l[4][16];
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kFewThreads)
kda_attn_few_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Attn A,
                    const Shares sh, const int box, const int slots_at_once) {
    using L = FewLay<D>;
    constexpr int NST = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ FewControl ct;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = A.G;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            sm100::mbar_init(&ct.full[i], 1);
            sm100::mbar_init(&ct.empty[i], 4);
        }
        sm100::fence_mbar_init();
    }
    auto need = [&](int n) {
        const AttnSeq s = attn_seq<true>(A, n);
        const int64_t rows = (s.b - s.a) * G;
        return AttnNeed{rows > 0 && rows <= kFewRows ? 1 : 0, (int32_t)((s.keys + kFewKeys - 1) / kFewKeys)};
    };
    int64_t slots;
    const bool some = attn_split_part<kFewThreads>(A.N, A.Hkv, blockIdx.x, slots_at_once, 8, 4, need, &ct.part, ct.scan,
                                                   &slots);
    if (blockIdx.x == 0 && tid == 0) *sh.count = (int32_t)slots;
    if (!some) return;
    const AttnPart part = ct.part;
    const AttnSeq sq = attn_seq<true>(A, part.n);
    const int32_t tokens = (int32_t)(sq.b - sq.a), rows = tokens * G;
    const int32_t behind = (int32_t)sq.keys - tokens, keys = (int32_t)sq.keys;
    const int n = part.j1 - part.j0;
    bool ok = true;
    if (warp == 4) {
        const int boxes = kFewKeys / box;
        const int unit = lane % (boxes * (D / 64)), mine = unit / boxes, which = unit % boxes;
        const bool values = lane >= boxes * (D / 64), issues = lane < 2 * boxes * (D / 64);
        const int32_t *row = A.table + (int64_t)part.n * A.wide;
        bool bad = false;
        int issued = 0;
        for (int j = 0; j < n; ++j) {
            const int64_t first = (int64_t)(part.j0 + j) * kFewKeys + which * box;
            int page = A.P;   // past the cache: reads zeros
            if (issues && first < keys) {
                const int p = row[first / A.page];
                if (p >= 0 && p < A.P) page = p; else bad = true;
            }
            const int st = j % NST;
            if (j >= NST) ok = attn_wait(&ct.empty[st], (j / NST - 1) & 1, &g_attn_status);
            if (!ok) break;
            uint8_t *to = ring + st * 2 * L::kTile + (values ? L::kTile : 0);
            if (lane == 0) sm100::mbar_arrive_expect_tx(&ct.full[st], 2 * L::kTile);
            __syncwarp();
            if (issues)
                tma_load_4d(to + mine * L::kBlock + which * box * 128, values ? &vmap : &kmap, &ct.full[st], mine * 64,
                            part.head, (int)(first % A.page), page);
            ++issued;
        }
        if (bad) atomicOr(&g_attn_status, kCacheBadPage);
        for (int j = max(0, issued - NST); j < issued; ++j) attn_wait(&ct.full[j % NST], (j / NST) & 1, &g_attn_status);
        __syncthreads();
        __syncthreads();
        return;
    }
    // the queries as the products' A operand: rows lane / 4 and + 8, two channels a register
    const int r0 = lane >> 2, r1 = r0 + 8;
    uint32_t qa[D / 16][4];
    {
        const uint16_t *q = static_cast<const uint16_t *>(A.q);
        const int t0 = r0 / G, t1 = r1 / G;
        const uint16_t *p0 = q + (sq.a + t0) * A.q_t + (int64_t)(part.head * G + r0 - t0 * G) * A.q_h + (lane & 3) * 2;
        const uint16_t *p1 = q + (sq.a + t1) * A.q_t + (int64_t)(part.head * G + r1 - t1 * G) * A.q_h + (lane & 3) * 2;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
            qa[s][0] = r0 < rows ? __ldg(reinterpret_cast<const uint32_t *>(p0 + s * 16)) : 0;
            qa[s][1] = r1 < rows ? __ldg(reinterpret_cast<const uint32_t *>(p1 + s * 16)) : 0;
            qa[s][2] = r0 < rows ? __ldg(reinterpret_cast<const uint32_t *>(p0 + s * 16 + 8)) : 0;
            qa[s][3] = r1 < rows ? __ldg(reinterpret_cast<const uint32_t *>(p1 + s * 16 + 8)) : 0;
        }
    }
    const int32_t seen0 = r0 < rows ? min(behind + r0 / G + 1, keys) : 0;
    const int32_t seen1 = r1 < rows ? min(behind + r1 / G + 1, keys) : 0;
    const float c = A.scale_log2;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
    // ldmatrix rows: keys 0..7 / 8..15 of the warp's 16, channel pieces 0 / 1
    const int krow = warp * 16 + (lane & 7) + ((lane >> 4) << 3), kpiece = (lane >> 3) & 1;
    const int vrow = warp * 16 + (lane & 15), vpiece = lane >> 4;
    for (int j = 0; j < n; ++j) {
        const int st = j % NST;
        ok = attn_wait(&ct.full[st], (j / NST) & 1, &g_attn_status);
        if (!ok) break;
        const uint32_t kb = sm100::smem_u32(ring + st * 2 * L::kTile), vb = kb + L::kTile;
        const int32_t first = (part.j0 + j) * kFewKeys + warp * 16;   // the warp's first key
        if (first + 16 > keys) {
            // value rows behind the last key hold anything; only this warp reads these
            uint8_t *v = ring + st * 2 * L::kTile + L::kTile;
            for (int x = lane; x < 16 * (D / 8); x += 32)
                if (first + x / (D / 8) >= keys)
                    *reinterpret_cast<uint4 *>(v + (x % (D / 8)) / 8 * L::kBlock + (warp * 16 + x / (D / 8)) * 128 +
                                               (x % 8) * 16) = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        float s[2][4] = {};
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            uint32_t b[4];
            const int piece = x * 2 + kpiece;
            ldsm4(b, kb + (piece >> 3) * L::kBlock + krow * 128 + (((piece & 7) ^ (krow & 7)) << 4));
            mma16816<BF16>(s[0], qa[x], b[0], b[1]);
            mma16816<BF16>(s[1], qa[x], b[2], b[3]);
        }
        const int32_t k0 = first + (lane & 3) * 2;
        if (first + 16 > behind + 1) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int32_t key = k0 + t * 8 + e;
                    if (key >= seen0) s[t][e] = -INFINITY;
                    if (key >= seen1) s[t][2 + e] = -INFINITY;
                }
        }
        float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
        }
        const bool g0 = t0 > m0 && (t0 - m0) * c > kGrowth, g1 = t1 > m1 && (t1 - m1) * c > kGrowth;
        if (__any_sync(0xffffffffu, g0 || g1)) {
            const float f0 = g0 ? ex2((m0 - t0) * c) : 1.f, f1 = g1 ? ex2((m1 - t1) * c) : 1.f;
            l0 *= f0;
            l1 *= f1;
            if (g0) m0 = t0;
            if (g1) m1 = t1;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) o[x][0] *= f0, o[x][1] *= f0, o[x][2] *= f1, o[x][3] *= f1;
        }
        const float h0 = m0 == -INFINITY ? 0.f : -m0 * c, h1 = m1 == -INFINITY ? 0.f : -m1 * c;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t][0] = ex2(fmaf(s[t][0], c, h0));
            s[t][1] = ex2(fmaf(s[t][1], c, h0));
            s[t][2] = ex2(fmaf(s[t][2], c, h1));
            s[t][3] = ex2(fmaf(s[t][3], c, h1));
        }
        l0 += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
        l1 += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
        const uint32_t pa[4] = {pack16<BF16>(s[0][0], s[0][1]), pack16<BF16>(s[0][2], s[0][3]),
                                pack16<BF16>(s[1][0], s[1][1]), pack16<BF16>(s[1][2], s[1][3])};
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            uint32_t b[4];
            const int piece = x * 2 + vpiece;
            ldsm4_t(b, vb + (piece >> 3) * L::kBlock + vrow * 128 + (((piece & 7) ^ (vrow & 7)) << 4));
            mma16816<BF16>(o[2 * x], pa, b[0], b[1]);
            mma16816<BF16>(o[2 * x + 1], pa, b[2], b[3]);
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&ct.empty[st]);
    }
    // join the four warps' shares
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, x);
        l1 += __shfl_xor_sync(0xffffffffu, l1, x);
    }
    __syncthreads();   // every stage has been read
    float *all = reinterpret_cast<float *>(ring);   // [4][16][D]
    if ((lane & 3) == 0) {
        ct.m[warp][r0] = m0;
        ct.m[warp][r1] = m1;
        ct.l[warp][r0] = l0;
        ct.l[warp][r1] = l1;
    }
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
        const int ch = x * 8 + (lane & 3) * 2;
        *reinterpret_cast<float2 *>(all + (warp * 16 + r0) * D + ch) = make_float2(o[x][0], o[x][1]);
        *reinterpret_cast<float2 *>(all + (warp * 16 + r1) * D + ch) = make_float2(o[x][2], o[x][3]);
    }
    __syncthreads();
    if (!ok) return;
    for (int x = tid; x < rows * (D / 8); x += 128) {
        const int r = x / (D / 8), ch = x % (D / 8) * 8;
        float top = fmaxf(fmaxf(ct.m[0][r], ct.m[1][r]), fmaxf(ct.m[2][r], ct.m[3][r]));
        const float ref = top == -INFINITY ? 0.f : top;
        float w[4], l = 0.f;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            w[y] = ex2((ct.m[y][r] - ref) * c);
            l += ct.l[y][r] * w[y];
        }
        const bool none = !(l > 0.f) && l == l;
        const float inv = none ? 0.f : 1.f / l;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float sum = 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) sum += w[y] * all[(y * 16 + r) * D + ch + e];
            v[e] = none ? 0.f : sum * inv;
        }
        const float lse = none ? -INFINITY : top * A.scale + logf(l);
        if (part.slot >= 0) {
            store8<BF16>(sh.out, true, ((int64_t)part.slot * kFewRows + r) * D + ch, v);
            if (ch == 0) sh.lse[(int64_t)part.slot * kFewRows + r] = lse;
        } else {
            const int tok = r / G;
            const int64_t at = (sq.a + tok) * A.Hq + part.head * G + (r - tok * G);
            store8<BF16>(A.out, A.out_dtype == KDA_DTYPE_F32, at * D + ch, v);
            if (ch == 0 && A.lse) A.lse[at] = lse;
        }
    }
    if (part.slot >= 0 && tid == 0) {
        int32_t *rec = sh.rec + (int64_t)part.slot * 8;
        rec[0] = part.n;
        rec[1] = 0;
        rec[2] = part.head;
        rec[3] = part.split;
        rec[4] = part.splits;
    }
}

// ---------------------------------------------------------------- host
// Sizes of a paged call's launches.  Which sequences have few rows is known on the device
// only (unless all are alike): each kernel passes by those that are the other's.
struct Sizes {
    bool many, few;               // launch the kernel of many rows, of few rows
    int64_t tiles, few_tiles;     // upper bounds on row tiles times heads
    int64_t parts, few_parts;     // blocks
    int64_t slots, few_slots;     // shares
};
constexpr int kFewAtOnce = 304;   // two blocks an SM

int64_t shares_bound(int64_t tiles, int at_once, int waves) {
    // a row tile that is cut has more than one run of keys: at most two parts a run
    const int64_t parts = attn_parts(tiles, at_once, waves);
    return parts < 2 * (int64_t)at_once * waves ? parts : 2 * (int64_t)at_once * waves;
}

Sizes sizes_of(const Attn &A) {
    Sizes z{};
    if (A.N == 0 || A.T == 0) return z;
    const int64_t rows = (int64_t)A.T * A.G;
    if (A.cu) {
        z.few = true;
        z.many = rows > kFewRows;
        z.tiles = rows / kTileRows + A.N;
        z.few_tiles = A.N;
    } else {
        z.few = A.seq_len * A.G <= kFewRows;
        z.many = !z.few;
        z.tiles = (A.seq_len * A.G + kTileRows - 1) / kTileRows * A.N;
        z.few_tiles = A.N;
    }
    z.tiles *= A.Hkv;
    z.few_tiles *= A.Hkv;
    if (z.many) {
        // the device knows the real number of row tiles: few of them, and it cuts for one
        // wave; more, for three
        z.parts = z.tiles * 2 <= 152 ? 152 : z.tiles + 3 * 152;
        z.slots = shares_bound(z.tiles, 152, 3);
    }
    if (z.few) {
        z.few_parts = attn_parts(z.few_tiles, kFewAtOnce, 8);
        z.few_slots = shares_bound(z.few_tiles, kFewAtOnce, 8);
    }
    return z;
}

int64_t up(int64_t x) { return (x + 255) / 256 * 256; }
int64_t shares_bytes(int64_t slots, int rows, int d) { return 256 + up(slots * 32) + up(slots * rows * 4) + slots * rows * d * 4; }

Shares shares_at(char *ws, int64_t slots, int rows) {
    Shares s;
    s.count = reinterpret_cast<int32_t *>(ws);
    s.rec = reinterpret_cast<int32_t *>(ws + 256);
    s.lse = reinterpret_cast<float *>(ws + 256 + up(slots * 32));
    s.out = reinterpret_cast<float *>(ws + 256 + up(slots * 32) + up(slots * rows * 4));
    return s;
}

template <typename Kernel>
cudaError_t roomy(Kernel kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <typename... Params, typename... Args>
cudaError_t launch(bool behind, void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                   const Args &...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cfg.attrs = behind ? &attr : nullptr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, bool BF16>
cudaError_t prefill(const Attn &A, cudaStream_t stream) {
    CUtensorMap km, vm;
    if (!kda_make_attn_map(&km, A.k, BF16, D, A.Hkv, A.T, 1, A.k_h, A.k_t, 0, kAttnKeys) ||
        !kda_make_attn_map(&vm, A.v, BF16, D, A.Hkv, A.T, 1, A.v_h, A.v_t, 0, kAttnKeys))
        return cudaErrorInvalidValue;
    const auto kernel = kda_attn_tc_kernel<D, BF16, false>;
    cudaError_t e = roomy(kernel, Lay<D>::kSmem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = A.cu ? (int64_t)A.T * A.G / kTileRows + A.N
                               : (A.seq_len * A.G + kTileRows - 1) / kTileRows * A.N;
    return launch(false, kernel, dim3((unsigned)(tiles * A.Hkv)), kThreads, Lay<D>::kSmem, stream, km, vm, A, Shares{},
                  kAttnKeys, 0);
}

template <int D, bool BF16>
cudaError_t paged(const Attn &A, char *ws, cudaStream_t stream) {
    const Sizes z = sizes_of(A);
    cudaError_t e = cudaSuccess;
    if (z.few) {
        const int box = A.page < kFewKeys ? A.page : kFewKeys;
        CUtensorMap km, vm;
        if (!kda_make_attn_map(&km, A.k, BF16, D, A.Hkv, A.page, A.P, A.k_h, A.k_t, A.k_p, box) ||
            !kda_make_attn_map(&vm, A.v, BF16, D, A.Hkv, A.page, A.P, A.v_h, A.v_t, A.v_p, box))
            return cudaErrorInvalidValue;
        const Shares sh = shares_at(ws, z.few_slots, kFewRows);
        const auto kernel = kda_attn_few_kernel<D, BF16>;
        e = roomy(kernel, FewLay<D>::kSmem);
        if (e == cudaSuccess)
            e = launch(false, kernel, dim3((unsigned)z.few_parts), kFewThreads, FewLay<D>::kSmem, stream, km, vm, A, sh,
                       box, kFewAtOnce);
        if (e == cudaSuccess)
            e = launch(true, kda_attn_join_kernel<D, BF16>, dim3((unsigned)z.few_slots, 4), 128, 0, stream, A, sh,
                       kFewRows);
        ws += up(shares_bytes(z.few_slots, kFewRows, D));
    }
    if (z.many && e == cudaSuccess) {
        const int box = A.page < kAttnKeys ? A.page : kAttnKeys;
        CUtensorMap km, vm;
        if (!kda_make_attn_map(&km, A.k, BF16, D, A.Hkv, A.page, A.P, A.k_h, A.k_t, A.k_p, box) ||
            !kda_make_attn_map(&vm, A.v, BF16, D, A.Hkv, A.page, A.P, A.v_h, A.v_t, A.v_p, box))
            return cudaErrorInvalidValue;
        const Shares sh = shares_at(ws, z.slots, kTileRows);
        const auto kernel = kda_attn_tc_kernel<D, BF16, true>;
        e = roomy(kernel, Lay<D>::kSmem);
        if (e == cudaSuccess)
            e = launch(false, kernel, dim3((unsigned)z.parts), kThreads, Lay<D>::kSmem, stream, km, vm, A, sh, box,
                       z.few ? kFewRows : 0);
        if (e == cudaSuccess)
            e = launch(true, kda_attn_join_kernel<D, BF16>, dim3((unsigned)z.slots, 16), 128, 0, stream, A, sh,
                       kTileRows);
    }
    return e;
}

}  // namespace

int64_t kda_attn_paged_ws(const Attn &A) {
    const Sizes z = sizes_of(A);
    return (z.few ? up(shares_bytes(z.few_slots, kFewRows, A.d)) : 0) +
           (z.many ? up(shares_bytes(z.slots, kTileRows, A.d)) : 0);
}

cudaError_t kda_launch_attn_prefill(const Attn &A, cudaStream_t stream) {
    const bool b = A.in_dtype == KDA_DTYPE_BF16;
    if (A.d == 128) return b ? prefill<128, true>(A, stream) : prefill<128, false>(A, stream);
    return b ? prefill<64, true>(A, stream) : prefill<64, false>(A, stream);
}

cudaError_t kda_launch_attn_paged(const Attn &A, void *workspace, cudaStream_t stream) {
    const bool b = A.in_dtype == KDA_DTYPE_BF16;
    char *ws = static_cast<char *>(workspace);
    if (A.d == 128) return b ? paged<128, true>(A, ws, stream) : paged<128, false>(A, ws, stream);
    return b ? paged<64, true>(A, ws, stream) : paged<64, false>(A, ws, stream);
}

cudaError_t kda_attn_read_status(unsigned *status) {
    unsigned w = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&w, g_attn_status, sizeof(w));
    if (e == cudaSuccess && w) {
        *status |= w;
        w = 0;
        e = cudaMemcpyToSymbol(g_attn_status, &w, sizeof(w));
    }
    return e;
}
